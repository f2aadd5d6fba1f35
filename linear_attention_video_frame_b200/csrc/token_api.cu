// Entry points of the token-wise operators: argument checks and dispatch.
#include <cmath>

#include "token.cuh"

namespace la {
namespace {

bool head_dim_ok(int D) { return D >= 16 && D <= 256 && D % 16 == 0; }
bool norm_width_ok(int N) { return N >= 16 && N <= 16384 && N % 16 == 0; }

size_t elem_size(int dt) { return dt == LA_BF16 ? 2 : 4; }

// Bytes from the first to behind the last element of [B, H, T, D] rows.
size_t span_bytes(const long long s[3], int B, int H, int T, int D, int dt) {
    if (T == 0) return 0;
    const long long last = (B - 1) * s[0] + (H - 1) * s[1] + (T - 1) * s[2] + D;
    return (size_t)last * elem_size(dt);
}

// Strides of rows that are read: whole 16-byte pieces, not negative, and a
// span that 63 bits hold.
bool strides_ok(const long long s[3], int B, int H, int T, int dt) {
    const long long unit = 16 / (long long)elem_size(dt);
    const int n[3] = {B, H, T};
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] % unit != 0 || (double)s[i] * n[i] > 2.0e18) return false;
    return true;
}

// Rows that are written must not share elements: taken from the smallest
// stride up, each stride steps over all of what the smaller ones span.
bool rows_disjoint(const long long s[3], int B, int H, int T, int D) {
    long long stride[3] = {s[0], s[1], s[2]};
    int n[3] = {B, H, T};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[j] < stride[i]) {
                const long long t = stride[i]; stride[i] = stride[j]; stride[j] = t;
                const int m = n[i]; n[i] = n[j]; n[j] = m;
            }
    long long extent = D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (stride[i] < extent) return false;
        extent = (n[i] - 1) * stride[i] + extent;
    }
    return true;
}

la_status check_delta(const la_delta* in) {
    if (!in) return LA_ERR_INVALID_ARG;
    if (in->dt != LA_F32 && in->dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if (in->B < 1 || in->Hk < 1 || in->Hv < 1 || in->T < 0) return LA_ERR_INVALID_ARG;
    if (in->B > 65535 || in->Hv > 65535 || in->Hv % in->Hk != 0) return LA_ERR_INVALID_ARG;
    // chunks are counted in 32 bits over all heads
    if ((double)in->B * in->Hv * (in->T / kChunk + 2.0) > 2.0e9) return LA_ERR_INVALID_ARG;
    if (!head_dim_ok(in->D)) return LA_ERR_UNSUPPORTED;
    if (!std::isfinite(in->k_scale) || !std::isfinite(in->q_scale)) return LA_ERR_INVALID_ARG;
    if (in->T > 0) {
        if (!in->q || !in->k || !in->v || !in->log_alpha || !in->beta) return LA_ERR_INVALID_ARG;
        if (!strides_ok(in->q_stride, in->B, in->Hk, in->T, in->dt) ||
            !strides_ok(in->k_stride, in->B, in->Hk, in->T, in->dt) ||
            !strides_ok(in->v_stride, in->B, in->Hv, in->T, in->dt))
            return LA_ERR_INVALID_ARG;
    }
    return LA_OK;
}

// `lengths` needs the alignment of its own type only.
la_status check_lengths(const int* p, int dev) {
    if (!p) return LA_OK;
    if (reinterpret_cast<uintptr_t>(p) & 3u) return LA_ERR_INVALID_ARG;
    return check_ptr(reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15)),
                     dev);
}

struct Region { const void* p; size_t n; };

// Device, pointers, and no output on top of an input or another output.
// `same` names the one input that output 0 may equal exactly.
la_status check_regions(const la_delta& in, const Region* ins, int n_in, const Region* outs,
                        int n_out, const void* same) {
    int dev = 0;
    la_status s = check_device(&dev);
    if (s != LA_OK) return s;
    for (int i = 0; i < n_in; ++i)
        if ((s = check_ptr(ins[i].p, dev)) != LA_OK) return s;
    for (int i = 0; i < n_out; ++i)
        if ((s = check_ptr(outs[i].p, dev)) != LA_OK) return s;
    if ((s = check_lengths(in.lengths, dev)) != LA_OK) return s;
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (!(o == 0 && outs[0].p && outs[0].p == same && ins[i].p == same) &&
                overlaps(outs[o].p, outs[o].n, ins[i].p, ins[i].n))
                return LA_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (overlaps(outs[o].p, outs[o].n, outs[i].p, outs[i].n)) return LA_ERR_INVALID_ARG;
    }
    return LA_OK;
}

la_status forward(const la_delta* in, void* o, const long long os[3], float* state_out, void* ws,
                  size_t ws_bytes, bool step, cudaStream_t st) {
    la_status s = check_delta(in);
    if (s != LA_OK) return s;
    const la_delta& a = *in;
    if (step && (a.T != 1 || !state_out)) return LA_ERR_INVALID_ARG;
    long long rs[3] = {0, 0, 0};
    if (a.T > 0) {
        if (!o || !os) return LA_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i) rs[i] = os[i];
        if (!strides_ok(rs, a.B, a.Hv, a.T, a.dt) || !rows_disjoint(rs, a.B, a.Hv, a.T, a.D))
            return LA_ERR_INVALID_ARG;
    }
    const size_t need = step ? 0 : delta_workspace_bytes(0, a.dt, a.B, a.Hk, a.Hv, a.T, a.D);
    if (!step && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < need))
        return LA_ERR_INVALID_ARG;
    const size_t gates = (size_t)a.B * a.Hv * a.T * 4, states = (size_t)a.B * a.Hv * a.D * a.D * 4;
    const Region ins[] = {{a.T ? a.q : nullptr, span_bytes(a.q_stride, a.B, a.Hk, a.T, a.D, a.dt)},
                          {a.T ? a.k : nullptr, span_bytes(a.k_stride, a.B, a.Hk, a.T, a.D, a.dt)},
                          {a.T ? a.v : nullptr, span_bytes(a.v_stride, a.B, a.Hv, a.T, a.D, a.dt)},
                          {a.T ? a.log_alpha : nullptr, gates},
                          {a.T ? a.beta : nullptr, gates},
                          {a.state_in, states}};
    const Region outs[] = {{state_out, states},
                           {a.T ? o : nullptr, span_bytes(rs, a.B, a.Hv, a.T, a.D, a.dt)},
                           {step ? nullptr : ws, need}};
    if ((s = check_regions(a, ins, 6, outs, 3, a.state_in)) != LA_OK) return s;
    if (a.lengths)
        for (const Region& r : outs)
            if (overlaps(r.p, r.n, a.lengths, (size_t)a.B * 4)) return LA_ERR_INVALID_ARG;
    const cudaError_t e = !step && delta_chunked(0, a.dt, a.B * a.Hv, a.T, a.D)
                              ? launch_delta_chunked(a, o, rs, state_out, ws, st)
                              : launch_delta_recurrent(a, o, rs, state_out,
                                                       static_cast<unsigned int*>(ws), st);
    if (e != cudaSuccess) { cudaGetLastError(); return LA_ERR_CUDA; }
    return LA_OK;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" la_status la_gated_delta_rule(const la_delta* in, void* o, const long long o_stride[3],
                                         float* state_out, void* workspace,
                                         size_t workspace_bytes, cudaStream_t stream) {
    return forward(in, o, o_stride, state_out, workspace, workspace_bytes, false, stream);
}

extern "C" la_status la_gated_delta_step(const la_delta* in, void* o, const long long o_stride[3],
                                         float* state_out, cudaStream_t stream) {
    return forward(in, o, o_stride, state_out, nullptr, 0, true, stream);
}

extern "C" size_t la_delta_workspace_size(int backward, la_dtype dt, int B, int Hk, int Hv, int T,
                                          int D) {
    if ((dt != LA_F32 && dt != LA_BF16) || B < 1 || Hk < 1 || Hv < 1 || T < 0 || Hv % Hk != 0 ||
        B > 65535 || Hv > 65535 || !head_dim_ok(D) || (backward && D > 128) ||
        (double)B * Hv * (T / kChunk + 2.0) > 2.0e9)
        return 0;
    return delta_workspace_bytes(backward, dt, B, Hk, Hv, T, D);
}

extern "C" const char* la_delta_plan(int backward, la_dtype dt, int B, int Hk, int Hv, int T,
                                     int D, int* kernels) {
    if (la_delta_workspace_size(backward, dt, B, Hk, Hv, T, D) == 0) return nullptr;
    const bool chunked = delta_chunked(backward, dt, B * Hv, T, D);
    if (kernels) *kernels = chunked ? delta_kernel_count(backward, dt, B, Hk, Hv, T) : 1;
    return chunked ? "delta_chunked" : "delta_recurrent";
}

extern "C" la_status la_add_rms_norm_fp8(const void* x, const void* residual, const float* weight,
                                         void* h, void* y8, float* scale, la_dtype dt,
                                         long long rows, int N, int group, float eps,
                                         cudaStream_t stream) {
    if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if (rows < 0 || rows > 0x7fffffffLL || (group != 0 && group != 128)) return LA_ERR_INVALID_ARG;
    if (!norm_width_ok(N)) return LA_ERR_UNSUPPORTED;
    if (!(std::isfinite(eps) && eps >= 0.f)) return LA_ERR_INVALID_ARG;
    if (rows == 0) return LA_OK;
    if (!x || !weight || !y8 || !scale) return LA_ERR_INVALID_ARG;
    int dev = 0;
    la_status s = check_device(&dev);
    if (s != LA_OK) return s;
    const size_t full = (size_t)rows * N * elem_size(dt);
    const size_t scales = (size_t)rows * (group ? (N + group - 1) / group : 1) * 4;
    const Region ins[] = {{x, full}, {residual, full}, {weight, (size_t)N * 4}};
    const Region outs[] = {{h, full}, {y8, (size_t)rows * N}, {scale, scales}};
    for (const Region& r : ins)
        if ((s = check_ptr(r.p, dev)) != LA_OK) return s;
    for (int o = 0; o < 3; ++o) {
        if ((s = check_ptr(outs[o].p, dev)) != LA_OK) return s;
        for (int i = 0; i < 3; ++i)
            if (!(o == 0 && i < 2 && h == ins[i].p) &&
                overlaps(outs[o].p, outs[o].n, ins[i].p, ins[i].n))
                return LA_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (overlaps(outs[o].p, outs[o].n, outs[i].p, outs[i].n)) return LA_ERR_INVALID_ARG;
    }
    if (launch_norm_fp8(x, residual, weight, h, y8, scale, dt == LA_BF16, rows, N, group, eps,
                        stream) != cudaSuccess) {
        cudaGetLastError();
        return LA_ERR_CUDA;
    }
    return LA_OK;
}

extern "C" size_t la_norm_workspace_size(long long rows, int N) {
    if (rows < 0 || rows > 0x7fffffffLL || !norm_width_ok(N)) return 0;
    return align_up((size_t)norm_backward_blocks(rows, N) * N * 4 + 256, 256);
}

extern "C" la_status la_add_rms_norm_backward(const void* dy, const void* h, const float* weight,
                                              const void* dh, void* dx, float* dweight,
                                              la_dtype dt, long long rows, int N, float eps,
                                              void* workspace, size_t workspace_bytes,
                                              cudaStream_t stream) {
    if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if (rows < 0 || rows > 0x7fffffffLL) return LA_ERR_INVALID_ARG;
    if (!norm_width_ok(N)) return LA_ERR_UNSUPPORTED;
    if (!(std::isfinite(eps) && eps >= 0.f)) return LA_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !h || !weight || !dx)) return LA_ERR_INVALID_ARG;
    const size_t need = dweight ? la_norm_workspace_size(rows, N) : 0;
    if (dweight && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                    workspace_bytes < need))
        return LA_ERR_INVALID_ARG;
    int dev = 0;
    la_status s = check_device(&dev);
    if (s != LA_OK) return s;
    const size_t full = (size_t)rows * N * elem_size(dt);
    const Region ins[] = {{dy, full}, {dh, full}, {h, full}, {weight, (size_t)N * 4}};
    const Region outs[] = {{dx, full}, {dweight, (size_t)N * 4},
                           {dweight ? workspace : nullptr, need}};
    for (const Region& r : ins)
        if ((s = check_ptr(r.p, dev)) != LA_OK) return s;
    for (int o = 0; o < 3; ++o) {
        if ((s = check_ptr(outs[o].p, dev)) != LA_OK) return s;
        for (int i = 0; i < 4; ++i)
            if (!(o == 0 && i < 2 && dx == ins[i].p) &&
                overlaps(outs[o].p, outs[o].n, ins[i].p, ins[i].n))
                return LA_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (overlaps(outs[o].p, outs[o].n, outs[i].p, outs[i].n)) return LA_ERR_INVALID_ARG;
    }
    if (launch_norm_backward(dy, h, weight, dh, dx, dweight, static_cast<float*>(workspace),
                             dt == LA_BF16, rows, N, eps, stream) != cudaSuccess) {
        cudaGetLastError();
        return LA_ERR_CUDA;
    }
    return LA_OK;
}

extern "C" la_status la_gated_delta_rule_backward(const la_delta* in, const void* d_o,
                                                  const long long do_stride[3],
                                                  const float* dstate_out, void* dq, void* dk,
                                                  void* dv, float* dlog_alpha, float* dbeta,
                                                  float* dstate_in, void* workspace,
                                                  size_t workspace_bytes, cudaStream_t stream) {
    la_status s = check_delta(in);
    if (s != LA_OK) return s;
    const la_delta& a = *in;
    if (a.D > 128) return LA_ERR_UNSUPPORTED;
    DeltaGrad g{d_o, {0, 0, 0}, dstate_out, dq, dk, dv, dlog_alpha, dbeta, dstate_in};
    if (a.T > 0) {
        if (!d_o || !do_stride || !dq || !dk || !dv || !dlog_alpha || !dbeta)
            return LA_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i) g.do_stride[i] = do_stride[i];
        if (!strides_ok(g.do_stride, a.B, a.Hv, a.T, a.dt)) return LA_ERR_INVALID_ARG;
    }
    const size_t need = delta_workspace_bytes(1, a.dt, a.B, a.Hk, a.Hv, a.T, a.D);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need)
        return LA_ERR_INVALID_ARG;
    const size_t gates = (size_t)a.B * a.Hv * a.T * 4, states = (size_t)a.B * a.Hv * a.D * a.D * 4;
    const size_t row = (size_t)a.B * a.T * a.D * elem_size(a.dt);
    auto if_t = [&](const void* p) { return a.T ? p : nullptr; };
    const Region ins[] = {{if_t(a.q), span_bytes(a.q_stride, a.B, a.Hk, a.T, a.D, a.dt)},
                          {if_t(a.k), span_bytes(a.k_stride, a.B, a.Hk, a.T, a.D, a.dt)},
                          {if_t(a.v), span_bytes(a.v_stride, a.B, a.Hv, a.T, a.D, a.dt)},
                          {if_t(a.log_alpha), gates},
                          {if_t(a.beta), gates},
                          {a.state_in, states},
                          {if_t(d_o), span_bytes(g.do_stride, a.B, a.Hv, a.T, a.D, a.dt)},
                          {dstate_out, states}};
    const Region outs[] = {{dstate_in, states}, {if_t(dq), row * a.Hk}, {if_t(dk), row * a.Hk},
                           {if_t(dv), row * a.Hv}, {if_t(dlog_alpha), gates},
                           {if_t(dbeta), gates}, {workspace, need}};
    if ((s = check_regions(a, ins, 8, outs, 7, dstate_out)) != LA_OK) return s;
    if (a.lengths)
        for (const Region& r : outs)
            if (overlaps(r.p, r.n, a.lengths, (size_t)a.B * 4)) return LA_ERR_INVALID_ARG;
    if (launch_delta_backward(a, g, workspace, stream) != cudaSuccess) {
        cudaGetLastError();
        return LA_ERR_CUDA;
    }
    return LA_OK;
}
