// Gated delta rule, token by token in float32: decoding (one token), calls too
// short for a chunk, and heads wider than 128.
//
// A block owns 32 columns of one head's state (the columns of S evolve
// independently: column c needs only k, q, the gates and v[c]) and keeps them
// in registers.  Per token, with m = kh S and p = qh S over the rows:
//     u = beta (v - alpha m),  S <- alpha S + kh u,  o = alpha p + (qh . kh) u,
// so the state is read once, both products share that read, and the output
// needs no second pass over the updated state.
//
// One token is bound by the state's traffic (8 D^2 bytes a head).  A block of 128
// threads holds 16 KB of a 128-row state: 8 threads side by side take one 128-byte
// row piece, so every access is a full line, each thread has its eight 16-byte loads
// in flight at once, and few warps wait for one another at a block's two barriers.
// 192 x 32 heads of 128: 125 to 130 us, 6.2 TB/s and more (256 threads of four loads:
// 157).  Eight blocks an SM leave a thread 64 registers; with six of 80, heads of 112
// and 256 take a tenth longer.
#include <cuda_bf16.h>

#include "token.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 32;                       // state columns of a block
constexpr int kRowGroups = kThreads / (kCols / 4);   // 32 threads down a column

template <typename T>
__device__ __forceinline__ float ld(const T* p) { return (float)*p; }
template <>
__device__ __forceinline__ float ld<__nv_bfloat16>(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
}
__device__ __forceinline__ void st_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void st_out(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// ROWS: state rows of a thread (rows rg, rg + 32, ...).
template <typename T, int ROWS>
__global__ void __launch_bounds__(kThreads)
delta_recurrent_kernel(la_delta in, T* o, Row3 os, float* state_out, unsigned int* status) {
    if (status && blockIdx.x + blockIdx.y + blockIdx.z == 0 && threadIdx.x < 2) status[threadIdx.x] = 0;
    // Per warp: partial k.S and q.S of the block's columns, and q.k; two
    // buffers so that one barrier a token is enough.
    __shared__ float4 part[2][kThreads / 32][kCols / 4][2];
    __shared__ float dots[2][kThreads / 32];

    const int h = blockIdx.y, b = blockIdx.z;
    const int hk = h / (in.Hv / in.Hk);
    const int D = in.D;
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * kCols + cg * 4;
    const bool live = col < D;
    const int n = seq_len(in.lengths, b, in.T);

    const size_t head = (size_t)b * in.Hv + h;
    const float* s_in = in.state_in ? in.state_in + head * D * D : nullptr;
    float4 S[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = rg + i * kRowGroups;
        S[i] = (s_in && live && r < D)
                   ? *reinterpret_cast<const float4*>(s_in + (size_t)r * D + col)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }

    const T* q = static_cast<const T*>(in.q) + row3(in.q_stride).at(b, hk, 0);
    const T* k = static_cast<const T*>(in.k) + row3(in.k_stride).at(b, hk, 0);
    const T* v = static_cast<const T*>(in.v) + row3(in.v_stride).at(b, h, 0);
    const float* la_p = in.log_alpha + head * in.T;
    const float* be_p = in.beta + head * in.T;

    for (int t = 0; t < n; ++t) {
        float kr[ROWS], qr[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = rg + i * kRowGroups;
            kr[i] = r < D ? ld(k + t * in.k_stride[2] + r) * in.k_scale : 0.f;
            qr[i] = r < D ? ld(q + t * in.q_stride[2] + r) * in.q_scale : 0.f;
        }
        float vv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) vv[j] = live ? ld(v + t * in.v_stride[2] + col + j) : 0.f;
        const float alpha = expf(la_p[t]), beta = be_p[t];

        float4 m = make_float4(0.f, 0.f, 0.f, 0.f), p = m;
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            m.x += kr[i] * S[i].x; m.y += kr[i] * S[i].y;
            m.z += kr[i] * S[i].z; m.w += kr[i] * S[i].w;
            p.x += qr[i] * S[i].x; p.y += qr[i] * S[i].y;
            p.z += qr[i] * S[i].z; p.w += qr[i] * S[i].w;
            qk += qr[i] * kr[i];
        }
        // the four rows of a warp that share a column group
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) {
            m.x += __shfl_xor_sync(~0u, m.x, d); m.y += __shfl_xor_sync(~0u, m.y, d);
            m.z += __shfl_xor_sync(~0u, m.z, d); m.w += __shfl_xor_sync(~0u, m.w, d);
            p.x += __shfl_xor_sync(~0u, p.x, d); p.y += __shfl_xor_sync(~0u, p.y, d);
            p.z += __shfl_xor_sync(~0u, p.z, d); p.w += __shfl_xor_sync(~0u, p.w, d);
            qk += __shfl_xor_sync(~0u, qk, d);
        }
        const int buf = t & 1;
        if (lane < 8) {
            part[buf][warp][cg][0] = m;
            part[buf][warp][cg][1] = p;
            if (lane == 0) dots[buf][warp] = qk;
        }
        __syncthreads();
        m = p = make_float4(0.f, 0.f, 0.f, 0.f);
        qk = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const float4 a = part[buf][w][cg][0], c = part[buf][w][cg][1];
            m.x += a.x; m.y += a.y; m.z += a.z; m.w += a.w;
            p.x += c.x; p.y += c.y; p.z += c.z; p.w += c.w;
            qk += dots[buf][w];
        }
        const float4 u = make_float4(beta * (vv[0] - alpha * m.x), beta * (vv[1] - alpha * m.y),
                                     beta * (vv[2] - alpha * m.z), beta * (vv[3] - alpha * m.w));
        if (rg == 0 && live) {
            T* out = o + os.at(b, h, t) + col;
            st_out(out, alpha * p.x + qk * u.x);
            st_out(out + 1, alpha * p.y + qk * u.y);
            st_out(out + 2, alpha * p.z + qk * u.z);
            st_out(out + 3, alpha * p.w + qk * u.w);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            S[i].x = alpha * S[i].x + kr[i] * u.x; S[i].y = alpha * S[i].y + kr[i] * u.y;
            S[i].z = alpha * S[i].z + kr[i] * u.z; S[i].w = alpha * S[i].w + kr[i] * u.w;
        }
    }
    if (!state_out || (n == 0 && state_out == in.state_in)) return;
    float* s_out = state_out + head * D * D;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = rg + i * kRowGroups;
        if (live && r < D) *reinterpret_cast<float4*>(s_out + (size_t)r * D + col) = S[i];
    }
}

// One token.  All of a block's state is asked for before anything else; k and q
// come through shared memory, so that a thread holds little beside its state.
template <typename T, int THREADS, int COLS, int ROWS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
delta_step_kernel(la_delta in, T* o, Row3 os, float* state_out, unsigned int* status) {
    if (status && blockIdx.x + blockIdx.y + blockIdx.z == 0 && threadIdx.x < 2) status[threadIdx.x] = 0;
    constexpr int CG = COLS / 4, RG = THREADS / CG;      // threads side by side, below
    __shared__ float4 part[THREADS / 32][CG][2];
    __shared__ float dots[THREADS / 32];
    __shared__ float2 kq[ROWS * RG];

    const int h = blockIdx.y, b = blockIdx.z;
    const int hk = h / (in.Hv / in.Hk);
    const int D = in.D;
    const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * COLS + cg * 4;
    const bool live = col < D;
    const size_t head = (size_t)b * in.Hv + h;
    const bool on = seq_len(in.lengths, b, 1) > 0;
    if (!on && (!state_out || state_out == in.state_in)) return;

    const float* s_in = in.state_in ? in.state_in + head * D * D : nullptr;
    float4 S[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = rg + i * RG;
        S[i] = (s_in && live && r < D)
                   ? __ldcs(reinterpret_cast<const float4*>(s_in + (size_t)r * D + col))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (on) {
        const T* q = static_cast<const T*>(in.q) + row3(in.q_stride).at(b, hk, 0);
        const T* k = static_cast<const T*>(in.k) + row3(in.k_stride).at(b, hk, 0);
        const T* v = static_cast<const T*>(in.v) + row3(in.v_stride).at(b, h, 0);
        const float alpha = expf(in.log_alpha[head]), beta = in.beta[head];
        if (threadIdx.x < ROWS * RG)
            kq[threadIdx.x] = threadIdx.x < D ? make_float2(ld(k + threadIdx.x) * in.k_scale,
                                                            ld(q + threadIdx.x) * in.q_scale)
                                              : make_float2(0.f, 0.f);
        float vv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) vv[j] = live ? ld(v + col + j) : 0.f;
        __syncthreads();
        float4 m = make_float4(0.f, 0.f, 0.f, 0.f), p = m;
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float2 f = kq[rg + i * RG];
            m.x += f.x * S[i].x; m.y += f.x * S[i].y;
            m.z += f.x * S[i].z; m.w += f.x * S[i].w;
            p.x += f.y * S[i].x; p.y += f.y * S[i].y;
            p.z += f.y * S[i].z; p.w += f.y * S[i].w;
            qk += f.x * f.y;
        }
        // the rows of a warp that share a column group
#pragma unroll
        for (int d = CG; d < 32; d <<= 1) {
            m.x += __shfl_xor_sync(~0u, m.x, d); m.y += __shfl_xor_sync(~0u, m.y, d);
            m.z += __shfl_xor_sync(~0u, m.z, d); m.w += __shfl_xor_sync(~0u, m.w, d);
            p.x += __shfl_xor_sync(~0u, p.x, d); p.y += __shfl_xor_sync(~0u, p.y, d);
            p.z += __shfl_xor_sync(~0u, p.z, d); p.w += __shfl_xor_sync(~0u, p.w, d);
            qk += __shfl_xor_sync(~0u, qk, d);
        }
        if (lane < CG) {
            part[warp][cg][0] = m;
            part[warp][cg][1] = p;
            if (lane == 0) dots[warp] = qk;
        }
        __syncthreads();
        m = p = make_float4(0.f, 0.f, 0.f, 0.f);
        qk = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            const float4 a = part[w][cg][0];
            m.x += a.x; m.y += a.y; m.z += a.z; m.w += a.w;
        }
        const float4 u = make_float4(beta * (vv[0] - alpha * m.x), beta * (vv[1] - alpha * m.y),
                                     beta * (vv[2] - alpha * m.z), beta * (vv[3] - alpha * m.w));
        if (rg == 0 && live) {
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                const float4 c = part[w][cg][1];
                p.x += c.x; p.y += c.y; p.z += c.z; p.w += c.w;
                qk += dots[w];
            }
            T* out = o + os.at(b, h, 0) + col;
            st_out(out, alpha * p.x + qk * u.x);
            st_out(out + 1, alpha * p.y + qk * u.y);
            st_out(out + 2, alpha * p.z + qk * u.z);
            st_out(out + 3, alpha * p.w + qk * u.w);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float f = kq[rg + i * RG].x;
            S[i].x = alpha * S[i].x + f * u.x; S[i].y = alpha * S[i].y + f * u.y;
            S[i].z = alpha * S[i].z + f * u.z; S[i].w = alpha * S[i].w + f * u.w;
        }
    }
    if (!state_out) return;
    float* s_out = state_out + head * D * D;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = rg + i * RG;
        if (live && r < D) __stcs(reinterpret_cast<float4*>(s_out + (size_t)r * D + col), S[i]);
    }
}

template <typename T>
void launch_typed(const la_delta& in, void* o, const long long os[3], float* state_out,
                  unsigned int* status, cudaStream_t st) {
    auto grid_of = [&](int cols) { return dim3((in.D + cols - 1) / cols, in.Hv, in.B); };
    const dim3 grid = grid_of(kCols);
    T* out = static_cast<T*>(o);
    const Row3 r = o ? row3(os) : Row3{0, 0, 0};
    if (in.T == 1) {
        if (in.D <= 64)
            delta_step_kernel<T, 128, 64, 8><<<grid_of(64), 128, 0, st>>>(in, out, r, state_out, status);
        else if (in.D <= 128)
            delta_step_kernel<T, 128, 32, 8><<<grid, 128, 0, st>>>(in, out, r, state_out, status);
        else
            delta_step_kernel<T, 256, 32, 8><<<grid, 256, 0, st>>>(in, out, r, state_out, status);
        return;
    }
    if (in.D <= 64)
        delta_recurrent_kernel<T, 2><<<grid, kThreads, 0, st>>>(in, out, r, state_out, status);
    else if (in.D <= 128)
        delta_recurrent_kernel<T, 4><<<grid, kThreads, 0, st>>>(in, out, r, state_out, status);
    else
        delta_recurrent_kernel<T, 8><<<grid, kThreads, 0, st>>>(in, out, r, state_out, status);
}

}  // namespace

cudaError_t launch_delta_recurrent(const la_delta& in, void* o, const long long o_stride[3],
                                   float* state_out, unsigned int* status, cudaStream_t st) {
    if (in.dt == LA_BF16) launch_typed<__nv_bfloat16>(in, o, o_stride, state_out, status, st);
    else launch_typed<float>(in, o, o_stride, state_out, status, st);
    return cudaGetLastError();
}

}  // namespace la
