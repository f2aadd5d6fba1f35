// The chain of the backward pass on tcgen05 (bf16 inputs), from a head's last
// chunk to its first; Kt, Pt and the mathematics are in delta_tc_prep.cu and
// delta_grad.cu, the operands' layout in delta_tc.cuh.
//
// With dS the gradient of the state after the chunk, transposed like everything:
//   MMA warp   dX = dO Pt + dS Kt^T               ->  compute warps  W = -k_scale gamma B dX
//   MMA warp   dS' = (q_scale gamma dO) Q + W K   ->  compute warps  dS = gamma_63 dS + dS'
// dO Pt and the first term of dS' do not depend on dS and run ahead.  dS (as it
// is before the chunk) and dX are left in float32 for delta_tc_grad_kernel.  32 heads
// of 128 in 64 chunks: 68 and 77 us in two passes, DRAM at 41 and 54 % of its peak.
#include "delta_tc.cuh"

namespace la {
namespace {
using namespace dtc;

template <int DP>
struct ReverseTc {
    static constexpr int kRows = (DP / 64) * 8192;      // K, Q or dO
    // with DP = 64 the second block of dO's columns is whatever lies behind it
    static constexpr int oK = 0, oQ = kRows, oO = 2 * kRows, oGates = 3 * kRows + (DP == 64 ? 8192 : 0),
                         kStage = oGates + 1024;
    static constexpr int kKt = 3 * kRows, kPt = 3 * kTri;
    static constexpr int oKt = 2 * kStage, oPt = oKt + kKt, kBytes = oPt + kPt + 1024;
};
// Tensor-memory columns: the first planes of dS, later dS' | its last plane |
// dX of the first planes | dX of the others | the planes of W | of gamma dO.
constexpr uint32_t cUpd = 0, cLo = 128, cXh = 192, cXl = 256, cW = 320, cG = 416;

struct ReverseArgs {
    la_delta in;
    DeltaGrad grad;
    DeltaWs ws;
    int pass;                       // 0: whole chains; 1, 2: the passes over segments
    int skip_rows;                  // tests: chunk of head 0 whose rows are not announced, or -1
};

// The part of a head's chain that a block runs.  seg_state now holds dS behind
// each segment.
struct Job {
    int head, c0, c1;
    bool emit;                      // dS and dX of the chunks
    const float* init;              // or NULL: zeros
    float* last;                    // or NULL
};
__device__ __forceinline__ Job reverse_job(const ReverseArgs& a) {
    const la_delta& in = a.in;
    const DeltaWs& ws = a.ws;
    const int segs = ws.seg.count, block = blockIdx.x;
    const size_t dd = (size_t)in.D * in.D;
    Job j{block, 0, 0, true, nullptr, nullptr};
    int s = 0;
    if (a.pass > 0) {
        j.head = block / (segs - 1);
        s = block % (segs - 1) + (a.pass == 1 ? 1 : 0);     // pass 1: 1 ..; pass 2: 0 .. segs - 2
    }
    const int n = (seq_len(in.lengths, j.head / in.Hv, in.T) + kChunk - 1) / kChunk;
    j.c0 = s * ws.seg.chunks;
    j.c1 = min(n, j.c0 + ws.seg.chunks);
    const bool is_last = n <= j.c0 + ws.seg.chunks, none = s > 0 && n <= j.c0;
    const float* outer = a.grad.dstate_out ? a.grad.dstate_out + j.head * dd : nullptr;
    if (none || (a.pass == 2 && s > 0 && is_last)) {        // behind the sequence, or run before
        j.c1 = j.c0;
        j.emit = false;
        return j;
    }
    j.emit = a.pass != 1 || is_last;
    j.init = is_last ? outer : j.emit ? ws.segment(ws.seg_state, j.head, s) : nullptr;
    if (s == 0) j.last = a.grad.dstate_in ? a.grad.dstate_in + j.head * dd : nullptr;
    else if (a.pass == 1)
        j.last = j.emit ? ws.segment(ws.seg_state, j.head, s - 1) : ws.segment(ws.seg_B, j.head, s);
    return j;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
delta_tc_reverse_kernel(ReverseArgs args) {
    using Sm = ReverseTc<DP>;
    constexpr int NK = DP / 4, kHalves = DP / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = tc::align1024(smem_raw);
    __shared__ uint64_t full[2], empty[2], full_kt, full_pt, ready_s[2], ready_g, ready_w;
    __shared__ uint64_t done_dx, done_upd[2], done_all;
    __shared__ uint32_t s_tmem, s_abort;

    const la_delta& in = args.in;
    const DeltaWs& ws = args.ws;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
    const Job job = reverse_job(args);
    const int head = job.head, b = head / in.Hv, h = head % in.Hv, hk = h / (in.Hv / in.Hk);
    const int D = in.D;
    const int len = seq_len(in.lengths, b, in.T);
    const int c1 = job.c1, n = c1 - job.c0;
    const tc::Abort ab{&s_abort, ws.status};

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&full[i], kRowThreads);
            tc::mbar_init(&empty[i], kComputeWarps);
            tc::mbar_init(&ready_s[i], kComputeWarps / kHalves);
            tc::mbar_init(&done_upd[i], 1);
        }
        for (uint64_t* bar : {&full_kt, &full_pt, &done_dx, &done_all}) tc::mbar_init(bar, 1);
        tc::mbar_init(&ready_g, kComputeWarps);
        tc::mbar_init(&ready_w, kComputeWarps);
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = s_tmem;

    if (warp >= kFirstCompute) {
        // ---------------------------------------------------------------- compute
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int cw = warp - kFirstCompute, quarter = warp & 3, part = cw >> 2;
        const bool alive = quarter * 32 < D;
        const int g = lane >> 2, tq = lane & 3, v0 = quarter * 32;
        const int k0 = part * NK, tok = part * 16, side = k0 / 64;
        const uint32_t at = tc::tmem_addr(tm, quarter * 32, 0);
        const uint32_t aS[3] = {at + k0, at + k0 + NK / 2, at + cLo + k0 / 2};
        const uint32_t aW[3] = {at + cW + part * 8, at + cW + 32 + part * 8, at + cW + 64 + part * 8};
        const uint32_t aG[3] = {at + cG + part * 8, at + cG + 32 + part * 8, at + cG + 64 + part * 8};

        Frag S[NK / 16];                            // dS
        auto each_state = [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < NK / 16; ++i)
                each([&](int hh, int j, int e) {
                    const int k = k0 + 16 * i + 8 * j + 2 * tq + (e & 1);
                    const int v = v0 + 16 * hh + 8 * (e >> 1) + g;
                    f(S[i][hh][j][e], (size_t)k * D + v, k < D && v < D);
                });
        };
        each_state([&](float& x, size_t p, bool on) {
            x = job.init && on ? job.init[p] : 0.f;
        });
        if (n > 0) {
            if (alive)
#pragma unroll
                for (int j = 0; j < NK / 16; ++j) store_a(aS, 8 * j, S[j]);
            arrive(&ready_s[side], lane);
        }

        for (int i = 0; i < n; ++i) {
            const int c = c1 - 1 - i, st = i & 1, ph = i & 1;
            const unsigned char* stage = smem + st * Sm::kStage;
            const float* gates = reinterpret_cast<const float*>(stage + Sm::oGates);
            Frag x, y;
            Factors ga, be;
            tc::mbar_wait(&full[st], (i >> 1) & 1, ab, 1);
            factors(ga, gates + tok, tq);
            factors(be, gates + 2 * kChunk + tok, tq);
            const float gc = gates[kChunk - 1];
            if (alive) {
                load_rows_frag(y, smem_u32(stage) + Sm::oO, 8192, tok, v0, lane);
                each([&](int a, int j, int e) { y[a][j][e] *= in.q_scale * factor(ga, j, e); });
                store_a(aG, 0, y);
            }
            arrive(&ready_g, lane);
            if (alive && job.emit)
#pragma unroll
                for (int j = 0; j < NK / 16; ++j)
                    save_frag(ws.dstate_frags(head, c), NK / 4, j, S[j], cw, lane);

            tc::mbar_wait(&done_dx, ph, ab, 2);
            tc::tc_fence_after();
            if (alive) {
                load_frag(x, at + cXh + tok);
                load_frag(y, at + cXl + tok);
                tc::tmem_wait_ld();
                each([&](int a, int j, int e) {
                    y[a][j][e] += x[a][j][e];
                    x[a][j][e] = -in.k_scale * (factor(ga, j, e) * factor(be, j, e)) * y[a][j][e];
                });
                store_a(aW, 0, x);
            }
            arrive(&ready_w, lane);
            if (alive && job.emit) save_frag(ws.dX_frags(head, c), 4, 0, y, cw, lane);

            tc::mbar_wait(&done_upd[side], ph, ab, 3);
            tc::tc_fence_after();
            if (alive) {
#pragma unroll
                for (int j = 0; j < NK / 16; ++j) {
                    load_frag(x, at + cUpd + k0 + 16 * j);
                    tc::tmem_wait_ld();
                    each([&](int a, int t, int e) {
                        S[j][a][t][e] = gc * S[j][a][t][e] + x[a][t][e];
                    });
                }
                // the planes go over this part's products: after all of them are read
                if (i + 1 < n)
#pragma unroll
                    for (int j = 0; j < NK / 16; ++j) store_a(aS, 8 * j, S[j]);
            }
            if (i + 1 < n) arrive(&ready_s[side], lane);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[st]);
        }
        if (job.last)
            each_state([&](float& x, size_t p, bool on) {
                if (on) job.last[p] = x;
            });
    } else if (warp > 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ------------------------------------------------------------------ load
        const int role = warp - 1;                      // K | dO and the gates | Kt and Pt
        if (role < 2) {
            const Row3 rows3 = row3(role ? args.grad.do_stride : in.k_stride), q3 = row3(in.q_stride);
            const __nv_bfloat16* src =
                static_cast<const __nv_bfloat16*>(role ? args.grad.d_o : in.k) +
                rows3.at(b, role ? h : hk, 0);
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(in.q) + q3.at(b, hk, 32 * role);
            for (int i = 0; i < n; ++i) {
                const int c = c1 - 1 - i, st = i & 1, t0 = c * kChunk, rows = len - t0;
                if (i >= 2 && !tc::mbar_wait(&empty[st], ((i >> 1) - 1) & 1, ab, 7)) break;
                const uint32_t sa = smem_u32(smem + st * Sm::kStage);
                load_tile(sa + (role ? Sm::oO : Sm::oK), 8192, src + t0 * rows3.t, rows3.t, rows, D,
                          lane);
                // rows behind the sequence read as 0, from an address that exists
                load_tile<32>(sa + Sm::oQ + 4096 * role, 8192,
                              rows > 32 * role ? q + t0 * q3.t : q - 32 * role * q3.t, q3.t,
                              rows - 32 * role, D, lane);
                if (role)
                    for (int k = lane; k < 3 * kChunk / 4; k += 32)
                        cp16(sa + Sm::oGates + k * 16, ws.gates(head, c) + k * 4, true);
                cp_commit();
                if (i + 1 < n)                          // the next chunk's, towards the L2
                    prefetch_lines(role == 0 ? ws.Kt(head, c - 1)
                                            : reinterpret_cast<const unsigned char*>(ws.P(head, c - 1)),
                                   role == 0 ? Sm::kKt : Sm::kPt, lane);
                cp_wait<0>();
                tc::fence_proxy_async_smem();
                if (role == 1 || head > 0 || c != args.skip_rows) tc::mbar_arrive(&full[st]);
            }
        } else if (lane == 0) {
            int armed = -1;                             // the chunk whose copies went out last
            for (int i = 0; i < n; ++i) {
                if (i >= 1 && !tc::mbar_wait(&done_dx, (i - 1) & 1, ab, 8)) break;
                tc::mbar_expect_tx(&full_pt, Sm::kPt);
                tc::bulk_load(smem + Sm::oPt, ws.P(head, c1 - 1 - i), Sm::kPt, &full_pt);
                tc::mbar_expect_tx(&full_kt, Sm::kKt);
                tc::bulk_load(smem + Sm::oKt, ws.Kt(head, c1 - 1 - i), Sm::kKt, &full_kt);
                armed = i;
            }
            if (armed >= 0 && tc::aborted(ab)) {
                tc::mbar_drain(&full_kt, armed & 1);
                tc::mbar_drain(&full_pt, armed & 1);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ------------------------------------------------------------------- MMA
        const uint32_t base = __shfl_sync(~0u, smem_u32(smem), 0);
        const uint32_t tm = __shfl_sync(~0u, s_tmem, 0);
        if (tc::elect_one()) {
            for (int i = 0; i < n; ++i) {
                const int st = i & 1, ph = i & 1;
                const uint32_t stage = base + st * Sm::kStage;
                // dX of the chunk before was read before its W came
                tc::mbar_wait(&full[st], (i >> 1) & 1, ab, 10);
                tc::mbar_wait(&full_pt, ph, ab, 11);
                if (ab.raised()) break;
                mma_rows_lower(tm + cXh, tm + cXl, stage + Sm::oO, 8192, base + Sm::oPt);
                tc::mbar_wait(&full_kt, ph, ab, 12);
                tc::mbar_wait(&ready_s[0], ph, ab, 13);
                if (ab.raised()) break;
                tc::tc_fence_after();
                mma_state_planes<DP, 0, 4>(tm + cXh, tm + cXl, tm, cLo, base + Sm::oKt, 3 * 8192,
                                           8192, D / 16);
                if constexpr (kHalves > 1) {
                    tc::mbar_wait(&ready_s[1], ph, ab, 14);
                    if (ab.raised()) break;
                    tc::tc_fence_after();
                    mma_state_planes<DP, 4, 8>(tm + cXh, tm + cXl, tm, cLo, base + Sm::oKt, 3 * 8192,
                                               8192, D / 16);
                }
                tc::mma_commit(&done_dx);
                tc::mbar_wait(&ready_g, ph, ab, 15);
                tc::mbar_wait(&done_dx, ph, ab, 16);        // it reads dS, which dS' replaces
                if (ab.raised()) break;
                tc::tc_fence_after();
#pragma unroll
                for (int j = 0; j < kHalves; ++j)
                    mma_planes_rows(tm + cUpd + 64 * j, tm + cG, stage + Sm::oQ + 8192 * j,
                                    D - 64 * j < 64 ? D - 64 * j : 64, false);
                tc::mbar_wait(&ready_w, ph, ab, 17);
                if (ab.raised()) break;
                tc::tc_fence_after();
#pragma unroll
                for (int j = 0; j < kHalves; ++j) {
                    mma_planes_rows(tm + cUpd + 64 * j, tm + cW, stage + Sm::oK + 8192 * j,
                                    D - 64 * j < 64 ? D - 64 * j : 64, true);
                    tc::mma_commit(&done_upd[j]);
                }
            }
            tc::mma_commit(&done_all);
            tc::mbar_drain(&done_all, 0);       // nothing in flight when the memory is freed
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

template <int DP>
cudaError_t reverse(const ReverseArgs& a, cudaStream_t st) {
    auto* kernel = delta_tc_reverse_kernel<DP>;
    constexpr int bytes = ReverseTc<DP>::kBytes;
    static_assert(bytes <= 227 * 1024, "shared memory of a block");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    const int heads = a.in.B * a.in.Hv, segs = a.ws.seg.count;
    ReverseArgs args = a;
    args.pass = segs > 1 ? 1 : 0;
    kernel<<<heads * (segs > 1 ? segs - 1 : 1), kThreads, bytes, st>>>(args);
    if (segs == 1 || (e = cudaGetLastError()) != cudaSuccess) return segs == 1 ? cudaGetLastError() : e;
    if (segs > 2 && (e = launch_delta_join(a.in, a.ws, true, st)) != cudaSuccess) return e;
    args.pass = 2;
    kernel<<<heads * (segs - 1), kThreads, bytes, st>>>(args);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tc_reverse(const la_delta& in, const DeltaGrad& g, const DeltaWs& ws,
                                    cudaStream_t st) {
    const ReverseArgs a{in, g, ws, 0, test_skip_rows(true)};
    return in.D <= 64 ? reverse<64>(a, st) : reverse<128>(a, st);
}

}  // namespace la
