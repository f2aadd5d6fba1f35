// The forward chain of the chunked gated delta rule on tcgen05 (bf16 inputs);
// Kt, Pt and the mathematics are in delta_tc_prep.cu, the operands' layout in
// delta_tc.cuh.
//
// One block walks the chunks of one head.  The chain itself is
//   MMA warp   KS = S^T K^T   ->   compute warps   X = B (V - gamma o KS)
//   MMA warp   X Kt           ->   compute warps   S = gamma_63 S + X Kt
// with an mbarrier each way; beside it run QS and X Pt^T with the outputs, or
// X L^T with Z = Y - X L^T for the backward pass.  Each of the 16 compute warps
// owns 32 value columns (its quarter of the lanes) and a quarter of the tokens
// (16) and of the key rows.  Three load warps keep the next chunk in flight.
//
// The chain of products and register work bounds it, not its bytes: 2300 cycles of
// products and as many of register work depend on one another, 4800 cycles a chunk in
// all, with outputs 5300 to 6000 (80 heads of 128, 32 chunks: 120 to 124 us, DRAM at
// 25 % of its peak).
#include "delta_tc.cuh"

namespace la {
namespace {
using namespace dtc;

// Shared memory: two stages of K, Q, V and the gates; one of Kt and Pt (or L),
// which are needed for a part of a chunk's time only.
template <int DP, bool STATES>
struct ChainTc {
    static constexpr int kHalf = STATES ? 8192 : 16384;     // K (and Q) rows of 64 columns
    static constexpr int oKQ = 0, oV = (DP / 64) * kHalf, oGates = oV + kChunk * DP * 2,
                         kStage = oGates + 1024;
    static constexpr int kKt = (DP / 64) * 3 * 8192, kPt = (STATES ? 3 : 2) * kTri;
    static constexpr int oKt = 2 * kStage, oPt = oKt + kKt, oOut = oPt + kPt;
    static constexpr int kOut = STATES ? 0 : 1024;      // a warp's outputs on their way
    static constexpr int kBytes = oOut + kComputeWarps * kOut + 1024;
};
// Tensor-memory columns: the first planes of S, later X Kt | the last plane of
// S | KS | QS | X Pt^T or X L^T | the planes of X.
constexpr uint32_t cUpd = 0, cLo = 128, cKS = 192, cQS = 256, cPX = 320, cX = 384;

struct ChainArgs {
    la_delta in;
    DeltaWs ws;
    void* o;
    Row3 os;
    float* state_out;
    int pass;                       // 0: whole chains; 1, 2: the passes over segments
    int skip_rows;                  // tests: chunk of head 0 whose rows are not announced, or -1
};

// The part of a head's chain that a block runs.
struct Job {
    int head, c0, c1;
    bool emit;                      // outputs (or states) and the final state
    bool identity;                  // from the identity, without values
    const float* init;              // or NULL: zeros
    float* last;                    // or NULL
};
__device__ __forceinline__ Job chain_job(const ChainArgs& a) {
    const la_delta& in = a.in;
    const DeltaWs& ws = a.ws;
    const int segs = ws.seg.count, block = blockIdx.x;
    const size_t dd = (size_t)in.D * in.D;
    Job j{block, 0, 0, true, false, nullptr, nullptr};
    int s = 0;
    if (a.pass == 1) {
        const int jobs = segs > 2 ? 2 * segs - 3 : 1, k = block % jobs;
        j.head = block / jobs;
        j.emit = k == 0;
        j.identity = k > segs - 2;
        s = j.identity ? k - (segs - 2) : k;
    } else if (a.pass == 2) {
        j.head = block / (segs - 1);
        s = block % (segs - 1) + 1;
    }
    const int n = (seq_len(in.lengths, j.head / in.Hv, in.T) + kChunk - 1) / kChunk;
    j.c0 = s * ws.seg.chunks;
    j.c1 = min(n, j.c0 + ws.seg.chunks);
    if (j.emit) {
        j.init = s > 0 ? ws.segment(ws.seg_state, j.head, s)
                       : in.state_in ? in.state_in + j.head * dd : nullptr;
        if (n <= j.c0 && s > 0) j.last = nullptr;       // behind the sequence
        else if (n <= j.c0 + ws.seg.chunks) j.last = a.state_out ? a.state_out + j.head * dd : nullptr;
        else if (a.pass == 1) j.last = ws.segment(ws.seg_state, j.head, 1);
    } else {
        j.last = ws.segment(j.identity ? ws.seg_A : ws.seg_B, j.head, s);
    }
    if (j.c1 < j.c0) j.c1 = j.c0;
    return j;
}

template <int DP, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
delta_tc_chain_kernel(ChainArgs args) {
    using Sm = ChainTc<DP, STATES>;
    constexpr int NK = DP / 4;                  // key rows of a thread
    // The update and the next KS go by halves of the key rows, so that half of
    // the warps work on their part of S while the other half's is multiplied.
    constexpr int kHalves = DP / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = tc::align1024(smem_raw);
    __shared__ uint64_t full[2], empty[2], full_kt, full_pt, ready_s[2], ready_x;
    __shared__ uint64_t done_ks, done_qs, done_upd[2], done_px, done_all;
    __shared__ uint32_t s_tmem, s_abort;

    const la_delta& in = args.in;
    const DeltaWs& ws = args.ws;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
    const Job job = chain_job(args);
    const int head = job.head, b = head / in.Hv, h = head % in.Hv, hk = h / (in.Hv / in.Hk);
    const int D = in.D;
    const int len = seq_len(in.lengths, b, in.T);
    const int c0 = job.c0, c1 = job.c1, n = c1 - c0;
    const bool emit = job.emit;
    const tc::Abort ab{&s_abort, ws.status};

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&full[i], kRowThreads);
            tc::mbar_init(&empty[i], kComputeWarps);
            tc::mbar_init(&ready_s[i], kComputeWarps / kHalves);
            tc::mbar_init(&done_upd[i], 1);
        }
        for (uint64_t* bar : {&full_kt, &full_pt, &done_ks, &done_qs, &done_px, &done_all})
            tc::mbar_init(bar, 1);
        tc::mbar_init(&ready_x, kComputeWarps);
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
        // 16 warps x 104 + 4 x 64 = the launch's 20 x 96 registers a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int quarter = warp & 3, part = (warp - kFirstCompute) >> 2;
        const bool alive = quarter * 32 < D;        // else the warp only keeps step
        const int g = lane >> 2, tq = lane & 3;
        const int v0 = quarter * 32;                // value columns v0 + 16 h + 8 r + g
        const int k0 = part * NK, tok = part * 16, side = k0 / 64;
        const uint32_t at = tc::tmem_addr(tm, quarter * 32, 0);
        const uint32_t aS[3] = {at + k0, at + k0 + NK / 2, at + cLo + k0 / 2};
        const uint32_t aX[3] = {at + cX + part * 8, at + cX + 32 + part * 8, at + cX + 64 + part * 8};
        unsigned char* buf = smem + Sm::oOut + (warp - kFirstCompute) * Sm::kOut;

        Frag S[NK / 16];                            // key rows k0 + 16 i + 8 j + 2 tq + (e & 1)
        auto each_state = [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < NK / 16; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = k0 + 16 * i + 8 * j + 2 * tq + (e & 1);
                            const int v = v0 + 16 * h + 8 * (e >> 1) + g;
                            f(S[i][h][j][e], (size_t)k * D + v, k < D && v < D, k == v);
                        }
        };
        each_state([&](float& x, size_t p, bool on, bool one) {
            x = job.identity && one ? 1.f : job.init && on ? job.init[p] : 0.f;
        });
        const int cw = warp - kFirstCompute;
        auto put_state = [&](int c) {               // for the backward pass
#pragma unroll
            for (int i = 0; i < NK / 16; ++i)
                save_frag(ws.state_frags(head, c), NK / 4, i, S[i], cw, lane);
        };
        if (n > 0) {
            if (alive)
#pragma unroll
                for (int j = 0; j < NK / 16; ++j) store_a(aS, 8 * j, S[j]);
            arrive(&ready_s[side], lane);
        }
        if constexpr (STATES)
            if (alive && emit && (n > 0 || c0 == 0)) put_state(c0);

        // The outputs of a chunk, 16 tokens x 32 columns a warp.  They leave one chunk
        // late, while the tensor core has the chain.
        uint32_t ow[2][2][2];
        auto put_out = [&](int c) {
            __syncwarp();
            stage_rows(smem_u32(buf), ow, lane);
            __syncwarp();
            const int col = v0 + (lane & 3) * 8, t0 = c * kChunk + tok + (lane >> 2);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (col < D && t0 + 8 * i < len)
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(args.o) +
                                              args.os.at(b, h, t0 + 8 * i) + col) =
                        staged_row(buf, i, lane);
        };
        for (int i = 0; i < n; ++i) {
            const int c = c0 + i, st = i & 1, ph = i & 1;
            const unsigned char* stage = smem + st * Sm::kStage;
            const float* gates = reinterpret_cast<const float*>(stage + Sm::oGates);
            Frag x, y;
            Factors ga, be, f;
            tc::mbar_wait(&full[st], (i >> 1) & 1, ab, 1);
            factors(ga, gates + tok, tq);
            factors(be, gates + 2 * kChunk + tok, tq);
            if (alive) {
                load_rows_frag(y, smem_u32(stage) + Sm::oV, 8192, tok, v0, lane);
                if (job.identity) each([&](int a, int j, int e) { y[a][j][e] = 0.f; });
            }
            const float gc = gates[kChunk - 1];
#pragma unroll
            for (int j = 0; j < 2; ++j) f[j] = make_float2(-in.k_scale * ga[j].x, -in.k_scale * ga[j].y);
            tc::mbar_wait(&done_ks, ph, ab, 2);
            tc::tc_fence_after();
            if (alive) {
                load_frag(x, at + cKS + tok);
                tc::tmem_wait_ld();
                each([&](int a, int j, int e) {
                    y[a][j][e] += factor(f, j, e) * x[a][j][e];
                    x[a][j][e] = factor(be, j, e) * y[a][j][e];
                });
                store_a(aX, 0, x);
            }
            arrive(&ready_x, lane);
            if (!STATES && emit) {
                if (alive && i > 0) put_out(c - 1);
                tc::mbar_wait(&done_qs, ph, ab, 5);
                tc::tc_fence_after();
                if (alive) {
                    load_frag(y, at + cQS + tok);
                    tc::tmem_wait_ld();
                    each([&](int a, int j, int e) {
                        y[a][j][e] *= in.q_scale * factor(ga, j, e);
                    });
                }
            }

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
                    // the planes go over this part's products, of which the second half
                    // is read after them: they are held back
                    if (NK == 16 && i + 1 < n) store_a(aS, 0, S[j]);
                }
                if (NK > 16 && i + 1 < n)
#pragma unroll
                    for (int j = 0; j < NK / 16; ++j) store_a(aS, 8 * j, S[j]);
            }
            if (i + 1 < n) arrive(&ready_s[side], lane);

            if (!emit) {
                // only the state goes on
            } else if constexpr (STATES) {
                // (the next segment writes the state that it starts from)
                if (alive && (i + 1 < n || (c + 1) * kChunk >= len)) put_state(c + 1);
                tc::mbar_wait(&done_px, ph, ab, 4);
                tc::tc_fence_after();
                if (alive) {
                    load_frag(x, at + cPX + tok);
                    tc::tmem_wait_ld();
                    each([&](int a, int j, int e) { y[a][j][e] -= x[a][j][e]; });
                    save_frag(ws.Z_frags(head, c), 4, 0, y, cw, lane);
                }
            } else {
                tc::mbar_wait(&done_px, ph, ab, 6);
                tc::tc_fence_after();
                if (alive) {
                    load_frag(x, at + cPX + tok);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int a = k >> 2, j = (k >> 1) & 1, r = k & 1;
                        ow[a][j][r] = pack_bf16(y[a][j][2 * r] + x[a][j][2 * r],
                                                y[a][j][2 * r + 1] + x[a][j][2 * r + 1]);
                    }
                }
            }
            // done_upd and, for outputs, done_px were waited for: the stage's products are done
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[st]);
        }
        if constexpr (!STATES)
            if (alive && emit && n > 0) put_out(c1 - 1);
        if (job.last)
            each_state([&](float& x, size_t p, bool on, bool) {
                if (on) job.last[p] = x;
            });
    } else if (warp > 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ------------------------------------------------------------------ load
        const int role = warp - 1;                      // K | V and the gates | Kt, Pt or L
        if (role < 2) {
            const Row3 rows3 = row3(role ? in.v_stride : in.k_stride), q3 = row3(in.q_stride);
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(role ? in.v : in.k) +
                                       rows3.at(b, role ? h : hk, 0);
            // and half of Q's rows each
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(in.q) + q3.at(b, hk, 32 * role);
            for (int i = 0; i < n; ++i) {
                const int c = c0 + i, st = i & 1, t0 = c * kChunk, rows = len - t0;
                if (i >= 2 && !tc::mbar_wait(&empty[st], ((i >> 1) - 1) & 1, ab, 7)) break;
                const uint32_t sa = smem_u32(smem + st * Sm::kStage);
                if (role == 0) {
                    load_tile(sa + Sm::oKQ, Sm::kHalf, src + t0 * rows3.t, rows3.t, rows, D,
                                        lane);
                } else {
                    load_tile(sa + Sm::oV, 8192, src + t0 * rows3.t, rows3.t, rows, D, lane);
                    for (int k = lane; k < 3 * kChunk / 4; k += 32)
                        cp16(sa + Sm::oGates + k * 16, ws.gates(head, c) + k * 4, true);
                }
                if constexpr (!STATES)
                    if (emit && rows > 32 * role)
                        load_tile<32>(sa + Sm::oKQ + 8192 + 4096 * role, Sm::kHalf,
                                                q + t0 * q3.t, q3.t, rows - 32 * role, D, lane);
                cp_commit();
                if (i + 1 < n)                          // the next chunk's, towards the L2
                    prefetch_lines(role == 0 ? ws.Kt(head, c + 1)
                                            : reinterpret_cast<const unsigned char*>(
                                                  STATES ? ws.L(head, c + 1) : ws.P(head, c + 1)),
                                   role == 0 ? Sm::kKt : Sm::kPt, lane);
                cp_wait<0>();
                tc::fence_proxy_async_smem();
                if (role == 1 || head > 0 || c != args.skip_rows) tc::mbar_arrive(&full[st]);
            }
        } else if (lane == 0) {
            // A barrier is armed again only once its last copy was read, so that after an
            // abort at most one copy to each is in flight.
            int kt = -1, pt = -1;                       // the chunks whose copies went out last
            for (int i = 0; i < n; ++i) {
                if (i >= 1 && !tc::mbar_wait(&done_upd[kHalves - 1], (i - 1) & 1, ab, 8)) break;
                tc::mbar_expect_tx(&full_kt, Sm::kKt);
                tc::bulk_load(smem + Sm::oKt, ws.Kt(head, c0 + i), Sm::kKt, &full_kt);
                kt = i;
                if (!emit) continue;
                if (i >= 1 && !tc::mbar_wait(&done_px, (i - 1) & 1, ab, 9)) break;
                tc::mbar_expect_tx(&full_pt, Sm::kPt);
                tc::bulk_load(smem + Sm::oPt, STATES ? ws.L(head, c0 + i) : ws.P(head, c0 + i),
                              Sm::kPt, &full_pt);
                pt = i;
            }
            if (tc::aborted(ab)) {
                if (kt >= 0) tc::mbar_drain(&full_kt, kt & 1);
                if (pt >= 0) tc::mbar_drain(&full_pt, pt & 1);
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
                tc::mbar_wait(&full[st], (i >> 1) & 1, ab, 10);
                tc::mbar_wait(&ready_s[0], ph, ab, 11);
                if (ab.raised()) break;
                tc::tc_fence_after();
                mma_state<3, DP, 0, 4>(tm + cKS, tm, cLo, stage + Sm::oKQ, Sm::kHalf, D / 16);
                if constexpr (kHalves > 1) {
                    tc::mbar_wait(&ready_s[1], ph, ab, 17);
                    if (ab.raised()) break;
                    tc::tc_fence_after();
                    mma_state<3, DP, 4, 8>(tm + cKS, tm, cLo, stage + Sm::oKQ, Sm::kHalf, D / 16);
                }
                tc::mma_commit(&done_ks);
                if (!STATES && emit) {
                    mma_state<2, DP, 0, DP / 16>(tm + cQS, tm, cLo, stage + Sm::oKQ + 8192, Sm::kHalf,
                                     D / 16);
                    tc::mma_commit(&done_qs);
                }
                tc::mbar_wait(&full_kt, ph, ab, 12);
                if (!STATES && emit) tc::mbar_wait(&done_qs, ph, ab, 16);     // it reads S
                tc::mbar_wait(&ready_x, ph, ab, 13);
                if (ab.raised()) break;
                tc::tc_fence_after();
#pragma unroll
                for (int j = 0; j < kHalves; ++j) {
                    mma_update<3>(tm + cUpd + 64 * j, tm + cX, base + Sm::oKt + j * 3 * 8192, 0, 8192,
                                  D - 64 * j < 64 ? D - 64 * j : 64);
                    tc::mma_commit(&done_upd[j]);
                }
                if (!emit) continue;
                tc::mbar_wait(&full_pt, ph, ab, 14);
                if (ab.raised()) break;
                mma_lower<STATES ? 3 : 2>(tm + cPX, tm + cX, base + Sm::oPt);
                tc::mma_commit(&done_px);
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

template <int DP, bool STATES>
cudaError_t chain(const ChainArgs& a, cudaStream_t st) {
    auto* kernel = delta_tc_chain_kernel<DP, STATES>;
    constexpr int bytes = ChainTc<DP, STATES>::kBytes;
    static_assert(bytes <= 227 * 1024, "shared memory of a block");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    const int heads = a.in.B * a.in.Hv, segs = a.ws.seg.count;
    ChainArgs args = a;
    args.pass = segs > 1 ? 1 : 0;
    kernel<<<heads * (segs > 2 ? 2 * segs - 3 : 1), kThreads, bytes, st>>>(args);
    if (segs == 1 || (e = cudaGetLastError()) != cudaSuccess) return segs == 1 ? cudaGetLastError() : e;
    if (segs > 2 && (e = launch_delta_join(a.in, a.ws, false, st)) != cudaSuccess) return e;
    args.pass = 2;
    kernel<<<heads * (segs - 1), kThreads, bytes, st>>>(args);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tc_chain(const la_delta& in, const DeltaWs& ws, void* o, Row3 os,
                                  float* state_out, bool states, cudaStream_t st) {
    const ChainArgs a{in, ws, o, os, state_out, 0, test_skip_rows(false)};
    if (states) return in.D <= 64 ? chain<64, true>(a, st) : chain<128, true>(a, st);
    return in.D <= 64 ? chain<64, false>(a, st) : chain<128, false>(a, st);
}

}  // namespace la
