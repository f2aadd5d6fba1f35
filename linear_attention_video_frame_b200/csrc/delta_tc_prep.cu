// What the tcgen05 chains of the gated delta rule need of every chunk (bf16
// inputs), formed for all chunks at once.
//
// With delta_chunk.cu's notation and T = (I + B N)^-1 = I - B L, a token's
// written value is U = T X with X = B (V - gamma o (Kh S0)), so
//     S = gamma_63 S0 + Kt^T X,      Kt = k_scale T^T (e^{G_63 - G} o Kh),
//     O = gamma o (Qh S0) + Pt X,    Pt = P T = P - (P B) L,
// and in the backward pass dX = T^T dU = Pt^T dO + Kt dS.  With Kt and Pt a
// chunk takes two dependent products in a chain in place of three.
//
// K K^T, Q K^T and Kt are tcgen05 products, one issue each.  What lies between goes
// by blocks of 16 on warp-level products, block column c by one warp, transposed, so
// that the tiles of one product are the a operand of the next.  L: the diagonal
// blocks by forward substitution (a column a lane), then
//     R = N_rc - sum_j N_rj (B L_jc),   L_rc = R - L_rr (B R).
// A block is one chunk's sequence of such steps, bound by their latency (27,000 cycles,
// of which the products take 2,000): four blocks share an SM.  2560 chunks of 128:
// 67 us, DRAM at 22 % of its peak; with K K^T, Q K^T and Kt on warp-level products 86.
#include "delta_tc.cuh"

namespace la {
namespace {
using namespace dtc;

constexpr int kPacked = 10 * 512;            // a plane of the blocks up to the diagonal

// 16-byte piece p (of 2) of row i of block (r, c) in a packed lower triangle.
__device__ __forceinline__ uint32_t packed_at(int r, int c, int i, int p) {
    return (uint32_t)((r * (r + 1) / 2 + c) * 512 + i * 32 + ((p ^ ((i >> 2) & 1)) << 4));
}
__device__ __forceinline__ uint32_t block_rows(int r, int c, int lane) {    // as at_rows
    return packed_at(r, c, lane & 15, lane >> 4);
}
__device__ __forceinline__ uint32_t block_cols(int r, int c, int lane) {    // as at_cols
    return packed_at(r, c, (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
}

template <int DP, bool BACKWARD>
struct PrepTc {
    // [half of the columns]: K | Q, 64 rows of 128 bytes each | planes of P that do not
    // fit where Q was | N | L.  Forward, only L's diagonal blocks are kept (one after
    // another).  A diagonal block of N in float32 lies where the block of L comes that
    // is made from it.
    static constexpr int kHalves = DP / 64, kHalf = 16384, kKQ = kHalves * kHalf;
    static constexpr int NP = BACKWARD ? 3 : 2;             // planes of P and Pt
    static constexpr int kExtra = NP > kHalves ? (NP - kHalves) * kPacked : 0;
    static constexpr int kP3 = 3 * kPacked, kPitch = 20;
    static constexpr int oN = kKQ + kExtra, oL = oN + kP3;
    static constexpr int kL = BACKWARD ? kP3 : 4 * 3 * 512;
    static constexpr int oDiag = BACKWARD ? oL + kL : oL, kDiag = 1536;
    static constexpr int kEnd = BACKWARD ? oDiag + 4 * kDiag : oL + kL, kBytes = kEnd + 1024;
    static __device__ __forceinline__ constexpr int plane_p(int e) {
        return e < kHalves ? e * kHalf + 8192 : kKQ + (e - kHalves) * kPacked;
    }
    // planes of M = k_scale tail o (I - B L), 8192 bytes each: where Q (and P) were, and
    // over N and L; Pt is staged over N and L before
    static __device__ __forceinline__ constexpr int plane_m(int e) {
        return e < kHalves ? e * kHalf + 8192 : oN + (e - kHalves) * 8192;
    }
    static_assert(kP3 + kL >= NP * kTri && kP3 + kL >= (3 - kHalves) * 8192, "staging");
    static_assert(kEnd >= kHalves * 3 * 8192, "staging of Kt, from the start");
    // a plane of L, and its block (r, r)
    static constexpr int kPlaneL = BACKWARD ? kPacked : 512;
    static __device__ __forceinline__ int block(int r) {
        return BACKWARD ? (r * (r + 1) / 2 + r) * 512 : r * 1536;
    }
};

// A wait of this kernel, which starts before the status word is known to be reset.
// False once it ran out.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, unsigned int* status) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::global_timer_ns();
    while (!tc::mbar_try_wait(bar, parity))
        if (tc::global_timer_ns() - t0 > tc::kWaitLimitNs) {
            atomicExch(status, (unsigned)LA_ERR_TIMEOUT);
            return false;
        }
    return true;
}

template <int DP, bool BACKWARD>
__global__ void __launch_bounds__(128, BACKWARD ? 3 : 4)
delta_tc_prep_kernel(la_delta in, DeltaWs ws, int chunks) {
    using Sm = PrepTc<DP, BACKWARD>;
    constexpr int NP = Sm::NP;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = tc::align1024(smem_raw);
    __shared__ __align__(16) float g_hi[kChunk], g_lo[kChunk], s_beta[kChunk], s_tail[kChunk];
    __shared__ uint64_t done, done_all;
    __shared__ uint32_t s_tmem;

    const int chunk = blockIdx.x % chunks, head = blockIdx.x / chunks;
    const int b = head / in.Hv, h = head % in.Hv, hk = h / (in.Hv / in.Hk), D = in.D;
    const int len = seq_len(in.lengths, b, in.T);
    const int t0 = chunk * kChunk, rows = len - t0;
    const int tid = threadIdx.x, lane = tid & 31;
    const int wid = __shfl_sync(~0u, tid >> 5, 0);
    // block column 0 has the most to do: its warp differs from block to block
    const int warp = (wid + blockIdx.x) & 3;
    if (blockIdx.x == 0 && tid < 2) ws.status[tid] = 0;
    if (rows <= 0) return;
    const uint32_t base = smem_u32(smem);
    const uint32_t sN = base + Sm::oN, sL = base + Sm::oL;
    const int g = lane >> 2, tq = lane & 3;

    RawGates raw;                     // asked for first: the sums over them take longest
    if (wid == 3) raw = fetch_gates(in, ((size_t)b * in.Hv + h) * in.T + t0, rows, lane);
    // K and Q, blocks of 16 rows in the order 0 3 1 2: lanes of the products are rows, and
    // so each warp has five blocks of 16 x 16 up to the diagonal.  Two warps each, their
    // own lanes' rows.
    const int rb[2] = {wid & 1, 3 - (wid & 1)};
    {
        const Row3 r3 = row3(wid < 2 ? in.k_stride : in.q_stride);
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(wid < 2 ? in.k : in.q) +
                                   r3.at(b, hk, t0);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int first = 16 * rb[hh];
            load_tile<16>(base + (wid >> 1) * 8192 + (32 * (wid & 1) + 16 * hh) * 128, Sm::kHalf,
                          rows > first ? src + first * r3.t : src, r3.t, rows - first, D, lane);
        }
        cp_commit();
    }
    if (wid == 0) {
        if (lane == 0) {
            tc::mbar_init(&done, 1);
            tc::mbar_init(&done_all, 1);
            tc::fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc(&s_tmem, 64);
        tc::tmem_relinquish();
    }
    if (wid == 3)
        chunk_gates(raw, ws.gates(head, chunk), g_hi, g_lo, s_beta, s_tail, lane);
    cp_wait<0>();
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(~0u, s_tmem, 0);
    if (wid == 0 && tc::elect_one()) {          // [K; Q] K^T: lanes 0 .. 63 and 64 .. 127
        const Desc k(base, 0, 1024);
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
            if (i < D / 16) {
                const uint64_t d = k.at((i >> 2) * Sm::kHalf + (i & 3) * 32);
                tc::mma_bf16(tm, d, d, tc::idesc_bf16(128, 64, false, false), i > 0);
            }
        tc::mma_commit(&done);
    }
    __syncwarp();
    bool ok = wait_bounded(&done, 0, ws.status);
    tc::tc_fence_after();

    // N (warps 0 and 1) and P (2 and 3), 32 rows each, up to the diagonal
    const float scale = in.k_scale * (wid < 2 ? in.k_scale : in.q_scale);
    const uint32_t at = tc::tmem_addr(tm, wid * 32, 0);
    float row_hi[2][2], row_lo[2][2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            row_hi[hh][r] = g_hi[rb[hh] * 16 + 8 * r + g];
            row_lo[hh][r] = g_lo[rb[hh] * 16 + 8 * r + g];
        }
#pragma unroll 1
    for (int cb = 0; cb <= rb[1]; ++cb) {
        Factors col_hi, col_lo;
        factors(col_hi, g_hi + cb * 16, tq);
        factors(col_lo, g_lo + cb * 16, tq);
        Frag x;
        load_frag(x, at + (cb == 0 ? 0 : cb == 3 ? 1 : cb + 1) * 16);     // where block cb is
        tc::tmem_wait_ld();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            if (cb > rb[hh]) continue;
            uint32_t w[3][2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int ti = rb[hh] * 16 + 8 * r + g, tj = cb * 16 + 8 * j + 2 * tq;
                    float y[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // masked places are selected away, never multiplied by 0
                        const float E = exp2_sum(row_hi[hh][r], row_lo[hh][r], factor(col_hi, j, e),
                                                 factor(col_lo, j, e));
                        const bool on = wid < 2 ? ti > tj + e : ti >= tj + e;
                        y[e] = on ? scale * E * x[hh][j][2 * r + e] : 0.f;
                    }
                    uint32_t p[3];
                    if (NP == 2 && wid >= 2) {
                        uint32_t q[2];
                        split_bf16<2>(y[0], y[1], q);
                        p[0] = q[0];
                        p[1] = q[1];
                        p[2] = 0;
                    } else {
                        cut_planes(y[0], y[1], p);
                    }
#pragma unroll
                    for (int e = 0; e < 3; ++e) w[e][j][r] = p[e];
                    if (wid < 2 && cb == rb[hh]) {
                        float* diag = reinterpret_cast<float*>(smem + Sm::oDiag + cb * Sm::kDiag);
                        *reinterpret_cast<float2*>(diag + (8 * r + g) * Sm::kPitch + 8 * j + 2 * tq) =
                            make_float2(y[0], y[1]);
                    }
                }
            const uint32_t to = packed_at(rb[hh], cb, (lane & 7) + 8 * ((lane >> 3) & 1), lane >> 4);
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                if (wid >= 2 && e >= NP) break;
                const uint32_t plane = wid < 2 ? sN + e * kPacked : base + Sm::plane_p(e);
                stsm4(plane + to, w[e][0][0], w[e][0][1], w[e][1][0], w[e][1][1]);
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    // the diagonal blocks of L: column `lane` of this warp's
    {
        const float* n = reinterpret_cast<const float*>(smem + Sm::oDiag + warp * Sm::kDiag);
        const int c = lane & 15;
        float l[16], bl[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < i; j += 4) {
                const float4 q = *reinterpret_cast<const float4*>(n + i * Sm::kPitch + j);
                const float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < i) s[e] += f[e] * bl[j + e];
            }
            l[i] = i > c ? n[i * Sm::kPitch + c] - ((s[0] + s[1]) + (s[2] + s[3])) : 0.f;
            bl[i] = s_beta[warp * 16 + i] * l[i];
        }
        __syncwarp();                 // all of the block has been read
        if (lane < 16)
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                uint32_t p[3];
                cut_planes(l[i], l[i + 1], p);
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    unsigned char* t = smem + Sm::oL + Sm::block(warp) + e * Sm::kPlaneL + (lane & 7) * 2;
                    *reinterpret_cast<uint16_t*>(t + packed_at(0, 0, i, lane >> 3)) = (uint16_t)p[e];
                    *reinterpret_cast<uint16_t*>(t + packed_at(0, 0, i + 1, lane >> 3)) =
                        (uint16_t)(p[e] >> 16);
                }
            }
    }
    __syncthreads();

    // (B L_rc)^T of block column c = warp, r = c + d, as product operands
    uint32_t bl[4][3][4];
    {
        uint32_t w[3][4];
#pragma unroll
        for (int e = 0; e < 3; ++e) ldsm4_t(w[e], sL + Sm::block(warp) + e * Sm::kPlaneL + block_cols(0, 0, lane));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = warp * 16 + 2 * tq + (i >> 1) * 8;
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int e = 2; e >= 0; --e) {
                x0 += __uint_as_float(w[e][i] << 16);
                x1 += __uint_as_float(w[e][i] & 0xffff0000u);
            }
            uint32_t p[3];
            cut_planes(s_beta[t] * x0, s_beta[t + 1] * x1, p);
#pragma unroll
            for (int e = 0; e < 3; ++e) bl[0][e][i] = p[e];
        }
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) {
        const int r = warp + d;
        if (r > 3) break;
        Acc C[2];
        C[0].zero();
        C[1].zero();
#pragma unroll
        for (int j = 0; j < d; ++j) {
            uint32_t n[3][4];
#pragma unroll
            for (int e = 0; e < 3; ++e) ldsm4(n[e], sN + e * kPacked + block_cols(r, warp + j, lane));
            product_planes<3, 3, 3>(C, bl[j], n);
        }
        float R[2][4] = {}, X[2][4];
#pragma unroll
        for (int e = 2; e >= 0; --e) {            // N_rc transposed
            uint32_t w[4];
            ldsm4_t(w, sN + e * kPacked + block_rows(r, warp, lane));
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    R[j][2 * i] += __uint_as_float(w[2 * i + j] << 16);
                    R[j][2 * i + 1] += __uint_as_float(w[2 * i + j] & 0xffff0000u);
                }
        }
        float be[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) be[j][e] = s_beta[r * 16 + j * 8 + 2 * tq + e];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                R[j][e] -= C[j][e];
                X[j][e] = be[j][e & 1] * R[j][e];
            }
        uint32_t x[3][4], l[3][4];
        cut_tiles(X[0], X[1], x);
        C[0].zero();
        C[1].zero();
#pragma unroll
        for (int e = 0; e < 3; ++e) ldsm4(l[e], sL + Sm::block(r) + e * Sm::kPlaneL + block_cols(0, 0, lane));
        product_planes<3, 3, 3>(C, x, l);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                R[j][e] -= C[j][e];
                X[j][e] = be[j][e & 1] * R[j][e];
            }
        cut_tiles(X[0], X[1], bl[d]);
        if constexpr (BACKWARD) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t w[2][3];
                cut_planes(R[j][0], R[j][1], w[0]);
                cut_planes(R[j][2], R[j][3], w[1]);
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    stsm2_t(sL + e * kPacked +
                                packed_at(r, warp, j * 8 + (lane & 7), (lane >> 3) & 1),
                            w[0][e], w[1][e]);
            }
        }
    }
    if constexpr (BACKWARD) {
        __syncthreads();              // L is complete
        unsigned char* out = reinterpret_cast<unsigned char*>(ws.L(head, chunk));
        for (int i = tid; i < 3 * 10 * 32; i += 128) {
            const int e = i / 320, k = i % 320, blk = k >> 5, row = (k >> 1) & 15, p = k & 1;
            const int r = blk < 1 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, c = blk - r * (r + 1) / 2;
            *reinterpret_cast<uint4*>(out + e * kTri + tile_at<8>(r * 16 + row, 2 * c + p)) =
                *reinterpret_cast<const uint4*>(smem + Sm::oL + e * kPacked +
                                                packed_at(r, c, row, p));
        }
    }
    __syncthreads();                  // N and L have been read: Pt is staged over them

    // Pt = P - P B L; outputs in bf16 need two planes of it, states' gradients three
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int i = warp + d;
        if (i > 3) break;
        Acc C[2];
        C[0].zero();
        C[1].zero();
#pragma unroll
        for (int r = 0; r <= d; ++r) {
            uint32_t p[3][4];
#pragma unroll
            for (int e = 0; e < NP; ++e) ldsm4(p[e], base + Sm::plane_p(e) + block_cols(i, warp + r, lane));
            product_planes<NP, 3, 3>(C, bl[r], p);
        }
        float R[2][4] = {};
#pragma unroll
        for (int e = NP - 1; e >= 0; --e) {
            uint32_t w[4];
            ldsm4_t(w, base + Sm::plane_p(e) + block_rows(i, warp, lane));
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    R[j][2 * k] += __uint_as_float(w[2 * k + j] << 16);
                    R[j][2 * k + 1] += __uint_as_float(w[2 * k + j] & 0xffff0000u);
                }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w[2][NP];
#pragma unroll
            for (int e = 0; e < 4; ++e) R[j][e] -= C[j][e];
            if constexpr (NP == 3) {
                cut_planes(R[j][0], R[j][1], w[0]);
                cut_planes(R[j][2], R[j][3], w[1]);
            } else {
                split_bf16<NP>(R[j][0], R[j][1], w[0]);
                split_bf16<NP>(R[j][2], R[j][3], w[1]);
            }
#pragma unroll
            for (int e = 0; e < NP; ++e)
                stsm2_t(sN + e * kTri + tile_at<8>(i * 16 + j * 8 + (lane & 7),
                                                   2 * warp + ((lane >> 3) & 1)),
                        w[0][e], w[1][e]);
        }
    }
    tc::fence_proxy_async_smem();
    __syncthreads();
    if (wid == 0 && lane == 0) {
        tc::bulk_store(ws.P(head, chunk), smem + Sm::oN, NP * kTri);
        tc::bulk_commit();
    }

    // (B L)^T to M^T = k_scale (tail o (I - B L))^T, and M's rows as operand tiles
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int r = warp + d;
        if (r > 3) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 2 * tq + (i >> 1) * 8;
            float x[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 2; e >= 0; --e) {
                x[0] += __uint_as_float(bl[d][e][i] << 16);
                x[1] += __uint_as_float(bl[d][e][i] & 0xffff0000u);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float one = d == 0 && g + 8 * (i & 1) == t + e ? 1.f : 0.f;
                x[e] = in.k_scale * s_tail[r * 16 + t + e] * (one - x[e]);
            }
            uint32_t p[3];
            cut_planes(x[0], x[1], p);
#pragma unroll
            for (int e = 0; e < 3; ++e) bl[d][e][i] = p[e];
        }
    }
    if (wid == 0 && lane == 0) tc::bulk_wait_read<0>();
    __syncthreads();                  // Pt has left
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int r = warp + d;
        if (r > 3) break;
        const int row = (r == 0 ? 0 : r == 3 ? 1 : r + 1) * 16 + 8 * (lane >> 4) + (lane & 7),
                  c = 2 * warp + ((lane >> 3) & 1);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            stsm4_t(base + Sm::plane_m(e) + row * 128 + ((c ^ (row & 7)) << 4), bl[d][e][0],
                    bl[d][e][1], bl[d][e][2], bl[d][e][3]);
    }
    tc::fence_proxy_async_smem();
    __syncthreads();
    if (wid == 0 && tc::elect_one()) {          // Kt^T = K^T M, block row r of M up to its diagonal
        tc::tc_fence_after();
        const Desc a(base, DP == 64 ? 0 : Sm::kHalf, 1024);
#pragma unroll
        for (int e = 2; e >= 0; --e) {
            const Desc m(base + Sm::plane_m(e), 0, 1024);
#pragma unroll
            for (int r = 3; r >= 0; --r) {      // the widest first: it sets all columns
                const int p = r == 0 ? 0 : r == 3 ? 1 : r + 1;
                tc::mma_bf16(tm, a.at(p * 2048), m.at(p * 2048),
                             tc::idesc_bf16(128, 16 * r + 16, true, true), e < 2 || r < 3);
            }
        }
        tc::mma_commit(&done);
    }
    __syncwarp();
    ok = wait_bounded(&done, 1, ws.status) && ok;
    tc::tc_fence_after();
    // its planes as rows of tokens, over everything
    if (wid < DP / 32)
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            Frag x;
            load_frag(x, at + 16 * i);
            tc::tmem_wait_ld();
            uint32_t w[3][2][2][2];
            planes_of<3>(w, x);
#pragma unroll
            for (int e = 0; e < 3; ++e)
                put_cols(base + ((wid >> 1) * 3 + e) * 8192, w[e], 32 * (wid & 1), 16 * i, lane);
        }
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    if (wid == 0) {
        if (!ok && tc::elect_one()) {           // nothing in flight when the memory is freed
            tc::mma_commit(&done_all);
            tc::mbar_drain(&done_all, 0);
        }
        __syncwarp();
        tc::tc_fence_after();
        tc::tmem_dealloc(tm, 64);
        if (lane == 0) {
            tc::bulk_store(ws.Kt(head, chunk), smem, Sm::kHalves * 3 * 8192);
            tc::bulk_commit();
            tc::bulk_wait_read<0>();
        }
    }
}

template <int DP, bool BACKWARD>
cudaError_t prep(const la_delta& in, const DeltaWs& ws, cudaStream_t st) {
    auto* kernel = delta_tc_prep_kernel<DP, BACKWARD>;
    constexpr int bytes = PrepTc<DP, BACKWARD>::kBytes;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(in.B * in.Hv) * (unsigned)ws.chunks, 128, bytes, st>>>(in, ws, ws.chunks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tc_prep(const la_delta& in, const DeltaWs& ws, bool backward,
                                 cudaStream_t st) {
    if (in.D <= 64) return backward ? prep<64, true>(in, ws, st) : prep<64, false>(in, ws, st);
    return backward ? prep<128, true>(in, ws, st) : prep<128, false>(in, ws, st);
}

}  // namespace la
