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
// Everything beyond K K^T and Q K^T goes by blocks of 16, block column c by one
// warp, transposed, so that the tiles of one product are the a operand of the
// next.  L: the diagonal blocks by forward substitution (a column a lane), then
//     R = N_rc - sum_j N_rj (B L_jc),   L_rc = R - L_rr (B R).
#include "delta_tiles.cuh"

namespace la {
namespace {

constexpr int kTri = kChunk * kChunk * 2;
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
    static constexpr int kTile = kChunk * DP * 2;
    // K | Q, later P | N | L.  Forward, only L's diagonal blocks are kept (one after
    // another), so that four blocks fit an SM.  A diagonal block of N in float32 lies
    // where the block of L comes that is made from it.
    static constexpr int kP3 = 3 * kPacked, kPitch = 17;
    static constexpr int oK = 0, oP = kTile, oN = oP + (kTile > kP3 ? kTile : kP3), oL = oN + kP3;
    static constexpr int kL = BACKWARD ? kP3 : 4 * 3 * 512;
    static constexpr int oDiag = BACKWARD ? oL + kL : oL, kDiag = BACKWARD ? 16 * kPitch * 4 : 1536;
    static constexpr int kBytes = BACKWARD ? oDiag + 4 * kDiag : oL + kL;
    // staging of Pt (over N and L) and of half of Kt's columns (over P and N)
    static_assert(kP3 + kL >= (BACKWARD ? 3 : 2) * kTri && oL - oP >= 3 * 8192, "staging");
    // a plane of L, and its block (r, r)
    static constexpr int kPlaneL = BACKWARD ? kPacked : 512;
    static __device__ __forceinline__ int block(int r) {
        return BACKWARD ? (r * (r + 1) / 2 + r) * 512 : r * 1536;
    }
};

template <int DP, bool BACKWARD>
__global__ void __launch_bounds__(128, BACKWARD ? 3 : 4)
delta_tc_prep_kernel(la_delta in, DeltaWs ws, int chunks) {
    using Sm = PrepTc<DP, BACKWARD>;
    constexpr int CH = DP / 8;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float g_hi[kChunk], g_lo[kChunk], s_beta[kChunk], s_tail[kChunk];

    const int chunk = blockIdx.x % chunks, head = blockIdx.x / chunks;
    const int b = head / in.Hv, h = head % in.Hv, hk = h / (in.Hv / in.Hk);
    const int len = seq_len(in.lengths, b, in.T);
    const int t0 = chunk * kChunk;
    const int tid = threadIdx.x, lane = tid & 31;
    // block column 0 has the most to do: its warp differs from block to block
    const int warp = ((tid >> 5) + blockIdx.x) & 3;
    if (blockIdx.x == 0 && tid < 2) ws.status[tid] = 0;
    if (t0 >= len) return;
    const uint32_t base = smem_u32(smem);
    const uint32_t sK = base + Sm::oK, sQ = base + Sm::oP, sP = sQ, sN = base + Sm::oN,
                   sL = base + Sm::oL;
    float* diag = reinterpret_cast<float*>(smem + Sm::oDiag + warp * Sm::kDiag);
    const int g = lane >> 2, tq = lane & 3;

    load_rows<DP>(sK, in.k, row3(in.k_stride).at(b, hk, 0), in.k_stride[2], t0, len, in.D,
                         tid, 128);
    load_rows<DP>(sQ, in.q, row3(in.q_stride).at(b, hk, 0), in.q_stride[2], t0, len, in.D,
                         tid, 128);
    cp_commit();
    if (warp == 3)
        chunk_gates(in, ((size_t)b * in.Hv + h) * in.T + t0, len - t0, ws.gates(head, chunk), g_hi,
                    g_lo, s_beta, s_tail, lane);
    cp_wait<0>();
    __syncthreads();

    // Rows 16 w .. 16 w + 15 of K K^T and Q K^T, up to the diagonal.
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[i][e] = qk[i][e] = 0.f;
#pragma unroll 2
    for (int ks = 0; ks < DP / 16; ++ks) {
        uint32_t ak[4], aq[4];
        ldsm4(ak, at_rows<CH>(sK, warp * 16, 2 * ks, lane));
        ldsm4(aq, at_rows<CH>(sQ, warp * 16, 2 * ks, lane));
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > warp) break;
            uint32_t bk[4];
            ldsm4(bk, at_cols<CH>(sK, np * 16, 2 * ks, lane));
            mma_bf16(kk[2 * np], ak, bk[0], bk[1]);
            mma_bf16(kk[2 * np + 1], ak, bk[2], bk[3]);
            mma_bf16(qk[2 * np], aq, bk[0], bk[1]);
            mma_bf16(qk[2 * np + 1], aq, bk[2], bk[3]);
        }
    }
    __syncthreads();                  // Q has been read
    const float k2 = in.k_scale * in.k_scale, qk_scale = in.k_scale * in.q_scale;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        if (nt >= 2 * (warp + 1)) break;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = warp * 16 + g + 8 * r, j = nt * 8 + 2 * tq;
            float n[2], p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // masked places are selected away, never multiplied by 0
                const float E = expf((g_hi[i] - g_hi[j + e]) + (g_lo[i] - g_lo[j + e]));
                n[e] = i > j + e ? k2 * E * kk[nt][2 * r + e] : 0.f;
                p[e] = i >= j + e ? qk_scale * E * qk[nt][2 * r + e] : 0.f;
                if ((nt >> 1) == warp)
                    diag[(i & 15) * Sm::kPitch + ((j + e) & 15)] = n[e];
            }
            uint32_t wn[3], wp[3];
            cut_planes(n[0], n[1], wn);
            cut_planes(p[0], p[1], wp);
            const uint32_t at = packed_at(warp, nt >> 1, i & 15, nt & 1) + 4 * tq;
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                *reinterpret_cast<uint32_t*>(smem + Sm::oP + e * kPacked + at) = wp[e];
                *reinterpret_cast<uint32_t*>(smem + Sm::oN + e * kPacked + at) = wn[e];
            }
        }
    }
    __syncwarp();
    // this warp's diagonal block: column `lane`
    {
        const float* n = diag;
        const int c = lane & 15;
        float l[16], bl[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) {
                if (j & 1) s1 += n[i * Sm::kPitch + j] * bl[j];
                else s0 += n[i * Sm::kPitch + j] * bl[j];
            }
            l[i] = i > c ? n[i * Sm::kPitch + c] - (s0 + s1) : 0.f;
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
    constexpr int NP = BACKWARD ? 3 : 2;
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
            for (int e = 0; e < NP; ++e) ldsm4(p[e], sP + e * kPacked + block_cols(i, warp + r, lane));
            product_planes<NP, 3, 3>(C, bl[r], p);
        }
        float R[2][4] = {};
#pragma unroll
        for (int e = 2; e >= 0; --e) {
            uint32_t w[4];
            ldsm4_t(w, sP + e * kPacked + block_rows(i, warp, lane));
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
    __syncthreads();
    {
        unsigned char* out = reinterpret_cast<unsigned char*>(ws.P(head, chunk));
        for (int i = tid; i < NP * kTri / 16; i += 128)
            reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(smem + Sm::oN)[i];
    }

    __syncthreads();                  // Pt has left, P has been read: Kt is staged there
    // (B L)^T to k_scale (tail o (I - B L))^T
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
    // Kt, 64 columns at a time: rows 16 w .. 16 w + 15
#pragma unroll 1
    for (int half = 0; half < DP / 64; ++half) {
        if (half > 0) __syncthreads();      // the staged values before have left
        unsigned char* stage = smem + Sm::oP;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
            Acc C[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) C[j].zero();
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int r = warp + d;
                if (r > 3) break;
#pragma unroll
                for (int np = 0; np < 2; ++np)
                    product_rows<3, 3, 1, CH>(C + 2 * np, bl[d], sK, Sm::kTile, r * 16,
                                              half * 8 + 4 * q + 2 * np, lane);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t w[3];
                    cut_planes(C[j][2 * r], C[j][2 * r + 1], w);
                    const uint32_t at = tile_at<8>(warp * 16 + g + 8 * r, 4 * q + j) + 4 * tq;
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        *reinterpret_cast<uint32_t*>(stage + e * 8192 + at) = w[e];
                }
        }
        __syncthreads();
        unsigned char* out = ws.Kt(head, chunk) + half * 3 * 8192;
        for (int i = tid; i < 3 * 8192 / 16; i += 128)
            reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(stage)[i];
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
