// Gated delta rule in chunks of 64 tokens: the mathematics, and the kernels for
// float32 inputs on warp-level products (bf16: delta_tc_prep.cu, delta_tc.cu).
//
// Within a chunk that starts from state S0, with G_i the sum of log_alpha up
// to token i, gamma_i = exp(G_i), E_ij = exp(G_i - G_j), B = diag(beta), every
// token writes a rank-one term kh_i u_i^T with
//     (I + B N) U = B (V - gamma o (Kh S0)),   N_ij = E_ij kh_i . kh_j  (i > j).
// Let L = N (I + B N)^-1 = N - N B L (strictly lower triangular).  Then
//     Y = V - gamma o (Kh S0),   Z = Y - L (B Y),   U = B Z,
//     O = gamma o (Qh S0) + P U,                P_ij = E_ij qh_i . kh_j (i >= j),
//     S = gamma_63 S0 + Kh^T (exp(G_63 - G) o U).
// L and P do not depend on the state: delta_prep_kernel forms them for all
// chunks at once; delta_chain_kernel walks the chunks of a head.
#include "delta_tiles.cuh"

namespace la {
namespace {

// ---------------------------------------------------------------------------
// L, P and the gates of every chunk
// ---------------------------------------------------------------------------
// A block of four warps forms one chunk of one value head.
//
// L goes by blocks of 16: the four diagonal blocks by forward substitution (a
// column a lane, 120 steps), then block column c by warp c from the top,
//     R = N_rc - sum_j N_rj (B L_jc),   L_rc = R - L_rr (B R),
// on tensor cores, transposed so that a block's result tiles are the next
// product's a operand; the serial part is 16 rows in place of 64.
//
// K and Q come 64 columns at a time, so that three blocks share an SM: 62 us for 640
// chunks of 128 (one block with all columns: 107).
struct PrepSmem {
    static constexpr int kTile = kChunk * 128, kTri = kChunk * kChunk * 2;
    static constexpr int NI = kPlanes, NP = kPlanes;
    // K and Q, later P, later L, and N; the diagonal blocks of N in float32
    static constexpr int kQ = NI * kTile, kN = kQ, kDiag = 2 * kQ, kPitch = 17;
    static_assert(kTri <= kTile, "P and N take the place of K and Q");
    static constexpr int kBytes = kDiag + 4 * 16 * kPitch * 4;
};

// 64 columns of rows t0 .. of a float32 matrix as tiles of planes, and, where `planes`
// is given, as pieces first .. of tiles of DP columns there.
template <int DP>
__device__ __forceinline__ void load_half(uint32_t dst, const float* src, long long stride, int t0,
                                          int len, int columns, unsigned char* planes, int first,
                                          int tid) {
#pragma unroll
    for (int i = tid; i < kChunk * 8; i += 128) {
        const int r = i >> 3, c = i & 7;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (t0 + r < len && c * 8 < columns) {
            const float4* p = reinterpret_cast<const float4*>(src + (t0 + r) * stride + c * 8);
            x = p[0];
            y = p[1];
        }
        const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint32_t w[4][kPlanes];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16<kPlanes>(f[2 * e], f[2 * e + 1], w[e]);
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) {
            const uint4 v = make_uint4(w[0][j], w[1][j], w[2][j], w[3][j]);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                         :: "r"(dst + j * PrepSmem::kTile + tile_at<8>(r, c)), "r"(v.x), "r"(v.y),
                            "r"(v.z), "r"(v.w) : "memory");
            if (planes)
                *reinterpret_cast<uint4*>(planes + j * kChunk * DP * 2 +
                                          tile_at<DP / 8>(r, first + c)) = v;
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(128, 3)
delta_prep_kernel(la_delta in, DeltaWs ws, int chunks) {
    using Sm = PrepSmem;
    constexpr int NI = Sm::NI, NP = Sm::NP, kTri = Sm::kTri;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float g_hi[kChunk], g_lo[kChunk], s_beta[kChunk];

    const int chunk = blockIdx.x % chunks, head = blockIdx.x / chunks;
    const int b = head / in.Hv, h = head % in.Hv, ratio = in.Hv / in.Hk, hk = h / ratio;
    const int len = seq_len(in.lengths, b, in.T);
    const int t0 = chunk * kChunk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0 && tid < 2) ws.status[tid] = 0;
    if (t0 >= len) return;
    const uint32_t base = smem_u32(smem);
    const uint32_t sK = base, sQ = base + Sm::kQ, sN = base + Sm::kN;
    float* diag = reinterpret_cast<float*>(smem + Sm::kDiag);

    if (warp == 0)
        chunk_gates(fetch_gates(in, ((size_t)b * in.Hv + h) * in.T + t0, len - t0, lane),
                    ws.gates(head, chunk), g_hi, g_lo, s_beta, nullptr, lane);

    // Warp w: rows 16 w .. 16 w + 15 of Kh Kh^T and Qh Kh^T, up to the diagonal.
    Acc kk[8], qk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        kk[i].zero();
        qk[i].zero();
    }
    const float* pk = static_cast<const float*>(in.k) + row3(in.k_stride).at(b, hk, 0);
    const float* pq = static_cast<const float*>(in.q) + row3(in.q_stride).at(b, hk, 0);
    // the planes of k and q that the chains load
    unsigned char* out = h % ratio == 0 ? ws.planes(b * in.Hk + hk, chunk) : nullptr;
#pragma unroll 1
    for (int half = 0; half < DP / 64; ++half) {
        if (half) __syncthreads();
        load_half<DP>(sK, pk + 64 * half, in.k_stride[2], t0, len, in.D - 64 * half, out, 8 * half,
                      tid);
        load_half<DP>(sQ, pq + 64 * half, in.q_stride[2], t0, len, in.D - 64 * half,
                      out ? out + NI * kChunk * DP * 2 : nullptr, 8 * half, tid);
        __syncthreads();
#pragma unroll 1
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t ak[NI][4], aq[NI][4];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                ldsm4(ak[i], at_rows<8>(sK + i * Sm::kTile, warp * 16, 2 * ks, lane));
                ldsm4(aq[i], at_rows<8>(sQ + i * Sm::kTile, warp * 16, 2 * ks, lane));
            }
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                if (np > warp) break;
                uint32_t bk[NI][4];
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    ldsm4(bk[j], at_cols<8>(sK + j * Sm::kTile, np * 16, 2 * ks, lane));
                product_planes<NI, NI, NI>(kk + 2 * np, ak, bk);
                product_planes<NI, NI, NI>(qk + 2 * np, aq, bk);
            }
        }
    }
    __syncthreads();                  // K and Q have been read
    const int g = lane >> 2, tq = lane & 3;
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
                const float E = exp2_sum(g_hi[i], g_lo[i], g_hi[j + e], g_lo[j + e]);
                n[e] = i > j + e ? k2 * E * kk[nt][2 * r + e] : 0.f;
                p[e] = i >= j + e ? qk_scale * E * qk[nt][2 * r + e] : 0.f;
                if ((nt >> 1) == warp)
                    diag[(warp * 16 + (i & 15)) * Sm::kPitch + ((j + e) & 15)] = n[e];
            }
            uint32_t wn[NP], wp[NP];
            split_bf16<NP>(n[0], n[1], wn);
            split_bf16<NP>(p[0], p[1], wp);
            const uint32_t at = tile_at<8>(i, j >> 3) + (j & 7) * 2;
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                *reinterpret_cast<uint32_t*>(smem + e * kTri + at) = wp[e];
                *reinterpret_cast<uint32_t*>(smem + Sm::kN + e * kTri + at) = wn[e];
            }
        }
    }
    __syncthreads();
    {
        unsigned char* to = reinterpret_cast<unsigned char*>(ws.P(head, chunk));
        for (int i = tid; i < NP * kTri / 16; i += 128)
            reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(smem)[i];
    }
    // the diagonal block of warp's rows: column `lane`
    float l[16];
    {
        const float* n = diag + warp * 16 * Sm::kPitch;
        const int c = lane & 15;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) s += n[i * Sm::kPitch + j] * (s_beta[warp * 16 + j] * l[j]);
            l[i] = i > c ? n[i * Sm::kPitch + c] - s : 0.f;
        }
    }
    __syncthreads();                  // P has left
    if (lane < 16)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = l[i];
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const __nv_bfloat16 w = __float2bfloat16_rn(x);
                *reinterpret_cast<__nv_bfloat16*>(
                    smem + e * kTri + tile_at<8>(warp * 16 + i, 2 * warp + (lane >> 3)) +
                    (lane & 7) * 2) = w;
                x -= __bfloat162float(w);
            }
        }
    __syncthreads();

    uint32_t bl[3][NP][4];            // (B L_jc)^T of the blocks so far
    {
        uint32_t w[NP][4];
#pragma unroll
        for (int e = 0; e < NP; ++e)
            ldsm4_t(w[e], at_cols<8>(base + e * kTri, warp * 16, 2 * warp, lane));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = warp * 16 + 2 * tq + (i >> 1) * 8;
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int e = NP - 1; e >= 0; --e) {
                x0 += __uint_as_float(w[e][i] << 16);
                x1 += __uint_as_float(w[e][i] & 0xffff0000u);
            }
            uint32_t p[NP];
            split_bf16<NP>(s_beta[t] * x0, s_beta[t + 1] * x1, p);
#pragma unroll
            for (int e = 0; e < NP; ++e) bl[0][e][i] = p[e];
        }
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) {     // block row r = c + d
        const int r = warp + d;
        if (r > 3) break;
        Acc C[2];
        C[0].zero();
        C[1].zero();
#pragma unroll
        for (int j = 0; j < d; ++j)
            product_cols<NP, NP, NP, 8>(C, bl[j], sN, kTri, r * 16, 2 * (warp + j), lane);
        float R[2][4] = {}, X[2][4];
#pragma unroll
        for (int e = NP - 1; e >= 0; --e) {       // N_rc transposed
            uint32_t w[4];
            ldsm4_t(w, at_rows<8>(sN + e * kTri, r * 16, 2 * warp, lane));
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    R[j][2 * i] += __uint_as_float(w[2 * i + j] << 16);
                    R[j][2 * i + 1] += __uint_as_float(w[2 * i + j] & 0xffff0000u);
                }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                R[j][e] -= C[j][e];
                X[j][e] = s_beta[r * 16 + j * 8 + 2 * tq + (e & 1)] * R[j][e];
            }
        uint32_t x[NP][4];
        split_tiles<NP>(X[0], X[1], x);
        C[0].zero();
        C[1].zero();
        product_cols<NP, NP, NP, 8>(C, x, base, kTri, r * 16, 2 * r, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w[2][NP];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                R[j][e] -= C[j][e];
                X[j][e] = s_beta[r * 16 + j * 8 + 2 * tq + (e & 1)] * R[j][e];
            }
            split_bf16<NP>(R[j][0], R[j][1], w[0]);
            split_bf16<NP>(R[j][2], R[j][3], w[1]);
#pragma unroll
            for (int e = 0; e < NP; ++e)
                stsm2_t(base + e * kTri + tile_at<8>(r * 16 + j * 8 + (lane & 7),
                                                     2 * warp + ((lane >> 3) & 1)),
                        w[0][e], w[1][e]);
        }
        if (d < 3) split_tiles<NP>(X[0], X[1], bl[d]);
    }
    __syncthreads();
    unsigned char* to = reinterpret_cast<unsigned char*>(ws.L(head, chunk));
    for (int i = tid; i < NP * kTri / 16; i += 128)
        reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(smem)[i];
}

// ---------------------------------------------------------------------------
// The chain over a head's chunks
// ---------------------------------------------------------------------------
// The columns of the state evolve independently, so a warp takes 16 of them
// and keeps S^T (16 value columns x key rows) as float32 product tiles in
// registers.  Everything is computed transposed: S^T is the a operand of
// (Kh S)^T = S^T Kh^T, whose result tiles are, rounded, the a operands of the
// products with L^T and P^T, and U^T in turn that of the update of S^T by Kh.
// No intermediate leaves registers; shared memory holds only the chunk's K, Q,
// L, P and V tiles, which the block's warps share.
//
// The chain's length, not its bytes, bounds it: a chunk costs a warp about 500
// products of 8 cycles each.  KS warps therefore share a slice's key rows (each
// holds DP / KS of them): their partial sums of Kh S and Qh S meet in shared
// memory, the middle part is computed by each, the outputs are split between
// them by token.  Their steps leave most of an SM's time unused, so that two blocks
// share it: Q and K, and L and P, come one after the other to the same place.  40 heads
// of 112 with 1000 tokens: 125 us (one block an SM, with places of their own: 187).
template <int DP, int KS, bool STATES>
struct ChainSmem {
    static constexpr int kTile = kChunk * DP * 2;                 // a plane of K or Q
    static constexpr int kLP = kChunk * kChunk * 2;               // a plane of L or P
    static constexpr int kGates = 3 * kChunk * 4;
    static constexpr int oK = 0, oL = oK + kPlanes * kTile, oV = oL + kPlanes * kLP,
                         oGates = oV + ValueTile::kBytes;      // of two chunks
    static constexpr int oExchange = oGates + 2 * kGates;
    // per warp: partial sums, 8 tiles of 512 bytes (twice with outputs)
    static constexpr int kExchange = KS * 8 * 512 * (STATES ? 1 : 2);
    static constexpr int oOut = oExchange + kExchange;
    static constexpr int kOut = STATES ? kChunk * 32 : 0;
    static constexpr int kBytes = oOut + kOut;
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two blocks on an SM");
};

// STATES: instead of outputs, the starting state of every chunk and the final
// one (as split S^T images) and Z (split) are written, for the backward pass.
template <int DP, int KS, bool STATES>
__global__ void __launch_bounds__(32 * KS, 2)
delta_chain_kernel(la_delta in, DeltaWs ws, void* o, Row3 os, float* state_out) {
    using Sm = ChainSmem<DP, KS, STATES>;
    constexpr int THREADS = 32 * KS;
    constexpr int CH = DP / 8;            // 16-byte pieces of a K row
    constexpr int DK = DP / KS;           // key rows of a warp
    constexpr int NT = DK / 8;            // tiles of S^T in a warp
    constexpr int NP = kPlanes, NI = kPlanes;
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t base = smem_u32(smem);

    const int tid = threadIdx.x, lane = tid & 31, part = tid >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int head = blockIdx.x, b = head / in.Hv, h = head % in.Hv, hk = h / (in.Hv / in.Hk);
    const int D = in.D;
    const int v0 = blockIdx.y * 16;           // first value column; D is a multiple of 16
    const int k0 = part * DK;
    const int len = seq_len(in.lengths, b, in.T);
    const int nc = (len + kChunk - 1) / kChunk;

    float S[NT][4];
    {
        const float* s_in = in.state_in ? in.state_in + (size_t)head * D * D : nullptr;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dk = k0 + nt * 8 + 2 * tq + (e & 1), v = v0 + g + 8 * (e >> 1);
                S[nt][e] = s_in && dk < D ? s_in[(size_t)dk * D + v] : 0.f;
            }
    }

    // the first of what the K place holds, V and the gates
    auto load = [&](int c) {
        copy_bytes(base + Sm::oK, ws.planes(b * in.Hk + hk, c) + (STATES ? 0 : NI * Sm::kTile),
                   NI * Sm::kTile, tid, THREADS);
        load_values(base + Sm::oV, in.v, row3(in.v_stride).at(b, h, 0), in.v_stride[2], v0,
                       c * kChunk, len, tid, THREADS);
        copy_bytes(base + Sm::oGates + (c & 1) * Sm::kGates, ws.gates(head, c), Sm::kGates, tid,
                   THREADS);
        cp_commit();
    };

    if (nc > 0) load(0);
    for (int c = 0; c < nc; ++c) {
        const float* gates =
            reinterpret_cast<const float*>(smem + Sm::oGates + (c & 1) * Sm::kGates);
        cp_wait<0>();
        __syncthreads();            // it has landed; L's place is free
        copy_bytes(base + Sm::oL, ws.L(head, c), NP * Sm::kLP, tid, THREADS);
        cp_commit();

        if constexpr (STATES) store_image<NP>(ws.states(head, c), S, v0, k0, DP, D, lane);

        // (Qh S0)^T and (Kh S0)^T, this warp's key rows; every warp adds the parts up in
        // the same order
        float M[8][4], O[8][4];
        float4* ex = reinterpret_cast<float4*>(smem + Sm::oExchange);
        float4* exo = ex + KS * 256;
        auto by_state = [&](float4* to) {
            Acc m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i].zero();
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                uint32_t a[NP][4];
                split_tiles<NP>(S[2 * ks], S[2 * ks + 1], a);
#pragma unroll
                for (int np = 0; np < 4; ++np)
                    product_cols<NP, NP, NI, CH>(m + 2 * np, a, base + Sm::oK, Sm::kTile, np * 16,
                                                 (k0 >> 3) + 2 * ks, lane);
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
                to[(part * 8 + nt) * 32 + lane] =
                    make_float4(m[nt][0], m[nt][1], m[nt][2], m[nt][3]);
        };
        if constexpr (!STATES) {
            by_state(exo);
            __syncthreads();        // Q has been read
            copy_bytes(base + Sm::oK, ws.planes(b * in.Hk + hk, c), NI * Sm::kTile, tid, THREADS);
            cp_commit();
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
                if (nt / (8 / KS) == part) sum_parts<KS>(O[nt], exo, nt, lane);
            cp_wait<0>();
            __syncthreads();        // K and L have landed
        }
        by_state(ex);
        cp_wait<0>();
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) sum_parts<KS>(M[nt], ex, nt, lane);

        // Y = V - gamma o (Kh S0), X = B Y (split), Z = Y - L X
        uint32_t x[4][NP][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            float V[2][4];
            load_v(V, smem + Sm::oV, np * 16, lane);
            float X[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int nt = 2 * np + j;
                const float2 ga = *reinterpret_cast<const float2*>(gates + nt * 8 + 2 * tq);
                const float2 be =
                    *reinterpret_cast<const float2*>(gates + 2 * kChunk + nt * 8 + 2 * tq);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    M[nt][e] = V[j][e] - in.k_scale * ((e & 1) ? ga.y : ga.x) * M[nt][e];
                    X[j][e] = ((e & 1) ? be.y : be.x) * M[nt][e];
                }
            }
            split_tiles<NP>(X[0], X[1], x[np]);
        }
#pragma unroll
        for (int ip = 0; ip < 4; ++ip) {          // tokens 16 ip .. 16 ip + 15
            Acc C[2];
            C[0].zero();
            C[1].zero();
#pragma unroll
            for (int jp = 0; jp <= ip; ++jp)
                product_cols<NP, NP, NP, 8>(C, x[jp], base + Sm::oL, Sm::kLP, ip * 16, 2 * jp, lane);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) M[2 * ip + j][e] -= C[j][e];
        }
        if constexpr (STATES) {
            if (part == 0) store_rows<NP>(ws.Z(head, c), M, smem + Sm::oOut, v0, DP, lane);
        } else {
            __syncthreads();        // L has been read
            copy_bytes(base + Sm::oL, ws.P(head, c), NP * Sm::kLP, tid, THREADS);
            cp_commit();
        }

        // U = B Z; W = exp(G_63 - G) o U for the update
        uint32_t u[4][NP][4], w[4][NP][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            float U[2][4], W[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int nt = 2 * np + j;
                const float2 be =
                    *reinterpret_cast<const float2*>(gates + 2 * kChunk + nt * 8 + 2 * tq);
                const float2 ta =
                    *reinterpret_cast<const float2*>(gates + kChunk + nt * 8 + 2 * tq);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    U[j][e] = ((e & 1) ? be.y : be.x) * M[nt][e];
                    W[j][e] = in.k_scale * ((e & 1) ? ta.y : ta.x) * U[j][e];
                }
            }
            if constexpr (!STATES) split_tiles<NP>(U[0], U[1], u[np]);
            split_tiles<NP>(W[0], W[1], w[np]);
        }

        // S^T <- gamma_63 S^T + W^T Kh, this warp's key rows
        const float gc = gates[kChunk - 1];
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
            Acc C[2];
            C[0].zero();
            C[1].zero();
#pragma unroll
            for (int ts = 0; ts < 4; ++ts)
                product_rows<NP, NP, NI, CH>(C, w[ts], base + Sm::oK, Sm::kTile, ts * 16,
                                             (k0 >> 3) + 2 * np, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S[2 * np][e] = gc * S[2 * np][e] + C[0][e];
                S[2 * np + 1][e] = gc * S[2 * np + 1][e] + C[1][e];
            }
        }

        cp_wait<0>();
        __syncthreads();            // K and V have been read, P has landed
        if (c + 1 < nc) load(c + 1);

        // O^T = gamma o (Qh S0)^T + U^T P^T, this warp's tokens
        if constexpr (!STATES) {
#pragma unroll
            for (int ip = 0; ip < 4; ++ip) {
                if (ip / (4 / KS) != part) continue;
                Acc C[2];
                C[0].zero();
                C[1].zero();
#pragma unroll
                for (int jp = 0; jp <= ip; ++jp)
                    product_cols<NP, NP, NP, 8>(C, u[jp], base + Sm::oL, Sm::kLP, ip * 16, 2 * jp,
                                                lane);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int nt = 2 * ip + j;
                    const float2 ga = *reinterpret_cast<const float2*>(gates + nt * 8 + 2 * tq);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        O[nt][e] = in.q_scale * ((e & 1) ? ga.y : ga.x) * O[nt][e] + C[j][e];
                }
            }
            store_out<KS>(o, os.at(b, h, c * kChunk), os.t, O, part, v0, len - c * kChunk, lane);
        }
    }
    if constexpr (STATES) store_image<NP>(ws.states(head, nc), S, v0, k0, DP, D, lane);
    if (state_out) {
        float* s_out = state_out + (size_t)head * D * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dk = k0 + nt * 8 + 2 * tq + (e & 1), v = v0 + g + 8 * (e >> 1);
                if (dk < D) s_out[(size_t)dk * D + v] = S[nt][e];
            }
    }
}

template <int DP>
cudaError_t prep(const la_delta& in, const DeltaWs& ws, cudaStream_t st) {
    using Sm = PrepSmem;
    const int chunks = (in.T + kChunk - 1) / kChunk;
    auto* kernel = delta_prep_kernel<DP>;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), Sm::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(in.B * in.Hv) * (unsigned)chunks, 128, Sm::kBytes, st>>>(in, ws, chunks);
    return cudaGetLastError();
}

template <int DP, int KS, bool STATES>
cudaError_t chain(const la_delta& in, const DeltaWs& ws, void* o, Row3 os, float* state_out,
                  cudaStream_t st) {
    using Sm = ChainSmem<DP, KS, STATES>;
    auto* kernel = delta_chain_kernel<DP, KS, STATES>;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), Sm::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<dim3(in.B * in.Hv, in.D / 16), 32 * KS, Sm::kBytes, st>>>(in, ws, o, os, state_out);
    return cudaGetLastError();
}

template <int DP>
cudaError_t forward(const la_delta& in, const DeltaWs& ws, void* o, Row3 os, float* state_out,
                    cudaStream_t st) {
    const cudaError_t e = prep<DP>(in, ws, st);
    return e != cudaSuccess ? e : chain<DP, 4, false>(in, ws, o, os, state_out, st);
}

template <int DP>
cudaError_t states(const la_delta& in, const DeltaWs& ws, cudaStream_t st) {
    const cudaError_t e = prep<DP>(in, ws, st);
    return e != cudaSuccess ? e : chain<DP, 4, true>(in, ws, nullptr, Row3{0, 0, 0}, nullptr, st);
}

}  // namespace

// From how many tokens on a call goes by chunks.  One chunk costs 20 to 27 us (bf16)
// or 23 to 33 (float32), with 160 heads of 128 37 and 66, however few of its tokens
// there are; token by token costs 6 us and 0.7 a token, 2.7 with 160 heads of 128.
bool delta_chunked(int backward, int dt, int heads, int T, int D) {
    if (backward) return true;
    if (D > 128) return false;
    return T >= (heads >= 64 ? (dt == LA_F32 ? 24 : 16) : dt == LA_F32 ? 40 : 24);
}

size_t delta_workspace_bytes(int backward, int dt, int B, int Hk, int Hv, int T, int D) {
    if (!delta_chunked(backward, dt, B * Hv, T, D)) return 256;
    return DeltaWs::layout(nullptr, backward, dt, B, Hk, Hv, T, D).bytes;
}

// prep, the chain (a chain over segments is two passes with a join between them)
// and, in the backward pass, the reverse chain and the gradients
int delta_kernel_count(int backward, int dt, int B, int Hk, int Hv, int T) {
    const int chunks = (T + kChunk - 1) / kChunk;
    const int segs = dt == LA_BF16 ? Segments::plan(backward, B * Hv, chunks).count : 1;
    const int chain = segs > 2 ? 3 : segs;
    const int shares = dt == LA_BF16 && Hv > Hk ? 1 : 0;      // dq and dk added up
    return backward ? (chunks ? 2 * chain + 2 + shares : 1) : 1 + chain;
}

cudaError_t launch_delta_chunked(const la_delta& in, void* o, const long long o_stride[3],
                                 float* state_out, void* ws_mem, cudaStream_t st) {
    const DeltaWs ws = DeltaWs::layout(ws_mem, 0, in.dt, in.B, in.Hk, in.Hv, in.T, in.D);
    const Row3 os = row3(o_stride);
    if (in.dt == LA_BF16) {
        const cudaError_t e = launch_delta_tc_prep(in, ws, false, st);
        return e != cudaSuccess ? e : launch_delta_tc_chain(in, ws, o, os, state_out, false, st);
    }
    return in.D <= 64 ? forward<64>(in, ws, o, os, state_out, st)
                      : forward<128>(in, ws, o, os, state_out, st);
}

cudaError_t launch_delta_states(const la_delta& in, const DeltaWs& ws, cudaStream_t st) {
    return in.D <= 64 ? states<64>(in, ws, st) : states<128>(in, ws, st);
}

}  // namespace la
