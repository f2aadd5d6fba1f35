// Backward pass of the gated delta rule in chunks of 64 tokens: the formulas, and
// the kernels for float32 inputs (bf16: delta_tc_reverse.cu, delta_tc_grad.cu).
//
// With the forward pass's notation (delta_chunk.cu), dS the gradient of the
// state after a chunk and dO that of its outputs:
//     dU = P^T dO + e^{G_63 - G} o (Kh dS),      dX = dU - L^T (B dU),
//     dS0 = gamma_63 dS + Qh^T (gamma o dO) - Kh^T (gamma B dX).
// delta_reverse_kernel walks a head's chunks from the last to the first with
// these and leaves dS and dX of every chunk.  delta_grad_kernel then forms, for
// all chunks at once, from S0, Z, dS and dX,
//     dV = B dX,   dbeta_i = dX_i . Z_i,   dP_ij = dO_i . U_j (i >= j),
//     dQh = gamma o (dO S0^T) + (dP o E) Kh,
//     dKh = -gamma B dX S0^T + (e^{G_63 - G} o U) dS^T + (dP o E)^T Qh + (N' + N'^T) Kh,
//           N'_ij = -beta_i E_ij dX_i . U_j (i > j),
//     dG_i = qh_i . dQh_i - v_i . dV_i,  and + <dS, S> (S after the chunk) at its last token,
// where dG_i follows from the invariance of the chunk's outputs under a scaling
// of what token i sees; dlog_alpha is dG summed from the chunk's end.
#include "delta_tiles.cuh"

namespace la {
namespace {

// ---------------------------------------------------------------------------
// The chain from the last chunk to the first
// ---------------------------------------------------------------------------
// The columns of dS evolve independently as those of S do, and the kernel is
// the forward chain's mirror: a warp holds dS^T of 16 value columns and DP / KS
// key rows; dO takes v's place.  K, Q and again K come to one place, P and L to
// another, so that two blocks share an SM.
template <int DP, int KS>
struct ReverseSmem {
    static constexpr int kTile = kChunk * DP * 2;
    static constexpr int kLP = kChunk * kChunk * 2;
    static constexpr int kGates = 3 * kChunk * 4;
    static constexpr int oK = 0, oP = oK + kPlanes * kTile, oV = oP + kPlanes * kLP,
                         oGates = oV + ValueTile::kBytes, oExchange = oGates + kGates,
                         oOut = oExchange + KS * 8 * 512, kBytes = oOut + kChunk * 32;
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two blocks on an SM");
};

template <int DP, int KS>
__global__ void __launch_bounds__(32 * KS, 2)
delta_reverse_kernel(la_delta in, DeltaGrad grad, DeltaWs ws) {
    using Sm = ReverseSmem<DP, KS>;
    constexpr int THREADS = 32 * KS;
    constexpr int CH = DP / 8, DK = DP / KS, NT = DK / 8;
    constexpr int NP = kPlanes, NI = kPlanes;
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t base = smem_u32(smem);

    const int tid = threadIdx.x, lane = tid & 31, part = tid >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int head = blockIdx.x, b = head / in.Hv, h = head % in.Hv, hk = h / (in.Hv / in.Hk);
    const int D = in.D;
    const int v0 = blockIdx.y * 16;
    const int k0 = part * DK;
    const int len = seq_len(in.lengths, b, in.T);
    const int nc = (len + kChunk - 1) / kChunk;

    float S[NT][4];                       // dS^T
    {
        const float* s = grad.dstate_out ? grad.dstate_out + (size_t)head * D * D : nullptr;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dk = k0 + nt * 8 + 2 * tq + (e & 1), v = v0 + g + 8 * (e >> 1);
                S[nt][e] = s && dk < D ? s[(size_t)dk * D + v] : 0.f;
            }
    }

    const unsigned char* planes = nullptr;       // of this chunk's K, then of Q
    auto load_place = [&](int which) {
        copy_bytes(base + Sm::oK, planes + which * NI * Sm::kTile, NI * Sm::kTile, tid, THREADS);
        cp_commit();
    };

    for (int c = nc - 1; c >= 0; --c) {
        planes = ws.planes(b * in.Hk + hk, c);
        const float* gates = reinterpret_cast<const float*>(smem + Sm::oGates);
        __syncthreads();            // the chunk behind has been read
        load_values(base + Sm::oV, grad.d_o, row3(grad.do_stride).at(b, h, 0),
                       grad.do_stride[2], v0, c * kChunk, len, tid, THREADS);
        copy_bytes(base + Sm::oP, ws.P(head, c), NP * Sm::kLP, tid, THREADS);
        copy_bytes(base + Sm::oGates, ws.gates(head, c), Sm::kGates, tid, THREADS);
        load_place(0);
        store_image<NP>(ws.dstates(head, c), S, v0, k0, DP, D, lane);
        cp_wait<0>();
        __syncthreads();

        // (Kh dS)^T, this warp's key rows, then the sum of all
        float M[8][4];
        {
            Acc m[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j].zero();
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                uint32_t a[NP][4];
                split_tiles<NP>(S[2 * ks], S[2 * ks + 1], a);
#pragma unroll
                for (int np = 0; np < 4; ++np)
                    product_cols<NP, NP, NI, CH>(m + 2 * np, a, base + Sm::oK, Sm::kTile, np * 16,
                                                 (k0 >> 3) + 2 * ks, lane);
            }
            float4* ex = reinterpret_cast<float4*>(smem + Sm::oExchange);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
                ex[(part * 8 + nt) * 32 + lane] =
                    make_float4(m[nt][0], m[nt][1], m[nt][2], m[nt][3]);
            __syncthreads();        // K has been read
            load_place(1);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) sum_parts<KS>(M[nt], ex, nt, lane);
        }

        // dO^T: its planes (rounded sums of planes are dO itself), and gamma o dO
        uint32_t d[4][NI][4], gd[4][NP][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            float V[2][4], W[2][4];
            load_v(V, smem + Sm::oV, np * 16, lane);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 ga =
                    *reinterpret_cast<const float2*>(gates + (2 * np + j) * 8 + 2 * tq);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    W[j][e] = in.q_scale * ((e & 1) ? ga.y : ga.x) * V[j][e];
            }
            split_tiles<NI>(V[0], V[1], d[np]);
            split_tiles<NP>(W[0], W[1], gd[np]);
        }
        // dU = P^T dO + tail o (Kh dS), X = B dU (split)
        uint32_t x[4][NP][4];
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) {          // tokens 16 jp .. 16 jp + 15
            Acc C[2];
            C[0].zero();
            C[1].zero();
#pragma unroll
            for (int ip = jp; ip < 4; ++ip)
                product_rows<NP, NI, NP, 8>(C, d[ip], base + Sm::oP, Sm::kLP, ip * 16, 2 * jp, lane);
            float X[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int nt = 2 * jp + j;
                const float2 ta =
                    *reinterpret_cast<const float2*>(gates + kChunk + nt * 8 + 2 * tq);
                const float2 be =
                    *reinterpret_cast<const float2*>(gates + 2 * kChunk + nt * 8 + 2 * tq);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    M[nt][e] = C[j][e] + in.k_scale * ((e & 1) ? ta.y : ta.x) * M[nt][e];
                    X[j][e] = ((e & 1) ? be.y : be.x) * M[nt][e];
                }
            }
            split_tiles<NP>(X[0], X[1], x[jp]);
        }
        cp_wait<0>();
        __syncthreads();            // Q has landed, P has been read
        copy_bytes(base + Sm::oP, ws.L(head, c), NP * Sm::kLP, tid, THREADS);
        cp_commit();
        // the update's part of Q: (gamma o dO)^T Qh
        Acc up[NT];
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
            up[2 * np].zero();
            up[2 * np + 1].zero();
#pragma unroll
            for (int ts = 0; ts < 4; ++ts)
                product_rows<NP, NP, NI, CH>(up + 2 * np, gd[ts], base + Sm::oK, Sm::kTile, ts * 16,
                                             (k0 >> 3) + 2 * np, lane);
        }
        cp_wait<0>();
        __syncthreads();            // L has landed, Q has been read
        load_place(0);
        // dX = dU - L^T X
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) {
            Acc C[2];
            C[0].zero();
            C[1].zero();
#pragma unroll
            for (int ip = jp; ip < 4; ++ip)
                product_rows<NP, NP, NP, 8>(C, x[ip], base + Sm::oP, Sm::kLP, ip * 16, 2 * jp, lane);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) M[2 * jp + j][e] -= C[j][e];
        }
        if (part == 0) store_rows<NP>(ws.dX(head, c), M, smem + Sm::oOut, v0, DP, lane);

        // dS^T <- gamma_63 dS^T + (gamma o dO)^T Qh - (gamma B dX)^T Kh
        uint32_t w[4][NP][4];
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            float W[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int nt = 2 * np + j;
                const float2 ga = *reinterpret_cast<const float2*>(gates + nt * 8 + 2 * tq);
                const float2 be =
                    *reinterpret_cast<const float2*>(gates + 2 * kChunk + nt * 8 + 2 * tq);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    W[j][e] = -in.k_scale * ((e & 1) ? ga.y * be.y : ga.x * be.x) * M[nt][e];
            }
            split_tiles<NP>(W[0], W[1], w[np]);
        }
        const float gc = gates[kChunk - 1];
        cp_wait<0>();
        __syncthreads();            // K has landed
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
            Acc* C = up + 2 * np;
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
    }
    if (grad.dstate_in) {
        float* s = grad.dstate_in + (size_t)head * D * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dk = k0 + nt * 8 + 2 * tq + (e & 1), v = v0 + g + 8 * (e >> 1);
                if (dk < D) s[(size_t)dk * D + v] = S[nt][e];
            }
    }
}

// ---------------------------------------------------------------------------
// The gradients of all chunks
// ---------------------------------------------------------------------------
// A block takes one chunk of one key head and adds up the value heads that
// share it, in their order.  Warp w: 16 tokens (w % 4) and a quarter of the columns.
// Shared memory holds one block an SM, whose warps wait for tiles and products in turn:
// 232 us for 640 chunks of 128 (8 warps of half the columns: 265).
constexpr int kGradThreads = 512;

template <int DP>
struct GradSmem {
    static constexpr int kTile = kChunk * DP * 2;
    static constexpr int NI = kPlanes, NP = kPlanes;
    static constexpr int kTri = kChunk * kChunk * 2;
    // half of the rows of a state image; dO, then dP o E and N' + N'^T; Z, then K; dX, then Q
    static constexpr int o0 = 0, o1 = o0 + NP * kTile,
                         k1 = NI * kTile > 2 * NP * kTri ? NI * kTile : 2 * NP * kTri,
                         o2 = o1 + k1, o3 = o2 + NP * kTile, kBytes = o3 + NP * kTile;
};

__device__ __forceinline__ void fetch8(float (&x)[8], const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void fetch8(float (&x)[8], const __nv_bfloat16* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void put8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ float2 fetch2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void put2(float* p, float x, float y) {
    *reinterpret_cast<float2*>(p) = make_float2(x, y);
}

// Eight values from planes `plane` elements apart.
template <int NP>
__device__ __forceinline__ void fetch_planes(float (&x)[8], const __nv_bfloat16* p, size_t plane) {
    fetch8(x, p + (NP - 1) * plane);
#pragma unroll
    for (int j = NP - 2; j >= 0; --j) {
        float y[8];
        fetch8(y, p + j * plane);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += y[e];
    }
}

// NP planes of rows of DP columns (`plane` elements apart) as tiles.
template <int NP, int DP>
__device__ __forceinline__ void load_planes(uint32_t dst, const __nv_bfloat16* src, size_t plane,
                                            int rows, int tid) {
    constexpr int CH = DP / 8;
    for (int i = tid; i < NP * kChunk * CH; i += kGradThreads) {
        const int p = i / (kChunk * CH), r = i / CH % kChunk, c = i % CH;
        if (r < rows)
            cp16(dst + p * (kChunk * DP * 2) + tile_at<CH>(r, c),
                 src + p * plane + (size_t)r * DP + c * 8, true);
    }
}

template <int DP>
__global__ void __launch_bounds__(kGradThreads)
delta_grad_kernel(la_delta in, DeltaGrad grad, DeltaWs ws, int chunks) {
    using Sm = GradSmem<DP>;
    using T = float;
    constexpr int CH = DP / 8, NP = Sm::NP, NI = Sm::NI, kTile = Sm::kTile, kTri = Sm::kTri;
    constexpr int NT = DP / 32;                 // tiles of a warp's columns
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float gates[kGateRows][kChunk];
    __shared__ float s_qdq[4][kChunk], s_vdv[kChunk], s_cross[kGradThreads / 32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rb = warp & 3, ch = warp >> 2, g = lane >> 2, tq = lane & 3;
    const int chunk = blockIdx.x % chunks, khead = blockIdx.x / chunks;
    const int b = khead / in.Hk, hk = khead % in.Hk, ratio = in.Hv / in.Hk, D = in.D;
    const int len = seq_len(in.lengths, b, in.T);
    const int t0 = chunk * kChunk, rows = in.T - t0 < kChunk ? in.T - t0 : kChunk;
    const int on = len - t0 < rows ? (len > t0 ? len - t0 : 0) : rows;   // rows of the sequence
    const uint32_t base = smem_u32(smem);
    const uint32_t r0 = base + Sm::o0, r1 = base + Sm::o1, r2 = base + Sm::o2, r3 = base + Sm::o3;
    const int row[2] = {rb * 16 + g, rb * 16 + g + 8};
    const int col = ch * (DP / 4) + 2 * tq;     // of tile 0
    const int piece0 = ch * (DP / 32);

    float dq[NT][4], dk[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dq[i][e] = dk[i][e] = 0.f;

    const T* q = static_cast<const T*>(in.q) + row3(in.q_stride).at(b, hk, t0);
    // sum over this thread's columns of q o x, per row, added to sum[]
    auto dot_q = [&](float (&sum)[2], const float (&x)[NT][4]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (row[r] >= on) continue;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (col + i * 8 < D) {
                    const float2 f = fetch2(q + row[r] * in.q_stride[2] + col + i * 8);
                    sum[r] += f.x * x[i][2 * r] + f.y * x[i][2 * r + 1];
                }
        }
    };

    for (int rep = 0; rep < ratio; ++rep) {
        const int h = hk * ratio + rep, head = b * in.Hv + h;
        const size_t gate_at = (size_t)head * in.T + t0;
        if (on == 0) {                          // behind the sequence
            for (int i = tid; i < rows; i += kGradThreads)
                grad.dlog_alpha[gate_at + i] = grad.dbeta[gate_at + i] = 0.f;
            T* dv = static_cast<T*>(grad.dv) + gate_at * D;
            const float zero[8] = {};
            for (int i = tid; i < rows * (D / 8); i += kGradThreads) put8(dv + i * 8, zero);
            continue;
        }
        __syncthreads();                        // the last head's readers are done
        for (int i = tid; i < kGateRows * kChunk; i += kGradThreads)
            (&gates[0][0])[i] = ws.gates(head, chunk)[i];
        load_rows_split<DP>(r1, grad.d_o, row3(grad.do_stride).at(b, h, 0), grad.do_stride[2], t0,
                           len, D, tid, kGradThreads);
        load_planes<NP, DP>(r2, ws.Z(head, chunk), (size_t)kChunk * DP, kChunk, tid);
        load_planes<NP, DP>(r3, ws.dX(head, chunk), (size_t)kChunk * DP, kChunk, tid);

        // dO S0^T, dX S0^T and Z dS^T, 64 rows of an image at a time
        float qdq[2] = {0.f, 0.f}, cross = 0.f;
#pragma unroll 1
        for (int image = 0; image < 2; ++image) {
            const __nv_bfloat16* src = image ? ws.dstates(head, chunk) : ws.states(head, chunk);
            Acc a0[NT], a1[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                a0[i].zero();
                a1[i].zero();
            }
#pragma unroll 1
            for (int vb = 0; vb < D; vb += kChunk) {
                const int n = D - vb < kChunk ? D - vb : kChunk;
                __syncthreads();                // the buffer's readers are done
                load_planes<NP, DP>(r0, src + (size_t)vb * DP, (size_t)D * DP, n, tid);
                cp_commit();
                cp_wait<0>();
                __syncthreads();
#pragma unroll 1
                for (int ks = 0; ks < n / 16; ++ks) {
                    const int piece = vb / 8 + 2 * ks;
                    uint32_t x[NP][4];
                    if (image == 0) {
                        uint32_t d[NI][4];
#pragma unroll
                        for (int i = 0; i < NI; ++i)
                            ldsm4(d[i], at_rows<CH>(r1 + i * kTile, rb * 16, piece, lane));
#pragma unroll
                        for (int i = 0; i < NP; ++i)
                            ldsm4(x[i], at_rows<CH>(r3 + i * kTile, rb * 16, piece, lane));
#pragma unroll
                        for (int np = 0; np < NT / 2; ++np) {
                            product_rows<NP, NI, NP, CH>(a0 + 2 * np, d, r0, kTile, ks * 16,
                                                         piece0 + 2 * np, lane);
                            product_rows<NP, NP, NP, CH>(a1 + 2 * np, x, r0, kTile, ks * 16,
                                                         piece0 + 2 * np, lane);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < NP; ++i)
                            ldsm4(x[i], at_rows<CH>(r2 + i * kTile, rb * 16, piece, lane));
#pragma unroll
                        for (int np = 0; np < NT / 2; ++np)
                            product_rows<NP, NP, NP, CH>(a0 + 2 * np, x, r0, kTile, ks * 16,
                                                         piece0 + 2 * np, lane);
                    }
                }
                if (image == 1) {               // <dS, S> with the state after the chunk
                    const __nv_bfloat16* s = ws.states(head, chunk + 1) + (size_t)vb * DP;
                    for (int i = tid; i < n * CH; i += kGradThreads) {
                        const int r = i / CH, c = i % CH;
                        float y[8], z[8];
                        fetch_planes<NP>(y, reinterpret_cast<const __nv_bfloat16*>(
                                                smem + Sm::o0 + tile_at<CH>(r, c)),
                                         (size_t)kChunk * DP);
                        fetch_planes<NP>(z, s + (size_t)r * DP + c * 8, (size_t)D * DP);
#pragma unroll
                        for (int e = 0; e < 8; ++e) cross += y[e] * z[e];
                    }
                }
            }
            float x[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = row[e >> 1];
                    if (image == 0) {
                        x[i][e] = gates[0][t] * a0[i][e];
                        dq[i][e] += x[i][e];
                        dk[i][e] -= gates[0][t] * gates[2][t] * a1[i][e];
                    } else {
                        dk[i][e] += gates[1][t] * gates[2][t] * a0[i][e];
                    }
                }
            if (image == 0) dot_q(qdq, x);
        }

        // dO Z^T and dX Z^T up to the diagonal: this warp's 16 rows, 16 columns
        Acc dp[2], dn[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            dp[i].zero();
            dn[i].zero();
        }
        if (ch <= rb) {
#pragma unroll 1
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t d[NI][4], x[NP][4];
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    ldsm4(d[i], at_rows<CH>(r1 + i * kTile, rb * 16, 2 * ks, lane));
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    ldsm4(x[i], at_rows<CH>(r3 + i * kTile, rb * 16, 2 * ks, lane));
                product_cols<NP, NI, NP, CH>(dp, d, r2, kTile, ch * 16, 2 * ks, lane);
                product_cols<NP, NP, NP, CH>(dn, x, r2, kTile, ch * 16, 2 * ks, lane);
            }
        }
        // dV, dbeta and v . dV: eight threads a row
        {
            const int r = tid >> 3;
            const T* v = static_cast<const T*>(in.v) + row3(in.v_stride).at(b, h, t0) +
                         r * in.v_stride[2];
            T* dv = static_cast<T*>(grad.dv) + (gate_at + r) * D;
            const float beta = gates[2][r];
            float xz = 0.f, vdv = 0.f;
            for (int c = tid & 7; c * 8 < D; c += 8) {
                float x[8], z[8], f[8];
                fetch_planes<NP>(x, reinterpret_cast<const __nv_bfloat16*>(
                                        smem + Sm::o3 + tile_at<CH>(r, c)),
                                 (size_t)kChunk * DP);
                fetch_planes<NP>(z, reinterpret_cast<const __nv_bfloat16*>(
                                        smem + Sm::o2 + tile_at<CH>(r, c)),
                                 (size_t)kChunk * DP);
                if (r < on) fetch8(f, v + c * 8);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xz += x[e] * z[e];
                    x[e] = r < on ? beta * x[e] : 0.f;
                    if (r < on) vdv += f[e] * x[e];
                }
                if (r < rows) put8(dv + c * 8, x);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {
                xz += __shfl_xor_sync(~0u, xz, d);
                vdv += __shfl_xor_sync(~0u, vdv, d);
            }
            if ((tid & 7) == 0) {
                s_vdv[r] = vdv;
                if (r < rows) grad.dbeta[gate_at + r] = r < on ? xz : 0.f;
            }
        }
        __syncthreads();                        // dO, Z and dX have been read

        // dP o E and N' + N'^T as split tiles
        if (ch <= rb) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int ti = row[e >> 1], tj = ch * 16 + i * 8 + 2 * tq + (e & 1);
                    // above the diagonal E may overflow: it is selected away
                    const float E = exp2_sum(gates[3][ti], gates[4][ti], gates[3][tj],
                                             gates[4][tj]) * gates[2][tj];
                    float p = ti >= tj ? E * dp[i][e] : 0.f;
                    float n = ti > tj ? -gates[2][ti] * E * dn[i][e] : 0.f;
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const __nv_bfloat16 ph = __float2bfloat16_rn(p), nh = __float2bfloat16_rn(n);
                        unsigned char* t = smem + Sm::o1 + j * kTri;
                        const uint32_t at = tile_at<8>(ti, tj >> 3) + (tj & 7) * 2;
                        *reinterpret_cast<__nv_bfloat16*>(t + at) = ph;
                        t += NP * kTri;
                        if (ti >= tj) *reinterpret_cast<__nv_bfloat16*>(t + at) = nh;
                        if (ti > tj)
                            *reinterpret_cast<__nv_bfloat16*>(t + tile_at<8>(tj, ti >> 3) +
                                                              (ti & 7) * 2) = nh;
                        p -= __bfloat162float(ph);
                        n -= __bfloat162float(nh);
                    }
                }
            }
        }
        load_rows_split<DP>(r2, in.k, row3(in.k_stride).at(b, hk, 0), in.k_stride[2], t0, len, D,
                           tid, kGradThreads);
        load_rows_split<DP>(r3, in.q, row3(in.q_stride).at(b, hk, 0), in.q_stride[2], t0, len, D,
                           tid, kGradThreads);
        cp_commit();
        cp_wait<0>();
        __syncthreads();

        const uint32_t rn = r1 + NP * kTri;
        {
            Acc a[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) a[i].zero();
#pragma unroll 1
            for (int jp = 0; jp <= rb; ++jp) {      // (dP o E) K
                uint32_t p[NP][4];
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    ldsm4(p[i], at_rows<8>(r1 + i * kTri, rb * 16, 2 * jp, lane));
#pragma unroll
                for (int np = 0; np < NT / 2; ++np)
                    product_rows<NP, NP, NI, CH>(a + 2 * np, p, r2, kTile, jp * 16,
                                                 piece0 + 2 * np, lane);
            }
            float x[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i][e] = in.k_scale * a[i][e];
                    dq[i][e] += x[i][e];
                    a[i].hi[e] = a[i].lo[e] = 0.f;
                }
            dot_q(qdq, x);
#pragma unroll 1
            for (int ip = rb; ip < 4; ++ip) {       // (dP o E)^T Q
                uint32_t p[NP][4];
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    ldsm4_t(p[i], at_cols<8>(r1 + i * kTri, ip * 16, 2 * rb, lane));
#pragma unroll
                for (int np = 0; np < NT / 2; ++np)
                    product_rows<NP, NP, NI, CH>(a + 2 * np, p, r3, kTile, ip * 16,
                                                 piece0 + 2 * np, lane);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dk[i][e] += in.q_scale * a[i][e];
                    a[i].hi[e] = a[i].lo[e] = 0.f;
                }
#pragma unroll 1
            for (int jp = 0; jp < 4; ++jp) {        // (N' + N'^T) K
                uint32_t p[NP][4];
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    ldsm4(p[i], at_rows<8>(rn + i * kTri, rb * 16, 2 * jp, lane));
#pragma unroll
                for (int np = 0; np < NT / 2; ++np)
                    product_rows<NP, NP, NI, CH>(a + 2 * np, p, r2, kTile, jp * 16,
                                                 piece0 + 2 * np, lane);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) dk[i][e] += in.k_scale * a[i][e];
        }

        // dG and its sums from the chunk's end
#pragma unroll
        for (int d = 1; d < 4; d <<= 1)
#pragma unroll
            for (int r = 0; r < 2; ++r) qdq[r] += __shfl_xor_sync(~0u, qdq[r], d);
#pragma unroll
        for (int d = 16; d; d >>= 1) cross += __shfl_xor_sync(~0u, cross, d);
        if (tq == 0)
#pragma unroll
            for (int r = 0; r < 2; ++r) s_qdq[ch][row[r]] = in.q_scale * qdq[r];
        if (lane == 0) s_cross[warp] = cross;
        __syncthreads();
        if (warp == 0) {
            double s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                s[i] = ((double)s_qdq[0][t] + (double)s_qdq[1][t]) +
                       ((double)s_qdq[2][t] + (double)s_qdq[3][t]) - (double)s_vdv[t];
            }
            if (lane == 31)
                for (int i = 0; i < kGradThreads / 32; ++i) s[1] += (double)s_cross[i];
            double run = s[0] + s[1];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double y = __shfl_down_sync(~0u, run, d);
                if (lane + d < 32) run += y;
            }
            const double sum[2] = {run, run - s[0]};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                if (t >= rows) continue;
                // where the decay is 0 the state before the token is forgotten, and before the
                // first one there may be none: exactly 0, where terms of the sum cancel
                const bool kept = t < on && (t > 0 || chunk > 0 || in.state_in) &&
                                  !(in.log_alpha[gate_at + t] <= kForgets);
                grad.dlog_alpha[gate_at + t] = kept ? (float)sum[i] : 0.f;
            }
        }
    }

    const size_t out = ((size_t)khead * in.T + t0) * D;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (row[r] >= rows) continue;
        T* pq = static_cast<T*>(grad.dq) + out + (size_t)row[r] * D;
        T* pk = static_cast<T*>(grad.dk) + out + (size_t)row[r] * D;
        const bool kept = row[r] < on;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int c = col + i * 8;
            if (c >= D) continue;
            put2(pq + c, kept ? in.q_scale * dq[i][2 * r] : 0.f,
                 kept ? in.q_scale * dq[i][2 * r + 1] : 0.f);
            put2(pk + c, kept ? in.k_scale * dk[i][2 * r] : 0.f,
                 kept ? in.k_scale * dk[i][2 * r + 1] : 0.f);
        }
    }
}

template <int DP>
cudaError_t reverse(const la_delta& in, const DeltaGrad& g, const DeltaWs& ws, cudaStream_t st) {
    constexpr int KS = 4;
    using Rs = ReverseSmem<DP, KS>;
    auto* kernel = delta_reverse_kernel<DP, KS>;
    const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), Rs::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<dim3(in.B * in.Hv, in.D / 16), 32 * KS, Rs::kBytes, st>>>(in, g, ws);
    return cudaGetLastError();
}

template <int DP>
cudaError_t backward(const la_delta& in, const DeltaGrad& g, const DeltaWs& ws, cudaStream_t st) {
    using Gs = GradSmem<DP>;
    static_assert(Gs::kBytes <= 220 * 1024, "shared memory of a block");
    cudaError_t e = cudaSuccess;
    if (ws.chunks > 0 && (e = launch_delta_states(in, ws, st)) != cudaSuccess) return e;
    e = reverse<DP>(in, g, ws, st);
    if (e != cudaSuccess || ws.chunks == 0) return e;
    auto* grads = delta_grad_kernel<DP>;
    if ((e = ensure_dyn_smem(reinterpret_cast<const void*>(grads), Gs::kBytes)) != cudaSuccess)
        return e;
    grads<<<(unsigned)(in.B * in.Hk) * (unsigned)ws.chunks, kGradThreads, Gs::kBytes, st>>>(
        in, g, ws, ws.chunks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_backward(const la_delta& in, const DeltaGrad& g, void* ws_mem,
                                  cudaStream_t st) {
    const DeltaWs ws = DeltaWs::layout(ws_mem, 1, in.dt, in.B, in.Hk, in.Hv, in.T, in.D);
    cudaError_t e = cudaSuccess;
    if (in.T == 0 && (e = cudaMemsetAsync(ws.status, 0, 8, st)) != cudaSuccess) return e;
    if (in.dt == LA_BF16) {
        if (in.T > 0) {
            if ((e = launch_delta_tc_prep(in, ws, true, st)) != cudaSuccess) return e;
            if ((e = launch_delta_tc_chain(in, ws, nullptr, Row3{0, 0, 0}, nullptr, true, st)) !=
                cudaSuccess)
                return e;
        }
        if ((e = launch_delta_tc_reverse(in, g, ws, st)) != cudaSuccess || in.T == 0) return e;
        return launch_delta_tc_grad(in, g, ws, st);
    }
    return in.D <= 64 ? backward<64>(in, g, ws, st) : backward<128>(in, g, ws, st);
}

}  // namespace la
