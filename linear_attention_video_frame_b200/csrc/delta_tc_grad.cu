// The gradients of all chunks on tcgen05 (bf16 inputs), from the states S0, Z, dS
// and dX that the two chains left; the formulas are in delta_grad.cu.
//
// A block takes one chunk of one key head and adds up the value heads that share
// it, in their order.  Its 16 warps hold fragments as the chains did (a quarter of
// the lanes, a quarter of the columns each).  Products, transposed where they
// are of key rows:
//   rows (dO | dX) Z^T     [tokens, 2 x 64 lanes] x [64 tokens]
//   S0 dO^T, S0 dX^T, dS Z^T, K^T dP', Q^T dP'^T, K^T (N' + N'^T)   [128 key rows] x [64 tokens]
// in bf16 planes: three where dlog_alpha (float32) depends on them, two for what
// only reaches the bf16 dk.
#include "delta_tc.cuh"

namespace la {
namespace {
using namespace dtc;

constexpr int kGradThreads = kComputeWarps * 32;

template <int DP>
struct GradTc {
    static constexpr int kHalves = DP / 64;
    static constexpr int kRows = kHalves * 8192;            // 64 rows of DP columns
    // With DP = 64 an operand of 128 lanes reads a second block of columns: what
    // lies behind the first, for lanes that nobody looks at.
    // [half]: dO | first planes of dX | second planes of dX; then N' in two planes, K, Q
    static constexpr int oX = 0, kXHalf = 3 * 8192, oN = oX, oK = oX + 2 * kTri, oQ = oK + kRows;
    static constexpr int kX = kHalves * kXHalf > oQ + kRows ? kHalves * kXHalf : oQ + kRows;
    static constexpr int oZ = oX + kX, kZHalf = 3 * 8192;                // [half][plane]
    // V, and dV on its way; then S0 [half][plane][128 rows of 128 bytes]; then dS, two
    // planes, and the planes of dP'; then the outputs on their way
    static constexpr int oS = oZ + kHalves * kZHalf, kSPlane = 16384, kSHalf = 3 * kSPlane;
    static constexpr int kS = kHalves * kSHalf > 32768 + 3 * kTri ? kHalves * kSHalf : 32768 + 3 * kTri;
    static constexpr int oP = oS + kHalves * 2 * kSPlane;
    static constexpr int kBytes = oS + kS + 1024;
    static_assert(oP + 3 * kTri <= oS + kS, "reused parts");
    // the second block of key rows of S0 and dS
    static constexpr int kS2 = DP == 64 ? 0 : kSHalf, kD2 = DP == 64 ? 0 : 2 * kSPlane;
};
// accumulators
constexpr uint32_t cDQ = 0, cDX = 64, cDS = 128, cPN = 192, cN2 = 256, cPK = 320, cPQ = 384, cNK = 448;

struct GradArgs {
    la_delta in;
    DeltaGrad grad;
    DeltaWs ws;
    int chunks;
};

// (A [64 keys x 2 blocks] x rows): A's planes of `plane_a` bytes, K (value columns)
// down its rows; rows planes K-major.  Pairs of planes below NP.
template <int NA, int NB, int NP>
__device__ __forceinline__ void mma_keys(uint32_t d, uint32_t a, int half_a, int plane_a, uint32_t b,
                                         int half_b, int plane_b, int steps) {
    constexpr uint32_t id = tc::idesc_bf16(128, 64, true, false);
    const Desc da(a, half_a, 1024), db(b, 0, 1024);
    uint32_t acc = 0;
#pragma unroll
    for (int s = NP - 1; s >= 0; --s)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int i = s - j;
            if (i < 0 || i >= NA) continue;
            for (int k = 0; k < steps; ++k) {
                tc::mma_bf16(d, da.at(i * plane_a + k * 2048),
                             db.at(j * plane_b + (k >> 2) * half_b + (k & 3) * 32), id, acc);
                acc = 1;
            }
        }
}
// 128 rows x planes of Z (64 rows), K = value columns.
template <int FIRST, int LAST>
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, int half_a, uint32_t b, int half_b,
                                           int plane_b, int steps) {
    constexpr uint32_t id = tc::idesc_bf16(128, 64, false, false);
    const Desc da(a, 0, 1024), db(b, 0, 1024);
    uint32_t acc = 0;
#pragma unroll
    for (int p = LAST; p >= FIRST; --p)
        for (int k = 0; k < steps; ++k) {
            tc::mma_bf16(d, da.at((k >> 2) * half_a + (k & 3) * 32),
                         db.at(p * plane_b + (k >> 2) * half_b + (k & 3) * 32), id, acc);
            acc = 1;
        }
}
// rows^T (64 tokens down, 128 columns as two blocks) x NP planes of a lower
// triangle T: sum over tokens j of rows[j, :] T[i, j] (BY_ROW), or over i.
template <int NP, bool BY_ROW>
__device__ __forceinline__ void mma_triangle(uint32_t d, uint32_t rows, uint32_t tri, bool add) {
    const Desc a(rows, 8192, 1024), b(tri, 0, 1024);
#pragma unroll
    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int k = BY_ROW ? q : 3 - q;
            const bool first = !add && p == NP - 1 && q == 0;
            if (BY_ROW)
                tc::mma_bf16(d + 16 * k, a.at(k * 2048), b.at(p * kTri + k * 2048 + k * 32),
                             tc::idesc_bf16(128, 64 - 16 * k, true, false), !first);
            else
                tc::mma_bf16(d, a.at(k * 2048), b.at(p * kTri + k * 2048),
                             tc::idesc_bf16(128, 16 * k + 16, true, true), !first);
        }
}

// Planes of a fragment pair by pair.
template <int NP>
__device__ __forceinline__ void planes_of(uint32_t (&w)[NP][2][2][2], const Frag& x) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float a = x[h][j][2 * r], b = x[h][j][2 * r + 1];
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    // the last of two planes is rounded: cutting errs to one side
                    const uint32_t p = e == NP - 1 && NP < 3
                                           ? pack_bf16(a, b)
                                           : __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                    w[e][h][j][r] = p;
                    if (e < NP - 1) minus_halves(a, b, p);
                }
            }
}
// A fragment's plane (rows = value columns or tokens from r0 on, 16 columns from
// c0 on) into a swizzled tile with the same rows ...
__device__ __forceinline__ void put_rows(uint32_t tile, const uint32_t (&w)[2][2][2], int r0, int c0,
                                         int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = r0 + 16 * h + 8 * ((lane >> 3) & 1) + (lane & 7), c = (c0 >> 3) + (lane >> 4);
        stsm4(tile + r * 128 + (((c & 7) ^ (r & 7)) << 4), w[h][0][0], w[h][0][1], w[h][1][0],
              w[h][1][1]);
    }
}
// ... or transposed: the tile's rows are the fragment's columns.
__device__ __forceinline__ void put_cols(uint32_t tile, const uint32_t (&w)[2][2][2], int r0, int c0,
                                         int lane) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = c0 + 8 * j + (lane & 7), c = (r0 >> 3) + (lane >> 3);
        stsm4_t(tile + r * 128 + (((c & 7) ^ (r & 7)) << 4), w[0][j][0], w[0][j][1], w[1][j][0],
                w[1][j][1]);
    }
}
// Sums over the lanes that share lane % 4.
__device__ __forceinline__ float sum_rows(float x) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

template <int DP>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_tc_grad_kernel(GradArgs args) {
    using Sm = GradTc<DP>;
    constexpr int NK = DP / 4;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = tc::align1024(smem_raw);
    __shared__ uint64_t done[3];
    __shared__ uint32_t s_tmem, s_abort;
    __shared__ __align__(16) float gates[kGateRows][kChunk];
    __shared__ float s_dbeta[4][kChunk], s_vdv[4][kChunk], s_qdq[4][kChunk], s_cross[kComputeWarps];

    const la_delta& in = args.in;
    const DeltaGrad& grad = args.grad;
    const DeltaWs& ws = args.ws;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
    const int chunk = blockIdx.x % args.chunks, khead = blockIdx.x / args.chunks;
    const int b = khead / in.Hk, hk = khead % in.Hk, ratio = in.Hv / in.Hk, D = in.D;
    const int len = seq_len(in.lengths, b, in.T);
    const int t0 = chunk * kChunk, rows = in.T - t0 < kChunk ? in.T - t0 : kChunk;
    const int on = len - t0 < rows ? (len > t0 ? len - t0 : 0) : rows;   // rows of the sequence
    const size_t out_row = (size_t)khead * in.T + t0;

    if (on == 0) {                              // behind the sequence
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int rep = 0; rep < ratio; ++rep) {
            const size_t row = ((size_t)b * in.Hv + hk * ratio + rep) * in.T + t0;
            for (int i = tid; i < rows; i += kGradThreads)
                grad.dlog_alpha[row + i] = grad.dbeta[row + i] = 0.f;
            for (int i = tid; i < rows * D / 8; i += kGradThreads)
                reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(grad.dv) + row * D)[i] = zero;
        }
        for (int i = tid; i < rows * D / 8; i += kGradThreads) {
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(grad.dq) + out_row * D)[i] = zero;
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(grad.dk) + out_row * D)[i] = zero;
        }
        return;
    }

    const tc::Abort ab{&s_abort, ws.status};
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < 3; ++i) tc::mbar_init(&done[i], 1);
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(~0u, s_tmem, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);

    const int quarter = warp & 3, part = warp >> 2, g = lane >> 2, tq = lane & 3;
    const bool alive = quarter * 32 < D;        // as value columns and as key rows
    const int v0 = quarter * 32, k0 = part * NK, tok = part * 16;
    const uint32_t at = tc::tmem_addr(tm, quarter * 32, 0);
    // a warp's rows on their way out: 16 tokens x 32 columns
    unsigned char* buf = smem + Sm::oS + 16384 + warp * 1024;
    auto put_out = [&](__nv_bfloat16* out, const Frag& x) {     // [rows, D]
        uint32_t w[2][2][2];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k >> 2][(k >> 1) & 1][k & 1] = pack_bf16(x[k >> 2][(k >> 1) & 1][2 * (k & 1)],
                                                       x[k >> 2][(k >> 1) & 1][2 * (k & 1) + 1]);
        __syncwarp();
        stage_rows(smem_u32(buf), w, lane);
        __syncwarp();
        const int col = v0 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = tok + (lane >> 2) + 8 * i;
            if (col < D && t < rows) {
                const uint4 y = staged_row(buf, i, lane);
                *reinterpret_cast<uint4*>(out + (size_t)t * D + col) =
                    t < on ? y : make_uint4(0, 0, 0, 0);
            }
        }
    };
    auto load64 = [&](uint32_t dst, int half, const void* src, long long offset, long long stride) {
        // 64 rows by the first eight warps, eight rows each
        if (warp < 8)
            load_tile<8>(dst + warp * 1024, half,
                         static_cast<const __nv_bfloat16*>(src) + offset +
                             (on > 8 * warp ? t0 + 8 * warp : t0) * stride,
                         stride, on - 8 * warp, D, lane);
    };
    Frag dq, dk;
    each([&](int a, int j, int e) { dq[a][j][e] = dk[a][j][e] = 0.f; });

    for (int rep = 0; rep < ratio; ++rep) {
        const int h = hk * ratio + rep, head = b * in.Hv + h, ph = rep & 1;
        const size_t row = (size_t)head * in.T + t0;
        __syncthreads();                        // the last head's tiles have been read
        load64(base + Sm::oX, Sm::kXHalf, grad.d_o, row3(grad.do_stride).at(b, h, 0),
               grad.do_stride[2]);
        load64(base + Sm::oS, 8192, in.v, row3(in.v_stride).at(b, h, 0), in.v_stride[2]);
        cp_commit();
        for (int i = tid; i < kGateRows * kChunk; i += kGradThreads)
            (&gates[0][0])[i] = ws.gates(head, chunk)[i];
        Frag x, z;
        if (alive) {
            fetch_frag(z, ws.Z_frags(head, chunk), 4, 0, warp, lane);
            fetch_frag(x, ws.dX_frags(head, chunk), 4, 0, warp, lane);
            {
                uint32_t w[3][2][2][2];
                planes_of<3>(w, z);
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    put_cols(base + Sm::oZ + (v0 >> 6) * Sm::kZHalf + e * 8192, w[e], v0 & 63, tok, lane);
            }
            uint32_t w[2][2][2][2];
            planes_of<2>(w, x);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                put_cols(base + Sm::oX + (v0 >> 6) * Sm::kXHalf + (1 + e) * 8192, w[e], v0 & 63, tok,
                         lane);
        }
        cp_wait<0>();
        tc::fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && tc::elect_one()) {
            // lanes 0 .. 63: dO Z^T; 64 .. 127: dX Z^T, whose second planes' part comes apart
            mma_tokens<0, 2>(tm + cPN, base + Sm::oX, Sm::kXHalf, base + Sm::oZ, Sm::kZHalf, 8192,
                             D / 16);
            mma_tokens<0, 0>(tm + cN2, base + Sm::oX + 8192, Sm::kXHalf, base + Sm::oZ, Sm::kZHalf,
                             8192, D / 16);
            tc::mma_commit(&done[0]);
        }
        __syncwarp();

        // dV = B dX, dbeta = dX . Z, v . dV
        {
            float xz[2][2] = {}, xv[2][2] = {};
            if (alive) {
                Frag v;
                load_rows_frag(v, base + Sm::oS, 8192, tok, v0, lane);
                Factors be;
                factors(be, gates[2] + tok, tq);
                each([&](int a, int j, int e) {
                    const bool live = v0 + 16 * a < D;
                    xz[j][e & 1] += live ? x[a][j][e] * z[a][j][e] : 0.f;
                    x[a][j][e] *= factor(be, j, e);
                    xv[j][e & 1] += live ? x[a][j][e] * v[a][j][e] : 0.f;
                });
                put_out(static_cast<__nv_bfloat16*>(grad.dv) + row * D, x);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a = sum_rows(xz[j][e]), c = sum_rows(xv[j][e]);
                    if (g == 0) {
                        s_dbeta[quarter][tok + 8 * j + 2 * tq + e] = a;
                        s_vdv[quarter][tok + 8 * j + 2 * tq + e] = c;
                    }
                }
        }
        Frag S[NK / 16];
        if (alive)
#pragma unroll
            for (int i = 0; i < NK / 16; ++i)
                fetch_frag(S[i], ws.state_frags(head, chunk), NK / 4, i, warp, lane);
        __syncthreads();                        // V has been read, dV has left
        if (alive)
#pragma unroll
            for (int i = 0; i < NK / 16; ++i) {
                const int key = k0 + 16 * i;
                uint32_t w[3][2][2][2];
                planes_of<3>(w, S[i]);
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    put_rows(base + Sm::oS + (key >> 6) * Sm::kSHalf + e * Sm::kSPlane, w[e], v0,
                             key & 63, lane);
            }
        tc::fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && tc::elect_one()) {
            mma_keys<3, 1, 3>(tm + cDQ, base + Sm::oS, Sm::kS2, Sm::kSPlane, base + Sm::oX,
                              Sm::kXHalf, 8192, D / 16);
            mma_keys<2, 2, 2>(tm + cDX, base + Sm::oS, Sm::kS2, Sm::kSPlane, base + Sm::oX + 8192,
                              Sm::kXHalf, 8192, D / 16);
            tc::mma_commit(&done[1]);
        }
        __syncwarp();

        // <dS, S> with the state after the chunk
        float cross = 0.f;
        if (alive)
#pragma unroll
            for (int i = 0; i < NK / 16; ++i) {
                fetch_frag(S[i], ws.dstate_frags(head, chunk), NK / 4, i, warp, lane);
                Frag y;
                fetch_frag(y, ws.state_frags(head, chunk + 1), NK / 4, i, warp, lane);
                each([&](int a, int j, int e) {
                    const bool live = v0 + 16 * a < D && k0 + 16 * i < D;
                    cross += live ? S[i][a][j][e] * y[a][j][e] : 0.f;
                });
            }
#pragma unroll
        for (int d = 16; d; d >>= 1) cross += __shfl_xor_sync(~0u, cross, d);
        if (lane == 0) s_cross[warp] = cross;

        // dP' = dP o E and N' as operand planes, once S0 and dX have been read
        tc::mbar_wait(&done[0], ph, ab, 1);
        tc::tc_fence_after();
        Frag p;
        load_frag(p, at + cPN + tok);
        if (quarter >= 2) load_frag(x, at + cN2 + tok);
        tc::tmem_wait_ld();
        const int i0 = (quarter & 1) * 32;      // rows i0 .. i0 + 31, columns tok .. tok + 15
        each([&](int a, int j, int e) {
            if (tok > i0 + 16 * a) return;      // above the diagonal: not read
            const int ti = i0 + 16 * a + 8 * (e >> 1) + g, tj = tok + 8 * j + 2 * tq + (e & 1);
            // above the diagonal E may overflow: it is selected away
            const float E = expf((gates[3][ti] - gates[3][tj]) + (gates[4][ti] - gates[4][tj])) *
                            gates[2][tj];
            if (quarter < 2) p[a][j][e] = ti >= tj ? E * p[a][j][e] : 0.f;
            else p[a][j][e] = ti > tj ? -gates[2][ti] * E * (p[a][j][e] + x[a][j][e]) : 0.f;
        });
        tc::mbar_wait(&done[1], ph, ab, 2);
        tc::tc_fence_after();
        load64(base + Sm::oK, 8192, in.k, row3(in.k_stride).at(b, hk, 0), in.k_stride[2]);
        load64(base + Sm::oQ, 8192, in.q, row3(in.q_stride).at(b, hk, 0), in.q_stride[2]);
        cp_commit();
        if (quarter < 2) {
            uint32_t w[3][2][2][2];
            planes_of<3>(w, p);
#pragma unroll
            for (int e = 0; e < 3; ++e) put_rows(base + Sm::oP + e * kTri, w[e], i0, tok, lane);
        } else {
            uint32_t w[2][2][2][2];
            planes_of<2>(w, p);
#pragma unroll
            for (int e = 0; e < 2; ++e) put_rows(base + Sm::oN + e * kTri, w[e], i0, tok, lane);
        }
        if (alive)
#pragma unroll
            for (int i = 0; i < NK / 16; ++i) {
                const int key = k0 + 16 * i;
                uint32_t w[2][2][2][2];
                planes_of<2>(w, S[i]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    put_rows(base + Sm::oS + (key >> 6) * 2 * Sm::kSPlane + e * Sm::kSPlane, w[e], v0,
                             key & 63, lane);
            }
        cp_wait<0>();
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncthreads();
        if (warp == 0 && tc::elect_one()) {
            tc::tc_fence_after();
            mma_triangle<3, true>(tm + cPK, base + Sm::oK, base + Sm::oP, false);
            mma_triangle<2, false>(tm + cPQ, base + Sm::oQ, base + Sm::oP, false);
            mma_triangle<2, true>(tm + cNK, base + Sm::oK, base + Sm::oN, false);
            mma_triangle<2, false>(tm + cNK, base + Sm::oK, base + Sm::oN, true);
            mma_keys<2, 2, 2>(tm + cDS, base + Sm::oS, Sm::kD2, Sm::kSPlane, base + Sm::oZ,
                              Sm::kZHalf, 8192, D / 16);
            tc::mma_commit(&done[2]);
        }
        __syncwarp();
        Factors ga, ta, be;
        factors(ga, gates[0] + tok, tq);
        factors(ta, gates[1] + tok, tq);
        factors(be, gates[2] + tok, tq);
        tc::mbar_wait(&done[2], ph, ab, 3);
        tc::tc_fence_after();
        float qdq[2][2] = {};
        if (alive) {
            Frag y;
            load_frag(x, at + cDQ + tok);
            load_frag(y, at + cPK + tok);
            load_rows_frag(z, base + Sm::oQ, 8192, tok, v0, lane);
            tc::tmem_wait_ld();
            each([&](int a, int j, int e) {
                x[a][j][e] = factor(ga, j, e) * x[a][j][e] + in.k_scale * y[a][j][e];
                dq[a][j][e] += x[a][j][e];
                if (v0 + 16 * a < D) qdq[j][e & 1] += z[a][j][e] * x[a][j][e];
            });
            load_frag(x, at + cDX + tok);
            load_frag(y, at + cDS + tok);
            tc::tmem_wait_ld();
            each([&](int a, int j, int e) {
                dk[a][j][e] += factor(be, j, e) * (factor(ta, j, e) * y[a][j][e] -
                                                   factor(ga, j, e) * x[a][j][e]);
            });
            load_frag(x, at + cPQ + tok);
            load_frag(y, at + cNK + tok);
            tc::tmem_wait_ld();
            each([&](int a, int j, int e) {
                dk[a][j][e] += in.q_scale * x[a][j][e] + in.k_scale * y[a][j][e];
            });
        }
        tc::tc_fence_before();                  // read before the next head's products
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float s = sum_rows(qdq[j][e]);
                if (g == 0) s_qdq[quarter][tok + 8 * j + 2 * tq + e] = in.q_scale * s;
            }
        __syncthreads();
        tc::tc_fence_after();
        if (warp == 0) {                        // dG, summed from the chunk's end
            double s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                s[i] = ((double)s_qdq[0][t] + (double)s_qdq[1][t]) +
                       ((double)s_qdq[2][t] + (double)s_qdq[3][t]) -
                       (((double)s_vdv[0][t] + (double)s_vdv[1][t]) +
                        ((double)s_vdv[2][t] + (double)s_vdv[3][t]));
            }
            if (lane == 31)
                for (int i = 0; i < kComputeWarps; ++i) s[1] += (double)s_cross[i];
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
                // below kLogAlphaMin the state before the token is forgotten
                const bool kept = t < on && !(in.log_alpha[row + t] < kLogAlphaMin);
                grad.dlog_alpha[row + t] = kept ? (float)sum[i] : 0.f;
                grad.dbeta[row + t] = t < on ? (s_dbeta[0][t] + s_dbeta[1][t]) +
                                                   (s_dbeta[2][t] + s_dbeta[3][t]) : 0.f;
            }
        }
    }
    if (alive) {
        each([&](int a, int j, int e) {
            dq[a][j][e] *= in.q_scale;
            dk[a][j][e] *= in.k_scale;
        });
        put_out(static_cast<__nv_bfloat16*>(grad.dq) + out_row * D, dq);
        put_out(static_cast<__nv_bfloat16*>(grad.dk) + out_row * D, dk);
    }
    if (warp == 0 && tc::elect_one() && tc::aborted(ab))
        for (int i = 0; i < 3; ++i) tc::mbar_drain(&done[i], (ratio - 1) & 1);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

template <int DP>
cudaError_t gradients(const GradArgs& a, cudaStream_t st) {
    auto* kernel = delta_tc_grad_kernel<DP>;
    constexpr int bytes = GradTc<DP>::kBytes;
    static_assert(bytes <= 225 * 1024 + 512, "shared memory of a block");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(a.in.B * a.in.Hk) * (unsigned)a.chunks, kGradThreads, bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tc_grad(const la_delta& in, const DeltaGrad& g, const DeltaWs& ws,
                                 cudaStream_t st) {
    const GradArgs a{in, g, ws, ws.chunks};
    return in.D <= 64 ? gradients<64>(a, st) : gradients<128>(a, st);
}

}  // namespace la
