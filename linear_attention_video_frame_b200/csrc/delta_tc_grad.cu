// The gradients of all chunks on tcgen05 (bf16 inputs), from the states S0, Z, dS
// and dX that the two chains left; the formulas are in delta_grad.cu.
//
// A block takes one chunk of one value head.  Where value heads share a key head,
// dq and dk leave in float32 and delta_share_kernel adds them up in their order.
// The warps hold fragments as the chains did.  Products, transposed where they
// are of key rows:
//   rows (dO | dX) Z^T     [tokens, 2 x 64 lanes] x [64 tokens]
//   S0 dO^T, S0 dX^T, dS Z^T, K^T dP', Q^T dP'^T, K^T (N' + N'^T)   [128 key rows] x [64 tokens]
// in bf16 planes: three where dlog_alpha (float32) depends on them, two for what
// only reaches the bf16 dk.
#include "delta_tc.cuh"

namespace la {
namespace {
using namespace dtc;

constexpr int kGradWarps = 8, kGradThreads = kGradWarps * 32;

// Value columns go 64 at a time, so that two blocks fit an SM: a block is a
// sequence of loads, conversions and products that wait for one another, and the
// second block fills its waits (one block of 16 warps with all columns at once:
// 317 us for 2048 chunks of 128, most of it waiting; as it is 212, DRAM at 36 % of its
// peak).
template <int DP>
struct GradTc {
    static constexpr int kHalves = DP / 64;                 // of the key rows
    static constexpr int kRows = kHalves * 8192;            // 64 rows of DP columns
    // dO | first plane of dX | zeros | second plane of dX, 64 tokens each
    static constexpr int oX = 0, oDX0 = 8192, oZero = 16384, oDX1 = 24576;
    static constexpr int oZ = 32768;                        // three planes
    // V, and dV on its way; then S0 [half][plane][64 rows of 128 bytes]; then dS, two planes
    static constexpr int oS = oZ + 3 * 8192, oOut = oS + 8192;
    // at the end, over Z and S: K | Q | two planes of N' | three of dP'
    static constexpr int oK = oZ, oQ = oK + kRows, oN = oQ + kRows, oP = oN + 2 * kTri,
                         oEnd = oP + 3 * kTri;
    static constexpr int kEnd = oS + kHalves * 3 * 8192 > oEnd ? oS + kHalves * 3 * 8192 : oEnd;
    static constexpr int kBytes = kEnd + 1024;
    // distance of the second 64 key rows; with DP = 64 lanes that nobody looks at
    // read the first once more
    static constexpr int kS2 = DP == 64 ? 0 : 3 * 8192, kD2 = DP == 64 ? 0 : 2 * 8192;
};
// accumulators; the first, third and fourth are used twice
constexpr uint32_t cPN = 0, cDQ = 64, cDX = 128, cDS = 192;
constexpr uint32_t cPK = cPN, cPQ = cDX, cNK = cDS, kGradCols = 256;

struct GradArgs {
    la_delta in;
    DeltaGrad grad;
    DeltaWs ws;
    int chunks;
};

// One plane each of A [64 rows down K x 128 keys] and rows [64 tokens x 64 of K].
__device__ __forceinline__ void mma_keys(uint32_t d, uint32_t a, int half_a, uint32_t b, bool add) {
    const Desc da(a, half_a, 1024), db(b, 0, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        tc::mma_bf16(d, da.at(k * 2048), db.at(k * 32), tc::idesc_bf16(128, 64, true, false),
                     add || k > 0);
}
// One plane each of A [128 rows x 64 of K] and rows [64 tokens x 64 of K].
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t b, bool add) {
    const Desc da(a, 0, 1024), db(b, 0, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        tc::mma_bf16(d, da.at(k * 32), db.at(k * 32), tc::idesc_bf16(128, 64, false, false),
                     add || k > 0);
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

// Sums over the lanes that share lane % 4.
__device__ __forceinline__ float sum_rows(float x) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

// SHARED: several value heads share a key head.
template <int DP, bool SHARED>
__global__ void __launch_bounds__(kGradThreads, 2)
delta_tc_grad_kernel(GradArgs args) {
    using Sm = GradTc<DP>;
    constexpr int NK = DP / 4;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = tc::align1024(smem_raw);
    __shared__ uint64_t done[2], done_all;
    __shared__ uint32_t s_tmem, s_abort;
    __shared__ __align__(16) float gates[kGateRows][kChunk];
    __shared__ float s_dbeta[2][kChunk], s_vdv[2][kChunk], s_qdq[4][kChunk], s_cross[kGradWarps];

    const la_delta& in = args.in;
    const DeltaGrad& grad = args.grad;
    const DeltaWs& ws = args.ws;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
    const int chunk = blockIdx.x % args.chunks, head = blockIdx.x / args.chunks;
    const int b = head / in.Hv, h = head % in.Hv, hk = SHARED ? h / (in.Hv / in.Hk) : h, D = in.D;
    const int len = seq_len(in.lengths, b, in.T);
    const int t0 = chunk * kChunk, rows = in.T - t0 < kChunk ? in.T - t0 : kChunk;
    const int on = len - t0 < rows ? (len > t0 ? len - t0 : 0) : rows;   // rows of the sequence
    const size_t row = (size_t)head * in.T + t0;

    if (on == 0) {                              // behind the sequence
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < rows; i += kGradThreads)
            grad.dlog_alpha[row + i] = grad.dbeta[row + i] = 0.f;
        for (int i = tid; i < rows * D / 8; i += kGradThreads) {
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(grad.dv) + row * D)[i] = zero;
            if (SHARED) continue;               // delta_share_kernel's
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(grad.dq) + row * D)[i] = zero;
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(grad.dk) + row * D)[i] = zero;
        }
        return;
    }
    // What is read later, towards the L2: the reads follow one another.
    {
        const void* from[3] = {ws.state_frags(head, chunk), ws.dstate_frags(head, chunk),
                               ws.state_frags(head, chunk + 1)};
        const int each_bytes = (int)ws.state_frag_bytes() / kGradWarps;
        const int warp_at = (tid >> 5) * each_bytes;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            prefetch_lines(static_cast<const char*>(from[i]) + warp_at, each_bytes, tid & 31);
    }

    const tc::Abort ab{&s_abort, ws.status};
    if (tid == 0) {
        s_abort = 0;
        for (uint64_t* bar : {&done[0], &done[1], &done_all}) tc::mbar_init(bar, 1);
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(&s_tmem, kGradCols);
        tc::tmem_relinquish();
    }
    for (int i = tid; i < 8192 / 16; i += kGradThreads)
        reinterpret_cast<uint4*>(smem + Sm::oZero)[i] = make_uint4(0, 0, 0, 0);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = __shfl_sync(~0u, s_tmem, 0), base = __shfl_sync(~0u, smem_u32(smem), 0);
    uint32_t phase[2] = {0, 0};
    auto wait = [&](int i) {
        tc::mbar_wait(&done[i], phase[i], ab, 1 + i);
        phase[i] ^= 1;
        tc::tc_fence_after();
    };

    const int g = lane >> 2, tq = lane & 3;
    // As a reader of accumulators: lanes 32 quarter .., columns 32 pair .. .
    const int quarter = warp & 3, pair = warp >> 2;
    const bool alive = quarter * 32 < D;        // as key rows
    const uint32_t at = tc::tmem_addr(tm, quarter * 32, 0);
    // As a reader of the chains' fragments: of 64 value columns its side, its tokens
    // and key rows.
    const int side = warp & 1, part = warp >> 1, tok = part * 16, k0 = part * NK;

    auto put_out = [&](unsigned char* buf, __nv_bfloat16* out, const Frag& x, int col0, int first) {
        uint32_t w[2][2][2];                    // rows of [rows, D]: 16 from `first`, 32 columns
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k >> 2][(k >> 1) & 1][k & 1] = pack_bf16(x[k >> 2][(k >> 1) & 1][2 * (k & 1)],
                                                       x[k >> 2][(k >> 1) & 1][2 * (k & 1) + 1]);
        __syncwarp();
        stage_rows(smem_u32(buf), w, lane);
        __syncwarp();
        const int col = col0 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = first + (lane >> 2) + 8 * i;
            if (col < D && t < rows) {
                const uint4 y = staged_row(buf, i, lane);
                *reinterpret_cast<uint4*>(out + (size_t)t * D + col) =
                    t < on ? y : make_uint4(0, 0, 0, 0);
            }
        }
    };
    // 64 rows x 64 columns from column `col` on, as a swizzled tile
    auto load64 = [&](uint32_t dst, const void* src, long long offset, long long stride, int col) {
        const int c = tid & 7;
        if (col + c * 8 >= D) return;
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(src) + offset +
                                 (long long)t0 * stride + col + c * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (tid >> 3) + 32 * i;
            cp16(dst + r * 128 + ((c ^ (r & 7)) << 4), r < on ? p + r * stride : p, r < on);
        }
    };

    for (int i = tid; i < kGateRows * kChunk; i += kGradThreads)
        (&gates[0][0])[i] = ws.gates(head, chunk)[i];
    {
        float xz[2][2] = {}, xv[2][2] = {}, cross = 0.f;

#pragma unroll 1
        for (int vh = 0; vh * 64 < D; ++vh) {
            const int v0 = vh * 64 + side * 32, cw = part * 4 + vh * 2 + side;   // the chains' warp
            const bool live = v0 < D;
            if (vh > 0) {
                wait(0);                        // the products before: all tiles are free
                __syncthreads();
            }
            load64(base + Sm::oX, grad.d_o, row3(grad.do_stride).at(b, h, 0), grad.do_stride[2],
                   vh * 64);
            load64(base + Sm::oS, in.v, row3(in.v_stride).at(b, h, 0), in.v_stride[2], vh * 64);
            cp_commit();
            Frag x, z;
            Frag S[NK / 16];
            if (live) {
                fetch_frag(z, ws.Z_frags(head, chunk), 4, 0, cw, lane);
                fetch_frag(x, ws.dX_frags(head, chunk), 4, 0, cw, lane);
#pragma unroll
                for (int i = 0; i < NK / 16; ++i)
                    fetch_frag(S[i], ws.state_frags(head, chunk), NK / 4, i, cw, lane);
                {
                    uint32_t w[3][2][2][2];
                    planes_of<3>(w, z);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        put_cols(base + Sm::oZ + e * 8192, w[e], side * 32, tok, lane);
                }
                uint32_t w[2][2][2][2];
                planes_of<2>(w, x);
                put_cols(base + Sm::oDX0, w[0], side * 32, tok, lane);
                put_cols(base + Sm::oDX1, w[1], side * 32, tok, lane);
            }
            cp_wait<0>();
            tc::fence_proxy_async_smem();
            __syncthreads();
            const int steps = D - vh * 64;      // value columns behind D are not there
            if (warp == 0 && tc::elect_one()) {
                // lanes 0 .. 63: dO Z^T; 64 .. 127: dX Z^T
                if (steps < 64) {
                    for (int k = 0; k * 16 < steps; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {       // pairs as below
                            const Desc da(base + (e == 2 ? Sm::oZero : Sm::oX), 0, 1024);
                            const Desc db(base + Sm::oZ + (e == 0 ? 16384 : e == 1 ? 8192 : 0), 0, 1024);
                            tc::mma_bf16(tm + cPN, da.at(k * 32), db.at(k * 32),
                                         tc::idesc_bf16(128, 64, false, false),
                                         vh > 0 || k > 0 || e > 0);
                        }
                } else {
                    mma_tokens(tm + cPN, base + Sm::oX, base + Sm::oZ + 16384, vh > 0);
                    mma_tokens(tm + cPN, base + Sm::oX, base + Sm::oZ + 8192, true);
                    mma_tokens(tm + cPN, base + Sm::oZero, base + Sm::oZ, true);
                    mma_tokens(tm + cPN, base + Sm::oX, base + Sm::oZ, true);
                }
            }
            __syncwarp();

            // dV = B dX, dbeta = dX . Z, v . dV
            if (live) {
                Frag v;
                load_rows_frag(v, base + Sm::oS, 0, tok, side * 32, lane);
                Factors be;
                factors(be, gates[2] + tok, tq);
                each([&](int a, int j, int e) {
                    const bool there = v0 + 16 * a < D;
                    xz[j][e & 1] += there ? x[a][j][e] * z[a][j][e] : 0.f;
                    x[a][j][e] *= factor(be, j, e);
                    xv[j][e & 1] += there ? x[a][j][e] * v[a][j][e] : 0.f;
                });
                put_out(smem + Sm::oOut + warp * 1024, static_cast<__nv_bfloat16*>(grad.dv) + row * D,
                        x, v0, tok);
            }
            __syncthreads();                    // V has been read, dV has left
            if (live)
#pragma unroll
                for (int i = 0; i < NK / 16; ++i) {
                    const int key = k0 + 16 * i;
                    uint32_t w[3][2][2][2];
                    planes_of<3>(w, S[i]);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        put_rows(base + Sm::oS + (key >> 6) * 3 * 8192 + e * 8192, w[e], side * 32,
                                 key & 63, lane);
                }
            tc::fence_proxy_async_smem();
            __syncthreads();
            // products with the rows of 64 value columns (or what there is) as K
            auto keys = [&](uint32_t d, uint32_t a, int half, uint32_t b_, bool add) {
                if (steps >= 64) {
                    mma_keys(d, a, half, b_, add);
                } else {
                    const Desc da(a, half, 1024), db(b_, 0, 1024);
                    for (int k = 0; k * 16 < steps; ++k)
                        tc::mma_bf16(d, da.at(k * 2048), db.at(k * 32),
                                     tc::idesc_bf16(128, 64, true, false), add || k > 0);
                }
            };
            if (warp == 0 && tc::elect_one()) {
#pragma unroll
                for (int e = 2; e >= 0; --e)
                    keys(tm + cDQ, base + Sm::oS + e * 8192, Sm::kS2, base + Sm::oX, vh > 0 || e < 2);
                keys(tm + cDX, base + Sm::oS + 8192, Sm::kS2, base + Sm::oDX0, vh > 0);
                keys(tm + cDX, base + Sm::oS, Sm::kS2, base + Sm::oDX1, true);
                keys(tm + cDX, base + Sm::oS, Sm::kS2, base + Sm::oDX0, true);
                tc::mma_commit(&done[1]);
            }
            __syncwarp();

            // <dS, S> with the state after the chunk
            if (live)
#pragma unroll
                for (int i = 0; i < NK / 16; ++i) {
                    Frag y;
                    fetch_frag(S[i], ws.dstate_frags(head, chunk), NK / 4, i, cw, lane);
                    fetch_frag(y, ws.state_frags(head, chunk + 1), NK / 4, i, cw, lane);
                    each([&](int a, int j, int e) {
                        const bool there = v0 + 16 * a < D && k0 + 16 * i < D;
                        cross += there ? S[i][a][j][e] * y[a][j][e] : 0.f;
                    });
                }
            wait(1);                            // S0 has been read
            if (live)
#pragma unroll
                for (int i = 0; i < NK / 16; ++i) {
                    const int key = k0 + 16 * i;
                    uint32_t w[2][2][2][2];
                    planes_of<2>(w, S[i]);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        put_rows(base + Sm::oS + (key >> 6) * 2 * 8192 + e * 8192, w[e], side * 32,
                                 key & 63, lane);
                }
            tc::fence_proxy_async_smem();
            __syncthreads();
            if (warp == 0 && tc::elect_one()) {
                keys(tm + cDS, base + Sm::oS + 8192, Sm::kD2, base + Sm::oZ, vh > 0);
                keys(tm + cDS, base + Sm::oS, Sm::kD2, base + Sm::oZ + 8192, true);
                keys(tm + cDS, base + Sm::oS, Sm::kD2, base + Sm::oZ, true);
                tc::mma_commit(&done[0]);
            }
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float a = sum_rows(xz[j][e]), c = sum_rows(xv[j][e]);
                if (g == 0) {
                    s_dbeta[side][tok + 8 * j + 2 * tq + e] = a;
                    s_vdv[side][tok + 8 * j + 2 * tq + e] = c;
                }
            }
#pragma unroll
        for (int d = 16; d; d >>= 1) cross += __shfl_xor_sync(~0u, cross, d);
        if (lane == 0) s_cross[warp] = cross;

        wait(0);
        __syncthreads();                        // every warp is past its waits: Z and S are free
#pragma unroll
        for (int half = 0; half < Sm::kHalves; ++half) {
            load64(base + Sm::oK + half * 8192, in.k, row3(in.k_stride).at(b, hk, 0), in.k_stride[2],
                   half * 64);
            load64(base + Sm::oQ + half * 8192, in.q, row3(in.q_stride).at(b, hk, 0), in.q_stride[2],
                   half * 64);
        }
        cp_commit();
        // dP' = dP o E and N' as operand planes
        const int i0 = (quarter & 1) * 32;      // rows i0 .. i0 + 31
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j0 = pair * 32 + i * 16;  // columns j0 .. j0 + 15
            Frag p;
            load_frag(p, at + cPN + j0);
            tc::tmem_wait_ld();
            each([&](int a, int j, int e) {
                if (j0 > i0 + 16 * a) return;   // above the diagonal: not read
                const int ti = i0 + 16 * a + 8 * (e >> 1) + g, tj = j0 + 8 * j + 2 * tq + (e & 1);
                // above the diagonal E may overflow: it is selected away
                const float E = exp2_sum(gates[3][ti], gates[4][ti], gates[3][tj], gates[4][tj]) *
                                gates[2][tj];
                if (quarter < 2) p[a][j][e] = ti >= tj ? E * p[a][j][e] : 0.f;
                else p[a][j][e] = ti > tj ? -gates[2][ti] * E * p[a][j][e] : 0.f;
            });
            if (quarter < 2) {
                uint32_t w[3][2][2][2];
                planes_of<3>(w, p);
#pragma unroll
                for (int e = 0; e < 3; ++e) put_rows(base + Sm::oP + e * kTri, w[e], i0, j0, lane);
            } else {
                uint32_t w[2][2][2][2];
                planes_of<2>(w, p);
#pragma unroll
                for (int e = 0; e < 2; ++e) put_rows(base + Sm::oN + e * kTri, w[e], i0, j0, lane);
            }
        }
        Frag dk[2];
        if (alive)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j0 = pair * 32 + i * 16;
                Frag x, y;
                Factors ga, ta, be;
                factors(ga, gates[0] + j0, tq);
                factors(ta, gates[1] + j0, tq);
                factors(be, gates[2] + j0, tq);
                load_frag(x, at + cDX + j0);
                load_frag(y, at + cDS + j0);
                tc::tmem_wait_ld();
                each([&](int a, int j, int e) {
                    dk[i][a][j][e] = factor(be, j, e) * (factor(ta, j, e) * y[a][j][e] -
                                                         factor(ga, j, e) * x[a][j][e]);
                });
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
            tc::mma_commit(&done[0]);
        }
        __syncwarp();
        wait(0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j0 = pair * 32 + i * 16;
            float qdq[2][2] = {};
            if (alive) {
                Frag x, y, q;
                Factors ga;
                factors(ga, gates[0] + j0, tq);
                load_frag(x, at + cDQ + j0);
                load_frag(y, at + cPK + j0);
                load_rows_frag(q, base + Sm::oQ, 8192, j0, quarter * 32, lane);
                tc::tmem_wait_ld();
                each([&](int a, int j, int e) {
                    x[a][j][e] = factor(ga, j, e) * x[a][j][e] + in.k_scale * y[a][j][e];
                    if (quarter * 32 + 16 * a < D) qdq[j][e & 1] += q[a][j][e] * x[a][j][e];
                });
                Frag z;
                load_frag(z, at + cPQ + j0);
                load_frag(y, at + cNK + j0);
                tc::tmem_wait_ld();
                each([&](int a, int j, int e) {
                    x[a][j][e] *= in.q_scale;
                    z[a][j][e] = in.k_scale * (dk[i][a][j][e] + in.q_scale * z[a][j][e] +
                                               in.k_scale * y[a][j][e]);
                });
                if (SHARED) {
                    float* pq = ws.dq_shares + row * D;
                    float* pk = ws.dk_shares + row * D;
                    each([&](int a, int j, int e) {
                        const int t = j0 + 8 * j + 2 * tq + (e & 1);
                        const int key = quarter * 32 + 16 * a + 8 * (e >> 1) + g;
                        if (t < on && key < D) {
                            pq[(size_t)t * D + key] = x[a][j][e];
                            pk[(size_t)t * D + key] = z[a][j][e];
                        }
                    });
                } else {
                    unsigned char* buf = smem + warp * 1024;
                    put_out(buf, static_cast<__nv_bfloat16*>(grad.dq) + row * D, x, quarter * 32, j0);
                    put_out(buf, static_cast<__nv_bfloat16*>(grad.dk) + row * D, z, quarter * 32, j0);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float s = sum_rows(qdq[j][e]);
                    if (g == 0) s_qdq[quarter][j0 + 8 * j + 2 * tq + e] = in.q_scale * s;
                }
        }
        __syncthreads();
        if (warp == 0) {                        // dG, summed from the chunk's end
            double s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                s[i] = ((double)s_qdq[0][t] + (double)s_qdq[1][t]) +
                       ((double)s_qdq[2][t] + (double)s_qdq[3][t]) -
                       ((double)s_vdv[0][t] + (double)s_vdv[1][t]);
            }
            if (lane == 31)
                for (int i = 0; i < kGradWarps; ++i) s[1] += (double)s_cross[i];
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
                                  !(in.log_alpha[row + t] <= kForgets);
                grad.dlog_alpha[row + t] = kept ? (float)sum[i] : 0.f;
                grad.dbeta[row + t] = t < on ? s_dbeta[0][t] + s_dbeta[1][t] : 0.f;
            }
        }
    }
    if (warp == 0 && tc::elect_one() && tc::aborted(ab)) {
        tc::mma_commit(&done_all);              // nothing in flight when the memory is freed
        tc::mbar_drain(&done_all, 0);
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tm, kGradCols);
    }
}

// dq and dk of the key heads: the sums of their value heads', four columns a thread.
__global__ void __launch_bounds__(256)
delta_share_kernel(GradArgs args) {
    const la_delta& in = args.in;
    const int D = in.D, ratio = in.Hv / in.Hk;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, row = i / (D / 4);
    const int c = (int)(i % (D / 4)) * 4;
    const long long khead = row / in.T;
    const int t = (int)(row % in.T), b = (int)(khead / in.Hk), hk = (int)(khead % in.Hk);
    if (b >= in.B) return;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f), k = q;
    if (t < seq_len(in.lengths, b, in.T))
        for (int r = 0; r < ratio; ++r) {
            const size_t at =
                (((size_t)b * in.Hv + hk * ratio + r) * in.T + t) * D + c;
            const float4 x = *reinterpret_cast<const float4*>(args.ws.dq_shares + at);
            const float4 y = *reinterpret_cast<const float4*>(args.ws.dk_shares + at);
            q.x += x.x; q.y += x.y; q.z += x.z; q.w += x.w;
            k.x += y.x; k.y += y.y; k.z += y.z; k.w += y.w;
        }
    const size_t out = (size_t)row * D + c;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(args.grad.dq) + out) =
        make_uint2(pack_bf16(q.x, q.y), pack_bf16(q.z, q.w));
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(args.grad.dk) + out) =
        make_uint2(pack_bf16(k.x, k.y), pack_bf16(k.z, k.w));
}

template <int DP, bool SHARED>
cudaError_t gradients(const GradArgs& a, cudaStream_t st) {
    auto* kernel = delta_tc_grad_kernel<DP, SHARED>;
    constexpr int bytes = GradTc<DP>::kBytes;
    static_assert(bytes <= 108 * 1024, "shared memory of two blocks");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(a.in.B * a.in.Hv) * (unsigned)a.chunks, kGradThreads, bytes, st>>>(a);
    if (!SHARED || (e = cudaGetLastError()) != cudaSuccess) return SHARED ? e : cudaGetLastError();
    const long long units = (long long)a.in.B * a.in.Hk * a.in.T * (a.in.D / 4);
    delta_share_kernel<<<(unsigned)((units + 255) / 256), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tc_grad(const la_delta& in, const DeltaGrad& g, const DeltaWs& ws,
                                 cudaStream_t st) {
    const GradArgs a{in, g, ws, ws.chunks};
    if (in.Hv == in.Hk) return in.D <= 64 ? gradients<64, false>(a, st) : gradients<128, false>(a, st);
    return in.D <= 64 ? gradients<64, true>(a, st) : gradients<128, true>(a, st);
}

}  // namespace la
