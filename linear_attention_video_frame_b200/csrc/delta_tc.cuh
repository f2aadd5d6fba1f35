// Shared parts of the tcgen05 kernels of the chunked gated delta rule (bf16
// inputs): the roles of a block, operand planes and their products.
//
// Everything is computed transposed, as in the warp-level kernels: lane v of
// tensor memory holds value column v of the state, whose row S^T[v, :] is the
// A operand of (K S)^T = S^T K^T; the results, scaled and split, are the A
// operands of the products with Kt and Pt (delta_tc_prep.cu).  A operands live
// in tensor memory, B operands in shared memory; float32 values enter as
// three bf16 planes that are cut, not rounded: 8 + 8 + 8 bits hold a float32
// exactly.  The float32 state itself stays in registers, so that products are
// added to it with rounding to nearest.
#pragma once

#include "delta_tiles.cuh"
#include "tc_common.cuh"

namespace la {
namespace dtc {

constexpr int kComputeWarps = 16, kLoadWarps = 3;      // 20 warps with the MMA warp: 96 registers
constexpr int kFirstCompute = 1 + kLoadWarps;       // warp 0 issues the products
constexpr int kRowThreads = 64;                      // load warps 0, 1: rows; 2: bulk copies
constexpr int kThreads = (kComputeWarps + kLoadWarps + 1) * 32;
constexpr int kTri = kChunk * kChunk * 2;            // a plane of L or P

// A compute warp's piece of 32 lanes x 16 columns, as fragments (tc_common.cuh):
// [16 lanes][8 columns][4].  Everything between tensor memory and registers is
// held like this: a thread's 16 values are of 4 tokens only, V comes by
// transposed matrix loads and outputs leave by transposed matrix stores.  (With
// a lane a thread the chain waited for shared memory: 16 two-byte loads and 12
// broadcast ones a thread beside the tensor core's own reads.)
typedef float Frag[2][2][4];

__device__ __forceinline__ void load_frag(Frag& x, uint32_t addr) {
#pragma unroll
    for (int h = 0; h < 2; ++h) tc::tmem_ld_frag2(addr + (h << 20), x[h]);     // lanes 16 h ..
}
// 16 consecutive K of the planes of an A operand: 8 packed columns each.
__device__ __forceinline__ void store_a(const uint32_t (&plane)[3], uint32_t col, const Frag& x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p[3];
            cut_planes(x[h][i >> 1][2 * (i & 1)], x[h][i >> 1][2 * (i & 1) + 1], p);
#pragma unroll
            for (int j = 0; j < 3; ++j) w[j][i] = p[j];
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) tc::tmem_st_frag2(plane[j] + col + (h << 20), w[j]);
    }
}
// A thread's factors of 16 tokens: [8 tokens][2].
typedef float2 Factors[2];
__device__ __forceinline__ void factors(Factors& f, const float* p, int tq) {
    f[0] = *reinterpret_cast<const float2*>(p + 2 * tq);
    f[1] = *reinterpret_cast<const float2*>(p + 8 + 2 * tq);
}
__device__ __forceinline__ float factor(const Factors& f, int j, int e) {
    return (e & 1) ? f[j].y : f[j].x;
}
// 16 tokens x 32 columns of a swizzled tile of rows of tokens, transposed.
__device__ __forceinline__ void load_rows_frag(Frag& x, uint32_t tile, int half, int tok, int col,
                                               int lane) {
    // matrices: tokens 0-7 and 8-15 of eight columns, then of the next eight
    const int r = tok + (lane & 15);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = (col >> 3) + 2 * h + (lane >> 4);
        uint32_t w[4];
        ldsm4_t(w, tile + (c >> 3) * half + r * 128 + (((c & 7) ^ (r & 7)) << 4));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                x[h][j][2 * k] = __uint_as_float(w[2 * k + j] << 16);
                x[h][j][2 * k + 1] = __uint_as_float(w[2 * k + j] & 0xffff0000u);
            }
    }
}
// A fragment to and from the workspace: [warp][N][lane] 16-byte units, `i` below N.
__device__ __forceinline__ void save_frag(float4* out, int units, int i, const Frag& x, int warp,
                                          int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float* p = x[k >> 1][k & 1];
        out[(warp * units + 4 * i + k) * 32 + lane] = make_float4(p[0], p[1], p[2], p[3]);
    }
}
__device__ __forceinline__ void fetch_frag(Frag& x, const float4* in, int units, int i, int warp,
                                           int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 p = in[(warp * units + 4 * i + k) * 32 + lane];
        float* q = x[k >> 1][k & 1];
        q[0] = p.x; q[1] = p.y; q[2] = p.z; q[3] = p.w;
    }
}
// f(h, j, e) for each place of a fragment.
template <typename F>
__device__ __forceinline__ void each(F&& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) f(h, j, e);
}
// Packed pairs of tokens (as [16 lanes][8 tokens][2]) to 16 rows of 64 bytes in
// shared memory, one row a token, pieces permuted; and a thread's piece of it
// (token lane / 4 + 8 i, columns 8 (lane % 4) ..).
__device__ __forceinline__ void stage_rows(uint32_t buf, const uint32_t (&w)[2][2][2], int lane) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = j * 8 + (lane & 7);
        stsm4_t(buf + t * 64 + (((lane >> 3) ^ ((t >> 1) & 3)) << 4), w[0][j][0], w[0][j][1],
                w[1][j][0], w[1][j][1]);
    }
}
__device__ __forceinline__ uint4 staged_row(const unsigned char* buf, int i, int lane) {
    const int t = (lane >> 2) + 8 * i;
    return *reinterpret_cast<const uint4*>(buf + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
}

// After this thread's tensor-memory stores and loads: tell the MMA warp.
__device__ __forceinline__ void arrive(uint64_t* bar, int lane) {
    tc::tmem_wait_st();
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}

// One warp's copy of ROWS (64) rows of a [T, D] matrix as 128-byte swizzled
// blocks of 64 columns, `half` bytes apart.  Rows behind the sequence are 0 and not
// read; columns behind D are left alone.
// A lane keeps to one 16-byte column, so that a copy costs three instructions
// (row and column taken from a running index cost 6000 cycles a chunk).
template <int ROWS = kChunk>
__device__ __forceinline__ void load_tile(uint32_t dst, int half, const __nv_bfloat16* src,
                                          long long stride, int rows, int D, int lane) {
    const int c = lane & 15, r0 = lane >> 4;
    if (c * 8 >= D) return;
    const __nv_bfloat16* p = src + r0 * stride + c * 8;
    const uint32_t d = dst + (c >> 3) * half + r0 * 128;
    uint32_t at[4];                             // rows r0, r0 + 2, r0 + 4, r0 + 6 of eight
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = d + j * 256 + (((c & 7) ^ (r0 + 2 * j)) << 4);
#pragma unroll
    for (int i = 0; i < ROWS / 2; ++i) {
        const bool on = r0 + 2 * i < rows;
        cp16(at[i & 3] + (i >> 2) * 1024, on ? p : src, on);
        p += 2 * stride;
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
// Asks the L2 for a run of bytes, by one warp.  (As one bulk prefetch it held up
// the issuing thread for 5000 cycles.)
__device__ __forceinline__ void prefetch_lines(const void* src, int bytes, int lane) {
    for (int i = lane * 128; i < bytes; i += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(src) + i));
}

// A shared-memory descriptor whose address moves by constants: one thread
// issues all products, and its instructions between two of them count.
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ Desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
        const uint64_t d = tc::sdesc_sw128(addr, lbo, sbo);
        lo = (uint32_t)d;
        hi = (uint32_t)(d >> 32);
    }
    __device__ __forceinline__ uint64_t at(uint32_t bytes) const {    // addresses stay below 2^18
        return ((uint64_t)hi << 32) | (lo + (bytes >> 4));
    }
};

// The planes of S^T, by parts of a quarter of the key rows: the first two of a
// part lie where the update's products of the same key rows come (columns
// DP / 4 * part ..), the last from `lo` on.  Each compute warp so overwrites
// only what it has read itself.
template <int DP>
__device__ __forceinline__ constexpr uint32_t state_col(int plane, int step, uint32_t lo) {
    return plane == 2 ? lo + 8 * step
                      : DP / 4 * (step / (DP / 64)) + plane * (DP / 8) + 8 * (step % (DP / 64));
}

// S^T x rows^T: N = 64 rows, K = 16-key steps FIRST .. LAST - 1 (below `steps`).
template <int NA, int DP, int FIRST, int LAST>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t tm, uint32_t lo, uint32_t tile,
                                          int half, int steps) {
    constexpr uint32_t id = tc::idesc_bf16(128, 64, false, false);
    const Desc b(tile, 0, 1024);
#pragma unroll
    for (int p = NA - 1; p >= 0; --p)
#pragma unroll
        for (int k = FIRST; k < LAST; ++k)
            if (k < steps)
                tc::mma_bf16_ta(d, tm + state_col<DP>(p, k, lo), b.at((k >> 2) * half + (k & 3) * 32),
                                id, FIRST > 0 || p < NA - 1 || k > 0);
}

// Plane pairs (i of A, j of B) with i + j < NP, the smallest products first: four
// bits each, i | j << 2.
template <int NP> struct Pairs;
template <> struct Pairs<3> {      // (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
    static constexpr uint32_t kCode = 0x041852;
    static constexpr int kCount = 6;
};
template <> struct Pairs<2> {      // (1,0) (0,1) (0,0)
    static constexpr uint32_t kCode = 0x041;
    static constexpr int kCount = 3;
};

// X x L^T with L lower triangular by blocks of 16: token block kp reaches the
// columns from 16 kp on.  X's planes are 32 columns apart.
template <int NP>
__device__ __forceinline__ void mma_lower(uint32_t d, uint32_t a, uint32_t tile) {
    const Desc b(tile, 0, 1024);
    uint32_t code = Pairs<NP>::kCode;
#pragma unroll
    for (int n = 0; n < Pairs<NP>::kCount; ++n, code >>= 4) {
        const uint32_t ai = a + 32 * (code & 3), bj = ((code >> 2) & 3) * kTri;
#pragma unroll
        for (int kp = 0; kp < 4; ++kp)
            tc::mma_bf16_ta(d + 16 * kp, ai + 8 * kp, b.at(bj + kp * 2048 + kp * 32),
                            tc::idesc_bf16(128, 64 - 16 * kp, false, false), n > 0 || kp > 0);
    }
}

// X x rows: n columns, K = 64 tokens (down the rows of the tile); X's planes
// are 32 columns apart, those of the rows `plane` bytes.
template <int NP>
__device__ __forceinline__ void mma_update(uint32_t d, uint32_t a, uint32_t tile, int half,
                                           int plane, int n) {
    const uint32_t id = tc::idesc_bf16(128, 0, false, true) | ((uint32_t)(n >> 3) << 17);
    const Desc b(tile, half, 1024);
    uint32_t code = Pairs<NP>::kCode;
#pragma unroll
    for (int i = 0; i < Pairs<NP>::kCount; ++i, code >>= 4) {
        const uint32_t ai = a + 32 * (code & 3), bj = ((code >> 2) & 3) * plane;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            tc::mma_bf16_ta(d, ai + k * 8, b.at(bj + k * 2048), id, i > 0 || k > 0);
    }
}

// S^T x rows^T with rows in planes (`plane` bytes apart): the product of the
// first planes and the products with a lower one in two accumulators.
template <int DP, int FIRST, int LAST>
__device__ __forceinline__ void mma_state_planes(uint32_t d_hi, uint32_t d_lo, uint32_t tm,
                                                 uint32_t lo, uint32_t tile, int half, int plane,
                                                 int steps) {
    constexpr uint32_t id = tc::idesc_bf16(128, 64, false, false);
    const Desc b(tile, 0, 1024);
    uint32_t code = Pairs<3>::kCode;
#pragma unroll
    for (int n = 0; n < 6; ++n, code >>= 4) {
        const int i = code & 3, j = (code >> 2) & 3;
#pragma unroll
        for (int k = FIRST; k < LAST; ++k)
            if (k < steps)
                tc::mma_bf16_ta(n == 5 ? d_hi : d_lo, tm + state_col<DP>(i, k, lo),
                                b.at(j * plane + (k >> 2) * half + (k & 3) * 32), id, 1);
    }
}

// rows^T x L, the rows (one bf16 plane, 128 columns as two blocks `half` bytes
// apart) down the product's K and L lower triangular in three planes: token block
// ip of the rows reaches the columns up to 16 ip + 15.
__device__ __forceinline__ void mma_rows_lower(uint32_t d_hi, uint32_t d_lo, uint32_t rows, int half,
                                               uint32_t tile) {
    const Desc a(rows, half, 1024), b(tile, 0, 1024);
#pragma unroll
    for (int j = 2; j >= 0; --j)
#pragma unroll
        for (int ip = 3; ip >= 0; --ip)             // the widest first: it sets all columns
            tc::mma_bf16(j ? d_lo : d_hi, a.at(ip * 2048), b.at(j * kTri + ip * 2048),
                         tc::idesc_bf16(128, 16 * ip + 16, true, true), j == 1 || ip < 3);
}

// planes of A (32 columns apart, three) x rows of one plane: n columns.
__device__ __forceinline__ void mma_planes_rows(uint32_t d, uint32_t a, uint32_t tile, int n,
                                                bool add) {
    const uint32_t id = tc::idesc_bf16(128, 0, false, true) | ((uint32_t)(n >> 3) << 17);
    const Desc b(tile, 0, 1024);
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            tc::mma_bf16_ta(d, a + 32 * p + 8 * k, b.at(k * 2048), id, add || p < 2 || k > 0);
}

}  // namespace dtc
}  // namespace la
