// Warp-level matrix products, matrix loads and stores, and asynchronous copies
// for the token-wise kernels.
//
// Products take bf16 operands into float32 sums.  A float32 operand enters as a
// sum of bf16 planes, each the rounding of what the planes before it leave:
// two planes hold x up to 2^-18 |x|, three up to 2^-27 |x|.  Of a product of
// two such sums the plane pairs (i, j) with i + j < planes are taken; the rest
// is below the last plane's rounding.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace la {

// c[16 x 8] += a[16 x 16] b[16 x 8].  Thread (g = lane / 4, t = lane % 4) holds
//   c: (g, 2t) (g, 2t+1) (g+8, 2t) (g+8, 2t+1)
//   a: pairs (g, 2t..) (g+8, 2t..) (g, 2t+8..) (g+8, 2t+8..)
//   b: pairs (2t.., g) (2t+8.., g)
// so two neighbouring c tiles, rounded, are the a operand of a next product.
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
// Four 8 x 8 matrices; lane i gives the address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Two 8 x 8 matrices stored transposed; lanes 0..15 give row addresses.
__device__ __forceinline__ void stsm2_t(uint32_t addr, uint32_t r0, uint32_t r1) {
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1,%2};"
                 :: "r"(addr), "r"(r0), "r"(r1) : "memory");
}

// Four 8 x 8 matrices; lane i gives the address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void stsm4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                      uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                        uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}

// Two floats as a bf16 pair (x0 in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x0, x1);
    return *reinterpret_cast<const uint32_t*>(&t);
}
// Planes of a pair of floats.
template <int NP>
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t (&p)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        p[i] = pack_bf16(x0, x1);
        x0 -= __uint_as_float(p[i] << 16);
        x1 -= __uint_as_float(p[i] & 0xffff0000u);
    }
}
// Two neighbouring c tiles as the planes of an a operand.
template <int NP>
__device__ __forceinline__ void split_tiles(const float (&c0)[4], const float (&c1)[4],
                                            uint32_t (&a)[NP][4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t p[NP];
        split_bf16<NP>(e < 2 ? c0[2 * e] : c1[2 * e - 4], e < 2 ? c0[2 * e + 1] : c1[2 * e - 3], p);
#pragma unroll
        for (int i = 0; i < NP; ++i) a[i][e] = p[i];
    }
}

// x - (the bf16 halves of p): one mixed-precision FMA each, exact where p was cut
// from x.  (Masking the halves out first costs 12 cycles a pair and plane set
// beside 7.)
__device__ __forceinline__ void minus_halves(float& x0, float& x1, uint32_t p) {
    asm("{\n\t.reg .b16 l, h, m;\n\tmov.b32 {l, h}, %2;\n\tmov.b16 m, 0xbf80;\n\t"     // -1
        "fma.rn.f32.bf16 %0, l, m, %0;\n\tfma.rn.f32.bf16 %1, h, m, %1;\n\t}"
        : "+f"(x0), "+f"(x1) : "r"(p));
}
// Planes of two floats by cutting; their sum is the float (values below 2^-110
// lose their last bits).
__device__ __forceinline__ void cut_planes(float x0, float x1, uint32_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
        if (i < 2) minus_halves(x0, x1, p[i]);
    }
}

// Two neighbouring c tiles as the three cut planes of an a operand.
__device__ __forceinline__ void cut_tiles(const float (&c0)[4], const float (&c1)[4],
                                          uint32_t (&a)[3][4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t p[3];
        cut_planes(e < 2 ? c0[2 * e] : c1[2 * e - 4], e < 2 ? c0[2 * e + 1] : c1[2 * e - 3], p);
#pragma unroll
        for (int i = 0; i < 3; ++i) a[i][e] = p[i];
    }
}

// 16 bytes to shared memory; zeros when `on` is false (src is not read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// Byte offset of 16-byte piece `c` of row `r` in a tile of CH pieces a row (a
// power of two): pieces are permuted within 128 bytes so that eight rows of
// one piece fall into different banks.
template <int CH>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    constexpr int S = CH >= 8 ? 0 : CH == 4 ? 1 : 2;     // rows that share 128 bytes, log2
    constexpr int M = CH >= 8 ? 7 : CH - 1;
    return (uint32_t)(r * CH + (c ^ ((r >> S) & M))) * 16u;
}

// Lane addresses for ldmatrix on such a tile.  rows: r0.., pieces: c0..
// A operand [16 rows x 16 columns], row-major; also a transposed pair of b
// operands whose k runs down the rows (ldsm4_t: r[0], r[1] are b0, b1 of the
// eight columns of piece c0, r[2], r[3] of piece c0 + 1).
template <int CH>
__device__ __forceinline__ uint32_t at_rows(uint32_t base, int r0, int c0, int lane) {
    return base + tile_at<CH>(r0 + (lane & 15), c0 + (lane >> 4));
}
// Two b operands whose k runs along the rows: r[0], r[1] are b0, b1 of the
// eight rows r0.., r[2], r[3] of rows r0 + 8...
template <int CH>
__device__ __forceinline__ uint32_t at_cols(uint32_t base, int r0, int c0, int lane) {
    return base + tile_at<CH>(r0 + (lane & 7) + ((lane >> 4) << 3), c0 + ((lane >> 3) & 1));
}

}  // namespace la
