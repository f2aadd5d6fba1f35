// Residual addition, RMSNorm and an e4m3 output with scales, and the backward
// pass of the addition and the norm.
//
// Both are bound by memory: every value is read once into registers, the
// sums are taken there in float32, and the results leave once.  A thread
// holds VPT vectors of 8 neighbouring columns (16 bytes of bf16); 16
// neighbouring lanes then hold the 128 columns of one scale group, so a
// group's maximum takes four shuffles and no shared memory.  28160 rows of 2560 in
// bf16 with a residual: 90 us, 5.6 TB/s (float32: 148 us, 6.4); backward, 8192 rows of 2560:
// 37 us, 4.5 TB/s (float32: 76 us, 4.4).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "mma.cuh"
#include "token.cuh"

namespace la {
namespace {

constexpr float kE4m3Max = 448.f;

struct Vec8 { float x[8]; };

__device__ __forceinline__ Vec8 load8(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
// Two products at once.
__device__ __forceinline__ void mul2(float& a, float& b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b) : "f"(c), "f"(d));
}
// (a, b) += (c, d) (e, f)
__device__ __forceinline__ void fma2(float& a, float& b, float c, float d, float e, float f) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mov.b64 z, {%4, %5};\n\tfma.rn.f32x2 x, y, z, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b) : "f"(c), "f"(d), "f"(e), "f"(f));
}
// sum + x^2 + y^2 of a bf16 pair, whose squares are exact in float32.
__device__ __forceinline__ float add_squares(float sum, uint32_t w) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tfma.rn.f32.bf16 %0, l, l, %0;\n\t"
        "fma.rn.f32.bf16 %0, h, h, %0;\n\t}" : "+f"(sum) : "r"(w));
    return sum;
}
// bf16 pairs' sums, rounded once (as the float32 sum rounded to bf16 is: a bit below
// float32's last cannot decide a tie between sums of 8-bit numbers).
__device__ __forceinline__ uint32_t add_pairs(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// Eight values as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ Vec8 value() const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        Vec8 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v.x[2 * i] = __uint_as_float(w[i] << 16);
            v.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        return v;
    }
    __device__ __forceinline__ void add(const Raw8& o) {       // as stored
        r = make_uint4(add_pairs(r.x, o.r.x), add_pairs(r.y, o.r.y), add_pairs(r.z, o.r.z),
                       add_pairs(r.w, o.r.w));
    }
    __device__ __forceinline__ float squares() const {
        return add_squares(add_squares(add_squares(add_squares(0.f, r.x), r.y), r.z), r.w);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ Vec8 value() const {
        return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    __device__ __forceinline__ void add(const Raw8& o) {
        a = make_float4(a.x + o.a.x, a.y + o.a.y, a.z + o.a.z, a.w + o.a.w);
        b = make_float4(b.x + o.b.x, b.y + o.b.y, b.z + o.b.z, b.w + o.b.w);
    }
    __device__ __forceinline__ float squares() const {
        return (((a.x * a.x + a.y * a.y) + (a.z * a.z + a.w * a.w)) +
                ((b.x * b.x + b.y * b.y) + (b.z * b.z + b.w * b.w)));
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Vec8& v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const Vec8& v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}
// Largest of two, NaN if either is NaN (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Eight values over their group's scale as e4m3.  The quotient is a product with
// the scale's reciprocal (1.5 roundings in place of 0.5, before one to 4 bits);
// scales whose reciprocal is not a normal number divide.
__device__ __forceinline__ uint2 quantise8(Vec8 v, float s, float inv) {
    if (inv != 0.f) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) mul2(v.x[j], v.x[j + 1], inv, inv);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.x[j] /= s;
    }
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        // the saturating conversion rounds to nearest even; only a quotient a
        // rounding above 448 saturates
        const __nv_fp8x4_e4m3 e4(make_float4(v.x[4 * j], v.x[4 * j + 1], v.x[4 * j + 2],
                                             v.x[4 * j + 3]));
        out[j] = *reinterpret_cast<const uint32_t*>(&e4);
    }
    return make_uint2(out[0], out[1]);
}
// y = h r weight, and its largest magnitude (NaN if one is).
__device__ __forceinline__ float norm8(Vec8& y, float r, const float* weight) {
    const Vec8 w = load8(weight);
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        mul2(y.x[j], y.x[j + 1], r, r);
        mul2(y.x[j], y.x[j + 1], w.x[j], w.x[j + 1]);
        asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(fabsf(y.x[j])), "f"(fabsf(y.x[j + 1])));
    }
    return top;
}
// The scale of a largest magnitude, and its reciprocal or 0 where that is to be
// divided by.  (NaN and infinity divide as well.)  A quotient that underflows to 0 is
// as good as 0: dividing by it would make NaN of the group's zeros.
__device__ __forceinline__ float scale_of(float top, float& inv) {
    const float q = top / kE4m3Max, s = q == 0.f ? 1.f : q;
    inv = s > 1e-36f && s < 1e36f ? 1.f / s : 0.f;
    return s;
}

// Sum (or NaN-keeping maximum) over the block, the same in every thread.
template <bool MAX>
__device__ float block_reduce(float x, float* smem) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float y = __shfl_xor_sync(~0u, x, d);
        x = MAX ? max_nan(x, y) : x + y;
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return x;
    __syncthreads();                       // the buffer's last readers are done
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = x;
    __syncthreads();
    x = smem[0];
    for (int w = 1; w < warps; ++w) x = MAX ? max_nan(x, smem[w]) : x + smem[w];
    return x;
}

// One row of at most 512 columns a warp.
__global__ void __launch_bounds__(256)
norm_fp8_warp_kernel(const __nv_bfloat16* x, const __nv_bfloat16* residual, const float* weight,
                     __nv_bfloat16* h, uint8_t* y8, float* scale, long long rows, int N, int group,
                     float eps) {
    using T = __nv_bfloat16;
    constexpr int V = 2;                   // vectors of 8 columns a lane
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31, nv = N / 8;
    Raw8<T> v[V];                          // h as stored
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < nv) v[i].load(x + row * N + (lane + 32 * i) * 8);
    if (residual) {
        Raw8<T> r[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < nv) r[i].load(residual + row * N + (lane + 32 * i) * 8);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < nv) v[i].add(r[i]);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < nv) {
            if (h) v[i].store(h + row * N + (lane + 32 * i) * 8);
            ss += v[i].squares();
        }
#pragma unroll
    for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
    const float r = 1.f / sqrtf(ss / (float)N + eps);
    // y of one vector, and its largest magnitude
    auto normed = [&](int i, Vec8& y) {
        if (lane + 32 * i >= nv) return 0.f;
        y = v[i].value();
        return norm8(y, r, weight + (lane + 32 * i) * 8);
    };
    float row_top = 0.f;
    if (group == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Vec8 y;
            row_top = max_nan(row_top, normed(i, y));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) row_top = max_nan(row_top, __shfl_xor_sync(~0u, row_top, d));
    }
    const int groups = group ? (N + group - 1) / group : 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        Vec8 y;
        float top = normed(i, y);
        if (group)
#pragma unroll
            for (int d = 8; d; d >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, d));
        const int c = lane + 32 * i;
        if (c >= nv) continue;
        float inv;
        const float s = scale_of(group ? top : row_top, inv);
        if (group ? (c & 15) == 0 : c == 0) scale[row * groups + (group ? c >> 4 : 0)] = s;
        *reinterpret_cast<uint2*>(y8 + row * N + c * 8) = quantise8(y, s, inv);
    }
}

// One row a block.
template <typename T, int VPT>
__global__ void __launch_bounds__(512)
norm_fp8_kernel(const T* x, const T* residual, const float* weight, T* h, uint8_t* y8,
                float* scale, int N, int group, float eps) {
    __shared__ float red[32];
    const long long row = blockIdx.x;
    const int nv = N / 8;
    Raw8<T> v[VPT];                        // h as stored
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nv) v[i].load(x + row * N + c * 8);
    }
    if (residual) {
        Raw8<T> r[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nv) r[i].load(residual + row * N + c * 8);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (threadIdx.x + i * blockDim.x < nv) v[i].add(r[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nv) {
            if (h) v[i].store(h + row * N + c * 8);
            ss += v[i].squares();
        }
    }
    ss = block_reduce<false>(ss, red);
    const float r = 1.f / sqrtf(ss / (float)N + eps);

    Vec8 y[VPT];
    float top[VPT], row_top = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        top[i] = 0.f;
        if (c < nv) {
            y[i] = v[i].value();
            top[i] = norm8(y[i], r, weight + c * 8);
        }
        row_top = max_nan(row_top, top[i]);
    }
    if (group == 0) {
        row_top = block_reduce<true>(row_top, red);
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int d = 8; d; d >>= 1) top[i] = max_nan(top[i], __shfl_xor_sync(~0u, top[i], d));
    }
    const int groups = group ? (N + group - 1) / group : 1;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nv) continue;
        const float a = group ? top[i] : row_top;
        float inv;
        const float s = scale_of(a, inv);
        if (group ? (c & 15) == 0 : c == 0) scale[row * groups + (group ? c >> 4 : 0)] = s;
        *reinterpret_cast<uint2*>(y8 + row * N + c * 8) = quantise8(y[i], s, inv);
    }
}

// A block takes every gridDim.x-th row and keeps its share of dweight in
// registers, with the weight beside it (up to 8192 columns); dweight's partial sums
// leave once a block.  With STAGES, the rows that come next are on their way to shared
// memory, each thread's own pieces, so that no barrier but the sums' is needed; they
// are read again after it, so that a thread needs no more than 96 registers and four
// blocks of 160 share an SM.  8192 rows of 2560 in bf16: 37 us with dweight's 6 (64
// registers and six blocks, which read the weight twice a row: 45; rows in registers
// and three blocks took a fifth longer than that).
constexpr int kNormStages = 2;
template <typename T, int VPT, bool STAGES>
__global__ void __maxnreg__(VPT > 2 ? 128 : 96)
norm_backward_kernel(const T* dy, const T* h, const float* weight, const T* dh, T* dx,
                     float* partial, long long rows, int N, float eps) {
    extern __shared__ __align__(16) unsigned char ring[];      // [stage][h, dy, dh][N]
    __shared__ float2 red[2][32];
    int buf = 0;
    const int nv = N / 8;
    const int warps = blockDim.x >> 5;
    constexpr bool KEEP = VPT <= 2;
    Vec8 dw[VPT], kept[KEEP ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i].x[j] = 0.f;
    if (KEEP)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nv) kept[i] = load8(weight + c * 8);
        }
    auto weights = [&](int i, int c) -> Vec8 {
        if constexpr (KEEP) return kept[i];
        else return load8(weight + c * 8);
    };
    constexpr int PIECES = sizeof(T) / 2;  // 16-byte pieces of a vector
    auto place = [&](int stage, int which, int c) {
        return ring + ((size_t)(stage * 3 + which) * N + c * 8) * sizeof(T);
    };
    auto send = [&](long long row, int stage) {
        if (row < rows)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c >= nv) continue;
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                    const long long at = row * N + c * 8 + p * (8 / PIECES);
                    cp16(smem_u32(place(stage, 0, c) + 16 * p), h + at, true);
                    cp16(smem_u32(place(stage, 1, c) + 16 * p), dy + at, true);
                    if (dh) cp16(smem_u32(place(stage, 2, c) + 16 * p), dh + at, true);
                }
            }
        cp_commit();
    };
    int stage = 0;
    if (STAGES)
#pragma unroll
        for (int i = 0; i < kNormStages - 1; ++i) send(blockIdx.x + (long long)i * gridDim.x, i);
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        if (STAGES) {
            // the stage read a row ago is free: its reader is this thread
            send(row + (long long)(kNormStages - 1) * gridDim.x,
                 stage == 0 ? kNormStages - 1 : stage - 1);
            cp_wait<kNormStages - 1>();
        }
        Raw8<T> f[VPT], g[VPT], more[VPT];     // h, dy, dh
        auto fetch = [&]() {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c >= nv) continue;
                if (STAGES) {
                    f[i].load(reinterpret_cast<const T*>(place(stage, 0, c)));
                    g[i].load(reinterpret_cast<const T*>(place(stage, 1, c)));
                    if (dh) more[i].load(reinterpret_cast<const T*>(place(stage, 2, c)));
                } else {
                    f[i].load(h + row * N + c * 8);
                    g[i].load(dy + row * N + c * 8);
                    if (dh) more[i].load(dh + row * N + c * 8);
                }
            }
        };
        fetch();
        float ss = 0.f, th[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nv) continue;
            ss += f[i].squares();
            const Vec8 w = weights(i, c), x = f[i].value();
            Vec8 t = g[i].value();
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                mul2(t.x[j], t.x[j + 1], w.x[j], w.x[j + 1]);
                fma2(th[0], th[1], t.x[j], t.x[j + 1], x.x[j], x.x[j + 1]);
            }
        }
        float tf = th[0] + th[1];
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            ss += __shfl_xor_sync(~0u, ss, d);
            tf += __shfl_xor_sync(~0u, tf, d);
        }
        if (warps > 1) {                   // two buffers: one barrier a row
            float2* red_row = red[buf];
            if ((threadIdx.x & 31) == 0) red_row[threadIdx.x >> 5] = make_float2(ss, tf);
            __syncthreads();
            ss = red_row[0].x;
            tf = red_row[0].y;
            for (int k = 1; k < warps; ++k) { ss += red_row[k].x; tf += red_row[k].y; }
            buf ^= 1;
        }
        const float r = 1.f / sqrtf(ss / (float)N + eps);
        // dx = r t - (h r) (r (r mean(t h))): of factors that are as large as their product
        // (r^3 would leave float32's range at a root mean square of 1e13, or of 1e-13)
        const float s = -(r * (r * (tf / (float)N)));
        if (STAGES) fetch();               // again, so that registers are free meanwhile
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nv) continue;
            const Vec8 w = weights(i, c), y = g[i].value();
            Vec8 x = f[i].value(), out = y;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                mul2(out.x[j], out.x[j + 1], w.x[j], w.x[j + 1]);
                mul2(out.x[j], out.x[j + 1], r, r);
                mul2(x.x[j], x.x[j + 1], r, r);
                fma2(out.x[j], out.x[j + 1], x.x[j], x.x[j + 1], s, s);
                fma2(dw[i].x[j], dw[i].x[j + 1], y.x[j], y.x[j + 1], x.x[j], x.x[j + 1]);
            }
            if (dh) {
                const Vec8 e = more[i].value();
#pragma unroll
                for (int j = 0; j < 8; ++j) out.x[j] += e.x[j];
            }
            store8(dx + row * N + c * 8, out);
        }
        stage = stage == kNormStages - 1 ? 0 : stage + 1;
    }
    if (!partial) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nv) store8(partial + (size_t)blockIdx.x * N + c * 8, dw[i]);
    }
}

// dweight = sum of the blocks' partial sums: COLS columns a block, 1024 / COLS threads
// down the partials of a column, joined in a fixed order.
template <int COLS>
__global__ void __launch_bounds__(1024)
norm_dweight_kernel(const float* partial, float* dweight, int blocks, int N) {
    constexpr int DOWN = 1024 / COLS;
    __shared__ float sum[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * COLS + threadIdx.x % COLS;
    float s = 0.f;
    if (c < N)
#pragma unroll 8
        for (int i = threadIdx.x / COLS; i < blocks; i += DOWN) s += partial[(size_t)i * N + c];
#pragma unroll
    for (int d = COLS; d < 32; d <<= 1) s += __shfl_xor_sync(~0u, s, d);
    if (lane < COLS) sum[warp][lane] = s;
    __syncthreads();
    if (warp >= COLS) return;
    float t = sum[lane][warp];
#pragma unroll
    for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(~0u, t, d);
    const int out = blockIdx.x * COLS + warp;
    if (lane == 0 && out < N) dweight[out] = t;
}

// Vectors a thread holds, and the threads of a row (at most 512 for N <= 16384).
int vectors_per_thread(int N) {
    const int nv = N / 8;
    return nv <= 128 ? 1 : nv <= 1024 ? 2 : 4;
}
int row_threads(int N, int vpt) {
    const int nv = N / 8;
    return ((nv + vpt - 1) / vpt + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_norm_fp8(const void* x, const void* residual, const float* weight, void* h,
                            void* y8, float* scale, int bf16, long long rows, int N, int group,
                            float eps, cudaStream_t st) {
    const int vpt = vectors_per_thread(N), threads = row_threads(N, vpt), nv = N / 8;
    const unsigned grid = (unsigned)rows;
    // Short rows in bf16 go a warp each, eight to a block: a block of one or two warps
    // a row leaves most of an SM's warps empty (60000 rows of 256: 37 us by blocks, 31
    // by warps; of 1024: the same; float32 is bound by memory either way).
    if (bf16 && nv <= 64) {
        norm_fp8_warp_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(
            static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(residual), weight,
            static_cast<__nv_bfloat16*>(h), static_cast<uint8_t*>(y8), scale, rows, N, group, eps);
        return cudaGetLastError();
    }
    auto run = [&](auto* kernel, auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        kernel<<<grid, threads, 0, st>>>(static_cast<const T*>(x), static_cast<const T*>(residual),
                                         weight, static_cast<T*>(h), static_cast<uint8_t*>(y8),
                                         scale, N, group, eps);
    };
    __nv_bfloat16* tb = nullptr;
    float* tf = nullptr;
    if (bf16) {
        if (vpt == 1) run(norm_fp8_kernel<__nv_bfloat16, 1>, tb);
        else if (vpt == 2) run(norm_fp8_kernel<__nv_bfloat16, 2>, tb);
        else run(norm_fp8_kernel<__nv_bfloat16, 4>, tb);
    } else {
        if (vpt == 1) run(norm_fp8_kernel<float, 1>, tf);
        else if (vpt == 2) run(norm_fp8_kernel<float, 2>, tf);
        else run(norm_fp8_kernel<float, 4>, tf);
    }
    return cudaGetLastError();
}

// Bytes of the backward pass's ring, or 0 where a row's stages do not fit.
static int ring_bytes(int N, int elem) {
    const int bytes = kNormStages * 3 * N * elem;
    return bytes <= 100 * 1024 ? bytes : 0;
}
// Blocks of the backward pass: what an SM holds (about 640 threads, and the rings),
// so that enough rows are in flight, and no more, so that few partial sums leave.
static int backward_blocks(long long rows, int N, int elem) {
    const int threads = row_threads(N, vectors_per_thread(N)), ring = ring_bytes(N, elem);
    int each = threads >= 640 ? 1 : 640 / threads;
    if (ring && each > 216 * 1024 / (ring + 2048)) each = 216 * 1024 / (ring + 2048);
    const long long most = (long long)kDefaultSmCount * each;
    return (int)(rows < most ? rows : most);
}
// The most of both types: the workspace's size depends on neither the type nor the device.
int norm_backward_blocks(long long rows, int N) {
    const int a = backward_blocks(rows, N, 2), b = backward_blocks(rows, N, 4);
    return a > b ? a : b;
}

cudaError_t launch_norm_backward(const void* dy, const void* h, const float* weight,
                                 const void* dh, void* dx, float* dweight, float* partial,
                                 int bf16, long long rows, int N, float eps, cudaStream_t st) {
    const int vpt = vectors_per_thread(N), threads = row_threads(N, vpt);
    const int blocks = backward_blocks(rows, N, bf16 ? 2 : 4), ring = ring_bytes(N, bf16 ? 2 : 4);
    if (!dweight) partial = nullptr;
    auto run = [&](auto* kernel, auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), ring);
        if (e != cudaSuccess) return e;
        kernel<<<blocks, threads, ring, st>>>(static_cast<const T*>(dy), static_cast<const T*>(h),
                                              weight, static_cast<const T*>(dh), static_cast<T*>(dx),
                                              partial, rows, N, eps);
        return cudaGetLastError();
    };
    auto pick = [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (vpt == 1) return run(norm_backward_kernel<T, 1, true>, t);      // N <= 1024
        if (vpt == 2)
            return ring ? run(norm_backward_kernel<T, 2, true>, t)
                        : run(norm_backward_kernel<T, 2, false>, t);
        return run(norm_backward_kernel<T, 4, false>, t);                   // N > 8192
    };
    if (blocks > 0) {
        const cudaError_t e = bf16 ? pick(static_cast<__nv_bfloat16*>(nullptr))
                                   : pick(static_cast<float*>(nullptr));
        if (e != cudaSuccess) return e;
    }
    // Few columns leave most SMs without a block: 8 columns a block take 8 us for N = 256
    // (32 a block 12), but 10 for N = 2560, whose rows are read by sectors then (6).
    if (dweight && N < 1024)
        norm_dweight_kernel<8><<<N / 8, 1024, 0, st>>>(partial, dweight, blocks, N);
    else if (dweight)
        norm_dweight_kernel<32><<<(N + 31) / 32, 1024, 0, st>>>(partial, dweight, blocks, N);
    return cudaGetLastError();
}

}  // namespace la
