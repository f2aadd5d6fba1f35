// Residual addition, RMSNorm and an e4m3 output with scales, and the backward
// pass of the addition and the norm.
//
// Both are bound by memory: every value is read once into registers, the
// sums are taken there in float32, and the results leave once.  A thread
// holds VPT vectors of 8 neighbouring columns (16 bytes of bf16); 16
// neighbouring lanes then hold the 128 columns of one scale group, so a
// group's maximum takes four shuffles and no shared memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "token.cuh"

namespace la {
namespace {

constexpr float kE4m3Max = 448.f;

struct Vec8 { float x[8]; };

__device__ __forceinline__ Vec8 load8(const __nv_bfloat16* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    Vec8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v.x[2 * i] = __uint_as_float(w[i] << 16);
        v.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return v;
}
__device__ __forceinline__ Vec8 load8(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
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
    __device__ __forceinline__ void set(const Vec8& v) {       // rounds
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&t);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
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
    __device__ __forceinline__ void set(const Vec8& v) {
        a = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
        b = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
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
__device__ __forceinline__ float as_stored(const __nv_bfloat16*, float x) {
    return __bfloat162float(__float2bfloat16_rn(x));
}
__device__ __forceinline__ float as_stored(const float*, float x) { return x; }

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
        for (int j = 0; j < 8; ++j) v.x[j] *= inv;
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
// The scale of a largest magnitude, and its reciprocal or 0 where that is to be
// divided by.  (NaN and infinity divide as well.)
__device__ __forceinline__ float scale_of(float top, float& inv) {
    const float s = top == 0.f ? 1.f : top / kE4m3Max;
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

// One row a warp, for many rows: all of a row's loads are in flight at once and
// no barrier waits for them.  V: vectors of 8 columns a lane.
template <typename T, int V>
__global__ void __launch_bounds__(256, V > 6 ? 2 : 3)
norm_fp8_warp_kernel(const T* x, const T* residual, const float* weight, T* h, uint8_t* y8,
                     float* scale, long long rows, int N, int group, float eps) {
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
            if (lane + 32 * i < nv) {
                Vec8 f = v[i].value();
                const Vec8 g = r[i].value();
#pragma unroll
                for (int j = 0; j < 8; ++j) f.x[j] += g.x[j];
                v[i].set(f);
            }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < nv) {
            if (h) v[i].store(h + row * N + (lane + 32 * i) * 8);
            const Vec8 f = v[i].value();
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) part += f.x[j] * f.x[j];
            ss += part;
        }
#pragma unroll
    for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
    const float r = 1.f / sqrtf(ss / (float)N + eps);
    // y of one vector, and its largest magnitude
    auto normed = [&](int i, Vec8& y) {
        float a = 0.f;
        if (lane + 32 * i < nv) {
            y = v[i].value();
            const Vec8 w = load8(weight + (lane + 32 * i) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y.x[j] = y.x[j] * r * w.x[j];
                a = max_nan(a, fabsf(y.x[j]));
            }
        }
        return a;
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
    Vec8 v[VPT];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nv) {
            v[i] = load8(x + row * N + c * 8);
            if (residual) {
                const Vec8 r = load8(residual + row * N + c * 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].x[j] = as_stored(x, v[i].x[j] + r.x[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += v[i].x[j] * v[i].x[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].x[j] = 0.f;
        }
    }
    if (h) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nv) store8(h + row * N + c * 8, v[i]);
        }
    }
    ss = block_reduce<false>(ss, red);
    const float r = 1.f / sqrtf(ss / (float)N + eps);

    float top[VPT], row_top = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        float a = 0.f;
        if (c < nv) {
            const Vec8 w = load8(weight + c * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i].x[j] = v[i].x[j] * r * w.x[j];
                a = max_nan(a, fabsf(v[i].x[j]));
            }
        }
        top[i] = a;
        row_top = max_nan(row_top, a);
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
        *reinterpret_cast<uint2*>(y8 + row * N + c * 8) = quantise8(v[i], s, inv);
    }
}

// A block takes every gridDim.x-th row and keeps its share of dweight in
// registers; dweight's partial sums leave once a block.
template <typename T, int VPT>
__global__ void __launch_bounds__(512)
norm_backward_kernel(const T* dy, const T* h, const float* weight, const T* dh, T* dx,
                     float* partial, long long rows, int N, float eps) {
    __shared__ float2 red[2][32];
    int buf = 0;
    const int nv = N / 8;
    const int warps = blockDim.x >> 5;
    Vec8 dw[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i].x[j] = 0.f;
    // h, dy and dh of the row that comes next, where registers hold them
    constexpr bool AHEAD = VPT <= 2;
    Raw8<T> next[3][VPT];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nv) {
                next[0][i].load(h + row * N + c * 8);
                next[1][i].load(dy + row * N + c * 8);
                if (dh) next[2][i].load(dh + row * N + c * 8);
            }
        }
    };
    if (AHEAD && blockIdx.x < rows) fetch(blockIdx.x);
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        Vec8 f[VPT], g[VPT];
        Raw8<T> more[VPT];
        if (!AHEAD) fetch(row);
        float ss = 0.f, th = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < nv) {
                f[i] = next[0][i].value();
                g[i] = next[1][i].value();
                more[i] = next[2][i];
                const Vec8 w = load8(weight + c * 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss += f[i].x[j] * f[i].x[j];
                    th += g[i].x[j] * w.x[j] * f[i].x[j];
                }
            }
        }
        if (AHEAD && row + gridDim.x < rows) fetch(row + gridDim.x);
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            ss += __shfl_xor_sync(~0u, ss, d);
            th += __shfl_xor_sync(~0u, th, d);
        }
        if (warps > 1) {                   // two buffers: one barrier a row
            float2* red_row = red[buf];
            if ((threadIdx.x & 31) == 0) red_row[threadIdx.x >> 5] = make_float2(ss, th);
            __syncthreads();
            ss = red_row[0].x;
            th = red_row[0].y;
            for (int k = 1; k < warps; ++k) { ss += red_row[k].x; th += red_row[k].y; }
            buf ^= 1;
        }
        const float r = 1.f / sqrtf(ss / (float)N + eps);
        const float s = r * r * r * (th / (float)N);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nv) continue;
            const Vec8 w = load8(weight + c * 8);
            Vec8 out;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i].x[j] += g[i].x[j] * f[i].x[j] * r;
                out.x[j] = r * g[i].x[j] * w.x[j] - f[i].x[j] * s;
            }
            if (dh) {
                const Vec8 e = more[i].value();
#pragma unroll
                for (int j = 0; j < 8; ++j) out.x[j] += e.x[j];
            }
            store8(dx + row * N + c * 8, out);
        }
    }
    if (!partial) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nv) store8(partial + (size_t)blockIdx.x * N + c * 8, dw[i]);
    }
}

// dweight = sum of the blocks' partial sums: 32 columns a block, 32 threads
// down the partials of a column, joined in a fixed order.
__global__ void __launch_bounds__(1024)
norm_dweight_kernel(const float* partial, float* dweight, int blocks, int N) {
    __shared__ float sum[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < N)
        for (int i = threadIdx.y; i < blocks; i += 32) s += partial[(size_t)i * N + c];
    sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    float t = sum[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(~0u, t, d);
    const int out = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out < N) dweight[out] = t;
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
    // A warp a row once the rows fill the SMs' warps twice over and fit a warp's
    // registers (28160 rows of 2560: 127 us by blocks, 92 by warps; one row: the block
    // is faster, ten loads a lane follow one another).
    if (rows >= 2 * 16 * kDefaultSmCount && nv <= 32 * (bf16 ? 16 : 10)) {
        auto by_warp = [&](auto* kernel, auto* t) {
            using T = std::remove_pointer_t<decltype(t)>;
            kernel<<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(
                static_cast<const T*>(x), static_cast<const T*>(residual), weight,
                static_cast<T*>(h), static_cast<uint8_t*>(y8), scale, rows, N, group, eps);
        };
        __nv_bfloat16* tb = nullptr;
        float* tf = nullptr;
        const int v = (nv + 31) / 32;
        if (bf16) {
            if (v <= 2) by_warp(norm_fp8_warp_kernel<__nv_bfloat16, 2>, tb);
            else if (v <= 4) by_warp(norm_fp8_warp_kernel<__nv_bfloat16, 4>, tb);
            else if (v <= 6) by_warp(norm_fp8_warp_kernel<__nv_bfloat16, 6>, tb);
            else if (v <= 10) by_warp(norm_fp8_warp_kernel<__nv_bfloat16, 10>, tb);
            else by_warp(norm_fp8_warp_kernel<__nv_bfloat16, 16>, tb);
        } else {
            if (v <= 2) by_warp(norm_fp8_warp_kernel<float, 2>, tf);
            else if (v <= 4) by_warp(norm_fp8_warp_kernel<float, 4>, tf);
            else if (v <= 6) by_warp(norm_fp8_warp_kernel<float, 6>, tf);
            else by_warp(norm_fp8_warp_kernel<float, 10>, tf);
        }
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

// Blocks of the backward pass: about 1024 threads an SM, so that enough rows
// are in flight, and no more, so that few partial sums leave.
int norm_backward_blocks(long long rows, int N) {
    const int threads = row_threads(N, vectors_per_thread(N));
    const long long most = (long long)kDefaultSmCount * (threads >= 1024 ? 1 : 1024 / threads);
    return (int)(rows < most ? rows : most);
}

cudaError_t launch_norm_backward(const void* dy, const void* h, const float* weight,
                                 const void* dh, void* dx, float* dweight, float* partial,
                                 int bf16, long long rows, int N, float eps, cudaStream_t st) {
    const int vpt = vectors_per_thread(N), threads = row_threads(N, vpt);
    const int blocks = norm_backward_blocks(rows, N);
    if (!dweight) partial = nullptr;
    auto run = [&](auto* kernel, auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        kernel<<<blocks, threads, 0, st>>>(static_cast<const T*>(dy), static_cast<const T*>(h),
                                           weight, static_cast<const T*>(dh), static_cast<T*>(dx),
                                           partial, rows, N, eps);
    };
    __nv_bfloat16* tb = nullptr;
    float* tf = nullptr;
    if (blocks > 0) {
        if (bf16) {
            if (vpt == 1) run(norm_backward_kernel<__nv_bfloat16, 1>, tb);
            else if (vpt == 2) run(norm_backward_kernel<__nv_bfloat16, 2>, tb);
            else run(norm_backward_kernel<__nv_bfloat16, 4>, tb);
        } else {
            if (vpt == 1) run(norm_backward_kernel<float, 1>, tf);
            else if (vpt == 2) run(norm_backward_kernel<float, 2>, tf);
            else run(norm_backward_kernel<float, 4>, tf);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (dweight)
        norm_dweight_kernel<<<(N + 31) / 32, dim3(32, 32), 0, st>>>(partial, dweight, blocks, N);
    return cudaGetLastError();
}

}  // namespace la
