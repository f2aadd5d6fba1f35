// Joins the segments of the chains (delta_tiles.cuh):
//   forward   S before segment s + 1 = A_s S + B_s,        s = 1, 2, ..
//   reverse   dS behind segment s - 1 = A_s^T dS + B'_s,   from the last one on
// in float32.  A block takes 32 value columns of a head, a thread four key rows
// of four of them, so that shared memory, which bounds it, gives 16 products for
// two 16-byte reads.  (A row a thread, from global memory: 60 us for 32 heads of
// 128 and 5 segments; two columns a thread: 35.)
#include "delta_tiles.cuh"

namespace la {
namespace {

constexpr int kCols = 32, kThreads = 256, kPitch = 132;
constexpr int kBytes = (128 * kPitch + 128 * kCols) * 4;

template <bool REVERSE>
__global__ void __launch_bounds__(kThreads)
delta_join_kernel(la_delta in, DeltaWs ws) {
    extern __shared__ __align__(16) float smem[];
    float* A = smem;                                // [128][kPitch]
    float* S = smem + 128 * kPitch;                 // [128][kCols]
    const int head = blockIdx.x, v0 = blockIdx.y * kCols, D = in.D, tid = threadIdx.x;
    const int n = (seq_len(in.lengths, head / in.Hv, in.T) + kChunk - 1) / kChunk;
    const int last = (n + ws.seg.chunks - 1) / ws.seg.chunks - 1;       // segment with tokens
    if (last < 2) return;
    const int lane = tid & 31, v = (tid >> 5) * 4;
    // key row i of a thread: 32 apart where A's rows are read, four in a row where
    // its columns are, for all lanes' reads to fall into different banks
    auto key = [&](int i) { return REVERSE ? 4 * lane + i : lane + 32 * i; };
    const bool there = v0 + v < D;
    auto at = [&](float* base, int s, int i) {
        return reinterpret_cast<float4*>(ws.segment(base, head, s) + (size_t)key(i) * D + v0 + v);
    };
    float4 x[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (there && key(i) < D) x[i] = *at(ws.seg_state, REVERSE ? last - 1 : 1, i);
    for (int step = 1; step < last; ++step) {
        const int s = REVERSE ? last - step : step;
        __syncthreads();                            // A and S have been read
        const float* a = ws.segment(ws.seg_A, head, s);
        for (int i = tid; i < D * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4);
            cp16(smem_u32(A + r * kPitch + c * 4), a + (size_t)i * 4, true);
        }
        cp_commit();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<float4*>(S + key(i) * kCols + v) = x[i];
            if (there && key(i) < D) x[i] = *at(ws.seg_B, s, i);
        }
        cp_wait<0>();
        __syncthreads();
#pragma unroll 2
        for (int j = 0; j < D; j += 4) {
            float m[4][4];                          // A[key(i)][j + e], or A[j + e][key(i)]
            float4 y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(
                    REVERSE ? A + (j + i) * kPitch + key(0) : A + key(i) * kPitch + j);
                const float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) m[REVERSE ? e : i][REVERSE ? i : e] = f[e];
                y[i] = *reinterpret_cast<const float4*>(S + (j + i) * kCols + v);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i].x += m[i][e] * y[e].x;
                    x[i].y += m[i][e] * y[e].y;
                    x[i].z += m[i][e] * y[e].z;
                    x[i].w += m[i][e] * y[e].w;
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (there && key(i) < D) *at(ws.seg_state, REVERSE ? s - 1 : s + 1, i) = x[i];
    }
}

}  // namespace

cudaError_t launch_delta_join(const la_delta& in, const DeltaWs& ws, bool reverse, cudaStream_t st) {
    auto* kernel = reverse ? delta_join_kernel<true> : delta_join_kernel<false>;
    const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<dim3(in.B * in.Hv, (in.D + kCols - 1) / kCols), kThreads, kBytes, st>>>(in, ws);
    return cudaGetLastError();
}

}  // namespace la
