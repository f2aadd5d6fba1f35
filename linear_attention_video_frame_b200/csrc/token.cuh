// Shared definitions of the token-wise operators (include/la_token.h).
#pragma once

#include <cstdlib>

#include "common.cuh"
#include "la_token.h"

namespace la {

// Tokens of one chunk of the chunked gated delta rule.
constexpr int kChunk = 64;
// At this log decay and below, the decay is 0 in float32 (2^-150 is e^-103.97): the token
// forgets the state.  In the running sums of a chunk it counts as kForgetSum, so that they
// stay finite and nothing comes back with the growth of 63 later tokens (e^88.7 each at most).
constexpr float kForgets = -104.f, kForgetSum = -6000.f;

struct DeltaGrad {           // outputs and extra inputs of the backward pass
    const void* d_o;
    long long do_stride[3];
    const float* dstate_out;
    void *dq, *dk, *dv;
    float *dlog_alpha, *dbeta, *dstate_in;
};

struct Row3 {                // element offset of (b, h, t)
    long long b, h, t;
    __host__ __device__ long long at(int ib, int ih, int it) const {
        return ib * b + ih * h + it * t;
    }
};
__host__ __device__ inline Row3 row3(const long long s[3]) { return Row3{s[0], s[1], s[2]}; }

__device__ __forceinline__ int seq_len(const int* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

// For tests of the bounded waits: LA_DELTA_TEST_SKIP_ROWS = c leaves out the arrival that
// announces the key rows of head 0's chunk c to a forward chain, -1 - c to a reverse one, so
// that the waits for it run out.  The chunk, or -1.
inline int test_skip_rows(bool reverse) {
    const char* e = std::getenv("LA_DELTA_TEST_SKIP_ROWS");
    if (!e) return -1;
    const int c = std::atoi(e);
    return reverse ? -1 - c : c;
}

// Launchers; each returns the CUDA error of its launches.
// status: the words that la_query_device_status reads, or NULL.
cudaError_t launch_delta_recurrent(const la_delta& in, void* o, const long long o_stride[3],
                                   float* state_out, unsigned int* status, cudaStream_t st);
// Chunked tensor-core path (delta_chunk.cu).
bool delta_chunked(int backward, int dt, int heads, int T, int D);
size_t delta_workspace_bytes(int backward, int dt, int B, int Hk, int Hv, int T, int D);
int delta_kernel_count(int backward, int dt, int B, int Hk, int Hv, int T);
cudaError_t launch_delta_chunked(const la_delta& in, void* o, const long long o_stride[3],
                                 float* state_out, void* ws, cudaStream_t st);
cudaError_t launch_delta_backward(const la_delta& in, const DeltaGrad& g, void* ws,
                                  cudaStream_t st);

cudaError_t launch_norm_fp8(const void* x, const void* residual, const float* weight, void* h,
                            void* y8, float* scale, int bf16, long long rows, int N, int group,
                            float eps, cudaStream_t st);
int norm_backward_blocks(long long rows, int N);
cudaError_t launch_norm_backward(const void* dy, const void* h, const float* weight,
                                 const void* dh, void* dx, float* dweight, float* partial,
                                 int bf16, long long rows, int N, float eps, cudaStream_t st);

}  // namespace la
