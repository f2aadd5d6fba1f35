// Workspace and tile helpers of the chunked gated delta rule.
#pragma once

#include "mma.cuh"
#include "token.cuh"

namespace la {

// bf16 planes of a float32 value (mma.cuh).  Computed values take three (2^-27):
// states and gate gradients leave in float32, where two planes would show (3e-6 of
// the state in place of 1e-7).  bf16 inputs are exact in one, float32 ones take
// three as well.
constexpr int kPlanes = 3;

// Per token: exp(G), exp(G_63 - G), beta, and G / ln 2 as the sum of two floats.
constexpr int kGateRows = 5;

// A head's chain may be cut into segments of chunks (bf16 inputs): with few heads
// most SMs have no chain.  Segments' transitions S -> A S + B come from running
// them on the identity without values and on zero with them.  In `segments`
// segments, the first pass runs the first segment outright and A and B of those
// between; the second runs the rest from their now known states.  The backward
// pass needs only B' in its first pass, as A^T takes A's place.
struct Segments {
    int count, chunks;           // of a head; of a segment

    // Chunk times (2 to 4 us) of the passes: rounds of jobs over the SMs, one job each;
    // the second pass's start costs about three more, a join (10 to 23 us) six.  For the
    // SMs of a B200, whatever the device: a workspace's size follows from the plan, and its
    // owner asks for it by shape alone.
    static Segments plan(int backward, int heads, int chunks) {
        auto rounds = [](long long jobs) {
            return (double)((jobs + kDefaultSmCount - 1) / kDefaultSmCount);
        };
        const double passes = backward ? 2.0 : 1.0;
        Segments best{1, chunks};
        double least = passes * rounds(heads) * chunks;
        for (int s = 2; s <= 64 && s * 4 <= chunks; ++s) {
            const int each = (chunks + s - 1) / s;
            if ((chunks + each - 1) / each != s) continue;      // fewer segments do
            const double forward = rounds((long long)heads * (s > 2 ? 2 * s - 3 : 1)) +
                                   rounds((long long)heads * (s - 1));
            const double reverse = backward ? 2.0 * rounds((long long)heads * (s - 1)) : 0.0;
            const double cost = (forward + reverse) * each + (s > 2 ? 9.0 : 3.0) * passes;
            if (cost < 0.9 * least) {
                least = cost;
                best = Segments{s, each};
            }
        }
        return best;
    }
};

// What the kernels of a call hand to one another.  L and P are [64][64] bf16
// planes as shared-memory tiles (tile_at<8>, which is also the tensor core's
// 128-byte swizzle); blocks of 16 above the diagonal hold anything.  States are images
// [value column][key row] of DP columns in planes; Z and dX are rows
// [token][value column] of DP columns in planes.
struct DeltaWs {
    unsigned int* status;        // header of the workspace (la_query_device_status)
    unsigned char *gates_, *L_, *P_, *Kt_, *planes_, *states_, *dstates_, *Z_, *dX_;
    int chunks;          // per head
    int DP, D;
    size_t bytes;
    Segments seg;
    float *seg_state, *seg_A, *seg_B;    // [head][segment][D][D], as states
    float *dq_shares, *dk_shares;        // [B, Hv, T, D], where value heads share a key head

    static DeltaWs layout(void* mem, int backward, int dt, int B, int Hk, int Hv, int T, int D) {
        DeltaWs w{};
        w.chunks = (T + kChunk - 1) / kChunk;
        w.DP = D <= 64 ? 64 : 128;
        w.D = D;
        const size_t n = (size_t)B * Hv * w.chunks, nk = (size_t)B * Hk * w.chunks;
        size_t at = kWsHeaderBytes;
        unsigned char* p = static_cast<unsigned char*>(mem);
        w.status = static_cast<unsigned int*>(mem);
        auto take = [&](size_t size) {
            unsigned char* r = p + at;
            at = align_up(at + size, 256);
            return r;
        };
        w.gates_ = take(n * kGateRows * kChunk * 4);
        w.L_ = take(n * kPlanes * 2 * kChunk * kChunk);
        w.P_ = take(n * kPlanes * 2 * kChunk * kChunk);
        w.Kt_ = take(dt == LA_BF16 ? n * 3 * w.plane_bytes() : 0);
        w.planes_ = take(dt == LA_F32 ? nk * 2 * kPlanes * w.plane_bytes() : 0);
        w.seg = dt == LA_BF16 ? Segments::plan(backward, B * Hv, w.chunks) : Segments{1, w.chunks};
        if (w.seg.count > 1) {
            const size_t all = (size_t)B * Hv * w.seg.count * D * D * 4;
            w.seg_state = reinterpret_cast<float*>(take(all));
            w.seg_A = reinterpret_cast<float*>(take(all));
            w.seg_B = reinterpret_cast<float*>(take(all));
        }
        if (backward) {
            const size_t image = dt == LA_F32 ? w.image_bytes() : w.state_frag_bytes();
            const size_t rows = dt == LA_F32 ? kPlanes * w.plane_bytes() : kRowFragBytes;
            w.states_ = take((size_t)B * Hv * (w.chunks + 1) * image);
            w.dstates_ = take(n * image);
            if (dt == LA_BF16 && Hv > Hk) {
                const size_t all = (size_t)B * Hv * T * D * 4;
                w.dq_shares = reinterpret_cast<float*>(take(all));
                w.dk_shares = reinterpret_cast<float*>(take(all));
            }
            w.Z_ = take(n * rows);
            w.dX_ = take(n * rows);
        }
        w.bytes = at;
        return w;
    }
    __host__ __device__ size_t plane_bytes() const { return (size_t)kChunk * DP * 2; }
    __host__ __device__ size_t image_bytes() const { return (size_t)D * DP * 2 * kPlanes; }
    __device__ float* segment(float* base, int head, int s) const {
        return base + ((size_t)head * seg.count + s) * D * D;
    }
    // bf16 inputs: states [128 x DP], Z and dX [128 x 64] in float32, each thread's
    // values as its chain holds them (delta_tc.cuh)
    static constexpr size_t kRowFragBytes = 128 * kChunk * 4;
    __host__ __device__ size_t state_frag_bytes() const { return (size_t)128 * DP * 4; }
    __device__ float4* state_frags(int head, int c) const {         // c = 0 .. chunks
        return reinterpret_cast<float4*>(
            states_ + ((size_t)head * (chunks + 1) + c) * state_frag_bytes());
    }
    __device__ float4* dstate_frags(int head, int c) const {
        return reinterpret_cast<float4*>(dstates_ + at(head, c) * state_frag_bytes());
    }
    __device__ float4* Z_frags(int head, int c) const {
        return reinterpret_cast<float4*>(Z_ + at(head, c) * kRowFragBytes);
    }
    __device__ float4* dX_frags(int head, int c) const {
        return reinterpret_cast<float4*>(dX_ + at(head, c) * kRowFragBytes);
    }
    __device__ size_t at(int head, int c) const { return (size_t)head * chunks + c; }
    __device__ float* gates(int head, int c) const {
        return reinterpret_cast<float*>(gates_) + at(head, c) * kGateRows * kChunk;
    }
    __device__ __nv_bfloat16* L(int head, int c) const {
        return reinterpret_cast<__nv_bfloat16*>(L_) + at(head, c) * kPlanes * kChunk * kChunk;
    }
    __device__ __nv_bfloat16* P(int head, int c) const {
        return reinterpret_cast<__nv_bfloat16*>(P_) + at(head, c) * kPlanes * kChunk * kChunk;
    }
    // bf16 inputs: Kt as [half of 64 columns][plane][64 rows of 128 bytes], swizzled
    __device__ unsigned char* Kt(int head, int c) const {
        return Kt_ + at(head, c) * 3 * plane_bytes();
    }
    // float32 inputs: the planes of K, then of Q, as shared-memory tiles
    __device__ unsigned char* planes(int khead, int c) const {
        return planes_ + ((size_t)khead * chunks + c) * 2 * kPlanes * plane_bytes();
    }
    __device__ __nv_bfloat16* states(int head, int c) const {       // c = 0 .. chunks
        return reinterpret_cast<__nv_bfloat16*>(
            states_ + ((size_t)head * (chunks + 1) + c) * image_bytes());
    }
    __device__ __nv_bfloat16* dstates(int head, int c) const {
        return reinterpret_cast<__nv_bfloat16*>(dstates_ + at(head, c) * image_bytes());
    }
    __device__ __nv_bfloat16* Z(int head, int c) const {
        return reinterpret_cast<__nv_bfloat16*>(Z_ + at(head, c) * kPlanes * plane_bytes());
    }
    __device__ __nv_bfloat16* dX(int head, int c) const {
        return reinterpret_cast<__nv_bfloat16*>(dX_ + at(head, c) * kPlanes * plane_bytes());
    }
};

// Kt, Pt (and L) of every chunk (delta_tc_prep.cu)
cudaError_t launch_delta_tc_prep(const la_delta& in, const DeltaWs& ws, bool backward,
                                 cudaStream_t st);
// forward chain on tcgen05 (delta_tc.cu), with outputs or with states for the
// backward pass
cudaError_t launch_delta_tc_chain(const la_delta& in, const DeltaWs& ws, void* o, Row3 os,
                                  float* state_out, bool states, cudaStream_t st);
// the joins between the passes over segments (delta_tc_join.cu)
cudaError_t launch_delta_join(const la_delta& in, const DeltaWs& ws, bool reverse, cudaStream_t st);
// its mirror (delta_tc_reverse.cu) and the gradients of all chunks
// (delta_tc_grad.cu), bf16 inputs
cudaError_t launch_delta_tc_reverse(const la_delta& in, const DeltaGrad& g, const DeltaWs& ws,
                                    cudaStream_t st);
cudaError_t launch_delta_tc_grad(const la_delta& in, const DeltaGrad& g, const DeltaWs& ws,
                                 cudaStream_t st);
// prep and forward chain of the backward pass (delta_chunk.cu)
cudaError_t launch_delta_states(const la_delta& in, const DeltaWs& ws, cudaStream_t st);

#ifdef __CUDACC__

// Rows t0 .. t0 + 63 of a float32 [T, D] matrix as tiles of DP columns, split into
// planes.  Rows from `len` on and columns from D on are 0 and not read.
template <int DP>
__device__ __forceinline__ void load_rows_split(uint32_t dst, const void* src, long long offset,
                                                long long stride, int t0, int len, int D, int tid,
                                                int threads) {
    constexpr int CH = DP / 8;
    for (int i = tid; i < kChunk * CH; i += threads) {
        const int r = i / CH, c = i % CH;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (t0 + r < len && c * 8 < D) {
            const float4* p = reinterpret_cast<const float4*>(
                static_cast<const float*>(src) + offset + (t0 + r) * stride + c * 8);
            x = p[0];
            y = p[1];
        }
        const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint32_t w[4][kPlanes];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16<kPlanes>(f[2 * e], f[2 * e + 1], w[e]);
#pragma unroll
        for (int j = 0; j < kPlanes; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                         :: "r"(dst + j * kChunk * DP * 2 + tile_at<CH>(r, c)), "r"(w[0][j]),
                            "r"(w[1][j]), "r"(w[2][j]), "r"(w[3][j]) : "memory");
    }
}

// A run of bytes as it lies (a multiple of 16).
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, int bytes, int tid,
                                           int threads) {
    for (int i = tid; i < bytes / 16; i += threads)
        cp16(dst + i * 16, static_cast<const unsigned char*>(src) + i * 16, true);
}

// A product tile in two sums: the leading planes' product, and the products
// with a lower plane.  The tensor core rounds its sums towards zero, so a sum
// loses up to half a last place for each product added to it: few are added to
// the large one, and none to a value that lives longer than its chunk (adding
// them to the state itself cost 5e-6 over 16 chunks).
struct Acc {
    float hi[4], lo[4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[e] = lo[e] = 0.f;
    }
    __device__ __forceinline__ float operator[](int e) const { return hi[e] + lo[e]; }
};

// c[0], c[1] += a b for two tiles of eight b rows each (k along the rows of the
// tile); a in NA planes, b in NB planes `plane` bytes apart, pairs whose
// indices add up to less than NP.
template <int NP, int NA, int NB>
__device__ __forceinline__ void product_planes(Acc* c, const uint32_t (&a)[NA][4],
                                               const uint32_t (&b)[NB][4]) {
#pragma unroll
    for (int s = NP - 1; s >= 0; --s)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int i = s - j;
            if (i < 0 || i >= NA) continue;
            mma_bf16(s ? c[0].lo : c[0].hi, a[i], b[j][0], b[j][1]);
            mma_bf16(s ? c[1].lo : c[1].hi, a[i], b[j][2], b[j][3]);
        }
}
template <int NP, int NA, int NB, int CH>
__device__ __forceinline__ void product_cols(Acc* c, const uint32_t (&a)[NA][4], uint32_t tile,
                                             int plane, int row, int piece, int lane) {
    uint32_t b[NB][4];
#pragma unroll
    for (int j = 0; j < NB; ++j) ldsm4(b[j], at_cols<CH>(tile + j * plane, row, piece, lane));
    product_planes<NP, NA, NB>(c, a, b);
}
// The same with k down the rows of the tile; two tiles of eight columns.
template <int NP, int NA, int NB, int CH>
__device__ __forceinline__ void product_rows(Acc* c, const uint32_t (&a)[NA][4], uint32_t tile,
                                             int plane, int row, int piece, int lane) {
    uint32_t b[NB][4];
#pragma unroll
    for (int j = 0; j < NB; ++j) ldsm4_t(b[j], at_rows<CH>(tile + j * plane, row, piece, lane));
    product_planes<NP, NA, NB>(c, a, b);
}

// The gates of a chunk's 64 tokens, by one warp: log_alpha and beta of tokens
// 2 lane, 2 lane + 1 (those from `on` on have alpha = 1 and beta = 0) ...
// 2^((a_hi - b_hi) + (a_lo - b_lo)) to 2 units in the last place.
__device__ __forceinline__ float exp2_sum(float a_hi, float a_lo, float b_hi, float b_lo) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((a_hi - b_hi) + (a_lo - b_lo)));
    return y;
}
struct RawGates { float g[2], beta[2]; };
__device__ __forceinline__ RawGates fetch_gates(const la_delta& in, size_t at, int on, int lane) {
    RawGates r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        r.g[i] = t < on ? in.log_alpha[at + t] : 0.f;
        r.beta[i] = t < on ? in.beta[at + t] : 0.f;
    }
    return r;
}
// ... and what follows from them.  Running sums of log_alpha in double, kept in
// powers of two as two floats: differences of sums far from 0 keep the accuracy of
// their own size, and exp2_sum takes them as they are.
__device__ __forceinline__ void chunk_gates(const RawGates& raw, float* gates, float* g_hi,
                                            float* g_lo, float* beta, float* tail, int lane) {
    double s[2];
    const float* bt = raw.beta;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        s[i] = raw.g[i] <= kForgets ? kForgetSum : raw.g[i];           // keeps NaN
    s[1] += s[0];
    double run = s[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(~0u, run, d);
        if (lane >= d) run += y;
    }
    s[0] += run - s[1];
    s[1] = run;
    const double last = __shfl_sync(~0u, run, 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const double p = s[i] * 1.4426950408889634;
        const float hi = (float)p, lo = (float)(p - (double)hi);
        const float to_end = expf((float)(last - s[i]));
        g_hi[t] = hi;
        g_lo[t] = lo;
        beta[t] = bt[i];
        if (tail) tail[t] = to_end;
        gates[t] = expf((float)s[i]);
        gates[kChunk + t] = to_end;
        gates[2 * kChunk + t] = bt[i];
        gates[3 * kChunk + t] = hi;
        gates[4 * kChunk + t] = lo;
    }
}

template <int KS>
__device__ __forceinline__ void sum_parts(float (&m)[4], const float4* ex, int nt, int lane) {
    float4 s = ex[nt * 32 + lane];
#pragma unroll
    for (int p = 1; p < KS; ++p) {
        const float4 x = ex[(p * 8 + nt) * 32 + lane];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    m[0] = s.x; m[1] = s.y; m[2] = s.z; m[3] = s.w;
}

// Value columns v0 .. v0 + 15 of a chunk's rows, as rows of 20 floats.  0 behind `len`.
struct ValueTile {
    static constexpr int kPitch = 20, kBytes = kChunk * kPitch * 4;
};
__device__ __forceinline__ void load_values(uint32_t dst, const void* src, long long offset,
                                            long long stride, int v0, int t0, int len, int tid,
                                            int threads) {
    for (int i = tid; i < kChunk * 4; i += threads) {
        const int r = i >> 2, c = i & 3;
        const bool on = t0 + r < len;
        cp16(dst + (r * ValueTile::kPitch + c * 4) * 4,
             static_cast<const float*>(src) + (on ? offset + (t0 + r) * stride + v0 + c * 4 : 0), on);
    }
}

// 16 tokens of it, transposed into two product tiles.
__device__ __forceinline__ void load_v(float (&V)[2][4], const unsigned char* ptr, int row, int lane) {
    const float* v = reinterpret_cast<const float*>(ptr) + (lane >> 2);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            V[j][e] = v[(row + j * 8 + 2 * (lane & 3) + (e & 1)) * ValueTile::kPitch + 8 * (e >> 1)];
}

// S^T tiles of a warp (16 value columns, key rows from k0) into an image.
template <int NP, int NT>
__device__ __forceinline__ void store_image(__nv_bfloat16* image, const float (&S)[NT][4], int v0,
                                            int k0, int DP, int D, int lane) {
    __nv_bfloat16* p = image + (size_t)(v0 + (lane >> 2)) * DP + k0 + 2 * (lane & 3);
    const size_t plane = (size_t)D * DP;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t w[NP];
            split_bf16<NP>(S[nt][2 * r], S[nt][2 * r + 1], w);
#pragma unroll
            for (int j = 0; j < NP; ++j)
                *reinterpret_cast<uint32_t*>(p + j * plane + (size_t)r * 8 * DP + nt * 8) = w[j];
        }
}

// 64 tokens of a warp's 16 value columns (transposed tiles) as planes of rows
// of DP columns.  `stage`: 64 x 32 bytes of the warp's own.
template <int NP>
__device__ __forceinline__ void store_rows(__nv_bfloat16* out, const float (&M)[8][4],
                                           unsigned char* stage, int v0, int DP, int lane) {
    const uint32_t sm = smem_u32(stage);
    uint32_t w[8][2][NP];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        split_bf16<NP>(M[nt][0], M[nt][1], w[nt][0]);
        split_bf16<NP>(M[nt][2], M[nt][3], w[nt][1]);
    }
#pragma unroll
    for (int plane = 0; plane < NP; ++plane) {
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
            stsm2_t(sm + (nt * 8 + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16, w[nt][0][plane],
                    w[nt][1][plane]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = i * 32 + lane, r = at >> 1, half = at & 1;
            *reinterpret_cast<uint4*>(out + (size_t)plane * kChunk * DP + r * DP + v0 + half * 8) =
                *reinterpret_cast<const uint4*>(stage + at * 16);
        }
    }
}

// A warp's share of the chunk's outputs: tokens 64 / KS * part .., `rows` of
// the chunk's tokens exist.
template <int KS>
__device__ __forceinline__ void store_out(void* o, long long offset, long long stride,
                                          const float (&O)[8][4], int part, int v0, int rows,
                                          int lane) {
    float* p = static_cast<float*>(o) + offset + v0 + (lane >> 2);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        if (nt / (8 / KS) != part) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = nt * 8 + 2 * (lane & 3) + (e & 1);
            if (t < rows) p[t * stride + 8 * (e >> 1)] = O[nt][e];
        }
    }
}

#endif  // __CUDACC__

}  // namespace la
