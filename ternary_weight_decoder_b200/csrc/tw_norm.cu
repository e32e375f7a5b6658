// tw_norm.cu — what stands between two blocks of a decoder layer, in one
// pass over a row: the norm of the block's output, its gate and scale, the
// residual sum, the norm of the sum, and the int8 codes of that for the next
// projection.
//   t = Npost(y);  h = x + alpha * gate * t;  n = Npre(h)
// with N one of: the identity; RMS, u / sqrt(mean(u^2) + eps) * w; layer,
// (u - mean(u)) / sqrt(var(u) + eps) * w + b.
// The codes are those of tw_quantize_act on n, bit for bit.
//
// A row of x and y is read once and held in registers from then on; sums are
// in 32 bits, the variance from the centred values.  Bound by memory: 16
// bytes per element (x, y in; h, n out).
#include "tw_device.cuh"
#include "tw_internal.h"

namespace tw {
namespace {

struct NormShape {
    int threads, per;   // threads a row, groups of V elements a thread
};

// Sum (or maximum) over the block, in a fixed order: the lanes by butterfly,
// then the warps' values in order by every thread.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *red, int warps)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (warps == 1)
        return v;
    __syncthreads();   // the last reduction's values are read
    if (lane == 0)
        red[warp] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < warps; ++w)
        v = MAX ? fmaxf(v, red[w]) : v + red[w];
    return v;
}

template <int V> struct Vec;
template <> struct Vec<4> {
    static __device__ __forceinline__ void load(const float *p, float (&v)[4])
    {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[4])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <> struct Vec<1> {
    static __device__ __forceinline__ void load(const float *p, float (&v)[1]) { v[0] = *p; }
    static __device__ __forceinline__ void store(float *p, const float (&v)[1]) { *p = v[0]; }
};

// Norm of the row held in u[PER][V], in place.
template <int V, int PER>
__device__ __forceinline__ void norm_row(float (&u)[PER][V], int kind, const float *w, const float *b,
                                         int K, float eps, float *red, int threads)
{
    const int tid = threadIdx.x, warps = threads / 32;
    if (kind == TW_NORM_NONE)
        return;
    const float inv = 1.0f / (float)K;
    if (kind == TW_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                s += u[i][j];
        const float mean = block_reduce<false>(s, red, warps) * inv;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                u[i][j] = (i * threads + tid) * V < K ? u[i][j] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
            q = fmaf(u[i][j], u[i][j], q);
    const float var = block_reduce<false>(q, red, warps) * inv;
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + eps));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = (i * threads + tid) * V;
        if (c >= K)
            continue;
        float wv[V], bv[V];
        if (w)
            Vec<V>::load(w + c, wv);
        if (b)
            Vec<V>::load(b + c, bv);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            u[i][j] *= r;
            if (w)
                u[i][j] *= wv[j];
            if (b)
                u[i][j] += bv[j];
        }
    }
}

// One block a row; thread t holds columns V * (t + i * threads).
template <int V, int PER>
__global__ void __launch_bounds__(1024) k_residual_norm(const ResidualNorm a)
{
    __shared__ float red[32];
    __shared__ int red_i[32];
    const int threads = blockDim.x, tid = threadIdx.x, K = (int)a.K;
    const int64_t m = blockIdx.x;
    float u[PER][V];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = (i * threads + tid) * V;
        if (c < K) {
            Vec<V>::load((a.y ? a.y + m * a.ldy : a.x + m * a.ldx) + c, u[i]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                u[i][j] = 0.f;
        }
    }
    if (a.y) {
        norm_row<V, PER>(u, a.post, a.post_w, a.post_b, K, a.eps, red, threads);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = (i * threads + tid) * V;
            if (c >= K)
                continue;
            float g[V], x[V];
            if (a.gate)
                Vec<V>::load(a.gate + m * a.ldg + c, g);
            Vec<V>::load(a.x + m * a.ldx + c, x);
#pragma unroll
            for (int j = 0; j < V; ++j)
                u[i][j] = fmaf(a.alpha, a.gate ? u[i][j] * g[j] : u[i][j], x[j]);
        }
    }
    if (a.h) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = (i * threads + tid) * V;
            if (c < K)
                Vec<V>::store(a.h + m * a.ldh + c, u[i]);
        }
    }
    if (!a.n && !a.xq)
        return;
    norm_row<V, PER>(u, a.pre, a.pre_w, a.pre_b, K, a.eps, red, threads);
    if (a.n) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = (i * threads + tid) * V;
            if (c < K)
                Vec<V>::store(a.n + m * a.ldn + c, u[i]);
        }
    }
    if (!a.xq)
        return;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
            top = fmaxf(top, (i * threads + tid) * V < K ? fabsf(u[i][j]) : 0.f);
    top = block_reduce<true>(top, red, threads / 32);
    const float scale = top == 0.f ? 0.f : __fdiv_rn(127.f, top);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = (i * threads + tid) * V;
        if (c >= K)
            continue;
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int q = top == 0.f ? 0 : min(max(__float2int_rn(__fmul_rn(u[i][j], scale)), -128), 127);
            sum += q;
            word |= (uint32_t)(q & 0xff) << (8 * j);
        }
        if (V == 4)
            *reinterpret_cast<uint32_t *>(a.xq + m * a.K + c) = word;
        else
            a.xq[m * a.K + c] = (int8_t)word;
    }
    if (a.qsum) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((tid & 31) == 0)
            red_i[tid >> 5] = sum;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < threads / 32; ++w)
                sum += red_i[w];
            a.qsum[m] = sum;
        }
    }
    if (tid == 0)
        a.amax[m] = top;
}

template <int V>
cudaError_t launch(const ResidualNorm &a, cudaStream_t stream)
{
    const int64_t groups = (a.K + V - 1) / V;
    // four groups a thread up to 128 threads, then more threads, then more groups
    int per = 4, threads = 128;
    while (threads < 1024 && (int64_t)threads * per < groups)
        threads *= 2;
    while ((int64_t)threads * per < groups)
        per *= 2;
    const unsigned grid = (unsigned)a.M;
    switch (per) {
    case 4: k_residual_norm<V, 4><<<grid, threads, 0, stream>>>(a); break;
    case 8: k_residual_norm<V, 8><<<grid, threads, 0, stream>>>(a); break;
    case 16: k_residual_norm<V, 16><<<grid, threads, 0, stream>>>(a); break;
    default: k_residual_norm<V, 32><<<grid, threads, 0, stream>>>(a); break;
    }
    return cudaGetLastError();
}

bool by16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

cudaError_t launch_residual_norm(const ResidualNorm &a, cudaStream_t stream)
{
    // Groups of four columns where every row of every operand starts on a
    // 16-byte boundary, single columns elsewhere (odd widths, odd strides).
    const bool quads = a.K % 4 == 0 && a.ldx % 4 == 0 && a.ldy % 4 == 0 && a.ldg % 4 == 0 &&
                       a.ldh % 4 == 0 && a.ldn % 4 == 0 && by16(a.x) && by16(a.y) && by16(a.gate) &&
                       by16(a.post_w) && by16(a.post_b) && by16(a.pre_w) && by16(a.pre_b) &&
                       by16(a.h) && by16(a.n) && by16(a.xq);
    return quads ? launch<4>(a, stream) : launch<1>(a, stream);
}

}  // namespace tw
