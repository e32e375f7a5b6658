// tw_attention.cu — attention of one new token per request over a paged
// key-value cache: for the query head i of request r over its visible keys j
// (first_r <= j < length_r)
//   s_j = scale * (q_i . k_j);  out_i = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
// with m the maximum of the s_j, in one pass with the running maximum and
// sum; lse_i = m + log(sum).  No visible key: out = 0, lse = -inf.
#include "tw_kv.cuh"

namespace tw {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kDims = 8;   // columns a lane holds: head_dim <= 256

// One block per request and query head; warps take keys in turn, a lane
// holds columns lane + 32 i.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_paged_attention(const PagedAttention a, uint32_t *err)
{
    using T = typename KvElem<DT>::type;
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][32 * kDims];
    const int64_t r = blockIdx.x / a.heads;
    const int head = (int)(blockIdx.x % a.heads), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = (int)a.cache.head_dim, P = (int)a.cache.page_size;
    const int kvh = head / (a.heads / (int)a.cache.kv_heads);
    int64_t len = a.lengths[r];
    int64_t from = a.first ? max(a.first[r], 0) : 0;
    if (len > a.max_pages * P) {
        if (tid == 0)
            atomicOr(err, EFLAG_BADDESC);
        len = a.max_pages * P;
    }
    float q[kDims], o[kDims], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
        const int c = lane + 32 * i;
        q[i] = c < D ? a.q[r * a.ldq + (int64_t)head * D + c] * a.scale : 0.f;
        o[i] = 0.f;
    }
    for (int64_t j = from + warp; j < len; j += kWarps) {
        const int64_t page = a.block_table[r * a.table_stride + j / P];
        if (page < 0 || page >= a.cache.num_pages) {
            if (lane == 0)
                atomicOr(err, EFLAG_BADDESC);
            continue;
        }
        const int64_t at = page * a.cache.page_stride + (j % P) * a.cache.token_stride + kvh * a.cache.head_stride;
        const T *k = static_cast<const T *>(a.cache.k) + at, *v = static_cast<const T *>(a.cache.v) + at;
        float ks = 1.f, vs = 1.f;
        if (DT == TW_KV_I8) {
            const int64_t sc = (page * P + j % P) * a.cache.kv_heads + kvh;
            ks = a.cache.k_scale[sc];
            vs = a.cache.v_scale[sc];
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kDims; ++i)
            if (lane + 32 * i < D)
                s = fmaf(q[i], kv_to_f32(k[lane + 32 * i]), s);
#pragma unroll
        for (int b = 16; b; b >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, b);
        s *= ks;
        const float top = fmaxf(m, s);
        const float old = m == -INFINITY ? 0.f : expf(m - top);
        const float p = top == -INFINITY ? 0.f : expf(s - top);
        m = top;
        l = l * old + p;
#pragma unroll
        for (int i = 0; i < kDims; ++i)
            if (lane + 32 * i < D)
                o[i] = fmaf(p * vs, kv_to_f32(v[lane + 32 * i]), o[i] * old);
    }
    if (lane == 0)
        sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
    for (int i = 0; i < kDims; ++i)
        sm_o[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w)
        top = fmaxf(top, sm_m[w]);
    for (int w = 0; w < kWarps; ++w)
        sum += sm_m[w] == -INFINITY ? 0.f : sm_l[w] * expf(sm_m[w] - top);
    for (int c = tid; c < D; c += kThreads) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w)
            x += sm_m[w] == -INFINITY ? 0.f : sm_o[w][c] * expf(sm_m[w] - top);
        a.out[r * a.ldo + (int64_t)head * D + c] = sum > 0.f || sum != sum ? x / sum : 0.f;
    }
    if (a.lse && tid == 0)
        a.lse[r * a.heads + head] = sum > 0.f || sum != sum ? top + logf(sum) : -INFINITY;
}

}  // namespace

int64_t paged_attention_ws_bytes(int64_t requests, int64_t heads, int64_t kv_heads, int64_t head_dim)
{
    (void)requests, (void)heads, (void)kv_heads, (void)head_dim;
    return 256;
}

cudaError_t launch_paged_attention(const PagedAttention &a, uint32_t *err, cudaStream_t stream)
{
    const unsigned grid = (unsigned)(a.requests * a.heads);
    switch ((int)a.cache.dtype) {
    case TW_KV_BF16: k_paged_attention<TW_KV_BF16><<<grid, kThreads, 0, stream>>>(a, err); break;
    case TW_KV_F16: k_paged_attention<TW_KV_F16><<<grid, kThreads, 0, stream>>>(a, err); break;
    default: k_paged_attention<TW_KV_I8><<<grid, kThreads, 0, stream>>>(a, err); break;
    }
    return cudaGetLastError();
}

}  // namespace tw
