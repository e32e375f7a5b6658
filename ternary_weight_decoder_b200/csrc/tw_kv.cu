// tw_kv.cu — what a paged key-value cache needs around attention: block
// tables and slots from request lengths (k_kv_assign), and the rotation of
// new queries and keys fused with the write of keys and values into their
// slots (k_rope_append).
#include <cooperative_groups.h>

#include "tw_kv.cuh"

namespace cg = cooperative_groups;

namespace tw {
namespace {

// ------------------------------------------------------------- assignment
constexpr int kAsThreads = 512;
constexpr int kAsCtas = 8;   // one portable cluster

// What one request does in a step.
struct Step {
    int64_t now;             // its length after the step
    int64_t held, need;      // its pages before and after
    int64_t grown;           // its new tokens
};

__device__ __forceinline__ Step step_of(int32_t len, int32_t delta, int64_t page)
{
    Step s;
    s.now = (int64_t)len + delta;
    s.now = s.now < 0 ? 0 : s.now;
    s.held = ((int64_t)len + page - 1) / page;
    s.need = (s.now + page - 1) / page;
    s.grown = s.now > len ? s.now - len : 0;
    return s;
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += u;
    }
    return v;
}

// One cluster of kAsCtas blocks.  Every block scans all requests for itself
// (at most kAssignMaxRequests lengths, read from L2), so that the only thing
// the blocks wait for is that the pages handed back are in the free list
// before any page is taken from it.  The pages then go out block by block
// over the requests, and the rows thread by thread: a row finds its request
// by bisection of the row starts in shared memory, and its page in the block
// table or, where this step takes it, straight in the free list.
__global__ void __launch_bounds__(kAsThreads) k_kv_assign(const KvAssign a, uint32_t *err)
{
    extern __shared__ int32_t sm[];
    const int64_t R = a.requests;
    int32_t *start = sm;                 // [R + 1] first row of each request
    int32_t *old = start + R + 1;        // [R]
    int32_t *take = old + R;             // [R] rank of its first page taken
    int32_t *give = take + R;            // [R] rank of its first page given back
    __shared__ int64_t part[3][kAsThreads / 32];
    __shared__ int64_t total[3];
    __shared__ uint32_t bad;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t gtid = (int64_t)cluster.block_rank() * kAsThreads + tid;
    const int64_t gthreads = (int64_t)kAsCtas * kAsThreads;
    if (tid == 0)
        bad = 0;
    __syncthreads();

    // Each thread sums a run of consecutive requests, then the runs are scanned.
    const int64_t per = (R + kAsThreads - 1) / kAsThreads;
    const int64_t lo = min((int64_t)tid * per, R), hi = min(lo + per, R);
    int64_t sum[3] = {0, 0, 0};
    uint32_t wrong = 0;
    for (int64_t r = lo; r < hi; ++r) {
        const int32_t len = a.lengths[r];
        const Step s = step_of(len, a.delta[r], a.page_size);
        if (len < 0 || s.held > a.max_pages)
            wrong |= EFLAG_BADDESC;
        else if (s.need > a.max_pages || s.now > INT32_MAX)
            wrong |= EFLAG_NOSPACE;
        sum[0] += s.grown;
        sum[1] += s.need > s.held ? s.need - s.held : 0;
        sum[2] += s.held > s.need ? s.held - s.need : 0;
    }
    int64_t incl[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        incl[i] = warp_inclusive(sum[i], lane);
        if (lane == 31)
            part[i][warp] = incl[i];
    }
    if (wrong)
        atomicOr(&bad, wrong);
    __syncthreads();
    if (warp < 3) {
        const int64_t v = lane < kAsThreads / 32 ? part[warp][lane] : 0;
        const int64_t w = warp_inclusive(v, lane);
        if (lane < kAsThreads / 32)
            part[warp][lane] = w - v;
        if (lane == 31)
            total[warp] = w;
    }
    const int64_t count = *a.free_count;
    __syncthreads();
    const int64_t top = count + total[2];   // height of the free list once pages are back
    uint32_t flags = bad;
    if (count < 0 || count > a.free_capacity || top > a.free_capacity)
        flags |= EFLAG_BADDESC;
    else if (total[1] > top || total[0] > a.rows)
        flags |= EFLAG_NOSPACE;
    const bool ok = flags == 0;

    int64_t at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i)
        at[i] = part[i][warp] + incl[i] - sum[i];
    if (ok)
        for (int64_t r = lo; r < hi; ++r) {
            const int32_t len = a.lengths[r];
            const Step s = step_of(len, a.delta[r], a.page_size);
            start[r] = (int32_t)at[0];
            old[r] = len;
            take[r] = (int32_t)at[1];
            give[r] = (int32_t)at[2];
            at[0] += s.grown;
            at[1] += s.need > s.held ? s.need - s.held : 0;
            at[2] += s.held > s.need ? s.held - s.need : 0;
        }
    if (ok && tid == 0)
        start[R] = (int32_t)total[0];
    __syncthreads();

    if (ok) {
        // pages handed back, on top of the list
        const int64_t gw = (int64_t)cluster.block_rank() * (kAsThreads / 32) + warp;
        for (int64_t r = gw; r < R; r += kAsCtas * (kAsThreads / 32)) {
            const Step s = step_of(old[r], a.delta[r], a.page_size);
            for (int64_t j = s.need + lane; j < s.held; j += 32)
                a.free_pages[count + give[r] + (j - s.need)] = a.block_table[r * a.table_stride + j];
        }
    }
    // Orders the list's new entries, and every read of the inputs that the
    // outputs may overwrite, before what follows in any block.
    cluster.sync();
    if (ok) {
        const int64_t gw = (int64_t)cluster.block_rank() * (kAsThreads / 32) + warp;
        for (int64_t r = gw; r < R; r += kAsCtas * (kAsThreads / 32)) {
            const Step s = step_of(old[r], a.delta[r], a.page_size);
            for (int64_t j = s.held + lane; j < s.need; j += 32)
                a.block_table[r * a.table_stride + j] = a.free_pages[top - 1 - take[r] - (j - s.held)];
        }
    }
    const int64_t used = ok ? total[0] : 0;
    for (int64_t t = gtid; t < a.rows; t += gthreads) {
        int32_t slot = -1, pos = 0, req = -1;
        if (t < used) {
            // the last request whose first row is at or before t (requests
            // without new rows share their start with the next one)
            int64_t l = 0, h = R;
            while (h - l > 1) {
                const int64_t m = (l + h) / 2;
                if (start[m] <= t)
                    l = m;
                else
                    h = m;
            }
            const int64_t held = ((int64_t)old[l] + a.page_size - 1) / a.page_size;
            const int64_t p = old[l] + (t - start[l]);
            const int64_t j = p / a.page_size;
            const int32_t page = j < held ? a.block_table[l * a.table_stride + j]
                                          : a.free_pages[top - 1 - take[l] - (j - held)];
            req = (int32_t)l;
            pos = (int32_t)p;
            slot = (int32_t)(page * a.page_size + (p - j * a.page_size));
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
        a.request_of_row[t] = req;
    }
    // lengths_out may be lengths and free_count_out free_count: every block
    // has its copy of both by now, except of delta, which no output aliases.
    for (int64_t r = gtid; r < R; r += gthreads) {
        if (ok)
            a.lengths_out[r] = (int32_t)step_of(old[r], a.delta[r], a.page_size).now;
        else if (a.lengths_out != a.lengths)
            a.lengths_out[r] = a.lengths[r];
    }
    if (a.row_start)
        for (int64_t r = gtid; r <= R; r += gthreads)
            a.row_start[r] = ok ? start[r] : 0;
    if (gtid == 0) {
        *a.free_count_out = (int32_t)(ok ? top - total[1] : count);
        if (flags)
            atomicOr(err, flags);
    }
}

// -------------------------------------------------- rotation and the cache
constexpr int kRaThreads = 256;
constexpr int kRaMaxHalf = 128;   // angles of a head of up to 256

// Angles of far positions: pos * inv_freq is formed in 64 bits and brought
// into [-pi, pi] there (two pi in two 64-bit parts, each product fused with
// its sum), and only the reduced angle is rounded to 32 bits, by at most
// 2^-23: sine and cosine are then as exact as those of a near position.
__device__ __forceinline__ void angle_sincos(int32_t pos, double freq, float *s, float *c)
{
    const double kTwoPiHi = 6.283185307179586232, kTwoPiLo = 2.4492935982947064e-16;
    const double a = (double)pos * freq;
    const double k = rint(a * 0.15915494309189535);
    const double r = fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, a));
    sincosf((float)r, s, c);
}

template <int DT>
__device__ __forceinline__ void store4(void *base, int64_t at, float4 v)
{
    if constexpr (DT == TW_KV_BF16) {
        // half to even, the type's own rounding: the cache's only loss
        __nv_bfloat162 p[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(base) + at) =
            *reinterpret_cast<uint2 *>(p);
    } else {
        __half2 p[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
        *reinterpret_cast<uint2 *>(static_cast<__half *>(base) + at) = *reinterpret_cast<uint2 *>(p);
    }
}

// One block per row (token), one warp per head of q, k or v: a lane holds up
// to two groups of four consecutive columns.  The row's cosines and sines are
// made once, in shared memory.
template <int DT>
__global__ void __launch_bounds__(kRaThreads) k_rope_append(const RopeAppend a, uint32_t *err)
{
    __shared__ __align__(16) float cs[kRaMaxHalf], sn[kRaMaxHalf];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = a.rotary / 2, D = a.head_dim;
    if (tid < half)
        angle_sincos(a.positions[t], a.inv_freq[tid], &sn[tid], &cs[tid]);
    const int64_t slot = a.slots[t];
    const int64_t slots = a.cache.num_pages * a.cache.page_size;
    const bool write = slot >= 0 && slot < slots;
    if (slot >= slots && tid == 0)
        atomicOr(err, EFLAG_BADDESC);
    const int64_t page = write ? slot / a.cache.page_size : 0;
    const int64_t off = write ? slot - page * a.cache.page_size : 0;
    __syncthreads();

    const int heads = a.heads + 2 * a.kv_heads;
    for (int i = warp; i < heads; i += kRaThreads / 32) {
        const bool is_q = i < a.heads, is_v = i >= a.heads + a.kv_heads;
        if (!is_q && !write)
            continue;
        const int h = is_q ? i : is_v ? i - a.heads - a.kv_heads : i - a.heads;
        const float *row = is_q   ? a.q + t * a.ldq + (int64_t)h * D
                           : is_v ? a.v + t * a.ldv + (int64_t)h * D
                                  : a.k + t * a.ldk + (int64_t)h * D;
        float4 x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int c = 4 * (lane + 32 * u);
            x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c >= D)
                continue;
            x[u] = *reinterpret_cast<const float4 *>(row + c);
            if (is_v || c >= a.rotary)
                continue;
            if (a.interleaved) {
                const float2 co = *reinterpret_cast<const float2 *>(cs + c / 2);
                const float2 si = *reinterpret_cast<const float2 *>(sn + c / 2);
                const float4 y = x[u];
                x[u] = make_float4(y.x * co.x - y.y * si.x, y.y * co.x + y.x * si.x,
                                   y.z * co.y - y.w * si.y, y.w * co.y + y.z * si.y);
            } else {
                const bool low = c < half;
                const int p = low ? c : c - half;
                const float4 y = *reinterpret_cast<const float4 *>(row + (low ? c + half : c - half));
                const float4 co = *reinterpret_cast<const float4 *>(cs + p);
                const float4 si = *reinterpret_cast<const float4 *>(sn + p);
                const float g = low ? -1.f : 1.f;
                x[u] = make_float4(x[u].x * co.x + g * y.x * si.x, x[u].y * co.y + g * y.y * si.y,
                                   x[u].z * co.z + g * y.z * si.z, x[u].w * co.w + g * y.w * si.w);
            }
        }
        if (is_q) {
            // (a warp has read the whole head before it writes: q_out may be q)
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = 4 * (lane + 32 * u);
                if (c < D)
                    *reinterpret_cast<float4 *>(a.q_out + t * a.ldqo + (int64_t)h * D + c) = x[u];
            }
            continue;
        }
        void *pool = is_v ? a.cache.v : a.cache.k;
        const int64_t at = page * a.cache.page_stride + off * a.cache.token_stride + h * a.cache.head_stride;
        if constexpr (DT == TW_KV_I8) {
            float m = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u)
                m = fmaxf(m, fmaxf(fmaxf(fabsf(x[u].x), fabsf(x[u].y)), fmaxf(fabsf(x[u].z), fabsf(x[u].w))));
#pragma unroll
            for (int o = 16; o; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float s = m == 0.f ? 0.f : __fdiv_rn(127.f, m);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = 4 * (lane + 32 * u);
                if (c >= D)
                    continue;
                const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                uint32_t w = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w |= (uint32_t)(min(max(__float2int_rn(__fmul_rn(v[j], s)), -127), 127) & 0xff) << (8 * j);
                *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(pool) + at + c) = w;
            }
            if (lane == 0)
                (is_v ? a.cache.v_scale : a.cache.k_scale)[slot * a.kv_heads + h] = __fdiv_rn(m, 127.f);
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = 4 * (lane + 32 * u);
                if (c < D)
                    store4<DT>(pool, at + c, x[u]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_assign(const KvAssign &a, uint32_t *err, cudaStream_t stream)
{
    const size_t smem = (size_t)(4 * a.requests + 1) * sizeof(int32_t);
    if (smem > 46 * 1024) {   // (with the static arrays, past the default limit)
        cudaError_t e = cudaFuncSetAttribute(k_kv_assign, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)((4 * kAssignMaxRequests + 1) * sizeof(int32_t)));
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kAsCtas);
    cfg.blockDim = dim3(kAsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kAsCtas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_kv_assign, a, err);
}

cudaError_t launch_rope_append(const RopeAppend &a, uint32_t *err, cudaStream_t stream)
{
    const unsigned grid = (unsigned)a.rows;
    switch ((int)a.cache.dtype) {
    case TW_KV_BF16: k_rope_append<TW_KV_BF16><<<grid, kRaThreads, 0, stream>>>(a, err); break;
    case TW_KV_F16: k_rope_append<TW_KV_F16><<<grid, kRaThreads, 0, stream>>>(a, err); break;
    default: k_rope_append<TW_KV_I8><<<grid, kRaThreads, 0, stream>>>(a, err); break;
    }
    return cudaGetLastError();
}

}  // namespace tw
