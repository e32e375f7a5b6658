// tw_kv.cu — what a paged key-value cache needs around attention: block
// tables and slots from request lengths (k_kv_assign), and the rotation of
// new queries and keys fused with the write of keys and values into their
// slots (k_rope_append).
#include <type_traits>
#include <cooperative_groups.h>

#include "tw_kv.cuh"

namespace cg = cooperative_groups;


namespace tw {
namespace {

// ------------------------------------------------------------- assignment
constexpr int kAsThreads = 1024;
constexpr int kAsCtas = 16;         // one cluster (of the largest size), or
// a single block up to as many requests and rows: more requests would not fit
// the shared memory that needs no asking (32 requests and rows 5.2 us, the
// cluster 5.8; 1400 of each 8.0, 8.8; 32 and 2700 rows 6.0, 6.7.  The cluster is
// ahead from some 5000 rows on: 32 and 4000 rows 7.2 us, a block 6.5; 6000 rows
// 7.0, 8.1).
constexpr int64_t kAsSmall = 2800;

__device__ __forceinline__ uint32_t pages_of(int32_t len, uint32_t page)   // len >= 0
{
    return ((uint32_t)len + page - 1) / page;
}

// What one request does in a step (of at most 2^31 - 1 tokens after it).
struct Step {
    int32_t now;             // its length after the step
    uint32_t held, need;     // its pages before and after
    int32_t grown;           // its new tokens
};

__device__ __forceinline__ Step step_of(int32_t len, int32_t delta, uint32_t page)
{
    Step s;
    const int64_t now = (int64_t)len + delta;
    s.now = (int32_t)min(max(now, (int64_t)0), (int64_t)INT32_MAX);
    s.held = pages_of(len, page);
    s.need = pages_of(s.now, page);
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

// One cluster of blocks.  Every block scans all requests for itself
// (at most kAssignMaxRequests lengths, read from L2), so that the only thing
// the blocks wait for is that the pages handed back are in the free list
// before any page is taken from it.  Bound by that: two passes over the requests
// with divisions by the page size and 64-bit sums, the same in every block, then
// dependent loads and bisections (1024 requests and 65536 rows: 10.8 us for 0.8 MB).  Pages and rows then go out thread by
// thread: each finds its request by bisection of the prefix sums in shared
// memory, and a row its page in the block table or, where this step takes it,
// straight in the free list.
__global__ void __launch_bounds__(kAsThreads) k_kv_assign(const KvAssign a, uint32_t *err)
{
    extern __shared__ int32_t sm[];
    const int64_t R = a.requests;
    const uint32_t page_size = (uint32_t)a.page_size;
    int32_t *start = sm;                 // [R + 1] first row of each request
    int32_t *old = start + R + 1;        // [R]
    int32_t *take = old + R;             // [R] rank of its first page taken
    int32_t *give = take + R;            // [R + 1] rank of its first page given back
    __shared__ int64_t part[3][kAsThreads / 32];
    __shared__ int64_t total[3];
    __shared__ uint32_t bad;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t gtid = (int64_t)cluster.block_rank() * kAsThreads + tid;
    const int64_t gthreads = (int64_t)gridDim.x * kAsThreads;
    const int64_t count = *a.free_count;
    if (tid == 0)
        bad = 0;
    __syncthreads();

    // Each thread sums a run of consecutive requests, then the runs are scanned.
    const int64_t per = (R + kAsThreads - 1) / kAsThreads;
    const int64_t lo = min((int64_t)tid * per, R), hi = min(lo + per, R);
    int64_t sum[3] = {0, 0, 0};
    uint32_t wrong = 0;
    for (int64_t r = lo; r < hi; ++r) {
        const int32_t len = max(a.lengths[r], 0), delta = a.delta[r];
        const Step s = step_of(len, delta, page_size);
        if (a.lengths[r] < 0 || s.held > a.max_pages)
            wrong |= EFLAG_BADDESC;
        else if (s.need > a.max_pages || (int64_t)len + delta > INT32_MAX)
            wrong |= EFLAG_NOSPACE;
        sum[0] += s.grown;
        sum[1] += s.need > s.held ? s.need - s.held : 0u;
        sum[2] += s.held > s.need ? s.held - s.need : 0u;
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
            const Step s = step_of(len, a.delta[r], page_size);
            start[r] = (int32_t)at[0];
            old[r] = len;
            take[r] = (int32_t)at[1];
            give[r] = (int32_t)at[2];
            at[0] += s.grown;
            at[1] += s.need > s.held ? s.need - s.held : 0;
            at[2] += s.held > s.need ? s.held - s.need : 0;
        }
    if (ok && tid == 0)
        start[R] = (int32_t)total[0], give[R] = (int32_t)total[2];
    __syncthreads();

    // The last request whose prefix is at or before x: requests that add
    // nothing share their prefix with the next one.
    auto owner = [&](const int32_t *prefix, int32_t x) {
        int l = 0, h = (int)R;
        while (h - l > 1) {
            const int m = (l + h) / 2;
            if (prefix[m] <= x)
                l = m;
            else
                h = m;
        }
        return l;
    };
    // pages handed back, on top of the list
    const int64_t given = ok ? total[2] : 0, taken = ok ? total[1] : 0;
    for (int64_t k = gtid; k < given; k += gthreads) {
        const int r = owner(give, (int32_t)k);
        // the last of its pages: entry `held` less those that are still to come
        const int64_t held = pages_of(old[r], page_size);
        a.free_pages[count + k] = a.block_table[r * a.table_stride + held - (give[r + 1] - k)];
    }
    // Orders the list's new entries, and every read of the inputs that the
    // outputs may overwrite, before what follows in any block.
    cluster.sync();
    for (int64_t k = gtid; k < taken; k += gthreads) {
        const int r = owner(take, (int32_t)k);
        const int64_t held = pages_of(old[r], page_size);
        a.block_table[r * a.table_stride + held + (k - take[r])] = a.free_pages[top - 1 - k];
    }
    // rows, four in turn to a thread: one bisection, four loads in flight
    const int64_t used = ok ? total[0] : 0;
    const bool quads = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions) |
                         reinterpret_cast<uintptr_t>(a.request_of_row)) & 15) == 0;
    for (int64_t t0 = 4 * gtid; t0 < a.rows; t0 += 4 * gthreads) {
        int32_t page[4], in[4], pos[4], req[4], slot[4];
        int r = t0 < used ? owner(start, (int32_t)t0) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t t = t0 + e;
            page[e] = in[e] = pos[e] = 0, req[e] = -1;
            if (t >= used)
                continue;
            while (start[r + 1] <= t)   // (start[R] = used)
                ++r;
            const int32_t p = old[r] + (int32_t)(t - start[r]);
            const int32_t held = (int32_t)pages_of(old[r], page_size), j = (int32_t)((uint32_t)p / page_size);
            page[e] = *(j < held ? a.block_table + r * a.table_stride + j
                                 : a.free_pages + (top - 1 - take[r] - (j - held)));
            in[e] = (int32_t)((uint32_t)p - (uint32_t)j * page_size);
            req[e] = r;
            pos[e] = p;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t s = page[e] * a.page_size + in[e];
            if (page[e] < 0 || s > INT32_MAX)   // no page of any pool: a table or list that holds something else
                atomicOr(err, EFLAG_BADDESC);
            slot[e] = req[e] < 0 || page[e] < 0 || s > INT32_MAX ? -1 : (int32_t)s;
        }
        if (quads && t0 + 4 <= a.rows) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(a.request_of_row + t0) = make_int4(req[0], req[1], req[2], req[3]);
            continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t0 + e < a.rows) {
                a.slots[t0 + e] = slot[e];
                a.positions[t0 + e] = pos[e];
                a.request_of_row[t0 + e] = req[e];
            }
    }
    // lengths_out may be lengths and free_count_out free_count: every block
    // has its copy of both by now, except of delta, which no output aliases.
    for (int64_t r = gtid; r < R; r += gthreads) {
        if (ok)
            a.lengths_out[r] = step_of(old[r], a.delta[r], page_size).now;
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
// Warps that a call is split into before a warp takes more heads: 32 on each
// of 148 SMs (8192 rows of 12 + 2 + 2 heads, 126 MB, in turn with two others:
// one row a warp 24.9 us, half a row 27.5 us, a quarter 31.6 us).
constexpr int64_t kRaWarps = 4736;

// Sine and cosine of pos * freq.  The angle is formed in 64 bits and brought
// into [-pi/4, pi/4] there by a whole number k of quarter turns (half a turn
// in two 64-bit parts, each product fused with its sum; adding 1.5 * 2^52
// rounds to a whole number and leaves it in the low bits).  What is left, r,
// is rounded to 32 bits, by at most 2^-25, so that far positions are as exact
// as near ones; its Taylor series leave out less than 2^-29 (sine, r^11 / 11! at
// pi/4) and 2^-33 (cosine, r^12 / 12!).  k mod 4 swaps and signs the two.
__device__ __forceinline__ void angle_sincos(int32_t pos, double freq, float *sin_out, float *cos_out)
{
    const double kQuarterHi = 1.5707963267948966, kQuarterLo = 6.123233995736766e-17;
    const double kRound = 6755399441055744.0;   // 1.5 * 2^52
    const double a = (double)pos * freq;
    const double sum = fma(a, 0.6366197723675814, kRound);   // 2 / pi
    const int k = __double2loint(sum);
    const double n = sum - kRound;
    const float r = (float)fma(-n, kQuarterLo, fma(-n, kQuarterHi, a)), q = r * r;
    float s = fmaf(q, 1.0f / 362880, -1.0f / 5040), c = fmaf(q, -1.0f / 3628800, 1.0f / 40320);
    s = fmaf(q, s, 1.0f / 120), c = fmaf(q, c, -1.0f / 720);
    s = fmaf(q, s, -1.0f / 6), c = fmaf(q, c, 1.0f / 24);
    s = fmaf(r * q, s, r), c = fmaf(q, c, -0.5f);
    c = fmaf(q, c, 1.0f);
    const float x = k & 1 ? c : s, y = k & 1 ? s : c;
    *sin_out = k & 2 ? -x : x;
    *cos_out = (k + 1) & 2 ? -y : y;
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

// A warp takes `per` consecutive heads (of q, then k, then v) of one row: a
// lane holds QUADS groups of four consecutive columns and makes the cosines
// and sines that they need once for all of the heads, so nothing is shared
// and kBatch heads are in flight at a time.  Large calls wait for their loads with
// two fifths of the warps resident (64 registers): 8192 rows of 12 + 2 + 2 heads,
// 126 MB of which L2 holds nothing, take 25.8 us (4.9 TB/s; into codes 28.2).
constexpr int kBatch = 4;
template <int DT, int QUADS, bool PAIRS>   // PAIRS: (2i, 2i + 1) are turned, else (i, i + rotary / 2)
__global__ void __launch_bounds__(kRaThreads, QUADS == 1 ? 4 : 2) k_rope_append(const RopeAppend a, int per,
                                                                                int parts, uint32_t *err)
{
    const int lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * (kRaThreads / 32) + (threadIdx.x >> 5);   // below 2^32: the launch sees to it
    const uint32_t t = item / (uint32_t)parts;
    if (t >= a.rows)
        return;
    const int D = a.head_dim, half = a.rotary / 2;
    const int first = (int)(item - t * (uint32_t)parts) * per;
    const int64_t slot = a.slots[t];
    const bool in_pools = slot < a.cache.num_pages * a.cache.page_size;
    if (!in_pools && first == 0 && lane == 0)
        atomicOr(err, EFLAG_BADDESC);
    const int pos = a.positions[t];

    // columns 4 * (lane + 32 u) .., and from there to their partners'
    int col[QUADS], to_other[QUADS];
    bool in[QUADS], turned[QUADS];
    float co[QUADS][4], si[QUADS][4];
#pragma unroll
    for (int u = 0; u < QUADS; ++u) {
        col[u] = 4 * (lane + 32 * u);
        in[u] = col[u] < D;
        turned[u] = col[u] < a.rotary;
        to_other[u] = col[u] < half ? half : -half;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            co[u][e] = 1.f, si[u][e] = 0.f;
    }
    auto make_angles = [&] {
#pragma unroll
        for (int u = 0; u < QUADS; ++u) {
            if (!turned[u])
                continue;
            const double *f = a.inv_freq + (PAIRS ? col[u] / 2 : col[u] < half ? col[u] : col[u] - half);
#pragma unroll
            for (int e = 0; e < (PAIRS ? 2 : 4); ++e) {
                angle_sincos(pos, f[e], &si[u][e], &co[u][e]);
                if (!PAIRS && col[u] < half)
                    si[u][e] = -si[u][e];
            }
        }
    };
    // n heads from src on, D columns apart, handed to put(head, u, values);
    // TURN: rotated.  (Every load of a batch is over before its first store:
    // q_out may be q.)
    bool have = false;
    auto each = [&](auto turn, const float *src, int n, auto put) {
        constexpr bool TURN = decltype(turn)::value;
        for (int b = 0; b < n; b += kBatch, src += kBatch * D) {
            float4 x[kBatch][QUADS], y[kBatch][QUADS];
            const float *p = src;
#pragma unroll
            for (int k = 0; k < kBatch; ++k, p += D) {
                const bool some = b + k < n;
#pragma unroll
                for (int u = 0; u < QUADS; ++u) {
                    x[k][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (some && in[u])
                        x[k][u] = *reinterpret_cast<const float4 *>(p + col[u]);
                    if (TURN && !PAIRS) {
                        y[k][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (some && turned[u])
                            y[k][u] = *reinterpret_cast<const float4 *>(p + col[u] + to_other[u]);
                    }
                }
            }
            if (TURN && !have) {   // while the first heads are on their way
                make_angles();
                have = true;
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (b + k >= n)
                    break;
#pragma unroll
                for (int u = 0; u < QUADS; ++u) {
                    const float4 v = x[k][u], w = y[k][u];
                    if (TURN && PAIRS && turned[u])
                        x[k][u] = make_float4(v.x * co[u][0] - v.y * si[u][0], v.y * co[u][0] + v.x * si[u][0],
                                              v.z * co[u][1] - v.w * si[u][1], v.w * co[u][1] + v.z * si[u][1]);
                    else if (TURN && !PAIRS)
                        x[k][u] = make_float4(v.x * co[u][0] + w.x * si[u][0], v.y * co[u][1] + w.y * si[u][1],
                                              v.z * co[u][2] + w.z * si[u][2], v.w * co[u][3] + w.w * si[u][3]);
                }
                put(b + k, x[k]);
            }
        }
    };
    const int q1 = min(first + per, a.heads);
    if (first < q1) {
        float *out = a.q_out + (int64_t)t * a.ldqo + first * D;
        each(std::true_type{}, a.q + (int64_t)t * a.ldq + first * D, q1 - first, [&](int k, const float4 (&v)[QUADS]) {
#pragma unroll
            for (int u = 0; u < QUADS; ++u)
                if (in[u])
                    *reinterpret_cast<float4 *>(out + k * D + col[u]) = v[u];
        });
    }
    if (slot < 0 || !in_pools || first + per <= a.heads)
        return;
    const uint32_t page = (uint32_t)slot / (uint32_t)a.cache.page_size;
    const int64_t token = page * a.cache.page_stride +
                          ((uint32_t)slot - page * (uint32_t)a.cache.page_size) * a.cache.token_stride;
    auto keep = [&](bool is_v, int h, const float4 (&x)[QUADS]) {
        void *pool = is_v ? a.cache.v : a.cache.k;
        const int64_t at = token + h * a.cache.head_stride;
        if constexpr (DT == TW_KV_I8) {
            float m = 0.f;
#pragma unroll
            for (int u = 0; u < QUADS; ++u)
                m = fmaxf(m, fmaxf(fmaxf(fabsf(x[u].x), fabsf(x[u].y)), fmaxf(fabsf(x[u].z), fabsf(x[u].w))));
#pragma unroll
            for (int o = 16; o; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float s = m == 0.f ? 0.f : __fdiv_rn(127.f, m);
#pragma unroll
            for (int u = 0; u < QUADS; ++u) {
                if (!in[u])
                    continue;
                const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                uint32_t w = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w |= (uint32_t)(min(max(__float2int_rn(__fmul_rn(v[j], s)), -127), 127) & 0xff) << (8 * j);
                *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(pool) + at + col[u]) = w;
            }
            if (lane == 0)
                (is_v ? a.cache.v_scale : a.cache.k_scale)[slot * a.kv_heads + h] = __fdiv_rn(m, 127.f);
        } else {
#pragma unroll
            for (int u = 0; u < QUADS; ++u)
                if (in[u])
                    store4<DT>(pool, at + col[u], x[u]);
        }
    };
    const int k0 = max(first - a.heads, 0), k1 = min(first + per - a.heads, a.kv_heads);
    if (k0 < k1)
        each(std::true_type{}, a.k + (int64_t)t * a.ldk + k0 * D, k1 - k0,
             [&](int k, const float4 (&v)[QUADS]) { keep(false, k0 + k, v); });
    const int v0 = max(first - a.heads - a.kv_heads, 0), v1 = min(first + per - a.heads - a.kv_heads, a.kv_heads);
    if (v0 < v1)
        each(std::false_type{}, a.v + (int64_t)t * a.ldv + v0 * D, v1 - v0,
             [&](int k, const float4 (&v)[QUADS]) { keep(true, v0 + k, v); });
}

template <int DT>
cudaError_t launch_append(const RopeAppend &a, uint32_t *err, cudaStream_t stream)
{
    // Few rows: two heads to a warp, for latency.  Many: a row's heads to as
    // few warps as leave kRaWarps of them, so that the angles are made less often.
    const int heads = a.heads + 2 * a.kv_heads;
    int per = 2;
    while (per < heads && (a.rows * ceil_div(heads, 2 * per) >= kRaWarps || a.rows * ceil_div(heads, per) > INT32_MAX))
        per *= 2;
    const int parts = (int)ceil_div(heads, per);
    const unsigned grid = (unsigned)ceil_div(a.rows * parts, kRaThreads / 32);
    auto *kernel = a.head_dim <= 128 ? a.interleaved ? k_rope_append<DT, 1, true> : k_rope_append<DT, 1, false>
                   : a.interleaved   ? k_rope_append<DT, 2, true>
                                     : k_rope_append<DT, 2, false>;
    kernel<<<grid, kRaThreads, 0, stream>>>(a, per, parts, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_assign(const KvAssign &a, uint32_t *err, cudaStream_t stream)
{
    const size_t smem = (size_t)(4 * a.requests + 2) * sizeof(int32_t);
    const unsigned ctas = a.requests + a.rows <= kAsSmall ? 1 : kAsCtas;
    if (ctas == 1) {   // (a block of its own is a cluster of one)
        k_kv_assign<<<1, kAsThreads, smem, stream>>>(a, err);
        return cudaGetLastError();
    }
    // the cluster's size and its shared memory are past what a kernel has without asking
    cudaError_t e = ask_once([] {
        cudaError_t e = cudaFuncSetAttribute(k_kv_assign, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(k_kv_assign, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)((4 * kAssignMaxRequests + 2) * sizeof(int32_t)));
    });
    if (e != cudaSuccess)
        return e;
    static_assert((4 * kAsSmall + 2) * sizeof(int32_t) < 46 * 1024, "a single block needs no asking");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kAsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_kv_assign, a, err);
}

cudaError_t launch_rope_append(const RopeAppend &a, uint32_t *err, cudaStream_t stream)
{
    switch ((int)a.cache.dtype) {
    case TW_KV_BF16: return launch_append<TW_KV_BF16>(a, err, stream);
    case TW_KV_F16: return launch_append<TW_KV_F16>(a, err, stream);
    default: return launch_append<TW_KV_I8>(a, err, stream);
    }
}

}  // namespace tw
