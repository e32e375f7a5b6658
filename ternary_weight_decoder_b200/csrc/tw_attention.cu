// tw_attention.cu — attention of one new token per request over a paged
// key-value cache: for the query head i of request r over its visible keys j
// (first_r <= j < length_r)
//   s_j = scale * (q_i . k_j);  out_i = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
// with m the maximum of the s_j, in one pass with the running maximum and
// sum; lse_i = m + log(sum).  No visible key: out = 0, lse = -inf.
//
// Bound by memory: every visible key and value is read once, and each element
// serves the few query heads of its group only (2 * heads / kv_heads
// multiply-adds per element), far below what tcgen05 tiles of 128 rows need
// to pay; mma.sync tiles keep up with the memory at a fraction of their rate.
//
// Split: the keys of all requests and KV heads are cut into tiles, laid end
// to end, and every block takes an equal run of them, whatever the lengths
// are.  A block whose run holds all of a (request, KV head) writes its
// output; the pieces of one that spans blocks go to the workspace and are
// joined in a fixed order, by the last block of every sixteen and then by the
// last of those.  Inside a block each warp takes 16 keys of every tile
// through its own ring of cp.async stages: no barrier until a piece ends.
//
// Matrix products: the 16 keys (or 16 columns of the values) are the rows of
// an MMA, eight query heads its columns, so no lane computes for nobody:
// scores^T = K q^T, out^T = V^T w^T.  The operands that are not in the cache
// are carried in parts, each the rounding of what the last one left: two of
// fp16 (22 bits), three of bf16 (24 bits); queries on codes in three int8
// digits (23 bits of the head's largest), whose products are exact integers.
// Scores and sums are fp32.
// Groups of more than eight heads are split into units of eight.
#include <cfloat>

#include "tw_kv.cuh"

#ifndef TW_ATT_WARPS
#define TW_ATT_WARPS 8
#endif
#ifndef TW_ATT_WARPS_CODES
#define TW_ATT_WARPS_CODES 12
#endif
#ifndef TW_ATT_BLOCKS
#define TW_ATT_BLOCKS 1
#endif
#ifndef TW_ATT_QS
#define TW_ATT_QS 0
#endif

namespace tw {
namespace {

constexpr int kKeys = 16;                    // keys of a warp's step
constexpr int kMaxCtas = 512;                // counters and partial results in the workspace
constexpr int kHeads = 8;                    // query heads of a unit
constexpr int kFan = 16;                     // pieces that one block joins
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// The shape of one variant: DP columns (head_dim rounded up) of type DT.
template <int DT, int DP>
struct Shape {
    static constexpr bool kCodes = DT == TW_KV_I8;
    static constexpr bool kBf = DT == TW_KV_BF16;
    static constexpr int kParts = kBf ? 3 : 2;         // of a weight
    static constexpr int kElem = kCodes ? 1 : 2;
    static constexpr int kRow = DP * kElem;            // bytes of a key
    static constexpr int kChunks = kRow / 16;
    static constexpr int kPool = kKeys * kRow;         // bytes of a step's keys
    static constexpr int kStage = 2 * kPool;
    static constexpr int kScales = kCodes ? 2 * kKeys * 4 : 0;   // of a stage, behind the rings
    static constexpr int kSteps = DP / 16;             // 16 columns of values each
    static constexpr int kQueryParts = kBf || kCodes ? 3 : 2;
    static constexpr int kQuerySteps = kCodes ? DP / 32 : DP / 16;   // MMA steps over a key
    static constexpr int kWarps = (kCodes ? TW_ATT_WARPS_CODES : TW_ATT_WARPS) / (DP > 128 ? 2 : 1);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTile = kKeys * kWarps;
    static constexpr int kBlocks = TW_ATT_BLOCKS;      // resident on an SM
    // Queries in registers up to 128 columns, in shared memory above.
    static constexpr bool kQueryShared = DP > 128 || TW_ATT_QS;
    static constexpr int kQueryBytes = kQueryShared ? kQuerySteps * 32 * 8 * kQueryParts : 0;
    static constexpr int kRoom = (227 * 1024) / kBlocks - 3072 - kQueryBytes;
    static constexpr int kFit = kRoom / (kWarps * (kStage + kScales));
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = kWarps * kStages * (kStage + kScales) + kQueryBytes;
    static_assert(kStages >= 2, "two stages at least");
    static_assert(kHeads * DP * 4 <= kStage, "a stage holds a warp's sums");
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 16 : 0;   // 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// D(16x8, f32) += A(16x16, row) * B(16x8, col) in fp16, or bf16.
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1)
{
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two values rounded to the operand's type, and what that leaves of them.
template <bool BF>
__device__ __forceinline__ uint32_t split2(float &x, float &y)
{
    uint32_t bits;
    if (BF) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
        x -= __bfloat162float(p.x), y -= __bfloat162float(p.y);
        bits = *reinterpret_cast<const uint32_t *>(&p);
    } else {
        const __half2 p = __floats2half2_rn(x, y);
        x -= __half2float(p.x), y -= __half2float(p.y);
        bits = *reinterpret_cast<const uint32_t *>(&p);
    }
    return bits;
}

// Bytes 0 and 2 of w, or 1 and 3, as exact fp16 codes: a code plus 128 under
// the exponent of 1024 is 1152 + code.
template <bool ODD>
__device__ __forceinline__ uint32_t codes2(uint32_t w)
{
    const uint32_t h = ((ODD ? w >> 8 : w) & 0x00ff00ffu) ^ 0x64806480u;
    const uint32_t off = 0x64806480u;   // 1152 twice
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// The 8 x 8 matrix of 16-bit values whose rows the lanes' quads hold, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Byte offset of 16-byte chunk c of key row in a step's pool: chunks are
// permuted by the row so that eight rows of one chunk fall on all banks.
template <int CHUNKS>
__device__ __forceinline__ int row_swap(int row)
{
    return CHUNKS >= 8 ? (row & 7) : ((row >> 1) & 3);
}
template <int CHUNKS>
__device__ __forceinline__ uint32_t place(int row, int c)
{
    return (uint32_t)(row * CHUNKS + (c ^ row_swap<CHUNKS>(row))) * 16;
}

// The visible keys of a request, as tiles.
struct Span {
    int lo, hi, first_tile, tiles;
};

template <int TILE>
__device__ __forceinline__ Span span_of(const PagedAttention &a, int64_t r, bool report, uint32_t *err)
{
    Span s;
    const int64_t cap = a.max_pages * a.cache.page_size;
    int64_t hi = a.lengths[r];
    if (hi > cap) {
        hi = cap;
        if (report)
            atomicOr(err, EFLAG_BADDESC);
    }
    s.hi = (int)hi;
    s.lo = a.first ? max(a.first[r], 0) : 0;
    s.first_tile = s.lo / TILE;
    s.tiles = s.hi > s.lo ? (s.hi - 1) / TILE + 1 - s.first_tile : 0;
    return s;
}

// A place in the run of tiles: tile t of unit u of request r.
template <int TILE>
struct Cursor {
    int64_t r;
    int u, t;
    Span s;
    __device__ __forceinline__ void next(const PagedAttention &a, int units)
    {
        if (++t < s.tiles)
            return;
        t = 0;
        if (++u < units)
            return;
        u = 0;
        do {
            ++r;
            if (r >= a.requests)
                return;
            s = span_of<TILE>(a, r, false, nullptr);
        } while (s.tiles == 0);
    }
};

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

// The pieces of one unit in the workspace: maxima and sums [piece][head][2],
// sums of values [piece][head][DP].
template <int DP>
struct Pieces {
    float *ml, *o;
    __device__ __forceinline__ float *at_ml(int64_t piece, int h) const { return ml + (piece * kHeads + h) * 2; }
    __device__ __forceinline__ float *at_o(int64_t piece, int h) const { return o + (piece * kHeads + h) * DP; }
};

// Join `count` <= 32 pieces of head h, piece i being piece_of(i), by one
// warp, in the order of i.  Columns 4 * lane + 128 q of the sum stay in x.
template <int DP, class F>
__device__ __forceinline__ void join(const Pieces<DP> &w, int count, int h, F piece_of,
                                     float4 (&x)[DP > 128 ? 2 : 1], float &top, float &sum)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f;
    if (lane < count) {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(w.at_ml(piece_of(lane), h)));
        m = v.x, l = v.y;
    }
    top = m;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = m == -INFINITY ? 0.f : ex2(m - top);
    sum = l * f;   // (a piece without a maximum can hold a NaN sum: it stays one)
    if (l != l)
        sum = l;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int q = 0; q < (DP > 128 ? 2 : 1); ++q) {
        x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int c = min(4 * lane + 128 * q, DP - 4);
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(w.at_o(piece_of(i), h) + c));
            const float g = __shfl_sync(0xffffffffu, f, i);
            x[q].x = fmaf(y.x, g, x[q].x), x[q].y = fmaf(y.y, g, x[q].y);
            x[q].z = fmaf(y.z, g, x[q].z), x[q].w = fmaf(y.w, g, x[q].w);
        }
    }
}

template <int DT, int DP>
__global__ void __launch_bounds__(Shape<DT, DP>::kThreads, Shape<DT, DP>::kBlocks)
    k_paged_attention(const PagedAttention a, uint32_t *err)
{
    using S = Shape<DT, DP>;
    constexpr bool BF = S::kBf;
    constexpr int W = S::kWarps, kThreads = S::kThreads, kTile = S::kTile;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t part[W];
    __shared__ int64_t start_r;
    __shared__ int start_u, start_t, last;
    __shared__ float sm_m[W][kHeads], sm_l[W][kHeads];
    __shared__ uint32_t sm_mask[W][S::kStages];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int D = (int)a.cache.head_dim, P = (int)a.cache.page_size, kvh = (int)a.cache.kv_heads;
    const int group = a.heads / kvh, per_kv = (group + kHeads - 1) / kHeads, units = kvh * per_kv;
    const int64_t R = a.requests;

    // ---- this block's run of tiles: lengths are scanned by every block
    const int64_t per = (R + kThreads - 1) / kThreads;
    const int64_t rlo = min((int64_t)tid * per, R), rhi = min(rlo + per, R);
    int64_t sum = 0;
    for (int64_t r = rlo; r < rhi; ++r)
        sum += span_of<kTile>(a, r, blockIdx.x == 0, err).tiles;
    const int64_t incl = warp_inclusive(sum, lane);
    if (lane == 31)
        part[warp] = incl;
    __syncthreads();
    int64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += w < warp ? part[w] : 0;
        total += part[w];
    }
    total *= units;
    const int64_t G = min((int64_t)gridDim.x, total);   // blocks with tiles: no run between two is empty
    const int64_t begin = blockIdx.x < G ? total * blockIdx.x / G : 0;
    const int64_t end = blockIdx.x < G ? total * (blockIdx.x + 1) / G : 0;
    if (begin < end && before * units <= begin && begin < (before + sum) * units) {
        int64_t at = before * units, r = rlo;
        for (;; ++r) {
            const int64_t n = (int64_t)span_of<kTile>(a, r, false, nullptr).tiles * units;
            if (begin < at + n) {
                const int64_t tiles = n / units;
                start_r = r;
                start_u = (int)((begin - at) / tiles);
                start_t = (int)((begin - at) % tiles);
                break;
            }
            at += n;
        }
    }
    // rows without keys
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        if (span_of<kTile>(a, r, false, nullptr).tiles)
            continue;
        for (int c = tid; c < a.heads * D; c += kThreads)
            a.out[r * a.ldo + c] = 0.f;
        if (a.lse)
            for (int h = tid; h < a.heads; h += kThreads)
                a.lse[r * a.heads + h] = -INFINITY;
    }
    __syncthreads();
    if (begin >= end)
        return;
    Cursor<kTile> load, use;
    load.r = start_r, load.u = start_u, load.t = start_t;
    load.s = span_of<kTile>(a, load.r, false, nullptr);
    use = load;

    // ---- the ring of stages
    constexpr int kRowsPer = S::kChunks >= 32 ? 1 : 32 / S::kChunks;   // rows of one pass of the warp
    const uint32_t ring = smem_u32(smem) + warp * S::kStages * S::kStage;
    const uint32_t scales = smem_u32(smem) + W * S::kStages * S::kStage + warp * S::kStages * S::kScales;
    const int row0 = lane / S::kChunks, chunk = lane % S::kChunks;
    const uint32_t lane_dst = ring + place<S::kChunks>(row0, chunk);
    const int64_t row_bytes = a.cache.token_stride * S::kElem;
    const uint8_t *kpool = static_cast<const uint8_t *>(a.cache.k) + row0 * row_bytes + chunk * 16;
    const int64_t v_of_k = static_cast<const uint8_t *>(a.cache.v) - static_cast<const uint8_t *>(a.cache.k);
    const float *scale_pool = (lane < 16 ? a.cache.k_scale : a.cache.v_scale) + (lane & 15) * kvh;
    const bool in_row = chunk < D * S::kElem / 16;
    // Steps whose 16 keys share a page, in pools with strides below 4 GB (one
    // wide multiply-add each), take the short way.
    const int64_t page_bytes = a.cache.page_stride * S::kElem, head_bytes = a.cache.head_stride * S::kElem;
    const bool short_way = P % kKeys == 0 && ((page_bytes | head_bytes | row_bytes) >> 32) == 0;
    const int page_shift = (P & (P - 1)) == 0 ? __ffs(P) - 1 : -1;
    auto fetch = [&](int stage) {
        const int head = load.u / per_kv;
        const int j0 = (load.s.first_tile + load.t) * kTile + warp * kKeys;
        const uint32_t base = stage * S::kStage;
        const int32_t *table = a.block_table + load.r * a.table_stride;
        if (short_way && j0 >= load.s.lo && j0 + kKeys <= load.s.hi) {
            const int p = page_shift >= 0 ? j0 >> page_shift : j0 / P;
            const int page = __ldg(table + p);
            if ((uint32_t)page < (uint32_t)a.cache.num_pages) {
                const int in = j0 - p * P;
                const uint8_t *ks = kpool + (uint64_t)(uint32_t)page * (uint32_t)page_bytes +
                                    (uint64_t)(uint32_t)in * (uint32_t)row_bytes +
                                    (uint64_t)(uint32_t)head * (uint32_t)head_bytes;
                const uint8_t *vs = ks + v_of_k;
                if (in_row) {
#pragma unroll
                    for (int i = 0; i < kKeys / kRowsPer; ++i) {
                        const uint32_t dst = (lane_dst + base) ^ (row_swap<S::kChunks>(kRowsPer * i) << 4);
                        cp_async16(dst + kRowsPer * i * S::kRow, ks, true);
                        cp_async16(dst + kRowsPer * i * S::kRow + S::kPool, vs, true);
                        ks += kRowsPer * row_bytes, vs += kRowsPer * row_bytes;
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < kKeys / kRowsPer; ++i) {
                        const uint32_t dst = (lane_dst + base) ^ (row_swap<S::kChunks>(kRowsPer * i) << 4);
                        cp_async16(dst + kRowsPer * i * S::kRow, a.cache.k, false);
                        cp_async16(dst + kRowsPer * i * S::kRow + S::kPool, a.cache.k, false);
                    }
                }
                if (S::kCodes)
                    cp_async4(scales + stage * S::kScales + lane * 4,
                              scale_pool + (uint64_t)(uint32_t)(page * P + in) * (uint32_t)kvh + head, true);
                if (lane == 0)
                    sm_mask[warp][stage] = 0xffffu;
                return;
            }
        }
        const int j = j0 + (lane & 15);
        bool ok = j >= load.s.lo && j < load.s.hi;
        int64_t off = 0, slot = 0;
        if (ok) {
            const int p = j / P;
            const int page = __ldg(table + p);
            if ((uint32_t)page < (uint32_t)a.cache.num_pages) {
                const int in = j - p * P;
                off = (page * a.cache.page_stride + in * a.cache.token_stride + head * a.cache.head_stride) *
                      S::kElem;
                slot = ((int64_t)page * P + in - (lane & 15)) * kvh + head;
            } else {
                ok = false;
                atomicOr(err, EFLAG_BADDESC);
            }
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
        if (lane == 0)
            sm_mask[warp][stage] = mask;
#pragma unroll 1
        for (int i = 0; i < kKeys / kRowsPer; ++i) {
            const int row = row0 + kRowsPer * i;
            const int64_t o = __shfl_sync(0xffffffffu, off, row) - row0 * row_bytes;
            const bool in = ((mask >> row) & 1) && in_row;
            const uint32_t dst = ring + base + place<S::kChunks>(row, chunk);
            cp_async16(dst, in ? kpool + o : a.cache.k, in);
            cp_async16(dst + S::kPool, in ? kpool + v_of_k + o : a.cache.k, in);
        }
        if (S::kCodes)
            cp_async4(scales + stage * S::kScales + lane * 4, ok ? scale_pool + slot : a.cache.k_scale, ok);
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    const int n = (int)(end - begin);
#pragma unroll 1
    for (int s = 0; s < S::kStages - 1; ++s) {
        if (s < n) {
            fetch(s);
            load.next(a, units);
        }
        commit();
    }

    // Queries as the MMA's B operand, in parts: [step][part] the pairs of
    // columns (head g of the unit) that this lane feeds.
    constexpr int kQ = S::kQueryShared ? 1 : S::kQuerySteps;
    uint32_t qb[kQ][S::kQueryParts][2];
    uint2 *qs = reinterpret_cast<uint2 *>(smem + W * S::kStages * (S::kStage + S::kScales));
    float o[S::kSteps][4];           // (columns g, g + 8 of 16) x (heads 2 t4, 2 t4 + 1)
    float m[2], l[2], unscale[2];    // of heads 2 t4, 2 t4 + 1
    int stage = 0;
    bool fresh = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        // ---- a new piece: its queries, split
        if (fresh) {
            const int h0 = (use.u / per_kv) * group + (use.u % per_kv) * kHeads;
            const bool live = (use.u % per_kv) * kHeads + g < group;
            const float *row = a.q + use.r * a.ldq + (int64_t)(h0 + (live ? g : 0)) * D;
            const float mul = a.scale * kLog2e;
            // a head's columns are spread over the four lanes of its quad:
            // pairs of fp16 or bf16, or four bytes, as the MMA takes them
            constexpr int kHold = S::kCodes ? 8 : 4;
            auto hold = [&](int j, float (&x)[kHold]) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int c = S::kCodes ? 32 * j + 16 * k + 4 * t4 : 16 * j + 8 * k + 2 * t4;
#pragma unroll
                    for (int e = 0; e < kHold / 2; e += 2) {
                        const float2 p = live && c + e < D ? *reinterpret_cast<const float2 *>(row + c + e)
                                                           : make_float2(0.f, 0.f);
                        x[k * (kHold / 2) + e] = p.x * mul, x[k * (kHold / 2) + e + 1] = p.y * mul;
                    }
                }
            };
            float norm = 1.f, back = 1.f;
            if (!BF) {
                // fp16 operands: the head's largest query is brought to 2^14
                // by a power of two, so that no part leaves the range.  For
                // codes it is brought below 2^23 - 2^15, the most that three
                // balanced digits of eight bits hold, and rounded there.
                float top = 0.f, poison = 0.f;   // poison: NaN if a query is, or is infinite
#pragma unroll
                for (int j = 0; j < S::kQuerySteps; ++j) {
                    float x[kHold];
                    hold(j, x);
#pragma unroll
                    for (int k = 0; k < kHold; ++k)
                        top = fmaxf(top, fabsf(x[k])), poison = fmaf(x[k], 0.f, poison);
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                poison += __shfl_xor_sync(0xffffffffu, poison, 1);
                poison += __shfl_xor_sync(0xffffffffu, poison, 2);
                const bool some = top > 0.f && top <= FLT_MAX;
                constexpr int kAt = S::kCodes ? 22 : 14;
                const int e = min(max((int)(__float_as_uint(S::kCodes ? top * 1.0078125f : top) >> 23) - 127, -100), 127);
                norm = some ? __uint_as_float((uint32_t)(127 + kAt - e) << 23) : 1.f;
                back = (some ? __uint_as_float((uint32_t)(127 - kAt + e) << 23) : 1.f) + poison;
            }
            unscale[0] = __shfl_sync(0xffffffffu, back, 8 * t4);
            unscale[1] = __shfl_sync(0xffffffffu, back, 8 * t4 + 4);
#pragma unroll
            for (int j = 0; j < S::kQuerySteps; ++j) {
                if (S::kQueryShared && j % W != warp)
                    continue;
                float x[kHold];
                hold(j, x);
                uint32_t b[S::kQueryParts][2];
                if constexpr (S::kCodes) {
#pragma unroll
                    for (int k = 0; k < S::kQueryParts; ++k)
                        b[k][0] = b[k][1] = 0;
#pragma unroll
                    for (int e = 0; e < kHold; ++e) {
                        int v = __float2int_rn(x[e] * norm);   // = 2^16 d0 + 2^8 d1 + d2
#pragma unroll
                        for (int k = S::kQueryParts - 1; k >= 0; --k) {
                            const int d = k ? ((v + 128) & 255) - 128 : v;
                            b[k][e / 4] |= (uint32_t)(d & 255) << (8 * (e & 3));
                            v = (v - d) >> 8;
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] *= norm;
#pragma unroll
                    for (int k = 0; k < S::kQueryParts; ++k)
                        b[k][0] = split2<BF>(x[0], x[1]), b[k][1] = split2<BF>(x[2], x[3]);
                }
#pragma unroll
                for (int k = 0; k < S::kQueryParts; ++k) {
                    if (S::kQueryShared)
                        qs[(j * S::kQueryParts + k) * 32 + lane] = make_uint2(b[k][0], b[k][1]);
                    else
                        qb[S::kQueryShared ? 0 : j][k][0] = b[k][0], qb[S::kQueryShared ? 0 : j][k][1] = b[k][1];
                }
            }
            if (S::kQueryShared)
                __syncthreads();
            m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.f;
#pragma unroll
            for (int c = 0; c < S::kSteps; ++c)
                o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
            fresh = false;
        }

        cp_async_wait<S::kStages - 2>();
        __syncwarp();   // every lane's copies of this stage are here, the last stage is read
        if (i + S::kStages - 1 < n) {
            fetch(stage == 0 ? S::kStages - 1 : stage - 1);
            load.next(a, units);
        }
        commit();

        const uint32_t base = ring + stage * S::kStage;
        const uint32_t mask = sm_mask[warp][stage];
        if (mask) {
            // ---- scores of keys g, g + 8 for heads 2 t4, 2 t4 + 1
            // (keys 0-7, 8-15) x (16 bytes at chunk 2 j, at 2 j + 1)
            const uint32_t kbase = base + place<S::kChunks>(lane & 15, lane >> 4);
            float sc[4];
            if constexpr (S::kCodes) {
                int acc[S::kQueryParts][4] = {};
#pragma unroll
                for (int j = 0; j < S::kQuerySteps; ++j) {
                    uint32_t f[4];
                    ldmatrix4<false>(f, kbase ^ (j << 5));
#pragma unroll
                    for (int k = 0; k < S::kQueryParts; ++k) {
                        const uint2 v = S::kQueryShared ? qs[(j * S::kQueryParts + k) * 32 + lane]
                                                        : make_uint2(qb[S::kQueryShared ? 0 : j][k][0],
                                                                     qb[S::kQueryShared ? 0 : j][k][1]);
                        mma_s8_16832(acc[k], f[0], f[1], f[2], f[3], v.x, v.y);
                    }
                }
                // exact sums of each digit (below 2^23); one rounding each below
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[e] = fmaf((float)(acc[0][e] * 256 + acc[1][e]), 256.f, (float)acc[2][e]);
            } else {
                float acc[S::kQueryParts][4] = {};
#pragma unroll
                for (int j = 0; j < S::kQuerySteps; ++j) {
                    uint32_t f[4];
                    ldmatrix4<false>(f, kbase ^ (j << 5));
#pragma unroll
                    for (int k = 0; k < S::kQueryParts; ++k) {
                        const uint2 v = S::kQueryShared ? qs[(j * S::kQueryParts + k) * 32 + lane]
                                                        : make_uint2(qb[S::kQueryShared ? 0 : j][k][0],
                                                                     qb[S::kQueryShared ? 0 : j][k][1]);
                        mma<BF>(acc[k], f[0], f[1], f[2], f[3], v.x, v.y);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[e] = acc[0][e] + acc[1][e];
                    if (S::kQueryParts == 3)
                        sc[e] += acc[S::kQueryParts - 1][e];
                }
            }
            // ---- running maximum and sum.  With codes the value's scale goes
            // into the weight (as its logarithm, so that weights stay within
            // fp16 whatever the scales are): w_j = 2^(s_j + log2 vs_j - m).
            float s[4], lv[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[e] = BF ? sc[e] : sc[e] * unscale[e & 1];
            if (S::kCodes) {
                const float *of = reinterpret_cast<const float *>(
                    smem + W * S::kStages * S::kStage + (warp * S::kStages + stage) * S::kScales);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float ks = of[g + 8 * k], vs = of[kKeys + g + 8 * k];
                    s[2 * k] *= ks, s[2 * k + 1] *= ks;
                    lv[k] = vs > 0.f ? __log2f(vs) : 0.f;
                }
            }
            if (mask != 0xffffu) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[e] = (mask >> (g + 8 * (e >> 1))) & 1 ? s[e] : -INFINITY;
            }
            float top[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                top[h] = S::kCodes ? fmaxf(s[h] + lv[0], s[2 + h] + lv[1]) : fmaxf(s[h], s[2 + h]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], x));
            if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
                float f[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float up = fmaxf(top[h], m[h]);
                    f[h] = up == -INFINITY ? 1.f : ex2(m[h] - up);
                    m[h] = up;
                    l[h] *= f[h];
                }
#pragma unroll
                for (int c = 0; c < S::kSteps; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[c][e] *= f[e & 1];
            }
            // fp16 weights are carried times 2^14 (as is the sum), so that
            // the second part of small ones stays clear of fp16's smallest
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float shift = (m[e & 1] == -INFINITY ? 0.f : m[e & 1]) - (BF ? 0.f : 14.f);
                const float x = s[e] - shift;
                p[e] = ex2(S::kCodes ? x + lv[e >> 1] : x);
                l[e & 1] += S::kCodes ? ex2(x) : p[e];
            }
            uint32_t w[S::kParts][2];
#pragma unroll
            for (int k = 0; k < S::kParts; ++k) {
                w[k][0] = transpose8(split2<BF>(p[0], p[1]));
                w[k][1] = transpose8(split2<BF>(p[2], p[3]));
            }
            // ---- weighted values: columns x heads
            if constexpr (S::kCodes) {
                // byte pairs: keys 2 t4 + {0, 1}, columns 2 g + {0, 1} of chunks
                // c, c + 1; even columns are the MMA's rows 0-7, odd ones 8-15
                const uint32_t vbase = base + S::kPool + place<S::kChunks>(lane & 15, lane >> 4);
#pragma unroll
                for (int c = 0; c < S::kSteps; c += 2) {
                    uint32_t f[4];
                    ldmatrix4<true>(f, vbase ^ (c << 4));
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t a0 = codes2<false>(f[2 * q]), a1 = codes2<true>(f[2 * q]);
                        const uint32_t a2 = codes2<false>(f[2 * q + 1]), a3 = codes2<true>(f[2 * q + 1]);
#pragma unroll
                        for (int k = 0; k < S::kParts; ++k)
                            mma<BF>(o[c + q], a0, a1, a2, a3, w[k][0], w[k][1]);
                    }
                }
            } else {
                // (columns 0-7, 8-15) x (keys 0-7, 8-15)
                const uint32_t vbase = base + S::kPool +
                                       place<S::kChunks>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
                for (int c = 0; c < S::kSteps; ++c) {
                    uint32_t f[4];
                    ldmatrix4<true>(f, vbase ^ (c << 5));
#pragma unroll
                    for (int k = 0; k < S::kParts; ++k)
                        mma<BF>(o[c], f[0], f[1], f[2], f[3], w[k][0], w[k][1]);
                }
            }
        }

        // ---- the end of a piece
        const bool unit_done = use.t + 1 == use.s.tiles;
        if (unit_done || i + 1 == n) {
            const int64_t ubeg = begin + i - use.t, uend = ubeg + use.s.tiles;
            const int h0 = (use.u / per_kv) * group + (use.u % per_kv) * kHeads;
            const int heads = min(kHeads, group - (use.u % per_kv) * kHeads);
            __syncwarp();   // the stage is read: it takes the warp's sums
            float *mine = reinterpret_cast<float *>(smem + (warp * S::kStages + stage) * S::kStage);
            // [head][column], columns permuted by the head against bank conflicts
            auto at = [](int h, int c) { return h * DP + (c ^ ((h >> 1) << 3)); };
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                    l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
                if (g == 0)
                    sm_m[warp][2 * t4 + h] = m[h], sm_l[warp][2 * t4 + h] = l[h];
#pragma unroll
                for (int c = 0; c < S::kSteps; ++c) {
                    if (S::kCodes) {
                        *reinterpret_cast<float2 *>(mine + at(2 * t4 + h, 16 * c + 2 * g)) =
                            make_float2(o[c][h], o[c][2 + h]);
                    } else {
                        mine[at(2 * t4 + h, 16 * c + g)] = o[c][h];
                        mine[at(2 * t4 + h, 16 * c + g + 8)] = o[c][2 + h];
                    }
                }
            }
            __syncthreads();
            const bool whole = unit_done && ubeg >= begin;
            uint32_t *ctr = reinterpret_cast<uint32_t *>(a.ws);
            Pieces<DP> pc;
            pc.ml = reinterpret_cast<float *>(ctr + 3 * kMaxCtas);
            pc.o = pc.ml + kMaxCtas * 2 * 2 * kHeads;
            const int64_t piece = 2 * (int64_t)blockIdx.x + (ubeg >= begin ? 1 : 0);
            const float shift = BF ? 0.f : 14.f;
            auto finish = [&](int h, int c, float4 x, float inv) {
                *reinterpret_cast<float4 *>(a.out + use.r * a.ldo + (int64_t)(h0 + h) * D + c) =
                    make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
            };
            auto finish_lse = [&](int h, float top, float sum_l) {
                if (a.lse && lane == 0)
                    a.lse[use.r * a.heads + h0 + h] = sum_l == 0.f ? -INFINITY : (top - shift) * kLn2 + logf(sum_l);
            };
            for (int h = warp; h < heads; h += W) {
                float top = -INFINITY, sum_l = 0.f, f[W];
#pragma unroll
                for (int w = 0; w < W; ++w)
                    top = fmaxf(top, sm_m[w][h]);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    f[w] = sm_m[w][h] == -INFINITY ? 0.f : ex2(sm_m[w][h] - top);
                    sum_l += sm_l[w][h] != sm_l[w][h] ? sm_l[w][h] : sm_l[w][h] * f[w];
                }
                const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
                for (int c = 4 * lane; c < D; c += 128) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float4 y = *reinterpret_cast<const float4 *>(
                            smem + (w * S::kStages + stage) * S::kStage + at(h, c) * 4);
                        x.x = fmaf(y.x, f[w], x.x), x.y = fmaf(y.y, f[w], x.y);
                        x.z = fmaf(y.z, f[w], x.z), x.w = fmaf(y.w, f[w], x.w);
                    }
                    if (whole)
                        finish(h, c, x, inv);
                    else
                        *reinterpret_cast<float4 *>(pc.at_o(piece, h) + c) = x;
                }
                if (whole)
                    finish_lse(h, top, sum_l);
                else if (lane == 0)
                    *reinterpret_cast<float2 *>(pc.at_ml(piece, h)) = make_float2(top, sum_l);
            }
            if (!whole) {
                // the blocks that hold a piece, from the one with the unit's
                // first tile (its second piece) to the one with its last
                // (their first pieces), sixteen to a bunch
                const int c0 = (int)(((ubeg + 1) * G + total - 1) / total - 1);
                const int c1 = (int)((uend * G + total - 1) / total - 1);
                const int bunches = (c1 - c0) / kFan + 1, bunch = ((int)blockIdx.x - c0) / kFan;
                const int b0 = c0 + bunch * kFan, count = min(kFan, c1 - b0 + 1);
                auto piece_of = [&](int b) { return 2 * (int64_t)b + (b == c0 ? 1 : 0); };
                auto arrive = [&](uint32_t *ctr, int of) {   // whether this block is the last of `of`
                    __threadfence();
                    __syncthreads();
                    if (tid == 0) {
                        const bool is = atomicAdd(ctr, 1u) == (uint32_t)of - 1;
                        if (is)
                            *ctr = 0;
                        last = is;
                    }
                    __syncthreads();
                    if (!last)
                        return false;
                    __threadfence();
                    return true;
                };
                auto join_all = [&](int count, auto from, bool out) {
                    for (int h = warp; h < heads; h += W) {
                        float4 x[DP > 128 ? 2 : 1];
                        float top, sum_l;
                        join<DP>(pc, count, h, from, x, top, sum_l);
                        const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
#pragma unroll
                        for (int q = 0; q < (DP > 128 ? 2 : 1); ++q) {
                            const int c = 4 * lane + 128 * q;
                            if (c >= D)
                                continue;
                            if (out)
                                finish(h, c, x[q], inv);
                            else
                                *reinterpret_cast<float4 *>(pc.at_o(piece_of(b0), h) + c) = x[q];
                        }
                        if (out)
                            finish_lse(h, top, sum_l);
                        else if (lane == 0)
                            *reinterpret_cast<float2 *>(pc.at_ml(piece_of(b0), h)) = make_float2(top, sum_l);
                    }
                };
                if (arrive(ctr + piece_of(b0), count)) {
                    join_all(count, [&](int i) { return piece_of(b0 + i); }, bunches == 1);
                    if (bunches > 1 && arrive(ctr + 2 * kMaxCtas + c0, bunches))
                        join_all(bunches, [&](int i) { return piece_of(c0 + i * kFan); }, true);
                }
            }
            __syncthreads();   // the stages and sums are read
            fresh = true;
        }
        use.next(a, units);
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
}

int padded(int64_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

template <int DT, int DP>
cudaError_t launch(const PagedAttention &a, uint32_t *err, cudaStream_t stream)
{
    using S = Shape<DT, DP>;
    auto *k = k_paged_attention<DT, DP>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    int dev = 0, sms = 0;
    if (e == cudaSuccess)
        e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    // As many blocks as are resident; no more than tiles that the block table
    // can hold.
    const int64_t group = a.heads / a.cache.kv_heads;
    const int64_t units = a.cache.kv_heads * ceil_div(group, kHeads);
    const int64_t span = a.max_pages * a.cache.page_size;
    const int64_t tiles = a.requests * units * ceil_div(span < INT32_MAX ? span : INT32_MAX, S::kTile);
    int64_t grid = (int64_t)sms * S::kBlocks;
    grid = grid < kMaxCtas ? grid : kMaxCtas;
    grid = grid < tiles ? grid : tiles;
    k<<<(unsigned)grid, S::kThreads, S::kSmem, stream>>>(a, err);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_type(const PagedAttention &a, uint32_t *err, cudaStream_t stream)
{
    switch (padded(a.cache.head_dim)) {
    case 64: return launch<DT, 64>(a, err, stream);
    case 128: return launch<DT, 128>(a, err, stream);
    default: return launch<DT, 256>(a, err, stream);
    }
}

}  // namespace

// Counters (one per piece, one per block), then maxima and sums, then sums of
// values of two pieces per block: the first and the last of its run.
int64_t paged_attention_ws_bytes(int64_t head_dim)
{
    return kMaxCtas * 3 * 4 + (int64_t)kMaxCtas * 2 * kHeads * 4 * (2 + padded(head_dim));
}

cudaError_t launch_paged_attention(const PagedAttention &a, uint32_t *err, cudaStream_t stream)
{
    switch ((int)a.cache.dtype) {
    case TW_KV_BF16: return launch_type<TW_KV_BF16>(a, err, stream);
    case TW_KV_F16: return launch_type<TW_KV_F16>(a, err, stream);
    default: return launch_type<TW_KV_I8>(a, err, stream);
    }
}

}  // namespace tw
