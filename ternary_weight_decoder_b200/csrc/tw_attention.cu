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
// joined in a fixed order, each head by the half warp that finishes it last,
// kFan pieces at a time and then those.  Inside a block each warp takes 16 keys (32
// of short rows) of every tile through its own ring of cp.async stages: no barrier
// until a piece ends.
//
// Matrix products: the 16 keys (or 16 columns of the values) are the rows of
// an MMA, eight query heads its columns, so no lane computes for nobody:
// scores^T = K q^T, out^T = V^T w^T.  The operands that are not in the cache
// are carried in parts, each the rounding of what the last one left: two of
// fp16 (22 bits), three of bf16 (24 bits); queries on codes in three int8
// digits (23 bits of the head's largest), whose products are exact integers.
// Scores and sums are fp32.  Groups of more than eight heads are split into
// units of eight, which read their keys again (from L2, mostly).
//
// Measured on B200 (12 heads over 2 KV heads of 128): past the first 262144
// keys of one request, another 262144 take 37 .. 41 us of bf16 or fp16 (6.6 ..
// 7.2 TB/s, of which L2 gives some) and 21.9 us of codes with their scales (6.3
// TB/s), the memory's rate; what is left is the start (scanning lengths, looking
// up pages, the first keys: about 5 us) and the joins (2 to 6 us).
#include <cfloat>

#include "tw_kv.cuh"

namespace tw {
namespace {

constexpr int kMaxCtas = 512;                // counters and partial results in the workspace
constexpr int kHeads = 8;                    // query heads of a unit
constexpr int kFan = 16;                     // pieces that half a warp joins, of one head
constexpr int kMinTile = 96;                 // keys of the smallest variant's tile
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
// The least log2 of a value's scale, as far as the running maximum goes: a key
// with a smaller one, or 0, adds to the sum of weights and hardly to the values.
// So low that the others' weights times scales keep their bits unless they are
// below 2^-80 of such a key's weight; not lower, as that is then 2^(80 + 12 + 3)
// at most, and the fp32 sum of 2^31 of them finite.
constexpr float kLeastScale = -80.f;

// A call, as the kernel reads it.
struct Args {
    // KV head and first of its query heads of a unit
    __device__ __forceinline__ int kv_of(int u) const { return per_kv == 1 ? u : u / per_kv; }
    __device__ __forceinline__ int skip_of(int u, int kv) const { return (u - kv * per_kv) * kHeads; }

    const float *q;
    float *out, *lse;
    const int32_t *table, *lengths, *first;
    const uint8_t *k;
    int64_t v_of_k;                  // bytes from the keys to the values
    const float *k_scale, *v_scale;
    uint8_t *ws;
    uint32_t *err;
    int64_t ldq, ldo, table_stride;
    int64_t page_bytes, row_bytes, head_bytes;
    int requests, heads, kv_heads, group;
    int per_kv, units;               // units of eight heads per KV head, and in all
    int D, P, page_shift;            // page_shift: log2 P, or -1
    int cap, pages;                  // keys that a table row can name, pages of the pools
    int short_way;                   // 16 keys share a page, byte strides below 2^32
    float mul;                       // scale * log2 e
};

// The shape of one variant: DP columns (head_dim rounded up) of type DT.
template <int DT, int DP>
struct Shape {
    static constexpr bool kCodes = DT == TW_KV_I8;
    static constexpr bool kBf = DT == TW_KV_BF16;
    static constexpr int kParts = kBf ? 3 : 2;         // of a weight
    static constexpr int kElem = kCodes ? 1 : 2;
    static constexpr int kRow = DP * kElem;            // bytes of a key
    static constexpr int kChunks = kRow / 16;
    // Keys of a warp's step: twice 16 where rows are short (codes, up to 64
    // columns), so that its fixed instructions count for less.  14 heads over 2
    // of 64 columns: 119 requests of 121 .. 231 keys 9.9 us (16 a step: 12.8),
    // 14 of 11500 .. 73268 49.1 us (50.7); but 212 of 24 .. 32 over 8 heads
    // 20.4 us (17.4), as fewer steps are on their way (the host, which chooses,
    // does not know the lengths).
    static constexpr int kHalves = kCodes || DP <= 64 ? 2 : 1;
    static constexpr int kKeys = 16 * kHalves;
    static constexpr uint32_t kAll = kHalves == 2 ? 0xffffffffu : 0xffffu;
    static constexpr int kPool = kKeys * kRow;         // bytes of a step's keys
    static constexpr int kStage = 2 * kPool;
    static constexpr int kScales = kCodes ? 2 * kKeys * 4 : 0;   // of a stage, behind the rings
    static constexpr int kSteps = DP / 16;             // 16 columns of values each
    static constexpr int kQueryParts = kBf || kCodes ? 3 : 2;
    static constexpr int kQuerySteps = kCodes ? DP / 32 : DP / 16;   // MMA steps over a key
    // The running maximum is raised once a score passes it by this much (in
    // powers of two), so that most steps leave the sums alone.  Weights are
    // then up to 2^slack; fp16 ones are carried times 2^12 (as is the sum),
    // so that the second part of small ones stays clear of fp16's smallest
    // number and large ones below its largest.
    static constexpr float kSlack = kBf ? 8.f : 3.f, kUp = kBf ? 0.f : 12.f;
    // Two blocks of six warps on an SM: while one ends a piece (a few thousand
    // cycles of latencies) the other streams.  256 requests of 512 .. 16384
    // keys of codes: 129 us, against 143 us with one block of twelve; 512 of
    // 20 .. 300 bf16 keys: 30.7 / 41.2 us; one of 131072: 34.3 / 36.7 us.
    // Rows of more than 128 columns take a whole SM's shared memory.
    static constexpr int kWarps = 6;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTile = kKeys * kWarps;
    static constexpr int kBlocks = DP > 128 ? 1 : 2;   // resident on an SM
    static constexpr int kQueryBytes = kQuerySteps * kQueryParts * 32 * 8;   // a unit's queries, as operands
    static constexpr int kRoom = (227 * 1024) / kBlocks - 3 * 1024 - kQueryBytes;
    static constexpr int kFit = kRoom / (kWarps * (kStage + kScales));
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = kWarps * kStages * (kStage + kScales) + kQueryBytes;
    static_assert(kStages >= 2, "two stages at least");
    static_assert(kFan * DP * 4 <= kStage, "a stage holds a warp's sums, or kFan pieces of one head");
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

// Element c of a row of the cache.
template <int DT>
__device__ __forceinline__ float element(const uint8_t *row, int c)
{
    if (DT == TW_KV_I8)
        return reinterpret_cast<const int8_t *>(row)[c];
    if (DT == TW_KV_BF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[c]);
    return __half2float(reinterpret_cast<const __half *>(row)[c]);
}

// The visible keys of a request, as tiles.
struct Span {
    int lo, hi, first_tile, tiles;
};

template <int TILE>
__device__ __forceinline__ Span span_of(const Args &a, int length, int first)
{
    Span s;
    s.hi = min(length, a.cap);
    s.lo = max(first, 0);
    s.first_tile = s.lo / TILE;
    s.tiles = s.hi > s.lo ? (s.hi - 1) / TILE + 1 - s.first_tile : 0;
    return s;
}

template <int TILE>
__device__ __forceinline__ Span span_of(const Args &a, int r)
{
    return span_of<TILE>(a, a.lengths[r], a.first ? a.first[r] : 0);
}

// A place in the run of tiles: tile t of unit u of request r.
template <int TILE>
struct Cursor {
    int r, u, t;
    Span s;
    int length, first;   // of request r + 1, read on entering r
    __device__ __forceinline__ void ahead(const Args &a)
    {
        if (r + 1 < a.requests) {
            length = a.lengths[r + 1];
            first = a.first ? a.first[r + 1] : 0;
        }
    }
    // One tile on; whether that is another unit.
    __device__ __forceinline__ bool next(const Args &a)
    {
        if (++t < s.tiles)
            return false;
        t = 0;
        if (++u < a.units)
            return true;
        u = 0;
        do {
            if (++r >= a.requests)
                return true;
            s = span_of<TILE>(a, length, first);
            ahead(a);
        } while (s.tiles == 0);
        return true;
    }
};

// Count one up at device scope, ordering what this thread has seen written
// before it and what it reads after it.
__device__ __forceinline__ uint32_t count_up(uint32_t *ctr)
{
    uint32_t was;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(was) : "l"(ctr) : "memory");
    return was;
}

// The pieces of one unit in the workspace: maxima and sums [piece][head][2],
// sums of values [piece][head][DP].
template <int DP>
struct Pieces {
    float *ml, *o;
    __device__ __forceinline__ float *at_ml(int64_t piece, int h) const { return ml + (piece * kHeads + h) * 2; }
    __device__ __forceinline__ float *at_o(int64_t piece, int h) const { return o + (piece * kHeads + h) * DP; }
};

// How `total` tiles fall to G blocks: the first `more` take one more than `each`.
struct Split {
    uint32_t each, more;
    __device__ __forceinline__ Split(uint32_t total, uint32_t G) : each(total / G), more(total - each * G) {}
    __device__ __forceinline__ uint32_t begin(uint32_t block) const { return block * each + min(block, more); }
    __device__ __forceinline__ int block_of(uint32_t tile) const
    {
        const uint32_t cut = more * (each + 1);
        const bool low = tile < cut;
        const uint32_t q = (low ? tile : tile - cut) / (low ? each + 1 : each);
        return (int)(low ? q : more + q);
    }
};

// A warp's keys of one piece, for it to sum in whole fp32 numbers.
struct Whole {
    Span s;
    int r, kv, h0, heads;        // request, KV head, first query head, query heads
    int tile, last;              // from which tile to which
};

// Where a warp's stage holds column c of head h: permuted by the head against
// bank conflicts.
template <int DP>
__device__ __forceinline__ int sum_at(int h, int c)
{
    return h * DP + (c ^ ((h >> 1) << 3));
}

// The maxima, sums of weights (2^up-fold) and sums of values of a piece's keys,
// head by head, with nothing carried in parts.
template <int DT, int DP>
__device__ __forceinline__ void whole_numbers(const Args &a, const Whole &u, float *sums, float *maxima, float *weights)
{
    using S = Shape<DT, DP>;
    constexpr int kCols = DP / 32, kTogether = DP > 128 ? 2 : 4;   // (keys)
    constexpr float kUp = S::kUp;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = kCols * lane, D = a.D;   // this lane's columns, and queries
    const int32_t *table = a.table + u.r * a.table_stride;
#pragma unroll 1
    for (int h = 0; h < u.heads; ++h) {
        const float *row = a.q + u.r * a.ldq + (int64_t)(u.h0 + h) * D;
        float q[kCols], x[kCols], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < kCols; ++e)
            q[e] = c0 + e < D ? row[c0 + e] * a.mul : 0.f, x[e] = 0.f;
#pragma unroll 1
        for (int i = 0; i < (u.last + 1 - u.tile) * S::kKeys && l == l; i += kTogether) {   // (NaN: so is all else)
            const int j0 = (u.tile + i / S::kKeys) * S::kTile + warp * S::kKeys + i % S::kKeys;
            const uint8_t *at_k[kTogether];
            float score[kTogether], v_scale[kTogether];
            bool some[kTogether];
#pragma unroll
            for (int k = 0; k < kTogether; ++k) {
                const int j = j0 + k, p = max(j, 0) / a.P, in = j - p * a.P;
                const int page = j >= u.s.lo && j < u.s.hi ? __ldg(table + p) : -1;
                some[k] = (uint32_t)page < (uint32_t)a.pages;
                at_k[k] = a.k + u.kv * a.head_bytes + (some[k] ? page * a.page_bytes + in * a.row_bytes : 0);
                float k_scale = 1.f;
                v_scale[k] = 1.f;
                if (S::kCodes) {
                    const int64_t at = (some[k] ? (int64_t)page * a.P + in : 0) * a.kv_heads + u.kv;
                    k_scale = a.k_scale[at], v_scale[k] = a.v_scale[at];
                }
                score[k] = 0.f;
#pragma unroll
                for (int e = 0; e < kCols; ++e)
                    if (some[k] && c0 + e < D)
                        score[k] = fmaf(q[e], element<DT>(at_k[k], c0 + e), score[k]);
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    score[k] += __shfl_xor_sync(0xffffffffu, score[k], o);
                score[k] *= k_scale;
            }
#pragma unroll
            for (int k = 0; k < kTogether; ++k) {
                if (!some[k])
                    continue;
                const float top = fmaxf(m, score[k]), f = top == m ? 1.f : ex2(m - top);
                const float w = ex2(score[k] - (top == -INFINITY ? 0.f : top) + kUp);
                m = top, l = fmaf(l, f, w);
#pragma unroll
                for (int e = 0; e < kCols; ++e)
                    if (c0 + e < D)
                        x[e] = fmaf(x[e], f, w * v_scale[k] * element<DT>(at_k[k] + a.v_of_k, c0 + e));
            }
        }
#pragma unroll
        for (int e = 0; e < kCols; ++e)
            sums[sum_at<DP>(h, c0 + e)] = x[e];
        if (lane == 0)
            maxima[h] = m, weights[h] = l;
    }
}

template <int DT, int DP>
__global__ void __launch_bounds__(Shape<DT, DP>::kThreads, Shape<DT, DP>::kBlocks)
    k_paged_attention(const Args a)
{
    using S = Shape<DT, DP>;
    constexpr bool BF = S::kBf;
    constexpr int W = S::kWarps, H = S::kHalves, kThreads = S::kThreads, kTile = S::kTile;
    constexpr float kSlack = S::kSlack, kUp = S::kUp;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t part[W];
    __shared__ int start[3];
    __shared__ uint32_t bounds[2];
    __shared__ float sm_m[W][kHeads], sm_l[W][kHeads], sm_back[kHeads];
    __shared__ uint32_t sm_mask[W][S::kStages];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int D = a.D;
    // Work per head goes to half warps, so that eight heads take one turn (eight
    // heads of one KV head, 5 requests of 4582 .. 9357 keys: 15.6 us, a warp a
    // head 21.9 us; six heads alike): this lane's head there, and its place.
    const int half_h = 2 * warp + (lane >> 4), half_lane = lane & 15;
    static_assert(2 * W >= kHeads, "a half warp for each head");

    // rows without keys
    auto clear_rows = [&] {
        for (int r = blockIdx.x; r < a.requests; r += gridDim.x) {
            if (span_of<kTile>(a, r).tiles)
                continue;
            for (int c = tid; c < a.heads * D; c += kThreads)
                a.out[r * a.ldo + c] = 0.f;
            if (a.lse)
                for (int h = tid; h < a.heads; h += kThreads)
                    a.lse[(int64_t)r * a.heads + h] = -INFINITY;
        }
    };

    // ---- this block's run of tiles: lengths are scanned by every block
    const int per = (a.requests + kThreads - 1) / kThreads;
    const int rlo = min(tid * per, a.requests), rhi = min(rlo + per, a.requests);
    uint32_t sum = 0;
#pragma unroll 1
    for (int r = rlo; r < rhi; ++r) {
        sum += span_of<kTile>(a, r).tiles;
        if (blockIdx.x == 0 && a.lengths[r] > a.cap)
            atomicOr(a.err, EFLAG_BADDESC);
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += u;
    }
    if (lane == 31)
        part[warp] = incl;
    __syncthreads();
    uint32_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += w < warp ? part[w] : 0;
        total += part[w];
    }
    total *= a.units;
    const uint32_t G = min(gridDim.x, total);   // blocks with tiles
    const Split split(total, max(G, 1u));
    uint32_t begin = split.begin(min(blockIdx.x, G)), end = split.begin(min(blockIdx.x + 1, G));
    // A run that would end within `near` tiles of a unit's edge ends there, for
    // this block and its neighbour alike: a few tiles more or less cost less
    // than another piece (256 requests on codes: 127.7 us, 128.4 us without;
    // with up to half a run 174.8 us).  Runs of one to four tiles (near = 0): one
    // whose last tile alone, or whose first alone, is another unit's than the
    // others leaves it to its neighbour, the last of two such ends only, so that
    // each run keeps a tile (25 requests of 12 .. 4404 keys, 8 heads of 256 over
    // one: 16.1 us, 18.5 us without; 64 of 200 .. 600, 12 over 2: 12.9, 14.5).
    const uint32_t near = min(split.each / 4, 3u);
    const bool alone = split.each == 1 && split.more == 0;   // a tile a block
    if (begin < end) {
        const uint32_t mine = before * a.units, past = (before + sum) * a.units;
        if (tid == 0 && (alone || end == total))
            bounds[1] = end;
#pragma unroll 1
        for (int k = 0; k < (alone ? 1 : 2); ++k) {
            const uint32_t at = k ? end : begin;
            if (at < mine || at >= past)
                continue;
            uint32_t in = at - mine;
            Cursor<kTile> c;
            for (c.r = rlo;; ++c.r) {
                c.s = span_of<kTile>(a, c.r);
                if (in < c.s.tiles * a.units)
                    break;
                in -= c.s.tiles * a.units;
            }
            c.u = in / c.s.tiles, c.t = in % c.s.tiles;
            uint32_t to = at;
            bool down = 2 * c.t < c.s.tiles, snap = (down ? c.t : c.s.tiles - c.t) <= near;
            if (near == 0) {
                const uint32_t edge = blockIdx.x + k;   // this run's begin or end, among all runs' (0: c.t is 0)
                down = c.t == 1 && split.begin(edge - 1) + 1 < at;
                snap = down || (c.t + 1 == c.s.tiles && split.begin(min(edge + 1, G)) >= at + 3);
            }
            if (c.t && snap) {
                to = down ? at - c.t : at + c.s.tiles - c.t;
                c.t = down ? 0 : c.s.tiles - 1;
                if (!down) {
                    c.ahead(a);
                    c.next(a);
                }
            }
            bounds[k] = to;
            if (k == 0)
                start[0] = c.r, start[1] = c.u, start[2] = c.t;
        }
    }
    __syncthreads();
    if (begin < end)
        begin = bounds[0], end = bounds[1];
    if (begin >= end) {
        clear_rows();
        return;
    }
    Cursor<kTile> load, use;
    load.r = start[0], load.u = start[1], load.t = start[2];
    load.s = span_of<kTile>(a, load.r);
    load.ahead(a);
    use = load;

    // ---- the ring of stages
    constexpr int kRowsPer = S::kChunks >= 32 ? 1 : 32 / S::kChunks;   // rows of one pass of the warp
    constexpr bool kWide = S::kChunks >= 32;                           // a pass is a row: all lanes stay in step
    const uint32_t ring = smem_u32(smem) + warp * S::kStages * S::kStage;
    const uint32_t scales = smem_u32(smem) + W * S::kStages * S::kStage + warp * S::kStages * S::kScales;
    const int row0 = lane / S::kChunks, chunk = lane % S::kChunks;
    const uint32_t lane_dst = ring + place<S::kChunks>(row0, chunk);
    const bool in_row = chunk < D * S::kElem / 16;
    // Of the unit that is being fetched: its table row, its head's pools.
    const int32_t *table;
    const uint8_t *kpool;
    int head;
    auto enter_unit = [&] {
        head = a.kv_of(load.u);
        table = a.table + load.r * a.table_stride;
        kpool = a.k + head * a.head_bytes + row0 * a.row_bytes + chunk * 16;
        // its queries are on their way to L1 while its keys are fetched
        const int skip = a.skip_of(load.u, head);
        const float *row = a.q + load.r * a.ldq + (int64_t)(head * a.group + skip + half_h) * D;
        if (half_h < min(kHeads, a.group - skip))
#pragma unroll
            for (int c = 8 * half_lane; c < DP; c += 128)
                if (c < D)
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(row + c));
    };
    // The next step's first key and, for every 16 keys of which some are
    // visible, their page (the short way: pages hold whole sixteens of keys),
    // looked up a step early.
    int next_j = 0, next_in[H] = {}, next_page[H];
    auto look_up = [&] {
        next_j = (load.s.first_tile + load.t) * kTile + warp * S::kKeys;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int j = next_j + 16 * h;
            next_page[h] = -1;
            if (a.short_way && j < load.s.hi && j + 16 > load.s.lo) {
                const int p = a.page_shift >= 0 ? j >> a.page_shift : j / a.P;
                next_in[h] = j - p * a.P;
                next_page[h] = __ldg(table + p);
            }
        }
    };
    uint32_t partial = 0;   // stages with keys left out: their masks are in sm_mask
    auto fetch = [&](int stage) {
        const uint32_t base = stage * S::kStage;
        uint32_t mask = 0;
        int64_t slot = -1;   // codes: this lane's key
        auto half = [&](int h, int page0, int in0) {
            const uint32_t rows = base + h * 16 * S::kRow;
            // Sixteen keys of which none is taken: their weights are 0, and 0
            // times what the stage holds has to be (codes are finite).  A whole
            // step of these is passed over.
            auto no_values = [&] {
                if (!S::kCodes && H == 2)
                    for (int i = 0; i < 16 / kRowsPer; ++i)
                        cp_async16(ring + rows + place<S::kChunks>(row0 + kRowsPer * i, chunk) + S::kPool, a.k, false);
            };
            if (a.short_way) {
                // visible keys of the sixteen, from which to which
                const int from = max(load.s.lo - next_j - 16 * h, 0), to = min(load.s.hi - next_j - 16 * h, 16);
                if (from >= to) {
                    no_values();
                    return;
                }
                if ((uint32_t)page0 >= (uint32_t)a.pages) {
                    if (lane == 0)
                        atomicOr(a.err, EFLAG_BADDESC);
                    no_values();
                    return;
                }
                const uint8_t *ks = kpool + (uint64_t)(uint32_t)page0 * (uint32_t)a.page_bytes +
                                    (uint64_t)(uint32_t)in0 * (uint32_t)a.row_bytes;
                const uint8_t *vs = ks + a.v_of_k;
                if (S::kCodes && (lane >> 4) == h && (lane & 15) >= from && (lane & 15) < to)
                    slot = (uint32_t)(page0 * a.P + in0) + (lane & 15);
                if (to - from == 16 && (kWide || in_row)) {
                    mask |= 0xffffu << (16 * h);
#pragma unroll
                    for (int i = 0; i < 16 / kRowsPer; ++i) {
                        const uint32_t dst = (lane_dst + rows) ^ (row_swap<S::kChunks>(kRowsPer * i) << 4);
                        cp_async16(dst + kRowsPer * i * S::kRow, !kWide || in_row ? ks : a.k, !kWide || in_row);
                        cp_async16(dst + kRowsPer * i * S::kRow + S::kPool, !kWide || in_row ? vs : a.k,
                                   !kWide || in_row);
                        ks += kRowsPer * a.row_bytes, vs += kRowsPer * a.row_bytes;
                    }
                } else {   // zeros for keys that are not visible and columns past head_dim
                    mask |= (0xffffu >> (16 - to + from)) << (16 * h + from);
#pragma unroll 1
                    for (int i = 0; i < 16 / kRowsPer; ++i) {
                        const uint32_t dst = (lane_dst + rows) ^ (row_swap<S::kChunks>(kRowsPer * i) << 4);
                        const int row = row0 + kRowsPer * i;
                        const bool in = in_row && row >= from && row < to;
                        cp_async16(dst + kRowsPer * i * S::kRow, in ? ks : a.k, in);
                        cp_async16(dst + kRowsPer * i * S::kRow + S::kPool, in ? vs : a.k, in);
                        ks += kRowsPer * a.row_bytes, vs += kRowsPer * a.row_bytes;
                    }
                }
                return;
            }
            const int j = next_j + 16 * h + (lane & 15);
            bool ok = j >= load.s.lo && j < load.s.hi;
            int64_t off = 0;
            if (ok) {
                const int p = j / a.P;
                const int page = __ldg(table + p);
                if ((uint32_t)page < (uint32_t)a.pages) {
                    const int in = j - p * a.P;
                    off = page * a.page_bytes + in * a.row_bytes;
                    if (S::kCodes && (lane >> 4) == h)
                        slot = (int64_t)page * a.P + in;
                } else {
                    ok = false;
                    atomicOr(a.err, EFLAG_BADDESC);
                }
            }
            const uint32_t some = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            mask |= some << (16 * h);
#pragma unroll 1
            for (int i = 0; i < 16 / kRowsPer; ++i) {
                const int row = row0 + kRowsPer * i;
                const int64_t o = __shfl_sync(0xffffffffu, off, row) - row0 * a.row_bytes;
                const bool in = ((some >> row) & 1) && in_row;
                const uint32_t dst = ring + rows + place<S::kChunks>(row, chunk);
                cp_async16(dst, in ? kpool + o : a.k, in);
                cp_async16(dst + S::kPool, in ? kpool + a.v_of_k + o : a.k, in);
            }
        };
        half(0, next_page[0], next_in[0]);
        if constexpr (H == 2)
            half(1, next_page[H - 1], next_in[H - 1]);
        if (S::kCodes) {
            const uint32_t dst = scales + stage * S::kScales + lane * 4;
            const int64_t at = slot < 0 ? 0 : slot * a.kv_heads + head;
            cp_async4(dst, a.k_scale + at, slot >= 0);
            cp_async4(dst + S::kKeys * 4, a.v_scale + at, slot >= 0);
        }
        partial &= ~(1u << stage);
        if (mask != S::kAll) {
            partial |= 1u << stage;
            if (lane == 0)
                sm_mask[warp][stage] = mask;
        }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    // ---- sums of a unit, whole or in pieces
    struct Unit {
        int r, h0, heads;         // request, first query head, heads (0: none)
        uint32_t beg, end;        // its tiles
    };
    Unit before_it{}, after{};    // this block's pieces: of a unit that began before its run, or ends after it
    Pieces<DP> pc;
    pc.ml = reinterpret_cast<float *>(a.ws) + 3 * kMaxCtas * kHeads;
    pc.o = pc.ml + kMaxCtas * 2 * 2 * kHeads;
    // Column c of head h into the output, or into a piece.
    auto put = [&](const Unit &u, bool out, int piece, int h, int c, float4 x, float inv) {
        float *to = out ? a.out + u.r * a.ldo + (int64_t)(u.h0 + h) * D : pc.at_o(piece, h);
        *reinterpret_cast<float4 *>(to + c) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    };
    auto put_sum = [&](const Unit &u, bool out, int piece, int h, float top, float sum_l) {
        if (!out)
            *reinterpret_cast<float2 *>(pc.at_ml(piece, h)) = make_float2(top, sum_l);
        else if (a.lse)
            a.lse[(int64_t)u.r * a.heads + u.h0 + h] = sum_l == 0.f ? -INFINITY : (top - kUp) * kLn2 + logf(sum_l);
    };
    // Maximum and sum over the parts that a half warp's lanes hold, two each,
    // and each part's factor.
    auto over_parts = [&](const float2 (&ml)[2], float (&f)[2], float &top, float &sum_l) {
        top = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
        for (int x = 8; x; x >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        sum_l = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            f[k] = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - top);
            sum_l += ml[k].y != ml[k].y ? ml[k].y : ml[k].y * f[k];   // (a NaN sum without a maximum stays one)
        }
#pragma unroll
        for (int x = 8; x; x >>= 1)
            sum_l += __shfl_xor_sync(0xffffffffu, sum_l, x);
    };
    const float2 no_part = make_float2(-INFINITY, 0.f);
    auto add = [](float4 &x, float4 y, float w) {
        x.x = fmaf(y.x, w, x.x), x.y = fmaf(y.y, w, x.y);
        x.z = fmaf(y.z, w, x.z), x.w = fmaf(y.w, w, x.w);
    };
    constexpr int kQuads = DP / 64;   // a lane's fours of columns: 4 * half_lane + 64 * q
    // The warps' parts, in stage `at_stage` of each.
    float odd = 0.f;   // NaN once a sum was, or was infinite
    auto join_warps = [&](const Unit &u, bool whole, int piece, int at_stage) {
        if (2 * warp >= u.heads)
            return;
        const int h = min(half_h, u.heads - 1);   // (two halves of the last head write the same)
        const float2 ml[2] = {half_lane < W ? make_float2(sm_m[half_lane % W][h], sm_l[half_lane % W][h]) : no_part,
                              no_part};
        float f[2], top, sum_l;
        over_parts(ml, f, top, sum_l);
        const float inv = !whole ? 1.f : sum_l == 0.f ? 0.f : 1.f / sum_l;
        float4 x[kQuads];
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
            x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float fw = __shfl_sync(0xffffffffu, f[0], w, 16);
            const uint8_t *part_w = smem + (w * S::kStages + at_stage) * S::kStage;
#pragma unroll
            for (int q = 0; q < kQuads; ++q)
                add(x[q], *reinterpret_cast<const float4 *>(part_w + sum_at<DP>(h, 4 * half_lane + 64 * q) * 4), fw);
        }
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            odd = fmaf(x[q].x, 0.f, fmaf(x[q].y, 0.f, fmaf(x[q].z, 0.f, fmaf(x[q].w, 0.f, odd))));
            if (4 * half_lane + 64 * q < D)
                put(u, whole, piece, h, 4 * half_lane + 64 * q, x[q], inv);
        }
        if (half_lane == 0)
            put_sum(u, whole, piece, h, top, sum_l);
    };

    // Queries as the MMA's B operand, in parts: [step][part][lane] the two
    // words that a lane feeds for head lane / 4 of the unit.
    uint2 *qs = reinterpret_cast<uint2 *>(smem + W * S::kStages * (S::kStage + S::kScales));
    float o[S::kSteps][4];           // (columns g, g + 8 of 16) x (heads 2 t4, 2 t4 + 1)
    float m[2], l[2], unscale[2];    // of heads 2 t4, 2 t4 + 1
    const int n = (int)(end - begin);
    int stage = 0;
    bool fresh = true, any_odd = false;
    enter_unit();
    look_up();
#pragma unroll 1
    for (int i = 1 - S::kStages; i < n; ++i) {
        // ---- a stage ahead
        if (i >= 0) {
            cp_async_wait<S::kStages - 2>();
            __syncwarp();   // every lane's copies of this stage are here, the last stage is read
        }
        if (i + S::kStages - 1 < n) {
            fetch(i < 0 ? i + S::kStages - 1 : stage == 0 ? S::kStages - 1 : stage - 1);
            if (i + S::kStages < n) {
                if (load.next(a))
                    enter_unit();
                look_up();
            }
        }
        commit();
        if (i < 0)
            continue;

        // ---- a new piece: its queries, split
        if (fresh) {
            const int kv = a.kv_of(use.u), skip = a.skip_of(use.u, kv);
            const int h0 = kv * a.group + skip, heads = min(kHeads, a.group - skip);
            if (const int h = half_h; h < kHeads) {   // (whole warps)
                const float *row = a.q + use.r * a.ldq + (int64_t)(h0 + h) * D;
                float x[kQuads][4];
                float top = 0.f, poison = 0.f;   // poison: NaN if a query is, or is infinite
#pragma unroll
                for (int q = 0; q < kQuads; ++q) {
                    const int c = 4 * half_lane + 64 * q;
                    const float4 v = h < heads && c < D ? *reinterpret_cast<const float4 *>(row + c)
                                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[q][0] = v.x * a.mul, x[q][1] = v.y * a.mul, x[q][2] = v.z * a.mul, x[q][3] = v.w * a.mul;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top = fmaxf(top, fabsf(x[q][k])), poison = fmaf(x[q][k], 0.f, poison);
                }
                float norm = 1.f, back = 1.f;
                if (!BF) {
                    // fp16 operands: the head's largest query is brought to 2^14
                    // by a power of two, so that no part leaves the range.  For
                    // codes it is brought below 2^23 - 2^15, the most that three
                    // balanced digits of eight bits hold, and rounded there.
#pragma unroll
                    for (int s = 8; s; s >>= 1) {
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                        poison += __shfl_xor_sync(0xffffffffu, poison, s);
                    }
                    const bool some = top > 0.f && top <= FLT_MAX;
                    constexpr int kAt = S::kCodes ? 22 : 14;
                    const int e = min(max((int)(__float_as_uint(S::kCodes ? top * 1.0078125f : top) >> 23) - 127, -100), 127);
                    norm = some ? __uint_as_float((uint32_t)(127 + kAt - e) << 23) : 1.f;
                    back = (some ? __uint_as_float((uint32_t)(127 - kAt + e) << 23) : 1.f) + poison;
                }
                if (half_lane == 0)
                    sm_back[h] = back;
#pragma unroll
                for (int q = 0; q < kQuads; ++q) {
                    const int c = 4 * half_lane + 64 * q;   // columns c .. c + 3
                    if constexpr (S::kCodes) {
                        uint32_t word[3] = {0, 0, 0};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            int v = __float2int_rn(x[q][e] * norm);   // = 2^16 d0 + 2^8 d1 + d2
#pragma unroll
                            for (int k = 2; k >= 0; --k) {
                                const int d = k ? ((v + 128) & 255) - 128 : v;
                                word[k] |= (uint32_t)(d & 255) << (8 * e);
                                v = (v - d) >> 8;
                            }
                        }
                        // step c / 32, half (c / 16) % 2, lane 4 h + (c / 4) % 4
                        uint32_t *to = reinterpret_cast<uint32_t *>(qs + (c / 32) * 3 * 32 + 4 * h + (c / 4) % 4) +
                                       (c / 16) % 2;
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            to[k * 64] = word[k];
                    } else {
                        // step c / 16, half (c / 8) % 2, lanes 4 h + (c / 2) % 4 + {0, 1}
                        uint32_t *to = reinterpret_cast<uint32_t *>(qs + (c / 16) * S::kQueryParts * 32 + 4 * h +
                                                                    (c / 2) % 4) + (c / 8) % 2;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[q][e] *= norm;
#pragma unroll
                        for (int k = 0; k < S::kQueryParts; ++k) {
                            to[k * 64] = split2<BF>(x[q][0], x[q][1]);
                            to[k * 64 + 2] = split2<BF>(x[q][2], x[q][3]);
                        }
                    }
                }
            }
            __syncthreads();
            unscale[0] = sm_back[2 * t4], unscale[1] = sm_back[2 * t4 + 1];
            m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.f;
#pragma unroll
            for (int c = 0; c < S::kSteps; ++c)
                o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
            fresh = false;
        }

        const uint32_t base = ring + stage * S::kStage;
        const uint32_t mask = (partial >> stage) & 1 ? sm_mask[warp][stage] : S::kAll;
        if (mask) {
            // ---- scores of keys g, g + 8 of 16 for heads 2 t4, 2 t4 + 1
            // (keys 0-7, 8-15) x (16 bytes at chunk 2 j, at 2 j + 1)
            const uint32_t kbase = base + place<S::kChunks>(lane & 15, lane >> 4);
            float s[H][4];
            if constexpr (S::kCodes) {
                int acc[H][3][4];
#pragma unroll
                for (int j = 0; j < S::kQuerySteps; ++j) {
                    uint32_t f[H][4];
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        ldmatrix4<false>(f[h], (kbase + h * 16 * S::kRow) ^ (j << 5));
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const uint2 v = qs[(j * 3 + k) * 32 + lane];
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            if (j == 0)
                                acc[h][k][0] = acc[h][k][1] = acc[h][k][2] = acc[h][k][3] = 0;
                            mma_s8_16832(acc[h][k], f[h][0], f[h][1], f[h][2], f[h][3], v.x, v.y);
                        }
                    }
                }
                // exact sums of each digit (below 2^23); one rounding each below
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[h][e] = fmaf((float)(acc[h][0][e] * 256 + acc[h][1][e]), 256.f, (float)acc[h][2][e]) *
                                  unscale[e & 1];
            } else {
                float acc[H][S::kQueryParts][4];
#pragma unroll
                for (int j = 0; j < S::kQuerySteps; ++j) {
                    uint32_t f[H][4];
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        ldmatrix4<false>(f[h], (kbase + h * 16 * S::kRow) ^ (j << 5));
#pragma unroll
                    for (int k = 0; k < S::kQueryParts; ++k) {
                        const uint2 v = qs[(j * S::kQueryParts + k) * 32 + lane];
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            if (j == 0)
                                acc[h][k][0] = acc[h][k][1] = acc[h][k][2] = acc[h][k][3] = 0.f;
                            mma<BF>(acc[h][k], f[h][0], f[h][1], f[h][2], f[h][3], v.x, v.y);
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[h][e] = acc[h][0][e] + acc[h][1][e];
                        if (S::kQueryParts == 3)
                            s[h][e] += acc[h][S::kQueryParts - 1][e];
                        if (!BF)
                            s[h][e] *= unscale[e & 1];
                    }
            }
            // ---- running maximum and sum.  With codes the value's scale goes
            // into the weight, 2^(s_j - m) vs_j, and into the maximum, that of
            // s_j + log2 vs_j, so that weights stay within fp16 whatever the
            // scales are (the sum of 2^(s_j - m) need not: it is fp32).
            float vs[H][2], lv[H][2];
            if (S::kCodes) {
                const float *of = reinterpret_cast<const float *>(
                    smem + W * S::kStages * S::kStage + (warp * S::kStages + stage) * S::kScales) + g;
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float ks = of[16 * h + 8 * k];
                        s[h][2 * k] *= ks, s[h][2 * k + 1] *= ks;
                        vs[h][k] = of[S::kKeys + 16 * h + 8 * k];
                        lv[h][k] = fmaxf(__log2f(vs[h][k]), kLeastScale);
                    }
            }
            if (mask != S::kAll) {
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[h][e] = (mask >> (16 * h + g + 8 * (e >> 1))) & 1 ? s[h][e] : -INFINITY;
            }
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top[e & 1] = fmaxf(top[e & 1], S::kCodes ? s[h][e] + lv[h][e >> 1] : s[h][e]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], x));
            if (__any_sync(0xffffffffu, top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float up = fmaxf(top[e], m[e]);
                    f[e] = up == -INFINITY ? 1.f : ex2(m[e] - up);
                    m[e] = up;
                    l[e] *= f[e];
                }
#pragma unroll
                for (int c = 0; c < S::kSteps; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[c][e] *= f[e & 1];
            }
            const float shift[2] = {(m[0] == -INFINITY ? 0.f : m[0]) - kUp, (m[1] == -INFINITY ? 0.f : m[1]) - kUp};
            uint32_t w[H][S::kParts][2];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(s[h][e] - shift[e & 1]);
                    l[e & 1] += p[e];
                    if (S::kCodes)
                        p[e] *= vs[h][e >> 1];
                }
#pragma unroll
                for (int k = 0; k < S::kParts; ++k) {
                    w[h][k][0] = transpose8(split2<BF>(p[0], p[1]));
                    w[h][k][1] = transpose8(split2<BF>(p[2], p[3]));
                }
            }
            // ---- weighted values: columns x heads
            if constexpr (S::kCodes) {
                // byte pairs: keys 2 t4 + {0, 1}, columns 2 g + {0, 1} of chunks
                // c, c + 1; even columns are the MMA's rows 0-7, odd ones 8-15
                const uint32_t vbase = base + S::kPool + place<S::kChunks>(lane & 15, lane >> 4);
#pragma unroll
                for (int c = 0; c < S::kSteps; c += 2)
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        uint32_t f[4];
                        ldmatrix4<true>(f, (vbase + h * 16 * S::kRow) ^ (c << 4));
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t a0 = codes2<false>(f[2 * q]), a1 = codes2<true>(f[2 * q]);
                            const uint32_t a2 = codes2<false>(f[2 * q + 1]), a3 = codes2<true>(f[2 * q + 1]);
#pragma unroll
                            for (int k = 0; k < S::kParts; ++k)
                                mma<BF>(o[c + q], a0, a1, a2, a3, w[h][k][0], w[h][k][1]);
                        }
                    }
            } else {
                // (columns 0-7, 8-15) x (keys 0-7, 8-15)
                const uint32_t vbase = base + S::kPool +
                                       place<S::kChunks>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
                for (int c = 0; c < S::kSteps; ++c)
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        uint32_t f[4];
                        ldmatrix4<true>(f, (vbase + h * 16 * S::kRow) ^ (c << 5));
#pragma unroll
                        for (int k = 0; k < S::kParts; ++k)
                            mma<BF>(o[c], f[0], f[1], f[2], f[3], w[h][k][0], w[h][k][1]);
                    }
            }
        }

        // ---- the end of a piece
        const bool unit_done = use.t + 1 == use.s.tiles;
        if (unit_done || i + 1 == n) {
            const uint32_t ubeg = begin + i - use.t, uend = ubeg + use.s.tiles;
            const int kv = a.kv_of(use.u), skip = a.skip_of(use.u, kv);
            const int h0 = kv * a.group + skip, heads = min(kHeads, a.group - skip);
            __syncwarp();   // the stage is read: it takes the warp's sums
            float *mine = reinterpret_cast<float *>(smem + (warp * S::kStages + stage) * S::kStage);
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
                        *reinterpret_cast<float2 *>(mine + sum_at<DP>(2 * t4 + h, 16 * c + 2 * g)) =
                            make_float2(o[c][h], o[c][2 + h]);
                    } else {
                        mine[sum_at<DP>(2 * t4 + h, 16 * c + g)] = o[c][h];
                        mine[sum_at<DP>(2 * t4 + h, 16 * c + g + 8)] = o[c][2 + h];
                    }
                }
            }
            const bool whole = unit_done && ubeg >= begin;
            const int mine_piece = 2 * (int)blockIdx.x + (ubeg >= begin ? 1 : 0);
            const Unit unit{use.r, h0, heads, ubeg, uend};
            __syncthreads();
            join_warps(unit, whole, mine_piece, stage);
            if (!whole)   // joined when the run is over: nothing in it waits for the counts
                (ubeg >= begin ? after : before_it) = unit;
            any_odd = __syncthreads_or(odd != odd);   // the stages and sums are read
            fresh = true;
        }
        use.next(a);
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncwarp();   // the warp's stages are its own again

    // ---- infinities.  One times the parts of a weight or a query, of which one
    // may be 0 or of the other sign, becomes NaN above: where a sum was not
    // finite, its piece comes again from whole fp32 numbers, into the same place.
    // (Looking for such sums costs 0.1 us of one short request's 8.3 us and 0.6 us
    // of 256 requests' 126.7 on codes; each warp among its own sums 3.5 us of them.)
    if (any_odd) {   // (by any thread, at the last piece's end)
        Cursor<kTile> c;
        c.r = start[0], c.u = start[1], c.t = start[2];
        c.s = span_of<kTile>(a, c.r);
        c.ahead(a);
#pragma unroll 1
        for (int left = n; left > 0;) {
            const int kv = a.kv_of(c.u), skip = a.skip_of(c.u, kv), tiles = min(c.s.tiles - c.t, left);
            const bool whole = c.t == 0 && tiles == c.s.tiles;
            const int piece = 2 * (int)blockIdx.x + (c.t == 0 ? 1 : 0);
            const Unit unit{c.r, kv * a.group + skip, min(kHeads, a.group - skip), 0, 0};
            bool again = false;
            for (int i = tid; i < unit.heads * D; i += kThreads) {
                const int h = i / D, col = i - h * D;
                const float x = whole ? a.out[unit.r * a.ldo + (int64_t)unit.h0 * D + i] : pc.at_o(piece, h)[col];
                again = again || !(fabsf(x) <= FLT_MAX);
            }
            if (__syncthreads_or(again)) {
                whole_numbers<DT, DP>(a, Whole{c.s, c.r, kv, unit.h0, unit.heads, c.s.first_tile + c.t,
                                               c.s.first_tile + c.t + tiles - 1},
                                      reinterpret_cast<float *>(smem + warp * S::kStages * S::kStage), sm_m[warp],
                                      sm_l[warp]);
                __syncthreads();
                join_warps(unit, whole, piece, 0);
                __syncthreads();
            }
            left -= tiles;
            c.t += tiles - 1;
            c.next(a);
        }
    }
    float *mine = reinterpret_cast<float *>(smem + (warp * S::kStages + (lane >> 4)) * S::kStage);
    // A unit's pieces: the second of the block with its first tile, the first
    // of the others.  kFan of them are joined into the first of them (into the
    // output if there are no more), then those; each head by the half warp that
    // counts to the last of them.
    struct Join {
        int b_first, b_last, b0, into, bunches;
    };
    auto piece_of = [](const Join &j, int b) { return 2 * b + (b == j.b_first ? 1 : 0); };
    auto join_of = [&](const Unit &u) {
        Join j;
        j.b_first = split.block_of(u.beg + near), j.b_last = split.block_of(u.end - near - 1);
        if (near == 0) {   // a neighbour may have taken over their only tile of the unit
            if (split.begin(j.b_last) + 1 == u.end && split.begin(j.b_last + 1) >= u.end + 2 &&
                !(u.beg + 2 == u.end && split.begin(j.b_last - 1) < u.beg))
                --j.b_last;
            if (split.begin(j.b_first + 1) == u.beg + 1 && split.begin(j.b_first) < u.beg)
                ++j.b_first;
        }
        j.bunches = (j.b_last - j.b_first) / kFan + 1;
        j.b0 = j.b_first + ((int)blockIdx.x - j.b_first) / kFan * kFan;
        j.into = piece_of(j, j.b0);
        return j;
    };
    auto in_bunch = [&](const Join &j) { return min(kFan, j.b_last - j.b0 + 1); };
    const Join join_0 = before_it.heads ? join_of(before_it) : Join{}, join_1 = after.heads ? join_of(after) : Join{};
    uint32_t *counters = reinterpret_cast<uint32_t *>(a.ws);
    auto last_of = [&](uint32_t *ctr, int count) {
        const bool is = count_up(ctr) == (uint32_t)count - 1;
        if (is)
            *ctr = 0;
        return is;
    };
    if (2 * warp < max(before_it.heads, after.heads)) {
        const int h = half_h;
        // lane 0 of a half counts for the first piece, lane 1 for the second, at once
        bool done = false;
        if (half_lane < 2 && h < (half_lane ? after.heads : before_it.heads))
            done = last_of(counters + (half_lane ? join_1.into : join_0.into) * kHeads + h,
                           in_bunch(half_lane ? join_1 : join_0));
        const uint32_t whose = __ballot_sync(0xffffffffu, done);
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            bool mine_too = (whose >> ((lane & 16) + k)) & 1;   // this half joins
            const Unit unit = k ? after : before_it;
            const Join j = k ? join_1 : join_0;
#pragma unroll 1
            for (int level = 0; level < 2; ++level) {
                const int from = level ? j.b_first : j.b0, step = level ? kFan : 1;
                const int count = level ? j.bunches : in_bunch(j);
                const bool out = level || j.bunches == 1;
                if (level) {
                    __syncwarp();
                    bool last = false;
                    if (mine_too && half_lane == 0)
                        last = last_of(counters + (2 * kMaxCtas + j.b_first) * kHeads + h, count);
                    mine_too = __shfl_sync(0xffffffffu, last, 0, 16);
                }
                if (!__any_sync(0xffffffffu, mine_too))
                    break;
                __syncwarp();   // (what the counts have seen, for every lane)
                // the pieces come through the half's stage, every lane fetching
                // the columns that it reads
                const uint32_t dst = smem_u32(mine) + 16 * half_lane;
                auto fill = [&](int i) {
#pragma unroll 4
                    for (int z = 0; z < kFan; ++z) {
                        const bool some = mine_too && i + z < count;
                        const float *p = pc.at_o(piece_of(j, from + (some ? i + z : 0) * step), h) + 4 * half_lane;
#pragma unroll
                        for (int q = 0; q < kQuads; ++q)
                            cp_async16(dst + (z * DP + 64 * q) * 4, p + 64 * q, some);
                    }
                    commit();
                };
                fill(0);
                float2 ml[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    ml[e] = mine_too && half_lane + 16 * e < count
                                ? __ldcg(reinterpret_cast<const float2 *>(
                                      pc.at_ml(piece_of(j, from + (half_lane + 16 * e) * step), h)))
                                : no_part;
                float f[2], top, sum_l;
                over_parts(ml, f, top, sum_l);
                float4 x[kQuads];
#pragma unroll
                for (int q = 0; q < kQuads; ++q)
                    x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int i = 0;;) {
                    cp_async_wait<0>();
#pragma unroll
                    for (int z = 0; z < kFan; ++z) {
                        const float w = __shfl_sync(0xffffffffu, i ? f[1] : f[0], z, 16);   // 0 past the last
#pragma unroll
                        for (int q = 0; q < kQuads; ++q)
                            add(x[q], *reinterpret_cast<const float4 *>(mine + z * DP + 4 * half_lane + 64 * q), w);
                    }
                    i += kFan;
                    if (i >= count)
                        break;
                    fill(i);
                }
                const float inv = !out ? 1.f : sum_l == 0.f ? 0.f : 1.f / sum_l;
                if (mine_too) {
#pragma unroll
                    for (int q = 0; q < kQuads; ++q)
                        if (4 * half_lane + 64 * q < D)
                            put(unit, out, j.into, h, 4 * half_lane + 64 * q, x[q], inv);
                    if (half_lane == 0)
                        put_sum(unit, out, j.into, h, top, sum_l);
                }
                if (out)
                    break;
            }
        }
    }
    clear_rows();
}

// Keys that a row of the block table can name.
int64_t key_cap(int64_t max_pages, int64_t page_size)
{
    const int64_t n = max_pages * page_size;
    return n < INT32_MAX ? n : INT32_MAX;
}

int padded(int64_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

template <int DT, int DP>
cudaError_t launch(const PagedAttention &p, uint32_t *err, cudaStream_t stream)
{
    using S = Shape<DT, DP>;
    static_assert(S::kTile >= kMinTile, "tile bound");
    auto *kernel = k_paged_attention<DT, DP>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = ask_once([] {
            return cudaFuncSetAttribute(k_paged_attention<DT, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        S::kSmem);
        });
    if (e != cudaSuccess)
        return e;
    const tw_kv_cache &c = p.cache;
    Args a{};
    a.q = p.q, a.out = p.out, a.lse = p.lse, a.table = p.block_table, a.lengths = p.lengths, a.first = p.first;
    a.k = static_cast<const uint8_t *>(c.k);
    a.v_of_k = static_cast<const uint8_t *>(c.v) - a.k;
    a.k_scale = c.k_scale, a.v_scale = c.v_scale, a.ws = p.ws, a.err = err;
    a.ldq = p.ldq, a.ldo = p.ldo, a.table_stride = p.table_stride;
    a.page_bytes = c.page_stride * S::kElem, a.row_bytes = c.token_stride * S::kElem;
    a.head_bytes = c.head_stride * S::kElem;
    a.requests = (int)p.requests, a.heads = p.heads, a.kv_heads = (int)c.kv_heads, a.group = a.heads / a.kv_heads;
    a.per_kv = (int)ceil_div(a.group, kHeads), a.units = a.kv_heads * a.per_kv;
    a.D = (int)c.head_dim, a.P = (int)c.page_size, a.pages = (int)c.num_pages;
    a.page_shift = -1;
    for (int b = 0; b < 31; ++b)
        if (a.P == 1 << b)
            a.page_shift = b;
    a.cap = (int)key_cap(p.max_pages, c.page_size);
    a.short_way = a.P % 16 == 0 && ((a.page_bytes | a.row_bytes | a.head_bytes) >> 32) == 0;
    a.mul = p.scale * kLog2e;
    // As many blocks as are resident; no more than tiles that the block table
    // can hold.
    const int64_t tiles = p.requests * a.units * ceil_div(a.cap, S::kTile);
    int64_t grid = (int64_t)sms * S::kBlocks;
    grid = grid < kMaxCtas ? grid : kMaxCtas;
    static_assert(2 * kFan * kFan >= kMaxCtas && S::kWarps <= kFan, "two parts a lane of a half");
    grid = grid < tiles ? grid : tiles;
    kernel<<<(unsigned)grid, S::kThreads, S::kSmem, stream>>>(a);
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

bool paged_attention_fits(int64_t requests, int64_t heads, int64_t kv_heads, int64_t max_pages, int64_t page_size)
{
    // (each factor is below 2^31; the whole product need not fit 64 bits)
    const int64_t units = requests * kv_heads * ceil_div(heads / kv_heads, kHeads);   // up to 2^24 * 2^16
    return units <= INT32_MAX / ceil_div(key_cap(max_pages, page_size), kMinTile);
}

// Counters per head (one for each piece, one for each block), then maxima and sums, then sums of
// values of two pieces per block: the first and the last of its run.
int64_t paged_attention_ws_bytes(int64_t head_dim)
{
    return (int64_t)kMaxCtas * kHeads * 4 * (3 + 2 * (2 + padded(head_dim)));
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
