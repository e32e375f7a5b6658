// tw_attention.cu — attention of one new token per request over a paged
// key-value cache: for the query head i of request r over its visible keys j
// (first_r <= j < length_r)
//   s_j = scale * (q_i . k_j);  out_i = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
// with m the maximum of the s_j, in one pass with the running maximum and
// sum; lse_i = m + log(sum).  No visible key: out = 0, lse = -inf.
//
// Bound by memory: every visible key and value is read once, and each element
// serves the few query heads of its group only (2 * heads / kv_heads
// multiply-adds per element and head), far below what tcgen05 tiles of 128
// rows need to pay; mma.sync tiles of 16 x 8 keep up with the memory at a
// fraction of their rate.
//
// Split: the keys of all requests and KV heads are cut into tiles of 64, laid
// end to end, and every block takes an equal run of them, whatever the
// lengths are.  A block whose run holds all of a (request, KV head) writes its
// output; the pieces of one that spans blocks go to the workspace, and the
// block that finishes last joins them in a fixed order.  Inside a block each
// of four warps takes 16 keys of every tile through its own ring of
// cp.async stages: no barrier until a piece ends.
//
// Eight query heads ride in one 16-row MMA operand together with what their
// first rounding left over: rows 0-7 hold the operand rounded to the cache's
// type, rows 8-15 the remainder, so that queries and weights are carried in 22
// bits (fp16) at no extra instruction.  bf16's eight bits need a third part,
// in a second MMA.  Larger groups are split into units of eight heads.
#include <cfloat>

#include "tw_kv.cuh"

namespace tw {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 16;                    // keys of a warp's step
constexpr int kTile = kKeys * kWarps;
constexpr int kMaxCtas = 512;                // counters and partial results in the workspace
constexpr int kHeads = 8;                    // query heads of a unit
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The shape of one variant: DP columns (head_dim rounded up) of type DT.
template <int DT, int DP>
struct Shape {
    static constexpr bool kCodes = DT == TW_KV_I8;
    static constexpr bool kThird = DT == TW_KV_BF16;   // a third part of queries and weights
    static constexpr int kElem = kCodes ? 1 : 2;
    static constexpr int kRow = DP * kElem;            // bytes of a key
    static constexpr int kChunks = kRow / 16;
    static constexpr int kPool = kKeys * kRow;         // bytes of a step's keys
    static constexpr int kStage = 2 * kPool + (kCodes ? 2 * kKeys * 4 : 0);
    static constexpr int kSteps = DP / 16;             // MMA steps over the columns
    static constexpr int kTiles = DP / 8;              // MMA tiles of output columns
    // Queries in registers up to 128 columns, in shared memory above (the
    // accumulators take half of the registers there).
    static constexpr bool kQueryShared = DP > 128;
    static constexpr int kQueryBytes = kQueryShared ? kSteps * 32 * (kThird ? 24 : 16) : 0;
    static constexpr int kStages = DP == 256 ? (kCodes ? 5 : 3) : DP == 128 ? (kCodes ? 5 : 3) : (kCodes ? 8 : 6);
    static constexpr int kSmem = kWarps * kStages * kStage + kQueryBytes;
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

// Two bytes of w ^ 0x80808080 (the codes plus 128) as exact fp16 codes: a
// byte b under the exponent of 1024 is 1024 + b, less 1152 the code.
template <int SEL>
__device__ __forceinline__ uint32_t codes2(uint32_t w)
{
    const uint32_t h = __byte_perm(w, 0x64646464u, SEL);
    const uint32_t off = 0x64806480u;   // 1152 twice
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// Byte offset of 16-byte chunk c of key row in a step's pool: chunks are
// permuted by the row so that eight rows of one chunk fall on all banks.
template <int CHUNKS>
__device__ __forceinline__ uint32_t place(int row, int c)
{
    const int x = CHUNKS >= 8 ? (row & 7) : ((row >> 1) & 3);
    return (uint32_t)(row * CHUNKS + (c ^ x)) * 16;
}

// The visible keys of a request, as tiles.
struct Span {
    int lo, hi, first_tile, tiles;
};

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
    s.first_tile = s.lo / kTile;
    s.tiles = s.hi > s.lo ? (s.hi - 1) / kTile + 1 - s.first_tile : 0;
    return s;
}

// A place in the run of tiles: tile t of unit u of request r.
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
            s = span_of(a, r, false, nullptr);
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

template <int DT, int DP>
__global__ void __launch_bounds__(kThreads, 2) k_paged_attention(const PagedAttention a, uint32_t *err)
{
    using S = Shape<DT, DP>;
    constexpr bool BF = DT == TW_KV_BF16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t part[kWarps];
    __shared__ int64_t start_r;
    __shared__ int start_u, start_t;
    __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
    __shared__ uint32_t sm_mask[kWarps][S::kStages];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int D = (int)a.cache.head_dim, P = (int)a.cache.page_size, kvh = (int)a.cache.kv_heads;
    const int group = a.heads / kvh, per_kv = (group + kHeads - 1) / kHeads, units = kvh * per_kv;
    const int64_t R = a.requests;

    // ---- this block's run of tiles: lengths are scanned by every block
    const int64_t per = (R + kThreads - 1) / kThreads;
    const int64_t rlo = min((int64_t)tid * per, R), rhi = min(rlo + per, R);
    int64_t sum = 0;
    for (int64_t r = rlo; r < rhi; ++r)
        sum += span_of(a, r, blockIdx.x == 0, err).tiles;
    const int64_t incl = warp_inclusive(sum, lane);
    if (lane == 31)
        part[warp] = incl;
    __syncthreads();
    int64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
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
            const int64_t n = (int64_t)span_of(a, r, false, nullptr).tiles * units;
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
        if (span_of(a, r, false, nullptr).tiles)
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
    Cursor load, use;
    load.r = start_r, load.u = start_u, load.t = start_t;
    load.s = span_of(a, load.r, false, nullptr);
    use = load;

    // ---- the ring of stages
    const uint32_t ring = smem_u32(smem) + warp * S::kStages * S::kStage;
    const uint8_t *kpool = static_cast<const uint8_t *>(a.cache.k);
    const uint8_t *vpool = static_cast<const uint8_t *>(a.cache.v);
    const int row_chunks = D * S::kElem / 16;
    auto fetch = [&](int stage) {
        const int head = load.u / per_kv;
        const int j = (load.s.first_tile + load.t) * kTile + warp * kKeys + (lane & 15);
        bool ok = j >= load.s.lo && j < load.s.hi;
        int64_t off = 0, slot = 0;
        if (ok) {
            const int p = j / P;
            const int page = __ldg(a.block_table + load.r * a.table_stride + p);
            if ((uint32_t)page < (uint32_t)a.cache.num_pages) {
                const int in = j - p * P;
                off = (page * a.cache.page_stride + in * a.cache.token_stride + head * a.cache.head_stride) *
                      S::kElem;
                slot = ((int64_t)page * P + in) * kvh + head;
            } else {
                ok = false;
                atomicOr(err, EFLAG_BADDESC);
            }
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
        if (lane == 0)
            sm_mask[warp][stage] = mask;
        const uint32_t base = ring + stage * S::kStage;
#pragma unroll
        for (int i = 0; i < S::kChunks / 2; ++i) {
            const int idx = i * 32 + lane, row = idx / S::kChunks, c = idx % S::kChunks;
            const int64_t o = __shfl_sync(0xffffffffu, off, row) + c * 16;
            const bool in = ((mask >> row) & 1) && c < row_chunks;
            const uint32_t dst = base + place<S::kChunks>(row, c);
            cp_async16(dst, kpool + (in ? o : 0), in);
            cp_async16(dst + S::kPool, vpool + (in ? o : 0), in);
        }
        if (S::kCodes) {
            const float *src = lane < 16 ? a.cache.k_scale : a.cache.v_scale;
            cp_async4(base + 2 * S::kPool + lane * 4, src + (ok ? slot : 0), ok);
        }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    const int64_t n = end - begin;
#pragma unroll 1
    for (int s = 0; s < S::kStages - 1; ++s) {
        if (s < n) {
            fetch(s);
            load.next(a, units);
        }
        commit();
    }

    uint32_t qa[S::kQueryShared ? 1 : S::kSteps][4], qb[S::kQueryShared || !S::kThird ? 1 : S::kSteps][2];
    uint4 *qs = reinterpret_cast<uint4 *>(smem + kWarps * S::kStages * S::kStage);
    uint2 *qs3 = reinterpret_cast<uint2 *>(qs + S::kSteps * 32);
    float o[S::kTiles][4], m = -INFINITY, l = 0.f, unscale = 1.f;
    int stage = 0;
    bool fresh = true;
#pragma unroll 1
    for (int64_t i = 0; i < n; ++i) {
        // ---- a new piece: its queries, split
        if (fresh) {
            const int h0 = (use.u / per_kv) * group + (use.u % per_kv) * kHeads;
            const bool live = (use.u % per_kv) * kHeads + g < group;
            const float *row = a.q + use.r * a.ldq + (int64_t)(h0 + (live ? g : 0)) * D;
            const float mul = a.scale * kLog2e;
            // columns of step j that this lane holds: two pairs, 16 bytes apart
            // in a 16-bit row; four in a row where the row holds codes
            auto load4 = [&](int j, float (&x)[4]) {
                const int c0 = S::kCodes ? 16 * j + 4 * t4 : 16 * j + 2 * t4;
                const int c1 = S::kCodes ? c0 + 2 : c0 + 8;
                const float2 p = live && c0 < D ? *reinterpret_cast<const float2 *>(row + c0) : make_float2(0.f, 0.f);
                const float2 q = live && c1 < D ? *reinterpret_cast<const float2 *>(row + c1) : make_float2(0.f, 0.f);
                x[0] = p.x * mul, x[1] = p.y * mul, x[2] = q.x * mul, x[3] = q.y * mul;
            };
            float norm = 1.f;
            unscale = 1.f;
            if (!BF) {
                // fp16 operands: the head's largest query is brought to 2^14
                // by a power of two, so that neither part leaves the range
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < S::kSteps; ++j) {
                    float x[4];
                    load4(j, x);
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
                norm = top > 0.f && top <= FLT_MAX ? __uint_as_float((uint32_t)(127 + 14 - e) << 23) : 1.f;
                unscale = top > 0.f && top <= FLT_MAX ? __uint_as_float((uint32_t)(127 - 14 + e) << 23) : 1.f;
            }
            if (S::kQueryShared)
                __syncthreads();   // the last piece's queries are read
#pragma unroll
            for (int j = 0; j < S::kSteps; ++j) {
                if (S::kQueryShared && (j & (kWarps - 1)) != warp)
                    continue;
                float x[4];
                load4(j, x);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] *= norm;
                uint32_t w[4], w3[2];
                w[0] = split2<BF>(x[0], x[1]);
                w[2] = split2<BF>(x[2], x[3]);
                w[1] = split2<BF>(x[0], x[1]);
                w[3] = split2<BF>(x[2], x[3]);
                if (S::kThird) {
                    w3[0] = split2<BF>(x[0], x[1]);
                    w3[1] = split2<BF>(x[2], x[3]);
                }
                if (S::kQueryShared) {
                    qs[j * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
                    if (S::kThird)
                        qs3[j * 32 + lane] = make_uint2(w3[0], w3[1]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        qa[S::kQueryShared ? 0 : j][k] = w[k];
                    if (S::kThird) {
                        qb[S::kQueryShared ? 0 : j][0] = w3[0];
                        qb[S::kQueryShared ? 0 : j][1] = w3[1];
                    }
                }
            }
            if (S::kQueryShared)
                __syncthreads();
            m = -INFINITY, l = 0.f;
#pragma unroll
            for (int c = 0; c < S::kTiles; ++c)
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

        const uint32_t kbase = ring + stage * S::kStage, vbase = kbase + S::kPool;
        const uint32_t mask = sm_mask[warp][stage];
        if (mask) {
            // ---- scores: heads g x keys 8 k + 2 t4 + {0, 1}
            float acc[2][4] = {}, third[2][4] = {};
            auto score_step = [&](int j, const uint32_t (&b)[2][2]) {
                uint32_t w[4], w3[2] = {0, 0};
                if (S::kQueryShared) {
                    const uint4 v = qs[j * 32 + lane];
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                    if (S::kThird) {
                        const uint2 v3 = qs3[j * 32 + lane];
                        w3[0] = v3.x, w3[1] = v3.y;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = qa[S::kQueryShared ? 0 : j][k];
                    if (S::kThird)
                        w3[0] = qb[S::kQueryShared ? 0 : j][0], w3[1] = qb[S::kQueryShared ? 0 : j][1];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mma<BF>(acc[k], w[0], w[1], w[2], w[3], b[k][0], b[k][1]);
                    if (S::kThird)
                        mma<BF>(third[k], w3[0], 0u, w3[1], 0u, b[k][0], b[k][1]);
                }
            };
            if (S::kCodes) {
#pragma unroll
                for (int j = 0; j < S::kSteps; j += 2) {
                    uint32_t f[4];
                    ldmatrix4<false>(f, kbase + place<S::kChunks>((lane & 7) + (lane & 8), j + (lane >> 4)));
                    uint32_t b[2][2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t x = f[2 * s + k] ^ 0x80808080u;
                            b[k][0] = codes2<0x4140>(x);
                            b[k][1] = codes2<0x4342>(x);
                        }
                        score_step(j + s, b);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < S::kSteps; ++j) {
                    uint32_t f[4];
                    ldmatrix4<false>(f, kbase + place<S::kChunks>((lane & 7) + ((lane >> 4) << 3),
                                                                   2 * j + ((lane >> 3) & 1)));
                    const uint32_t b[2][2] = {{f[0], f[1]}, {f[2], f[3]}};
                    score_step(j, b);
                }
            }
            // ---- running maximum and sum.  With codes the value's scale goes
            // into the weight (as its logarithm, so that weights stay within
            // fp16 whatever the scales are): w_j = 2^(s_j + log2 vs_j - m).
            float s[2][2], lv[2][2], top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = 8 * k + 2 * t4 + e;
                    float x = acc[k][e] + acc[k][2 + e];
                    if (S::kThird)
                        x += third[k][e];
                    lv[k][e] = 0.f;
                    if (S::kCodes) {
                        const float *sc = reinterpret_cast<const float *>(
                            smem + (warp * S::kStages + stage) * S::kStage + 2 * S::kPool);
                        x *= unscale * sc[key];
                        const float vs = sc[kKeys + key];
                        lv[k][e] = vs > 0.f ? log2f(vs) : 0.f;
                    } else if (!BF) {
                        x *= unscale;
                    }
                    s[k][e] = (mask >> key) & 1 ? x : -INFINITY;
                    top = fmaxf(top, s[k][e] + lv[k][e]);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (__any_sync(0xffffffffu, top > m)) {
                const float up = fmaxf(top, m);
                const float f = up == -INFINITY ? 1.f : ex2(m - up);
                m = up;
                l *= f;
#pragma unroll
                for (int c = 0; c < S::kTiles; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[c][e] *= f;
            }
            // fp16 weights are carried times 2^14 (as is the sum), so that
            // the second part of small ones stays clear of fp16's smallest
            const float shift = (m == -INFINITY ? 0.f : m) - (BF ? 0.f : 14.f);
            float p[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    p[k][e] = ex2(s[k][e] + lv[k][e] - shift);
                    l += S::kCodes ? ex2(s[k][e] - shift) : p[k][e];
                }
            uint32_t w[4], w3[2] = {0, 0};
            w[0] = split2<BF>(p[0][0], p[0][1]);
            w[2] = split2<BF>(p[1][0], p[1][1]);
            w[1] = split2<BF>(p[0][0], p[0][1]);
            w[3] = split2<BF>(p[1][0], p[1][1]);
            if (S::kThird) {
                w3[0] = split2<BF>(p[0][0], p[0][1]);
                w3[1] = split2<BF>(p[1][0], p[1][1]);
            }
            // ---- weighted values
            if (S::kCodes) {
                // a transposed 8 x 8 matrix of byte pairs: keys 2 t4 + {0, 1}, columns 2 g + {0, 1}
#pragma unroll
                for (int c = 0; c < S::kChunks; c += 2) {
                    uint32_t f[4];
                    ldmatrix4<true>(f, vbase + place<S::kChunks>((lane & 7) + (lane & 8), c + (lane >> 4)));
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t x0 = f[2 * q] ^ 0x80808080u, x1 = f[2 * q + 1] ^ 0x80808080u;
                        mma<false>(o[2 * (c + q)], w[0], w[1], w[2], w[3], codes2<0x4240>(x0), codes2<0x4240>(x1));
                        mma<false>(o[2 * (c + q) + 1], w[0], w[1], w[2], w[3], codes2<0x4341>(x0), codes2<0x4341>(x1));
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < S::kTiles; c += 2) {
                    uint32_t f[4];
                    ldmatrix4<true>(f, vbase + place<S::kChunks>((lane & 7) + (lane & 8), c + (lane >> 4)));
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        mma<BF>(o[c + q], w[0], w[1], w[2], w[3], f[2 * q], f[2 * q + 1]);
                        if (S::kThird)
                            mma<BF>(o[c + q], w3[0], 0u, w3[1], 0u, f[2 * q], f[2 * q + 1]);
                    }
                }
            }
        }

        // ---- the end of a piece
        const bool unit_done = use.t + 1 == use.s.tiles;
        if (unit_done || i + 1 == n) {
            const int64_t ubeg = begin + i - use.t, uend = ubeg + use.s.tiles;
            const int h0 = (use.u / per_kv) * group + (use.u % per_kv) * kHeads;
            const int heads = min(kHeads, group - (use.u % per_kv) * kHeads);
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            __syncwarp();   // the stage is read: it takes the warp's sums
            float *mine = reinterpret_cast<float *>(smem + (warp * S::kStages + stage) * S::kStage);
            // [head][column], columns permuted by the head against bank conflicts
            auto at = [](int h, int c) { return h * DP + (c ^ (h << 3)); };
            if (S::kCodes) {
#pragma unroll
                for (int c = 0; c < S::kChunks; ++c)
                    *reinterpret_cast<float4 *>(mine + at(g, 16 * c + 4 * t4)) =
                        make_float4(o[2 * c][0] + o[2 * c][2], o[2 * c + 1][0] + o[2 * c + 1][2],
                                    o[2 * c][1] + o[2 * c][3], o[2 * c + 1][1] + o[2 * c + 1][3]);
            } else {
#pragma unroll
                for (int c = 0; c < S::kTiles; ++c)
                    *reinterpret_cast<float2 *>(mine + at(g, 8 * c + 2 * t4)) =
                        make_float2(o[c][0] + o[c][2], o[c][1] + o[c][3]);
            }
            if (t4 == 0)
                sm_m[warp][g] = m, sm_l[warp][g] = l;
            __syncthreads();
            const bool whole = unit_done && ubeg >= begin;
            float *ws_ml = reinterpret_cast<float *>(a.ws + kMaxCtas * 4);
            float *ws_o = ws_ml + kMaxCtas * 2 * 2 * kHeads;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (ubeg >= begin ? 1 : 0);
            for (int h = warp; h < heads; h += kWarps) {
                float top = -INFINITY, sum_l = 0.f, f[kWarps];
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    top = fmaxf(top, sm_m[w][h]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    f[w] = top == -INFINITY ? 0.f : ex2(sm_m[w][h] - top);
                    sum_l = fmaf(sm_l[w][h], f[w], sum_l);
                }
                const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
                for (int c = 4 * lane; c < D; c += 128) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float4 y = *reinterpret_cast<const float4 *>(
                            smem + (w * S::kStages + stage) * S::kStage + at(h, c) * 4);
                        x.x = fmaf(y.x, f[w], x.x), x.y = fmaf(y.y, f[w], x.y);
                        x.z = fmaf(y.z, f[w], x.z), x.w = fmaf(y.w, f[w], x.w);
                    }
                    if (whole)
                        *reinterpret_cast<float4 *>(a.out + use.r * a.ldo + (int64_t)(h0 + h) * D + c) =
                            make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
                    else
                        *reinterpret_cast<float4 *>(ws_o + (slot * kHeads + h) * DP + c) = x;
                }
                if (lane == 0) {
                    if (!whole) {
                        ws_ml[(slot * kHeads + h) * 2] = top;
                        ws_ml[(slot * kHeads + h) * 2 + 1] = sum_l;
                    } else if (a.lse) {
                        a.lse[use.r * a.heads + h0 + h] =
                            sum_l == 0.f ? -INFINITY : (top - (BF ? 0.f : 14.f)) * kLn2 + logf(sum_l);
                    }
                }
            }
            if (!whole) {
                // the blocks that hold a piece: from the one with the unit's
                // first tile to the one with its last
                const int64_t c0 = ((ubeg + 1) * G + total - 1) / total - 1;
                const int64_t c1 = (uend * G + total - 1) / total - 1;
                uint32_t *ctr = reinterpret_cast<uint32_t *>(a.ws) + c0;
                __threadfence();
                __syncthreads();
                if (tid == 0)
                    last = atomicAdd(ctr, 1u) == (uint32_t)(c1 - c0);
                __syncthreads();
                if (last) {
                    __threadfence();
                    const int64_t first_slot = 2 * c0 + 1;   // the unit begins in block c0, ...
                    for (int h = warp; h < heads; h += kWarps) {
                        float top = -INFINITY, sum_l = 0.f;
                        for (int64_t b = c0 + lane; b <= c1; b += 32) {
                            const int64_t sl = b == c0 ? first_slot : 2 * b;   // ... and goes on in the others
                            top = fmaxf(top, __ldcg(ws_ml + (sl * kHeads + h) * 2));
                        }
#pragma unroll
                        for (int x = 16; x; x >>= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                        float4 x[DP / 128 ? DP / 128 : 1] = {};
                        for (int64_t b = c0; b <= c1; ++b) {
                            const int64_t sl = b == c0 ? first_slot : 2 * b;
                            const float f = top == -INFINITY ? 0.f : ex2(__ldcg(ws_ml + (sl * kHeads + h) * 2) - top);
                            sum_l = fmaf(__ldcg(ws_ml + (sl * kHeads + h) * 2 + 1), f, sum_l);
#pragma unroll
                            for (int q = 0; q < (DP / 128 ? DP / 128 : 1); ++q) {
                                const int c = 4 * lane + 128 * q;
                                if (c >= D)
                                    continue;
                                const float4 y = __ldcg(reinterpret_cast<const float4 *>(ws_o + (sl * kHeads + h) * DP + c));
                                x[q].x = fmaf(y.x, f, x[q].x), x[q].y = fmaf(y.y, f, x[q].y);
                                x[q].z = fmaf(y.z, f, x[q].z), x[q].w = fmaf(y.w, f, x[q].w);
                            }
                        }
                        const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
#pragma unroll
                        for (int q = 0; q < (DP / 128 ? DP / 128 : 1); ++q) {
                            const int c = 4 * lane + 128 * q;
                            if (c < D)
                                *reinterpret_cast<float4 *>(a.out + use.r * a.ldo + (int64_t)(h0 + h) * D + c) =
                                    make_float4(x[q].x * inv, x[q].y * inv, x[q].z * inv, x[q].w * inv);
                        }
                        if (a.lse && lane == 0)
                            a.lse[use.r * a.heads + h0 + h] =
                                sum_l == 0.f ? -INFINITY : (top - (BF ? 0.f : 14.f)) * kLn2 + logf(sum_l);
                    }
                    if (tid == 0)
                        *ctr = 0;
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
    // Two blocks an SM where the stages allow it; no more blocks than tiles
    // that the block table can hold.
    const int per_sm = 2 * (S::kSmem + 2048) <= 227 * 1024 ? 2 : 1;
    const int64_t group = a.heads / a.cache.kv_heads;
    const int64_t units = a.cache.kv_heads * ceil_div(group, kHeads);
    const int64_t span = a.max_pages * a.cache.page_size;
    const int64_t tiles = a.requests * units * ceil_div(span < INT32_MAX ? span : INT32_MAX, kTile);
    int64_t grid = (int64_t)sms * per_sm;
    grid = grid < kMaxCtas ? grid : kMaxCtas;
    grid = grid < tiles ? grid : tiles;
    k<<<(unsigned)grid, kThreads, S::kSmem, stream>>>(a, err);
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

// A counter per block, then maxima and sums, then sums of values of two
// pieces per block (the first and the last of its run).
int64_t paged_attention_ws_bytes(int64_t head_dim)
{
    return kMaxCtas * 4 + (int64_t)kMaxCtas * 2 * kHeads * 4 * (2 + padded(head_dim));
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
