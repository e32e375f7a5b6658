// tw_norm.cu — what stands between two blocks of a decoder layer, in one
// pass over a row: the norm of the block's output, its gate and scale, the
// residual sum, the norm of the sum, and the int8 codes of that for the next
// projection.
//   t = Npost(y);  h = x + alpha * gate * t;  n = Npre(h)
// with N one of: the identity; RMS, u / sqrt(mean(u^2) + eps) * w; layer,
// (u - mean(u)) / sqrt(var(u) + eps) * w + b.
// The codes are those of tw_quantize_act on n, bit for bit.
//
// A row is read once: y (or x alone) into registers, x and a gate per token
// meanwhile into registers, shared memory or L2; sums are in 32 bits, the
// variance from the centred values.  What it has to move is 16 bytes per element
// (x, y in; h, n out).  4096 rows of 1536 with both norms and a gate take 21.9 us
// where L2 holds nothing of them (4.6 TB/s; 19.8 us into buffers that it holds),
// of 8960 in 1000 rows 37.5 us (3.8 TB/s), odd widths, column by column, 30 .. 45 us
// for as many bytes.  That is not the memory's rate (6.5 TB/s): a row's reductions
// and barriers leave too few bytes on their way, and 1000 rows in three blocks an
// SM are two and a quarter turns of the GPU.  Where nothing else is said, the times
// of one choice against another below are of passes whose outputs L2 holds.
// Measured and left out: persistent blocks with the next rows on their way into
// shared memory (24.9 and 47.1 us: with one row at a time in a block the
// reductions' latency shows), a warp a row (35.1 us at 1536), odd widths in groups
// of four between memory's boundaries with their ends apart (2492 rows of 2407:
// 33 us, single columns 26 us).
#include "tw_device.cuh"
#include "tw_internal.h"
#include "tw_kv.cuh"

namespace tw {
namespace {

constexpr int64_t kSms = 148;   // of a B200

// Sums (or maxima) over the threads of a row, in a fixed order: the lanes by
// butterfly, then the warps' values by butterfly in every warp.  The warps'
// values of one reduction and the next go to different places, so that one
// barrier each is enough.
struct Reduction {
    float (&red)[2][32];
    int turn = 0;
    template <bool MAX>
    __device__ __forceinline__ static float butterfly(float v)
    {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, v, o);
            v = MAX ? fmaxf(v, u) : v + u;
        }
        return v;
    }
    template <bool MAX>
    __device__ __forceinline__ float over_row(float v, int warps)
    {
        const int lane = threadIdx.x & 31;
        v = butterfly<MAX>(v);
        if (warps == 1)
            return v;
        if (lane == 0)
            red[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? red[turn][lane] : 0.f;   // (0 is the least maximum of magnitudes too)
        turn ^= 1;
        return butterfly<MAX>(v);
    }
};

// V columns of fp32.  `once`: of a row that is read once, kept out of L1 for
// the weights' sake.
template <int V> struct Vec;
template <> struct Vec<4> {
    static __device__ __forceinline__ void once(const float *p, float (&v)[4])
    {
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p) : "memory");
    }
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

// The row that a block's threads hold in u (of y, or of x without y): its
// norm, residual sum, norm and codes.  Thread t has columns
// V * (t + i * STRIDE) + 0 .. V - 1 (STRIDE 0: blockDim); x_at(i, v) and gate_at(i, v) give x and
// the gate there.
template <int V, int PER, int STRIDE, class A, class X, class G>
__device__ __forceinline__ void finish_row(const ResidualNorm &a, int64_t m, float (&u)[PER][V], Reduction &sums,
                                           int *red_i, A arrive, X x_at, G gate_at)
{
    const int threads = STRIDE ? STRIDE : blockDim.x, tid = threadIdx.x, K = (int)a.K, warps = threads / 32;
    const float inv = 1.0f / (float)K;
    auto col = [&](int i) { return (i * threads + tid) * V; };
    auto write = [&](float *row, float (&v)[PER][V]) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (col(i) < K)
                Vec<V>::store(row + col(i), v[i]);
    };
    // Norm of the row in v, in place (columns past K stay 0 until the last step).
    auto norm = [&](float (&v)[PER][V], int kind, const float *w, const float *b) {
        if (kind == TW_NORM_NONE)
            return;
        if (kind == TW_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    s += v[i][j];
            const float mean = sums.over_row<false>(s, warps) * inv;
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[i][j] = col(i) < K ? v[i][j] - mean : 0.f;
        }
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                q = fmaf(v[i][j], v[i][j], q);
        const float var = sums.over_row<false>(q, warps) * inv;
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (col(i) >= K)
                continue;
            float wv[V], bv[V];
            if (w)
                Vec<V>::load(w + col(i), wv);
            if (b)
                Vec<V>::load(b + col(i), bv);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] *= r;
                if (w)
                    v[i][j] *= wv[j];
                if (b)
                    v[i][j] += bv[j];
            }
        }
    };

    if (a.y) {
        norm(u, a.post, a.post_w, a.post_b);
        arrive();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (col(i) >= K)
                continue;
            float g[V], x[V];
            if (a.gate)
                gate_at(i, g);
            x_at(i, x);
#pragma unroll
            for (int j = 0; j < V; ++j)
                u[i][j] = fmaf(a.alpha, a.gate ? u[i][j] * g[j] : u[i][j], x[j]);
        }
    }
    if (a.h)
        write(a.h + m * a.ldh, u);
    if (!a.n && !a.xq)
        return;
    norm(u, a.pre, a.pre_w, a.pre_b);
    if (a.n)
        write(a.n + m * a.ldn, u);
    if (!a.xq)
        return;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
            top = fmaxf(top, col(i) < K ? fabsf(u[i][j]) : 0.f);
    top = sums.over_row<true>(top, warps);
    const float scale = top == 0.f ? 0.f : __fdiv_rn(127.f, top);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (col(i) >= K)
            continue;
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int q = top == 0.f ? 0 : min(max(__float2int_rn(__fmul_rn(u[i][j], scale)), -128), 127);
            sum += q;
            word |= (uint32_t)(q & 0xff) << (8 * j);
        }
        if (V == 4)
            *reinterpret_cast<uint32_t *>(a.xq + m * a.K + col(i)) = word;
        else
            a.xq[m * a.K + col(i)] = (int8_t)word;
    }
    if (a.qsum) {
        sum = __reduce_add_sync(0xffffffffu, sum);
        if ((tid & 31) == 0)
            red_i[tid >> 5] = sum;
        __syncthreads();
        if (tid < 32) {
            sum = __reduce_add_sync(0xffffffffu, tid < warps ? red_i[tid] : 0);
            if (tid == 0)
                a.qsum[m] = sum;
        }
    }
    if (tid == 0)
        a.amax[m] = top;
}

// Blocks that share an SM, so that one loads while another reduces: of 512
// threads three where a thread has few columns (4096 rows of 1536: 19.0 us, two
// 20.3 us), else two.
template <int VALUES, int THREADS>
constexpr int kBlocks = (VALUES <= 16 && THREADS <= 512 ? 1536 : 1024) / THREADS;

// Where x waits while y is normed: shared memory leaves registers to the row
// and so another block to the SM (1000 rows of 8960: three blocks 27.5 us, two
// with x in registers 30.3 us).
enum Wait { kL2, kRegisters, kShared };
template <int VALUES, int THREADS, int BLOCKS>
constexpr Wait kWait = VALUES <= 8 || (VALUES <= 20 && BLOCKS * THREADS <= 1024) ? kRegisters : kL2;

// One block a row: of THREADS threads (STRIDE), or of as many as fill it.
template <int V, int PER, int THREADS, int STRIDE, int BLOCKS, Wait WAIT>
__global__ void __launch_bounds__(THREADS, BLOCKS) k_residual_norm(const ResidualNorm a)
{
    __shared__ float red[2][32];
    __shared__ int red_i[32];
    Reduction sums{red};
    const int threads = STRIDE ? STRIDE : blockDim.x, tid = threadIdx.x, K = (int)a.K;
    const int64_t m = blockIdx.x;
    auto col = [&](int i) { return (i * threads + tid) * V; };
    auto read = [&](const float *row, auto &v) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (col(i) < K) {
                // 4096 rows of 1536 into buffers that L2 holds: 19.2 us, through
                // L1 20.3 us (into others alike); wide rows lose by it
                if constexpr (V == 4 && PER <= 2)
                    Vec<V>::once(row + col(i), v[i]);
                else
                    Vec<V>::load(row + col(i), v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[i][j] = 0.f;
            }
        }
    };
    // x is on its way while y is normed, and a gate per token: into shared
    // memory, where a thread finds what it fetched itself, or x into registers
    // where they hold both, else into L2
    extern __shared__ __align__(16) float staged[];
    auto stage = [&](const float *row, float *to) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (col(i) >= K)
                continue;
            else if (V == 4)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + col(i))),
                             "l"(row + col(i)) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to + col(i))),
                             "l"(row + col(i)) : "memory");
    };
    auto ahead = [&](const float *row) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (col(i) < K && (V > 1 || tid % 8 == 0))
                asm volatile("prefetch.global.L2 [%0];" ::"l"(row + col(i)));
    };
    const bool gate_row = a.gate && a.ldg;
    float *const staged_gate = staged + K;
    float u[PER][V], x[WAIT == kRegisters ? PER : 1][V];
    read((a.y ? a.y + m * a.ldy : a.x + m * a.ldx), u);
    if (a.y) {
        if constexpr (WAIT == kRegisters)
            read(a.x + m * a.ldx, x);
        else if constexpr (WAIT == kShared)
            stage(a.x + m * a.ldx, staged);
        else
            ahead(a.x + m * a.ldx);
        if (gate_row) {
            if constexpr (WAIT == kShared)
                stage(a.gate + m * a.ldg, staged_gate);
            else
                ahead(a.gate + m * a.ldg);
        }
    }
    finish_row<V, PER, STRIDE>(
        a, m, u, sums, red_i,
        [] {
            if constexpr (WAIT == kShared)
                asm volatile("cp.async.wait_all;" ::: "memory");
        },
        [&](int i, float (&v)[V]) {
            if constexpr (WAIT == kRegisters) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = x[i][j];
            } else {
                Vec<V>::load((WAIT == kShared ? staged : a.x + m * a.ldx) + col(i), v);
            }
        },
        [&](int i, float (&v)[V]) {
            Vec<V>::load((WAIT == kShared && gate_row ? staged_gate : a.gate + m * a.ldg) + col(i), v);
        });
}

constexpr int kSharedMost = 224 * 1024;   // of a block, beside its static shared memory

// A row of x, and of a gate per token.
int64_t shared_bytes(const ResidualNorm &a) { return (a.y ? a.gate && a.ldg ? 2 : 1 : 0) * a.K * (int64_t)sizeof(float); }

template <int V, int PER, int THREADS = 512, int BLOCKS = kBlocks<V * PER, THREADS>>
cudaError_t launch(const ResidualNorm &a, cudaStream_t stream)
{
    // whole warps, PER groups a thread
    const int64_t groups = (a.K + V - 1) / V, threads = (groups + 32 * PER - 1) / (32 * PER) * 32;
    k_residual_norm<V, PER, THREADS, 0, BLOCKS, kWait<V * PER, THREADS, BLOCKS>>
        <<<(unsigned)a.M, (unsigned)threads, 0, stream>>>(a);
    return cudaGetLastError();
}

// Every thread of THREADS, its groups a constant apart: where they are many,
// addresses and bounds of any other distance would not fit the registers (by
// single columns 1280 rows of 4687: 32 us, 69 us; quads from shared memory,
// 1785 rows of 8960: 44.1 us, 51.2 us).
template <int V, int PER, int THREADS, int BLOCKS = kBlocks<V * PER, THREADS>>
cudaError_t launch_all(const ResidualNorm &a, cudaStream_t stream)
{
    k_residual_norm<V, PER, THREADS, THREADS, BLOCKS, kWait<V * PER, THREADS, BLOCKS>>
        <<<(unsigned)a.M, THREADS, 0, stream>>>(a);
    return cudaGetLastError();
}

// x and a gate per token wait in shared memory (STRIDE as the kernel's).
template <int V, int PER, int BLOCKS, int THREADS = 512, int STRIDE = 0>
cudaError_t launch_shared(const ResidualNorm &a, cudaStream_t stream)
{
    auto *kernel = k_residual_norm<V, PER, THREADS, STRIDE, BLOCKS, kShared>;
    cudaError_t e = ask_once([] {
        return cudaFuncSetAttribute(k_residual_norm<V, PER, THREADS, STRIDE, BLOCKS, kShared>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedMost);
    });
    if (e != cudaSuccess)
        return e;
    const int64_t groups = (a.K + V - 1) / V, threads = (groups + 32 * PER - 1) / (32 * PER) * 32;
    kernel<<<(unsigned)a.M, STRIDE ? STRIDE : (unsigned)threads, (size_t)shared_bytes(a), stream>>>(a);
    return cudaGetLastError();
}

bool by16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows too few for every SM, or narrow ones for it twice, get threads enough
// for one group of columns each, for latency (one row of 1536: 2.1 us, with two
// groups a thread 2.4; 296 rows 3.7, 3.95; one of 16384 with four groups 7.3,
// with eight 8.7).
cudaError_t launch_quads(const ResidualNorm &a, cudaStream_t stream)
{
    const int64_t groups = a.K / 4;
    if (groups <= 512 && a.M <= 2 * kSms)
        return launch<4, 1>(a, stream);
    if (a.M < kSms) {
        if (groups <= 1024)
            return launch<4, 1, 1024>(a, stream);
        if (groups <= 2048)
            return launch<4, 2, 1024>(a, stream);
        if (groups <= 4096)
            return launch_all<4, 4, 1024>(a, stream);
    }
    // as few groups a thread as 512 threads allow, two at least; a row and its
    // gate wait in L2 where an SM holds fewer of them than blocks
    switch ((groups + 511) / 512) {
    case 1: case 2: return launch_shared<4, 2, 3>(a, stream);
    case 3: return launch_shared<4, 3, 3, 512, 512>(a, stream);
    case 4: return launch_shared<4, 4, 3, 512, 512>(a, stream);
    case 5: return launch_shared<4, 5, 3, 512, 512>(a, stream);
    case 6: return launch_shared<4, 6, 2, 512, 512>(a, stream);
    case 7: case 8:
        return 2 * shared_bytes(a) <= kSharedMost ? launch_shared<4, 8, 2, 512, 512>(a, stream)
                                                  : launch_all<4, 8, 512>(a, stream);
    default:
        return shared_bytes(a) <= kSharedMost ? launch_shared<4, 8, 1, 1024, 1024>(a, stream)
                                              : launch_all<4, 8, 1024>(a, stream);
    }
}

// Odd widths and strides.
cudaError_t launch_singles(const ResidualNorm &a, cudaStream_t stream)
{
    if (a.K <= 1024 && a.M <= 2 * kSms)
        return launch<1, 1, 1024>(a, stream);
    if (a.M < kSms) {
        if (a.K <= 2048)
            return launch<1, 2, 1024>(a, stream);
        if (a.K <= 4096)
            return launch_all<1, 4, 1024>(a, stream);
        if (a.K <= 8192)
            return launch_all<1, 8, 1024>(a, stream);
    }
    // eight columns a thread (3903 rows of 1537: 26 us, four 39 us), more in
    // rows that 512 threads cannot hold so
    if (a.K <= 256)   // a warp a row where there are rows enough (4096 of 171: 5.9 us, 128 threads 7.5; 300: 4.1, 3.0)
        return a.M > 12 * kSms ? launch_all<1, 8, 32, 32>(a, stream) : launch_all<1, 2, 128>(a, stream);
    // As few threads as hold the row so: of 512 most would have no column (6.3
    // million values in rows of 385, 601, 901, 1301, 1601, 2201 and 2559 columns,
    // nothing in L2: 30, 30, 30, 29, 30, 31 and 31 us, with 512 threads 122, 83, 59,
    // 45, 40, 35 and 33).
    if (a.K <= 512)
        return launch_all<1, 4, 128>(a, stream);
    if (a.K <= 1024)
        return launch_all<1, 8, 128>(a, stream);
    if (a.K <= 1536)
        return launch_all<1, 8, 192>(a, stream);
    if (a.K <= 2048)
        return launch_all<1, 8, 256>(a, stream);
    if (a.K <= 2560)
        return launch_all<1, 8, 320>(a, stream);
    if (a.K <= 4096)
        return launch_all<1, 8, 512>(a, stream);
    // Rows waiting in shared memory, three blocks an SM (nothing in L2): with a gate
    // per token, layer norms and codes 1280 rows of 4687 take 42.0 us, with sixteen
    // columns a thread and two blocks 53.9, 300 rows 15.7 and 23.3; with a gate per
    // column and RMS norms 38.1 and 38.5, 300 rows 15.3 and 18.9 (976 of 6143: 45.4
    // and 40.8).
    if (a.K <= 6144)
        return launch_shared<1, 12, 3, 512, 512>(a, stream);
    if (a.K <= 8192)
        return launch_all<1, 16, 512, 2>(a, stream);
    return a.K <= 16384 ? launch_all<1, 16, 1024>(a, stream) : launch_all<1, 32, 1024>(a, stream);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNorm &a, cudaStream_t stream)
{
    if (a.K < 1 || a.K > kNormMaxK)   // columns past the widest block's would be left out
        return cudaErrorInvalidValue;
    // Groups of four columns where every row of every operand starts on a
    // 16-byte boundary, single columns elsewhere (odd widths, odd strides).
    const bool quads = a.K % 4 == 0 && a.ldx % 4 == 0 && a.ldy % 4 == 0 && a.ldg % 4 == 0 &&
                       a.ldh % 4 == 0 && a.ldn % 4 == 0 && by16(a.x) && by16(a.y) && by16(a.gate) &&
                       by16(a.post_w) && by16(a.post_b) && by16(a.pre_w) && by16(a.pre_b) &&
                       by16(a.h) && by16(a.n) && by16(a.xq);
    if (!quads)
        return launch_singles(a, stream);
    return launch_quads(a, stream);
}

}  // namespace tw
