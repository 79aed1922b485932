// block_select.cu -- which blocks of a long cache a query should read.
//
// CS336 lecture 10 §"Арифметическая интенсивность инференса" (decoding reads the whole
// KV cache for every token and is bound by that) and §"PagedAttention" (the cache is
// blocks of 16 tokens, found through a table): a query whose weights lie on few blocks
// need read only those.  What stands for a block is, per KV head and element d, the
// largest and the smallest key of its rows; for any q
//     sum_d max(q_d max_d, q_d min_d) >= <q, k>   for every key k of the block
// bounds every score in it, at a thirtieth of the block's bytes:
//   bounds  int8 [num_blocks][K][2][H]  (0: largest, 1: smallest), and a scale
//           fp32 [num_blocks][K]: s = max |k| / 127 over the block's rows held,
//           ceil(max_d / s) and floor(min_d / s) (outwards: still a bound, up to the
//           divisions' rounding), within [-127, 127]
// The query's rows become 8-bit codes as well, c = rn(q / t) with t = max |q| / 127, so
// that the sums are whole numbers, at most 127 * 127 * 128 < 2^21 + 2^19, the same in any
// order, exact in fp32; a block's score for a KV head is the largest over its G queries of
//     (t * s) * sum_d max(c_d max_d, c_d min_d)       (both products rounded in fp32)
// (a bound for t c; for q itself, of which c holds the nearest codes, an estimate: <q, k> may
// pass it by up to t / 2 sum_d |k_d|), and equal scores go to the lower block: the choice does
// not depend on the schedule.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBoundThreads = 256;
constexpr float kMaxFinite = 3.402823466e38f;

// ---- bounds ------------------------------------------------------------------------
struct BoundParams {
    const uint4* k_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_new;
    int8_t* bounds;
    float* scale;
    int32_t* status;
    int B, K, max_blocks, num_blocks;
};

// Largest and smallest magnitude-limited value: a NaN counts as 0, an infinity as the
// largest finite number.
template <bool BF16>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
    auto one = [&](uint32_t x) {
        const uint32_t m = x & 0x7fffu;
        return m > kInf ? 0u : m == kInf ? (x & 0x8000u) | (kInf - 1) : x;
    };
    return one(w & 0xffffu) | one(w >> 16) << 16;
}

template <bool BF16>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (BF16)
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t smaller2(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (BF16)
        asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A warp per block and KV head: 16 rows of H elements, 16 bytes a lane and row (H = 128:
// two rows at a time).  The units of 256 sequences at a time lie end to end (a prefix
// sum of the CTA), a warp takes every W-th of them.  Bound by reading the keys once: 36,060
// rows of 8 heads of 128 (74 MB, 4 MB written) take 16.9 us on the device, of them 4 the start
// (lengths, prefix, the first table entries); the quotients as divisions took 18.8.
template <bool BF16, int H>
__global__ void __launch_bounds__(kBoundThreads, 4) block_bounds_kernel(const BoundParams p) {
    constexpr int P = H / 8, R = 32 / P;  // lanes per row, rows at a time
    __shared__ int s_end[kBoundThreads], s_first[kBoundThreads], s_ctx[kBoundThreads];
    __shared__ int s_warp[kBoundThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, c = lane % P, sub = lane / P;
    const uint32_t K = (uint32_t)p.K;
    const long long W = (long long)gridDim.x * (kBoundThreads / 32);
    long long id = (long long)blockIdx.x * (kBoundThreads / 32) + (threadIdx.x >> 5);
    long long base = 0;  // units of the sequences before b0
    for (int b0 = 0; b0 < p.B; b0 += kBoundThreads) {
        const int b = b0 + (int)threadIdx.x;
        int ctx = 0, i0 = 0, n = 0;  // length; first touched block and how many
        if (b < p.B) {
            ctx = __ldg(p.context_lens + b);
            const int add = __ldg(p.cu_new + b + 1) - __ldg(p.cu_new + b);
            if (add < 0 || (add > 0 && (ctx < add || ctx > p.max_blocks * 16))) {
                if (blockIdx.x == 0) report(p.status, GQA_ERR_CONTEXT);
            } else if (add > 0) {
                i0 = (ctx - add) >> 4;
                n = ((ctx + 15) >> 4) - i0;
            }
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += x;
        }
        if (b0 > 0) __syncthreads();  // the last sequences' entries have been read
        if (lane == 31) s_warp[threadIdx.x >> 5] = incl;
        __syncthreads();
        int blocks = 0;
#pragma unroll
        for (int w = 0; w < kBoundThreads / 32; ++w) {
            if (w < (int)(threadIdx.x >> 5)) incl += s_warp[w];
            blocks += s_warp[w];
        }
        s_end[threadIdx.x] = incl;
        s_first[threadIdx.x] = i0 - (incl - n);
        s_ctx[threadIdx.x] = ctx;
        __syncthreads();
        const long long units = (long long)blocks * K;
        // block id, KV head and rows held of unit x
        auto find = [&](long long x, int* blk, uint32_t* k, int* held) {
            if (x >= base + units) return;
            const uint32_t v = (uint32_t)(x - base), u = v / K;
            *k = v - u * K;
            int src = 0;  // whose it is
#pragma unroll
            for (int o = kBoundThreads / 2; o > 0; o >>= 1)
                if (s_end[src + o - 1] <= (int)u) src += o;
            const int at = s_first[src] + (int)u;
            *held = min(16, s_ctx[src] - at * 16);
            *blk = __ldg(p.block_tables + (size_t)(b0 + src) * p.max_blocks + at);
        };
        int blk_next = 0, held_next = 0;
        uint32_t k_next = 0;
        find(id, &blk_next, &k_next, &held_next);
        for (; id < base + units; id += W) {
            const int blk = blk_next, held = held_next;
            const uint32_t k = k_next;
            find(id + W, &blk_next, &k_next, &held_next);
            if (blk < 0 || blk >= p.num_blocks) {
                if (lane == 0) report(p.status, GQA_ERR_BLOCK_ID);
                continue;
            }
            const uint4* rows = p.k_cache + ((size_t)blk * 16 * p.K + k) * P + c;
            uint4 w[16 / R];
#pragma unroll
            for (int j = 0; j < 16 / R; ++j) {
                const int r = j * R + sub;  // (rows past the last repeat the first)
                w[j] = __ldg(rows + (size_t)(r < held ? r : 0) * p.K * P);
            }
            uint32_t m2 = 0;  // largest magnitudes
#pragma unroll
            for (int j = 0; j < 16 / R; ++j)
                m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(w[j].x & 0x7fff7fffu, w[j].y & 0x7fff7fffu),
                                           __vmaxu2(w[j].z & 0x7fff7fffu, w[j].w & 0x7fff7fffu)));
            uint32_t m = max(m2 & 0xffffu, m2 >> 16);
            if (m >= (BF16 ? 0x7f80u : 0x7c00u)) {  // rare
                m = 0;
#pragma unroll
                for (int j = 0; j < 16 / R; ++j) {
                    w[j] = make_uint4(finite2<BF16>(w[j].x), finite2<BF16>(w[j].y),
                                      finite2<BF16>(w[j].z), finite2<BF16>(w[j].w));
                    const uint32_t a[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m = max(m, max(a[e] & 0x7fffu, a[e] >> 16 & 0x7fffu));
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
            uint32_t top[4], low[4];  // two elements a word
#pragma unroll
            for (int j = 0; j < 16 / R; ++j) {
                const uint32_t a[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    top[e] = j ? larger2<BF16>(top[e], a[e]) : a[e];
                    low[e] = j ? smaller2<BF16>(low[e], a[e]) : a[e];
                }
            }
#pragma unroll
            for (int o = P; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    top[e] = larger2<BF16>(top[e], __shfl_xor_sync(kFull, top[e], o));
                    low[e] = smaller2<BF16>(low[e], __shfl_xor_sync(kFull, low[e], o));
                }
            const float s = __fdiv_rn(Elt<BF16>::lo(m), 127.f);
            if (sub < 2) {  // lanes of the first row write the largest, of the second the smallest
                uint32_t word[2] = {0u, 0u};
                if (s > 0.f) {
                    // largest values as they are, smallest ones with the sign turned: both
                    // are codes ceil(x / s)
                    const float sign = sub ? -1.f : 1.f;
                    float x[8], z[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t w2 = sub ? low[e >> 1] : top[e >> 1];
                        x[e] = sign * (e & 1 ? Elt<BF16>::hi(w2) : Elt<BF16>::lo(w2));
                    }
                    // x / s is at most 127 and a bit, so x * (1 / s) is off by less than 2^-15: the
                    // same ceiling as the quotient's unless an integer is nearer than that,
                    // or the code 127 all the same
                    const float r = __frcp_rn(s);
                    bool near = !(s >= 1e-30f);  // (no reciprocal to speak of)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = x[e] * r;
                        z[e] = ceilf(y);
                        near |= fabsf(y - rintf(y)) < 0x1p-13f && y < 126.5f;
                    }
                    if (near) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e] = ceilf(__fdiv_rn(x[e], s));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int code = (int)(sign * fminf(fmaxf(z[e], -127.f), 127.f));
                        word[e >> 2] |= (uint32_t)(code & 0xff) << (8 * (e & 3));
                    }
                }
                const size_t row = (size_t)blk * p.K + k;
                reinterpret_cast<uint2*>(p.bounds)[(row * 2 + sub) * P + c] =
                    make_uint2(word[0], word[1]);
                if (lane == 0) p.scale[row] = s;
            }
        }
        base += units;
    }
}

// ---- scores and the choice -----------------------------------------------------------
constexpr int kMaxSelectThreads = 1024;
struct SelectParams {
    const void* q;
    const int8_t* bounds;
    const float* scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* tables;
    int32_t* lens;
    int32_t* blocks;
    float* scores;  // [B][K][max_blocks], of sequences of more blocks than `hold`
    int32_t* status;
    int B, N, K, G, max_blocks, num_blocks;
    int keep, first, recent;
    int hold;       // scores that a CTA holds in shared memory, behind the queries' codes
};

__device__ __forceinline__ int blocks_of(const SelectParams& p, int ctx) {
    return ctx >= 1 && ctx <= p.max_blocks * 16 ? (ctx + 15) >> 4 : 0;
}
// D += A(16 x 32, row) * B(32 x 8, col), 8-bit integers
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Order-preserving bits of a score (-0 as 0; a NaN, the score of a block without bounds,
// below every number).
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Scores of a sequence's blocks for a KV head, by a cluster of CTAs, each a part of them: as
// keys in the first CTA's shared memory (`keys`), or, of more than that holds, in memory.
// The score is one product of a block's row [largest | smallest] with [max(c, 0) | min(c, 0)]
// of each query, 16 blocks by 8 queries at a time.  A product's k positions are in the
// order in which 16-byte loads bring them, the same for both sides.  Bound by reading the
// bounds: 64 contexts of 30,000 .. 32,768 tokens, 8 heads of 128 (264 MB), take 66 us with the
// choice, 4.0 TB/s over all of it and 78 % of DRAM's peak while scores are made.  (More CTAs
// per row than are resident at once, so that one row's choice overlaps another's scores,
// took 72 to 91 us.)
template <bool BF16, int H>
__device__ void block_scores(const SelectParams& p, int bk, int nb, int part, int parts,
                             uint4* codes, const uint32_t* keys) {
    constexpr int V = 2 * H / 16;  // 16-byte pieces of a row
    const int b = bk / p.K, k = bk - b * p.K, warps = blockDim.x / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G8 = (p.G + 7) / 8 * 8;
    float* qs = reinterpret_cast<float*>(codes + (size_t)G8 * V);
    for (int g = warp; g < G8; g += warps) {
        constexpr int E = H / 32;  // elements of a lane
        float x[E], a = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = 0.f;
            if (g < p.G) {
                const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                                      ((size_t)b * p.N + (size_t)k * p.G + g) * H + lane * E;
                const uint32_t w = (uint32_t)finite2<BF16>(src[e]);
                x[e] = Elt<BF16>::lo(w);
            }
            a = fmaxf(a, fabsf(x[e]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, o));
        const float t = __fdiv_rn(a, 127.f);
        int8_t* row = reinterpret_cast<int8_t*>(codes + (size_t)g * V);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int code = t > 0.f ? __float2int_rn(fminf(fmaxf(__fdiv_rn(x[e], t), -127.f), 127.f)) : 0;
            row[lane * E + e] = (int8_t)max(code, 0);
            row[H + lane * E + e] = (int8_t)min(code, 0);
        }
        if (lane == 0) qs[g] = t;
    }
    __syncthreads();
    const bool held = nb <= p.hold;
    uint32_t dst;  // of the first CTA's keys
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_addr(keys)));
    if (parts > 1)  // it has begun
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int32_t* table = p.block_tables + (size_t)b * p.max_blocks;
    float* out = p.scores + (size_t)bk * p.max_blocks;
    auto store = [&](int i, float x) {
        if (held)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + 4u * (uint32_t)i),
                         "r"(score_key(x))
                         : "memory");
        else
            out[i] = x;
    };
    const int tiles = (nb + 15) / 16, g = lane >> 2, t = lane & 3;
    const int stride = parts * warps;
    int tile = part * warps + warp;
    auto load_id = [&](int x) {
        const int i = x * 16 + (lane & 15);
        return i < nb ? __ldg(table + i) : 0;
    };
    int ahead = load_id(tile);
    for (; tile < tiles; tile += stride) {
        int id = ahead;
        ahead = load_id(tile + stride);
        const bool bad = id < 0 || id >= p.num_blocks;
        if (bad) id = 0;
        if (bad && k == 0 && lane < 16) report(p.status, GQA_ERR_BLOCK_ID);
        const unsigned bads = __ballot_sync(kFull, bad);
        const int ida = __shfl_sync(kFull, id, g), idb = __shfl_sync(kFull, id, g + 8);
        const uint4* ra = reinterpret_cast<const uint4*>(p.bounds) + ((size_t)ida * p.K + k) * V;
        const uint4* rb = reinterpret_cast<const uint4*>(p.bounds) + ((size_t)idb * p.K + k) * V;
        uint4 wa[V / 4], wb[V / 4];
#pragma unroll
        for (int x = 0; x < V / 4; ++x) {
            wa[x] = __ldg(ra + 4 * x + t);
            wb[x] = __ldg(rb + 4 * x + t);
        }
        const float sa = __ldg(p.scale + (size_t)ida * p.K + k);
        const float sb = __ldg(p.scale + (size_t)idb * p.K + k);
        float va = -INFINITY, vb = -INFINITY;
        for (int n0 = 0; n0 < G8; n0 += 8) {
            int d[4] = {0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < V / 4; ++x) {
                const uint4 w = codes[(size_t)(n0 + g) * V + 4 * x + t];
                mma_s8(d, wa[x].x, wb[x].x, wa[x].y, wb[x].y, w.x, w.y);
                mma_s8(d, wa[x].z, wb[x].z, wa[x].w, wb[x].w, w.z, w.w);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = n0 + 2 * t + e;
                if (n < p.G) {  // (a product past fp32's range counts as its largest number)
                    const float u = qs[n];
                    va = fmaxf(va, __fmul_rn(fminf(__fmul_rn(u, sa), kMaxFinite), (float)d[e]));
                    vb = fmaxf(vb, __fmul_rn(fminf(__fmul_rn(u, sb), kMaxFinite), (float)d[2 + e]));
                }
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            va = fmaxf(va, __shfl_xor_sync(kFull, va, o));
            vb = fmaxf(vb, __shfl_xor_sync(kFull, vb, o));
        }
        if (t == 0) {
            // (the limit above made a number of a scale that is none, or minus infinity)
            if (!(sa >= -kMaxFinite)) va = NAN;
            if (!(sb >= -kMaxFinite)) vb = NAN;
            const int ia = tile * 16 + g;
            if (ia < nb) store(ia, bads >> g & 1 ? -INFINITY : va);
            if (ia + 8 < nb) store(ia + 8, bads >> (g + 8) & 1 ? -INFINITY : vb);
        }
    }
}

// Sum of the first `warp` of a CTA's per-warp counts (whole warp).
__device__ __forceinline__ int before_warp(const int* sums, int warp, int lane, int warps) {
    return __reduce_add_sync(kFull, lane < warp && lane < warps ? sums[lane] : 0);
}

// The choice, by one CTA: the key of the last block to take by passes over as many bits
// as give a bin per thread (a histogram of the candidates that share the bits found so far), from the
// first bit in which any two candidates differ -- the leading ones, sign and exponent, are
// mostly alike, and a histogram of them would be one bin --, or, once no more than 32 are
// left, by comparing those with one another; then the blocks above it and as many of those
// at it as are left, in order.
__device__ void block_pick(const SelectParams& p, int bk, int nb, const uint32_t* keys) {
    __shared__ int hist[kMaxSelectThreads];  // a bin per thread
    __shared__ int sums[2][32];
    __shared__ uint32_t s_or, s_and, s_prefix, s_few[32];
    __shared__ int s_left, s_bin, s_count;
    const int b = bk / p.K, tid = threadIdx.x, threads = blockDim.x;
    const int lane = tid & 31, warp = tid >> 5;
    const int32_t* table = p.block_tables + (size_t)b * p.max_blocks;
    int32_t* tables = p.tables + (size_t)bk * p.keep;
    int32_t* blocks = p.blocks + (size_t)bk * p.keep;
    // blocks [lo, hi) compete for `left` places
    const int lo = p.first, hi = nb - p.recent, count = hi - lo;
    int left = p.keep - p.first - p.recent;
    for (int i = tid; i < p.first + p.recent; i += threads) {
        const int at = i < p.first ? i : hi + i - p.first;
        const int to = i < p.first ? i : p.keep - p.recent + i - p.first;
        tables[to] = __ldg(table + at);
        blocks[to] = at;
    }
    if (left == 0) return;
    const float* scores = p.scores + (size_t)bk * p.max_blocks + lo;
    const bool held = nb <= p.hold;
    auto key = [&](int i) { return held ? keys[lo + i] : score_key(__ldcg(scores + i)); };
    if (tid == 0) {
        s_or = 0u;
        s_and = ~0u;
    }
    __syncthreads();
    uint32_t any = 0u, all = ~0u;
    for (int i = tid; i < count; i += threads) {
        const uint32_t u = key(i);
        any |= u;
        all &= u;
    }
    any = __reduce_or_sync(kFull, any);
    all = __reduce_and_sync(kFull, all);
    if (lane == 0) {
        atomicOr(&s_or, any);
        atomicAnd(&s_and, all);
    }
    __syncthreads();
    int bits = 32 - __clz(s_or ^ s_and);  // low bits in which keys differ
    uint32_t prefix = bits == 32 ? 0u : s_and >> bits << bits;
    while (bits > 0) {
        const int take = min(bits, 31 - __clz(threads)), shift = bits - take, bins = 1 << take;
        hist[tid] = 0;
        __syncthreads();
        const uint32_t known = bits == 32 ? 0u : ~0u << bits;
        for (int i = tid; i < count; i += threads) {
            const uint32_t u = key(i);
            if ((u & known) == prefix) atomicAdd(&hist[u >> shift & (bins - 1)], 1);
        }
        __syncthreads();
        // bin of the left-th largest: thread t has the t-th from the top
        const int bin = bins - 1 - tid, own = bin >= 0 ? hist[bin] : 0;
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sums[0][warp] = incl;
        __syncthreads();
        incl += before_warp(sums[0], warp, lane, threads / 32);
        if (incl - own < left && left <= incl) {
            s_prefix = prefix | (uint32_t)bin << shift;
            s_left = left - (incl - own);
            s_bin = own;
            s_count = 0;
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
        bits = shift;
        if (bits == 0 || s_bin > 32) continue;
        const uint32_t same = ~0u << bits;
        for (int i = tid; i < count; i += threads) {
            const uint32_t u = key(i);
            if ((u & same) == prefix) s_few[atomicAdd(&s_count, 1)] = u;
        }
        __syncthreads();
        const int few = s_bin;
        const uint32_t mine = lane < few ? s_few[lane] : 0u;
        int more = 0, equal = 0;
        for (int i = 0; i < few; ++i) {
            const uint32_t u = __shfl_sync(kFull, mine, i);
            more += u > mine;
            equal += u == mine;
        }
        // (every warp finds the same)
        const unsigned at = __ballot_sync(kFull, lane < few && more < left && left <= more + equal);
        prefix = __shfl_sync(kFull, mine, __ffs(at) - 1);
        left -= __shfl_sync(kFull, more, __ffs(at) - 1);
        bits = 0;
    }
    // a run of blocks per thread: how many lie above the key and at it, before it too
    const int run = (count + threads - 1) / threads;
    const int from = min(count, tid * run), to = min(count, from + run);
    int above = 0, equal = 0;
    for (int i = from; i < to; ++i) {
        const uint32_t u = key(i);
        above += u > prefix;
        equal += u == prefix;
    }
    int ia = above, ie = equal;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, ia, o), y = __shfl_up_sync(kFull, ie, o);
        if (lane >= o) {
            ia += x;
            ie += y;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sums[0][warp] = ia;
        sums[1][warp] = ie;
    }
    __syncthreads();
    ia += before_warp(sums[0], warp, lane, threads / 32);
    ie += before_warp(sums[1], warp, lane, threads / 32);
    int a = ia - above, e = ie - equal;
    for (int i = from; i < to; ++i) {
        const uint32_t u = key(i);
        if (u > prefix || (u == prefix && e < left)) {
            const int at = p.first + a + min(e, left);
            tables[at] = __ldg(table + lo + i);
            blocks[at] = lo + i;
        }
        a += u > prefix;
        e += u == prefix;
    }
}

// A cluster per sequence and KV head: scores, then its first CTA's choice.
template <bool BF16, int H>
__global__ void __launch_bounds__(kMaxSelectThreads, 1024 / kMaxSelectThreads)
    block_select_kernel(const SelectParams p) {
    extern __shared__ uint4 scratch[];  // the queries' codes and scales, then the scores' keys
    griddep_launch_dependents();
    griddep_wait();
    uint32_t part, parts;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(part));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
    const int bk = blockIdx.x / parts, b = bk / p.K, k = bk - b * p.K, tid = threadIdx.x;
    const int ctx = __ldg(p.context_lens + b), nb = blocks_of(p, ctx);
    const int held = min(nb, p.keep);
    int32_t* tables = p.tables + (size_t)bk * p.keep;
    int32_t* blocks = p.blocks + (size_t)bk * p.keep;
    if (part == 0) {
        if (k == 0 && tid == 0) {
            p.lens[b] = nb ? (held - 1) * 16 + ctx - (nb - 1) * 16 : 0;
            if (nb == 0) report(p.status, GQA_ERR_CONTEXT);
        }
        for (int i = held + tid; i < p.keep; i += blockDim.x) tables[i] = blocks[i] = -1;
        if (nb <= p.keep)
            for (int i = tid; i < nb; i += blockDim.x) {
                tables[i] = __ldg(p.block_tables + (size_t)b * p.max_blocks + i);
                blocks[i] = i;
            }
    }
    if (nb <= p.keep) return;  // all of them (the whole cluster)
    if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    uint32_t* const keys =
        reinterpret_cast<uint32_t*>(scratch) + (p.G + 7) / 8 * 8 * (2 * H / 4 + 1);
    block_scores<BF16, H>(p, bk, nb, (int)part, (int)parts, scratch, keys);
    __syncthreads();
    if (parts > 1)  // every part of the scores is there
        asm volatile(
            "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                : "memory");
    if (part == 0) block_pick(p, bk, nb, keys);
}

}  // namespace

gqa_status launch_block_bounds(const gqa_shape& s, const void* k_cache,
                               const int32_t* block_tables, const int32_t* context_lens,
                               const int32_t* cu_new, int8_t* bounds, float* bounds_scale,
                               int32_t* dev_status, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return GQA_ERR_CUDA;
    BoundParams p = {static_cast<const uint4*>(k_cache), block_tables, context_lens, cu_new,
                     bounds, bounds_scale, dev_status, s.B, s.K, s.max_blocks_per_seq,
                     s.num_blocks};
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kBoundThreads);
    cfg.gridDim = dim3((unsigned)(sms * 4));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (s.flags & (GQA_FLAG_PDL | GQA_FLAG_EARLY_KV)) ? 1 : 0;
    return launch_status(
        s.dtype == GQA_BF16
            ? (s.H == 64 ? cudaLaunchKernelEx(&cfg, block_bounds_kernel<true, 64>, p)
                         : cudaLaunchKernelEx(&cfg, block_bounds_kernel<true, 128>, p))
            : (s.H == 64 ? cudaLaunchKernelEx(&cfg, block_bounds_kernel<false, 64>, p)
                         : cudaLaunchKernelEx(&cfg, block_bounds_kernel<false, 128>, p)));
}

size_t select_workspace_bytes(const gqa_shape& s) {
    return (size_t)s.B * s.K * s.max_blocks_per_seq * sizeof(float);
}

gqa_status launch_select_blocks(const gqa_shape& s, int keep, int first, int recent,
                                const void* q, const int8_t* bounds, const float* bounds_scale,
                                const int32_t* block_tables, const int32_t* context_lens,
                                int32_t* tables, int32_t* lens, int32_t* blocks, void* workspace,
                                int32_t* dev_status, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return GQA_ERR_CUDA;
    SelectParams p = {q, bounds, bounds_scale, block_tables, context_lens, tables, lens, blocks,
                      static_cast<float*>(workspace), dev_status, s.B, s.N, s.K, s.N / s.K,
                      s.max_blocks_per_seq, s.num_blocks, keep, first, recent, 0};
    const long long bk = (long long)s.B * s.K;
    const size_t codes = (size_t)(p.G + 7) / 8 * 8 * (2 * s.H + sizeof(float));
    constexpr size_t most = 39 * 1024;  // with what is static, what needs no opt-in
    if (codes > most || bk * 8 > (1ll << 31) - 1) return GQA_ERR_SHAPE;
    p.hold = (int)std::min((most - codes) / sizeof(uint32_t), (size_t)s.max_blocks_per_seq);
    const size_t smem = codes + p.hold * sizeof(uint32_t);
    // As many CTAs per row as are resident at once (four of 256 threads on an SM), up to a
    // cluster's eight, and no more than there are tiles of 16 blocks for their warps; rows
    // so few that this leaves SMs idle get CTAs of 1,024 (one sequence of 6,251 blocks, 8 heads:
    // 17.2 us, of 512 18.1, with the scores by way of memory 19.3).
    const int threads = bk * 8 <= sms ? kMaxSelectThreads : 256;
    const long long tiles = (s.max_blocks_per_seq + 15) / 16;
    int parts = 1;
    while (parts < 8 && bk * parts * 2 <= sms * (1024 / threads) &&
           parts * 2 * (threads / 32) <= tiles)
        parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.gridDim = dim3((unsigned)(bk * parts));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (s.flags & (GQA_FLAG_PDL | GQA_FLAG_EARLY_KV)) ? 2 : 1;
    return launch_status(
        s.dtype == GQA_BF16
            ? (s.H == 64 ? cudaLaunchKernelEx(&cfg, block_select_kernel<true, 64>, p)
                         : cudaLaunchKernelEx(&cfg, block_select_kernel<true, 128>, p))
            : (s.H == 64 ? cudaLaunchKernelEx(&cfg, block_select_kernel<false, 64>, p)
                         : cudaLaunchKernelEx(&cfg, block_select_kernel<false, 128>, p)));
}

}  // namespace gqa
