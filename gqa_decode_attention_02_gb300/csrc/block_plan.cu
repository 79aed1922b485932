// block_plan.cu -- block tables, slot maps and lengths of a step, made on the
// GPU from the requests' lengths.
//
// CS336 lecture 10 §"PagedAttention": a sequence's tokens live in fixed-size
// blocks found through its block table, blocks are handed out as sequences
// grow.  The accepted length of a speculative step is known on the device only
// ("Болжау арқылы Sonar модельдерін жылдамдату" §"Спекулятивті кодтан шығару
// арқылы инференс": no GPU->CPU sync), so the block bookkeeping is done there
// too:
//     target_b = ctx_b + new_b (0 if new_b = -1),  need_b = ceil(target_b / 16)
//     need_b > held_b: the next need_b - held_b ids from the head of the free
//     ring go to the table; need_b < held_b: the ids past need_b go to its tail
//     slot of token t of b: table[b][(ctx_b + t) / 16] * 16 + (ctx_b + t) % 16
// Free ids sit in a ring of num_blocks entries, taken at the head and returned
// at the tail: within one call the two ranges cannot meet, so nothing orders
// them.  All sums are integers: the result does not depend on any order.
//
// One cluster of up to 8 CTAs (one CTA for small steps).  Every CTA scans all
// sequences itself (two block-wide prefix sums), then all of them write table
// entries (a warp per sequence) and slots (four per thread, their sequence by
// binary search of the prefix in shared memory).  What a later step reads and
// this one also reads -- lengths, counts, the ring's state, which may be
// updated in place -- is written after a cluster barrier.  A step of a few
// hundred sequences is bound by the launch and two dependent reads; a batch of
// prompts by writing 8 bytes a token.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxB = 16384;    // 12 bytes of shared memory per sequence
constexpr int kPlanCluster = 8;
constexpr int kPlanOneCta = 4096;   // tokens that one CTA handles alone

struct PlanParams {
    const int32_t* ctx;
    const int32_t* add;
    const int32_t* held;
    const int32_t* state;  // {head, count}
    int32_t* ring;
    int32_t* tables;
    int32_t* ctx_out;
    int32_t* held_out;
    int32_t* state_out;
    int32_t* cu;
    int32_t* slots;
    int32_t* positions;
    int32_t* status;
    int B, max_blocks, num_blocks;
    int tokens;  // entries of slots and positions
    int limit;   // most new tokens granted (-1 tokens: no slot map and no limit)
};

struct Demand {  // of one sequence
    int ctx, add, held, need, grow, give;
    bool bad;
};

__device__ __forceinline__ Demand demand(const PlanParams& p, int b) {
    Demand d;
    d.ctx = p.ctx[b];
    d.held = p.held[b];
    const int n = p.add[b];
    const long long target = n < 0 ? 0 : (long long)d.ctx + n;
    d.bad = d.ctx < 0 || n < -1 || d.held < 0 || d.held > p.max_blocks ||
            (long long)d.held * 16 < d.ctx || target > 16ll * p.max_blocks;
    d.add = d.bad ? 0 : max(n, 0);
    d.need = d.bad ? d.held : (int)((target + 15) >> 4);
    d.grow = max(0, d.need - d.held);
    d.give = max(0, d.held - d.need);
    return d;
}

// Exclusive prefix over the block of (a, b), and the totals.
struct Two {
    long long a, b;
};
__device__ Two scan2(Two v, Two* warp_sums, Two* total) {
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Two s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(FULL, s.a, o), b = __shfl_up_sync(FULL, s.b, o);
        if (lane >= o) {
            s.a += a;
            s.b += b;
        }
    }
    __syncthreads();  // the sums of an earlier scan have been read
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    Two before = {0, 0}, all = {0, 0};
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const Two x = warp_sums[w];
        if (w < warp) {
            before.a += x.a;
            before.b += x.b;
        }
        all.a += x.a;
        all.b += x.b;
    }
    *total = all;
    return {before.a + s.a - v.a, before.b + s.b - v.b};
}

__global__ void __launch_bounds__(kPlanThreads) block_plan_kernel(const PlanParams p) {
    extern __shared__ int plan_smem[];
    int* cu = plan_smem;              // [B + 1] first token of each sequence
    int* take = cu + p.B + 1;         // [B] its first id in the taken range, -1: refused
    int* back = take + p.B;           // [B] its first id in the returned range
    __shared__ Two sums[kPlanThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const bool lead = blockIdx.x == 0;
    const int C = p.num_blocks;
    int head = p.state[0], count = p.state[1];
    const bool ring_ok = head >= 0 && head < C && count >= 0 && count <= C;
    if (!ring_ok) {
        if (lead && tid == 0) report(p.status, GQA_ERR_BLOCKS);
        head = 0;
        count = 0;
    }
    const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
    // 1. What every sequence asks for, in order; one that does not fit is refused.
    Two v = {0, 0}, total;
    for (int b = lo; b < hi; ++b) {
        const Demand d = demand(p, b);
        if (d.bad && lead) report(p.status, GQA_ERR_CONTEXT);
        v.a += d.grow;
        v.b += d.add;
    }
    Two at = scan2(v, sums, &total);
    Two got = {0, 0};  // {taken, tokens} granted
    long long ret = 0;
    for (int b = lo; b < hi; ++b) {
        const Demand d = demand(p, b);
        at.a += d.grow;
        at.b += d.add;
        const bool fits = (d.grow == 0 || at.a <= count) &&
                          (d.add == 0 || at.b <= p.limit) &&
                          (ring_ok || d.give == 0);
        take[b] = fits ? 0 : -1;
        if (!fits && lead) report(p.status, GQA_ERR_BLOCKS);
        if (fits) {
            got.a += d.grow;
            got.b += d.add;
            ret += d.give;
        }
    }
    // 2. Where the granted ids and tokens start.
    Two sum;
    Two off = scan2(got, sums, &sum);
    Two rsum;
    long long roff = scan2({ret, 0}, sums, &rsum).a;
    const bool full = count + rsum.a > C;  // more ids than blocks: keep them
    if (full && lead && tid == 0) report(p.status, GQA_ERR_BLOCKS);
    for (int b = lo; b < hi; ++b) {
        const Demand d = demand(p, b);
        const bool fits = take[b] == 0;
        cu[b] = (int)off.b;
        take[b] = fits ? (int)off.a : -1;
        back[b] = (int)roff;
        if (fits) {
            off.a += d.grow;
            off.b += d.add;
            roff += d.give;
        }
    }
    if (tid == 0) cu[p.B] = (int)sum.b;
    __syncthreads();
    // 3. Table entries taken from the ring, ids returned to it: a warp per sequence.
    const int warps = gridDim.x * (kPlanThreads / 32);
    for (int b = blockIdx.x * (kPlanThreads / 32) + (tid >> 5); b < p.B; b += warps) {
        if (take[b] < 0) continue;
        const Demand d = demand(p, b);
        int32_t* row = p.tables + (size_t)b * p.max_blocks;
        for (int j = lane; j < d.grow; j += 32) {
            const int id = p.ring[((long long)head + take[b] + j) % C];
            if (id < 0 || id >= p.num_blocks) report(p.status, GQA_ERR_BLOCK_ID);
            row[d.held + j] = id;
        }
        if (!full)
            for (int j = lane; j < d.give; j += 32)
                p.ring[((long long)head + count + back[b] + j) % C] = row[d.need + j];
    }
    // 4. A slot and a position per new token; -1 past the last.
    if (p.slots) {
        const int n = cu[p.B];
        for (long long i0 = ((long long)blockIdx.x * kPlanThreads + tid) * 4; i0 < p.tokens;
             i0 += (long long)gridDim.x * kPlanThreads * 4) {
            int s[4], q[4];
            int l = 0, r = p.B;  // the last sequence that starts at or before i0
            while (r - l > 1) {
                const int m = (l + r) >> 1;
                if (cu[m] <= i0)
                    l = m;
                else
                    r = m;
            }
            int b = l, held = 0, c = 0, last = -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = (int)i0 + e;
                s[e] = q[e] = -1;
                if (i < n) {
                    while (cu[b + 1] <= i) ++b;
                    if (b != last) {
                        held = p.held[b];
                        c = p.ctx[b];
                        last = b;
                    }
                    const int pos = c + i - cu[b], j = pos >> 4;
                    const int id = j < held ? p.tables[(size_t)b * p.max_blocks + j]
                                            : p.ring[((long long)head + take[b] + j - held) % C];
                    q[e] = pos;
                    s[e] = (id >= 0 && id < p.num_blocks) ? id * 16 + (pos & 15) : -1;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (i0 + e < p.tokens) {
                    p.slots[i0 + e] = s[e];
                    if (p.positions) p.positions[i0 + e] = q[e];
                }
            }
        }
    }
    // 5. What may be updated in place, once every CTA has read it.
    cooperative_groups::this_cluster().sync();
    if (!lead) return;
    for (int b = tid; b <= p.B; b += kPlanThreads) p.cu[b] = cu[b];
    for (int b = tid; b < p.B; b += kPlanThreads) {
        const Demand d = demand(p, b);
        const int n = p.add[b];
        const bool fits = take[b] >= 0 && !d.bad;
        p.ctx_out[b] = fits ? (n < 0 ? 0 : d.ctx + n) : d.ctx;
        p.held_out[b] = fits && !(full && d.give > 0) ? d.need : d.held;
    }
    __syncthreads();  // state is read above by every thread of this CTA only
    if (tid == 0 && ring_ok) {
        const long long back_n = full ? 0 : rsum.a;
        p.state_out[0] = (int)((head + sum.a) % C);
        p.state_out[1] = (int)(count - sum.a + back_n);
    } else if (tid == 0) {
        p.state_out[0] = p.state[0];
        p.state_out[1] = p.state[1];
    }
}

}  // namespace

gqa_status launch_plan_blocks(int B, int max_blocks, int num_blocks, int tokens,
                              const int32_t* context_lens, const int32_t* new_lens,
                              const int32_t* held, const int32_t* ring_state, int32_t* free_ring,
                              int32_t* block_tables, int32_t* context_lens_out,
                              int32_t* held_out, int32_t* ring_state_out, int32_t* cu_new,
                              int32_t* slots, int32_t* positions, bool pdl, int32_t* dev_status,
                              cudaStream_t stream) {
    PlanParams p = {};
    p.ctx = context_lens;
    p.add = new_lens;
    p.held = held;
    p.state = ring_state;
    p.ring = free_ring;
    p.tables = block_tables;
    p.ctx_out = context_lens_out;
    p.held_out = held_out;
    p.state_out = ring_state_out;
    p.cu = cu_new;
    p.slots = slots;
    p.positions = positions;
    p.status = dev_status;
    p.B = B;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.tokens = tokens > 0 ? tokens : 0;
    p.limit = tokens < 0 ? 0x7fffffff : tokens;
    if (B > kPlanMaxB) return GQA_ERR_SHAPE;
    const size_t smem = ((size_t)3 * B + 1) * sizeof(int);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(reinterpret_cast<const void*>(&block_plan_kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(((size_t)3 * kPlanMaxB + 1) * sizeof(int))) != cudaSuccess)
        return GQA_ERR_CUDA;
    const unsigned ctas = tokens <= kPlanOneCta ? 1 : kPlanCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    void* args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(
        &cfg, reinterpret_cast<const void*>(&block_plan_kernel), args);
    return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa
