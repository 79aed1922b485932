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
// One CTA; for many tokens a CTA per 4,096, or one cluster of 8 where an output
// shares its input's buffer (in place).  Every CTA scans all sequences
// itself (one block-wide prefix sum; a second one only if something does not
// fit).  The thread that owns a sequence writes its few new table entries and
// slots itself; a sequence with more is left to a pass of whole warps (table
// entries) and of all threads (four slots each, their sequence by binary search
// of the prefix in shared memory).  What a later step reads and this one also
// reads -- lengths, counts, the ring's state, which may be updated in place -- is
// written after a barrier of the
// cluster.  A step of a few hundred sequences is bound by the
// launch and two dependent reads, a batch of prompts by writing 8 bytes a token.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

#include "launch.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int kPlanThreads = 1024;  // at most
constexpr int kPlanMaxB = 16384;    // 12 bytes of shared memory per sequence
constexpr int kPlanKeepB = 4096;    // ... 24 with its length and count and the long rows' list
constexpr size_t plan_smem_bytes(bool keep, int B) {
    return ((size_t)(keep ? 6 : 3) * B + 1) * sizeof(int);
}
constexpr int kPlanCluster = 8;
constexpr int kPlanOneCta = 4096;   // tokens that one CTA handles alone
constexpr int kPlanOwn = 8;         // table entries or tokens a thread writes alone

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
    int in_place;  // the grid is one cluster: some output is its input's buffer
    int wide;    // slots and positions are 16-byte aligned
    int limit;   // most new tokens granted (-1 tokens: no slot map and no limit)
};

struct Demand {  // of one sequence
    int ctx, add, held, target, need, grow, give;
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
    d.target = (int)(d.bad ? 0 : target);
    d.need = d.bad ? d.held : (int)((target + 15) >> 4);
    d.grow = max(0, d.need - d.held);
    d.give = max(0, d.held - d.need);
    return d;
}

struct Sums {
    int grow, give, rows;  // rows: long table rows
    long long add;
};
__device__ __forceinline__ Sums plus(const Sums& x, const Sums& y) {
    return {x.grow + y.grow, x.give + y.give, x.rows + y.rows, x.add + y.add};
}
__device__ __forceinline__ Sums scan_step(const Sums& s, int o, int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    const Sums t = {__shfl_up_sync(FULL, s.grow, o), __shfl_up_sync(FULL, s.give, o),
                    __shfl_up_sync(FULL, s.rows, o), __shfl_up_sync(FULL, s.add, o)};
    return lane >= o ? plus(s, t) : s;
}
// Exclusive prefix over the block, and the total.
__device__ Sums scan(const Sums& v, Sums* warp_sums, Sums* total) {
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    Sums s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s = scan_step(s, o, lane);
    __syncthreads();  // the sums of an earlier scan have been read
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    Sums w = {};  // every warp scans the warps' sums
    if (lane < W) w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) w = scan_step(w, o, lane);
    auto get = [&](int lane_) -> Sums {
        return {__shfl_sync(FULL, w.grow, lane_), __shfl_sync(FULL, w.give, lane_),
                __shfl_sync(FULL, w.rows, lane_), __shfl_sync(FULL, w.add, lane_)};
    };
    *total = get(31);
    Sums base = get(max(warp - 1, 0));
    if (warp == 0) base = {};
    return {base.grow + s.grow - v.grow, base.give + s.give - v.give, base.rows + s.rows - v.rows,
            base.add + s.add - v.add};
}

// What a sequence adds to the sums.
__device__ __forceinline__ Sums sums_of(const Demand& d) {
    return {d.grow, d.give, d.grow + d.give > kPlanOwn ? 1 : 0, (long long)d.add};
}

// KEEP: lengths, counts and a list of the sequences with long rows stay in shared
// memory beside the offsets.
template <bool KEEP>
__global__ void __launch_bounds__(kPlanThreads) block_plan_kernel(const PlanParams p) {
    extern __shared__ int plan_smem[];
    int* cu = plan_smem;              // [B + 1] first token of each sequence
    int* take = cu + p.B + 1;         // [B] its first id in the taken range, -1: refused
    int* back = take + p.B;           // [B] its first id in the returned range
    int* s_ctx = back + p.B;
    int* s_held = s_ctx + p.B;
    int* s_rows = s_held + p.B;
    __shared__ Sums sums[32];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    const bool lead = blockIdx.x == 0;
    const int C = p.num_blocks;
    const int per = (p.B + threads - 1) / threads;
    const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
    Demand own = {};  // of the one sequence of this thread, if it has one
    if (lo < hi) own = demand(p, lo);
    auto of = [&](int b) { return per == 1 ? own : demand(p, b); };
    int head = p.state[0], count = p.state[1];
    const bool ring_ok = head >= 0 && head < C && count >= 0 && count <= C;
    if (!ring_ok) {
        if (lead && tid == 0) report(p.status, GQA_ERR_BLOCKS);
        head = 0;
        count = 0;
    }
    // entry i of the ring past its head; i < 2C
    auto at = [&](int i) {
        i += head;
        i -= i >= C ? C : 0;
        return i >= C ? i - C : i;
    };
    // 1. What every sequence asks for, in order.
    Sums v = {}, total;
    for (int b = lo; b < hi; ++b) {
        const Demand d = of(b);
        if (d.bad && lead) report(p.status, GQA_ERR_CONTEXT);
        v = plus(v, sums_of(d));
    }
    Sums off = scan(v, sums, &total);
    // 2. Where its ids and tokens start.  One that does not fit into what is left
    //    after all before it asked is refused.
    const bool all = ring_ok && total.grow <= count && total.add <= p.limit;
    if (!all) {
        Sums got = {}, at_ = off;
        for (int b = lo; b < hi; ++b) {
            const Demand d = of(b);
            at_ = plus(at_, sums_of(d));
            const bool fits = (d.grow == 0 || at_.grow <= count) &&
                              (d.add == 0 || at_.add <= p.limit) && (ring_ok || d.give == 0);
            take[b] = fits ? 0 : -1;
            if (!fits && lead) report(p.status, GQA_ERR_BLOCKS);
            if (fits) got = plus(got, sums_of(d));
        }
        off = scan(got, sums, &total);
    }
    const bool full = total.give > C - count;  // more ids than blocks: keep them
    if (full && lead && tid == 0) report(p.status, GQA_ERR_BLOCKS);
    // 3. Offsets to shared memory; small demands are met on the way.
    bool many_tokens = false;
    for (int b = lo; b < hi; ++b) {
        const Demand d = of(b);
        const bool fits = all || take[b] == 0;
        cu[b] = (int)off.add;
        take[b] = fits ? off.grow : -1;
        back[b] = off.give;
        if (KEEP) {
            s_ctx[b] = d.ctx;
            s_held[b] = d.held;
        }
        if (!fits) continue;
        int32_t* row = p.tables + (size_t)b * p.max_blocks;
        if (d.grow + d.give > kPlanOwn) {
            if (KEEP) s_rows[off.rows] = b;
        } else if (lead) {
            for (int j = 0; j < d.grow; ++j) {
                const int id = p.ring[at(off.grow + j)];
                if (id < 0 || id >= p.num_blocks) report(p.status, GQA_ERR_BLOCK_ID);
                row[d.held + j] = id;
            }
            if (!full)
                for (int j = 0; j < d.give; ++j)
                    p.ring[at(count + off.give + j)] = row[d.need + j];
        }
        if (d.add > kPlanOwn) {
            many_tokens = true;
        } else if (lead && p.slots) {
            for (int t = 0; t < d.add; ++t) {
                const int pos = d.ctx + t, j = pos >> 4;
                const int id = j < d.held ? row[j] : p.ring[at(off.grow + j - d.held)];
                const long long i = off.add + t;
                p.slots[i] = (id >= 0 && id < p.num_blocks) ? id * 16 + (pos & 15) : -1;
                if (p.positions) p.positions[i] = pos;
            }
        }
        off = plus(off, sums_of(d));
    }
    if (tid == 0) cu[p.B] = (int)total.add;
    many_tokens = __syncthreads_or(many_tokens);
    // 4. The long table rows, each in as many parts as there are warps for it.
    if (total.rows > 0) {
        const int warps = gridDim.x * (threads >> 5);
        const int rows = KEEP ? total.rows : p.B, parts = max(1, warps / rows);
        for (int x = blockIdx.x * (threads >> 5) + (tid >> 5); x < rows * parts; x += warps) {
            const int part = x / rows, b = KEEP ? s_rows[x - part * rows] : x - part * rows;
            const int first = take[b];
            if (first < 0) continue;
            const Demand d = demand(p, b);
            if (!KEEP && d.grow + d.give <= kPlanOwn) continue;
            int32_t* row = p.tables + (size_t)b * p.max_blocks;
#pragma unroll 4
            for (int j = part * 32 + lane; j < d.grow; j += parts * 32) {
                const int id = p.ring[at(first + j)];
                if (id < 0 || id >= p.num_blocks) report(p.status, GQA_ERR_BLOCK_ID);
                row[d.held + j] = id;
            }
            if (!full)
#pragma unroll 4
                for (int j = part * 32 + lane; j < d.give; j += parts * 32)
                    p.ring[at(count + back[b] + j)] = row[d.need + j];
        }
    }
    // 5. A slot and a position per new token, of sequences not done above; -1 past
    //    the last.  (Without long ones only the tail is left.)
    const int n = cu[p.B];
    const long long from = many_tokens ? 0 : n & ~3;
    for (long long i0 = from + ((long long)blockIdx.x * threads + tid) * 4; i0 < p.tokens;
         i0 += (long long)gridDim.x * threads * 4) {
        int s[4], q[4];
        int b = 0;
        if (i0 < n) {  // the last sequence that starts at or before i0
            int r = p.B;
            while (r - b > 1) {
                const int m = (b + r) >> 1;
                if (cu[m] <= i0)
                    b = m;
                else
                    r = m;
            }
        }
        unsigned mine = 0;  // entries this thread writes
        int last = -1, jlast = -1, id = 0, held = 0, c = 0, base = 0, len = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = (int)i0 + e;
            s[e] = q[e] = -1;
            if (i >= n) {
                mine |= 1u << e;
                continue;
            }
            while (cu[b + 1] <= i) ++b;
            if (b != last) {
                held = KEEP ? s_held[b] : p.held[b];
                c = KEEP ? s_ctx[b] : p.ctx[b];
                base = cu[b];
                len = cu[b + 1] - base;
                last = b;
                jlast = -1;
            }
            if (len <= kPlanOwn) continue;
            mine |= 1u << e;
            const int pos = c + i - base, j = pos >> 4;
            if (j != jlast) {
                id = j < held ? p.tables[(size_t)b * p.max_blocks + j]
                              : p.ring[at(take[b] + j - held)];
                jlast = j;
            }
            q[e] = pos;
            s[e] = (id >= 0 && id < p.num_blocks) ? id * 16 + (pos & 15) : -1;
        }
        if (mine == 15u && i0 + 4 <= p.tokens && p.wide) {
            *reinterpret_cast<int4*>(p.slots + i0) = make_int4(s[0], s[1], s[2], s[3]);
            if (p.positions)
                *reinterpret_cast<int4*>(p.positions + i0) = make_int4(q[0], q[1], q[2], q[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if ((mine >> e & 1u) && i0 + e < p.tokens) {
                    p.slots[i0 + e] = s[e];
                    if (p.positions) p.positions[i0 + e] = q[e];
                }
            }
        }
    }
    // 6. What may be updated in place, once every CTA has read it.
    if (p.in_place)
        cooperative_groups::this_cluster().sync();
    else
        __syncthreads();
    if (!lead) return;
    for (int b = lo; b < hi; ++b) {
        const Demand d = of(b);
        const bool fits = take[b] >= 0 && !d.bad;
        p.cu[b] = cu[b];
        p.ctx_out[b] = fits ? d.target : d.ctx;
        p.held_out[b] = fits && !(full && d.give > 0) ? d.need : d.held;
    }
    if (tid == 0) {
        p.cu[p.B] = n;
        const int back_n = full ? 0 : total.give;
        p.state_out[0] = ring_ok ? at(total.grow) : p.state[0];
        p.state_out[1] = ring_ok ? count - total.grow + back_n : p.state[1];
    }
}

// The kernel's shared-memory limit on the current device, once, to the most that any
// batch takes: the limit belongs to the kernel, so a smaller one set for this call
// would refuse a larger one of another thread.
bool plan_ready(const void* kernel, bool keep) {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[2][kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < kDevices && done[keep][dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)plan_smem_bytes(keep, keep ? kPlanKeepB : kPlanMaxB)) !=
        cudaSuccess)
        return false;
    if (dev < kDevices) done[keep][dev].store(true, std::memory_order_release);
    return true;
}

// Whether an output array overlaps the input that it replaces.
bool updates_in_place(const PlanParams& p) {
    const int n[3] = {p.B, p.B, 2};
    const int32_t* in[3] = {p.ctx, p.held, p.state};
    const int32_t* out[3] = {p.ctx_out, p.held_out, p.state_out};
    for (int i = 0; i < 3; ++i)
        for (int o = 0; o < 3; ++o)
            if (in[i] < out[o] + n[o] && out[o] < in[i] + n[i]) return true;
    return false;
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
    p.wide = ((reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(positions)) & 15) == 0;
    if (B > kPlanMaxB) return GQA_ERR_SHAPE;
    const bool keep = B <= kPlanKeepB;
    const void* kernel = keep ? reinterpret_cast<const void*>(&block_plan_kernel<true>)
                              : reinterpret_cast<const void*>(&block_plan_kernel<false>);
    if (!plan_ready(kernel, keep)) return GQA_ERR_CUDA;
    // Outputs in buffers of their own need no barrier between the CTAs, so as many
    // run as there are tokens for (262,000 tokens: 64 CTAs 13 us, one cluster 22).
    p.in_place = updates_in_place(p);
    const int sms = device_sm_count();
    if (sms <= 0) return GQA_ERR_CUDA;
    const int want = (int)(((long long)p.tokens + kPlanOneCta - 1) / kPlanOneCta);
    const unsigned ctas = want <= 1 ? 1 : p.in_place ? kPlanCluster : want < sms ? want : sms;
    if (ctas == 1) p.in_place = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(B <= 256 && ctas == 1 ? 256 : kPlanThreads);
    cfg.dynamicSmemBytes = plan_smem_bytes(keep, B);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.in_place ? 2 : pdl ? 1 : 0;
    void* args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
    return launch_status(e);
}

}  // namespace gqa
