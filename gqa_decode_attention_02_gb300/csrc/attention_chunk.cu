// attention_chunk.cu -- attention of chunks of new tokens of several requests over
// a paged cache: prompts, parts of prompts behind a cached prefix, single tokens,
// any mix of them in one call.
//
// CS336 lecture 10 §"Арифметическая интенсивность инференса" (prefill works on all
// tokens of a prompt at once and is bound by arithmetic, generation by memory),
// GQA from §"Уменьшаем KV-кэш", block tables from §"PagedAttention".  For row i of
// sequence b, at position a, query head n of KV head k = n / G:
//     out[i][n] = sum_j softmax_j(scale <q[i][n], K_b[j][k]>) V_b[j][k]
// over the positions j <= a (with a window W: a - W < j <= a), by an online softmax
// over tiles of 128 positions: O += exp2(S - m) V and l += sum exp2(S - m) for a
// running reference m, O and l scaled when a row's maximum passes m by more than 8
// (in log2), O / l at the end.
//
// An item of work is a KV head and two tiles of 128 query rows of one sequence (a row
// = a token and one of the G heads), and walks the 128-position tiles that its rows
// see.  Both row tiles use one copy of K and V from shared memory, and while one
// tile's softmax runs the tensor cores work for the other.  Items lie end to end
// in units (a few for a start-up, then one per KV tile); every CTA takes an equal
// range of units, so that ragged batches, one short chunk behind a long prefix and
// single tokens all fill the GPU.  The pieces of an item that a range boundary cuts
// are folded with log-sum-exp weights, in order, by the piece that finishes last
// (no CTA waits for another; the result does not depend on which it is).
//
// One CTA per SM: warp 0 issues the MMAs, warp 1 loads K and V (one TMA box per
// cache block and KV head), warp 2 loads Q, warps 4..7 and 8..11 are the softmax of
// row tiles 0 and 1, one thread per row.
//   S_i[128 x 128] = Q_i K^T     Q_i and K from shared memory
//   P_i = exp2(S_i scale - m)    in q's dtype, over the first half of S_i's columns
//   O_i[128 x H]  += P_i V       P_i from tensor memory, V MN-major
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each.  The issuer's order is PV_0(j),
// QK_0(j + 1), PV_1(j), QK_1(j + 1): S_i is overwritten by a product that
// follows, in issue order, the one that reads P_i.
// Shared memory: Q_0, Q_1 and a ring of slots, each a tile of K or V: per cache
// block [2 groups of 8 rows][H / 64 halves][8 rows x 128 B], 128-byte swizzled, so a
// block is one box and both operand layouts have one stride between row groups.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "launch.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace gqa {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRows = 128;     // query rows of a tile (MMA M)
constexpr int kStep = 128;     // positions of a KV tile
constexpr int kBlocks = kStep / 16;
constexpr int kSoftWarp = 4;   // first softmax warp
constexpr int kThreadsCh = 384;
constexpr int kStart = 2;      // units of an item's start-up and end
constexpr int kQuota = 4;      // units per CTA at least
constexpr float kSlack = 8.f;  // log2 slack before O is rescaled
constexpr int kSeqCache = 128;
constexpr int kBadRing = 8;    // items in flight at most (the ring holds 8 tiles)
constexpr int kMaxSeqs = 16384;
constexpr uint32_t kColS = 0, kColO = 256;  // tensor-memory columns, 128 per tile

template <int H>
struct Ch {
    static constexpr int kHalves = H / 64;
    static constexpr int kTile = 128 * H * 2;        // a tile of Q, K or V
    static constexpr int kSlots = H == 128 ? 5 : 8;  // K and V tiles in flight
    static constexpr int kGroup = kHalves * 1024;    // 8 rows of a K or V tile
    static constexpr int kPart = kRows * (H + 2);    // floats of a partial result
};

struct ChunkParams {
    void* out;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* cu_new;  // nullptr: sequence b has the one row b
    int32_t* status;
    int32_t* flags;         // tickets: two per CTA that holds a first piece
    float* partials;        // [grid][2][2][kPart]: slot 0 a later piece, slot 1 a first one
    int B, M, N, K, G;
    int tpc, hpc, cpt, KC;  // tokens and heads of a row tile; head chunks per KV head
    int max_blocks, num_blocks, window;
    long long table_b, table_k;  // strides of the block tables
    float scale_log2;
};

struct ChunkSmem {
    uint64_t full[8], empty[8];
    uint64_t q_full, q_free;
    uint64_t s_ready[2], p_ready[2], o_ready[2], o_free[2], group[2];
    uint64_t done;
    long long c0, c1, base;  // range of units; first unit of the first item
    long long quota;
    int b0, vh0, qi0;
    uint32_t tmem;
    volatile int abort_flag;
    volatile int bad[kBadRing];
    int ticket[2];
    int ctxs[kSeqCache], rows[kSeqCache + 1];
};

// A sequence's new rows, or none where its lengths are out of range.
struct Seq {
    int n, ctx, r0;
    int code;  // 0, or the error
};
__device__ __forceinline__ Seq seq_of(const ChunkParams& p, int r0, int r1, int ctx) {
    Seq s = {r1 - r0, ctx, r0, 0};
    if (r0 < 0 || r1 < r0 || r1 > p.M) {
        s.n = 0;
        s.code = 2;  // its rows are not known
    } else if (s.n > 0 && (ctx < s.n || ctx > p.max_blocks * 16)) {
        s.code = 1;
        s.n = 0;
    }
    return s;
}
__device__ __forceinline__ Seq read_seq(const ChunkParams& p, int b) {
    return p.cu_new ? seq_of(p, __ldg(p.cu_new + b), __ldg(p.cu_new + b + 1),
                             __ldg(p.context_lens + b))
                    : seq_of(p, b, b + 1, __ldg(p.context_lens + b));
}
__device__ __forceinline__ Seq cached_seq(const ChunkSmem& sm, const ChunkParams& p, int b) {
    const int i = b - sm.b0;
    if (i < kSeqCache) return seq_of(p, sm.rows[i], sm.rows[i + 1], sm.ctxs[i]);
    return read_seq(p, b);
}
__device__ __forceinline__ int items_of(const ChunkParams& p, const Seq& s) {
    return (s.n + 2 * p.tpc - 1) / (2 * p.tpc);
}
// KV tiles [lo, hi) that tokens f .. e - 1 of a sequence see.
__device__ __forceinline__ int tile_lo(const ChunkParams& p, const Seq& s, int f) {
    return p.window > 0 ? max(0, s.ctx - s.n + f - p.window + 1) / kStep : 0;
}
__device__ __forceinline__ int tile_hi(const Seq& s, int e) {
    return (s.ctx - s.n + e - 1) / kStep + 1;
}
__device__ __forceinline__ int item_units(const ChunkParams& p, const Seq& s, int qi) {
    const int f = qi * 2 * p.tpc;
    return tile_hi(s, min(s.n, f + 2 * p.tpc)) - tile_lo(p, s, f) + kStart;
}

__device__ __forceinline__ void give_up(ChunkSmem& sm, const ChunkParams& p) {
    report(p.status, GQA_ERR_TIMEOUT);
    sm.abort_flag = 1;
}

// KV tiles [t0, t1) of an item, of those [lo, hi) that it has.
struct Piece {
    Seq s;
    int b, vh, f;  // first token
    int lo, hi, t0, t1;
    long long first;  // unit of tile lo
};
// Tokens of row tile i, and its KV tiles within the piece.
struct Sub {
    int f, e, a, b;
};
__device__ __forceinline__ Sub sub_of(const ChunkParams& p, const Piece& pc, int i) {
    Sub x;
    x.f = pc.f + i * p.tpc;
    x.e = min(pc.s.n, x.f + p.tpc);
    x.a = x.b = pc.t0;
    if (x.f < x.e) {
        x.a = max(pc.t0, tile_lo(p, pc.s, x.f));
        x.b = max(x.a, min(pc.t1, tile_hi(pc.s, x.e)));
    }
    return x;
}

// The pieces of the CTA's range in order; every role walks the same.
struct Walk {
    long long pos, c1, base;
    int b, vh, qi, nq;
    Seq s;
    __device__ void init(const ChunkSmem& sm, const ChunkParams& p) {
        pos = sm.c0;
        c1 = sm.c1;
        base = sm.base;
        b = sm.b0;
        vh = sm.vh0;
        qi = sm.qi0;
        nq = 0;
        if (pos < c1) {
            s = cached_seq(sm, p, b);
            nq = items_of(p, s);
        }
    }
    __device__ bool next(const ChunkSmem& sm, const ChunkParams& p, Piece& pc) {
        while (pos < c1) {
            if (nq == 0) {
                if (++b >= p.B) break;
                s = cached_seq(sm, p, b);
                nq = items_of(p, s);
                continue;
            }
            const int f = qi * 2 * p.tpc;
            const int lo = tile_lo(p, s, f), hi = tile_hi(s, min(s.n, f + 2 * p.tpc));
            const long long first = base + kStart, end = first + (hi - lo);
            if (pos < end) {
                const long long from = max(pos, first), to = min(c1, end);
                pos = to;
                if (to <= from) break;  // only start-up units
                pc.s = s;
                pc.b = b;
                pc.vh = vh;
                pc.f = f;
                pc.lo = lo;
                pc.hi = hi;
                pc.first = first;
                pc.t0 = lo + (int)(from - first);
                pc.t1 = lo + (int)(to - first);
                return true;
            }
            base = end;
            if (++qi == nq) {
                qi = 0;
                if (++vh == p.KC) {
                    vh = 0;
                    nq = 0;
                }
            }
        }
        pos = c1;
        return false;
    }
};

__device__ __forceinline__ long long shfl_ll(long long v, int src) {
    return __shfl_sync(kAll, v, src);
}
__device__ __forceinline__ long long scan_ll(long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// Rows [r0, r0 + n) of the output become zeros (whole warp).
template <int H>
__device__ void zero_rows(const ChunkParams& p, int r0, int n) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (size_t)r0 * p.N * H);
    const long long count = (long long)n * p.N * (H / 8);
    for (long long i = threadIdx.x & 31; i < count; i += 32) o[i] = make_uint4(0, 0, 0, 0);
}

// All threads: units of every sequence (in `cost`, shared memory), then this CTA's
// range and the item it starts in.
template <int H>
__device__ void chunk_plan(const ChunkParams& p, ChunkSmem& sm, long long* cost) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int first = warp * 32; first < p.B; first += kThreadsCh) {
        const int b = first + lane;
        Seq s = {0, 0, 0, 0};
        if (b < p.B) s = read_seq(p, b);
        const int nq = items_of(p, s);
        long long c = 0;
        if (nq <= 8)
            for (int qi = 0; qi < nq; ++qi) c += item_units(p, s, qi);
        unsigned many = __ballot_sync(kAll, nq > 8);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            Seq t;
            t.n = __shfl_sync(kAll, s.n, src);
            t.ctx = __shfl_sync(kAll, s.ctx, src);
            const int m = __shfl_sync(kAll, nq, src);
            long long x = 0;
            for (int qi = lane; qi < m; qi += 32) x += item_units(p, t, qi);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
            if (lane == src) c = x;
        }
        if (b < p.B) cost[b] = c;
        if (blockIdx.x == 0) {
            if (s.code) report(p.status, GQA_ERR_CONTEXT);
            unsigned zero = __ballot_sync(kAll, s.code == 1);
            while (zero) {
                const int src = __ffs(zero) - 1;
                zero &= zero - 1;
                const int at = first + src;
                const int r0 = p.cu_new ? __ldg(p.cu_new + at) : at;
                const int r1 = p.cu_new ? __ldg(p.cu_new + at + 1) : at + 1;
                zero_rows<H>(p, r0, r1 - r0);
            }
        }
    }
    __syncthreads();
    if (warp != 0) return;
    const int per = (p.B + 31) / 32;
    const int lo = min(p.B, lane * per), hi = min(p.B, lo + per);
    long long local = 0;
    for (int b = lo; b < hi; ++b) local += cost[b];
    const long long incl = scan_ll(local, lane), excl = incl - local;
    const long long total = shfl_ll(incl, 31) * p.KC;
    const long long quota = max((total + gridDim.x - 1) / gridDim.x, (long long)kQuota);
    const long long c0 = blockIdx.x * quota, c1 = min(total, c0 + quota);
    const bool mine = c0 < c1 && excl * p.KC <= c0 && c0 < incl * p.KC;
    const unsigned owners = __ballot_sync(kAll, mine);
    int b0 = 0;
    long long base = 0;
    if (mine) {
        base = excl * p.KC;
        b0 = lo;
        while (c0 >= base + cost[b0] * p.KC) base += cost[b0++] * p.KC;
    }
    const int owner = owners ? __ffs(owners) - 1 : 0;
    b0 = __shfl_sync(kAll, b0, owner);
    base = shfl_ll(base, owner);
    if (lane == 0) {
        sm.c0 = c0;
        sm.c1 = max(c0, c1);
        sm.quota = quota;
        sm.b0 = b0;
    }
    if (owners) {
        // the virtual head, then the item in it (a run of items per lane)
        const Seq s = read_seq(p, b0);
        const int nq = items_of(p, s);
        const int vh = (int)((c0 - base) / cost[b0]);
        base += vh * cost[b0];
        const int run = (nq + 31) / 32;
        const int qlo = min(nq, lane * run), qhi = min(nq, qlo + run);
        long long x = 0;
        for (int qi = qlo; qi < qhi; ++qi) x += item_units(p, s, qi);
        const long long xi = scan_ll(x, lane), xe = xi - x;
        if (base + xe <= c0 && c0 < base + xi) {
            long long at = base + xe;
            int qi = qlo;
            while (true) {
                const int u = item_units(p, s, qi);
                if (c0 < at + u) break;
                at += u;
                ++qi;
            }
            sm.vh0 = vh;
            sm.qi0 = qi;
            sm.base = at;
        }
    }
    for (int i = lane; i <= kSeqCache; i += 32) {
        const int b = min(b0 + i, p.B);
        sm.rows[i] = p.cu_new ? __ldg(p.cu_new + b) : b;
        if (i < kSeqCache) sm.ctxs[i] = b < p.B ? __ldg(p.context_lens + b) : 0;
    }
}

// ---------------------------------------------------------------------------
// Warp 1: K and V tiles into the ring, K(j) then V(j).  A lane per cache block; block
// ids are read 32 at a time, the next ones while these are in use.
template <int H>
__device__ void chunk_load(const CUtensorMap* tmk, const CUtensorMap* tmv, const ChunkParams& p,
                           uint8_t* ring, ChunkSmem& sm) {
    using C = Ch<H>;
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        tma_prefetch_desc(tmk);
        tma_prefetch_desc(tmv);
    }
    Walk wk;
    wk.init(sm, p);
    Piece pc;
    int it = 0, item = 0;
    bool aborted = false;
    while (!aborted && wk.next(sm, p, pc)) {
        const int kv = pc.vh / p.cpt;
        const int32_t* table = p.block_tables + pc.b * p.table_b + kv * p.table_k;
        // blocks that the item's rows see: none below the window, none past its last token
        const int pos0 = pc.s.ctx - pc.s.n + pc.f;
        const int blo = p.window > 0 ? max(0, pos0 - p.window + 1) / 16 : 0;
        const int bhi = (pc.s.ctx - pc.s.n + min(pc.s.n, pc.f + 2 * p.tpc) - 1) / 16 + 1;
        if (lane == 0) sm.bad[item % kBadRing] = 0;
        auto load_ids = [&](int from) {
            const int i = from + lane;
            return i >= blo && i < bhi ? __ldg(table + i) : 0;
        };
        int win = pc.t0 * kBlocks, ids = load_ids(win), nxt = load_ids(win + 32);
        for (int j = pc.t0; j < pc.t1 && !aborted; ++j) {
            if (j * kBlocks - win == 32) {
                win += 32;
                ids = nxt;
                nxt = load_ids(win + 32);
            }
            const int id = __shfl_sync(kAll, ids, (j * kBlocks - win + lane) & 31);
            const int blk = j * kBlocks + lane;
            const bool mine = lane < kBlocks && blk >= blo && blk < bhi;
            const unsigned on = __ballot_sync(kAll, mine);
            const bool bad = __any_sync(kAll, mine && (id < 0 || id >= p.num_blocks));
            const uint32_t bytes = __popc(on) * (16 * H * 2);
#pragma unroll 1
            for (int kvsel = 0; kvsel < 2; ++kvsel, ++it) {
                const int s = it % C::kSlots;
                const uint32_t bar = smem_addr(&sm.full[s]);
                if (lane == 0) {
                    bool ok = true;
                    if (it >= C::kSlots)
                        ok = mbar_wait(smem_addr(&sm.empty[s]), (it / C::kSlots - 1) & 1);
                    if (!ok) give_up(sm, p);
                    aborted = !ok || sm.abort_flag;
                    if (!aborted) {
                        if (bad) {
                            report(p.status, GQA_ERR_BLOCK_ID);
                            sm.bad[item % kBadRing] = 1;
                            __threadfence_block();
                            mbar_arrive(bar);
                        } else {
                            mbar_arrive_expect_tx(bar, bytes);
                        }
                    }
                }
                aborted = __shfl_sync(kAll, aborted, 0);
                if (aborted) break;
                if (mine && !bad)
                    tma_load_5d(smem_addr(ring + (size_t)s * C::kTile) + lane * 2 * C::kGroup,
                                kvsel ? tmv : tmk, bar, 0, 0, 0, 2 * id, kv);
            }
        }
        ++item;
    }
    if (lane == 0 && aborted)  // copies in flight land before the CTA ends
        for (int j = max(0, it - C::kSlots); j < it; ++j)
            mbar_wait(smem_addr(&sm.full[j % C::kSlots]), (j / C::kSlots) & 1);
}

// ---------------------------------------------------------------------------
// Warp 2, one lane: the Q tiles of every piece, once the products of the last one have
// read theirs.  Rows past the sequence's last token are the next sequence's (or zeros
// past the tensor): their results are not stored.
template <int H>
__device__ void chunk_queries(const CUtensorMap* tmq, const ChunkParams& p, uint8_t* qbuf,
                              ChunkSmem& sm) {
    using C = Ch<H>;
    if ((threadIdx.x & 31) != 0) return;
    tma_prefetch_desc(tmq);
    Walk wk;
    wk.init(sm, p);
    Piece pc;
    int k = 0;
    bool aborted = false;
    while (wk.next(sm, p, pc)) {
        if (k >= 1 && !mbar_wait(smem_addr(&sm.q_free), (k - 1) & 1)) give_up(sm, p);
        aborted = sm.abort_flag != 0;
        if (aborted) break;
        const int kv = pc.vh / p.cpt, h0 = (pc.vh % p.cpt) * p.hpc;
        const int tiles = pc.f + p.tpc < pc.s.n ? 2 : 1;
        mbar_arrive_expect_tx(smem_addr(&sm.q_full),
                              (uint32_t)(tiles * C::kHalves * 128 * p.tpc * p.hpc));
        for (int i = 0; i < tiles; ++i)
            for (int h = 0; h < C::kHalves; ++h)
                tma_load_4d(smem_addr(qbuf) + i * C::kTile + h * (kRows * 128), tmq,
                            smem_addr(&sm.q_full), 64 * h, h0, kv, pc.s.r0 + pc.f + i * p.tpc);
        ++k;
    }
    if (aborted && k >= 1) mbar_wait(smem_addr(&sm.q_full), (k - 1) & 1);
}

// ---------------------------------------------------------------------------
// Warp 0, one lane: every MMA.
template <bool BF16, int H>
__device__ void chunk_mma(const ChunkParams& p, uint8_t* ring, uint8_t* qbuf, ChunkSmem& sm) {
    using C = Ch<H>;
    if ((threadIdx.x & 31) != 0) return;
    constexpr uint32_t id_s = umma_idesc_ct(BF16, kRows, kStep, false);
    constexpr uint32_t id_o = umma_idesc_ct(BF16, kRows, H, true);
    const uint32_t tmem = sm.tmem;
    const uint64_t dq = umma_desc_sw128(smem_addr(qbuf), 16, 1024);
    const uint64_t dk = umma_desc_sw128(smem_addr(ring), 16, C::kGroup);
    const uint64_t dv = umma_desc_sw128(smem_addr(ring), 1024, C::kGroup);
    auto landed = [&](int n) {
        return mbar_wait(smem_addr(&sm.full[n % C::kSlots]), (n / C::kSlots) & 1);
    };
    auto qk = [&](int i, int n) {  // S_i = Q_i K^T, K in ring tile n
        const uint64_t a = dq + (uint64_t)(i * (C::kTile >> 4));
        const uint64_t b = dk + (uint64_t)((n % C::kSlots) * (C::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < H / 16; ++kk)
            umma_ss(tmem + kColS + i * 128,
                    a + (uint64_t)(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4),
                    b + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_s, kk > 0);
        umma_commit(smem_addr(&sm.s_ready[i]));
    };
    auto pv = [&](int i, int n, bool add) {  // O_i += P_i V, V in ring tile n
        const uint64_t b = dv + (uint64_t)((n % C::kSlots) * (C::kTile >> 4));
        umma_ts(tmem + kColO + i * 128, tmem + kColS + i * 128, b, id_o, add);
#pragma unroll
        for (int ks = 1; ks < kBlocks; ++ks)
            umma_ts(tmem + kColO + i * 128, tmem + kColS + i * 128 + 8 * ks,
                    b + (uint64_t)((ks * 2 * C::kGroup) >> 4), id_o, true);
        umma_commit(smem_addr(&sm.o_ready[i]));
    };
    Walk wk;
    wk.init(sm, p);
    Piece pc;
    int n = 0, k = 0;  // ring tiles and pieces so far
    int steps[2] = {0, 0}, used[2] = {0, 0};
    bool ok = true;
    while (ok && wk.next(sm, p, pc)) {
        const Sub sub[2] = {sub_of(p, pc, 0), sub_of(p, pc, 1)};
        ok = mbar_wait(smem_addr(&sm.q_full), k & 1) && !sm.abort_flag && landed(n);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (sub[i].a < sub[i].b && sub[i].a == pc.t0) qk(i, n);
        umma_commit(smem_addr(&sm.empty[n % C::kSlots]));
        if (pc.t0 + 1 == pc.t1) umma_commit(smem_addr(&sm.q_free));
        for (int j = pc.t0; j < pc.t1 && ok; ++j, n += 2) {
            ok = landed(n + 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok) break;
                if (j >= sub[i].a && j < sub[i].b) {
                    ok = mbar_wait(smem_addr(&sm.p_ready[i]), steps[i] & 1);
                    ++steps[i];
                    if (j == sub[i].a) {
                        if (used[i] > 0)
                            ok = ok && mbar_wait(smem_addr(&sm.o_free[i]), (used[i] - 1) & 1);
                        ++used[i];
                    }
                    if (!ok || sm.abort_flag) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    pv(i, n + 1, j > sub[i].a);
                }
                if (j + 1 >= sub[i].a && j + 1 < sub[i].b) {
                    ok = landed(n + 2);
                    if (ok) qk(i, n + 2);
                }
            }
            if (!ok) break;
            umma_commit(smem_addr(&sm.empty[(n + 1) % C::kSlots]));
            if (j + 1 < pc.t1) {
                umma_commit(smem_addr(&sm.empty[(n + 2) % C::kSlots]));
                if (j + 2 == pc.t1) umma_commit(smem_addr(&sm.q_free));
            }
        }
        ++k;
    }
    if (!ok) give_up(sm, p);
    umma_commit(smem_addr(&sm.done));  // every MMA ends before tensor memory is freed
    if (!mbar_wait(smem_addr(&sm.done), 0)) give_up(sm, p);
}

// ---------------------------------------------------------------------------
// Softmax of row tile i, a thread per row.
template <bool BF16, int H>
__device__ void chunk_softmax(const ChunkParams& p, uint8_t* ring, ChunkSmem& sm) {
    using C = Ch<H>;
    using E = Elt<BF16>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = (warp - kSoftWarp) >> 2;           // row tile
    const int row = 32 * (warp & 3) + lane;          // tensor-memory lane
    const int tid = row;                             // within the tile's 128 threads
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = sm.tmem + kColS + i * 128 + lanes, tO = sm.tmem + kColO + i * 128 + lanes;
    const uint32_t bS = smem_addr(&sm.s_ready[i]), bP = smem_addr(&sm.p_ready[i]),
                   bO = smem_addr(&sm.o_ready[i]), bF = smem_addr(&sm.o_free[i]),
                   bG = smem_addr(&sm.group[i]);
    int meets = 0;
    auto meet = [&]() {  // the tile's 128 threads
        mbar_arrive(bG);
        const bool ok = mbar_wait(bG, meets & 1);
        ++meets;
        return ok;
    };
    Walk wk;
    wk.init(sm, p);
    Piece pc;
    int step = 0, item = -1, n0 = 0;
    bool ok = true;
    while (ok && wk.next(sm, p, pc)) {
        ++item;
        const int ring0 = n0;
        n0 += 2 * (pc.t1 - pc.t0);
        const Sub sub = sub_of(p, pc, i);
        if (sub.f >= sub.e) continue;  // no tokens for this row tile
        const int h0 = (pc.vh % p.cpt) * p.hpc;
        const int heads = min(p.hpc, p.G - h0);
        const int count = (sub.e - sub.f - 1) * p.hpc + heads;  // rows in use
        const bool active = row < count;
        const bool warp_on = 32 * (warp & 3) < count;
        const int at = pc.s.ctx - pc.s.n;  // position of the first new token
        const int lim = at + sub.f + (active ? row / p.hpc : 0);
        const int low = p.window > 0 ? lim - p.window + 1 : 0;
        // positions that the item's rows see at all
        const int see_lo = p.window > 0 ? max(0, at + pc.f - p.window + 1) : 0;
        const int see_hi = at + min(pc.s.n, pc.f + 2 * p.tpc);
        float m = -INFINITY, l = 0.f;
        for (int j = sub.a; j < sub.b; ++j, ++step) {
            ok = __all_sync(kAll, mbar_wait(bS, step & 1));
            if (!ok) break;
            const int tok = j * kStep;
            if (warp_on) {
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s[c]);
                tmem_wait_ld();
                const int from = low - tok, to = lim + 1 - tok;  // columns seen
                if (!__all_sync(kAll, from <= 0 && to >= kStep)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (32 * c + x < from || 32 * c + x >= to) s[c][x] = 0xff800000u;
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float a = __uint_as_float(s[c][0]), b = __uint_as_float(s[c][1]);
#pragma unroll
                    for (int x = 2; x < 32; x += 2) {
                        a = fmaxf(a, __uint_as_float(s[c][x]));
                        b = fmaxf(b, __uint_as_float(s[c][x + 1]));
                    }
                    mx[c] = fmaxf(a, b);
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                const bool need = top > m + kSlack;
                if (__any_sync(kAll, need)) {
                    const float f = need && m != -INFINITY ? fast_exp2(m - top) : 1.f;
                    if (j > sub.a && __any_sync(kAll, f != 1.f)) {  // the last PV has ended
                        ok = __all_sync(kAll, mbar_wait(bO, (step - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < H / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tO + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x)
                                o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tmem_st16(tO + 16 * c, o);
                        }
                        tmem_wait_st();
                    }
                    if (need) {
                        l *= f;
                        m = top;
                    }
                }
                const float ref = m == -INFINITY ? 0.f : -m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        w[x] = E::pack(
                            fast_exp2(fmaf(__uint_as_float(s[c][2 * x]), p.scale_log2, ref)),
                            fast_exp2(fmaf(__uint_as_float(s[c][2 * x + 1]), p.scale_log2, ref)));
                        sum[x & 1] += E::lo(w[x]);
                        sum[2 + (x & 1)] += E::hi(w[x]);
                    }
                    tmem_st16(tS + 16 * c, w);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
            }
            // V rows that no row of the item sees hold anything: zeros, since 0 * NaN counts
            const int v0 = max(0, see_lo - tok), v1 = min(kStep, see_hi - tok);
            if (v0 > 0 || v1 < kStep) {
                const int nv = ring0 + 2 * (j - pc.t0) + 1;
                ok = __all_sync(kAll, mbar_wait(smem_addr(&sm.full[nv % C::kSlots]),
                                                (nv / C::kSlots) & 1));
                if (!ok) break;
                const uint32_t vb = smem_addr(ring + (size_t)(nv % C::kSlots) * C::kTile);
                // (every 16 bytes of a row, wherever the swizzle puts them)
                for (int x = tid; x < kStep * (H / 8); x += kRows) {
                    const int r = x / (H / 8), c = x % (H / 8);
                    if (r < v0 || r >= v1)
                        st_shared_v4(vb + (r >> 3) * C::kGroup + (c >> 3) * 1024 + (r & 7) * 128 +
                                         (c & 7) * 16,
                                     make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async_shared();
            }
            tc_fence_before();
            mbar_arrive(bP);
        }
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        // ---- the tile's rows ------------------------------------------------------
        const bool some = sub.a < sub.b;  // any KV tile in this piece
        if (some) {
            ok = __all_sync(kAll, mbar_wait(bO, (step - 1) & 1));
            if (!ok) break;
            tc_fence_after();
        }
        // (set before the tiles landed; without one, nothing has been waited for)
        const bool bad = some && sm.bad[item % kBadRing] != 0;
        const int first_cta = (int)(pc.first / sm.quota);
        const int last_cta = (int)((pc.first + (pc.hi - pc.lo) - 1) / sm.quota);
        const size_t head0 = (size_t)(pc.vh / p.cpt) * p.G + h0;  // query head of the tile's first
        uint16_t* const out = static_cast<uint16_t*>(p.out);
        auto out_row = [&](int r) {
            return out + (((size_t)pc.s.r0 + sub.f + r / p.hpc) * p.N + head0 + r % p.hpc) * H;
        };
        if (first_cta == last_cta) {
            if (warp_on) {
                const float inv = bad || !(l > 0.f) ? 0.f : 1.f / l;
                uint16_t* dst = active ? out_row(row) : nullptr;
#pragma unroll 1
                for (int c = 0; c < H / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        w[x] = inv == 0.f ? 0u
                                          : E::pack(__uint_as_float(o[2 * x]) * inv,
                                                    __uint_as_float(o[2 * x + 1]) * inv);
                    if (active)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            reinterpret_cast<uint4*>(dst + 32 * c)[x] =
                                make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                }
            }
            tc_fence_before();
            if (some) mbar_arrive(bF);
            continue;
        }
        // a piece of an item that several CTAs share: [H/4][128 rows][4] values, maxima, sums
        const int me = blockIdx.x, pieces = last_cta - first_cta + 1;
        {
            float* part = p.partials + ((size_t)(me * 2 + (me == first_cta)) * 2 + i) * C::kPart;
            if (warp_on && some) {
#pragma unroll 1
                for (int c = 0; c < H / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
                    if (active)
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            __stcg(reinterpret_cast<uint4*>(part) + (8 * c + x) * kRows + row,
                                   make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
                }
            }
            tc_fence_before();
            if (some) mbar_arrive(bF);
            __stcg(part + kRows * H + row, m);
            __stcg(part + kRows * (H + 1) + row, bad ? -1.f : l);  // a bad block shows as -1
        }
        __threadfence();
        int32_t* const flag = p.flags + 2 * first_cta + i;
        ok = meet();
        if (ok && tid == 0) {
            unsigned v;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                         : "=r"(v)
                         : "l"(flag)
                         : "memory");
            sm.ticket[i] = (int)v;
        }
        ok = __all_sync(kAll, ok && meet());
        if (!ok) break;
        const bool last = sm.ticket[i] == pieces - 1;
        if (last) {
            __threadfence();
            auto part_of = [&](int c) {
                return p.partials + ((size_t)(c * 2 + (c == first_cta)) * 2 + i) * C::kPart;
            };
            for (int x = tid; x < count * (H / 4); x += kRows) {
                const int r = x % count, d = x / count;
                float M = -INFINITY;
                bool any_bad = false;
                for (int c = first_cta; c <= last_cta; ++c) {
                    const float* q = part_of(c) + kRows * H + r;
                    M = fmaxf(M, __ldcg(q));
                    any_bad |= __ldcg(q + kRows) < 0.f;
                }
                float acc[4] = {0.f, 0.f, 0.f, 0.f}, L = 0.f;
                for (int c = first_cta; c <= last_cta; ++c) {
                    const float* q = part_of(c);
                    const float lc = __ldcg(q + kRows * (H + 1) + r);
                    if (!(lc > 0.f)) continue;  // nothing seen in this piece
                    const float w = fast_exp2(__ldcg(q + kRows * H + r) - M);
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(q) + d * kRows + r);
                    L = fmaf(w, lc, L);
                    acc[0] = fmaf(w, v.x, acc[0]);
                    acc[1] = fmaf(w, v.y, acc[1]);
                    acc[2] = fmaf(w, v.z, acc[2]);
                    acc[3] = fmaf(w, v.w, acc[3]);
                }
                const bool zero = any_bad || !(L > 0.f);
                const float inv = zero ? 0.f : 1.f / L;
                uint2 y = make_uint2(0u, 0u);
                if (!zero)
                    y = make_uint2(E::pack(acc[0] * inv, acc[1] * inv),
                                   E::pack(acc[2] * inv, acc[3] * inv));
                *reinterpret_cast<uint2*>(out_row(r) + 4 * d) = y;
            }
            if (tid == 0) *flag = 0;  // as the next call wants it
        }
        // (no thread writes the ticket again before every thread has read it)
        ok = __all_sync(kAll, meet());
    }
    if (!ok) give_up(sm, p);
}

template <bool BF16, int H>
__global__ void __launch_bounds__(kThreadsCh, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap tmk,
                           const __grid_constant__ CUtensorMap tmv,
                           const __grid_constant__ CUtensorMap tmq, const ChunkParams p) {
    using C = Ch<H>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* qbuf = base;
    uint8_t* ring = qbuf + 2 * C::kTile;
    ChunkSmem& sm = *reinterpret_cast<ChunkSmem*>(ring + C::kSlots * C::kTile);
    const int warp = threadIdx.x >> 5;
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < 8; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        mbar_init(smem_addr(&sm.q_full), 1);
        mbar_init(smem_addr(&sm.q_free), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sm.s_ready[i]), 1);
            mbar_init(smem_addr(&sm.p_ready[i]), kRows);
            mbar_init(smem_addr(&sm.o_ready[i]), 1);
            mbar_init(smem_addr(&sm.o_free[i]), kRows);
            mbar_init(smem_addr(&sm.group[i]), kRows);
        }
        mbar_init(smem_addr(&sm.done), 1);
        sm.abort_flag = 0;
        sm.base = 0;
        sm.vh0 = sm.qi0 = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(smem_addr(&sm.tmem), 512);
    griddep_wait();  // everything read or written follows earlier kernels
    __syncthreads();  // (the plan's scratch is the ring; the range's start is set above)
    chunk_plan<H>(p, sm, reinterpret_cast<long long*>(ring));
    fence_proxy_async_shared();  // the scratch before the copies that overwrite it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        chunk_mma<BF16, H>(p, ring, qbuf, sm);
    else if (warp == 1)
        chunk_load<H>(&tmk, &tmv, p, ring, sm);
    else if (warp == 2)
        chunk_queries<H>(&tmq, p, qbuf, sm);
    else if (warp >= kSoftWarp)
        chunk_softmax<BF16, H>(p, ring, sm);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(sm.tmem, 512);
}

template <int H>
constexpr size_t chunk_smem() {
    return 1024 + (size_t)(2 + Ch<H>::kSlots) * Ch<H>::kTile + sizeof(ChunkSmem);
}
static_assert(chunk_smem<128>() <= 227 * 1024 && chunk_smem<64>() <= 227 * 1024, "shared memory");
static_assert(kMaxSeqs * sizeof(long long) <= (size_t)Ch<64>::kSlots * Ch<64>::kTile &&
                  kMaxSeqs * sizeof(long long) <= (size_t)Ch<128>::kSlots * Ch<128>::kTile,
              "the plan's scratch fits in the ring");

// K or V of a cache: (64 elements, 8 rows, half, group of 8 rows, KV head); a box is a
// cache block of one head.
bool block_map(CUtensorMap* m, const void* base, const gqa_shape& s) {
    const cuuint64_t row = (cuuint64_t)s.K * s.H * 2;
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)s.H / 64, 2 * (cuuint64_t)s.num_blocks,
                                (cuuint64_t)s.K};
    const cuuint64_t strides[4] = {row, 128, 8 * row, (cuuint64_t)s.H * 2};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)s.H / 64, 2, 1};
    return make_tensor_map(m, s.dtype, 5, base, dims, strides, box);
}
// q: (dim, head of the group, KV head, row)
bool query_map(CUtensorMap* m, const void* q, const gqa_shape& s, long long rows,
               long long stride, int hpc, int tpc) {
    const cuuint64_t G = (cuuint64_t)(s.N / s.K), H = (cuuint64_t)s.H;
    const cuuint64_t dims[4] = {H, G, (cuuint64_t)s.K, (cuuint64_t)rows};
    const cuuint64_t strides[3] = {H * 2, G * H * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)hpc, 1, (cuuint32_t)tpc};
    return make_tensor_map(m, s.dtype, 4, q, dims, strides, box);
}

}  // namespace

size_t chunk_workspace_bytes(const gqa_shape& s, size_t flags_bytes) {
    const int sms = device_sm_count();
    if (sms < 1 || (size_t)sms * 2 * sizeof(int32_t) > flags_bytes) return 0;
    return flags_bytes + (size_t)sms * 4 * kRows * (s.H + 2) * sizeof(float);
}

gqa_status launch_chunk_attention(const gqa_shape& s, long long rows, long long q_stride,
                                  const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, bool head_tables,
                                  const int32_t* context_lens, const int32_t* cu_new, void* out,
                                  void* workspace, size_t flags_bytes, int32_t* dev_status,
                                  cudaStream_t stream) {
    if (s.B == 0 || rows == 0) return GQA_OK;
    if (s.B > kMaxSeqs) return GQA_ERR_SHAPE;
    const void* kern =
        s.dtype == GQA_BF16
            ? (s.H == 64 ? reinterpret_cast<const void*>(&chunk_attention_kernel<true, 64>)
                         : reinterpret_cast<const void*>(&chunk_attention_kernel<true, 128>))
            : (s.H == 64 ? reinterpret_cast<const void*>(&chunk_attention_kernel<false, 64>)
                         : reinterpret_cast<const void*>(&chunk_attention_kernel<false, 128>));
    const size_t smem = s.H == 64 ? chunk_smem<64>() : chunk_smem<128>();
    {
        // the shared-memory opt-in, once per device and kernel
        static std::mutex mu;
        static bool done[64][4] = {};
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GQA_ERR_CUDA;
        std::lock_guard<std::mutex> lock(mu);
        bool& d = done[dev][(s.dtype == GQA_BF16 ? 2 : 0) + (s.H == 64 ? 1 : 0)];
        if (!d && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem) != cudaSuccess)
            return GQA_ERR_CUDA;
        d = true;
    }
    ChunkParams p = {};
    p.G = s.N / s.K;
    p.cpt = (p.G + kRows - 1) / kRows;
    p.hpc = (p.G + p.cpt - 1) / p.cpt;
    p.tpc = p.cpt > 1 ? 1 : kRows / p.G;
    p.KC = s.K * p.cpt;
    p.out = out;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.cu_new = cu_new;
    p.status = dev_status;
    p.flags = static_cast<int32_t*>(workspace);
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + flags_bytes);
    p.B = s.B;
    p.M = (int)rows;
    p.N = s.N;
    p.K = s.K;
    p.max_blocks = s.max_blocks_per_seq;
    p.num_blocks = s.num_blocks;
    p.window = s.window;
    p.table_k = head_tables ? s.max_blocks_per_seq : 0;
    p.table_b = (long long)s.max_blocks_per_seq * (head_tables ? s.K : 1);
    const double scale = s.scale > 0.f ? (double)s.scale : 1.0 / sqrt((double)s.H);
    p.scale_log2 = (float)(scale * 1.4426950408889634);
    CUtensorMap tmk, tmv, tmq;
    if (!block_map(&tmk, k_cache, s) || !block_map(&tmv, v_cache, s) ||
        !query_map(&tmq, q, s, rows, q_stride, p.hpc, p.tpc))
        return GQA_ERR_CUDA;
    const int sms = device_sm_count();
    if (sms < 1) return GQA_ERR_CUDA;
    // no more CTAs than units can be (every item at the tables' width)
    const long long items = (rows + 2 * p.tpc - 1) / (2 * p.tpc) + s.B;
    const long long most = items * p.KC * ((s.max_blocks_per_seq + kBlocks - 1) / kBlocks + kStart);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max<long long>(
        1, std::min<long long>(sms, (most + kQuota - 1) / kQuota)));
    cfg.blockDim = dim3(kThreadsCh);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (s.flags & (GQA_FLAG_PDL | GQA_FLAG_EARLY_KV)) ? 1 : 0;
    void* args[] = {&tmk, &tmv, &tmq, &p};
    return launch_status(cudaLaunchKernelExC(&cfg, kern, args));
}

}  // namespace gqa
