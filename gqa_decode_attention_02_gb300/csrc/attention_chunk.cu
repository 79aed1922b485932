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
// running reference m (the row's maximum when it is set, in f16 7 less), O and l scaled when
// the maximum passes the one it was set by by more than 8 (in log2), O / l at the end.
//
// An item of work is a KV head and two row tiles (128 query rows each: tokens, and the G
// heads of each) of one sequence, and walks the 128-position KV tiles that its rows
// see.  Both row tiles use one copy of K and V in shared memory, and while one's softmax
// runs the tensor cores work for the other.  Items lie end to end in units of about
// equal time; every CTA takes an equal range of them, so that ragged batches, one short
// chunk behind a long prefix and single tokens all fill the GPU.  An item that a range
// boundary cuts (not near its ends) is shared: its pieces go to the workspace, and the CTA
// that draws the item's last ticket folds them, in order, with log-sum-exp weights (no
// CTA waits for another; the result does not depend on which CTA folds).
//
// One CTA per SM.  A row tile in the works has a slot: its Q in shared memory, S and O in
// tensor memory, four softmax warps and an issuer.
//   warps 0, 3    issue the MMAs of slots 0 and 1 (in turns: chunk_mma)
//   warp 1        loads K and V, one TMA box per cache block and KV head
//   warp 2        makes the list of pieces (KV tiles of an item) and loads Q
//   warps 4 - 11  softmax of slots 0 and 1, one thread per row, and the outputs
//   S_i[128 x 128] = Q_i K^T     Q_i and K from shared memory
//   P_i = exp2(S_i scale - m)    in q's dtype, over the first half of S_i's columns
//   O_i[128 x H]  += P_i V       P_i from tensor memory, V MN-major
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each, all there is.  An issuer's order is
// PV(j), QK(j + 1): S is overwritten by a product that follows, from the same thread, the
// one that reads P.  Shared memory: Q_0, Q_1 and a ring of K and V tiles, each per cache
// block [2 groups of 8 rows][H / 64 halves][8 rows x 128 B], 128-byte swizzled, so a block
// is one box and both operand layouts have one stride between row groups.
//
// What it rounds: probabilities to q's dtype before the product with V (by half a step, in f16
// at most 2^-32 of the row's sum where that is more), the result; sums of probabilities are taken before
// that rounding, in fp32 as the scores and O.
//
// Measured (one GB300, H = 128, bf16, 32 / 8 heads): 2,048 tokens behind 30,720 765 us, 1.39
// PFLOP/s, 72 % of what a library product of 8192^3 reaches; a step takes 1.75 us (3,300 cycles)
// for 2,048 cycles of MMAs.  A slot's chain is that long: softmax 1,350 cycles, hand-overs 400,
// its PV and QK 1,600 from the first to the last (issued by one thread that waits for nothing,
// the same products take 1,024; with the issuers' waits, turns and commits alone 1,310; the
// rest is the other slot's, still in the queue).  Short prompts (24 of 200..3,001): 519 us, of
// it some 100 at the items' ends, where both slots store outputs at once.  Single tokens,
// 256 x 2,048: 353 us, 6.1 TB/s.
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
// Registers per thread: the softmax warps hold 128 scores each.  Together no more than the
// launch's 384 x 168.
constexpr int kRegsIssue = 88, kRegsSoft = 208;
static_assert(128 * kRegsIssue + 256 * kRegsSoft <= kThreadsCh * 168, "register split");
// Units of work: a KV tile of an item with one row tile (its bytes: 1.5 us) or two (its
// MMAs: 1.8 us), an item's start and end; and per CTA at least.  Measured at H = 128, 16-bit
// rows, G = 4, and used for H = 64 and every G too: they only steer the balance.
constexpr int kLone = 5, kPair = 6, kStart = 10, kQuota = 10;
// A range boundary this near to an item's start or end moves there: a smaller piece is not
// worth its fold (some 5 us with one row tile of few rows, 20 with two full ones; for one
// row tile 2 KV tiles are: 4,096 tokens of 8 heads 21.2 us, with twice kNearLone and kQuota
// 23.7).
constexpr int kNearLone = kLone, kNearPair = 8 * kPair;
constexpr float kSlack = 8.f;  // log2 slack before O is rescaled
// How far below a row's maximum its reference is set (log2).  In f16 the largest probability
// is then 2^7 .. 2^15, near the top of the type's range, and what rounding takes from small
// ones (2^-25 each) is 2^-32 of it: with the reference at the maximum, positions 17 nats behind
// it were lost altogether, however many they are.  bf16 has fp32's range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;
// Scores from which on fp32 numbers are so far apart (2 in f16, 64 in bf16) that a score
// scaled in the fma that takes the reference off, not rounded as the reference was, could
// lie above the slack by more than the type's range (see far_tile).
template <bool BF16>
constexpr float kFar = BF16 ? 0x1p29f : 0x1p24f;
constexpr int kFarBit = 1 << 30;  // positions are below
constexpr int kPieces = 8;      // pieces between the scheduler and the last role
constexpr int kMaxSeqs = 16384;
constexpr uint32_t kColS = 0, kColO = 256;  // tensor-memory columns, 128 per slot

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
    int32_t* flags;         // tickets: of the item whose first piece a CTA holds
    float* partials;        // [grid][2][2][kPart]: slot 0 a later piece, slot 1 a first one
    int B, M, N, G;
    int tpc, hpc, cpt, KC;  // tokens and heads of a row tile; head chunks per KV head
    int max_blocks, num_blocks, window;
    long long table_b, table_k;  // strides of the block tables
    float scale_log2;
};

// A sequence's new rows, or none where its lengths are out of range.
struct Seq {
    int n, ctx, r0;
    int code;  // 0, or the error
};
// KV tiles [t0, t1) of an item, as the scheduler hands them to the other roles (t0 < 0: no
// more).  Per slot: its row tile's KV tiles [a, b) within the piece, rows in use (0: none),
// first row of q and out and its position.
struct Piece {
    int t0, t1;
    int a[2], b[2], count[2], row0[2], pos[2], tile[2];
    int kv, h0;              // KV head, first query head in its group
    int see_lo, see_hi;      // positions that the item's rows see
    int first_cta, last_cta; // CTAs that share the item
    long long table;         // its row of the block tables
};
struct ChunkSmem {
    uint64_t full[8], empty[8];
    uint64_t piece_full[kPieces], piece_free[kPieces];
    // per slot (a row tile in the works: its Q, S, O and softmax warps)
    uint64_t q_full[2], q_free[2], s_ready[2], p_ready[2], o_ready[2], o_free[2], done[2];
    uint64_t all;  // the softmax threads
    long long c0, c1, base;  // range of units; first unit of the first item
    long long quota;
    int b0, vh0, qi0, nq0;
    Seq seq0;                // sequence b0, its items per virtual head
    uint32_t tmem, lock;
    volatile int abort_flag;
    volatile int bad[kPieces];
    // the items that the CTA shares: 0 as a later piece of one, 1 as the first
    struct {
        int first_cta, pieces, kv, h0;
    } shared[2];
    int shared_rows[2][2], shared_count[2][2];  // per row tile
    int ticket[2];
    Piece pieces[kPieces];
};

// Waits for the phase of a barrier with the given parity; false after some four seconds: a
// poll that fails lasts 1.97 us (measured).  (ptx.cuh's wait reads a clock; this kernel waits
// in some thirty places, and what it runs in turn has to stay in the instruction cache: with
// the clock prompts took 3 to 7 % longer.)
constexpr uint32_t kPolls = 1u << 21;
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t n = 0; n < kPolls; ++n)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

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
__device__ __noinline__ int item_units(const ChunkParams& p, const Seq& s, int qi) {
    const int f = qi * 2 * p.tpc, e = min(s.n, f + 2 * p.tpc);
    return (tile_hi(s, e) - tile_lo(p, s, f)) * (f + p.tpc < e ? kPair : kLone) + kStart;
}

__device__ __forceinline__ void give_up(ChunkSmem& sm, const ChunkParams& p) {
    report(p.status, GQA_ERR_TIMEOUT);
    sm.abort_flag = 1;
}

// a / b for a >= 0, b > 0 (32 bits where they do)
__device__ __noinline__ long long div_ll(long long a, long long b) {
    if ((a | b) >> 32 == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// The pieces of the CTA's range in order.  Lone row tiles take the two slots in turn, so
// that one's end and the next one's start overlap.
struct Walk {
    long long c0, c1, base, quota;
    int b, vh, qi, nq, turn;
    Seq s, ahead;  // of sequences b and b + 1
    __device__ void load(const ChunkParams& p) {
        s = ahead;
        nq = items_of(p, s);
        if (b + 1 < p.B) ahead = read_seq(p, b + 1);
    }
    __device__ void init(const ChunkSmem& sm, const ChunkParams& p) {
        c0 = sm.c0;
        c1 = sm.c1;
        base = sm.base;
        quota = sm.quota;
        b = sm.b0;
        vh = sm.vh0;
        qi = sm.qi0;
        nq = turn = 0;
        if (c0 < c1) {
            s = sm.seq0;
            nq = sm.nq0;
            if (b + 1 < p.B) ahead = read_seq(p, b + 1);
        } else {
            base = c1;  // nothing for this CTA
        }
    }
    __device__ bool next(const ChunkParams& p, Piece& pc) {
        while (base < c1) {
            if (nq == 0) {
                if (++b >= p.B) break;
                load(p);
                continue;
            }
            const int f = qi * 2 * p.tpc, e = min(s.n, f + 2 * p.tpc), mid = min(e, f + p.tpc);
            const int lo = tile_lo(p, s, f), hi = tile_hi(s, e);
            // (a KV tile is the CTA's in whose range its first unit lies)
            const int each = mid < e ? kPair : kLone, near = mid < e ? kNearPair : kNearLone;
            const long long first = base + kStart, end = first + (long long)(hi - lo) * each;
            int from = lo, to = hi;
            if (c0 > first + near)
                from = end - c0 <= near ? hi : lo + (int)div_ll(c0 - first + each - 1, each);
            if (c1 < end) {
                if (c1 <= first + near)
                    to = lo;
                else if (end - c1 > near)
                    to = lo + (int)div_ll(c1 - first + each - 1, each);
            }
            if (from < to) {
                pc.t0 = from;
                pc.t1 = to;
                const int kv = p.cpt > 1 ? vh / p.cpt : vh;
                pc.kv = kv;
                pc.h0 = (vh - kv * p.cpt) * p.hpc;
                pc.table = b * p.table_b + kv * p.table_k;
                const int at = s.ctx - s.n;  // position of the first new token
                pc.see_lo = p.window > 0 ? max(0, at + f - p.window + 1) : 0;
                pc.see_hi = at + e;
                // the CTAs whose ranges begin in the item, but for its ends
                const bool cut = to - from != hi - lo;
                pc.first_cta = cut ? (int)div_ll(first + near, quota) : -1;
                pc.last_cta = cut ? (int)div_ll(end - near - 1, quota) : -1;
                const int heads = min(p.hpc, p.G - pc.h0);
                const bool lone = mid == e;
                for (int i = 0; i < 2; ++i) {
                    const int tile = lone ? i ^ turn : i;
                    const int tf = tile ? mid : f, te = tile ? e : mid;
                    pc.tile[i] = tile;
                    pc.row0[i] = s.r0 + tf;
                    pc.pos[i] = at + tf;
                    pc.count[i] = tf < te ? (te - tf - 1) * p.hpc + heads : 0;
                    pc.a[i] = pc.b[i] = pc.t0;
                    if (tf < te) {
                        pc.a[i] = max(pc.t0, tile_lo(p, s, tf));
                        pc.b[i] = max(pc.a[i], min(pc.t1, tile_hi(s, te)));
                    }
                }
                if (lone) turn ^= 1;
            }
            base = end;
            if (++qi == nq) {
                qi = 0;
                if (++vh == p.KC) {
                    vh = 0;
                    nq = 0;
                }
            }
            if (from < to) return true;
        }
        return false;
    }
};

__device__ __forceinline__ long long shfl_ll(long long v, int src) {
    return __shfl_sync(kAll, v, src);
}
__device__ __forceinline__ long long scan_ll(long long v, int lane) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += x;
    }
    return v;
}
// Rows [r0, r0 + n) of the output become zeros (whole warp).
template <int H>
__device__ __noinline__ void zero_rows(const ChunkParams& p, int r0, int n) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (size_t)r0 * p.N * H);
    const long long count = (long long)n * p.N * (H / 8);
#pragma unroll 1
    for (long long i = threadIdx.x & 31; i < count; i += 32) o[i] = make_uint4(0, 0, 0, 0);
}

// (The plan's loops stay rolled and its helpers calls: its code runs once, and fetching it
// counts: 64 x 2,048 tokens 101.4 us with everything inline, 99.5 so.)
// Units of one virtual head of sequences first .. first + 31, a lane each (whole warp);
// CTA 0 also reports and clears those out of range.
template <int H>
__device__ long long warp_units(const ChunkParams& p, int first, Seq& s) {
    const int lane = threadIdx.x & 31, b = first + lane;
    s = {0, 0, 0, 0};
    if (b < p.B) s = read_seq(p, b);
    const int nq = items_of(p, s);
    long long c = 0;
    if (nq <= 4)
#pragma unroll 1
        for (int qi = 0; qi < nq; ++qi) c += item_units(p, s, qi);
    unsigned many = __ballot_sync(kAll, nq > 4);
    while (many) {
        const int src = __ffs(many) - 1;
        many &= many - 1;
        Seq t;
        t.n = __shfl_sync(kAll, s.n, src);
        t.ctx = __shfl_sync(kAll, s.ctx, src);
        const int m = __shfl_sync(kAll, nq, src);
        long long x = 0;
#pragma unroll 1
        for (int qi = lane; qi < m; qi += 32) x += item_units(p, t, qi);
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
        if (lane == src) c = x;
    }
    if (blockIdx.x == 0 && __any_sync(kAll, s.code != 0)) {
        if (s.code) report(p.status, GQA_ERR_CONTEXT);
        unsigned zero = __ballot_sync(kAll, s.code == 1);
        while (zero) {
            const int at = first + __ffs(zero) - 1;
            zero &= zero - 1;
            const int r0 = p.cu_new ? __ldg(p.cu_new + at) : at;
            const int r1 = p.cu_new ? __ldg(p.cu_new + at + 1) : at + 1;
            zero_rows<H>(p, r0, r1 - r0);
        }
    }
    return c;
}

// All warps: units of every sequence (`cost`, shared memory; with no more than a lane each
// warp 0 alone), then warp 0: this CTA's range and the item it starts in.
template <int H>
__device__ void chunk_plan(const ChunkParams& p, ChunkSmem& sm, long long* cost) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool few = p.B <= 32;
    Seq s;
    long long local = 0;
    int lo = lane, hi = min(p.B, lane + 1);  // this lane's sequences
    if (few) {
        if (warp != 0) return;
        local = warp_units<H>(p, 0, s);
    } else {
        for (int first = warp * 32; first < p.B; first += kThreadsCh) {
            const long long c = warp_units<H>(p, first, s);
            if (first + lane < p.B) cost[first + lane] = c;
        }
        __syncthreads();
        if (warp != 0) return;
        const int per = (p.B + 31) / 32;
        lo = min(p.B, lane * per);
        hi = min(p.B, lo + per);
        for (int b = lo; b < hi; ++b) local += cost[b];
    }
    const long long incl = scan_ll(local, lane), excl = incl - local;
    const long long total = shfl_ll(incl, 31) * p.KC;
    const long long quota =
        max(div_ll(total + gridDim.x - 1, gridDim.x), (long long)kQuota);
    const long long c0 = blockIdx.x * quota, c1 = min(total, c0 + quota);
    const bool mine = c0 < c1 && excl * p.KC <= c0 && c0 < incl * p.KC;
    const unsigned owners = __ballot_sync(kAll, mine);
    int b0 = 0;
    long long base = 0, one = 0;  // first unit of b0; units of a virtual head of it
    if (mine) {
        base = excl * p.KC;
        b0 = lo;
        one = local;
        if (!few) {
            while (c0 >= base + cost[b0] * p.KC) base += cost[b0++] * p.KC;
            one = cost[b0];
        }
    }
    const int owner = owners ? __ffs(owners) - 1 : 0;
    b0 = __shfl_sync(kAll, b0, owner);
    base = shfl_ll(base, owner);
    one = shfl_ll(one, owner);
    if (lane == 0) {
        sm.c0 = c0;
        sm.c1 = max(c0, c1);
        sm.quota = quota;
        sm.b0 = b0;
        sm.qi0 = 0;
    }
    __syncwarp();
    if (owners) {
        // the virtual head, then the item in it (a run of items per lane)
        Seq t;
        if (few) {
            t.n = __shfl_sync(kAll, s.n, owner);
            t.ctx = __shfl_sync(kAll, s.ctx, owner);
            t.r0 = __shfl_sync(kAll, s.r0, owner);
            t.code = 0;
        } else {
            t = read_seq(p, b0);
        }
        const int nq = items_of(p, t);
        const int vh = (int)div_ll(c0 - base, one);
        base += vh * one;
        if (lane == 0) {
            sm.seq0 = t;
            sm.nq0 = nq;
            sm.vh0 = vh;
            sm.base = base;
        }
        if (nq == 1) return;
        __syncwarp();
        const int run = (nq + 31) / 32;
        const int qlo = min(nq, lane * run), qhi = min(nq, qlo + run);
        long long x = 0;
#pragma unroll 1
        for (int qi = qlo; qi < qhi; ++qi) x += item_units(p, t, qi);
        const long long xi = scan_ll(x, lane), xe = xi - x;
        if (base + xe <= c0 && c0 < base + xi) {
            long long at = base + xe;
            int qi = qlo;
            while (true) {
                const int u = item_units(p, t, qi);
                if (c0 < at + u) break;
                at += u;
                ++qi;
            }
            sm.qi0 = qi;
            sm.base = at;
        }
    }
}

// ---------------------------------------------------------------------------
// Waits for piece k of the CTA; false after a time-out or an abort.
__device__ __forceinline__ bool piece_ready(ChunkSmem& sm, int k) {
    return wait_for(smem_addr(&sm.piece_full[k % kPieces]), (k / kPieces) & 1) && !sm.abort_flag;
}
__device__ __forceinline__ void piece_done(ChunkSmem& sm, int k) {
    mbar_arrive(smem_addr(&sm.piece_free[k % kPieces]));
}

// Warp 1: K and V tiles into the ring, K(j) then V(j).  A lane per cache block; block
// ids are read 32 at a time, the next ones while these are in use.
template <int H>
__device__ void chunk_load(const CUtensorMap* tmk, const CUtensorMap* tmv, const ChunkParams& p,
                           uint8_t* ring, ChunkSmem& sm) {
    using C = Ch<H>;
    const int lane = threadIdx.x & 31;
    int it = 0, r = 0;
    uint32_t ph = 1;  // phase whose end frees slot r (none at first)
    bool aborted = false;
    for (int k = 0;; ++k) {
        aborted = __any_sync(kAll, !piece_ready(sm, k));
        if (aborted) break;
        const Piece& pc = sm.pieces[k % kPieces];
        const int t0 = pc.t0, t1 = pc.t1, kv = pc.kv;
        if (t0 < 0) break;
        const int32_t* table = p.block_tables + pc.table;
        // blocks that the item's rows see: none below the window, none past its last token
        const int blo = pc.see_lo / 16, bhi = (pc.see_hi + 15) / 16;
        __syncwarp();
        if (lane == 0) {
            sm.bad[k % kPieces] = 0;
            piece_done(sm, k);
        }
        auto load_ids = [&](int from) {
            const int i = from + lane;
            return i >= blo && i < bhi ? __ldg(table + i) : 0;
        };
        int win = t0 * kBlocks, ids = load_ids(win), nxt = load_ids(win + 32);
        for (int j = t0; j < t1 && !aborted; ++j) {
            if (j * kBlocks - win == 32) {
                win += 32;
                ids = nxt;
                nxt = load_ids(win + 32);
            }
            const int id = __shfl_sync(kAll, ids, (j * kBlocks - win + lane) & 31);
            const int blk = j * kBlocks + lane;
            const bool mine = lane < kBlocks && blk >= blo && blk < bhi;
            const bool bad = __any_sync(kAll, mine && (id < 0 || id >= p.num_blocks));
            // (a block that no row sees: past the tensor's end, which reads as zeros)
            const int at = mine ? 2 * id : 2 * p.num_blocks;
#pragma unroll 1
            for (int kvsel = 0; kvsel < 2; ++kvsel) {
                const uint32_t bar = smem_addr(&sm.full[r]);
                if (lane == 0) {
                    bool ok = it < C::kSlots || wait_for(smem_addr(&sm.empty[r]), ph);
                    if (!ok) give_up(sm, p);
                    aborted = !ok || sm.abort_flag;
                    if (!aborted) {
                        if (bad) {
                            report(p.status, GQA_ERR_BLOCK_ID);
                            sm.bad[k % kPieces] = 1;
                            __threadfence_block();
                            mbar_arrive(bar);
                        } else {
                            mbar_arrive_expect_tx(bar, (uint32_t)C::kTile);
                        }
                    }
                }
                aborted = __shfl_sync(kAll, aborted, 0);
                if (aborted) break;
                if (lane < kBlocks && !bad)
                    tma_load_5d(smem_addr(ring + (size_t)r * C::kTile) + lane * 2 * C::kGroup,
                                kvsel ? tmv : tmk, bar, 0, 0, 0, at, kv);
                ++it;
                if (++r == C::kSlots) {
                    r = 0;
                    ph ^= 1;
                }
            }
        }
        if (aborted) break;
    }
    if (lane == 0 && aborted)  // copies in flight land before the CTA ends
        for (int j = max(0, it - C::kSlots); j < it; ++j)
            wait_for(smem_addr(&sm.full[j % C::kSlots]), (j / C::kSlots) & 1);
}

// ---------------------------------------------------------------------------
// Warp 2, one lane: the pieces, two ahead of the queries it loads, and the Q tiles of each,
// a slot's once the products of the last one have read theirs.  Rows past the
// sequence's last token are the next sequence's (or zeros past the tensor): their
// results are not stored.
template <int H>
__device__ void chunk_schedule(const CUtensorMap* tmq, const ChunkParams& p, uint8_t* qbuf,
                               ChunkSmem& sm) {
    using C = Ch<H>;
    if ((threadIdx.x & 31) != 0) return;
    Walk wk;
    wk.init(sm, p);
    int out = 0, in = 0;  // pieces handed out; pieces whose queries are on their way
    uint32_t loads[2] = {0, 0};
    bool more = true, ok = true;
    while (ok) {
        if (more && out < in + 3) {
            const int e = out % kPieces;
            if (out >= kPieces)
                ok = wait_for(smem_addr(&sm.piece_free[e]), (out / kPieces - 1) & 1);
            if (!ok) break;
            more = wk.next(p, sm.pieces[e]);
            if (!more) sm.pieces[e].t0 = -1;
            mbar_arrive(smem_addr(&sm.piece_full[e]));
            if (more) ++out;
            continue;
        }
        if (in == out) break;
        const Piece& pc = sm.pieces[in % kPieces];
#pragma unroll 1
        for (int i = 0; i < 2 && ok; ++i) {
            if (pc.a[i] >= pc.b[i]) continue;
            if (loads[i] > 0) ok = wait_for(smem_addr(&sm.q_free[i]), (loads[i] - 1) & 1);
            if (!ok || sm.abort_flag) {
                ok = false;
                break;
            }
            const uint32_t bar = smem_addr(&sm.q_full[i]);
            mbar_arrive_expect_tx(bar, (uint32_t)(C::kHalves * 128 * p.tpc * p.hpc));
#pragma unroll 1
            for (int h = 0; h < C::kHalves; ++h)
                tma_load_4d(smem_addr(qbuf) + i * C::kTile + h * (kRows * 128), tmq, bar, 64 * h,
                            pc.h0, pc.kv, pc.row0[i]);
            ++loads[i];
        }
        ++in;
    }
    if (!ok) {
        give_up(sm, p);
        for (int i = 0; i < 2; ++i)  // copies in flight land before the CTA ends
            if (loads[i] > 0) wait_for(smem_addr(&sm.q_full[i]), (loads[i] - 1) & 1);
    }
}

// ---------------------------------------------------------------------------
// Warps 0 and 3, one lane each: the MMAs of a slot.  QK of a KV tile, PV of it once its
// probabilities are written, QK of the next one behind it.  An issuer's wait costs some
// 100 cycles even when there is nothing to wait for, and the tensor cores' queue is a few
// MMAs deep: two issuers hide each other's waits.  They take turns by a lock, a PV and the
// QK behind it at a time: interleaved, both slots' products would end together, then
// both softmaxes run while the tensor cores rest (measured 2.4 us per pair of tiles).  A
// turn ends two MMAs before its products do, about what handing it over takes (24 prompts:
// none 523.6 us, one 523.8, two 521.6, three 523.0, four 525.3, six 540.3).
__device__ __forceinline__ bool take_turn(ChunkSmem& sm) {
    const uint32_t lock = smem_addr(&sm.lock);
#pragma unroll 1
    for (uint32_t n = 0; n < 32 * kPolls; ++n) {  // bounded: 17 ns a try
        uint32_t old;
        asm volatile("atom.acquire.cta.shared::cta.exch.b32 %0, [%1], 1;"
                     : "=r"(old)
                     : "r"(lock)
                     : "memory");
        if (old == 0) return true;
    }
    return false;
}
__device__ __forceinline__ void end_turn(ChunkSmem& sm) {
    asm volatile("st.release.cta.shared::cta.b32 [%0], 0;" ::"r"(smem_addr(&sm.lock)) : "memory");
}

template <bool BF16, int H>
__device__ void chunk_mma(const ChunkParams& p, uint8_t* ring, uint8_t* qbuf, ChunkSmem& sm,
                          int I) {
    using C = Ch<H>;
    if ((threadIdx.x & 31) != 0) return;
    constexpr uint32_t id_s = umma_idesc_ct(BF16, kRows, kStep, false);
    constexpr uint32_t id_o = umma_idesc_ct(BF16, kRows, H, true);
    const uint32_t tS = sm.tmem + kColS + I * 128, tO = sm.tmem + kColO + I * 128;
    const uint64_t dq = umma_desc_sw128(smem_addr(qbuf) + I * C::kTile, 16, 1024);
    const uint64_t dk0 = umma_desc_sw128(smem_addr(ring), 16, C::kGroup);
    const uint64_t dv0 = umma_desc_sw128(smem_addr(ring), 1024, C::kGroup);
    const uint32_t full = smem_addr(&sm.full[0]), empty = smem_addr(&sm.empty[0]);
    int r = 0;         // ring slot of the next tile
    uint32_t ph = 0;   // and its phase
    uint32_t steps = 0, pieces = 0;
    auto advance = [&]() {
        if (++r == C::kSlots) {
            r = 0;
            ph ^= 1;
        }
    };
    bool ok = true;
    auto qk = [&](bool last) {  // S = Q K^T, K in ring slot r
        const uint64_t dk = dk0 + (uint32_t)(r * (C::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < H / 16; ++kk) {
            if (kk == H / 16 - 2) end_turn(sm);
            umma_ss(tS, dq + (uint64_t)(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4),
                    dk + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_s, kk > 0);
        }
        umma_commit(smem_addr(&sm.s_ready[I]));
        umma_commit(empty + 8 * r);
        if (last) umma_commit(smem_addr(&sm.q_free[I]));
        advance();
    };
    for (int k = 0; ok; ++k) {
        ok = piece_ready(sm, k);
        if (!ok) break;
        const Piece& pc = sm.pieces[k % kPieces];
        const int t0 = pc.t0, t1 = pc.t1, ja = pc.a[I], jb = pc.b[I];
        if (t0 < 0) break;
        piece_done(sm, k);
        bool begun = false;  // QK of tile j has been issued
        for (int j = t0; j < t1 && ok; ++j) {
            if (j < ja || j >= jb) {  // not seen by this slot's rows
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    ok = wait_for(full + 8 * r, ph);
                    mbar_arrive(empty + 8 * r);
                    advance();
                }
                continue;
            }
            if (j == ja) ok = wait_for(smem_addr(&sm.q_full[I]), pieces & 1);
            if (!begun) {
                ok = ok && wait_for(full + 8 * r, ph) && take_turn(sm);
                if (!ok) break;
                qk(j + 1 == jb);
            }
            begun = false;
            ok = wait_for(full + 8 * r, ph) && wait_for(smem_addr(&sm.p_ready[I]), steps & 1);
            ++steps;
            if (j == ja && pieces > 0)  // O of the last piece has been read
                ok = ok && wait_for(smem_addr(&sm.o_free[I]), (pieces - 1) & 1);
            ok = ok && !sm.abort_flag && take_turn(sm);
            if (!ok) break;
            tc_fence_after();
            const int rk = r + 1 == C::kSlots ? 0 : r + 1;
            begun = j + 1 < jb && mbar_test(full + 8 * rk, rk ? ph : ph ^ 1);
            {
                const uint64_t dv = dv0 + (uint32_t)(r * (C::kTile >> 4));
                umma_ts(tO, tS, dv, id_o, j > ja);
#pragma unroll
                for (int ks = 1; ks < kBlocks; ++ks) {
                    if (ks == kBlocks - 2 && !begun) end_turn(sm);
                    umma_ts(tO, tS + 8 * ks, dv + (uint64_t)((ks * 2 * C::kGroup) >> 4), id_o, true);
                }
                umma_commit(smem_addr(&sm.o_ready[I]));
                umma_commit(empty + 8 * r);
                advance();
            }
            if (begun) qk(j + 2 == jb);
        }
        if (ja < jb) ++pieces;
    }
    if (!ok) give_up(sm, p);
    umma_commit(smem_addr(&sm.done[I]));  // every MMA ends before tensor memory is freed
    if (!wait_for(smem_addr(&sm.done[I]), 0)) give_up(sm, p);
}

// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lo2(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// O's row scaled by f.
template <int H>
__device__ __forceinline__ void scale_o(uint32_t tO, float f) {
#pragma unroll 1
    for (int c = 0; c < H / 16; ++c) {
        uint32_t o[16];
        tmem_ld16(tO + 16 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
        tmem_st16(tO + 16 * c, o);
    }
    tmem_wait_st();
}
// Columns [a, b) of the 32 from 0 on, as bits.
__device__ __forceinline__ uint32_t columns(int a, int b) {
    return (b >= 32 ? ~0u : b <= 0 ? 0u : ~(~0u << b)) & (a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a);
}

// The softmax of a tile whose scores, or an earlier tile's, lie beyond kFar, of a warp's 32
// rows: as chunk_softmax does it, but with the scaled scores rounded before the reference
// is taken off.  Rare, and a call: with the mask's loop scaling the scores too, inline, prompts
// took 3.5 % longer; so 24 prompts 543 us, 543 without any of it.
struct Sums {
    float m, l;
    bool ok;
};
template <bool BF16, int H>
__device__ __noinline__ Sums far_tile(uint32_t tS, uint32_t tO, int from, int to, float scale,
                                      float m, float l, uint32_t bO, int o_phase) {
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        const uint32_t seen = columns(from - 32 * c, to - 32 * c);
        uint32_t x[32];
        tmem_ld32(tS + 32 * c, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const float y = seen >> e & 1u ? __fmul_rn(__uint_as_float(x[e]), scale) : -INFINITY;
            top = fmaxf(top, y);
            x[e] = __float_as_uint(y);
        }
        tmem_st32(tS + 32 * c, x);
    }
    tmem_wait_st();
    const bool need = __fsub_rn(top, m) > kSlack + kLift<BF16>;
    if (__any_sync(kAll, need)) {
        const float next = __fsub_rn(top, kLift<BF16>);
        const float f = need && m != -INFINITY ? fast_exp2(m - next) : 1.f;
        if (o_phase >= 0 && __any_sync(kAll, f != 1.f)) {
            if (!__all_sync(kAll, wait_for(bO, o_phase))) return {m, l, false};
            tc_fence_after();
            scale_o<H>(tO, f);
        }
        if (need) {
            l *= f;
            m = next;
        }
    }
    const float ref = m == -INFINITY ? 0.f : -m;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t x[32], w[16];
        tmem_ld32(tS + 32 * c, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float a = fast_exp2(__fadd_rn(__uint_as_float(x[2 * e]), ref));
            const float b = fast_exp2(__fadd_rn(__uint_as_float(x[2 * e + 1]), ref));
            w[e] = Elt<BF16>::pack(a, b);
            l += a + b;
        }
        tmem_st16(tS + 16 * c, w);
    }
    tmem_wait_st();
    return {m, l, true};
}

// Softmax of the row tiles in slot i, a thread per row.
template <bool BF16, int H>
__device__ bool chunk_softmax(const ChunkParams& p, uint8_t* ring, ChunkSmem& sm) {
    using C = Ch<H>;
    using E = Elt<BF16>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = (warp - kSoftWarp) >> 2;           // slot
    const int row = 32 * (warp & 3) + lane;          // tensor-memory lane
    const int tid = row;                             // within the slot's 128 threads
    const int row_t = row / p.hpc;
    // Outputs are stored by quads of threads, each 64 bytes of a row of the quad at a time:
    // the four rows, in 16-byte pieces from the tile's first
    uint32_t quad[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int r = (row & ~3) + x;
        quad[x] = ((uint32_t)(r / p.hpc) * p.N + r % p.hpc) * (H / 8) + (lane & 3);
    }
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = sm.tmem + kColS + i * 128 + lanes, tO = sm.tmem + kColO + i * 128 + lanes;
    const uint32_t bS = smem_addr(&sm.s_ready[i]), bP = smem_addr(&sm.p_ready[i]),
                   bO = smem_addr(&sm.o_ready[i]), bF = smem_addr(&sm.o_free[i]);
    const uint64_t scale2 = pair2(p.scale_log2, p.scale_log2);
    int step = 0, n0 = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        ok = __all_sync(kAll, piece_ready(sm, k));
        if (!ok) break;
        const Piece& pc = sm.pieces[k % kPieces];
        const int t0 = pc.t0, ja = pc.a[i], jb = pc.b[i], count = pc.count[i];
        if (t0 < 0) break;
        const int ring0 = n0;
        n0 += 2 * (pc.t1 - t0);
        auto release = [&]() {
            __syncwarp();
            if (lane == 0) piece_done(sm, k);
        };
        if (count == 0) {  // no tokens for this slot
            release();
            continue;
        }
        const bool active = row < count;
        const bool warp_on = 32 * (warp & 3) < count;
        const int lim = pc.pos[i] + (active ? row_t : 0);
        // (with kFarBit once a row of the warp had scores beyond kFar: no tile is seen whole)
        int low = p.window > 0 ? max(0, lim - p.window + 1) : 0;
        const int see_lo = pc.see_lo, see_hi = pc.see_hi;
        float m = -INFINITY, l = 0.f;
        for (int j = ja; j < jb; ++j, ++step) {
            ok = __all_sync(kAll, wait_for(bS, step & 1));
            if (!ok) break;
            const int tok = j * kStep;
            auto far = [&]() {
                low |= kFarBit;
                const Sums x = far_tile<BF16, H>(tS, tO, low - kFarBit - tok, lim + 1 - tok,
                                                 p.scale_log2, m, l, bO,
                                                 j > ja ? (step - 1) & 1 : -1);
                m = x.m;
                l = x.l;
                ok = x.ok;
            };
            if (warp_on) do {
                tc_fence_after();
                const int from = low - tok, to = lim + 1 - tok;  // columns seen
                if (!__all_sync(kAll, from <= 0 && to >= kStep)) {
                    if (low >= kFarBit) {
                        far();
                        break;
                    }
                    // some are not: -inf there, in tensor memory (a loop of its own, so
                    // that the code of the tiles seen whole stays short)
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t seen = columns(from - 32 * c, to - 32 * c);
                        if (__all_sync(kAll, seen == ~0u)) continue;
                        uint32_t x[32];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen >> e & 1u)) x[e] = 0xff800000u;
                        tmem_st32(tS + 32 * c, x);
                    }
                    tmem_wait_st();
                }
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s[c]);
                tmem_wait_ld();
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                    for (int x = 2; x < 32; x += 2)
                        mx[c] = max3(mx[c], __uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1]));
                }
                const float top =
                    __fmul_rn(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), p.scale_log2);
                const bool need = __fsub_rn(top, m) > kSlack + kLift<BF16>;
                if (__any_sync(kAll, need)) {
                    if (__any_sync(kAll, need && active && fabsf(top) >= kFar<BF16>)) {
                        far();
                        break;
                    }
                    const float next = __fsub_rn(top, kLift<BF16>);
                    const float f = need && m != -INFINITY ? fast_exp2(m - next) : 1.f;
                    if (j > ja && __any_sync(kAll, f != 1.f)) {  // the last PV has ended
                        ok = __all_sync(kAll, wait_for(bO, (step - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        scale_o<H>(tO, f);
                    }
                    if (need) {
                        l *= f;
                        m = next;
                    }
                }
                const float ref = m == -INFINITY ? 0.f : -m;
                const uint64_t ref2 = pair2(ref, ref);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const uint64_t y = fma2(pair2(__uint_as_float(s[c][2 * x]),
                                                      __uint_as_float(s[c][2 * x + 1])),
                                                scale2, ref2);
                        const float a = fast_exp2(lo2(y)), b = fast_exp2(hi2(y));
                        w[x] = E::pack(a, b);
                        sum[x & 1] = add2(sum[x & 1], pair2(a, b));
                    }
                    tmem_st16(tS + 16 * c, w);
                }
                const uint64_t both = add2(sum[0], sum[1]);
                l += lo2(both) + hi2(both);
                tmem_wait_st();
            } while (false);
            if (!ok) break;
            // V rows of a block that rows of the item see in part: the others hold anything
            // and become zeros, since 0 * NaN counts (whole blocks came as zeros)
            const int v0 = max(0, see_lo - tok), v1 = min(kStep, see_hi - tok);
            const int z0 = v0 & 15, z = z0 + (-v1 & 15);  // rows before v0 and from v1 on
            if (z > 0) {
                const int nv = ring0 + 2 * (j - t0) + 1;
                ok = __all_sync(kAll, wait_for(smem_addr(&sm.full[nv % C::kSlots]),
                                                (nv / C::kSlots) & 1));
                if (!ok) break;
                const uint32_t vb = smem_addr(ring + (size_t)(nv % C::kSlots) * C::kTile);
                // (every 16 bytes of a row, wherever the swizzle puts them)
                for (int x = tid; x < z * (H / 8); x += kRows) {
                    const int k = x / (H / 8), c = x % (H / 8);
                    const int r = k < z0 ? v0 - 1 - k : v1 + k - z0;
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
        const bool some = ja < jb;  // any KV tile in this piece
        if (some) {
            ok = __all_sync(kAll, wait_for(bO, (step - 1) & 1));
            if (!ok) break;
            tc_fence_after();
        }
        // (set before the tiles landed; without one, nothing has been waited for)
        const bool bad = some && sm.bad[k % kPieces] != 0;
        const int first_cta = pc.first_cta, tile = pc.tile[i];
        uint4* const out = reinterpret_cast<uint4*>(
            static_cast<uint16_t*>(p.out) +
            ((size_t)pc.row0[i] * p.N + (size_t)pc.kv * p.G + pc.h0) * H);
        const int w = (int)blockIdx.x == first_cta;  // an item's first piece ends its CTA's range
        if (first_cta >= 0 && tid == 0)
            sm.shared[w] = {first_cta, pc.last_cta - first_cta + 1, pc.kv, pc.h0};
        if (first_cta >= 0 && tid == 0) {
            sm.shared_rows[w][tile] = pc.row0[i];
            sm.shared_count[w][tile] = count;
        }
        release();
        // O_i in q's dtype, or, of a piece of an item that several CTAs share, as it is,
        // [128 rows][H], then the rows' references and sums.  64 bytes of a row at a time, in a
        // loop (code that runs once a piece is not in the instruction cache), stored by
        // quads of threads.
        const bool whole = first_cta < 0;
        float* const part =
            p.partials + ((size_t)((int)blockIdx.x * 2 + w) * 2 + tile) * C::kPart;
        const float inv = bad || l == 0.f ? 0.f : 1.f / l;  // (a NaN score: a NaN row)
        uint4* const dst = whole ? out : reinterpret_cast<uint4*>(part);
        if (warp_on && some) {
#pragma unroll 1
            for (int c = 0; c < (whole ? H / 32 : H / 16); ++c) {
                uint32_t w[4][4];
                if (whole) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        w[x >> 2][x & 3] = inv == 0.f
                                               ? 0u
                                               : E::pack(__uint_as_float(o[2 * x]) * inv,
                                                         __uint_as_float(o[2 * x + 1]) * inv);
                } else {
                    uint32_t o[16];
                    tmem_ld16(tO + 16 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 16; ++x) w[x >> 2][x & 3] = o[x];
                }
                // piece x of this thread's row <-> piece (lane & 3) of the quad's row x
#pragma unroll
                for (int y = 0; y < 4; ++y) {
#pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        const uint32_t u = __shfl_xor_sync(kAll, lane & 1 ? w[x][y] : w[x + 1][y], 1);
                        w[x][y] = lane & 1 ? u : w[x][y];
                        w[x + 1][y] = lane & 1 ? w[x + 1][y] : u;
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t u = __shfl_xor_sync(kAll, lane & 2 ? w[x][y] : w[x + 2][y], 2);
                        w[x][y] = lane & 2 ? u : w[x][y];
                        w[x + 2][y] = lane & 2 ? w[x + 2][y] : u;
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = (row & ~3) + x;
                    const uint32_t at = whole ? quad[x] : (uint32_t)(r * (H / 4) + (lane & 3));
                    if (r < count)
                        __stcg(dst + at + 4 * c, make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]));
                }
            }
        }
        tc_fence_before();
        if (some) mbar_arrive(bF);
        if (!whole) {
            __stcg(part + kRows * H + row, m);
            __stcg(part + kRows * (H + 1) + row, bad ? -1.f : l);  // a bad block shows as -1
            __threadfence();  // before the item's ticket
        }
    }
    if (!ok) give_up(sm, p);
    return ok;
}

// The softmax warps, when every piece of the CTA is done: for the items that it shares with
// others (the one that its range begins in, the one that it ends in), a ticket; the CTA
// that draws an item's last one folds the pieces.
template <bool BF16, int H>
__device__ void chunk_shared(const ChunkParams& p, ChunkSmem& sm, float* weight) {
    using C = Ch<H>;
    const int tid = threadIdx.x - 32 * kSoftWarp;
    int meets = 0;
    auto meet = [&]() {  // the softmax threads
        mbar_arrive(smem_addr(&sm.all));
        const bool ok = wait_for(smem_addr(&sm.all), meets & 1);
        ++meets;
        return ok;
    };
    if (!meet()) return give_up(sm, p);
    if (tid % kRows == 0 && sm.shared[tid / kRows].pieces > 0) {
        const int w = tid / kRows;
        int32_t* const flag = p.flags + sm.shared[w].first_cta;
        unsigned v;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(v) : "l"(flag) : "memory");
        sm.ticket[w] = (int)v;
        if ((int)v == sm.shared[w].pieces - 1) *flag = 0;  // as the next call wants it
    }
    if (!meet()) return give_up(sm, p);
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        const int first_cta = sm.shared[w].first_cta, pieces = sm.shared[w].pieces;
        if (pieces == 0 || sm.ticket[w] != pieces - 1) continue;
        __threadfence();
        auto part_of = [&](int c, int tile) {
            return p.partials + ((size_t)((first_cta + c) * 2 + (c == 0)) * 2 + tile) * C::kPart;
        };
        // weights of the pieces' rows, a thread per row of both tiles (in the shared memory
        // that tiles were in)
        {
            const float* const rows = part_of(0, tid / kRows) + kRows * H + tid % kRows;
            const float* const rest = part_of(1, tid / kRows) + kRows * H + tid % kRows;
            const bool on = tid % kRows < sm.shared_count[w][tid / kRows];
            float M = -INFINITY, L = 0.f;
            bool bad = false;
#pragma unroll 4
            for (int c = 0; c < pieces; ++c) {
                const float* q = c ? rest + (size_t)(c - 1) * 4 * C::kPart : rows;
                const float mc = on ? __ldcg(q) : 0.f, lc = on ? __ldcg(q + kRows) : 0.f;
                bad |= lc < 0.f;
                const bool seen = !(lc <= 0.f);  // else nothing in this piece
                const float top = seen ? fmaxf(M, mc) : M;
                const float f = M == -INFINITY ? 0.f : fast_exp2(M - top);
                L = fmaf(L, f, seen ? lc * fast_exp2(mc - top) : 0.f);
                M = top;
                weight[c * 2 * kRows + tid] = seen ? mc : -INFINITY;
            }
            const float inv = bad || L == 0.f ? 0.f : 1.f / L;
            for (int c = 0; c < pieces; ++c) {
                float& x = weight[c * 2 * kRows + tid];
                x = (x == -INFINITY ? 0.f : fast_exp2(x - M)) * inv;  // (a NaN stays one)
            }
        }
        if (!meet()) return give_up(sm, p);
        // four dims of a row at a time, in the pieces' order: four of them a thread and four
        // pieces at once, so that their reads overlap
        constexpr int V = H / 4, kEach = 4, kAtOnce = 4;
        const int n0 = sm.shared_count[w][0], total = (n0 + sm.shared_count[w][1]) * V;
#pragma unroll 1
        for (int x0 = tid; x0 < total; x0 += 2 * kRows * kEach) {
            float acc[kEach][4] = {};
            int row[kEach];  // of both tiles
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int r = (x0 + e * 2 * kRows) / V;
                row[e] = r < n0 ? r : r - n0 + kRows;
            }
#pragma unroll 1
            for (int c0 = 0; c0 < pieces; c0 += kAtOnce) {
                float4 v[kAtOnce][kEach];
                float f[kAtOnce][kEach];
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        f[c][e] = 0.f;
                        if (x0 + e * 2 * kRows < total && c0 + c < pieces)
                            f[c][e] = weight[(c0 + c) * 2 * kRows + row[e]];
                        v[c][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (f[c][e] != 0.f)  // (else nothing may be there)
                            v[c][e] = __ldcg(reinterpret_cast<const float4*>(
                                                 part_of(c0 + c, row[e] / kRows)) +
                                             row[e] % kRows * V + x0 % V);
                    }
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        acc[e][0] = fmaf(f[c][e], v[c][e].x, acc[e][0]);
                        acc[e][1] = fmaf(f[c][e], v[c][e].y, acc[e][1]);
                        acc[e][2] = fmaf(f[c][e], v[c][e].z, acc[e][2]);
                        acc[e][3] = fmaf(f[c][e], v[c][e].w, acc[e][3]);
                    }
            }
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (x0 + e * 2 * kRows >= total) continue;
                const int r = row[e] % kRows;
                uint16_t* const out =
                    static_cast<uint16_t*>(p.out) +
                    ((size_t)(sm.shared_rows[w][row[e] / kRows] + r / p.hpc) * p.N +
                     (size_t)sm.shared[w].kv * p.G + sm.shared[w].h0 + r % p.hpc) * H;
                reinterpret_cast<uint2*>(out)[x0 % V] =
                    make_uint2(Elt<BF16>::pack(acc[e][0], acc[e][1]),
                               Elt<BF16>::pack(acc[e][2], acc[e][3]));
            }
        }
        if (!meet()) return give_up(sm, p);  // the weights have been read
    }
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
    if (threadIdx.x == 32) {
        for (int s = 0; s < 8; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), 2);
            mbar_init(smem_addr(&sm.piece_full[s]), 1);
            mbar_init(smem_addr(&sm.piece_free[s]), 3 + 8);  // issuers, loader, softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sm.q_full[i]), 1);
            mbar_init(smem_addr(&sm.q_free[i]), 1);
            mbar_init(smem_addr(&sm.s_ready[i]), 1);
            mbar_init(smem_addr(&sm.p_ready[i]), kRows);
            mbar_init(smem_addr(&sm.o_ready[i]), 1);
            mbar_init(smem_addr(&sm.o_free[i]), kRows);
            mbar_init(smem_addr(&sm.done[i]), 1);
        }
        sm.abort_flag = 0;
        sm.lock = 0;
        mbar_init(smem_addr(&sm.all), 2 * kRows);
        sm.shared[0].pieces = sm.shared[1].pieces = 0;
        for (int i = 0; i < 4; ++i) sm.shared_count[i >> 1][i & 1] = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
        tma_prefetch_desc(&tmq);
    }
    if (warp == 2) tmem_alloc(smem_addr(&sm.tmem), 512);
    griddep_wait();  // everything read or written follows earlier kernels
    chunk_plan<H>(p, sm, reinterpret_cast<long long*>(ring));
    fence_proxy_async_shared();  // the plan's scratch before the copies that overwrite it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < kSoftWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == 1)
            chunk_load<H>(&tmk, &tmv, p, ring, sm);
        else if (warp == 2)
            chunk_schedule<H>(&tmq, p, qbuf, sm);
        else
            chunk_mma<BF16, H>(p, ring, qbuf, sm, warp == 0 ? 0 : 1);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        if (chunk_softmax<BF16, H>(p, ring, sm))
            chunk_shared<BF16, H>(p, sm, reinterpret_cast<float*>(qbuf));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(sm.tmem, 512);
}

template <int H>
constexpr size_t chunk_smem() {
    return 1024 + (size_t)(2 + Ch<H>::kSlots) * Ch<H>::kTile + sizeof(ChunkSmem);
}
static_assert(chunk_smem<128>() <= 227 * 1024 && chunk_smem<64>() <= 227 * 1024, "shared memory");
constexpr int kMaxCtas = 152;  // pieces whose weights the fold holds
static_assert(kMaxCtas * 2 * kRows * sizeof(float) <= (size_t)(2 + Ch<64>::kSlots) * Ch<64>::kTile &&
                  kMaxCtas * 2 * kRows * sizeof(float) <=
                      (size_t)(2 + Ch<128>::kSlots) * Ch<128>::kTile,
              "the fold's weights fit where tiles were");
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
    if (sms < 1 || (size_t)sms * sizeof(int32_t) > flags_bytes) return 0;
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
    const int sms = std::min(device_sm_count(), kMaxCtas);
    if (sms < 1) return GQA_ERR_CUDA;
    // no more CTAs than units can be (every item at the tables' width)
    const long long items = (rows + 2 * p.tpc - 1) / (2 * p.tpc) + s.B;
    const long long most =
        items * p.KC * (((s.max_blocks_per_seq + kBlocks - 1) / kBlocks) * (long long)kPair + kStart);
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
