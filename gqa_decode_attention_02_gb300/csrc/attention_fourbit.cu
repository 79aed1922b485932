// attention_fourbit.cu -- decode / verify attention over a paged cache held in
// 4 bits (codes and scales: fourbit.cuh).
//
// For sequence b, new token t and query head n of KV head k = n / G:
//     s_j = scale * <q[b,t,n,:], K_b[j,k,:]>,   out = sum_j softmax(s)_j V_b[j,k,:]
// over the positions j that token t sees (causal, window, tree mask as in the
// other attention calls), K and V being code * group scale.
//
// What bounds it.  A position costs 2 * (H/2 + H/32) bytes per KV head (136 at
// H = 128), so at the measured copy rate a 16-token tile (2,176 bytes) could arrive
// every 95 cycles per SM; the copies alone, without the arithmetic, run at 97 % of
// that rate.  The arithmetic takes longer: 64 sequences of 32,768 tokens (4 query
// rows per KV head) need 142 cycles per tile and SM, 504 us, 67 % of the
// copy rate.  Taking parts out one by one, of a form with 18 mma.sync a tile (17 now)
// and 148 cycles, showed its shares: about 47 cycles for the mma.sync, 43 for turning
// the codes into f16 operands, the rest for the softmax, the copies' addresses and the
// loop.
// (In loops of their own an mma.sync takes 8 cycles of a scheduler, lop3 and hfma2
// two each, two of each in turn 6.1: the pipes overlap only in part.)  So
// instructions per code word are what is saved first:
//
//  * No producer warp, no barriers in the loop: each warp copies its own tiles
//    with 16-byte cp.async into three slots of its own (two steps in flight, one
//    computed) and waits for its own copies only.
//  * Natural storage order, fragments by permutation.  Lane (g, q4) (g = lane /
//    4) reads K dims H/4*q4 .. of its two tokens with one wide load each: one
//    group per lane, one scale per token; V dims H/8*g .. of its four tokens:
//    one group per lane again, and the output leaves as contiguous dims.  q is
//    permuted to match once per segment.
//  * Codes become f16 operands exactly, one or and one fma per pair (q4_values).
//    One more row tile of PV sums the probabilities.
//  * S^T[16 tokens x 8 rows] and O^T[H x 8 rows] on mma.sync m16n8k16, tokens
//    (dims) on M.  Up to three row tiles share one conversion; more rows run in
//    chunks of 24 (chunks of 16: 68 us against 59 for 16 sequences of 40 rows, 364
//    against 244 for 64 of 8,192 tokens and 24 rows).
//    Four tiles no longer fit the registers with two tiles of tokens: 32 rows over
//    64 sequences of 8,192 tokens in 368 us against 387, over 4 of 500 in 24 against
//    20; five: no gain anywhere.
//    tcgen05 would take the mma off the schedulers but wants its operands in
//    shared memory as f16, four times the codes' bytes, written there by the
//    same warps; that trade was not built.
//
// Work split.  The batch's segments (sequence, KV head, row chunk) are laid end
// to end in units (a segment's start-up units, then its tiles) and CTA c takes
// the c-th equal range.  The warps of a CTA take tile pairs of a segment in
// turn and meet in shared memory when it ends; a segment cut by a range
// boundary goes through the workspace, the CTA that finishes last folding the
// pieces in order (deterministic; nobody waits).  Where there is a CTA for every
// segment and none is long, each CTA takes one whole segment.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "fourbit.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kStepTiles = 2;    // tiles a warp computes per step
constexpr int kSlots = 3;        // steps in a warp's buffer: one computed, two in flight
// Start-up cost of a segment, in tiles per warp (256 ragged sequences, one row tile,
// 4 warps: some 6 us a segment against 0.27 us a tile; with 3 units 240 us, 6 228, 9
// 234.  Three row tiles: 7 us against 0.15-0.18 us; 16 sequences of 40 rows with 5 units
// 62 us, 10 59, 15 62).
constexpr int q4_seg_units(int NW) { return NW == 1 ? 6 : NW == 2 ? 7 : 10; }
// Longest segment of a planless launch, in tiles per warp.  Such a launch against a
// planned one (us, in a chain of calls in a graph): 295 tokens 5.8 against 6.8, 64 of
// 16..1,024 9.1 against 10.4, 8 of 2,560 (the longest it takes at 16 warps) 21.5 against
// 22.9; of 5,000 tokens 33.7 against 28.0, which is why it ends there.
constexpr int kQ4Direct = 10;
// What cutting segments costs a CTA, in tiles per warp.  Whole segments where the longest
// passes an equal share by up to 0, 6 or 24 tiles a warp (us): 12 sequences of 16,000
// tokens 68.5, 68.0, 86.3; 16 of 12,000..16,000 79.5, 79.1, 84.4; 30 of 8,000 78.4, 78.2,
// 84.6; 8 of 5,000 27.9, 27.9, 35.2; but 16 of 16..5,000 31.1, 34.3, 34.1.
constexpr int kQ4CutCost = 6;
// Reference where no score was seen: below all, and finite, so references need no test.
constexpr float kQ4None = -3.402823466e38f;
// A probability is 2^(score - reference).  The reference of a row is set 7 below its
// largest score, and again once a score is 15 above it, so that the largest probability
// is 2^7 .. 2^15, near the top of f16's range, and what f16 takes from small ones (2^-25
// each) is 2^-32 of it.  (A reference at the maximum would lose positions 18 nats behind
// it altogether, however many they are.)
constexpr float kQ4Top = 7.0f;
constexpr float kQ4Gap = 8.0f + kQ4Top;
constexpr size_t kQ4FlagBytes = 262144; // tickets, one per CTA (as large as the other kernels' region)
constexpr long long kQ4MaxRows = 8192;  // T*G
constexpr int kQ4MaxTiles = 3;          // row tiles of 8 per warp

struct Q4Params {
    const void* q;
    void* out;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const uint8_t* k_scale;
    const uint8_t* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const uint64_t* tree_mask;  // nullptr: the chain
    float* partials;
    int32_t* tickets;
    int32_t* status;
    int B, T, N, K, G, R;
    int C, Rc, KC;  // row chunks per KV head, rows per chunk, virtual heads K*C
    int max_blocks, num_blocks;
    int window;
    int direct;  // a CTA per segment (the host's rule)
    float scale_log2;
    uint32_t code_stride, scale_stride;  // bytes of a block's codes, scales
    uint32_t ex[2];  // 0x64006400, 0x54005400 (see q4_values)
};

template <int H>
struct Q4 {
    static constexpr int kRow = H / 2;             // code bytes of a row
    static constexpr int kCodes = 16 * kRow;       // ... of a tile
    static constexpr int kGroups = H / kQ4Group;   // scales of a row
    static constexpr int kScales = 16 * kGroups;   // scale bytes of a tile
    static constexpr int kTile = 2 * (kCodes + kScales);
    static constexpr int kSlot = kStepTiles * kTile;
    static constexpr int kSteps = H / 16;          // k16 steps of QK^T, m16 tiles of PV
    static constexpr int kKWords = H / 32;         // K words per lane and token
    static constexpr int kVWords = H / 64;         // V words per lane and token
    static constexpr int kRowFloats = H + 4;       // row stride of the combine scratch
};

__device__ __forceinline__ int q4_first_block(int ctx, int T, int window) {
    return window > 0 ? max(0, ctx - T - window + 1) >> 4 : 0;
}
__device__ __forceinline__ int q4_blocks(int ctx, int T, int max_blocks, int window) {
    return (ctx >= T && ctx >= 1 && ctx <= max_blocks * 16)
               ? ((ctx + 15) >> 4) - q4_first_block(ctx, T, window)
               : 0;
}
__device__ __forceinline__ int q4_units(int nblk, int seg) { return nblk > 0 ? nblk + seg : 0; }

// The pieces of segments in one CTA's range of units, in order.
struct Pieces {
    int b, k;        // sequence, virtual head
    int ctx, nblk, f0;
    int start;       // unit of the segment's first tile
    int i0, i1;      // this CTA's tiles of it
    int c0, c1;      // the range
    int seg;         // a segment's start-up units

    __device__ void load(const Q4Params& p) {
        ctx = __ldg(p.context_lens + b);
        nblk = q4_blocks(ctx, p.T, p.max_blocks, p.window);
        f0 = q4_first_block(ctx, p.T, p.window);
    }
    // Virtual head k_ of sequence b_, whole; false for an invalid length.
    __device__ bool one(const Q4Params& p, int b_, int k_) {
        b = b_;
        k = k_;
        load(p);
        seg = start = c0 = i0 = 0;
        i1 = c1 = nblk;
        return nblk > 0;
    }
    __device__ bool clip() {
        i0 = max(0, c0 - start);
        i1 = min(nblk, c1 - start);
        return i1 > i0;
    }
    // From the segment holding unit c0 (sequence b_, whose first unit is base):
    // the first piece with tiles; false if the range holds none.
    __device__ bool begin(const Q4Params& p, int b_, int base, int lo, int hi, int seg_) {
        c0 = lo;
        c1 = hi;
        b = b_;
        if (c0 >= c1) return false;
        load(p);
        seg = seg_;
        const int u = q4_units(nblk, seg);
        k = (c0 - base) / u;
        start = base + k * u + seg;
        return clip() || next(p);
    }
    __device__ bool next(const Q4Params& p) {
        while (true) {
            start += nblk + seg;
            if (start >= c1) return false;  // later segments start later still
            if (++k == p.KC) {
                k = 0;
                do {
                    if (++b >= p.B) return false;  // (units remain: one with tiles follows)
                    load(p);
                } while (nblk == 0);
            }
            if (clip()) return true;
        }
    }
};

// 16-byte cp.async with constant offsets on both sides.
template <int DST, int SRC>
__device__ __forceinline__ void q4_cp16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src),
                 "n"(DST), "n"(SRC)
                 : "memory");
}

// A lane's part of copying tiles of one KV head into a slot.  K rows go to row
// r ^ ((r >> 2) & 1) at H = 128 (r ^ 2 * that at H = 64) and V chunks to
// c ^ 2 * ((r >> 1) & 1): the fragment loads are then free of bank conflicts.
template <int H>
struct Q4Copy {
    using L = Q4<H>;
    static constexpr int kSc = L::kScales / 16;  // 16-byte pieces of a scale tile
    const uint8_t *k, *v, *s;  // of block 0
    uint32_t ko, vo, so;       // offsets in a tile

    __device__ void lane_offsets(int lane) {
        if constexpr (H == 128) {
            const int r = lane >> 2, c = lane & 3;  // rows 8..15: the same swizzle
            ko = (uint32_t)((r ^ ((r >> 2) & 1)) * 64 + c * 16);
            vo = (uint32_t)(L::kCodes + r * 64 + ((c ^ (r & 2)) << 4));
        } else {
            const int r = lane >> 1, c = lane & 1;
            ko = (uint32_t)((r ^ ((r >> 1) & 2)) * 32 + c * 16);
            vo = (uint32_t)(L::kCodes + lane * 16);
        }
        so = (uint32_t)(2 * L::kCodes + lane * 16);
    }
    __device__ void head(const Q4Params& p, int kv, int lane) {
        k = p.k_cache + (size_t)kv * L::kCodes + lane * 16;
        v = p.v_cache + (size_t)kv * L::kCodes + lane * 16;
        s = lane < kSc ? p.k_scale + (size_t)kv * L::kScales + lane * 16
                       : p.v_scale + (size_t)kv * L::kScales + (lane - kSc) * 16;
    }
    // base + blk * stride, one instruction
    static __device__ __forceinline__ const uint8_t* at(const uint8_t* base, uint32_t blk,
                                                        uint32_t stride) {
        uint64_t r;
        asm("mad.wide.u32 %0, %1, %2, %3;"
            : "=l"(r)
            : "r"(blk), "r"(stride), "l"(reinterpret_cast<uint64_t>(base)));
        return reinterpret_cast<const uint8_t*>(r);
    }
    template <int J>  // tile J of the slot at dst
    __device__ __forceinline__ void tile(uint32_t dst, uint32_t blk, const Q4Params& p,
                                         int lane) const {
        const uint8_t* ks = at(k, blk, p.code_stride);
        const uint8_t* vs = at(v, blk, p.code_stride);
        q4_cp16<J * L::kTile, 0>(dst + ko, ks);
        q4_cp16<J * L::kTile, 0>(dst + vo, vs);
        if constexpr (H == 128) {
            q4_cp16<J * L::kTile + 512, 512>(dst + ko, ks);
            q4_cp16<J * L::kTile + 512, 512>(dst + vo, vs);
        }
        if (lane < 2 * kSc) q4_cp16<J * L::kTile, 0>(dst + so, at(s, blk, p.scale_stride));
    }
};

__device__ __forceinline__ __half2 as_h2(uint32_t x) {
    return *reinterpret_cast<__half2*>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// W words of shared memory
template <int W>
__device__ __forceinline__ void q4_words(const uint8_t* at, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(at);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    }
}

__device__ __forceinline__ void q4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scales of the two codes of a pair, times 2^-7, as f16x2 (exact: the smallest
// scale is 2^-17, f16's last bit 2^-24), and what turns biased codes into values.
// The 2^7 comes back with the score factors and the final rows.  s has four
// significant bits, so 129 s has eleven and 9 s eight: f16 holds both.
constexpr float kQ4Unit = 128.f;
struct Q4Scale {
    __half2 s, n10, n6;  // s, -1032 s, -72 s
    __device__ __forceinline__ explicit Q4Scale(uint32_t bits) {
        s = __hmul2(as_h2(bits), as_h2(0x20002000u));    // 2^-7
        n10 = __hmul2(as_h2(bits), as_h2(0xc808c808u));  // -129 / 16
        n6 = __hmul2(as_h2(bits), as_h2(0xb880b880u));   // -9 / 16
    }
};

// Four code pairs of a word -- nibbles i of its two halves, i = 0..3 -- times
// their scales.  Or-ed under an exponent a nibble n = c + 8 is 1024 + n (bits
// 0-3 under 0x6400, ex[0]) or 64 + n (bits 4-7 under 0x5400, ex[1]; both come as
// kernel parameters, or each of these lines is two instructions).
// FAST: one fma each, (1024 + n) s - 1032 s = c s, every term and the result exact
// (scales below 8192: 1032 s stays in range).  Otherwise in two steps.
// (Another form, (1024 + n) s - 1024 s = n s with 8 s per code taken off the sums at the
// end, loses what fp32 drops beside 8 sum(p s): f16 outputs of 113,000 positions were
// 6.4e-5 off (rms, scales of 1/4), a hundred times their rounding; this form 6.6e-7.)
template <bool FAST>
__device__ __forceinline__ void q4_values(uint32_t x, const Q4Scale& f, const uint32_t (&ex)[2],
                                          uint32_t (&v)[4]) {
    const uint32_t y = x >> 8;
    const __half2 t0 = as_h2((x & 0x000f000fu) | ex[0]);
    const __half2 t1 = as_h2((x & 0x00f000f0u) | ex[1]);
    const __half2 t2 = as_h2((y & 0x000f000fu) | ex[0]);
    const __half2 t3 = as_h2((y & 0x00f000f0u) | ex[1]);
    if constexpr (FAST) {
        v[0] = as_u32(__hfma2(t0, f.s, f.n10));
        v[1] = as_u32(__hfma2(t1, f.s, f.n6));
        v[2] = as_u32(__hfma2(t2, f.s, f.n10));
        v[3] = as_u32(__hfma2(t3, f.s, f.n6));
    } else {
        const __half2 o10 = as_h2(0x64086408u), o6 = as_h2(0x54805480u);  // 1032, 72
        v[0] = as_u32(__hmul2(__hsub2(t0, o10), f.s));
        v[1] = as_u32(__hmul2(__hsub2(t1, o6), f.s));
        v[2] = as_u32(__hmul2(__hsub2(t2, o10), f.s));
        v[3] = as_u32(__hmul2(__hsub2(t3, o6), f.s));
    }
}

// The q rows of a piece, in shared memory: every warp of the CTA needs the same.
// Row u*8+g, dims H/4*q4 .. as B fragments: word j of a token's codes meets k-steps 2j
// (nibbles 0|4, 1|5) and 2j+1 (2|6, 3|7).  Rows are scaled by a power of two that
// puts their largest element in [64, 128): f16 then holds an element of either
// type exactly down to 2^-20 of the largest, and to within 2^-31 of it below.
template <int H, int NW, bool BF16>
struct Q4Rows {
    uint2 frag[NW][Q4<H>::kSteps][32];
    float factor[8 * NW];  // of the rows' scores, to the log2 domain

    // This lane's raw words of row 8u + g of virtual head k of sequence b.
    static __device__ __forceinline__ void load(const Q4Params& p, int b, int k, int u,
                                                uint32_t (&w)[H / 8]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
        const int kv = k / p.C, rb = (k - kv * p.C) * p.Rc, re = min(p.R, rb + p.Rc);
        const int r = rb + 8 * u + g, t = r / p.G, gg = r - t * p.G;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) +
            (((size_t)b * p.T + t) * p.N + (size_t)kv * p.G + gg) * H + q4 * (H / 4));
#pragma unroll
        for (int i = 0; i < H / 32; ++i) {
            const uint4 x = r < re ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
        }
    }
    __device__ __forceinline__ void make(const Q4Params& p, int u, uint32_t (&w)[H / 8]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
        auto lo = [&](uint32_t x) { return Elt<BF16>::lo(x); };
        auto hi = [&](uint32_t x) { return Elt<BF16>::hi(x); };
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < H / 8; ++i) top = fmaxf(top, fmaxf(fabsf(lo(w[i])), fabsf(hi(w[i]))));
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
        const int e = min(max(127 + 6 - (int)(__float_as_uint(top) >> 23), -112), 112);
        const float f = __uint_as_float((uint32_t)(127 + e) << 23);  // row times 2^e
        const float back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < H / 8; ++i) w[i] = Elt<false>::pack(lo(w[i]) * f, hi(w[i]) * f);
        // never 0, which a hidden position's -inf must not meet
        if (q4 == 0) factor[8 * u + g] = fmaxf(kQ4Unit * p.scale_log2 * back, 1.17549435e-38f);
#pragma unroll
        for (int j = 0; j < H / 32; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                frag[u][2 * j + h][lane] =
                    make_uint2(prmt(w[4 * j + h], w[4 * j + 2 + h], 0x5410u),
                               prmt(w[4 * j + h], w[4 * j + 2 + h], 0x7632u));
    }
};

// A warp's state for one piece of a segment: NW tiles of 8 query rows.  Several
// tiles share every converted code, and read the q fragments from shared memory.
template <int H, int NW, bool BF16>
struct Q4Warp {
    using L = Q4<H>;
    static constexpr bool kKeepQ = NW == 1;  // q fragments in registers
    const Q4Params& p;
    const Q4Rows<H, NW, BF16>* qr;
    const int lane, g, q4;
    const uint32_t ex[2];
    uint32_t kro, vro, sko, svo;  // this lane's offsets in a tile
    uint32_t cko;                 // ... and of the 8 scale bytes it looks over
    int rbase, rend, b, kv, ctx;
    int edge_lo, edge_hi;  // tiles <= edge_lo or >= edge_hi hold hidden positions
    uint32_t qf[kKeepQ ? NW : 1][L::kSteps][2];
    float acc[NW][L::kSteps][4];
    // sum p, which rides along with the PV product as one more row tile (of ones): [0],
    // [1] of rows 2*q4, 2*q4 + 1; [2], [3] the same
    float sum[NW][4];
    float sl0[NW], sl1[NW];  // score factor to the log2 domain, per row
    float m0[NW], m1[NW];    // references of the rows' probabilities
    bool bad;

    __device__ Q4Warp(const Q4Params& p_, const Q4Rows<H, NW, BF16>* qr_)
        : p(p_), qr(qr_), lane(threadIdx.x & 31), g((threadIdx.x & 31) >> 2), q4(threadIdx.x & 3),
          ex{p_.ex[0], p_.ex[1]} {
        const int ta = token();
        const int ra = H == 128 ? (ta ^ ((ta >> 2) & 1)) : (ta ^ ((ta >> 1) & 2));
        kro = (uint32_t)(ra * L::kRow + q4 * (L::kRow / 4));
        vro = L::kCodes + (H == 128 ? (uint32_t)(q4 * 64 + ((((g >> 1) ^ (q4 & 2)) << 4) |
                                                            ((g & 1) << 3)))
                                    : (uint32_t)(q4 * 32 + g * 4));
        sko = (uint32_t)(2 * L::kCodes + ta * L::kGroups + q4 * L::kGroups / 4);
        svo = (uint32_t)(2 * L::kCodes + L::kScales + q4 * L::kGroups + g * L::kGroups / 8);
        cko = (uint32_t)((lane >> 4) * L::kTile + 2 * L::kCodes + (lane & 15) * (L::kScales / 8));
    }
    // Score rows g, g + 8 are tokens token(), token() + 8 of a tile; V's k pairs
    // are then tokens q4, q4 + 4 and q4 + 8, q4 + 12.
    __device__ __forceinline__ int token() const { return (g >> 1) + 4 * (g & 1); }

    // Start a piece, whose q rows are in *qr.
    __device__ __forceinline__ void begin(const Pieces& s) {
        b = s.b;
        ctx = s.ctx;
        kv = s.k / p.C;
        rbase = (s.k - kv * p.C) * p.Rc;
        rend = min(p.R, rbase + p.Rc);
        bad = false;
        // hidden somewhere: new positions (the first only by a tree mask, but then a
        // chain mask and none take the same steps), past the end, or at or below the
        // last row's window
        edge_hi = ((ctx - p.T) >> 4) - s.f0;
        edge_lo = p.window > 0 && ctx > p.window ? ((ctx - 1 - p.window) >> 4) - s.f0 : -1;
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            m0[u] = m1[u] = kQ4None;
            sl0[u] = qr->factor[8 * u + 2 * q4];
            sl1[u] = qr->factor[8 * u + 2 * q4 + 1];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[u][e] = 0.f;
#pragma unroll
            for (int mt = 0; mt < L::kSteps; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[u][mt][e] = 0.f;
                if constexpr (kKeepQ) {
                    const uint2 f = qr->frag[u][mt][lane];
                    qf[u][mt][0] = f.x;
                    qf[u][mt][1] = f.y;
                }
            }
        }
    }

    // Hide score entries of tile position tb (of this lane's tokens) from the rows
    // that do not see them.
    __device__ __forceinline__ void mask(float (&sc)[4], int u, int tb) const {
        const int wl = p.window > 0 ? p.window : (1 << 30);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // row rbase + 8u + 2*q4 + h, of new token t
            const int t = min((rbase + 8 * u + 2 * q4 + h) / p.G, p.T - 1), lim = ctx - p.T + t;
            const uint64_t row = p.tree_mask ? __ldg(p.tree_mask + (size_t)b * p.T + t) : ~0ull;
#pragma unroll
            for (int e = h; e < 4; e += 2) {
                const int pos = tb + token() + (e >> 1) * 8, j = pos - (ctx - p.T);
                const bool off = pos > lim || pos <= lim - wl ||
                                 (j >= 0 && j < t && j < 64 && !((row >> j) & 1ull));
                if (off) sc[e] = -INFINITY;
            }
        }
    }

    // Scores of NT tiles.
    template <bool FAST, int NT>
    __device__ __forceinline__ void scores(float (&sc)[NT][NW][4], const uint8_t* tiles) {
        uint32_t wa[NT][L::kKWords], wb[NT][L::kKWords];
        uint32_t sa[NT], sb[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint8_t* tile = tiles + j * L::kTile;
            sa[j] = (uint32_t)tile[sko] * 0x00800080u;
            sb[j] = (uint32_t)tile[sko + 8 * L::kGroups] * 0x00800080u;
            q4_words(tile + kro, wa[j]);
            q4_words(tile + kro + 8 * L::kRow, wb[j]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int u = 0; u < NW; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][u][e] = 0.f;
#pragma unroll
        for (int i = 0; i < L::kKWords; ++i) {
            uint32_t va[NT][4], vb[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                q4_values<FAST>(wa[j][i], Q4Scale(sa[j]), ex, va[j]);
                q4_values<FAST>(wb[j][i], Q4Scale(sb[j]), ex, vb[j]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < NW; ++u) {
                    uint2 f;
                    if constexpr (kKeepQ)
                        f = make_uint2(qf[u][2 * i + h][0], qf[u][2 * i + h][1]);
                    else
                        f = qr->frag[u][2 * i + h][lane];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        q4_mma(sc[j][u], va[j][2 * h], vb[j][2 * h], va[j][2 * h + 1],
                               vb[j][2 * h + 1], f.x, f.y);
                }
        }
    }

    // O^T += V^T P^T of a tile.  The probabilities enter the product as f16, off by
    // 2^-11 of themselves (or 2^-25, see kQ4Top), an eighth of a bf16 output's half step.
    // An f16 output's half step is no more than that, so there what rounding left over
    // enters as a second f16 term (64 sequences of 8,192 tokens, f16, H = 128: 4 rows per
    // KV head 160 us with it, 144 without; 24 rows 281 against 244).  The sum takes the
    // same terms, so the weights still add up to one.
    template <bool FAST>
    __device__ __forceinline__ void values(const float (&sc)[NW][4], const uint8_t* tile, int tb) {
        constexpr int kTerms = BF16 ? 1 : 2;
        uint32_t pb[kTerms][NW][2];
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            // product and difference rounded one by one, as in raise(): where fp32 numbers
            // are far apart an fma's would lie beyond the reference's 15.  (A mul.rn.f32x2
            // before the add.rn.f32x2 gave an fma's results.)
            auto x = [&](int e) { return __fmul_rn(sc[u][e], e & 1 ? sl1[u] : sl0[u]); };
            const uint64_t m = q4_pair(-m0[u], -m1[u]);
            const uint64_t x01 = q4_add2(q4_pair(x(0), x(1)), m);
            const uint64_t x23 = q4_add2(q4_pair(x(2), x(3)), m);
            const float e0 = fast_exp2(q4_lo(x01)), e1 = fast_exp2(q4_hi(x01));
            const float e2 = fast_exp2(q4_lo(x23)), e3 = fast_exp2(q4_hi(x23));
            const uint32_t w0 = Elt<false>::pack(e0, e1), w1 = Elt<false>::pack(e2, e3);
            pb[0][u][0] = movm_t(w0);
            pb[0][u][1] = movm_t(w1);
            if constexpr (kTerms == 2) {
                pb[1][u][0] =
                    movm_t(Elt<false>::pack(e0 - Elt<false>::lo(w0), e1 - Elt<false>::hi(w0)));
                pb[1][u][1] =
                    movm_t(Elt<false>::pack(e2 - Elt<false>::lo(w1), e3 - Elt<false>::hi(w1)));
            }
        }
        uint32_t s[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] = tile[svo + 4 * x * L::kGroups];  // tokens q4 + 4x
        if constexpr (!FAST) {
            // Rows past the context or below every window may hold anything: scale 0
            // makes their values zeros.
            const int lo = p.window > 0 ? ctx - p.T - p.window + 1 : 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int pos = tb + q4 + 4 * x;
                if (pos >= ctx || pos < lo) s[x] = 0u;
            }
        }
        const Q4Scale f01((s[0] << 7) | (s[1] << 23)), f23((s[2] << 7) | (s[3] << 23));
        constexpr uint32_t kOnes = 0x3c003c00u;
#pragma unroll
        for (int z = 0; z < kTerms; ++z)
#pragma unroll
            for (int u = 0; u < NW; ++u)
                q4_mma(sum[u], kOnes, kOnes, kOnes, kOnes, pb[z][u][0], pb[z][u][1]);
        uint32_t w[4][L::kVWords];
#pragma unroll
        for (int i = 0; i < 4; ++i) q4_words(tile + vro + i * 4 * L::kRow, w[i]);
#pragma unroll
        for (int i = 0; i < L::kVWords; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h ? 0x7632u : 0x5410u;
                uint32_t va[4], vc[4];
                q4_values<FAST>(prmt(w[0][i], w[1][i], sel), f01, ex, va);
                q4_values<FAST>(prmt(w[2][i], w[3][i], sel), f23, ex, vc);
#pragma unroll
                for (int z = 0; z < kTerms; ++z)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int u = 0; u < NW; ++u)
                            q4_mma(acc[u][4 * i + 2 * h + x], va[2 * x], va[2 * x + 1], vc[2 * x],
                                   vc[2 * x + 1], pb[z][u][0], pb[z][u][1]);
            }
    }

    // References of the rows (kQ4Top below a running maximum) after the scores of a
    // step: rescale only when one of them is more than kQ4Gap above.
    __device__ __forceinline__ void raise(const float (&sc)[kStepTiles][NW][4]) {
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            float x0 = sc[0][u][0], x1 = sc[0][u][1];
#pragma unroll
            for (int j = 0; j < kStepTiles; ++j) {
                x0 = fmaxf(x0, fmaxf(sc[j][u][0], sc[j][u][2]));
                x1 = fmaxf(x1, fmaxf(sc[j][u][1], sc[j][u][3]));
            }
            x0 = __fmul_rn(x0, sl0[u]);
            x1 = __fmul_rn(x1, sl1[u]);
            auto above = [](float x, float m) { return __fsub_rn(x, m) > kQ4Gap; };
            if (__any_sync(FULL, above(x0, m0[u]) || above(x1, m1[u]))) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(FULL, x0, o));
                    x1 = fmaxf(x1, __shfl_xor_sync(FULL, x1, o));
                }
                const bool up0 = above(x0, m0[u]), up1 = above(x1, m1[u]);
                x0 -= kQ4Top;
                x1 -= kQ4Top;
                const float f0 = up0 ? fast_exp2(m0[u] - x0) : 1.f;
                const float f1 = up1 ? fast_exp2(m1[u] - x1) : 1.f;
                if (up0) m0[u] = x0;
                if (up1) m1[u] = x1;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[u][e] *= (e & 1) ? f1 : f0;
#pragma unroll
                for (int mt = 0; mt < L::kSteps; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[u][mt][e] *= (e & 1) ? f1 : f0;
            }
        }
    }

    // One step: nt tiles (1 or 2) from tile i of the segment (first position tb),
    // in the given slot.  Nearly every step is whole, sees all its positions and
    // has scales below 8192, and takes the straight path.
    __device__ __forceinline__ void step(const uint8_t* slot, int i, int tb, int nt) {
        uint32_t c[L::kScales / 32];  // this lane's share of the step's scale bytes
        q4_words(slot + cko, c);
        uint32_t top = 0u;
#pragma unroll
        for (int x = 0; x < L::kScales / 32; ++x) top |= c[x] & (c[x] << 1) & (c[x] << 2);
        const bool large = (top & 0x80808080u) != 0u;  // a byte of 224 or more
        float sc[kStepTiles][NW][4];
        if (!__any_sync(FULL, large) && nt == kStepTiles && i + nt <= edge_hi && i > edge_lo) {
            scores<true, kStepTiles>(sc, slot);
            raise(sc);
#pragma unroll
            for (int j = 0; j < kStepTiles; ++j)
                values<true>(sc[j], slot + j * L::kTile, 0);
            return;
        }
#pragma unroll
        for (int j = 0; j < kStepTiles; ++j) {
            if (j < nt) {
                scores<false, 1>(*reinterpret_cast<float (*)[1][NW][4]>(&sc[j]),
                                 slot + j * L::kTile);
#pragma unroll
                for (int u = 0; u < NW; ++u) mask(sc[j][u], u, tb + 16 * j);
            } else {
#pragma unroll
                for (int u = 0; u < NW; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[j][u][e] = -INFINITY;
            }
        }
        raise(sc);
#pragma unroll
        for (int j = 0; j < kStepTiles; ++j)
            if (j < nt) values<false>(sc[j], slot + j * L::kTile, tb + 16 * j);
    }

    // This warp's maxima and sums of every row, and the accumulators of row tile U.
    __device__ __forceinline__ void save_head(float* head) const {
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int r = 8 * u + 2 * q4;
            if (g == 0) {
                head[r] = m0[u];
                head[r + 1] = m1[u];
                head[8 * NW + r] = sum[u][0];
                head[8 * NW + r + 1] = sum[u][1];
            }
        }
        if (lane == 0) head[16 * NW] = bad ? 1.f : 0.f;
    }
    template <int U>
    __device__ __forceinline__ void save_rows(float* rows) const {
        float* d0 = rows + 2 * q4 * L::kRowFloats + g * (H / 8);
        float* d1 = d0 + L::kRowFloats;
#pragma unroll
        for (int i = 0; i < L::kSteps / 2; ++i) {
            reinterpret_cast<float4*>(d0)[i] =
                make_float4(acc[U][2 * i][0], acc[U][2 * i][2], acc[U][2 * i + 1][0],
                            acc[U][2 * i + 1][2]);
            reinterpret_cast<float4*>(d1)[i] =
                make_float4(acc[U][2 * i][1], acc[U][2 * i][3], acc[U][2 * i + 1][1],
                            acc[U][2 * i + 1][3]);
        }
    }
};

__device__ __forceinline__ float q4_weight(float m, float M) {
    return fast_exp2(m - M);  // 0 for kQ4None unless all are
}

template <int H, bool BF16>
__device__ __forceinline__ void q4_store4(const Q4Params& p, int b, int kv, int r, int d,
                                          float4 v) {
    const int t = r / p.G, gg = r - t * p.G;
    uint16_t* dst = static_cast<uint16_t*>(p.out) +
                    (((size_t)b * p.T + t) * p.N + (size_t)kv * p.G + gg) * H + d;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(Elt<BF16>::pack(v.x, v.y), Elt<BF16>::pack(v.z, v.w));
}

// Partial of one piece in the workspace: max[8*NW], sum[8*NW], bad, pad, then
// the rows' accumulators.
template <int H, int NW>
struct Q4Part {
    static constexpr int kHead = 16 * NW + 4;
    static constexpr int kFloats = kHead + 8 * NW * H;
};

// Where the warps' scratch is: the slot a warp has computed last is free until the
// CTA leaves the piece.  (Shared memory is what bounds the copies in flight.)
template <int H>
struct Q4Free {
    uint8_t* smem;       // the warps' rings
    const uint32_t* at;  // offset of each warp's free slot
    __device__ __forceinline__ uint8_t* of(int w) const { return smem + at[w]; }
    __device__ __forceinline__ float* rows(int w) const { return reinterpret_cast<float*>(of(w)); }
};

// Fold pieces first .. last of a split segment (the whole block).  A warp per row
// turns the pieces' maxima and sums into weights, lanes over the pieces; meanwhile
// every thread's first accumulators are on their way.  Then the threads, in groups
// that take a share of the pieces each, add up.  All orders are fixed by the sizes.
// (Every thread going through its row's 20 maxima and sums itself: the fold of one
// sequence of 100,003 tokens took 10 us, so 5, and the call 51 us, so 46.)
template <int H, int NW, bool BF16>
__device__ __forceinline__ void fold_pieces(const Q4Params& p, int b, int kv, int rbase, int nrows,
                                         int first, int last, Q4Free<H> fr) {
    using Part = Q4Part<H, NW>;
    constexpr int kRows = 8 * NW, kAhead = 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = blockDim.x >> 5;
    const int n = last - first + 1;
    auto sec = [&](int c) {  // piece c
        return p.partials + ((size_t)(first + c) * 2 + (c == 0 ? 1 : 0)) * Part::kFloats;
    };
    // a free slot holds 16 bytes a lane for the groups' sums, then the weights of
    // every W-th row; too many of them take the place of the maxima
    const bool fits = (nrows + W - 1) / W * n * 4 <= Q4<H>::kSlot - 512;
    auto weight = [&](int c, int r) {
        return fits ? reinterpret_cast<float*>(fr.of(r % W) + 512) + r / W * n + c : sec(c) + r;
    };
    const int items = nrows * (H / 4);
    const int groups = max(1, min((int)blockDim.x / items, n));
    const int each = (n + groups - 1) / groups;
    const int gi = groups > 1 ? tid / items : 0;
    const int lo = gi * each, hi = gi < groups ? min(n, lo + each) : lo;
    int x = groups > 1 ? tid - gi * items : tid;
    float4 v[kAhead];
    auto load = [&](int c0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (x < items && c0 + j < hi)
                v[j] = __ldcg(reinterpret_cast<const float4*>(sec(c0 + j) + Part::kHead) + x);
    };
    load(lo);
    bool bad = false;
    for (int r0 = warp; r0 < nrows; r0 += NW * W) {
        float m0[NW], l0[NW];
        const float flag = lane < n ? __ldcg(sec(lane) + 16 * NW) : 0.f;
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const bool in = lane < n && r0 + u * W < nrows;
            m0[u] = in ? __ldcg(sec(lane) + r0 + u * W) : kQ4None;
            l0[u] = in ? __ldcg(sec(lane) + kRows + r0 + u * W) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            const int r = r0 + u * W;
            if (r >= nrows) break;
            float M = m0[u];
            for (int c = lane + 32; c < n; c += 32) M = fmaxf(M, __ldcg(sec(c) + r));
#pragma unroll
            for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
            const float f = q4_weight(m0[u], M);
            float l = f * l0[u];
            for (int c = lane + 32; c < n; c += 32)
                l = fmaf(q4_weight(__ldcg(sec(c) + r), M), __ldcg(sec(c) + kRows + r), l);
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
            const float iv = kQ4Unit / l;
            if (lane < n) *weight(lane, r) = f * iv;
            for (int c = lane + 32; c < n; c += 32)
                *weight(c, r) = q4_weight(__ldcg(sec(c) + r), M) * iv;
        }
        bad |= flag != 0.f;
        for (int c = lane + 32; c < n; c += 32) bad |= __ldcg(sec(c) + 16 * NW) != 0.f;
    }
    bad = __syncthreads_or(bad);
    for (int x0 = 0; x0 < items; x0 += blockDim.x) {
        const int r = min(x, items - 1) / (H / 4), d = x % (H / 4) * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = lo; c0 < hi; c0 += kAhead) {
            if (c0 > lo || x0 > 0) load(c0);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (c0 + j < hi) {
                    const float f = *weight(c0 + j, r);
                    o.x = fmaf(f, v[j].x, o.x);
                    o.y = fmaf(f, v[j].y, o.y);
                    o.z = fmaf(f, v[j].z, o.z);
                    o.w = fmaf(f, v[j].w, o.w);
                }
            }
        }
        if (groups > 1) {  // (one round of items then)
            auto sums = [&](int t) { return reinterpret_cast<float4*>(fr.of(t >> 5)) + (t & 31); };
            if (gi < groups) *sums(tid) = o;
            __syncthreads();
            if (gi == 0) {
                for (int y = 1; y < groups; ++y) {
                    const float4 w = *sums(y * items + x);
                    o.x += w.x;
                    o.y += w.y;
                    o.z += w.z;
                    o.w += w.w;
                }
            }
        }
        if (gi == 0 && x < items) {
            if (bad) o = make_float4(0.f, 0.f, 0.f, 0.f);
            q4_store4<H, BF16>(p, b, kv, rbase + r, d, o);
        }
        x += blockDim.x;
    }
}

// Warps an SM's registers hold at each row count: 128, 168 and 255 registers a thread.
// At H = 128 some spill (one row tile 340 bytes, two 706, three 16), nearly all outside
// the loop over the steps: 0.6 spilled accesses a tile.  One row tile with 12 warps (168
// registers, next to no spills) and with 8 (none) against 16: 64 x 32,768 513 and 544 us
// against 504, 256 ragged 232 and 253 against 228; shorter and f16 batches like 12 better
// (32 x 8,192 79.5 us against 85.5; 64 x 8,192, f16, 152 against 160).  Two row tiles
// with 8 warps (no spills): 64 x 8,192, 16 rows, 193 us against 203.
constexpr int q4_sm_warps(int NW) { return NW == 1 ? 16 : NW == 2 ? 12 : 8; }

template <int H, int NW, bool BF16>
__global__ void __launch_bounds__(32 * q4_sm_warps(NW), 1) q4_attention_kernel(const Q4Params p) {
    using L = Q4<H>;
    using Part = Q4Part<H, NW>;
    constexpr int kRows = 8 * NW;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_scan[16], s_long[16], s_b, s_base, s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = blockDim.x >> 5;
    auto* qr = reinterpret_cast<Q4Rows<H, NW, BF16>*>(smem + (size_t)W * kSlots * L::kSlot);
    float* heads = reinterpret_cast<float*>(qr + 1);
    __shared__ uint32_t s_free[16];
    const Q4Free<H> fr = {smem, s_free};
    griddep_launch_dependents();
    griddep_wait();

    uint32_t qw[H / 8];  // warp u: raw words of row tile u of the next piece
    Pieces piece;
    bool more, whole = p.direct;
    int quota = 1;
    int ids = 0, fl = 32;  // block ids of 16 steps (two a step), the next one's place
    // An invalid length: zeros for sequence b.
    auto refuse = [&](int b) {
        if (tid == 0) report(p.status, GQA_ERR_CONTEXT);
        const size_t n16 = (size_t)p.T * p.N * H / 8;
        uint4* dst = static_cast<uint4*>(p.out) + (size_t)b * n16;
        for (size_t i = tid; i < n16; i += blockDim.x) dst[i] = make_uint4(0, 0, 0, 0);
    };
    if (p.direct) {
        // ---- this CTA's segment: q, the first block ids and the length in one trip ------
        const int b = blockIdx.x / p.KC, k = blockIdx.x - b * p.KC;
        if (warp < NW) qr->load(p, b, k, warp, qw);
        const int i = kStepTiles * (warp + W * (lane >> 1)) + (lane & 1);
        if (p.window == 0 && i < p.max_blocks) ids = __ldg(p.block_tables + (size_t)b * p.max_blocks + i);
        more = piece.one(p, b, k);
        if (!more) {
            if (k == 0) refuse(b);
            return;
        }
        if (p.window == 0) {
            fl = 0;
            if (i >= piece.i1) ids = 0;  // an entry past the length
        }
    } else {
        // ---- this CTA's range of units --------------------------------------------------
        // Every warp adds up all lengths itself (up to 256 sequences; then the block does
        // it together).
        constexpr int seg_per_warp = q4_seg_units(NW);
        const int seg = seg_per_warp * W;
        const bool block = p.B > 256;
        const int own = block ? tid : lane, owners = block ? (int)blockDim.x : 32;
        const int per = (p.B + owners - 1) / owners;
        const int lo = min(p.B, own * per), hi = min(p.B, lo + per);
        int local = 0, longest = 0;
        bool bad = false;
#pragma unroll 4
        for (int b = lo; b < hi; ++b) {
            const int n = q4_blocks(__ldg(p.context_lens + b), p.T, p.max_blocks, p.window);
            local += q4_units(n, seg);
            longest = max(longest, n);
            bad |= n == 0;
        }
        longest = __reduce_max_sync(FULL, longest);
        int incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += v;
        }
        int before = 0, total = __shfl_sync(FULL, incl, 31);
        if (block) {
            if (lane == 31) {
                s_scan[warp] = incl;
                s_long[warp] = longest;
            }
            bad = __syncthreads_or(bad);
            total = 0;
            for (int w = 0; w < W; ++w) {
                before += w < warp ? s_scan[w] : 0;
                total += s_scan[w];
                longest = max(longest, s_long[w]);
            }
        } else {
            bad = __any_sync(FULL, bad);
        }
        total *= p.KC;
        const int excl = (before + incl - local) * p.KC, grid = gridDim.x;
        quota = total / grid + (total % grid != 0);
        quota = max(quota, 2 * kStepTiles * W);
        // Whole segments, one per CTA, where there is a CTA for each and the longest
        // exceeds an equal share by less than cutting segments costs (two more trips
        // through L2 and a fold).
        whole = p.B * p.KC <= grid && longest <= quota + kQ4CutCost * W;
        const int c0 = (int)min((long long)total, (long long)blockIdx.x * quota);
        const int c1 = (int)min((long long)total, (long long)c0 + quota);
        int at_b = 0, at_base = 0;
        const bool mine = c0 < c1 && excl <= c0 && c0 < excl + local * p.KC;
        if (mine) {  // the sequence that holds unit c0, and its first unit
            at_base = excl;
            for (at_b = lo;; ++at_b) {
                const int n = p.KC * q4_units(q4_blocks(__ldg(p.context_lens + at_b), p.T,
                                                        p.max_blocks, p.window), seg);
                if (c0 < at_base + n) break;
                at_base += n;
            }
        }
        if (bad)
            for (int b = blockIdx.x; b < p.B; b += grid)
                if (q4_blocks(p.context_lens[b], p.T, p.max_blocks, p.window) == 0) refuse(b);
        if (whole) {
            const int b = blockIdx.x / p.KC;
            more = b < p.B && piece.one(p, b, blockIdx.x - b * p.KC);
        } else {
            if (block) {
                if (mine) {
                    s_b = at_b;
                    s_base = at_base;
                }
                __syncthreads();
                at_b = s_b;
                at_base = s_base;
            } else {
                const int from = max(__ffs(__ballot_sync(FULL, mine)) - 1, 0);
                at_b = __shfl_sync(FULL, at_b, from);
                at_base = __shfl_sync(FULL, at_base, from);
            }
            more = piece.begin(p, at_b, at_base, c0, c1, seg);
        }
        if (!more) return;
        if (warp < NW) qr->load(p, piece.b, piece.k, warp, qw);
    }

    // ---- stream the range -------------------------------------------------------------
    // The piece being computed and the one being copied; their state is looked at
    // only when a piece ends, so it lives in shared memory.
    __shared__ Pieces s_piece[2][16];
    Pieces& cur = s_piece[0][warp];
    Pieces& fet = s_piece[1][warp];
    const uint8_t* ring = smem + (size_t)warp * kSlots * L::kSlot;
    const uint32_t ring_at = smem_addr(ring);
    float* head = heads + warp * Part::kHead;
    Q4Copy<H> cp;
    cp.lane_offsets(lane);
    cp.head(p, piece.k / p.C, lane);
    bool fmore = true;
    int fi = piece.i0 + kStepTiles * warp, fend = piece.i1;  // next tile to copy, its piece's end
    const uint32_t ring_end = kSlots * L::kSlot;
    uint32_t fslot = 0;  // slot to copy into
    unsigned badq = 0;   // bit i: the i-th step from the one computed has a bad block id
    if (lane == 0) cur = fet = piece;
    __syncwarp();
    const int hop = kStepTiles * W;
    // Copy this warp's next step, in whichever piece it lies.
    auto fetch = [&]() {
        if (fi >= fend && fmore) {
            Pieces t = fet;
            do {
                fmore = t.next(p);
                fi = t.i0 + kStepTiles * warp;
            } while (fmore && fi >= t.i1);
            fend = fmore ? t.i1 : 0;
            fl = 32;
            if (fmore) cp.head(p, t.k / p.C, lane);
            __syncwarp();
            if (lane == 0) fet = t;
            __syncwarp();
        }
        if (fmore) {
            if (fl == 32) {
                fl = 0;
                const int i = fi + hop * (lane >> 1) + (lane & 1);
                ids = i < fend ? __ldg(p.block_tables + (size_t)fet.b * p.max_blocks + fet.f0 + i)
                               : 0;
            }
            const uint32_t dst = ring_at + fslot;
            const uint32_t blk0 = __shfl_sync(FULL, ids, fl), blk1 = __shfl_sync(FULL, ids, fl + 1);
            const bool two = fi + 1 < fend;  // (else blk1 is 0, no id being held for it)
            if (max(blk0, blk1) < (uint32_t)p.num_blocks) {
                cp.template tile<0>(dst, blk0, p, lane);
                if (two) cp.template tile<1>(dst, blk1, p, lane);
            } else {
                badq |= 1u << (kSlots - 1);
                if (lane == 0) report(p.status, GQA_ERR_BLOCK_ID);
            }
            fi += hop;
            fl += 2;
            fslot += L::kSlot;
            if (fslot == ring_end) fslot = 0;
        }
        cp_async_commit();  // empty past the end: the count of groups stays in step
    };
#pragma unroll
    for (int i = 0; i < kSlots - 1; ++i) {
        fetch();
        badq >>= 1;
    }
    if (warp < NW) qr->make(p, warp, qw);
    __syncthreads();
    Q4Warp<H, NW, BF16> cs(p, qr);
    uint32_t slot = 0;  // of the step being computed
    while (more) {
        cs.begin(cur);
        const int iend = cur.i1, f0 = cur.f0;
        for (int i = cur.i0 + kStepTiles * warp; i < iend; i += hop) {
            __syncwarp();  // every lane is done with the slot the copy overwrites
            fetch();
            asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
            __syncwarp();  // the other lanes' copies too
            if (badq & 1u)
                cs.bad = true;
            else
                cs.step(ring + slot, i, (f0 + i) * 16, min(kStepTiles, iend - i));
            badq >>= 1;
            slot += L::kSlot;
            if (slot == ring_end) slot = 0;
        }
        // ---- the warps meet, one row tile after another -------------------------------
        cs.save_head(head);
        // the slot computed last, or the one that would have been
        const uint32_t mine = (slot == 0 ? ring_end : slot) - L::kSlot;
        float* rows = reinterpret_cast<float*>(smem + (size_t)warp * ring_end + mine);
        if (lane == 0) s_free[warp] = (uint32_t)warp * ring_end + mine;
        __syncwarp();  // every lane is done with it
        const int nrows = cs.rend - cs.rbase;
        const int first = cur.start / quota, last = (cur.start + cur.nblk - 1) / quota;
        const bool split = !whole && first != last;
        const int me = blockIdx.x;
        float* part = p.partials + ((size_t)me * 2 + (me == first ? 1 : 0)) * Part::kFloats;
        piece = cur;
        more = piece.next(p);
        if (more && warp < NW) qr->load(p, piece.b, piece.k, warp, qw);  // lands meanwhile
        bool bad = false;
        auto meet = [&](auto u_) {
            constexpr int U = decltype(u_)::value;
            if (U > 0) __syncthreads();  // the scratch is free again
            cs.template save_rows<U>(rows);
            __syncthreads();
            if (U == 0) {
                for (int w = 0; w < W; ++w) bad |= heads[w * Part::kHead + 16 * NW] != 0.f;
            }
            if (U == NW - 1 && more && warp < NW) qr->make(p, warp, qw);  // the old rows are done with
            for (int x = tid; x < min(8, nrows - 8 * U) * (H / 4); x += blockDim.x) {
                const int r = 8 * U + x / (H / 4), d = x % (H / 4) * 4;
                float M = kQ4None;
#pragma unroll 4
                for (int w = 0; w < W; ++w) M = fmaxf(M, heads[w * Part::kHead + r]);
                float l = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int w = 0; w < W; ++w) {
                    const float f = q4_weight(heads[w * Part::kHead + r], M);
                    l += f * heads[w * Part::kHead + kRows + r];
                    const float4 v = *reinterpret_cast<const float4*>(
                        fr.rows(w) + (r - 8 * U) * L::kRowFloats + d);
                    o.x += f * v.x;
                    o.y += f * v.y;
                    o.z += f * v.z;
                    o.w += f * v.w;
                }
                if (!split) {
                    const float iv = (!bad && l != 0.f) ? kQ4Unit / l : 0.f;
                    if (bad)
                        o = make_float4(0.f, 0.f, 0.f, 0.f);
                    else
                        o = make_float4(o.x * iv, o.y * iv, o.z * iv, o.w * iv);
                    q4_store4<H, BF16>(p, cs.b, cs.kv, cs.rbase + r, d, o);
                } else {
                    *reinterpret_cast<float4*>(part + Part::kHead + r * H + d) = o;
                    if (d == 0) {
                        part[r] = M;
                        part[kRows + r] = l;
                    }
                }
            }
        };
        meet(std::integral_constant<int, 0>{});
        if constexpr (NW > 1) meet(std::integral_constant<int, 1>{});
        if constexpr (NW > 2) meet(std::integral_constant<int, 2>{});
        if (split) {
            if (tid == 0) part[16 * NW] = bad ? 1.f : 0.f;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = atomicAdd(p.tickets + first, 1);
                s_last = n == last - first;
                if (s_last) p.tickets[first] = 0;  // ready for the next call
                __threadfence();
            }
            __syncthreads();
            if (s_last) fold_pieces<H, NW, BF16>(p, cs.b, cs.kv, cs.rbase, nrows, first, last, fr);
        }
        __syncthreads();  // the scratch is free again, the next piece's q rows are there
        if (lane == 0) cur = piece;
        __syncwarp();
    }
    cp_async_wait_all();
}

// ---- host -----------------------------------------------------------------------------
struct Q4Plan {
    int NW, W, grid, C, Rc, direct;
    size_t smem, part_floats, workspace;
    const void* kernel;
};

template <int H, int NW>
void q4_pick(Q4Plan* pl, bool bf16) {
    pl->kernel = bf16 ? reinterpret_cast<const void*>(&q4_attention_kernel<H, NW, true>)
                      : reinterpret_cast<const void*>(&q4_attention_kernel<H, NW, false>);
    pl->part_floats = Q4Part<H, NW>::kFloats;
    static_assert(8 * Q4<H>::kRowFloats * 4 <= Q4<H>::kSlot, "a row tile's scratch in a free slot");
    pl->smem = (size_t)pl->W * (kSlots * Q4<H>::kSlot + Q4Part<H, NW>::kHead * 4) +
               sizeof(Q4Rows<H, NW, true>);
}
template <int H>
void q4_pick(Q4Plan* pl, bool bf16) {
    if (pl->NW == 1)
        q4_pick<H, 1>(pl, bf16);
    else if (pl->NW == 2)
        q4_pick<H, 2>(pl, bf16);
    else
        q4_pick<H, 3>(pl, bf16);
}

std::mutex q4_mu;
std::map<std::tuple<int, const void*, int>, int> q4_resident;  // CTAs per SM

gqa_status q4_plan(const gqa_shape& s, Q4Plan* pl) {
    const long long R = (long long)s.T * (s.N / s.K);
    if (R > kQ4MaxRows) return GQA_ERR_SHAPE;
    if (s.K > (1 << 20)) return GQA_ERR_SHAPE;  // a block's code bytes in 32 bits
    // row chunks of up to 24 rows: every chunk converts the codes again
    pl->C = (int)((R + 8 * kQ4MaxTiles - 1) / (8 * kQ4MaxTiles));
    pl->Rc = (int)((R + pl->C - 1) / pl->C);
    pl->NW = (pl->Rc + 7) / 8;
    const long long segs = (long long)s.B * s.K * pl->C;
    // units are 32-bit in the kernel
    if (segs * ((long long)s.max_blocks_per_seq + 16 * q4_seg_units(kQ4MaxTiles)) > (1ll << 31) - 1)
        return GQA_ERR_SHAPE;
    const int sms = device_sm_count();
    if (sms <= 0) return GQA_ERR_CUDA;
    // Warps per CTA.  Many segments: small CTAs, so that few warps wait for one
    // another when a segment ends; few segments: large ones, so that a segment
    // is cut into few pieces.  Between (one to two an SM), half of the most against all of
    // them and against 4 (us): 160 segments of 1,024 tokens 17.9, 24.2, 18.8, of 8,192 58.7,
    // 63.0, 55.7; 256 of 8,192 85.5, 90.6, 81.6, with a window of 1,024 17.8, -, 25.2; 74 of
    // 4,096, H = 64, 33.3, 45.7, 39.8: never far from the best.
    const int most = q4_sm_warps(pl->NW);
    pl->W = segs > 2 * sms ? 4 : segs > sms ? most / 2 : most;
    if (s.H == 128)
        q4_pick<128>(pl, s.dtype == GQA_BF16);
    else
        q4_pick<64>(pl, s.dtype == GQA_BF16);
    int dev = 0, resident = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GQA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(q4_mu);
        const auto key = std::make_tuple(dev, pl->kernel, pl->W);
        auto it = q4_resident.find(key);
        if (it == q4_resident.end()) {
            if (cudaFuncSetAttribute(pl->kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     226 * 1024 - 2048) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, pl->kernel, 32 * pl->W,
                                                              pl->smem) != cudaSuccess ||
                resident < 1) {
                cudaGetLastError();
                return GQA_ERR_CUDA;
            }
            it = q4_resident.emplace(key, resident).first;
        }
        resident = it->second;
    }
    pl->grid = sms * resident;
    if ((size_t)pl->grid * 4 > kQ4FlagBytes) pl->grid = (int)(kQ4FlagBytes / 4);
    // A CTA per segment where there are CTAs for all and even the longest segment the
    // table allows is short: nothing is planned, cut or folded then.
    const long long reach =
        s.window > 0 ? ((long long)s.window + s.T + 14) / 16 + 1 : s.max_blocks_per_seq;
    pl->direct = segs <= pl->grid &&
                 (reach < s.max_blocks_per_seq ? reach : s.max_blocks_per_seq) <= kQ4Direct * pl->W;
    if (pl->direct) pl->grid = (int)segs;
    pl->workspace = kQ4FlagBytes + (size_t)pl->grid * 2 * pl->part_floats * 4;
    return GQA_OK;
}

}  // namespace

gqa_status fourbit_workspace_bytes(const gqa_shape& s, size_t* bytes) {
    Q4Plan pl;
    const gqa_status st = q4_plan(s, &pl);
    if (st == GQA_OK) *bytes = pl.workspace;
    return st;
}

gqa_status launch_attention_fourbit(const gqa_shape& s, const void* q, const uint8_t* k_cache,
                                    const uint8_t* v_cache, const uint8_t* k_scale,
                                    const uint8_t* v_scale, const int32_t* block_tables,
                                    const int32_t* context_lens, const uint64_t* tree_mask,
                                    void* out, void* workspace, size_t ws_bytes,
                                    int32_t* dev_status, cudaStream_t stream) {
    Q4Plan pl;
    const gqa_status st = q4_plan(s, &pl);
    if (st != GQA_OK) return st;
    if (!workspace || ws_bytes < pl.workspace) return GQA_ERR_WORKSPACE;
    Q4Params p = {};
    p.q = q;
    p.out = out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.tree_mask = tree_mask;
    p.tickets = static_cast<int32_t*>(workspace);
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kQ4FlagBytes);
    p.status = dev_status;
    p.B = s.B;
    p.T = s.T;
    p.N = s.N;
    p.K = s.K;
    p.G = s.N / s.K;
    p.R = s.T * p.G;
    p.C = pl.C;
    p.Rc = pl.Rc;
    p.KC = s.K * pl.C;
    p.max_blocks = s.max_blocks_per_seq;
    p.num_blocks = s.num_blocks;
    p.window = s.window;
    p.direct = pl.direct;
    const float scale = s.scale > 0.f ? s.scale : 1.f / sqrtf((float)s.H);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.code_stride = (uint32_t)s.K * (uint32_t)(16 * s.H / 2);
    p.scale_stride = (uint32_t)s.K * (uint32_t)(16 * s.H / kQ4Group);
    p.ex[0] = 0x64006400u;
    p.ex[1] = 0x54005400u;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pl.grid);
    cfg.blockDim = dim3(32u * pl.W);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (s.flags & (GQA_FLAG_PDL | GQA_FLAG_EARLY_KV)) ? 1 : 0;
    void* args[] = {&p};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, pl.kernel, args);
    return launch_status(e);
}

}  // namespace gqa
