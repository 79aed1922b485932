// attention_fourbit.cu -- decode / verify attention over a paged cache held in
// 4 bits (codes and scales: fourbit.cuh).
//
// For sequence b, new token t and query head n of KV head k = n / G:
//     s_j = scale * <q[b,t,n,:], K_b[j,k,:]>,   out = sum_j softmax(s)_j V_b[j,k,:]
// over the positions j that token t sees (causal, window, tree mask as in the
// other attention calls), K and V being code * group scale.
//
// What bounds it.  A position costs 2 * (H/2 + H/32) bytes per KV head (136 at
// H = 128).  At 6.78 TB/s over 152 SMs a 16-token tile (2,176 bytes) arrives
// every ~93 cycles per SM, in which its four schedulers issue ~370
// instructions: the 16 words a lane holds of the tile must become f16 operands
// within that, so instructions per code word, not bytes, are what is saved
// first.  Everything below is chosen for that.
//
//  * No producer warp, no barriers in the loop: each warp copies its own tiles
//    with 16-byte cp.async (9 instructions per two tiles) into a double buffer
//    of its own and waits for its own copies only.
//  * Natural storage order, fragments by permutation.  Lane (g, q4) (g = lane /
//    4) reads K dims H/4*q4 .. of its two tokens with one wide load each: one
//    group per lane, one scale per token; V dims H/8*g .. of its four tokens:
//    one group per lane again, and the output leaves as contiguous dims.  q is
//    permuted to match once per segment.
//  * Codes become f16 by or-ing a nibble under an exponent (0x6400: 1024 + n;
//    nibbles one place up, 0x5400: 64 + n), subtracting the offset and
//    multiplying by the scale: all exact (fourbit.cuh), so products are those
//    of the cached values and sums are fp32.
//  * S^T[16 tokens x 8 rows] and O^T[H x 8 rows] on mma.sync m16n8k16, tokens
//    (dims) on M: up to 8 query rows cost 16 mma per tile.  Decode attention
//    has T*G = 1..16 rows; tcgen05's M = 128 would be empty there, and its
//    operands would have to pass through shared memory as f16.
//
// Work split.  The batch's segments (sequence, KV head, row chunk) are laid end
// to end in units (a segment's start-up units, then its tiles) and CTA c takes
// the c-th equal range.  The warps of a CTA take tile pairs of a segment in
// turn and meet in shared memory when it ends; a segment cut by a range
// boundary goes through the workspace, the CTA that finishes last folding the
// pieces in order (deterministic; nobody waits).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <map>
#include <mutex>
#include <tuple>

#include "fourbit.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kStepTiles = 2;    // tiles a warp computes per step
constexpr int kSlots = 2;        // steps in a warp's buffer
constexpr int kQ4SegUnits = 6;   // start-up cost of a segment, in tiles
constexpr float kQ4Gap = 8.0f;   // log2-domain slack before rescaling
constexpr size_t kQ4FlagBytes = 262144; // tickets, one per CTA (as large as the other kernels' region)
constexpr long long kQ4MaxRows = 8192;  // T*G

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
    float scale_log2;
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
__device__ __forceinline__ int q4_units(int nblk) { return nblk > 0 ? nblk + kQ4SegUnits : 0; }

// The pieces of segments in one CTA's range of units, in order.
struct Pieces {
    int b, k;        // sequence, virtual head
    int ctx, nblk, f0;
    int start;       // unit of the segment's first tile
    int i0, i1;      // this CTA's tiles of it
    int c0, c1;      // the range

    __device__ void load(const Q4Params& p) {
        ctx = __ldg(p.context_lens + b);
        nblk = q4_blocks(ctx, p.T, p.max_blocks, p.window);
        f0 = q4_first_block(ctx, p.T, p.window);
    }
    __device__ bool clip() {
        i0 = max(0, c0 - start);
        i1 = min(nblk, c1 - start);
        return i1 > i0;
    }
    // From the segment holding unit c0 (sequence b_, whose first unit is base):
    // the first piece with tiles; false if the range holds none.
    __device__ bool begin(const Q4Params& p, int b_, int base, int lo, int hi) {
        c0 = lo;
        c1 = hi;
        b = b_;
        if (c0 >= c1) return false;
        load(p);
        const int u = q4_units(nblk);
        k = (c0 - base) / u;
        start = base + k * u + kQ4SegUnits;
        return clip() || next(p);
    }
    __device__ bool next(const Q4Params& p) {
        while (true) {
            start += nblk + kQ4SegUnits;
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

// Copies of one step (tiles i, i+1 of a piece, those below i1) into a slot.
// K rows go to row r ^ ((r >> 2) & 1) at H = 128 (r ^ 2 * that at H = 64) and V
// chunks to c ^ 2 * ((r >> 1) & 1): the fragment loads are then free of bank
// conflicts.
template <int H>
__device__ __forceinline__ void q4_copy_tile(uint32_t dst, const Q4Params& p, int blk, int kv,
                                             int lane) {
    using L = Q4<H>;
    const size_t tile = (size_t)blk * p.K + kv;
    const uint8_t* kc = p.k_cache + tile * L::kCodes + lane * 16;
    const uint8_t* vc = p.v_cache + tile * L::kCodes + lane * 16;
    if constexpr (H == 128) {
        const int r = lane >> 2, c = lane & 3;
        const uint32_t ko = (uint32_t)((r ^ ((r >> 2) & 1)) * 64 + c * 16);
        const uint32_t vo = (uint32_t)(r * 64 + ((c ^ (r & 2)) << 4));
        cp_async_16(dst + ko, kc);
        cp_async_16(dst + 512 + ko, kc + 512);  // rows 8..15: the same swizzle
        cp_async_16(dst + L::kCodes + vo, vc);
        cp_async_16(dst + L::kCodes + 512 + vo, vc + 512);
    } else {
        const int r = lane >> 1, c = lane & 1;
        const uint32_t ko = (uint32_t)((r ^ ((r >> 1) & 2)) * 32 + c * 16);
        cp_async_16(dst + ko, kc);
        cp_async_16(dst + L::kCodes + lane * 16, vc);
    }
    constexpr int kSc = L::kScales / 16;  // 16-byte pieces of each scale tile
    if (lane < 2 * kSc) {
        const bool v = lane >= kSc;
        const int c = v ? lane - kSc : lane;
        cp_async_16(dst + 2 * L::kCodes + lane * 16,
                    (v ? p.v_scale : p.k_scale) + tile * L::kScales + c * 16);
    }
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 v = ld_shared_v4(addr);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (W == 2) {
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    }
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) {
    return *reinterpret_cast<__half2*>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Four code pairs of a word -- nibbles i of its two halves, i = 0..3 -- times
// their scales (low half, high half), as f16x2; exact.
__device__ __forceinline__ void q4_values(uint32_t x, __half2 s, uint32_t (&v)[4]) {
    const __half2 o0 = as_h2(0x64086408u);  // 1024 + 8
    const __half2 o1 = as_h2(0x54805480u);  // 64 + 8
    const uint32_t y = x >> 8;
    v[0] = as_u32(__hmul2(__hsub2(as_h2((x & 0x000f000fu) | 0x64006400u), o0), s));
    v[1] = as_u32(__hmul2(__hsub2(as_h2((x & 0x00f000f0u) | 0x54005400u), o1), s));
    v[2] = as_u32(__hmul2(__hsub2(as_h2((y & 0x000f000fu) | 0x64006400u), o0), s));
    v[3] = as_u32(__hmul2(__hsub2(as_h2((y & 0x00f000f0u) | 0x54005400u), o1), s));
}

// A warp's state for one piece of a segment: NW tiles of 8 query rows.
template <int H, bool BF16, int NW>
struct Q4Warp {
    using L = Q4<H>;
    using E = Elt<false>;  // the mma's operands are f16 for either type of q
    const Q4Params& p;
    const int lane, g, q4;
    int r0[NW];  // first of this lane's two query rows (of R), per tile
    int lim0[NW], lim1[NW];       // last position rows r0, r0 + 1 see
    int rbase, rend, b, kv, ctx;
    uint32_t qf[NW][L::kSteps][2];
    float acc[NW][L::kSteps][4];
    float sl0[NW], sl1[NW];  // score factor to the log2 domain, per row
    float m0[NW], m1[NW], l0[NW], l1[NW];
    bool bad;

    __device__ Q4Warp(const Q4Params& p_)
        : p(p_), lane(threadIdx.x & 31), g((threadIdx.x & 31) >> 2), q4(threadIdx.x & 3) {}

    // q rows of the segment as B fragments.  Row u*8+g, dims H/4*q4 ..: word j
    // of a token's codes meets steps 2j (nibbles 0|4, 1|5) and 2j+1 (2|6, 3|7).
    // bf16 rows are scaled by a power of two that puts their largest element
    // near 2^14: f16 then holds every bf16 q exactly down to 2^-31 of it.
    __device__ void begin(const Pieces& s) {
        b = s.b;
        ctx = s.ctx;
        kv = s.k / p.C;
        rbase = (s.k - kv * p.C) * p.Rc;
        rend = min(p.R, rbase + p.Rc);
        bad = false;
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            r0[u] = rbase + 8 * u + 2 * q4;
            lim0[u] = ctx - p.T + min(r0[u] / p.G, p.T - 1);
            lim1[u] = ctx - p.T + min((r0[u] + 1) / p.G, p.T - 1);
            m0[u] = m1[u] = -INFINITY;
            l0[u] = l1[u] = 0.f;
#pragma unroll
            for (int mt = 0; mt < L::kSteps; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[u][mt][e] = 0.f;
            const int r = rbase + 8 * u + g;
            uint32_t w[H / 8];
#pragma unroll
            for (int i = 0; i < H / 8; ++i) w[i] = 0u;
            if (r < rend) {
                const int t = r / p.G, gg = r - t * p.G;
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(p.q) +
                    (((size_t)b * p.T + t) * p.N + (size_t)kv * p.G + gg) * H + q4 * (H / 4));
#pragma unroll
                for (int i = 0; i < H / 32; ++i) {
                    const uint4 x = __ldg(src + i);
                    w[4 * i] = x.x;
                    w[4 * i + 1] = x.y;
                    w[4 * i + 2] = x.z;
                    w[4 * i + 3] = x.w;
                }
            }
            float back = 1.f;
            if constexpr (BF16) {
                uint32_t top = 0u;  // largest exponent field of the row
#pragma unroll
                for (int i = 0; i < H / 8; ++i)
                    top = max(top, max((w[i] >> 7) & 0xffu, (w[i] >> 23) & 0xffu));
                top = max(top, __shfl_xor_sync(FULL, top, 1));
                top = max(top, __shfl_xor_sync(FULL, top, 2));
                const int e = min(max(127 + 14 - (int)top, -112), 112);  // row times 2^e
                const float f = __uint_as_float((uint32_t)(127 + e) << 23);
                back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int i = 0; i < H / 8; ++i)
                    w[i] = E::pack(__uint_as_float(w[i] << 16) * f,
                                   __uint_as_float(w[i] & 0xffff0000u) * f);
            }
            // the factors of the rows this lane's scores belong to (rows 2*q4 and
            // 2*q4 + 1 sit in lanes 8*q4 and 8*q4 + 4); never 0, which a hidden
            // position's -inf must not meet
            sl0[u] = fmaxf(p.scale_log2 * __shfl_sync(FULL, back, 8 * q4), 1.17549435e-38f);
            sl1[u] = fmaxf(p.scale_log2 * __shfl_sync(FULL, back, 8 * q4 + 4), 1.17549435e-38f);
#pragma unroll
            for (int j = 0; j < L::kKWords; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    qf[u][2 * j + h][0] = prmt(w[4 * j + h], w[4 * j + 2 + h], 0x5410u);
                    qf[u][2 * j + h][1] = prmt(w[4 * j + h], w[4 * j + 2 + h], 0x7632u);
                }
        }
    }

    // Hide score entries of tile position tb (of this lane's tokens tb + ta and
    // tb + ta + 8) from the rows that do not see them.
    __device__ __forceinline__ void mask(float (&sc)[4], int u, int tb) const {
        const int ta = (g >> 1) + 4 * (g & 1);
        const int wl = p.window > 0 ? p.window : (1 << 30);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int pos = tb + ta + (e >> 1) * 8;
            const int lim = (e & 1) ? lim1[u] : lim0[u];
            bool off = pos > lim || pos <= lim - wl;
            if (p.tree_mask) {
                const int fn = ctx - p.T;
                if (pos >= fn && pos < lim) {
                    const uint64_t row = __ldg(p.tree_mask + (size_t)b * p.T + (lim - fn));
                    off |= !((row >> (pos - fn)) & 1ull);
                }
            }
            if (off) sc[e] = -INFINITY;
        }
    }

    // One step: nt tiles (1 or 2) whose first position is tb, in the slot at sm.
    __device__ __forceinline__ void step(uint32_t sm, int tb, int nt) {
        const int ta = (g >> 1) + 4 * (g & 1);  // this lane's K tokens: ta, ta + 8
        float sc[kStepTiles][NW][4];
#pragma unroll
        for (int j = 0; j < kStepTiles; ++j) {
#pragma unroll
            for (int u = 0; u < NW; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][u][e] = 0.f;
            const uint32_t kb = sm + j * L::kTile;
            const int ra = H == 128 ? (ta ^ ((ta >> 2) & 1)) : (ta ^ ((ta >> 1) & 2));
            uint32_t wa[L::kKWords], wb[L::kKWords];
            lds_words(kb + ra * L::kRow + q4 * (L::kRow / 4), wa);
            lds_words(kb + (ra + 8) * L::kRow + q4 * (L::kRow / 4), wb);
            const uint32_t sb = kb + 2 * L::kCodes + ta * L::kGroups + q4 * L::kGroups / 4;
            const __half2 s_a = as_h2(lds_u8(sb) * 0x00800080u);
            const __half2 s_b = as_h2(lds_u8(sb + 8 * L::kGroups) * 0x00800080u);
#pragma unroll
            for (int i = 0; i < L::kKWords; ++i) {
                uint32_t va[4], vb[4];
                q4_values(wa[i], s_a, va);
                q4_values(wb[i], s_b, vb);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a[4] = {va[2 * h], vb[2 * h], va[2 * h + 1], vb[2 * h + 1]};
#pragma unroll
                    for (int u = 0; u < NW; ++u)
                        E::mma(sc[j][u], a, qf[u][2 * i + h][0], qf[u][2 * i + h][1]);
                }
            }
        }
        // masks: only where some position of the step is hidden from some row
        const int last = tb + 16 * nt - 1;
        const bool edge = nt < kStepTiles || last > ctx - p.T - (p.tree_mask ? 1 : 0) ||
                          (p.window > 0 && tb < ctx - p.window);
        if (edge) {
#pragma unroll
            for (int j = 0; j < kStepTiles; ++j)
#pragma unroll
                for (int u = 0; u < NW; ++u) {
                    if (j < nt) {
                        mask(sc[j][u], u, tb + 16 * j);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[j][u][e] = -INFINITY;
                    }
                }
        }
        // running maximum: rescale only when it grows by more than 2^kQ4Gap
        float ref0[NW], ref1[NW];
#pragma unroll
        for (int u = 0; u < NW; ++u) {
            float x0 = sc[0][u][0], x1 = sc[0][u][1];
#pragma unroll
            for (int j = 0; j < kStepTiles; ++j) {
                x0 = fmaxf(x0, fmaxf(sc[j][u][0], sc[j][u][2]));
                x1 = fmaxf(x1, fmaxf(sc[j][u][1], sc[j][u][3]));
            }
            x0 *= sl0[u];
            x1 *= sl1[u];
            if (__any_sync(FULL, x0 > m0[u] + kQ4Gap || x1 > m1[u] + kQ4Gap)) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(FULL, x0, o));
                    x1 = fmaxf(x1, __shfl_xor_sync(FULL, x1, o));
                }
                const bool up0 = x0 > m0[u] + kQ4Gap, up1 = x1 > m1[u] + kQ4Gap;
                const float f0 = up0 ? fast_exp2(m0[u] - x0) : 1.f;
                const float f1 = up1 ? fast_exp2(m1[u] - x1) : 1.f;
                if (up0) m0[u] = x0;
                if (up1) m1[u] = x1;
                l0[u] *= f0;
                l1[u] *= f1;
#pragma unroll
                for (int mt = 0; mt < L::kSteps; ++mt) {
                    acc[u][mt][0] *= f0;
                    acc[u][mt][1] *= f1;
                    acc[u][mt][2] *= f0;
                    acc[u][mt][3] *= f1;
                }
            }
            ref0[u] = m0[u] == -INFINITY ? 0.f : m0[u];
            ref1[u] = m1[u] == -INFINITY ? 0.f : m1[u];
        }
        // O^T += V^T P^T, tile by tile.  The probabilities enter the product as
        // f16 (half an ulp is 2^-12 of them, below the output's own rounding);
        // their sum stays fp32.
#pragma unroll
        for (int j = 0; j < kStepTiles; ++j) {
            if (j >= nt) break;  // warp-uniform
            uint32_t pb[NW][2];
#pragma unroll
            for (int u = 0; u < NW; ++u) {
                const float e0 = fast_exp2(fmaf(sc[j][u][0], sl0[u], -ref0[u]));
                const float e1 = fast_exp2(fmaf(sc[j][u][1], sl1[u], -ref1[u]));
                const float e2 = fast_exp2(fmaf(sc[j][u][2], sl0[u], -ref0[u]));
                const float e3 = fast_exp2(fmaf(sc[j][u][3], sl1[u], -ref1[u]));
                l0[u] += e0 + e2;
                l1[u] += e1 + e3;
                pb[u][0] = movm_t(E::pack(e0, e1));
                pb[u][1] = movm_t(E::pack(e2, e3));
            }
            const uint32_t vb = sm + j * L::kTile + L::kCodes;
            const uint32_t sb = sm + j * L::kTile + 2 * L::kCodes + L::kScales +
                                q4 * L::kGroups + g * L::kGroups / 8;
            uint32_t w[4][L::kVWords], s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // tokens q4 + 4i
                const int r = q4 + 4 * i;
                const uint32_t off =
                    H == 128 ? (uint32_t)(r * 64 + ((((g >> 1) ^ (q4 & 2)) << 4) | ((g & 1) << 3)))
                             : (uint32_t)(r * 32 + g * 4);
                lds_words(vb + off, w[i]);
                s[i] = lds_u8(sb + 4 * i * L::kGroups);
            }
            // Rows past the context or below every window may hold anything:
            // scale 0 makes their values zeros.
            const int t0 = tb + 16 * j, lo = p.window > 0 ? ctx - p.T - p.window + 1 : 0;
            if (t0 + 16 > ctx || t0 < lo) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int pos = t0 + q4 + 4 * i;
                    if (pos >= ctx || pos < lo) s[i] = 0u;
                }
            }
            const __half2 s01 = as_h2((s[0] << 7) | (s[1] << 23));
            const __half2 s23 = as_h2((s[2] << 7) | (s[3] << 23));
#pragma unroll
            for (int i = 0; i < L::kVWords; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h ? 0x7632u : 0x5410u;
                    uint32_t va[4], vc[4];
                    q4_values(prmt(w[0][i], w[1][i], sel), s01, va);
                    q4_values(prmt(w[2][i], w[3][i], sel), s23, vc);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int mt = 4 * i + 2 * h + x;
                        const uint32_t a[4] = {va[2 * x], va[2 * x + 1], vc[2 * x],
                                               vc[2 * x + 1]};
#pragma unroll
                        for (int u = 0; u < NW; ++u) E::mma(acc[u][mt], a, pb[u][0], pb[u][1]);
                    }
                }
        }
    }

    // This warp's (max, sum, accumulator) of every row to its scratch rows.
    __device__ void save(float* head, float* rows) {
#pragma unroll
        for (int u = 0; u < NW; ++u) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l0[u] += __shfl_xor_sync(FULL, l0[u], o);
                l1[u] += __shfl_xor_sync(FULL, l1[u], o);
            }
            const int r = 8 * u + 2 * q4;
            if (g == 0) {
                head[r] = m0[u];
                head[r + 1] = m1[u];
                head[8 * NW + r] = l0[u];
                head[8 * NW + r + 1] = l1[u];
            }
            float* d0 = rows + r * L::kRowFloats + g * (H / 8);
            float* d1 = d0 + L::kRowFloats;
#pragma unroll
            for (int i = 0; i < L::kSteps / 2; ++i) {
                reinterpret_cast<float4*>(d0)[i] =
                    make_float4(acc[u][2 * i][0], acc[u][2 * i][2], acc[u][2 * i + 1][0],
                                acc[u][2 * i + 1][2]);
                reinterpret_cast<float4*>(d1)[i] =
                    make_float4(acc[u][2 * i][1], acc[u][2 * i][3], acc[u][2 * i + 1][1],
                                acc[u][2 * i + 1][3]);
            }
        }
        if (lane == 0) head[16 * NW] = bad ? 1.f : 0.f;
    }
};

__device__ __forceinline__ float q4_weight(float m, float M) {
    return m == -INFINITY ? 0.f : fast_exp2(m - M);
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

template <int H, bool BF16, int NW>
__global__ void __launch_bounds__(NW == 1 ? 512 : 384, 1) q4_attention_kernel(const Q4Params p) {
    using L = Q4<H>;
    using Part = Q4Part<H, NW>;
    constexpr int kRows = 8 * NW;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_scan[16], s_b, s_base, s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = blockDim.x >> 5;
    float* heads = reinterpret_cast<float*>(smem + (size_t)W * kSlots * L::kSlot);
    float* scratch = heads + W * Part::kHead;
    griddep_launch_dependents();
    griddep_wait();

    // ---- this CTA's range of units --------------------------------------------------
    const int per = (p.B + blockDim.x - 1) / blockDim.x;
    const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
    int local = 0;
    for (int b = lo; b < hi; ++b)
        local += q4_units(q4_blocks(p.context_lens[b], p.T, p.max_blocks, p.window));
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < W; ++w) {
        before += w < warp ? s_scan[w] : 0;
        total += s_scan[w];
    }
    total *= p.KC;
    const int excl = (before + incl - local) * p.KC;
    const int quota = max((int)(((long long)total + gridDim.x - 1) / gridDim.x), 2 * kStepTiles * W);
    const int c0 = min((long long)total, (long long)blockIdx.x * quota);
    const int c1 = min((long long)total, (long long)c0 + quota);
    if (c0 < c1 && excl <= c0 && c0 < excl + local * p.KC) {
        int base = excl;
        for (int b = lo; b < hi; ++b) {
            const int n = p.KC * q4_units(q4_blocks(p.context_lens[b], p.T, p.max_blocks, p.window));
            if (c0 < base + n) {
                s_b = b;
                s_base = base;
                break;
            }
            base += n;
        }
    }
    // sequences of an invalid length: zeros
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (q4_blocks(p.context_lens[b], p.T, p.max_blocks, p.window) == 0) {
            if (tid == 0) report(p.status, GQA_ERR_CONTEXT);
            const size_t n16 = (size_t)p.T * p.N * H / 8;
            uint4* dst = static_cast<uint4*>(p.out) + (size_t)b * n16;
            for (size_t i = tid; i < n16; i += blockDim.x) dst[i] = make_uint4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    if (c0 >= c1) return;

    // ---- stream the range -------------------------------------------------------------
    const uint32_t ring = smem_addr(smem + (size_t)warp * kSlots * L::kSlot);
    float* head = heads + warp * Part::kHead;
    float* rows = scratch + (size_t)warp * kRows * L::kRowFloats;
    Q4Warp<H, BF16, NW> cs(p);
    Pieces cur, fet;  // the piece being computed, and the one being copied
    bool more = cur.begin(p, s_b, s_base, c0, c1);
    fet = cur;
    bool fmore = more;
    int fi = fet.i0 + kStepTiles * warp;  // next tile to copy
    int fst = 0, fkv = fet.k / p.C;       // its step within the piece, its KV head
    int ids = 0;                          // block ids of 16 steps, from step fst & ~15
    int fs = 0;                           // steps copied (ring position)
    unsigned badbits = 0;                 // per slot: an invalid block id
    // Copy this warp's next step, in whichever piece it lies.
    auto fetch = [&]() {
        while (fmore && fi >= fet.i1) {
            fmore = fet.next(p);
            fi = fet.i0 + kStepTiles * warp;
            fst = 0;
            fkv = fet.k / p.C;
        }
        if (fmore) {
            if ((fst & 15) == 0) {
                const int i = fi + kStepTiles * W * (lane >> 1) + (lane & 1);
                ids = i < fet.i1 ? __ldg(p.block_tables + (size_t)fet.b * p.max_blocks + fet.f0 + i)
                                 : 0;
            }
            const uint32_t dst = ring + (fs % kSlots) * L::kSlot;
            bool bad = false;
#pragma unroll
            for (int j = 0; j < kStepTiles; ++j) {
                const int blk = __shfl_sync(FULL, ids, 2 * (fst & 15) + j);
                if (fi + j < fet.i1) {
                    if (blk >= 0 && blk < p.num_blocks)
                        q4_copy_tile<H>(dst + j * L::kTile, p, blk, fkv, lane);
                    else
                        bad = true;
                }
            }
            const unsigned bit = 1u << (fs % kSlots);
            badbits = bad ? badbits | bit : badbits & ~bit;
            if (bad && lane == 0) report(p.status, GQA_ERR_BLOCK_ID);
            fi += kStepTiles * W;
            ++fst;
            ++fs;
        }
        cp_async_commit();  // empty past the end: the count of groups stays in step
    };
#pragma unroll
    for (int i = 0; i < kSlots - 1; ++i) fetch();
    int done = 0;  // steps computed
    while (more) {
        cs.begin(cur);
        for (int i = cur.i0 + kStepTiles * warp; i < cur.i1; i += kStepTiles * W) {
            __syncwarp();  // every lane is done with the slot the copy overwrites
            fetch();
            asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
            __syncwarp();  // the other lanes' copies too
            if (badbits >> (done % kSlots) & 1u)
                cs.bad = true;
            else
                cs.step(ring + (done % kSlots) * L::kSlot, (cur.f0 + i) * 16,
                        min(kStepTiles, cur.i1 - i));
            ++done;
        }
        // ---- the warps meet -----------------------------------------------------------
        cs.save(head, rows);
        __syncthreads();
        const int nrows = cs.rend - cs.rbase;
        const int first = cur.start / quota, last = (cur.start + cur.nblk - 1) / quota;
        const bool split = first != last;
        const int me = blockIdx.x;
        float* part = p.partials + ((size_t)me * 2 + (me == first ? 1 : 0)) * Part::kFloats;
        bool bad = false;
        for (int w = 0; w < W; ++w) bad |= heads[w * Part::kHead + 16 * NW] != 0.f;
        for (int x = tid; x < nrows * (H / 4); x += blockDim.x) {
            const int r = x / (H / 4), d = x % (H / 4) * 4;
            float M = -INFINITY;
            for (int w = 0; w < W; ++w) M = fmaxf(M, heads[w * Part::kHead + r]);
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < W; ++w) {
                const float f = q4_weight(heads[w * Part::kHead + r], M);
                l += f * heads[w * Part::kHead + kRows + r];
                const float4 v = *reinterpret_cast<const float4*>(
                    scratch + ((size_t)w * kRows + r) * L::kRowFloats + d);
                o.x += f * v.x;
                o.y += f * v.y;
                o.z += f * v.z;
                o.w += f * v.w;
            }
            if (!split) {
                const float iv = (!bad && l != 0.f) ? 1.f / l : 0.f;
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
            if (s_last) {  // every piece is in: fold them in order
                auto sec = [&](int c) {
                    return p.partials + ((size_t)c * 2 + (c == first ? 1 : 0)) * Part::kFloats;
                };
                for (int x = tid; x < nrows * (H / 4); x += blockDim.x) {
                    const int r = x / (H / 4), d = x % (H / 4) * 4;
                    float M = -INFINITY;
                    bool any = false;
                    for (int c = first; c <= last; ++c) {
                        M = fmaxf(M, __ldcg(sec(c) + r));
                        any |= __ldcg(sec(c) + 16 * NW) != 0.f;
                    }
                    float l = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = first; c <= last; ++c) {
                        const float f = q4_weight(__ldcg(sec(c) + r), M);
                        l += f * __ldcg(sec(c) + kRows + r);
                        const float4 v = __ldcg(
                            reinterpret_cast<const float4*>(sec(c) + Part::kHead + r * H + d));
                        o.x += f * v.x;
                        o.y += f * v.y;
                        o.z += f * v.z;
                        o.w += f * v.w;
                    }
                    const float iv = 1.f / l;
                    if (any)
                        o = make_float4(0.f, 0.f, 0.f, 0.f);
                    else
                        o = make_float4(o.x * iv, o.y * iv, o.z * iv, o.w * iv);
                    q4_store4<H, BF16>(p, cs.b, cs.kv, cs.rbase + r, d, o);
                }
            }
        }
        __syncthreads();  // the scratch is free again
        more = cur.next(p);
    }
    cp_async_wait_all();
}

// ---- host -----------------------------------------------------------------------------
struct Q4Plan {
    int NW, W, grid, C, Rc;
    size_t smem, part_floats, workspace;
    const void* kernel;
};

template <int H, bool BF16>
const void* q4_pick(int NW) {
    return NW == 1 ? reinterpret_cast<const void*>(&q4_attention_kernel<H, BF16, 1>)
                   : reinterpret_cast<const void*>(&q4_attention_kernel<H, BF16, 2>);
}

std::mutex q4_mu;
std::map<std::tuple<int, const void*, int>, int> q4_resident;  // CTAs per SM

gqa_status q4_plan(const gqa_shape& s, Q4Plan* pl) {
    const long long R = (long long)s.T * (s.N / s.K);
    if (R > kQ4MaxRows) return GQA_ERR_SHAPE;
    pl->NW = R <= 8 ? 1 : 2;
    pl->C = (int)((R + 8 * pl->NW - 1) / (8 * pl->NW));
    pl->Rc = (int)((R + pl->C - 1) / pl->C);
    const long long segs = (long long)s.B * s.K * pl->C;
    // units are 32-bit in the kernel
    if (segs * ((long long)s.max_blocks_per_seq + kQ4SegUnits) > (1ll << 31) - 1)
        return GQA_ERR_SHAPE;
    const int sms = device_sm_count();
    if (sms <= 0) return GQA_ERR_CUDA;
    // Warps per CTA.  Many segments: small CTAs, so that few warps wait for one
    // another when a segment ends; few segments: large ones, so that a segment
    // is cut into few pieces.
    const int most = pl->NW == 1 ? 16 : 12;
    pl->W = segs >= 2 * sms ? 4 : most;
    const int slot = (s.H == 128 ? Q4<128>::kSlot : Q4<64>::kSlot);
    pl->part_floats = (size_t)(16 * pl->NW + 4) + (size_t)8 * pl->NW * s.H;
    pl->smem = (size_t)pl->W * (kSlots * slot + (16 * pl->NW + 4) * 4 +
                                (size_t)8 * pl->NW * (s.H + 4) * 4);
    pl->kernel = s.H == 128 ? (s.dtype == GQA_BF16 ? q4_pick<128, true>(pl->NW)
                                                   : q4_pick<128, false>(pl->NW))
                            : (s.dtype == GQA_BF16 ? q4_pick<64, true>(pl->NW)
                                                   : q4_pick<64, false>(pl->NW));
    int dev = 0, resident = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return GQA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(q4_mu);
        const auto key = std::make_tuple(dev, pl->kernel, pl->W);
        auto it = q4_resident.find(key);
        if (it == q4_resident.end()) {
            if (cudaFuncSetAttribute(pl->kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     227 * 1024 - 1024) != cudaSuccess ||
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
    const float scale = s.scale > 0.f ? s.scale : 1.f / sqrtf((float)s.H);
    p.scale_log2 = scale * 1.4426950408889634f;
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
    return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa
