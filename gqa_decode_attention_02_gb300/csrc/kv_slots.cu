// kv_slots.cu -- rows written into and read from a paged cache by position:
//   kv_append_fourbit  the T newest tokens of every sequence into a 4-bit cache,
//                      by block table (as gqa_kv_append)
//   kv_append_slots    packed rows [M][K][H] of any number of requests into a
//                      cache of any kind, by a slot per row (block * 16 + row)
//   kv_gather_slots    the way back: rows [M][K][H] in the dtype of the shape
//
// CS336 lecture 10 §"PagedAttention" (fixed-size blocks; a token's place is its
// block and its row); the quantization is that of kv_quant.cu (one byte) and
// fourbit.cuh (4 bits).
//
// All of it is moving bytes: the floor is the 16-bit side plus the cache side
// once.  A thread owns 8 consecutive elements (one 16-byte access on the 16-bit
// side) of a key and a value row, or 16 on the way to 4 bits; two threads share a
// 4-bit group and H/8 an 8-bit row, so maxima take one (or log2(H/8)) shuffles
// inside the warp and every row is written as one contiguous piece.  At 4 bits the
// arithmetic comes close to the bytes: maxima are taken on the packed 16-bit
// patterns, codes without a division and two to an instruction (fourbit.cuh), and
// clipping is left to the warps whose scales need it.  36,060 rows of prompts
// (8 heads of 128, bf16) at 4 bits, on the device: put 30 us and take 32 us for
// 187 MB each, 6.2 and 5.8 TB/s of the 6.8 that a copy reaches.  (Take with two
// parts a thread: no faster.)  16-bit caches: 45 and 46 us for 295 MB, 6.6 and 6.5 TB/s.
// One-byte caches: take 37 us for 224 MB, 6.0 TB/s, put 74 us (int8) and 65 us (e4m3), 3.0
// and 3.4 TB/s, bound by a division and a conversion per element.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fourbit.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int kSlotThreads = 256;
constexpr int kKvFourbit = GQA_KV_INT4;

struct SlotParams {
    const uint4* k_new;  // rows [M][K][H]
    const uint4* v_new;
    uint4* k_out;
    uint4* v_out;
    uint8_t* k_cache;
    uint8_t* v_cache;
    void* k_scale;
    void* v_scale;
    const int32_t* slots;  // [M]; nullptr: by block table
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* status;
    uint32_t rows, T, K;
    uint32_t kmul, kshift;  // i / K = (umulhi(i, kmul) + i) >> kshift, i < 2^31
    int max_blocks, num_blocks;
};

template <bool BF16>
__device__ __forceinline__ void widen8(uint4 w, float (&x)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = Elt<BF16>::lo(a[i]);
        x[2 * i + 1] = Elt<BF16>::hi(a[i]);
    }
}

// Max over the N threads (a power of two, aligned in the warp) that share it.
template <int N>
__device__ __forceinline__ float max_over(float a) {
#pragma unroll
    for (int o = 1; o < N; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// Cache slot of row i (token t of sequence b by block table), -1: none.
__device__ __forceinline__ int slot_of(const SlotParams& p, uint32_t i, bool reporter) {
    if (p.slots) {
        const int s = __ldg(p.slots + i);
        if (s >= 0 && (s >> 4) < p.num_blocks) return s;
        if (s != -1 && reporter) report(p.status, GQA_ERR_BLOCK_ID);
        return -1;
    }
    const uint32_t b = i / p.T, t = i - b * p.T;
    const int ctx = __ldg(p.context_lens + b);
    if (ctx < (int)p.T || ctx > p.max_blocks * 16) {
        if (reporter) report(p.status, GQA_ERR_CONTEXT);
        return -1;
    }
    const int pos = ctx - (int)p.T + (int)t;
    const int blk = __ldg(p.block_tables + (size_t)b * p.max_blocks + (pos >> 4));
    if (blk < 0 || blk >= p.num_blocks) {
        if (reporter) report(p.status, GQA_ERR_BLOCK_ID);
        return -1;
    }
    return blk * 16 + (pos & 15);
}

// Row, KV head and part of item it, H/8 parts a row.
template <int H>
__device__ __forceinline__ void item_of(const SlotParams& p, uint32_t it, uint32_t* row,
                                        uint32_t* k, uint32_t* c) {
    const uint32_t rk = it / (H / 8);
    *c = it % (H / 8);
    *row = (__umulhi(rk, p.kmul) + rk) >> p.kshift;
    *k = rk - *row * p.K;
}

// Largest magnitude of a group, of which a thread has two quarters; a NaN element
// becomes zero.  Magnitudes of 16-bit floats compare as integers, two at a time.
template <bool BF16>
__device__ __forceinline__ float group_max(uint4 (&w)[2]) {
    constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
    auto four = [&](const uint4& v) {
        return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                        __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    };
    auto top = [&]() {
        const uint32_t m = __vmaxu2(four(w[0]), four(w[1]));
        return max(m & 0xffffu, m >> 16);
    };
    uint32_t m = top();
    if (m > kInf) {  // rare: drop the NaN elements
        auto clean = [&](uint32_t x) {
            if ((x & 0x7fffu) > kInf) x &= 0xffff0000u;
            if ((x >> 16 & 0x7fffu) > kInf) x &= 0x0000ffffu;
            return x;
        };
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[j] = make_uint4(clean(w[j].x), clean(w[j].y), clean(w[j].z), clean(w[j].w));
        m = top();
    }
    return Elt<BF16>::lo(max(m, __shfl_xor_sync(0xffffffffu, m, 1)));
}

// A thread's 16-byte pieces of a row.  At 4 bits two: what a group costs once
// (maximum, scale, addresses) is then shared by 16 elements (24 prompts of 200 to
// 3,001 tokens, 8 heads of 128: 42 us with one piece, 30 with two).
template <int KIND>
constexpr int kPieces = KIND == kKvFourbit ? 2 : 1;

// The elements of part c of a row of KV head k into slot s.
template <bool BF16, int KIND, int H>
__device__ __forceinline__ void put(const SlotParams& p, uint8_t* cache, void* scale, int s, int k,
                                    int c, uint4 (&w)[kPieces<KIND>]) {
    constexpr int P = H / 8 / kPieces<KIND>;  // threads per row
    const size_t blk = (size_t)(s >> 4);
    const int row = s & 15;
    if constexpr (KIND == GQA_KV_SAME) {
        if (s >= 0)
            reinterpret_cast<uint4*>(cache)[((blk * 16 + row) * p.K + k) * P + c] = w[0];
        return;
    }
    float x[8];
    if constexpr (KIND == kKvFourbit) {
        const uint32_t sc = q4_scale_code(group_max<BF16>(w));
        const float r = q4_scale_inverse(q4_scale_value(sc));
        uint2 word;
        if (__any_sync(0xffffffffu, q4_scale_clips(sc))) {
            widen8<BF16>(w[0], x);
            word.x = q4_word<true>(x, r);
            widen8<BF16>(w[1], x);
            word.y = q4_word<true>(x, r);
        } else {
            widen8<BF16>(w[0], x);
            word.x = q4_word<false>(x, r);
            widen8<BF16>(w[1], x);
            word.y = q4_word<false>(x, r);
        }
        if (s >= 0) {
            const size_t r = (blk * p.K + k) * 16 + row;
            reinterpret_cast<uint2*>(cache)[r * P + c] = word;
            if ((c & 1) == 0)
                static_cast<uint8_t*>(scale)[r * (H / kQ4Group) + (c >> 1)] = (uint8_t)sc;
        }
    } else {
        widen8<BF16>(w[0], x);
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
        a = max_over<P>(a);
        const float sv = __fdiv_rn(a, KIND == GQA_KV_INT8 ? 127.f : 448.f);
        uint32_t word[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t code = 0;
            if (sv != 0.f) {
                const float y = __fdiv_rn(x[e], sv);
                if (KIND == GQA_KV_INT8) {
                    int r = (y != y) ? 0 : __float2int_rn(y);
                    code = (uint32_t)(min(127, max(-128, r)) & 0xff);
                } else {
                    code = (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
                }
            }
            word[e >> 2] |= code << (8 * (e & 3));
        }
        if (s >= 0) {
            reinterpret_cast<uint2*>(cache)[((blk * 16 + row) * p.K + k) * P + c] =
                make_uint2(word[0], word[1]);
            if (c == 0) static_cast<float*>(scale)[(blk * p.K + k) * 16 + row] = sv;
        }
    }
}

// Items: row i, KV head k, part c, keys and values of one item together.
template <bool BF16, int KIND, int H>
__global__ void __launch_bounds__(kSlotThreads) kv_put_kernel(const SlotParams p) {
    constexpr int V = kPieces<KIND>;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t items = p.rows * p.K * (H / 8 / V), stride = gridDim.x * kSlotThreads;
    // whole warps stay in the loop together (the shuffles); it < 2^31 + 2^24
    for (uint32_t it = blockIdx.x * kSlotThreads + threadIdx.x; it - (threadIdx.x & 31) < items;
         it += stride) {
        const bool on = it < items;
        uint32_t i, k, c;
        item_of<H / V>(p, on ? it : items - 1, &i, &k, &c);
        uint4 kw[V], vw[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            kw[j] = vw[j] = make_uint4(0, 0, 0, 0);
            if (on) {
                kw[j] = __ldg(p.k_new + (size_t)it * V + j);
                vw[j] = __ldg(p.v_new + (size_t)it * V + j);
            }
        }
        const int s = on ? slot_of(p, i, c == 0 && k == 0) : -1;
        put<BF16, KIND, H>(p, p.k_cache, p.k_scale, s, k, c, kw);
        put<BF16, KIND, H>(p, p.v_cache, p.v_scale, s, k, c, vw);
    }
}

// Eight 4-bit values as 16-bit numbers, exactly: a nibble n = c + 8 or-ed under an
// exponent is 1024 + n (f16) or 128 + n (bf16); minus the offset, times the scale.
template <bool BF16>
__device__ __forceinline__ uint4 expand8(uint32_t w, uint32_t sc) {
    uint32_t v[4];  // nibbles i and i + 4
    if constexpr (BF16) {
        const uint32_t sb = __float_as_uint(q4_scale_value(sc)) >> 16;  // 4 bits: exact
        const uint32_t s2 = sb | sb << 16, off = 0x43084308u;           // 128 + 8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t t = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
            const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                                     *reinterpret_cast<const __nv_bfloat162*>(&off)),
                                             *reinterpret_cast<const __nv_bfloat162*>(&s2));
            v[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
    } else {
        const uint32_t s2 = sc * 0x00800080u, off = 0x64086408u;  // 1024 + 8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t t = ((w >> (4 * i)) & 0x000f000fu) | 0x64006400u;
            const __half2 y = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&t),
                                              *reinterpret_cast<const __half2*>(&off)),
                                      *reinterpret_cast<const __half2*>(&s2));
            v[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
    }
    return make_uint4(prmt(v[0], v[1], 0x5410u), prmt(v[2], v[3], 0x5410u),
                      prmt(v[0], v[1], 0x7632u), prmt(v[2], v[3], 0x7632u));
}

// Eight elements of KV head k's row in slot s, in the 16-bit type.
template <bool BF16, int KIND, int H>
__device__ __forceinline__ uint4 take8(const SlotParams& p, const uint8_t* cache,
                                       const void* scale, int s, int k, int c) {
    constexpr int P = H / 8;
    if (s < 0) return make_uint4(0, 0, 0, 0);
    const size_t blk = (size_t)(s >> 4);
    const int row = s & 15;
    if constexpr (KIND == GQA_KV_SAME) {
        return __ldg(reinterpret_cast<const uint4*>(cache) + ((blk * 16 + row) * p.K + k) * P + c);
    } else if constexpr (KIND == kKvFourbit) {
        const size_t r = (blk * p.K + k) * 16 + row;
        return expand8<BF16>(
            __ldg(reinterpret_cast<const uint32_t*>(cache) + r * P + c),
            __ldg(static_cast<const uint8_t*>(scale) + r * (H / kQ4Group) + (c >> 2)));
    } else {
        float x[8];
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(cache) +
                              ((blk * 16 + row) * p.K + k) * P + c);
        const float sv = __ldg(static_cast<const float*>(scale) + (blk * p.K + k) * 16 + row);
        const uint32_t a[2] = {w.x, w.y};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t code = (a[e >> 2] >> (8 * (e & 3))) & 0xffu;
            if (KIND == GQA_KV_INT8)
                x[e] = (float)(int8_t)code * sv;
            else
                x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code,
                                                                  __NV_E4M3))) * sv;
        }
        return make_uint4(Elt<BF16>::pack(x[0], x[1]), Elt<BF16>::pack(x[2], x[3]),
                          Elt<BF16>::pack(x[4], x[5]), Elt<BF16>::pack(x[6], x[7]));
    }
}

template <bool BF16, int KIND, int H>
__global__ void __launch_bounds__(kSlotThreads) kv_take_kernel(const SlotParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t items = p.rows * p.K * (H / 8);
    for (uint32_t it = blockIdx.x * kSlotThreads + threadIdx.x; it < items;
         it += gridDim.x * kSlotThreads) {
        uint32_t i, k, c;
        item_of<H>(p, it, &i, &k, &c);
        const int s = slot_of(p, i, c == 0 && k == 0);
        const uint4 kw = take8<BF16, KIND, H>(p, p.k_cache, p.k_scale, s, k, c);
        const uint4 vw = take8<BF16, KIND, H>(p, p.v_cache, p.v_scale, s, k, c);
        p.k_out[it] = kw;
        p.v_out[it] = vw;
    }
}

template <bool PUT, bool BF16, int KIND, int H>
const void* slot_kernel() {
    return PUT ? reinterpret_cast<const void*>(&kv_put_kernel<BF16, KIND, H>)
               : reinterpret_cast<const void*>(&kv_take_kernel<BF16, KIND, H>);
}
template <bool PUT, bool BF16, int H>
const void* slot_kernel_kind(int kind) {
    switch (kind) {
        case GQA_KV_SAME: return slot_kernel<PUT, BF16, GQA_KV_SAME, H>();
        case GQA_KV_INT8: return slot_kernel<PUT, BF16, GQA_KV_INT8, H>();
        case GQA_KV_E4M3: return slot_kernel<PUT, BF16, GQA_KV_E4M3, H>();
        default: return slot_kernel<PUT, BF16, kKvFourbit, H>();
    }
}
template <bool PUT>
const void* pick_slot_kernel(const gqa_shape& s) {
    const bool bf16 = s.dtype == GQA_BF16;
    if (s.H == 128)
        return bf16 ? slot_kernel_kind<PUT, true, 128>(s.kv_dtype)
                    : slot_kernel_kind<PUT, false, 128>(s.kv_dtype);
    return bf16 ? slot_kernel_kind<PUT, true, 64>(s.kv_dtype)
                : slot_kernel_kind<PUT, false, 64>(s.kv_dtype);
}

// `rows` rows from `p`, in launches of fewer than 2^31 items.
gqa_status launch_slots(const gqa_shape& s, const void* kernel, SlotParams p, long long rows,
                        cudaStream_t stream) {
    const long long per_row = (long long)s.K * (s.H / 8);
    if (rows == 0) return GQA_OK;
    const int sms = device_sm_count();
    if (sms <= 0) return GQA_ERR_CUDA;
    p.T = (uint32_t)s.T;
    p.K = (uint32_t)s.K;
    p.max_blocks = s.max_blocks_per_seq;
    p.num_blocks = s.num_blocks;
    while ((1ll << p.kshift) < s.K) ++p.kshift;
    p.kmul = (uint32_t)(((1ull << 32) * ((1ull << p.kshift) - (uint64_t)s.K)) / (uint64_t)s.K + 1);
    if (per_row >= (1ll << 31)) return GQA_ERR_SHAPE;
    long long most = ((1ll << 31) - 1) / per_row;
    if (!p.slots) most = most / s.T * s.T;  // whole sequences
    if (most < 1) return GQA_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kSlotThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (s.flags & (GQA_FLAG_PDL | GQA_FLAG_EARLY_KV)) ? 1 : 0;
    while (rows > 0) {
        const long long n = rows < most ? rows : most, items = n * per_row;
        const long long need = (items + kSlotThreads - 1) / kSlotThreads, cap = (long long)sms * 32;
        p.rows = (uint32_t)n;
        cfg.gridDim = dim3((unsigned)(need < cap ? need : cap));
        void* args[] = {&p};
        const gqa_status st = launch_status(cudaLaunchKernelExC(&cfg, kernel, args));
        if (st != GQA_OK) return st;
        rows -= n;
        if (p.k_new) {
            p.k_new += items;
            p.v_new += items;
        } else {
            p.k_out += items;
            p.v_out += items;
        }
        if (p.slots) {
            p.slots += n;
        } else {
            p.block_tables += n / s.T * s.max_blocks_per_seq;
            p.context_lens += n / s.T;
        }
    }
    return GQA_OK;
}

}  // namespace

gqa_status launch_kv_append_slots(const gqa_shape& s, long long rows, const void* k_new,
                                  const void* v_new, void* k_cache, void* v_cache, void* k_scale,
                                  void* v_scale, const int32_t* slots,
                                  const int32_t* block_tables, const int32_t* context_lens,
                                  int32_t* dev_status, cudaStream_t stream) {
    SlotParams p = {};
    p.k_new = static_cast<const uint4*>(k_new);
    p.v_new = static_cast<const uint4*>(v_new);
    p.k_cache = static_cast<uint8_t*>(k_cache);
    p.v_cache = static_cast<uint8_t*>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.slots = slots;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.status = dev_status;
    return launch_slots(s, pick_slot_kernel<true>(s), p, rows, stream);
}

gqa_status launch_kv_gather_slots(const gqa_shape& s, long long rows, const void* k_cache,
                                  const void* v_cache, const void* k_scale, const void* v_scale,
                                  const int32_t* slots, void* k_out, void* v_out,
                                  int32_t* dev_status, cudaStream_t stream) {
    SlotParams p = {};
    p.k_out = static_cast<uint4*>(k_out);
    p.v_out = static_cast<uint4*>(v_out);
    p.k_cache = static_cast<uint8_t*>(const_cast<void*>(k_cache));
    p.v_cache = static_cast<uint8_t*>(const_cast<void*>(v_cache));
    p.k_scale = const_cast<void*>(k_scale);
    p.v_scale = const_cast<void*>(v_scale);
    p.slots = slots;
    p.status = dev_status;
    return launch_slots(s, pick_slot_kernel<false>(s), p, rows, stream);
}

}  // namespace gqa
