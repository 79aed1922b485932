// api.cu -- the extern "C" entry points declared in include/gqa_decode.h:
// host-side argument validation, then one launch per operation.
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gqa_status check_common(const gqa_shape* s) {
    if (!s) return GQA_ERR_NULL;
    if (s->dtype != GQA_F16 && s->dtype != GQA_BF16) return GQA_ERR_DTYPE;
    if (s->B < 0 || s->T < 1 || s->N < 1 || s->K < 1 || s->N % s->K != 0) return GQA_ERR_SHAPE;
    if (s->H != 64 && s->H != 128) return GQA_ERR_SHAPE;
    if (s->block_size != 16 || s->num_blocks < 1 || s->max_blocks_per_seq < 1)
        return GQA_ERR_SHAPE;
    if ((long long)s->num_blocks * 16 > (1ll << 31) - 1) return GQA_ERR_SHAPE;
    if ((long long)s->max_blocks_per_seq * 16 > (1ll << 30)) return GQA_ERR_SHAPE;
    if ((long long)s->B * s->K * s->max_blocks_per_seq > (1ll << 31) - 1) return GQA_ERR_SHAPE;
    if (s->window < 0) return GQA_ERR_SHAPE;
    if (s->kv_dtype < GQA_KV_SAME || s->kv_dtype > GQA_KV_E4M3) return GQA_ERR_DTYPE;
    return GQA_OK;
}

// The shape of a 4-bit call: the common checks on everything but kv_dtype.
gqa_status check_fourbit(const gqa_shape* s) {
    if (!s) return GQA_ERR_NULL;
    if (s->kv_dtype != GQA_KV_INT4) return GQA_ERR_DTYPE;
    gqa_shape sh = *s;
    sh.kv_dtype = GQA_KV_SAME;
    const gqa_status st = check_common(&sh);
    if (st != GQA_OK) return st;
    // the other kernels do not serve it
    if (s->flags & (GQA_FLAG_WARP_MMA | GQA_FLAG_TENSOR_MEMORY | GQA_FLAG_DIRECT))
        return GQA_ERR_SHAPE;
    return GQA_OK;
}

gqa_status attention_fourbit_entry(const gqa_shape* s, bool fused, const void* q,
                                   const void* k_new, const void* v_new, const uint8_t* k_cache,
                                   const uint8_t* v_cache, const uint8_t* k_scale,
                                   const uint8_t* v_scale, const int32_t* block_tables,
                                   const int32_t* context_lens, const uint64_t* tree_mask,
                                   void* out, void* workspace, size_t ws_bytes,
                                   int32_t* dev_status, void* stream) {
    gqa_status st = check_fourbit(s);
    if (st != GQA_OK) return st;
    if (tree_mask && (s->window > 0 || s->T > 64)) return GQA_ERR_SHAPE;
    if (s->B == 0) return GQA_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens ||
        !out || (fused && (!k_new || !v_new)))
        return GQA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) ||
        !aligned16(v_scale) || !aligned16(out) || (fused && (!aligned16(k_new) || !aligned16(v_new))))
        return GQA_ERR_ALIGN;
    if (tree_mask && (reinterpret_cast<uintptr_t>(tree_mask) & 7u) != 0) return GQA_ERR_ALIGN;
    if (!workspace) return GQA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQA_ERR_ALIGN;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (fused) {
        size_t need = 0;  // nothing is appended by a call that then refuses
        st = gqa::fourbit_workspace_bytes(*s, &need);
        if (st != GQA_OK) return st;
        if (ws_bytes < need) return GQA_ERR_WORKSPACE;
        st = gqa::launch_kv_append_slots(
            *s, (long long)s->B * s->T, k_new, v_new, const_cast<uint8_t*>(k_cache),
            const_cast<uint8_t*>(v_cache), const_cast<uint8_t*>(k_scale),
            const_cast<uint8_t*>(v_scale), nullptr, block_tables, context_lens, dev_status, cs);
        if (st != GQA_OK) return st;
    }
    return gqa::launch_attention_fourbit(*s, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                         context_lens, tree_mask, out, workspace, ws_bytes,
                                         dev_status, cs);
}

// Arguments of the calls that move rows by slot.
gqa_status check_slots(const gqa_shape* s, long long rows, const void* k, const void* v,
                       const void* k_cache, const void* v_cache, const void* k_scale,
                       const void* v_scale, const int32_t* slots) {
    if (!s) return GQA_ERR_NULL;
    gqa_shape sh = *s;
    if (sh.kv_dtype == GQA_KV_INT4) sh.kv_dtype = GQA_KV_SAME;
    const gqa_status st = check_common(&sh);
    if (st != GQA_OK) return st;
    if (rows < 0 || rows > (1ll << 31) - 1) return GQA_ERR_SHAPE;
    const bool scaled = s->kv_dtype != GQA_KV_SAME;
    if (!scaled && (k_scale || v_scale)) return GQA_ERR_DTYPE;  // the rows carry no scales
    if (rows == 0) return GQA_OK;
    if (!k || !v || !k_cache || !v_cache || !slots || (scaled && (!k_scale || !v_scale)))
        return GQA_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(k_scale) || !aligned16(v_scale))
        return GQA_ERR_ALIGN;
    return GQA_OK;
}

gqa_status attention_entry(const gqa_shape* s, bool decode_only, bool fused, const void* q,
                           const void* k_new, const void* v_new, const void* k_cache,
                           const void* v_cache, const int32_t* block_tables,
                           const int32_t* context_lens, const uint64_t* tree_mask, void* out,
                           void* workspace, size_t ws_bytes, int32_t* dev_status,
                           void* stream, const float* k_scale = nullptr,
                           const float* v_scale = nullptr) {
    gqa_status st = check_common(s);
    if (st != GQA_OK) return st;
    if (decode_only && s->T != 1) return GQA_ERR_SHAPE;
    // one-byte caches come with their row scales (the _quant calls), others without
    if ((s->kv_dtype != GQA_KV_SAME) != (k_scale != nullptr)) return GQA_ERR_DTYPE;
    if (k_scale && !v_scale) return GQA_ERR_NULL;
    if (k_scale && (!aligned16(k_scale) || !aligned16(v_scale))) return GQA_ERR_ALIGN;
    if (s->B == 0) return GQA_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
        return GQA_ERR_NULL;
    if (fused && (!k_new || !v_new)) return GQA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return GQA_ERR_ALIGN;
    if (fused && (!aligned16(k_new) || !aligned16(v_new))) return GQA_ERR_ALIGN;
    if (tree_mask && s->window > 0) return GQA_ERR_SHAPE;  // not combined
    if (tree_mask && s->T > 64) return GQA_ERR_SHAPE;      // one 64-bit row per new token
    if (tree_mask && (reinterpret_cast<uintptr_t>(tree_mask) & 7u) != 0) return GQA_ERR_ALIGN;
    const bool force_warp = (s->flags & GQA_FLAG_WARP_MMA) != 0;
    const bool force_tc = (s->flags & GQA_FLAG_TENSOR_MEMORY) != 0;
    const bool force_direct = (s->flags & GQA_FLAG_DIRECT) != 0;
    if ((int)force_warp + (int)force_tc + (int)force_direct > 1) return GQA_ERR_SHAPE;
    if (force_tc && !gqa::tc_attention_supported(*s)) return GQA_ERR_SHAPE;
    gqa::AttnPlan plan;
    st = gqa::attention_plan(*s, tree_mask != nullptr, &plan);
    if (st != GQA_OK) return st;
    if (!workspace || ws_bytes < plan.workspace) return GQA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQA_ERR_ALIGN;
    if (force_tc || (!force_warp && !force_direct && gqa::tc_attention_preferred(*s))) {
        if (ws_bytes < gqa::tc_workspace_bytes(*s, plan.flags_bytes)) return GQA_ERR_WORKSPACE;
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        if (fused) {
            st = gqa::launch_kv_append(*s, k_new, v_new, const_cast<void*>(k_cache),
                                       const_cast<void*>(v_cache), block_tables, context_lens,
                                       dev_status, cs);
            if (st != GQA_OK) return st;
        }
        return gqa::launch_tc_attention(*s, q, k_cache, v_cache, block_tables, context_lens,
                                        tree_mask, out, workspace, plan.flags_bytes, dev_status,
                                        cs);
    }
    if (fused && k_scale) {
        // One-byte cache: the append is a launch of its own just before the
        // attention launch.  (Both one-launch forms measured slower on the
        // 256-sequence int8 batch, whose attention kernel is bound by its
        // producer warp's issue rate and its consumers' registers: the rows
        // quantized by the consumers 467 us, by the producer 417 us, against
        // 360 + 9 us for the two launches.)
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        st = gqa::launch_kv_append_quant(*s, k_new, v_new, const_cast<void*>(k_cache),
                                         const_cast<void*>(v_cache),
                                         const_cast<float*>(k_scale),
                                         const_cast<float*>(v_scale), block_tables,
                                         context_lens, dev_status, cs);
        if (st != GQA_OK) return st;
        return gqa::launch_attention(*s, plan, q, nullptr, nullptr, k_cache, v_cache,
                                     block_tables, context_lens, tree_mask, k_scale, v_scale,
                                     out, workspace, dev_status, cs);
    }
    return gqa::launch_attention(*s, plan, q, fused ? k_new : nullptr, fused ? v_new : nullptr,
                                 k_cache, v_cache, block_tables, context_lens, tree_mask,
                                 k_scale, v_scale, out, workspace, dev_status,
                                 static_cast<cudaStream_t>(stream));
}

// Shape of a call over a cache in q's dtype whose kernel is not a matter of flags.
gqa_status check_plain(const gqa_shape* s) {
    const gqa_status st = check_common(s);
    if (st != GQA_OK) return st;
    if (s->kv_dtype != GQA_KV_SAME) return GQA_ERR_DTYPE;
    if (s->flags & (GQA_FLAG_WARP_MMA | GQA_FLAG_TENSOR_MEMORY | GQA_FLAG_DIRECT))
        return GQA_ERR_SHAPE;
    return s->N / s->K <= 8192 && s->B <= 16384 ? GQA_OK : GQA_ERR_SHAPE;
}

gqa_status chunk_entry(const gqa_shape* s, int64_t rows, int64_t q_stride, const void* q,
                       const void* k_cache, const void* v_cache, const int32_t* block_tables,
                       bool head_tables, const int32_t* context_lens, const int32_t* cu_new,
                       void* out, void* workspace, size_t ws_bytes, int32_t* dev_status,
                       void* stream) {
    const gqa_status st = check_plain(s);
    if (st != GQA_OK) return st;
    if (rows < 0 || rows > (1ll << 31) - 1) return GQA_ERR_SHAPE;
    const long long row = (long long)s->N * s->H;
    // (the tensor map's strides; a row tile's outputs within 32 bits of 16-byte pieces)
    if (row > (1ll << 27) || q_stride < row || q_stride % 8 != 0 || q_stride >= (1ll << 39))
        return GQA_ERR_SHAPE;
    if (s->B == 0 || rows == 0) return GQA_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out ||
        (!head_tables && !cu_new))
        return GQA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return GQA_ERR_ALIGN;
    const size_t flags = gqa::workspace_flags_bytes();
    const size_t need = gqa::chunk_workspace_bytes(*s, flags);
    if (need == 0) return GQA_ERR_CUDA;
    if (!workspace || ws_bytes < need) return GQA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQA_ERR_ALIGN;
    return gqa::launch_chunk_attention(*s, rows, q_stride, q, k_cache, v_cache, block_tables,
                                       head_tables, context_lens, cu_new, out, workspace, flags,
                                       dev_status, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int gqa_version(void) { return 400; }

const char* gqa_status_string(int status) {
    switch (status) {
        case GQA_OK: return "ok";
        case GQA_ERR_NULL: return "a required pointer is NULL";
        case GQA_ERR_SHAPE: return "unsupported or inconsistent sizes";
        case GQA_ERR_DTYPE: return "unsupported dtype";
        case GQA_ERR_ALIGN: return "pointer not 16-byte aligned";
        case GQA_ERR_WORKSPACE: return "workspace missing or too small";
        case GQA_ERR_CUDA: return "CUDA call failed";
        case GQA_ERR_CONTEXT: return "context length out of range";
        case GQA_ERR_BLOCK_ID: return "block id out of range";
        case GQA_ERR_TIMEOUT: return "bounded wait inside a kernel timed out";
        case GQA_ERR_PROBS: return "invalid probability, uniform or empty distribution";
        case GQA_ERR_TREE: return "draft tree parent or accepted path out of range";
        case GQA_ERR_BLOCKS: return "no free blocks or token slots left, or an inconsistent free ring";
        default: return "unknown status";
    }
}

gqa_status gqa_kv_append(const gqa_shape* shape, const void* k_new, const void* v_new,
                         void* k_cache, void* v_cache, const int32_t* block_tables,
                         const int32_t* context_lens, int32_t* dev_status, void* stream) {
    gqa_status st = check_common(shape);
    if (st != GQA_OK) return st;
    if (shape->kv_dtype != GQA_KV_SAME) return GQA_ERR_DTYPE;  // use gqa_kv_append_quant
    if (shape->B == 0) return GQA_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !block_tables || !context_lens)
        return GQA_ERR_NULL;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache))
        return GQA_ERR_ALIGN;
    return gqa::launch_kv_append(*shape, k_new, v_new, k_cache, v_cache, block_tables,
                                 context_lens, dev_status, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_kv_append_quant(const gqa_shape* shape, const void* k_new, const void* v_new,
                               void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                               const int32_t* block_tables, const int32_t* context_lens,
                               int32_t* dev_status, void* stream) {
    gqa_status st = check_common(shape);
    if (st != GQA_OK) return st;
    if (shape->kv_dtype != GQA_KV_INT8 && shape->kv_dtype != GQA_KV_E4M3) return GQA_ERR_DTYPE;
    if (shape->B == 0) return GQA_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables ||
        !context_lens)
        return GQA_ERR_NULL;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(k_scale) || !aligned16(v_scale))
        return GQA_ERR_ALIGN;
    return gqa::launch_kv_append_quant(*shape, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                       block_tables, context_lens, dev_status,
                                       static_cast<cudaStream_t>(stream));
}

int gqa_attention_engine(const gqa_shape* shape) {
    if (shape && shape->kv_dtype == GQA_KV_INT4)
        return check_fourbit(shape) == GQA_OK ? GQA_ENGINE_FOURBIT : 0;
    if (check_common(shape) != GQA_OK) return 0;
    const bool force_warp = (shape->flags & GQA_FLAG_WARP_MMA) != 0;
    const bool force_tc = (shape->flags & GQA_FLAG_TENSOR_MEMORY) != 0;
    const bool force_direct = (shape->flags & GQA_FLAG_DIRECT) != 0;
    if ((int)force_warp + (int)force_tc + (int)force_direct > 1) return 0;
    if (force_tc) return gqa::tc_attention_supported(*shape) ? GQA_ENGINE_TENSOR_MEMORY : 0;
    if (force_direct) return gqa::direct_attention_supported(*shape, false) ? GQA_ENGINE_DIRECT : 0;
    if (force_warp) return GQA_ENGINE_WARP_MMA;
    if (gqa::tc_attention_preferred(*shape)) return GQA_ENGINE_TENSOR_MEMORY;
    return gqa::direct_attention_preferred(*shape, false) ? GQA_ENGINE_DIRECT
                                                          : GQA_ENGINE_WARP_MMA;
}

size_t gqa_attention_workspace_size(const gqa_shape* shape) {
    if (shape && shape->kv_dtype == GQA_KV_INT4) {
        size_t need = 0;
        if (check_fourbit(shape) != GQA_OK) return 0;
        return gqa::fourbit_workspace_bytes(*shape, &need) == GQA_OK ? need : 0;
    }
    if (check_common(shape) != GQA_OK) return 0;
    // the largest need of the kernels that may serve the shape (the direct
    // kernel uses none, so its flag does not change the size)
    gqa_shape sh = *shape;
    sh.flags &= ~GQA_FLAG_DIRECT;
    gqa::AttnPlan plain, general;
    if (gqa::attention_plan(sh, false, &plain) != GQA_OK) return 0;
    if (gqa::attention_plan(sh, true, &general) != GQA_OK) return 0;
    size_t w = plain.workspace > general.workspace ? plain.workspace : general.workspace;
    const size_t tc = gqa::tc_workspace_bytes(*shape, plain.flags_bytes);  // 0: not served
    return tc > w ? tc : w;
}

gqa_status gqa_workspace_clear(void* workspace, size_t bytes, void* stream) {
    if (bytes == 0) return GQA_OK;
    if (!workspace) return GQA_ERR_NULL;
    return cudaMemsetAsync(workspace, 0, bytes, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GQA_OK
               : GQA_ERR_CUDA;
}

gqa_status gqa_decode_attention(const gqa_shape* shape, const void* q, const void* k_cache,
                                const void* v_cache, const int32_t* block_tables,
                                const int32_t* context_lens, void* out, void* workspace,
                                size_t workspace_bytes, int32_t* dev_status, void* stream) {
    return attention_entry(shape, true, false, q, nullptr, nullptr, k_cache, v_cache,
                           block_tables, context_lens, nullptr, out, workspace,
                           workspace_bytes, dev_status, stream);
}

gqa_status gqa_verify_attention(const gqa_shape* shape, const void* q, const void* k_cache,
                                const void* v_cache, const int32_t* block_tables,
                                const int32_t* context_lens, void* out, void* workspace,
                                size_t workspace_bytes, int32_t* dev_status, void* stream) {
    return attention_entry(shape, false, false, q, nullptr, nullptr, k_cache, v_cache,
                           block_tables, context_lens, nullptr, out, workspace,
                           workspace_bytes, dev_status, stream);
}

gqa_status gqa_append_decode_attention(const gqa_shape* shape, const void* q,
                                       const void* k_new, const void* v_new, void* k_cache,
                                       void* v_cache, const int32_t* block_tables,
                                       const int32_t* context_lens, void* out, void* workspace,
                                       size_t workspace_bytes, int32_t* dev_status,
                                       void* stream) {
    return attention_entry(shape, true, true, q, k_new, v_new, k_cache, v_cache, block_tables,
                           context_lens, nullptr, out, workspace, workspace_bytes, dev_status,
                           stream);
}

gqa_status gqa_append_verify_attention(const gqa_shape* shape, const void* q,
                                       const void* k_new, const void* v_new, void* k_cache,
                                       void* v_cache, const int32_t* block_tables,
                                       const int32_t* context_lens, void* out, void* workspace,
                                       size_t workspace_bytes, int32_t* dev_status,
                                       void* stream) {
    return attention_entry(shape, false, true, q, k_new, v_new, k_cache, v_cache, block_tables,
                           context_lens, nullptr, out, workspace, workspace_bytes, dev_status,
                           stream);
}

gqa_status gqa_tree_verify_attention(const gqa_shape* shape, const void* q,
                                     const void* k_cache, const void* v_cache,
                                     const int32_t* block_tables, const int32_t* context_lens,
                                     const uint64_t* tree_mask, void* out, void* workspace,
                                     size_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (!tree_mask) return GQA_ERR_NULL;
    return attention_entry(shape, false, false, q, nullptr, nullptr, k_cache, v_cache,
                           block_tables, context_lens, tree_mask, out, workspace,
                           workspace_bytes, dev_status, stream);
}

gqa_status gqa_append_tree_verify_attention(const gqa_shape* shape, const void* q,
                                            const void* k_new, const void* v_new,
                                            void* k_cache, void* v_cache,
                                            const int32_t* block_tables,
                                            const int32_t* context_lens,
                                            const uint64_t* tree_mask, void* out,
                                            void* workspace, size_t workspace_bytes,
                                            int32_t* dev_status, void* stream) {
    if (!tree_mask) return GQA_ERR_NULL;
    return attention_entry(shape, false, true, q, k_new, v_new, k_cache, v_cache, block_tables,
                           context_lens, tree_mask, out, workspace, workspace_bytes, dev_status,
                           stream);
}

gqa_status gqa_decode_attention_quant(const gqa_shape* shape, const void* q,
                                      const void* k_cache, const void* v_cache,
                                      const float* k_scale, const float* v_scale,
                                      const int32_t* block_tables,
                                      const int32_t* context_lens, void* out, void* workspace,
                                      size_t workspace_bytes, int32_t* dev_status,
                                      void* stream) {
    if (!k_scale || !v_scale) return GQA_ERR_NULL;
    return attention_entry(shape, true, false, q, nullptr, nullptr, k_cache, v_cache,
                           block_tables, context_lens, nullptr, out, workspace,
                           workspace_bytes, dev_status, stream, k_scale, v_scale);
}

gqa_status gqa_verify_attention_quant(const gqa_shape* shape, const void* q,
                                      const void* k_cache, const void* v_cache,
                                      const float* k_scale, const float* v_scale,
                                      const int32_t* block_tables,
                                      const int32_t* context_lens, void* out, void* workspace,
                                      size_t workspace_bytes, int32_t* dev_status,
                                      void* stream) {
    if (!k_scale || !v_scale) return GQA_ERR_NULL;
    return attention_entry(shape, false, false, q, nullptr, nullptr, k_cache, v_cache,
                           block_tables, context_lens, nullptr, out, workspace,
                           workspace_bytes, dev_status, stream, k_scale, v_scale);
}

gqa_status gqa_tree_verify_attention_quant(const gqa_shape* shape, const void* q,
                                          const void* k_cache, const void* v_cache,
                                          const float* k_scale, const float* v_scale,
                                          const int32_t* block_tables,
                                          const int32_t* context_lens,
                                          const uint64_t* tree_mask, void* out, void* workspace,
                                          size_t workspace_bytes, int32_t* dev_status,
                                          void* stream) {
    if (!k_scale || !v_scale || !tree_mask) return GQA_ERR_NULL;
    return attention_entry(shape, false, false, q, nullptr, nullptr, k_cache, v_cache,
                           block_tables, context_lens, tree_mask, out, workspace,
                           workspace_bytes, dev_status, stream, k_scale, v_scale);
}

gqa_status gqa_append_decode_attention_quant(const gqa_shape* shape, const void* q,
                                             const void* k_new, const void* v_new,
                                             void* k_cache, void* v_cache, float* k_scale,
                                             float* v_scale, const int32_t* block_tables,
                                             const int32_t* context_lens, void* out,
                                             void* workspace, size_t workspace_bytes,
                                             int32_t* dev_status, void* stream) {
    if (!k_scale || !v_scale) return GQA_ERR_NULL;
    return attention_entry(shape, true, true, q, k_new, v_new, k_cache, v_cache, block_tables,
                           context_lens, nullptr, out, workspace, workspace_bytes, dev_status,
                           stream, k_scale, v_scale);
}

gqa_status gqa_append_verify_attention_quant(const gqa_shape* shape, const void* q,
                                             const void* k_new, const void* v_new,
                                             void* k_cache, void* v_cache, float* k_scale,
                                             float* v_scale, const int32_t* block_tables,
                                             const int32_t* context_lens, void* out,
                                             void* workspace, size_t workspace_bytes,
                                             int32_t* dev_status, void* stream) {
    if (!k_scale || !v_scale) return GQA_ERR_NULL;
    return attention_entry(shape, false, true, q, k_new, v_new, k_cache, v_cache, block_tables,
                           context_lens, nullptr, out, workspace, workspace_bytes, dev_status,
                           stream, k_scale, v_scale);
}

size_t gqa_accept_workspace_size(int B, int T) { return gqa::accept_workspace_bytes(B, T); }

gqa_status gqa_accept_prefix(int B, int T, int V, const float* target_logits,
                             const int32_t* draft_ids, int32_t* accepted, int32_t* next_token,
                             int32_t* context_lens_inout, void* workspace,
                             size_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (B < 0 || T < 1 || T > 64 || V < 1) return GQA_ERR_SHAPE;
    if (!workspace && B > 65535) return GQA_ERR_SHAPE;  // one cluster per sequence (grid y)
    if (B == 0) return GQA_OK;
    if (!target_logits || !accepted || !next_token || (T > 1 && !draft_ids))
        return GQA_ERR_NULL;
    if (!aligned16(target_logits)) return GQA_ERR_ALIGN;
    if ((long long)T * V > (1ll << 31) - 1) return GQA_ERR_SHAPE;
    if (workspace) {
        if (workspace_bytes < gqa::accept_workspace_bytes(B, T)) return GQA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return GQA_ERR_ALIGN;
    }
    return gqa::launch_accept_prefix(B, T, V, target_logits, draft_ids, nullptr, accepted,
                                     next_token, nullptr, context_lens_inout, workspace,
                                     dev_status, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_accept_tree(int B, int T, int V, const float* target_logits,
                           const int32_t* draft_ids, const int32_t* parents, int32_t* accepted,
                           int32_t* next_token, int32_t* path, int32_t* context_lens_inout,
                           void* workspace, size_t workspace_bytes, int32_t* dev_status,
                           void* stream) {
    if (B < 0 || T < 1 || T > 64 || V < 1) return GQA_ERR_SHAPE;
    if (!workspace && B > 65535) return GQA_ERR_SHAPE;  // one cluster per sequence (grid y)
    if (B == 0) return GQA_OK;
    if (!target_logits || !parents || !accepted || !next_token ||
        (T > 1 && (!draft_ids || !path)))
        return GQA_ERR_NULL;
    if (!aligned16(target_logits)) return GQA_ERR_ALIGN;
    if ((long long)T * V > (1ll << 31) - 1) return GQA_ERR_SHAPE;
    if (workspace) {
        if (workspace_bytes < gqa::accept_workspace_bytes(B, T)) return GQA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return GQA_ERR_ALIGN;
    }
    return gqa::launch_accept_prefix(B, T, V, target_logits, draft_ids, parents, accepted,
                                     next_token, path, context_lens_inout, workspace,
                                     dev_status, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_kv_compact(const gqa_shape* shape, void* k_cache, void* v_cache, float* k_scale,
                          float* v_scale, const int32_t* block_tables,
                          const int32_t* context_lens, const int32_t* path,
                          const int32_t* accepted, int32_t* dev_status, void* stream) {
    gqa_status st = check_common(shape);
    if (st != GQA_OK) return st;
    if (shape->T > 64) return GQA_ERR_SHAPE;
    const bool one_byte = shape->kv_dtype != GQA_KV_SAME;
    if (!one_byte && (k_scale || v_scale)) return GQA_ERR_DTYPE;  // scales: one-byte caches only
    if (one_byte && (!k_scale || !v_scale)) return GQA_ERR_NULL;
    if (shape->B == 0 || shape->T == 1) return GQA_OK;  // nothing can move
    if (!k_cache || !v_cache || !block_tables || !context_lens || !path || !accepted)
        return GQA_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return GQA_ERR_ALIGN;
    return gqa::launch_kv_compact(*shape, k_cache, v_cache, k_scale, v_scale, block_tables,
                                  context_lens, path, accepted, dev_status,
                                  static_cast<cudaStream_t>(stream));
}

gqa_status gqa_accept_sampled(int B, int T, int V, const float* target_probs,
                              const float* draft_probs, const int32_t* draft_ids,
                              const double* uniforms, int32_t* accepted, int32_t* next_token,
                              int32_t* context_lens_inout, int32_t* dev_status, void* stream) {
    if (B < 0 || T < 1 || T > 64 || V < 1 || B > (1 << 28)) return GQA_ERR_SHAPE;
    if (B == 0) return GQA_OK;
    if (!target_probs || !uniforms || !accepted || !next_token) return GQA_ERR_NULL;
    if (T > 1 && (!draft_probs || !draft_ids)) return GQA_ERR_NULL;
    return gqa::launch_accept_sampled(B, T, V, target_probs, T > 1 ? draft_probs : nullptr,
                                      T > 1 ? draft_ids : nullptr, uniforms, accepted,
                                      next_token, context_lens_inout, dev_status,
                                      static_cast<cudaStream_t>(stream));
}

gqa_status gqa_kv_append_fourbit(const gqa_shape* shape, const void* k_new, const void* v_new,
                                 uint8_t* k_cache, uint8_t* v_cache, uint8_t* k_scale,
                                 uint8_t* v_scale, const int32_t* block_tables,
                                 const int32_t* context_lens, int32_t* dev_status, void* stream) {
    const gqa_status st = check_fourbit(shape);
    if (st != GQA_OK) return st;
    if (shape->B == 0) return GQA_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables ||
        !context_lens)
        return GQA_ERR_NULL;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(k_scale) || !aligned16(v_scale))
        return GQA_ERR_ALIGN;
    return gqa::launch_kv_append_slots(*shape, (long long)shape->B * shape->T, k_new, v_new,
                                       k_cache, v_cache, k_scale, v_scale, nullptr, block_tables,
                                       context_lens, dev_status, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_attention_fourbit(const gqa_shape* shape, const void* q, const uint8_t* k_cache,
                                 const uint8_t* v_cache, const uint8_t* k_scale,
                                 const uint8_t* v_scale, const int32_t* block_tables,
                                 const int32_t* context_lens, const uint64_t* tree_mask,
                                 void* out, void* workspace, size_t workspace_bytes,
                                 int32_t* dev_status, void* stream) {
    return attention_fourbit_entry(shape, false, q, nullptr, nullptr, k_cache, v_cache, k_scale,
                                   v_scale, block_tables, context_lens, tree_mask, out,
                                   workspace, workspace_bytes, dev_status, stream);
}

gqa_status gqa_append_attention_fourbit(const gqa_shape* shape, const void* q, const void* k_new,
                                        const void* v_new, uint8_t* k_cache, uint8_t* v_cache,
                                        uint8_t* k_scale, uint8_t* v_scale,
                                        const int32_t* block_tables, const int32_t* context_lens,
                                        const uint64_t* tree_mask, void* out, void* workspace,
                                        size_t workspace_bytes, int32_t* dev_status,
                                        void* stream) {
    return attention_fourbit_entry(shape, true, q, k_new, v_new, k_cache, v_cache, k_scale,
                                   v_scale, block_tables, context_lens, tree_mask, out,
                                   workspace, workspace_bytes, dev_status, stream);
}

gqa_status gqa_kv_compact_fourbit(const gqa_shape* shape, uint8_t* k_cache, uint8_t* v_cache,
                                  uint8_t* k_scale, uint8_t* v_scale,
                                  const int32_t* block_tables, const int32_t* context_lens,
                                  const int32_t* path, const int32_t* accepted,
                                  int32_t* dev_status, void* stream) {
    const gqa_status st = check_fourbit(shape);
    if (st != GQA_OK) return st;
    if (shape->T > 64) return GQA_ERR_SHAPE;
    if (shape->B == 0 || shape->T == 1) return GQA_OK;  // nothing can move
    if (!k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens || !path ||
        !accepted)
        return GQA_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
        return GQA_ERR_ALIGN;
    return gqa::launch_kv_compact(*shape, k_cache, v_cache, k_scale, v_scale, block_tables,
                                  context_lens, path, accepted, dev_status,
                                  static_cast<cudaStream_t>(stream));
}

gqa_status gqa_kv_append_slots(const gqa_shape* shape, int64_t rows, const void* k_new,
                               const void* v_new, void* k_cache, void* v_cache, void* k_scale,
                               void* v_scale, const int32_t* slots, int32_t* dev_status,
                               void* stream) {
    const gqa_status st = check_slots(shape, rows, k_new, v_new, k_cache, v_cache, k_scale,
                                      v_scale, slots);
    if (st != GQA_OK || rows == 0) return st;
    return gqa::launch_kv_append_slots(*shape, rows, k_new, v_new, k_cache, v_cache, k_scale,
                                       v_scale, slots, nullptr, nullptr, dev_status,
                                       static_cast<cudaStream_t>(stream));
}

gqa_status gqa_kv_gather_slots(const gqa_shape* shape, int64_t rows, const void* k_cache,
                               const void* v_cache, const void* k_scale, const void* v_scale,
                               const int32_t* slots, void* k_out, void* v_out,
                               int32_t* dev_status, void* stream) {
    const gqa_status st = check_slots(shape, rows, k_out, v_out, k_cache, v_cache, k_scale,
                                      v_scale, slots);
    if (st != GQA_OK || rows == 0) return st;
    return gqa::launch_kv_gather_slots(*shape, rows, k_cache, v_cache, k_scale, v_scale, slots,
                                       k_out, v_out, dev_status,
                                       static_cast<cudaStream_t>(stream));
}

gqa_status gqa_kv_append_rotary(const gqa_shape* shape, int64_t rows, const void* q,
                                const void* k_new, const void* v_new, int64_t q_stride,
                                int64_t k_stride, int64_t v_stride, void* k_cache, void* v_cache,
                                void* k_scale, void* v_scale, const int32_t* slots,
                                const int32_t* positions, const float* cos_sin, int table_rows,
                                int rotary_dims, int interleaved, void* q_out,
                                int32_t* dev_status, void* stream) {
    const gqa_status st = check_slots(shape, rows, k_new, v_new, k_cache, v_cache, k_scale,
                                      v_scale, slots);
    if (st != GQA_OK) return st;
    if (table_rows < 1 || rotary_dims < 16 || rotary_dims > shape->H || rotary_dims % 16 != 0)
        return GQA_ERR_SHAPE;
    const long long q_row = (long long)shape->N * shape->H, k_row = (long long)shape->K * shape->H;
    if (q_stride < q_row || k_stride < k_row || v_stride < k_row || q_stride % 8 != 0 ||
        k_stride % 8 != 0 || v_stride % 8 != 0)
        return GQA_ERR_SHAPE;
    if (rows == 0) return GQA_OK;
    if (!q || !q_out || !positions || !cos_sin) return GQA_ERR_NULL;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(cos_sin)) return GQA_ERR_ALIGN;
    return gqa::launch_kv_append_rotary(*shape, rows, q, k_new, v_new, q_stride, k_stride,
                                        v_stride, k_cache, v_cache, k_scale, v_scale, slots,
                                        positions, cos_sin, table_rows, rotary_dims,
                                        interleaved != 0, q_out, dev_status,
                                        static_cast<cudaStream_t>(stream));
}

size_t gqa_chunk_workspace_size(const gqa_shape* shape) {
    return check_plain(shape) == GQA_OK
               ? gqa::chunk_workspace_bytes(*shape, gqa::workspace_flags_bytes())
               : 0;
}

gqa_status gqa_chunk_attention(const gqa_shape* shape, int64_t rows, const void* q,
                               int64_t q_stride, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, const int32_t* context_lens,
                               const int32_t* cu_new, void* out, void* workspace,
                               size_t workspace_bytes, int32_t* dev_status, void* stream) {
    return chunk_entry(shape, rows, q_stride, q, k_cache, v_cache, block_tables, false,
                       context_lens, cu_new, out, workspace, workspace_bytes, dev_status, stream);
}

gqa_status gqa_sparse_decode_attention(const gqa_shape* shape, const void* q, const void* k_cache,
                                       const void* v_cache, const int32_t* tables,
                                       const int32_t* lens, void* out, void* workspace,
                                       size_t workspace_bytes, int32_t* dev_status,
                                       void* stream) {
    if (shape && (shape->T != 1 || shape->window != 0)) return GQA_ERR_SHAPE;
    return chunk_entry(shape, shape ? shape->B : 0, shape ? (int64_t)shape->N * shape->H : 0, q,
                       k_cache, v_cache, tables, true, lens, nullptr, out, workspace,
                       workspace_bytes, dev_status, stream);
}

gqa_status gqa_kv_block_bounds(const gqa_shape* shape, const void* k_cache,
                               const int32_t* block_tables, const int32_t* context_lens,
                               const int32_t* cu_new, int8_t* bounds, float* bounds_scale,
                               int32_t* dev_status, void* stream) {
    const gqa_status st = check_plain(shape);
    if (st != GQA_OK || shape->B == 0) return st;
    if (!k_cache || !block_tables || !context_lens || !cu_new || !bounds || !bounds_scale)
        return GQA_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(bounds)) return GQA_ERR_ALIGN;
    return gqa::launch_block_bounds(*shape, k_cache, block_tables, context_lens, cu_new, bounds,
                                    bounds_scale, dev_status, static_cast<cudaStream_t>(stream));
}

size_t gqa_select_workspace_size(const gqa_shape* shape) {
    return check_plain(shape) == GQA_OK ? gqa::select_workspace_bytes(*shape) : 0;
}

gqa_status gqa_select_blocks(const gqa_shape* shape, int keep, int first, int recent,
                             const void* q, const int8_t* bounds, const float* bounds_scale,
                             const int32_t* block_tables, const int32_t* context_lens,
                             int32_t* tables, int32_t* lens, int32_t* blocks, void* workspace,
                             size_t workspace_bytes, int32_t* dev_status, void* stream) {
    const gqa_status st = check_plain(shape);
    if (st != GQA_OK) return st;
    if (shape->T != 1 || shape->N / shape->K > 128) return GQA_ERR_SHAPE;
    // (a table of the chosen blocks is a block table again)
    if (keep < 1 || first < 0 || recent < 1 || (long long)first + recent > keep ||
        (long long)keep * 16 > (1ll << 30) ||
        (long long)shape->B * shape->K * keep > (1ll << 31) - 1)
        return GQA_ERR_SHAPE;
    if (shape->B == 0) return GQA_OK;
    if (!q || !bounds || !bounds_scale || !block_tables || !context_lens || !tables || !lens ||
        !blocks)
        return GQA_ERR_NULL;
    if (!aligned16(q) || !aligned16(bounds)) return GQA_ERR_ALIGN;
    if (!workspace || workspace_bytes < gqa::select_workspace_bytes(*shape))
        return GQA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQA_ERR_ALIGN;
    return gqa::launch_select_blocks(*shape, keep, first, recent, q, bounds, bounds_scale,
                                     block_tables, context_lens, tables, lens, blocks, workspace,
                                     dev_status, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_plan_blocks(int B, int max_blocks_per_seq, int num_blocks, int max_tokens,
                           const int32_t* context_lens, const int32_t* new_lens,
                           const int32_t* held, const int32_t* ring_state, int32_t* free_ring,
                           int32_t* block_tables, int32_t* context_lens_out, int32_t* held_out,
                           int32_t* ring_state_out, int32_t* cu_new, int32_t* slots,
                           int32_t* positions, unsigned int flags, int32_t* dev_status,
                           void* stream) {
    if (B < 0 || B > 16384 || max_blocks_per_seq < 1 || num_blocks < 1 || max_tokens < -1)
        return GQA_ERR_SHAPE;
    if ((long long)num_blocks * 16 > (1ll << 31) - 1 ||
        (long long)max_blocks_per_seq * 16 > (1ll << 30) ||
        (long long)B * max_blocks_per_seq > (1ll << 31) - 1)
        return GQA_ERR_SHAPE;
    if (!ring_state || !free_ring || !ring_state_out || !cu_new) return GQA_ERR_NULL;
    if (B > 0 && (!context_lens || !new_lens || !held || !block_tables || !context_lens_out ||
                  !held_out))
        return GQA_ERR_NULL;
    if ((max_tokens > 0) != (slots != nullptr) || (positions && !slots)) return GQA_ERR_NULL;
    return gqa::launch_plan_blocks(B, max_blocks_per_seq, num_blocks, max_tokens,
                                   context_lens, new_lens, held, ring_state, free_ring,
                                   block_tables, context_lens_out, held_out, ring_state_out,
                                   cu_new, slots, positions,
                                   (flags & (GQA_FLAG_PDL | GQA_FLAG_EARLY_KV)) != 0, dev_status,
                                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
