// kvd_latent_api.cu — the latent cache's entry points: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/kvd.h"
#include "kvd_common.cuh"
#include "kvd_latent.h"
#include "kvd_pool.h"

using namespace kvd;

namespace {

static_assert(KVD_LATENT_DIM == kLatDim && KVD_LATENT_ROPE == kLatRope, "the header's sizes");

bool is_fp8(const kvd_pool* pool) { return pool->desc.kv_dtype == KVD_LATENT_FP8; }

uint8_t* layer_mem(const kvd_pool* pool, int layer) { return pool->mem + static_cast<size_t>(layer) * pool->layer_bytes; }

kvd_status check_pool(const kvd_pool* pool, int layer) {
    if (!pool || layer < 0 || layer >= pool->desc.num_layers) return KVD_ERR_INVALID;
    return is_latent(pool) ? KVD_OK : KVD_ERR_UNSUPPORTED;
}

bool overlaps_pool(const kvd_pool* pool, const void* x, size_t bytes) {
    return overlap(x, bytes, pool->mem, pool->layer_bytes * static_cast<size_t>(pool->desc.num_layers));
}

// Bytes from the first row's start to the last row's end.
size_t span(size_t n, int64_t stride, size_t row) { return (n - 1) * 2 * static_cast<size_t>(stride) + row; }

struct LatentLayout {
    size_t part, ml, seg, total;
};

// Two partials a CTA (its first and its last unit may be cut), one CTA per SM.
LatentLayout latent_layout(const kvd_pool* pool) {
    const size_t slots = 2 * static_cast<size_t>(pool->num_sms);
    LatentLayout w;
    w.part = 0;
    w.ml = align256(w.part + slots * kLatUnitRows * kLatDim * sizeof(float));
    w.seg = align256(w.ml + slots * kLatUnitRows * 3 * sizeof(float));
    w.total = align256(w.seg + slots * sizeof(int4));
    return w;
}

kvd_status check_heads(const kvd_pool* pool, int n_q, int batch) {
    if (!pool || n_q < 1 || batch < 0) return KVD_ERR_INVALID;
    if (!is_latent(pool) || n_q > kLatMaxHeads || batch > kMaxBatch) return KVD_ERR_UNSUPPORTED;
    return KVD_OK;
}

}  // namespace

extern "C" {

kvd_status kvd_latent_append(kvd_pool* pool, int layer, const void* latent, int64_t latent_stride, const void* k_rope,
                             int64_t k_rope_stride, const void* norm_weight, float norm_eps, const void* q_rope,
                             int64_t q_stride, int64_t q_head_stride, int n_q, const int32_t* positions,
                             const kvd_rope_desc* rope, const int64_t* slot_mapping, int n_tokens, void* q_rope_out,
                             int64_t q_out_stride, int64_t q_out_head_stride, void* stream) {
    kvd_status st = check_pool(pool, layer);
    if (st != KVD_OK) return st;
    if (n_q < 0 || n_tokens < 0 || (n_q > 0 && !rope)) return KVD_ERR_INVALID;
    if (rope && (rope->rot_dim < 2 || (rope->rot_dim & 1) || !rope->turns || (rope->interleaved != 0 && rope->interleaved != 1)))
        return KVD_ERR_INVALID;
    if (norm_weight && !(norm_eps >= 0.f && std::isfinite(norm_eps))) return KVD_ERR_INVALID;
    if ((rope && rope->rot_dim > kLatRope) || n_q > kLatMaxHeads) return KVD_ERR_UNSUPPORTED;
    if (n_tokens == 0) return KVD_OK;
    if (!latent || !k_rope || !slot_mapping || (rope && !positions) || (n_q > 0 && (!q_rope || !q_rope_out))) return KVD_ERR_INVALID;
    if (latent_stride < kLatDim || k_rope_stride < kLatRope || (latent_stride & 7) || (k_rope_stride & 7)) return KVD_ERR_INVALID;
    if (!aligned16(latent) || !aligned16(k_rope) || !aligned16(norm_weight)) return KVD_ERR_INVALID;
    if (rope && (reinterpret_cast<uintptr_t>(rope->turns) & 7u)) return KVD_ERR_INVALID;
    const size_t n = static_cast<size_t>(n_tokens);
    if (n_q > 0) {
        // heads of a token apart from each other, tokens apart from each other
        if (q_head_stride < kLatRope || q_out_head_stride < kLatRope || (q_head_stride & 7) || (q_out_head_stride & 7) ||
            (q_stride & 7) || (q_out_stride & 7) || !aligned16(q_rope) || !aligned16(q_rope_out))
            return KVD_ERR_INVALID;
        const int64_t q_row = (n_q - 1) * q_head_stride + kLatRope, out_row = (n_q - 1) * q_out_head_stride + kLatRope;
        if (q_stride < q_row || q_out_stride < out_row) return KVD_ERR_INVALID;
        const size_t out_bytes = 2 * static_cast<size_t>(out_row), pitch = 2 * static_cast<size_t>(q_out_stride);
        // a warp reads rows while another writes its own (q itself is read by the warp that writes it)
        const bool in_place = q_rope_out == q_rope && q_out_stride == q_stride && q_out_head_stride == q_head_stride;
        if (!in_place && rows_overlap(q_rope, 2 * static_cast<size_t>(q_row), 2 * static_cast<size_t>(q_stride), q_rope_out, out_bytes, pitch, n)) {
            // slices of one tensor's heads have one pitch, and each its own dims of every head
            if (q_stride != q_out_stride || q_head_stride != q_out_head_stride || q_stride % q_head_stride != 0 ||
                rows_overlap(q_rope, 2 * kLatRope, 2 * static_cast<size_t>(q_head_stride), q_rope_out, 2 * kLatRope,
                             2 * static_cast<size_t>(q_head_stride), (n - 1) * (q_stride / q_head_stride) + n_q))
                return KVD_ERR_INVALID;
        }
        if (rows_overlap(latent, 2 * kLatDim, 2 * static_cast<size_t>(latent_stride), q_rope_out, out_bytes, pitch, n) ||
            rows_overlap(k_rope, 2 * kLatRope, 2 * static_cast<size_t>(k_rope_stride), q_rope_out, out_bytes, pitch, n) ||
            overlaps_pool(pool, q_rope_out, span(n, q_out_stride, out_bytes)))
            return KVD_ERR_INVALID;
    }
    st = check_device(pool->device);
    if (st != KVD_OK) return st;
    LatentAppendParams p;
    p.latent = static_cast<const uint16_t*>(latent);
    p.k_rope = static_cast<const uint16_t*>(k_rope);
    p.q_rope = static_cast<const uint16_t*>(q_rope);
    p.q_out = static_cast<uint16_t*>(q_rope_out);
    p.norm = static_cast<const uint16_t*>(norm_weight);
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.turns = rope ? reinterpret_cast<const float2*>(rope->turns) : nullptr;
    p.mem = layer_mem(pool, layer);
    p.err = pool->err;
    p.latent_stride = latent_stride;
    p.k_stride = k_rope_stride;
    p.q_stride = q_stride;
    p.q_head = q_head_stride;
    p.out_stride = q_out_stride;
    p.out_head = q_out_head_stride;
    p.num_blocks = pool->desc.num_blocks;
    p.n_tokens = n_tokens;
    p.n_q = n_q;
    p.rot = rope ? rope->rot_dim : 0;
    p.interleaved = rope ? rope->interleaved : 1;
    p.heads = 0;
    p.mscale = rope ? rope->mscale : 1.f;
    p.eps = norm_eps;
    return cuda_status(launch_latent_append(p, is_fp8(pool), pool->num_sms, static_cast<cudaStream_t>(stream)));
}

kvd_status kvd_latent_gather(kvd_pool* pool, int layer, const int32_t* block_table, int max_blocks_per_seq,
                             const int32_t* row_start, const int32_t* first, int batch, int n_rows, void* out,
                             int64_t out_stride, void* stream) {
    kvd_status st = check_pool(pool, layer);
    if (st != KVD_OK) return st;
    if (batch < 0 || n_rows < 0 || max_blocks_per_seq < 1) return KVD_ERR_INVALID;
    if (batch > kMaxBatch) return KVD_ERR_UNSUPPORTED;
    if (batch == 0 || n_rows == 0) return KVD_OK;
    if (!block_table || !row_start || !out || !aligned16(out) || out_stride < kLatKey || (out_stride & 7)) return KVD_ERR_INVALID;
    if (overlaps_pool(pool, out, span(static_cast<size_t>(n_rows), out_stride, 2 * kLatKey))) return KVD_ERR_INVALID;
    st = check_device(pool->device);
    if (st != KVD_OK) return st;
    LatentGatherParams p;
    p.mem = layer_mem(pool, layer);
    p.block_table = block_table;
    p.row_start = row_start;
    p.first = first;
    p.out = static_cast<uint16_t*>(out);
    p.err = pool->err;
    p.out_stride = out_stride;
    p.num_blocks = pool->desc.num_blocks;
    p.n_rows = n_rows;
    p.max_blocks = max_blocks_per_seq;
    p.B = batch;
    return cuda_status(launch_latent_gather(p, is_fp8(pool), pool->num_sms, static_cast<cudaStream_t>(stream)));
}

kvd_status kvd_latent_workspace_bytes(const kvd_pool* pool, int n_q, int batch, size_t* bytes_out) {
    kvd_status st = check_heads(pool, n_q, batch);
    if (st != KVD_OK) return st;
    if (!bytes_out) return KVD_ERR_INVALID;
    *bytes_out = latent_layout(pool).total;
    return KVD_OK;
}

kvd_status kvd_latent_attn(kvd_pool* pool, int layer, const void* q, int n_q, const int32_t* q_start, int n_tokens,
                           const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens, int batch,
                           const uint16_t* retain_mask, float softmax_scale, void* workspace, size_t workspace_bytes,
                           void* out, int out_dtype, float* lse_out, void* stream) {
    kvd_status st = check_heads(pool, n_q, batch);
    if (st != KVD_OK) return st;
    if (layer < 0 || layer >= pool->desc.num_layers || n_tokens < 0 || max_blocks_per_seq < 1) return KVD_ERR_INVALID;
    if (out_dtype != KVD_BF16 && out_dtype != KVD_F32) return KVD_ERR_INVALID;
    if (!std::isfinite(softmax_scale * kLog2e)) return KVD_ERR_INVALID;
    if (batch == 0 || n_tokens == 0) return KVD_OK;
    if (!q || !q_start || !block_table || !seq_lens || !workspace || !out) return KVD_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return KVD_ERR_INVALID;
    const LatentLayout w = latent_layout(pool);
    if (workspace_bytes < w.total) return KVD_ERR_NOMEM;
    const size_t rows = static_cast<size_t>(n_tokens) * n_q, value = out_dtype == KVD_F32 ? 4 : 2;
    if (overlap(q, 2 * rows * kLatKey, out, value * rows * kLatDim) || overlaps_pool(pool, out, value * rows * kLatDim) ||
        overlap(workspace, w.total, out, value * rows * kLatDim) || overlap(workspace, w.total, q, 2 * rows * kLatKey))
        return KVD_ERR_INVALID;
    st = check_device(pool->device);
    if (st != KVD_OK) return st;
    LatentAttnParams p;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.mem = layer_mem(pool, layer);
    p.q = static_cast<const uint16_t*>(q);
    p.q_start = q_start;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.retain = retain_mask;
    p.out = out;
    p.lse_out = lse_out;
    p.part = reinterpret_cast<float*>(ws + w.part);
    p.part_ml = reinterpret_cast<float*>(ws + w.ml);
    p.part_seg = reinterpret_cast<int4*>(ws + w.seg);
    p.err = pool->err;
    p.num_blocks = pool->desc.num_blocks;
    p.n_tokens = n_tokens;
    p.max_blocks = max_blocks_per_seq;
    p.B = batch;
    p.n_q = n_q;
    p.out_f32 = out_dtype == KVD_F32;
    p.scale_log2 = softmax_scale * kLog2e;
    return cuda_status(launch_latent_attn(p, is_fp8(pool), pool->num_sms, static_cast<cudaStream_t>(stream)));
}

kvd_status kvd_latent_prefill(kvd_pool* pool, const void* q, int n_q, const int32_t* q_start, int n_tokens,
                              const void* k_nope, int64_t k_stride, int64_t k_head_stride, const void* v, int64_t v_stride,
                              int64_t v_head_stride, const void* k_rope, int64_t k_rope_stride, const int32_t* kv_start,
                              int n_keys, int batch, int causal, float softmax_scale, void* out, int out_dtype,
                              float* lse_out, void* stream) {
    kvd_status st = check_heads(pool, n_q, batch);
    if (st != KVD_OK) return st;
    if (n_tokens < 0 || n_keys < 0 || (causal != 0 && causal != 1)) return KVD_ERR_INVALID;
    if (out_dtype != KVD_BF16 && out_dtype != KVD_F32) return KVD_ERR_INVALID;
    if (!std::isfinite(softmax_scale * kLog2e)) return KVD_ERR_INVALID;
    if (batch == 0 || n_tokens == 0) return KVD_OK;
    if (!q || !q_start || !kv_start || !out || !aligned16(q) || !aligned16(out)) return KVD_ERR_INVALID;
    const size_t rows = static_cast<size_t>(n_tokens) * n_q, out_bytes = (out_dtype == KVD_F32 ? 4 : 2) * rows * kExpVal;
    if (overlap(q, 2 * rows * kExpKey, out, out_bytes)) return KVD_ERR_INVALID;
    if (n_keys > 0) {
        if (!k_nope || !v || !k_rope || !aligned16(k_nope) || !aligned16(v) || !aligned16(k_rope)) return KVD_ERR_INVALID;
        if (k_head_stride < kNope || v_head_stride < kExpVal || ((k_stride | k_head_stride | v_stride | v_head_stride | k_rope_stride) & 7))
            return KVD_ERR_INVALID;
        const int64_t k_row = (n_q - 1) * k_head_stride + kNope, v_row = (n_q - 1) * v_head_stride + kExpVal;
        if (k_stride < k_row || v_stride < v_row || k_rope_stride < kLatRope) return KVD_ERR_INVALID;
        const size_t n = static_cast<size_t>(n_keys);
        if (overlap(k_nope, span(n, k_stride, 2 * static_cast<size_t>(k_row)), out, out_bytes) ||
            overlap(v, span(n, v_stride, 2 * static_cast<size_t>(v_row)), out, out_bytes) ||
            overlap(k_rope, span(n, k_rope_stride, 2 * kLatRope), out, out_bytes))
            return KVD_ERR_INVALID;
    }
    st = check_device(pool->device);
    if (st != KVD_OK) return st;
    LatentPrefillParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k_nope = static_cast<const uint16_t*>(k_nope);
    p.v = static_cast<const uint16_t*>(v);
    p.k_rope = static_cast<const uint16_t*>(k_rope);
    p.q_start = q_start;
    p.kv_start = kv_start;
    p.out = out;
    p.lse_out = lse_out;
    p.err = pool->err;
    p.k_stride = k_stride;
    p.k_head = k_head_stride;
    p.v_stride = v_stride;
    p.v_head = v_head_stride;
    p.rope_stride = k_rope_stride;
    p.n_keys = n_keys;
    p.n_tokens = n_tokens;
    p.B = batch;
    p.n_q = n_q;
    p.causal = causal;
    p.out_f32 = out_dtype == KVD_F32;
    p.scale_log2 = softmax_scale * kLog2e;
    return cuda_status(launch_latent_prefill(p, pool->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
