// kvd_latent.h — kernel parameter blocks and launchers of the latent cache's operators.
#pragma once

#include "kvd_internal.h"

namespace kvd {

constexpr int kLatDim = 512;           // values of a token's latent vector: the keys' first part, and the values
constexpr int kLatRope = 64;           // rotated dims of its key
constexpr int kLatKey = kLatDim + kLatRope;
constexpr int kNope = 128;             // a head's own key dims, expanded
constexpr int kExpKey = kNope + kLatRope;
constexpr int kExpVal = 128;           // a head's value dims, expanded
constexpr int kLatMaxHeads = 256;

// Records of 16 tokens.  bf16: 16-byte piece i (dims 8i .. 8i+7) of token t at latent_piece(t, i).  8 bits: codes at
// latent_code(t, i), the rotated dims' pieces behind them as pieces 0 .. 7 of a tile one chunk wide, then 16 scales.
constexpr int kLatCodes = 16 * kLatDim;
constexpr int kLatScales = kLatCodes + 16 * kLatRope * 2;
__host__ __device__ constexpr int latent_record_bytes(bool fp8) { return fp8 ? kLatScales + 16 * 4 : 16 * kLatKey * 2; }
__host__ __device__ constexpr int latent_piece(int t, int i) {
    return (t >> 3) * 9216 + (i >> 3) * 1024 + (t & 7) * 128 + (((i & 7) ^ (t & 7)) << 4);
}
__host__ __device__ constexpr int latent_code(int t, int i) { return (t >> 3) * 4096 + (i >> 3) * 512 + (t & 7) * 64 + ((i & 7) << 3); }
__host__ __device__ constexpr int latent_rope_piece(int t, int i) {
    return kLatCodes + (t >> 3) * 1024 + (t & 7) * 128 + (((i & 7) ^ (t & 7)) << 4);
}

struct LatentAppendParams {
    const uint16_t* latent;      // bf16 bits, token n at n·stride
    const uint16_t* k_rope;
    const uint16_t* q_rope;      // head h of token n at n·q_stride + h·q_head
    uint16_t* q_out;
    const uint16_t* norm;        // [512] or null
    const int32_t* positions;
    const int64_t* slot_mapping;
    const float2* turns;         // [rot/2] (hi, lo), or null: nothing is rotated
    uint8_t* mem;                // this layer's records
    int32_t* err;
    int64_t latent_stride, k_stride, q_stride, q_head, out_stride, out_head;
    int64_t num_blocks;
    int64_t n_tokens;
    int n_q;
    int rot;
    int interleaved;
    int heads;                   // query heads a warp: set by the launcher
    float mscale;
    float eps;
};
cudaError_t launch_latent_append(LatentAppendParams p, bool fp8, int num_sms, cudaStream_t stream);

struct LatentGatherParams {
    const uint8_t* mem;          // this layer's records
    const int32_t* block_table;  // [B][max_blocks]
    const int32_t* row_start;    // [B + 1]
    const int32_t* first;        // [B] or null
    uint16_t* out;
    int32_t* err;
    int64_t out_stride;
    int64_t num_blocks;
    int64_t n_rows;
    int max_blocks;
    int B;
};
cudaError_t launch_latent_gather(const LatentGatherParams& p, bool fp8, int num_sms, cudaStream_t stream);

struct LatentAttnParams {
    const uint8_t* mem;          // this layer's records
    const uint16_t* q;           // bf16 bits [n_tokens][n_q][576]
    const int32_t* q_start;      // [B + 1]
    const int32_t* block_table;  // [B][max_blocks]
    const int32_t* seq_lens;     // [B]
    const uint16_t* retain;      // [num_blocks] or null
    void* out;                   // [n_tokens][n_q][512]
    float* lse_out;              // [n_tokens][n_q] or null
    float* part;                 // workspace: [2·CTAs][64 rows · 512] unnormalised sums, in the order of part_at
    float* part_ml;              // workspace: [2·CTAs][3][64] maximum (log2 domain), sum of weights, of rounded ones
    int4* part_seg;              // workspace: [2·CTAs]
    int32_t* err;
    int64_t num_blocks;
    int n_tokens;
    int max_blocks;
    int B;
    int n_q;
    int out_f32;
    float scale_log2;            // softmax_scale·log2(e)
};
constexpr int kLatUnitRows = 64;       // rows of a unit of work
cudaError_t launch_latent_attn(const LatentAttnParams& p, bool fp8, int num_sms, cudaStream_t stream);

struct LatentPrefillParams {
    const uint16_t* q;           // bf16 bits [n_tokens][n_q][192]
    const uint16_t* k_nope;      // head h of key n at n·k_stride + h·k_head
    const uint16_t* v;
    const uint16_t* k_rope;      // key n at n·rope_stride
    const int32_t* q_start;      // [B + 1]
    const int32_t* kv_start;     // [B + 1]
    void* out;                   // [n_tokens][n_q][128]
    float* lse_out;              // [n_tokens][n_q] or null
    int32_t* err;
    int64_t k_stride, k_head, v_stride, v_head, rope_stride;
    int64_t n_keys;
    int n_tokens;
    int B;
    int n_q;
    int causal;
    int out_f32;
    float scale_log2;
};
cudaError_t launch_latent_prefill(const LatentPrefillParams& p, int num_sms, cudaStream_t stream);

}  // namespace kvd
