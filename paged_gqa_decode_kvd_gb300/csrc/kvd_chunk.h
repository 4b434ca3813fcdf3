// kvd_chunk.h — kernel parameter blocks and launchers of the chunk operators (rotary append, chunk
// attention, compaction).
#pragma once

#include "kvd_internal.h"

namespace kvd {

constexpr int kMaxRopePos = 1 << 24;   // positions a float holds exactly

struct RopeParams {
    const uint16_t* q;           // bf16 bits, token n's heads at n·stride
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const int32_t* positions;
    const int64_t* slot_mapping;
    const float2* turns;         // [rot/2] (hi, lo)
    uint8_t* kv;                 // this layer's records
    uint8_t* host_kv;            // this layer's host-tier records (device address), or null
    const uint8_t* block_fmt;
    int32_t* err;
    int64_t num_blocks;
    int64_t host_blocks;
    int n_tokens;
    int n_q;
    int n_kv;
    int ng;
    int rot;
    int interleaved;
    int heads_per_cta, kv_heads_per_cta;           // set by the launcher
    float mscale;
};
cudaError_t launch_rope_append(RopeParams p, int kind, int num_sms, cudaStream_t stream);

struct ChunkParams {
    const uint8_t* kv;           // this layer's records
    const uint8_t* stage;        // host-tier records to read (staged copy, or the host's), or null
    const uint8_t* block_fmt;
    const uint16_t* q;           // bf16 bits [n_tokens][n_q][128]
    const int32_t* q_start;      // [B + 1]
    const int32_t* block_table;  // [B][max_blocks]
    const int32_t* seq_lens;     // [B]
    const uint16_t* retain;      // [num_blocks + host_blocks] or null
    void* out;
    float* lse_out;
    float* part;                 // workspace: [2·CTAs][128 dims][256 rows] unnormalised sums
    float* part_ml;              // workspace: [2·CTAs][2][256] maximum (log2 domain), sum of weights
    int4* part_seg;              // workspace: [2·CTAs] (request or −1, unit, head << 1 | not its first part, end tile)
    int32_t* err;
    int64_t num_blocks;
    int64_t host_blocks;
    int64_t record_bytes;
    int host_direct;             // host-tier records are read from host memory, by cp.async
    int n_tokens;
    int max_blocks;
    int B;
    int n_q;
    int n_kv;
    int g;
    int ng;
    int out_f32;
    float scale_log2;            // softmax_scale·log2(e)
};
constexpr int kChunkUnitRows = 256;    // rows of a unit of work
cudaError_t launch_chunk(const ChunkParams& p, int kind, int ctas, cudaStream_t stream);
cudaError_t launch_chunk_lowbit(const ChunkParams& p, int kind, int ctas, cudaStream_t stream);   // INT4 / INT2

struct CompactParams {
    const int32_t* block_table;  // [B][max_blocks]
    const int32_t* seq_lens;     // [B]
    const int32_t* new_table;    // [B][new_max_blocks]
    uint16_t* retain;            // [num_blocks + host_blocks] or null
    int32_t* new_lens;           // [B]
    const float* scores;         // [B][scores_stride] or null
    float* new_scores;
    int64_t scores_stride, new_scores_stride;
    uint32_t* source;            // workspace: [B][max_blocks·16] old slot (block·16 + offset) of every new one
    uint32_t* claim;             // workspace: [num_blocks + host_blocks]
    uint8_t* kv;                 // the whole pool (every layer)
    uint8_t* host_kv;            // the whole host tier (device address), or null
    int32_t* err;
    int64_t num_blocks;
    int64_t host_blocks;
    int max_blocks;
    int new_max_blocks;
    int B;
    int L;
    int n_kv;
};
cudaError_t launch_compact(const CompactParams& p, int kind, int ng, int num_sms, cudaStream_t stream);

}  // namespace kvd
