// kvd_compact.cu — the retained slots of a batch copied to dense blocks.
//
// The retain mask leaves evicted slots in the middle of blocks: the decode skips them, but their
// pages stay taken and their bytes are still streamed.  Compaction copies position p of request b,
// if retained, to position rank(p) = Σ_{p' < p} retained(p') of a row of new blocks, for every layer
// and KV head; order is kept, so causal attention over the new row equals masked attention over
// the old one.  With nothing evicted it is a copy (a fork of the request).
//
// Three launches: the ranks (one CTA per request, a prefix sum over its blocks' popcounts), the
// blocks' claims (a new block named twice, or one that is also read, is skipped), and the gather.
// Bound of the gather: HBM, each retained byte read and written once.
#include "kvd_chunk.h"
#include "kvd_common.cuh"

namespace kvd {
namespace {

constexpr int kRankThreads = 256;
constexpr uint32_t kNoSource = 0xffffffffu;

__device__ __forceinline__ int request_blocks(const CompactParams& p, int b) {
    const int len = p.seq_lens[b];
    if (len < 0 || static_cast<int64_t>(len) > static_cast<int64_t>(p.max_blocks) * kBs) return -1;
    return (len + kBs - 1) / kBs;
}

// Slots of logical block j that are kept.
__device__ __forceinline__ uint32_t kept_slots(const CompactParams& p, int len, int phys, int j) {
    const int64_t ids = p.num_blocks + p.host_blocks;
    if (phys < 0 || phys >= ids) return 0;
    const int left = len - j * kBs;
    const uint32_t in = left >= kBs ? 0xffffu : (1u << left) - 1u;
    return p.retain ? p.retain[phys] & in : in;
}

// One CTA per request: source of every new slot, the new length, the scores.  Clears the claims.
__global__ void __launch_bounds__(kRankThreads) compact_rank_kernel(const CompactParams p) {
    __shared__ int scan[kRankThreads];
    __shared__ int base;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x, tid = threadIdx.x;
    for (int64_t i = static_cast<int64_t>(b) * kRankThreads + tid; i < p.num_blocks + p.host_blocks;
         i += static_cast<int64_t>(gridDim.x) * kRankThreads)
        p.claim[i] = 0;
    const int len = p.seq_lens[b];
    int nb = request_blocks(p, b);
    if (nb < 0) {
        if (tid == 0) report(p.err, KVD_ERR_OOB);
        nb = 0;
    }
    if (tid == 0) base = 0;
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    uint32_t* source = p.source + static_cast<int64_t>(b) * p.max_blocks * kBs;
    const float* from = p.scores ? p.scores + static_cast<int64_t>(b) * p.scores_stride : nullptr;
    float* to = p.scores ? p.new_scores + static_cast<int64_t>(b) * p.new_scores_stride : nullptr;
    __syncthreads();
    for (int j0 = 0; j0 < nb; j0 += kRankThreads) {
        const int j = j0 + tid;
        uint32_t kept = 0;
        int phys = 0;
        if (j < nb) {
            phys = table[j];
            kept = kept_slots(p, len, phys, j);
            if (phys < 0 || phys >= p.num_blocks + p.host_blocks) report(p.err, KVD_ERR_OOB);
        }
        const int n = __popc(kept);
        scan[tid] = n;
        __syncthreads();
        for (int off = 1; off < kRankThreads; off <<= 1) {
            const int v = tid >= off ? scan[tid - off] : 0;
            __syncthreads();
            scan[tid] += v;
            __syncthreads();
        }
        int r = base + scan[tid] - n;
        while (kept) {
            const int t = __ffs(kept) - 1;
            kept &= kept - 1;
            source[r] = static_cast<uint32_t>(phys) * kBs + t;
            if (to && r < p.new_scores_stride) {
                const int64_t pos = static_cast<int64_t>(j) * kBs + t;
                to[r] = pos < p.scores_stride ? from[pos] : 0.f;
            }
            ++r;
        }
        __syncthreads();
        if (tid == kRankThreads - 1) base += scan[tid];
        __syncthreads();
    }
    int total = base;
    if (total > static_cast<int64_t>(p.new_max_blocks) * kBs) {   // the new row cannot hold it: an empty request
        if (tid == 0) report(p.err, KVD_ERR_OOB);
        total = 0;
    }
    if (tid == 0) p.new_lens[b] = total;
    const int tail = (kBs - total % kBs) % kBs;   // the last block's other slots
    if (tid < tail) source[total + tid] = kNoSource;
    if (to)
        for (int64_t i = total + tid; i < p.new_scores_stride; i += kRankThreads) to[i] = 0.f;
}

// claim[id]: bit 0 = read as a source, then 2 for every new-table entry in use that names it.
__global__ void __launch_bounds__(kRankThreads) compact_claim_kernel(const CompactParams p) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y;
    const int j = blockIdx.x * kRankThreads + threadIdx.x;
    const int64_t ids = p.num_blocks + p.host_blocks;
    if (j < request_blocks(p, b)) {
        const int phys = p.block_table[static_cast<int64_t>(b) * p.max_blocks + j];
        if (phys >= 0 && phys < ids) atomicOr(&p.claim[phys], 1u);
    }
    if (static_cast<int64_t>(j) * kBs >= p.new_lens[b]) return;   // ≤ new_max_blocks·16
    const int to = p.new_table[static_cast<int64_t>(b) * p.new_max_blocks + j];
    if (to >= 0 && to < ids) atomicAdd(&p.claim[to], 2u);
}

// ------------------------------------------------------------------ gather
// The record's 16-byte pieces, by kind.  unit(piece, k): the slot offset t whose bytes fill unit k
// of the piece, and where those bytes are in a source record that holds the token at offset u.
template <int KIND, int NG>
struct Rec {
    static constexpr int kBits = KIND == kKindInt4 ? 4 : 2;
    static constexpr bool kLow = is_lowbit(KIND);
    static constexpr bool kWide = KIND == kKindBf16;
    static constexpr int kBytes = kWide ? kRecordBf16 : kLow ? lowbit_record_bytes(kBits, NG) : kRecordFp8;
    static constexpr int kTile = kWide ? kTileBf16 : kLow ? lowbit_tile_bytes(kBits) : kTileFp8;
    static constexpr int kPieces = kBytes / 16;
};

// K tile of a 16- or 8-bit record: 16-byte piece = fragment lane (r, x); token t = r + 8·((k >> 1) & 1)
// for element e, elements in pairs (W = bytes of an element).
template <int W>
__device__ __forceinline__ uint4 gather_k(const uint8_t* const* rec, const int* off, int piece) {
    const int l = piece & 31, x = l & 3, r = l >> 2, group = piece >> 5;
    uint4 out;
    uint32_t* o = reinterpret_cast<uint32_t*>(&out);
    auto at = [&](int t) -> const uint8_t* {   // the piece of token t's source that holds its pairs
        const int u = off[t];
        return rec[t] + (group * 32 + 4 * (u & 7) + x) * 16 + (u >> 3) * 2 * W;
    };
    const uint8_t* a = rec[r] ? at(r) : nullptr;
    const uint8_t* b = rec[r + 8] ? at(r + 8) : nullptr;
    if constexpr (W == 2) {
        o[0] = a ? *reinterpret_cast<const uint32_t*>(a) : 0u;
        o[1] = b ? *reinterpret_cast<const uint32_t*>(b) : 0u;
        o[2] = a ? *reinterpret_cast<const uint32_t*>(a + 8) : 0u;
        o[3] = b ? *reinterpret_cast<const uint32_t*>(b + 8) : 0u;
    } else {
        #pragma unroll
        for (int k = 0; k < 4; ++k) {   // group 2i (k < 2) and 2i + 1; dims + 0 and + 8
            const uint32_t lo = a ? *reinterpret_cast<const uint16_t*>(a + 4 * k) : 0u;
            const uint32_t hi = b ? *reinterpret_cast<const uint16_t*>(b + 4 * k) : 0u;
            o[k] = lo | (hi << 16);
        }
    }
    return out;
}

// V tile: 16-byte piece = fragment lane (r, x); elements of tokens 2x, 2x+1, 2x+8, 2x+9, dims r and r + 8.
template <int W>
__device__ __forceinline__ uint4 gather_v(const uint8_t* const* rec, const int* off, int piece) {
    const int l = piece & 31, x = l & 3, r = l >> 2, group = piece >> 5;
    uint32_t e[2][2][4] = {};   // [group half (8-bit)][dim half][token]
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = 2 * x + (k & 1) + 8 * (k >> 1);
        if (!rec[t]) continue;
        const int u = off[t];
        const uint8_t* base = rec[t] + Rec<W == 2 ? kKindBf16 : kKindFp8, 1>::kTile +
                              (group * 32 + 4 * r + ((u & 7) >> 1)) * 16 + ((u & 1) + 4 * (u >> 3)) * W;
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (W == 2) {
                e[0][h][k] = *reinterpret_cast<const uint16_t*>(base + h * 4);
            } else {
                e[0][h][k] = base[h * 2];
                e[1][h][k] = base[8 + h * 2];
            }
        }
    }
    if constexpr (W == 2) {
        return make_uint4(e[0][0][0] | e[0][0][1] << 16, e[0][1][0] | e[0][1][1] << 16, e[0][0][2] | e[0][0][3] << 16,
                          e[0][1][2] | e[0][1][3] << 16);
    } else {
        auto word = [&](int g, int hi) {
            const int k = 2 * hi;
            return e[g][0][k] | e[g][0][k + 1] << 8 | e[g][1][k] << 16 | e[g][1][k + 1] << 24;
        };
        return make_uint4(word(0, 0), word(0, 1), word(1, 0), word(1, 1));
    }
}

// A low-bit tile's piece: words (kg parity, th) of lane l.  K words hold one token's codes, V bytes
// two tokens of one dim each.
__device__ __forceinline__ uint4 gather_low(const uint8_t* const* rec, const int* off, int piece, int tile, bool value) {
    const int l = piece & 31, x = l & 3, r = l >> 2, group = piece >> 5;
    uint32_t o[4];
    #pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int par = w >> 1, th = w & 1;
        if (!value) {
            const int t = r + 8 * th;
            o[w] = 0;
            if (rec[t])
                o[w] = *reinterpret_cast<const uint32_t*>(
                    rec[t] + ((group * 32 + 4 * (off[t] & 7) + x) * 4 + par * 2 + (off[t] >> 3)) * 4);
        } else {
            uint32_t v = 0;
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = 2 * x + k + 8 * th;
                if (!rec[t]) continue;
                const int u = off[t];
                const uint8_t* base =
                    rec[t] + tile + ((group * 32 + 4 * r + ((u & 7) >> 1)) * 4 + par * 2 + (u >> 3)) * 4 + (u & 1);
                v |= static_cast<uint32_t>(base[0]) << (8 * k) | static_cast<uint32_t>(base[2]) << (8 * k + 16);
            }
            o[w] = v;
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Words after the tiles: [2][16 tokens][words per token]; four words a piece.
template <int WORDS>
__device__ __forceinline__ uint4 gather_words(const uint8_t* const* rec, const int* off, int piece, int tiles) {
    uint32_t o[4];
    #pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int i = piece * 4 + w;
        const int side = i / (kBs * WORDS), t = i / WORDS % kBs, g = i % WORDS;
        o[w] = rec[t] ? reinterpret_cast<const uint32_t*>(rec[t] + tiles)[(side * kBs + off[t]) * WORDS + g] : 0u;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int KIND, int NG>
__device__ __forceinline__ uint4 gather_piece(const uint8_t* const* rec, const int* off, int c) {
    using R = Rec<KIND, NG>;
    constexpr int kT = R::kTile / 16;
    if constexpr (R::kWide) {
        return c < kT ? gather_k<2>(rec, off, c) : gather_v<2>(rec, off, c - kT);
    } else if constexpr (R::kLow) {
        if (c < 2 * kT) return gather_low(rec, off, c < kT ? c : c - kT, R::kTile, c >= kT);
        return gather_words<NG>(rec, off, c - 2 * kT, 2 * R::kTile);
    } else {
        if (c < kT) return gather_k<1>(rec, off, c);
        if (c < 2 * kT) return gather_v<1>(rec, off, c - kT);
        return gather_words<1>(rec, off, c - 2 * kT, 2 * R::kTile);
    }
}

constexpr int kGatherThreads = 256;

// CTA (new block j of request b, share of the (layer, KV head) pairs).
template <int KIND, int NG>
__global__ void __launch_bounds__(kGatherThreads) compact_gather_kernel(const CompactParams p) {
    using R = Rec<KIND, NG>;
    __shared__ const uint8_t* rec[2][kBs];
    __shared__ int off[kBs];
    __shared__ uint32_t src[kBs];
    pdl_wait();
    const int tid = threadIdx.x;
    const int b = blockIdx.z, j = blockIdx.x;
    const int n = p.new_lens[b];
    if (static_cast<int64_t>(j) * kBs >= n) return;
    const int to = p.new_table[static_cast<int64_t>(b) * p.new_max_blocks + j];
    if (to < 0 || to >= p.num_blocks + p.host_blocks || p.claim[to] != 2u) {   // no block, or not this one's alone
        if (tid == 0 && blockIdx.y == 0) report(p.err, KVD_ERR_OOB);
        return;
    }
    if (tid == 0 && blockIdx.y == 0 && p.retain) p.retain[to] = 0xffffu;   // `to` is no source: nobody reads its mask
    if (tid < kBs) {
        src[tid] = p.source[(static_cast<int64_t>(b) * p.max_blocks + j) * kBs + tid];
        off[tid] = static_cast<int>(src[tid] % kBs);
    }
    __syncthreads();
    auto record = [&](int64_t id, int layer, int h) -> uint8_t* {
        return id < p.num_blocks
                   ? p.kv + ((static_cast<int64_t>(layer) * p.num_blocks + id) * p.n_kv + h) * R::kBytes
                   : p.host_kv + ((static_cast<int64_t>(layer) * p.host_blocks + (id - p.num_blocks)) * p.n_kv + h) * R::kBytes;
    };
    const int pairs = p.L * p.n_kv;
    int k = 0;
    for (int i = blockIdx.y; i < pairs; i += gridDim.y, k ^= 1) {
        const int layer = i / p.n_kv, h = i % p.n_kv;
        if (tid < kBs) rec[k][tid] = src[tid] == kNoSource ? nullptr : record(src[tid] / kBs, layer, h);
        __syncthreads();
        uint4* out = reinterpret_cast<uint4*>(record(to, layer, h));
        for (int c = tid; c < R::kPieces; c += kGatherThreads) out[c] = gather_piece<KIND, NG>(rec[k], off, c);
    }
}

template <int KIND, int NG>
cudaError_t launch_gather(const CompactParams& p, dim3 grid, cudaStream_t stream) {
    return launch_dependent(compact_gather_kernel<KIND, NG>, grid, dim3(kGatherThreads), 0, -1, stream, p);
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, int kind, int ng, cudaStream_t stream) {
    cudaError_t e = launch_dependent(compact_rank_kernel, dim3(static_cast<unsigned>(p.B)), dim3(kRankThreads), 0, -1,
                                     stream, p);
    if (e != cudaSuccess) return e;
    const dim3 claims(static_cast<unsigned>((p.max_blocks + kRankThreads - 1) / kRankThreads), static_cast<unsigned>(p.B));
    e = launch_dependent(compact_claim_kernel, claims, dim3(kRankThreads), 0, -1, stream, p);
    if (e != cudaSuccess) return e;
    const int pairs = p.L * p.n_kv;
    const dim3 grid(static_cast<unsigned>(p.max_blocks), static_cast<unsigned>(pairs < 8 ? pairs : 8),
                    static_cast<unsigned>(p.B));
    switch (kind) {
        case kKindFp8:
        case kKindAngle: return launch_gather<kKindFp8, 1>(p, grid, stream);
        case kKindInt4:
            return ng == 4   ? launch_gather<kKindInt4, 4>(p, grid, stream)
                   : ng == 2 ? launch_gather<kKindInt4, 2>(p, grid, stream)
                             : launch_gather<kKindInt4, 1>(p, grid, stream);
        case kKindInt2:
            return ng == 4   ? launch_gather<kKindInt2, 4>(p, grid, stream)
                   : ng == 2 ? launch_gather<kKindInt2, 2>(p, grid, stream)
                             : launch_gather<kKindInt2, 1>(p, grid, stream);
        default: return launch_gather<kKindBf16, 1>(p, grid, stream);
    }
}

}  // namespace kvd
