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
// Bound of the gather: HBM, each retained byte read and written once, and with them the evicted ones of the same
// 16-byte pieces.  Eight traces of 7,000 to 8,192 positions in 28 layers, 3% evicted: 1,092 us, 6.4 TB/s (96% of the
// measured bandwidth); one 8-bit request of 16,411 in 80 layers, a third evicted: 828 us (67%; 84% with the bytes that
// come along).  A short call is its three launches.
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
    __shared__ int sums[kRankThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    for (int64_t i = static_cast<int64_t>(b) * kRankThreads + tid; i < p.num_blocks + p.host_blocks;
         i += static_cast<int64_t>(gridDim.x) * kRankThreads)
        p.claim[i] = 0;
    const int len = p.seq_lens[b];
    int nb = request_blocks(p, b);
    if (nb < 0) {
        if (tid == 0) report(p.err, KVD_ERR_OOB);
        nb = 0;
    }
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    uint32_t* source = p.source + static_cast<int64_t>(b) * p.max_blocks * kBs;
    const float* from = p.scores ? p.scores + static_cast<int64_t>(b) * p.scores_stride : nullptr;
    float* to = p.scores ? p.new_scores + static_cast<int64_t>(b) * p.new_scores_stride : nullptr;
    int base = 0;
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
        int up = n;   // of this block and those before it in the warp
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, up, o);
            if (lane >= o) up += v;
        }
        if (lane == 31) sums[tid >> 5] = up;
        __syncthreads();
        int before = 0, all = 0;
        #pragma unroll
        for (int w = 0; w < kRankThreads / 32; ++w) {
            before += w < (tid >> 5) ? sums[w] : 0;
            all += sums[w];
        }
        int r = base + before + up - n;
        base += all;
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

// The sources of a block's 16 slots in the record of one (layer, KV head): offset of the token in its record, and the
// record's place in the first layer's first head's, to which a pair adds its own, by tier.
struct Sources {
    const uint8_t* const* rec;
    const int* off;
    const bool* host;
    int64_t device_pair, host_pair;
    __device__ __forceinline__ const uint8_t* operator[](int t) const {
        return rec[t] ? rec[t] + (host[t] ? host_pair : device_pair) : nullptr;
    }
};

// The source piece of new slot t's token: piece(u) gives its number in the tile for slot offset u.  All lanes load
// whole 16-byte pieces and pick the token's part: a fourth of the loads that the parts alone would take.
template <class F>
__device__ __forceinline__ uint4 source_piece(const Sources& s, int t, F piece) {
    const uint8_t* from = s[t];
    if (!from) return make_uint4(0, 0, 0, 0);
    return __ldg(reinterpret_cast<const uint4*>(from) + piece(s.off[t]));
}

// K tile: 16-byte piece = fragment lane (r, x) of a group: tokens r and r + 8.  W = bytes of an element; 0: low-bit codes.
template <int W>
__device__ __forceinline__ uint4 gather_k(const Sources& s, int piece) {
    const int l = piece & 31, x = l & 3, r = l >> 2, group = piece >> 5;
    auto number = [&](int u) { return group * 32 + 4 * (u & 7) + x; };
    const uint4 a = source_piece(s, r, number), b = source_piece(s, r + 8, number);
    const bool ah = s.off[r] >> 3, bh = s.off[r + 8] >> 3;   // which of the piece's tokens
    if constexpr (W == 1) {   // pairs of codes: the halves of each word
        const uint32_t pick = (ah ? 0x32u : 0x10u) | (bh ? 0x7600u : 0x5400u);
        return make_uint4(__byte_perm(a.x, b.x, pick), __byte_perm(a.y, b.y, pick), __byte_perm(a.z, b.z, pick),
                          __byte_perm(a.w, b.w, pick));
    } else {                  // words 0, 2: the first token; 1, 3: the second
        return make_uint4(ah ? a.y : a.x, bh ? b.y : b.x, ah ? a.w : a.z, bh ? b.w : b.z);
    }
}

// V tile at `tile`: 16-byte piece = fragment lane (r, x): tokens 2x, 2x+1, 2x+8, 2x+9 of dims r and r + 8 (of two groups:
// 8-bit and low-bit codes, alike here).
template <int W>
__device__ __forceinline__ uint4 gather_v(const Sources& s, int piece, int tile) {
    const int l = piece & 31, x = l & 3, r = l >> 2, group = piece >> 5;
    auto number = [&](int u) { return tile / 16 + group * 32 + 4 * r + ((u & 7) >> 1); };
    uint32_t lo[4], hi[4], odd[4];   // the words that hold the token
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = 2 * x + (k & 1) + 8 * (k >> 1);
        const uint4 v = source_piece(s, t, number);
        const bool second = s.off[t] >> 3;
        if constexpr (W == 2) {   // words 0, 1 or 2, 3: dims r and r + 8, a half each
            lo[k] = second ? v.z : v.x;
            hi[k] = second ? v.w : v.y;
        } else {                  // words 0, 2 or 1, 3: the two groups, bytes 0, 2 or 1, 3
            lo[k] = second ? v.y : v.x;
            hi[k] = second ? v.w : v.z;
        }
        odd[k] = s.off[t] & 1;
    }
    uint32_t o[4];
    #pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const uint32_t pick = W == 2 ? (odd[k] ? 0x32u : 0x10u) | (odd[k + 1] ? 0x7600u : 0x5400u)
                                     : 0x6240u + odd[k] * 0x0101u + odd[k + 1] * 0x1010u;
        const uint32_t a = __byte_perm(lo[k], lo[k + 1], pick), b = __byte_perm(hi[k], hi[k + 1], pick);
        if constexpr (W == 2) {   // words: (r, first), (r + 8, first), (r, second), (r + 8, second tokens)
            o[k] = a;
            o[k + 1] = b;
        } else {                  // words: (group, first), (group, second), (group + 1, first), (group + 1, second)
            o[k / 2] = a;
            o[2 + k / 2] = b;
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Words after the tiles: [2][16 tokens][words per token]; four words a piece.
template <int WORDS>
__device__ __forceinline__ uint4 gather_words(const Sources& s, int piece, int tiles) {
    uint32_t o[4];
    #pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int i = piece * 4 + w;
        const int side = i / (kBs * WORDS), t = i / WORDS % kBs, g = i % WORDS;
        const uint8_t* from = s[t];
        o[w] = from ? __ldg(reinterpret_cast<const uint32_t*>(from + tiles) + (side * kBs + s.off[t]) * WORDS + g) : 0u;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int KIND, int NG>
__device__ __forceinline__ uint4 gather_piece(const Sources& s, int c) {
    using R = Rec<KIND, NG>;
    constexpr int kT = R::kTile / 16;
    if (c < kT) return gather_k<R::kWide ? 2 : R::kLow ? 0 : 1>(s, c);
    if (c < 2 * kT) return gather_v<R::kWide ? 2 : 1>(s, c - kT, R::kTile);
    if constexpr (R::kWide) return make_uint4(0, 0, 0, 0);
    else return gather_words<R::kLow ? NG : 1>(s, c - 2 * kT, 2 * R::kTile);
}

// A thread holds a piece or two: an 8-bit record has 264, a 16-bit one 512.  Every thread slot of an SM is taken (32
// registers): the gather waits for memory.
template <int KIND>
constexpr int gather_threads() { return KIND == kKindFp8 ? 288 : 256; }

// CTA (new block j of request b, share of the (layer, KV head) pairs).
template <int KIND, int NG>
__global__ void __launch_bounds__(gather_threads<KIND>(), 2048 / gather_threads<KIND>()) compact_gather_kernel(const CompactParams p) {
    using R = Rec<KIND, NG>;
    __shared__ const uint8_t* rec[kBs];
    __shared__ int off[kBs];
    __shared__ bool host[kBs];
    pdl_wait();
    const int tid = threadIdx.x;
    const int b = blockIdx.z, j = blockIdx.x;
    if (j >= p.new_max_blocks) return;
    const int n = p.new_lens[b];   // these three are under way at once
    const int to = p.new_table[static_cast<int64_t>(b) * p.new_max_blocks + j];
    const uint32_t from = tid < kBs ? p.source[(static_cast<int64_t>(b) * p.max_blocks + j) * kBs + tid] : 0;
    if (static_cast<int64_t>(j) * kBs >= n) return;
    if (to < 0 || to >= p.num_blocks + p.host_blocks || p.claim[to] != 2u) {   // no block, or not this one's alone
        if (tid == 0 && blockIdx.y == 0) report(p.err, KVD_ERR_OOB);
        return;
    }
    if (tid == 0 && blockIdx.y == 0 && p.retain) p.retain[to] = 0xffffu;   // `to` is no source: nobody reads its mask
    auto record = [&](int64_t id) -> uint8_t* {   // of the first layer and head
        return id < p.num_blocks ? p.kv + id * p.n_kv * R::kBytes : p.host_kv + (id - p.num_blocks) * p.n_kv * R::kBytes;
    };
    if (tid < kBs) {
        const int64_t id = from / kBs;
        rec[tid] = from == kNoSource ? nullptr : record(id);
        off[tid] = static_cast<int>(from % kBs);
        host[tid] = id >= p.num_blocks;
    }
    __syncthreads();
    uint8_t* const first = record(to);
    const int pairs = p.L * p.n_kv;
    #pragma unroll 1
    for (int i = blockIdx.y; i < pairs; i += gridDim.y) {
        const int64_t layer = i / p.n_kv, h = i % p.n_kv;
        const Sources s{rec, off, host, (layer * p.num_blocks * p.n_kv + h) * R::kBytes,
                        (layer * p.host_blocks * p.n_kv + h) * R::kBytes};
        uint4* out = reinterpret_cast<uint4*>(first + (to < p.num_blocks ? s.device_pair : s.host_pair));
        #pragma unroll
        for (int c0 = 0; c0 < R::kPieces; c0 += gather_threads<KIND>())
            if (c0 + tid < R::kPieces) out[c0 + tid] = gather_piece<KIND, NG>(s, c0 + tid);
    }
}

template <int KIND, int NG>
cudaError_t launch_gather(const CompactParams& p, dim3 grid, cudaStream_t stream) {
    return launch_dependent(compact_gather_kernel<KIND, NG>, grid, dim3(gather_threads<KIND>()), 0, -1, stream, p);
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, int kind, int ng, int num_sms, cudaStream_t stream) {
    cudaError_t e = launch_dependent(compact_rank_kernel, dim3(static_cast<unsigned>(p.B)), dim3(kRankThreads), 0, -1,
                                     stream, p);
    if (e != cudaSuccess) return e;
    const dim3 claims(static_cast<unsigned>((p.max_blocks + kRankThreads - 1) / kRankThreads), static_cast<unsigned>(p.B));
    e = launch_dependent(compact_claim_kernel, claims, dim3(kRankThreads), 0, -1, stream, p);
    if (e != cudaSuccess) return e;
    const int pairs = p.L * p.n_kv;
    // Eight shares of the (layer, KV head) pairs a block; more where the blocks alone leave SMs without their
    // eight CTAs: a share is a chain of loads and stores.
    const int64_t blocks = static_cast<int64_t>(p.max_blocks) * p.B;
    const int64_t want = (8 * static_cast<int64_t>(num_sms) + blocks - 1) / blocks;
    const int64_t shares = min(static_cast<int64_t>(pairs), max(want, static_cast<int64_t>(8)));
    const dim3 grid(static_cast<unsigned>(p.max_blocks), static_cast<unsigned>(shares), static_cast<unsigned>(p.B));
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
