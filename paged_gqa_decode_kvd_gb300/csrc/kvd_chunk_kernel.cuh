// kvd_chunk_kernel.cuh — causal attention of a chunk of new tokens over the paged cache: the kernel
// template shared by the translation units that instantiate its pool kinds.
//
// Row (token i of the T new tokens of request b, query head h): with len = seq_lens[b] and
// position P = len − T + i,
//   l_t = softmax_scale · q·K_t for t ≤ P (−inf where slot t is evicted),
//   out = Σ_t softmax(l)_t · V_t,  lse = log Σ_t exp(l_t).
//
// Work.  A unit is (request, KV head, TQ = ⌊256/g⌋ new tokens): up to 256 rows (token, head of the
// group) that share every K and V.  Its cost is its tiles of 64 positions up to its last row's, and a few
// tiles' time for its start and end.  The units' costs, laid end to end, are cut into equal shares, one per CTA
// (one CTA per SM), so every CTA does the same work whatever the batch holds; a unit cut by a border leaves
// fp32 partials (unnormalised sum, maximum, sum of weights) that chunk_combine_kernel joins.
//
// One CTA, 20 warps:
//  * producer warp: follows the block table and bulk-copies (TMA engine) the four 16-token records
//    of a tile into a raw ring;
//  * two repack warpgroups, one for K and one for V: turn the records' mma.m16n8k16 fragment order into the
//    128-byte-swizzled K-major operands the tensor cores read, by 16-byte shared loads and stores and register
//    renaming only.  A K piece holds four dims of tokens t and t + 8: two pieces give eight dims of each, so
//    the operand's dims stand in the order 32j + {2x, 2x+1, 2x+8, 2x+9, 16 + the same} (q is laid
//    out alike, the product does not care).  A V piece holds four tokens of dims r and r + 8: the pieces
//    of two blocks give eight tokens of each, which fixes the order of a tile's 64 columns:
//    column 32p + 8x + 4u + w = token 2x + (w & 1) + 8(w >> 1) of block 2p + u.  8-bit codes become
//    bf16 exactly on the way; a low-bit code becomes the fp32 value code·scale + zero as two bf16, each in an operand
//    of its own (rounded once, outputs whose terms cancel would be off by more than the decode's tolerance);
//  * two warps that issue S = Q·K^T, one for each softmax warpgroup, and one that issues O += P·V for both; Q, K and V
//    from shared memory, P and the accumulators in tensor memory;
//  * two softmax warpgroups, one thread a row: online softmax in fp32 (exp2 domain), P back to tensor
//    memory, over the S it came from, as two bf16, its leading bits and the remainder (two products: a weight is off
//    by 2^-16; rounded once, by 2^-8, an output whose terms cancel would be off by more than the tolerance of the
//    decode's outputs, 2e-3 + 1e-2 of the value).  A warpgroup has two S: the next is ready when a step ends, so a step
//    has one wait and one arrival.  The reference maximum moves only when a row's maximum passes it by 8
//    (weights up to 2^8), so O is rarely rescaled.
// With more than 128 rows the warpgroups take 128 rows each and share every tile; with fewer they
// take the even and the odd tiles of the same rows and are merged at the unit's end.
//
// Waits.  Each barrier's waiter is at most one phase behind it: a tile's stages, its S and its P are handed on in
// order, and where a warpgroup might be ahead or behind (tiles of one warpgroup only, a segment's end) it waits for
// the phase before first.  Every wait gives up after a second or so; the kernel then reports it and ends.
//
// Bound, BF16, 32 + 8 heads: 2,048 tokens behind 8,192 take 341 us, 906 TFLOP/s (48% of the measured matrix rate; with P's
// second product the tensor pipe is 64% busy).  A tile of 256 rows takes about 2,400 cycles: the MMAs 1,800 (S 768, bound
// by its operands in shared memory, and twice 512 for the two products with V).  In a graph, 331 us: without its repack it
// would take 317, without its exponentials 328: no one role stands out.  32 × 5 tokens behind 8,187 stream the cache at
// 5.1 TB/s (76% of the measured bandwidth).
// The other pool kinds take, one call on a cold cache (BF16: 326 us): FP8 383, angle 434, mixed 542, INT4 832, INT2 839 (a
// second operand for K and for V doubles their repack).
//
// 8-bit records: the K scale multiplies the fp32 logit, the V scale the fp32 weight before it is
// rounded, so codes enter the MMAs exactly.  Angle-domain keys: q enters as its direction code, with
// ||q||/||d_q|| in the row's scale and the key's factor in the column's.
//
// Masked positions: logits become −inf by selection and V is zeroed, so what a slot holds does not
// matter.  Inside the chunk a token's V is attended by later rows and masked for earlier ones, and
// 0·NaN would reach the earlier ones: non-finite V there is zeroed too, noted, and added at the end
// to the rows that attend it.  An 8-bit V whose scale is not finite (its token held an infinity: every code is zero
// or NaN, every product NaN) is left out everywhere and makes NaN of the rows that attend it.
#pragma once

#include "kvd_chunk.h"
#include "kvd_tcgen.cuh"

namespace kvd {
namespace chunk {

constexpr int kTile = 64;              // positions per tile: four blocks
constexpr int kWgRows = 128;           // rows of one MMA (tensor memory lanes)
constexpr int kUnitRows = 2 * kWgRows;
constexpr int kThreads = 640;          // softmax 2 × 128, repack of K 128, of V 128, producer 32, S 2 × 32, O 32
constexpr int kKeyWarp = 8, kValueWarp = 12, kProducerWarp = 16, kScoreWarp = 17, kOutWarp = 19;
constexpr int kOpBytes = 16384;
constexpr float kLazy = 8.f;           // log2: how far a row's maximum may pass its reference
constexpr uint64_t kWaitNs = 1000000000ull;   // of what must land before the block leaves
constexpr int kTries = 200000;         // tries of a wait, which suspend: a second or so (a clock read a try costs more than the wait)
constexpr int kColS = 0, kColO = 256;   // tensor memory columns: S and P 2 × 2 × 64, O 2 × 128
// Smallest share of a CTA.  In a graph, four tokens behind 1,019 take 31.4, 21.8, 24.8, 18.6, 23.7, 19.7 us with 1, 2, 3,
// 4, 6, 8: a smaller share leaves more parts to join, and a share that does not divide the units leaves two parts a CTA.
constexpr int kMinTiles = 4;
// What a unit costs beside its tiles (its Q, its first S, its rows out), in tiles.  A serving batch (units of 1 to 260
// tiles) takes 711, 530, 440, 404, 416, 441 us with 0, 2, 4, 6, 8, 12; a whole prompt of 8,192 711, 660, 617, 603, 608, 619.
constexpr int kUnitTiles = 6;
// P as two bf16: the weight times this, cut to 16 bits, is below the weight (by a step where 16 bits hold it, else by
// less), and the remainder, rounded, is off by half a step of what has at most 8 bits less: 2^-16 of the weight.  Neither
// term is zero or negative unless the weight is zero (or nearly: below 2^-104), so an infinity in V that every row
// attends stays one (a rounded weight's remainder would have either sign, and make NaN of it).
constexpr float kBelow = 1.f - 0x1p-22f;
constexpr uint32_t kStop = 0x80000000u;   // block word behind the last tile

constexpr bool has_factors(int kind) { return kind == kKindFp8 || kind == kKindMixed || kind == kKindAngle; }
// A raw slot holds a tile's four records.
constexpr int max_record(int kind) {
    return kind == kKindBf16 || kind == kKindMixed ? kRecordBf16
           : kind == kKindInt4                     ? lowbit_record_bytes(4, 4)
           : kind == kKindInt2                     ? lowbit_record_bytes(2, 4)
                                                   : kRecordFp8;
}
constexpr bool is_wide(int kind) { return kind == kKindBf16 || kind == kKindMixed; }
// What fits beside Q: raw tiles, and operand stages of 16 KiB (32 KiB low-bit) for K and for V.  A tile's masks and factors are
// read until its P is there.  K may be as far ahead as the stages' tiles behind the other S that a warpgroup has
// been given before: with a warpgroup on every second tile, four tiles and the stages.
constexpr int raw_tiles(int kind) { return kind == kKindMixed ? 2 : 3; }
// Low-bit values have two operands, the rounded value and the rounded remainder.
constexpr int op_parts(int kind) { return is_lowbit(kind) ? 2 : 1; }
constexpr int op_stages(int kind) { return is_wide(kind) || is_lowbit(kind) ? 2 : 3; }
constexpr int info_sets(int kind) { return op_stages(kind) == 2 ? 6 : 8; }

struct TileInfo {
    alignas(16) float limit[kTile];   // column: −inf where the position may not be attended, else +inf
    unsigned long long mask;          // bit 16·block + t: position may be attended
    unsigned long long nonfin[4];     // by repack warp; column n: its V has non-finite elements, zeroed in the operand
    unsigned long long wild;          // like mask: the V factor is not finite, and zero in the table
};
constexpr int kFlags = 5;           // tiles that hold positions of a unit's own tokens: ⌈(63 + 256)/64⌉

struct Request {
    int s0, T, len;   // first row, new tokens, context (−1: bad length, nothing is attended)
};
struct WalkState {
    int64_t remaining;
    int b, h, qt, off, extra;
    Request r;
};

template <int KIND>
struct Smem {
    static constexpr int kStages = op_stages(KIND), kRaw = raw_tiles(KIND), kInfos = info_sets(KIND);
    uint8_t k[kStages][op_parts(KIND) * kOpBytes], v[kStages][op_parts(KIND) * kOpBytes];   // operands; 1,024-byte aligned
    uint8_t q[2][2 * kOpBytes];                                 // 128 rows each
    uint8_t raw[kRaw][4][max_record(KIND)];
    alignas(16) float factor[has_factors(KIND) ? kInfos : 1][2][has_factors(KIND) ? kTile : 1];   // column: K factor, V factor
    TileInfo info[kInfos];
    uint32_t word[kRaw][4];                                     // block words
    WalkState walks[8];                                         // by softmax warp: it has no registers to spare
    unsigned long long flags[8][kFlags];                        // by softmax warp: nonfin of the unit's last tiles
    uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];         // [warpgroup][S and P buffer]
    uint64_t q_ready[2], q_one, merge_full, merge_empty, drain[3];
    int64_t remaining;   // the CTA's share of the schedule: length, first unit, and where in it, see Walk
    int b, h, qt, off, extra;
    uint32_t tmem, tiles;   // tiles: of all segments, when the producer is through
    int abort;
    // the merge of the two warpgroups: WG 1's maximum and sum, where no query of its own is
    __device__ __forceinline__ float* ml() { return reinterpret_cast<float*>(q[1]); }
};

// ------------------------------------------------------------------ schedule
// Σ_{i<n} ⌊(a·i + c)/64⌋: the sum without the floors less that of the remainders, which repeat every 64 terms
// (64/d values d apart, d = gcd(a, 64), each d times).
__device__ inline int64_t tile_sum(int64_t n, int a, int64_t c) {
    static_assert(kTile == 64, "the period of the remainders");
    const int low = a & 63, d = low ? low & -low : 64;
    int64_t rest = (n >> 6) * (64 * (c & (d - 1)) + 32 * (64 - d));
    uint32_t at = static_cast<uint32_t>(c);
    if (low == 0) rest += (n & 63) * (at & 63u);
    else for (int i = 0; i < static_cast<int>(n & 63); ++i, at += low) rest += at & 63u;
    return (a * (n * (n - 1) / 2) + c * n - rest) >> 6;
}

__device__ __forceinline__ Request load_request(const ChunkParams& p, int b, bool tell) {
    Request r;
    r.s0 = p.q_start[b];
    const int s1 = p.q_start[b + 1], len = p.seq_lens[b];
    r.T = 0;
    r.len = -1;
    if (r.s0 < 0 || s1 < r.s0 || s1 > p.n_tokens) {
        if (tell) report(p.err, KVD_ERR_OOB);
        return r;
    }
    r.T = s1 - r.s0;
    if (r.T == 0) return r;
    r.len = len;
    if (r.len < r.T || static_cast<int64_t>(r.len) > static_cast<int64_t>(p.max_blocks) * kBs) {
        if (tell) report(p.err, KVD_ERR_OOB);
        r.len = -1;
    }
    return r;
}
__device__ __forceinline__ int unit_end(const Request& r, int qt, int tq) {   // positions the unit attends
    return r.len < 0 ? 0 : r.len - r.T + min((qt + 1) * tq, r.T);
}
__device__ __forceinline__ int unit_tiles(const Request& r, int qt, int tq) {
    return r.len < 0 ? 1 : (unit_end(r, qt, tq) + kTile - 1) / kTile;
}
__device__ inline int64_t tiles_before(const Request& r, int k, int tq) {   // tiles of units 0 .. k-1 of one head
    if (r.len < 0) return k;
    const int n = (r.T + tq - 1) / tq;
    const int whole = min(k, n - 1);
    int64_t s = tile_sum(whole, tq, static_cast<int64_t>(r.len) - r.T + tq + kTile - 1);
    if (k == n) s += unit_tiles(r, n - 1, tq);
    return s;
}

struct Segment {
    int b, h, qt;
    int t0, t1, tiles;       // this CTA's tiles of the unit's
    int s0, T, len;
    int end;                 // positions the unit attends
    int first;               // position of its first row
    int tok0, rows;
    bool two;                // the warpgroups take 128 rows each
};

// The CTA's segments in order; every role walks them on its own.  A unit takes `extra` + tiles of the schedule's
// length, its tiles last: a share that ends before them has none of it.
struct Walk : WalkState {
    template <class S>
    __device__ __forceinline__ Walk(const ChunkParams& p, const S& s)
        : WalkState{s.remaining, s.b, s.h, s.qt, s.off, s.extra, Request{0, 0, -1}} {
        if (remaining > 0) r = load_request(p, b, false);
    }
    __device__ __forceinline__ explicit Walk(const WalkState& w) : WalkState(w) {}
    __device__ __forceinline__ bool next(const ChunkParams& p, Segment& g) {
        if (remaining <= 0) return false;
        const int tq = kUnitRows / p.g;
        g.b = b;
        g.h = h;
        g.qt = qt;
        g.tiles = unit_tiles(r, qt, tq);
        const int take = static_cast<int>(min(static_cast<int64_t>(g.tiles) + extra - off, remaining));
        g.t0 = max(off - extra, 0);
        g.t1 = off + take - extra;
        g.s0 = r.s0;
        g.T = r.T;
        g.len = r.len;
        g.end = unit_end(r, qt, tq);
        g.tok0 = qt * tq;
        g.first = r.len < 0 ? -1 : r.len - r.T + g.tok0;
        g.rows = min(tq, r.T - g.tok0) * p.g;
        g.two = g.rows > kWgRows;
        remaining -= take;
        off = 0;
        if (remaining > 0) {
            if (++qt * tq >= r.T) {
                qt = 0;
                if (++h == p.n_kv) {
                    h = 0;
                    do {
                        if (++b >= p.B) {
                            remaining = 0;
                            break;
                        }
                        r = load_request(p, b, false);
                    } while (r.T == 0);
                }
            }
        }
        return g.t1 > g.t0;
    }
};

// A CTA's share of the schedule, by every thread of the block; scratch holds 2·p.B int64.
template <class S>
__device__ inline void make_schedule(const ChunkParams& p, S& s, int64_t* scratch) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int tq = kUnitRows / p.g;
    for (int b = tid; b < p.B; b += kThreads) {
        const Request r = load_request(p, b, blockIdx.x == 0);
        const int units = (r.T + tq - 1) / tq;
        scratch[2 * b] = r.T ? tiles_before(r, units, tq) * p.n_kv : 0;
        scratch[2 * b + 1] = static_cast<int64_t>(units) * p.n_kv;
    }
    __syncthreads();
    if (tid < 32) {
        int64_t tiles = 0, units = 0;
        for (int b = lane; b < p.B; b += 32) {
            tiles += scratch[2 * b];
            units += scratch[2 * b + 1];
        }
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            tiles += __shfl_xor_sync(kFull, tiles, o);
            units += __shfl_xor_sync(kFull, units, o);
        }
        // a small call is cut into its smallest shares; there the border must not fall beside the tiles
        const int extra = static_cast<int>(min(static_cast<int64_t>(kUnitTiles), tiles / (8 * gridDim.x)));
        const int64_t total = tiles + units * extra;
        const int64_t most = (total + kMinTiles - 1) / kMinTiles;
        const int64_t ctas = most < gridDim.x ? (most < 1 ? 1 : most) : gridDim.x;
        const int64_t lo = blockIdx.x < ctas ? total * blockIdx.x / ctas : 0;
        const int64_t hi = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : 0;
        if (lane == 0) {
            s.remaining = hi - lo;
            s.extra = extra;
        }
        int64_t before = 0;
        for (int b0 = 0; hi > lo && b0 < p.B; b0 += 32) {
            const int64_t c = b0 + lane < p.B ? scratch[2 * (b0 + lane)] + extra * scratch[2 * (b0 + lane) + 1] : 0;
            int64_t up = c;
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(kFull, up, o);
                if (lane >= o) up += v;
            }
            up += before;
            const unsigned at = __ballot_sync(kFull, lo >= up - c && lo < up);
            if (at) {
                const int src = __ffs(at) - 1, b = b0 + src;
                const int64_t cost = __shfl_sync(kFull, c, src), from = __shfl_sync(kFull, up, src) - cost;
                const Request r = load_request(p, b, false);
                const int64_t head = cost / p.n_kv, rem = lo - from;
                const int h = static_cast<int>(rem / head);
                const int64_t in = rem - h * head;
                int a = 0, z = (r.T + tq - 1) / tq;   // the last unit of [a, z) that starts at or before `in`
                while (z - a > 1) {
                    const int step = (z - a + 31) / 32, mid = a + lane * step;
                    const bool at_or_before = mid < z && tiles_before(r, mid, tq) + static_cast<int64_t>(mid) * extra <= in;
                    const int n = __popc(__ballot_sync(kFull, at_or_before));
                    a += (n - 1) * step;
                    z = min(z, a + step);
                }
                if (lane == 0) {
                    s.b = b;
                    s.h = h;
                    s.qt = a;
                    s.off = static_cast<int>(in - tiles_before(r, a, tq) - static_cast<int64_t>(a) * extra);
                }
            }
            before = __shfl_sync(kFull, up, 31);
            if (before > lo) break;
        }
    }
}

// ------------------------------------------------------------------- repack
// Column of token t of block k of a tile, and the position within the tile of a column.
__host__ __device__ constexpr int column_of(int k, int t) {
    return 32 * (k >> 1) + 8 * ((t & 7) >> 1) + 4 * (k & 1) + (t & 1) + 2 * (t >> 3);
}
__host__ __device__ constexpr int place_of(int n) {
    return 16 * (2 * (n >> 5) + ((n >> 2) & 1)) + 2 * ((n >> 3) & 3) + (n & 1) + 8 * ((n >> 1) & 1);
}

__device__ __forceinline__ void put16(uint8_t* base, int row, int piece, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    *reinterpret_cast<uint4*>(base + row * 128 + ((piece ^ (row & 7)) << 4)) = make_uint4(a, b, c, d);
}
__device__ __forceinline__ void put_k(uint8_t* op, int n, int j, int x, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    put16(op + (j >> 1) * 8192, n, 4 * (j & 1) + x, a, b, c, d);
}

__device__ __forceinline__ uint32_t pair_mask(uint32_t m, int t) {
    return ((m >> t & 1u) ? 0xffffu : 0u) | ((m >> (t + 1) & 1u) ? 0xffff0000u : 0u);
}
// Whether a pair of bf16 has an infinity or a NaN (in the top bits of its halves).
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// V words of a lane, one dim: tokens (2x, 2x+1), (2x+8, 2x+9) of blocks 2p and 2p+1; masked tokens are zeroed
// and, where rows of the unit differ in which they attend, non-finite elements zeroed and noted.
struct VPut {
    uint8_t* op;
    uint32_t keep[4];          // the lane's valid bits, by word
    unsigned long long bad;    // columns with non-finite elements
    bool whole;                // every position of the tile is valid
    bool look;                 // the tile holds positions some rows attend and others do not
    __device__ __forceinline__ VPut(uint8_t* o, const uint32_t (&word)[4], bool l, int lane) : op(o), bad(0), look(l) {
        whole = (word[0] & word[1] & word[2] & word[3] & 0xffffu) == 0xffffu;
        const int x = lane & 3;
        const uint32_t m0 = (lane & 4) ? word[2] : word[0], m1 = (lane & 4) ? word[3] : word[1];
        keep[0] = pair_mask(m0, 2 * x);
        keep[1] = pair_mask(m0, 2 * x + 8);
        keep[2] = pair_mask(m1, 2 * x);
        keep[3] = pair_mask(m1, 2 * x + 8);
    }
    // Dim d, columns 32p + 8x + 0 .. 7, element by element.
    __device__ __forceinline__ void put(int d, int lane, uint32_t a, uint32_t b, uint32_t c, uint32_t e) {
        const int x = lane & 3, p = (lane >> 2) & 1;
        uint32_t w[4] = {a & keep[0], b & keep[1], c & keep[2], e & keep[3]};
        if (look) {
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t n = nonfinite(w[i]);
                if (n & 0x8000u) bad |= 1ull << (32 * p + 8 * x + 2 * i);
                if (n & 0x80000000u) bad |= 2ull << (32 * p + 8 * x + 2 * i);
                w[i] &= ~((n & 0x8000u ? 0xffffu : 0u) | (n & 0x80000000u ? 0xffff0000u : 0u));
            }
        }
        put16(op, d, 4 * p + x, w[0], w[1], w[2], w[3]);
    }
};

// Four 8-bit codes -> two packed bf16 pairs, exact for numbers.  An E4M3 (E5M2) code is moved into a bf16's
// sign, exponent and mantissa bits and scaled by 2^120 (2^112), the difference of the exponent biases.
// `special` collects codes that are no numbers: those go through the conversion instruction (any_code_to_bf16).
template <int FMT>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi, uint32_t& special) {
    constexpr uint32_t kBits = FMT == kFmtE5m2 ? 0x0fe00fe0u : 0x07f007f0u;
    constexpr int kShift = FMT == kFmtE5m2 ? 3 : 4;
    constexpr uint32_t kUp = FMT == kFmtE5m2 ? 0x77807780u : 0x7b807b80u;
    special |= FMT == kFmtE5m2 ? (w & 0x7c7c7c7cu) + 0x04040404u : (w & 0x7f7f7f7fu) + 0x01010101u;
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
    uint32_t pa = ((a >> kShift) & kBits) | (a & 0x80008000u), pb = ((b >> kShift) & kBits) | (b & 0x80008000u);
    const uint32_t up = kUp;
    const __nv_bfloat162 u = *reinterpret_cast<const __nv_bfloat162*>(&up);
    __nv_bfloat162 ra = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&pa), u);
    __nv_bfloat162 rb = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&pb), u);
    lo = *reinterpret_cast<uint32_t*>(&ra);
    hi = *reinterpret_cast<uint32_t*>(&rb);
}
template <int FMT>
__device__ __forceinline__ void any_code_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    uint32_t a, b;
    f8x4_to_f16x2x2<FMT>(w, a, b);
    const float2 x = unpack_f16(a), y = unpack_f16(b);
    lo = pack_bf16(x.x, x.y);
    hi = pack_bf16(y.x, y.y);
}

// A lane's byte offsets, the same for every tile; [q] for the even and the odd pieces.  K: the warp's block; V: the
// warp's 32 dims of all four blocks.  Lanes of an eight read one 64-byte half each and write all eight pieces of
// two rows' 128-byte lines, so neither side has bank conflicts.
struct Offsets {
    int k_ld[2], k_st[2][2];   // [q] (16-bit records: twice the part before the + of the 8-bit ones), [q][token t, t + 8]
    int v_ld[2], v_st[2];
    int k_half, v_warp;        // the parts that differ between 16- and 8-bit records
    __device__ __forceinline__ Offsets(int warp, int lane) {
        const int x = lane & 3, h = (lane >> 2) & 1, l = lane >> 3;
        k_half = h * 512;
        v_warp = warp * 512;
        #pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = 2 * l + (q ^ h);   // K: token (mod 8); V: dim (mod 8)
            const int n = column_of(warp, t);
            k_ld[q] = (4 * t + x) * 16;
            k_st[q][0] = n * 128 + (((4 * h + x) ^ (n & 7)) << 4);
            k_st[q][1] = (n + 2) * 128 + (((4 * h + x) ^ ((n + 2) & 7)) << 4);
            v_ld[q] = (4 * t + x) * 16;
            v_st[q] = warp * 4096 + t * 128 + (((4 * h + x) ^ t) << 4);
        }
    }
};

__device__ __forceinline__ uint4 ld16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(uint8_t* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}

// K of one block (codes) by one warp, every load before the stores.
template <int FMT>
__device__ __forceinline__ void repack_k(const uint8_t* code, uint8_t* op, const Offsets& o) {
    if constexpr (FMT == kFmtBf16) {
        #pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint4 a[2], b[2];
            #pragma unroll
            for (int q = 0; q < 2; ++q) {
                a[q] = ld16(code + 2 * o.k_half + o.k_ld[q] + j * 2048);
                b[q] = ld16(code + 2 * o.k_half + o.k_ld[q] + j * 2048 + 512);
            }
            #pragma unroll
            for (int q = 0; q < 2; ++q) {
                st16(op + o.k_st[q][0] + j * 8192, a[q].x, a[q].z, b[q].x, b[q].z);
                st16(op + o.k_st[q][1] + j * 8192, a[q].y, a[q].w, b[q].y, b[q].w);
            }
        }
    } else {
        uint4 a[4];
        uint32_t special = 0;
        #pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = ld16(code + o.k_half + o.k_ld[i & 1] + (i >> 1) * 1024);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo[4], hi[4];
            codes_to_bf16<FMT>(a[i].x, lo[0], hi[0], special);
            codes_to_bf16<FMT>(a[i].y, lo[1], hi[1], special);
            codes_to_bf16<FMT>(a[i].z, lo[2], hi[2], special);
            codes_to_bf16<FMT>(a[i].w, lo[3], hi[3], special);
            st16(op + o.k_st[i & 1][0] + (i >> 1) * 8192, lo[0], lo[1], lo[2], lo[3]);
            st16(op + o.k_st[i & 1][1] + (i >> 1) * 8192, hi[0], hi[1], hi[2], hi[3]);
        }
        if (special & 0x80808080u) {   // rare
            #pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const uint4 c = ld16(code + o.k_half + o.k_ld[0] + (i & 1) * (o.k_ld[1] - o.k_ld[0]) + (i >> 1) * 1024);
                const int s0 = i & 1 ? o.k_st[1][0] : o.k_st[0][0], s1 = i & 1 ? o.k_st[1][1] : o.k_st[0][1];
                uint32_t lo[4], hi[4];
                any_code_to_bf16<FMT>(c.x, lo[0], hi[0]);
                any_code_to_bf16<FMT>(c.y, lo[1], hi[1]);
                any_code_to_bf16<FMT>(c.z, lo[2], hi[2]);
                any_code_to_bf16<FMT>(c.w, lo[3], hi[3]);
                st16(op + s0 + (i >> 1) * 8192, lo[0], lo[1], lo[2], lo[3]);
                st16(op + s1 + (i >> 1) * 8192, hi[0], hi[1], hi[2], hi[3]);
            }
        }
    }
}

// A V piece of two dims as bf16: group i (dims 16i + r and 16i + r + 8), lane 4r + x: tokens
// (2x, 2x+1) of dim r, of dim r + 8, tokens (2x+8, 2x+9) of dim r, of dim r + 8.
template <int FMT>
__device__ __forceinline__ uint4 v_piece(const uint8_t* code, int i, int l) {
    if constexpr (FMT == kFmtBf16) {
        return ld16(code + (i * 32 + l) * 16);
    } else {
        const uint2 a = *reinterpret_cast<const uint2*>(code + ((i >> 1) * 32 + l) * 16 + (i & 1) * 8);
        uint4 o;
        any_code_to_bf16<FMT>(a.x, o.x, o.y);
        any_code_to_bf16<FMT>(a.y, o.z, o.w);
        return o;
    }
}
template <int KIND>
__device__ __forceinline__ uint4 v_piece_kind(const uint8_t* rec, uint32_t word, int i, int l) {
    if constexpr (KIND == kKindBf16) {
        return v_piece<kFmtBf16>(rec + kTileBf16, i, l);
    } else if constexpr (KIND == kKindMixed) {
        const int f = (word >> 17) & 3u;
        return f == kFmtBf16 ? v_piece<kFmtBf16>(rec + kTileBf16, i, l)
               : f == kFmtE4m3 ? v_piece<kFmtE4m3>(rec + kTileFp8, i, l) : v_piece<kFmtE5m2>(rec + kTileFp8, i, l);
    } else {
        return v_piece<kFmtE4m3>(rec + kTileFp8, i, l);
    }
}

// V of the tile, 32 dims by one warp; pair: the lane's two blocks' codes.  MASK: some position is not valid; LOOK:
// non-finite elements matter.  Returns whether the lane met something that wants the element-wise path.
template <int KIND, bool MASK, bool LOOK>
__device__ __forceinline__ bool repack_v_fast(const uint8_t* pair, const VPut& out, const Offsets& o) {
    constexpr int kNext = max_record(KIND);
    const uint8_t* code = pair + (KIND == kKindBf16 ? kTileBf16 : kTileFp8);
    uint32_t odd = 0, special = 0;
    auto put = [&](uint8_t* to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        if constexpr (MASK) {
            a &= out.keep[0];
            b &= out.keep[1];
            c &= out.keep[2];
            d &= out.keep[3];
        }
        if constexpr (LOOK) odd |= nonfinite(a) | nonfinite(b) | nonfinite(c) | nonfinite(d);
        st16(to, a, b, c, d);
    };
    if constexpr (KIND == kKindBf16) {
        #pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint4 a[2], b[2];
            #pragma unroll
            for (int q = 0; q < 2; ++q) {
                a[q] = ld16(code + 2 * o.v_warp + o.v_ld[q] + j * 512);
                b[q] = ld16(code + 2 * o.v_warp + o.v_ld[q] + j * 512 + kNext);
            }
            #pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint8_t* to = out.op + o.v_st[q] + j * 2048;
                put(to, a[q].x, a[q].z, b[q].x, b[q].z);
                put(to + 1024, a[q].y, a[q].w, b[q].y, b[q].w);
            }
        }
    } else {
        uint4 a[2], b[2];
        #pragma unroll
        for (int q = 0; q < 2; ++q) {
            a[q] = ld16(code + o.v_warp + o.v_ld[q]);
            b[q] = ld16(code + o.v_warp + o.v_ld[q] + kNext);
        }
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = i & 1;
            uint32_t lo[4], hi[4];
            codes_to_bf16<kFmtE4m3>(i >> 1 ? a[q].z : a[q].x, lo[0], hi[0], special);
            codes_to_bf16<kFmtE4m3>(i >> 1 ? a[q].w : a[q].y, lo[1], hi[1], special);
            codes_to_bf16<kFmtE4m3>(i >> 1 ? b[q].z : b[q].x, lo[2], hi[2], special);
            codes_to_bf16<kFmtE4m3>(i >> 1 ? b[q].w : b[q].y, lo[3], hi[3], special);
            uint8_t* to = out.op + o.v_st[q] + (i >> 1) * 2048;
            put(to, lo[0], lo[1], lo[2], lo[3]);
            put(to + 1024, hi[0], hi[1], hi[2], hi[3]);
        }
    }
    return odd != 0 || (special & 0x80808080u) != 0;
}
template <int KIND>
__device__ __forceinline__ void repack_v(const uint8_t* pair, const uint32_t (&word)[4], VPut& out, const Offsets& o, int warp,
                                         int lane) {
    if constexpr (KIND != kKindMixed) {
        bool slow;
        if (out.look) slow = repack_v_fast<KIND, true, true>(pair, out, o);
        else if (!out.whole) slow = repack_v_fast<KIND, true, false>(pair, out, o);
        else slow = repack_v_fast<KIND, false, false>(pair, out, o);
        if (!__any_sync(kFull, slow)) return;
    }
    const int x = lane & 3, p = (lane >> 2) & 1, rl = lane >> 3;
    #pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const int group = 2 * warp + (i >> 1), r = 2 * rl + ((i & 1) ^ p);
        const uint4 a = v_piece_kind<KIND>(pair, word[2 * p], group, 4 * r + x);
        const uint4 b = v_piece_kind<KIND>(pair + max_record(KIND), word[2 * p + 1], group, 4 * r + x);
        out.put(16 * group + r, lane, a.x, a.z, b.x, b.z);
        out.put(16 * group + r + 8, lane, a.y, a.w, b.y, b.w);
    }
}

// Low-bit codes: values fp32(code·scale + zero), as bf16 and the bf16 of what is left.
struct LowPair {
    uint32_t hi, lo;
};
template <int BITS>
__device__ __forceinline__ LowPair low_pair(uint32_t word, int h, int j, float2 sz0, float2 sz1) {
    const uint32_t c0 = word >> (8 * j + BITS * h) & ((1u << BITS) - 1), c1 = word >> (8 * (j + 1) + BITS * h) & ((1u << BITS) - 1);
    const float a = fmaf(static_cast<float>(c0), sz0.x, sz0.y), b = fmaf(static_cast<float>(c1), sz1.x, sz1.y);
    const uint32_t hi = pack_bf16(a, b);
    const float2 r = unpack_bf16(hi);
    return {hi, pack_bf16(a - r.x, b - r.y)};
}
template <int BITS>
__device__ __forceinline__ void repack_k_low(const uint8_t* rec, uint8_t* op, int k, int ng, int lane) {
    constexpr int kPer = 8 / BITS, kTileB = lowbit_tile_bytes(BITS);
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(rec + 2 * kTileB);
    const int x = lane & 3, r = lane >> 2;
    const int n = column_of(k, r);
    #pragma unroll
    for (int kg = 0; kg < 8 / kPer; ++kg) {
        #pragma unroll
        for (int th = 0; th < 2; ++th) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + lowbit_word(kg, lane, th) * 4);
            #pragma unroll
            for (int q = 0; q < kPer / 2; ++q) {   // 32 dims each: one group of the row
                const int j = kg * (kPer / 2) + q;
                const float2 sz = unpack_f16(meta[(r + 8 * th) * ng + j * ng / 4]);
                const LowPair a = low_pair<BITS>(w, 2 * q, 0, sz, sz), b = low_pair<BITS>(w, 2 * q, 2, sz, sz);
                const LowPair c = low_pair<BITS>(w, 2 * q + 1, 0, sz, sz), d = low_pair<BITS>(w, 2 * q + 1, 2, sz, sz);
                put_k(op, n + 2 * th, j, x, a.hi, b.hi, c.hi, d.hi);
                put_k(op + kOpBytes, n + 2 * th, j, x, a.lo, b.lo, c.lo, d.lo);
            }
        }
    }
}
template <int KIND, int BITS>
__device__ __forceinline__ void repack_v_low(const uint8_t* pair, VPut& out, int ng, int warp, int lane) {
    constexpr int kPer = 8 / BITS, kTileB = lowbit_tile_bytes(BITS);
    const int x = lane & 3, p = (lane >> 2) & 1, rl = lane >> 3;
    #pragma unroll 1
    for (int i = 0; i < 2; ++i) {   // eight groups of 16 dims: 2·warp and 2·warp + 1
        const int group = 2 * warp + i, kg = group / kPer, h = group % kPer;
        #pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = 2 * rl + (s ^ p);
            LowPair o[2][4];   // dims r, r + 8: tokens (2x, 2x+1), (2x+8, 2x+9) of blocks 2p, 2p+1
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* b = pair + u * max_record(KIND);
                const uint32_t* meta = reinterpret_cast<const uint32_t*>(b + 2 * kTileB) + kBs * ng;
                const int gi = group * ng / 8;
                #pragma unroll
                for (int th = 0; th < 2; ++th) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(b + kTileB + lowbit_word(kg, 4 * r + x, th) * 4);
                    const int t = 2 * x + 8 * th;
                    const float2 s0 = unpack_f16(meta[t * ng + gi]), s1 = unpack_f16(meta[(t + 1) * ng + gi]);
                    o[0][2 * u + th] = low_pair<BITS>(w, h, 0, s0, s1);
                    o[1][2 * u + th] = low_pair<BITS>(w, h, 2, s0, s1);
                }
            }
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = 16 * group + r + 8 * e;
                out.put(d, lane, o[e][0].hi, o[e][1].hi, o[e][2].hi, o[e][3].hi);
                put16(out.op + kOpBytes, d, 4 * p + x, o[e][0].lo & out.keep[0], o[e][1].lo & out.keep[1],
                      o[e][2].lo & out.keep[2], o[e][3].lo & out.keep[3]);
            }
        }
    }
}

// -------------------------------------------------------------------- pool
__device__ __forceinline__ const uint8_t* record_at(const ChunkParams& p, int64_t id, int h) {
    return id < p.num_blocks ? p.kv + (id * p.n_kv + h) * p.record_bytes
                             : p.stage + ((id - p.num_blocks) * p.n_kv + h) * p.record_bytes;
}

// Block word: bits 0-15 positions that may be attended, bit 16 the record is copied, bits 17-18 its
// format (mixed pools).
template <int KIND>
__device__ __forceinline__ uint32_t block_word_of(const ChunkParams& p, int phys, int j, int end) {
    if (phys < 0 || phys >= p.num_blocks + p.host_blocks) {
        report(p.err, KVD_ERR_OOB);
        return 0;
    }
    const int left = end - j * kBs;
    uint32_t m = left >= kBs ? 0xffffu : (1u << left) - 1u;
    if (p.retain) m &= p.retain[phys];
    int f = kFmtBf16;
    if constexpr (KIND == kKindMixed) {
        f = block_format(p.block_fmt[phys]);
        if (f < 0) {
            report(p.err, KVD_ERR_OOB);
            return 0;
        }
    }
    return m ? m | 0x10000u | static_cast<uint32_t>(f) << 17 : 0u;
}

// V of (position, dim) as attention reads it: only for positions with non-finite values.
template <int KIND>
__device__ __noinline__ float pool_value(const ChunkParams& p, int b, int h, int pos, int d) {
    const int phys = p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kBs];
    if (phys < 0 || phys >= p.num_blocks + p.host_blocks) return 0.f;
    const uint8_t* rec = record_at(p, phys, h);
    const int t = pos % kBs;
    int fl, fe;
    const int i = v_frag_i(t, d, &fl, &fe);
    if constexpr (is_lowbit(KIND)) {
        constexpr int kBits = KIND == kKindInt4 ? 4 : 2, kT = lowbit_tile_bytes(kBits);
        const uint32_t* meta = reinterpret_cast<const uint32_t*>(rec + 2 * kT) + kBs * p.ng;
        const float2 sz = unpack_f16(meta[t * p.ng + d * p.ng / kDh]);
        const uint32_t c = rec[kT + lowbit_v_byte(kBits, t, d)] >> (kBits * ((d / 16) % (8 / kBits))) & ((1 << kBits) - 1);
        return static_cast<float>(c) * sz.x + sz.y;
    } else {
        int f = KIND == kKindBf16 ? kFmtBf16 : kFmtE4m3;
        if constexpr (KIND == kKindMixed) f = block_format(p.block_fmt[phys]);
        if (f == kFmtBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(rec)[kBs * kDh + bf16_tile_index(i, fl, fe)]);
        const __half_raw v = __nv_cvt_fp8_to_halfraw(rec[kTileFp8 + fp8_tile_index(i, fl, fe)], f == kFmtE5m2 ? __NV_E5M2 : __NV_E4M3);
        return __half2float(__half(v)) * reinterpret_cast<const float*>(rec + 2 * kTileFp8)[kBs + t];
    }
}

// ------------------------------------------------------------------ the roles
// Wait of a whole warp for a barrier's phase; one answer for all its lanes.  A try suspends the warp for
// some 8,000 cycles at most and wakes within about 130, so the limit, a second or so, is a count of tries;
// reading the timer would add 700 cycles to every wait that is not over at once.
template <int KIND>
__device__ __forceinline__ bool wait_bar(Smem<KIND>& s, uint64_t* bar, uint32_t phase) {
    #pragma unroll 1
    for (int i = 0; i < kTries; ++i)
        if (__all_sync(kFull, mbar_try_wait(bar, phase & 1u))) return true;
    s.abort = 1;   // reported at the kernel's end
    return false;
}

// Two waits with one vote; the second only if `second`.
template <int KIND>
__device__ __forceinline__ bool wait_two(Smem<KIND>& s, uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, bool second = true) {
    #pragma unroll 1
    for (int i = 0; i < kTries; ++i) {
        const bool x = mbar_try_wait(a, pa & 1u), y = !second || mbar_try_wait(b, pb & 1u);
        if (__all_sync(kFull, x && y)) return true;
    }
    s.abort = 1;   // reported at the kernel's end
    return false;
}

template <int KIND>
__device__ __forceinline__ void producer(Smem<KIND>& s, const ChunkParams& p, int lane) {
    constexpr int kRaw = Smem<KIND>::kRaw;
    Walk walk(p, s);
    Segment g;
    uint32_t k = 0;
    bool ok = true;
    while (ok && walk.next(p, g)) {
        const int32_t* row = p.block_table + static_cast<int64_t>(g.b) * p.max_blocks;
        auto block_at = [&](int j) { return j < 4 * g.t1 && j * kBs < g.end ? row[j] : -1; };
        int phys = block_at(4 * g.t0 + lane);   // 32 blocks: eight tiles; the next eight's are fetched meanwhile
        for (int tb = g.t0; ok && tb < g.t1; tb += 8) {
            const int j = 4 * tb + lane;
            uint32_t word = 0;
            const uint8_t* rec = nullptr;
            bool host = false;
            if (j < 4 * g.t1 && j * kBs < g.end) {
                word = block_word_of<KIND>(p, phys, j, g.end);
                if (word) rec = record_at(p, phys, g.h);
                host = word && p.host_direct && phys >= p.num_blocks;
            }
            phys = block_at(j + 32);
            uint32_t bytes = 0;
            if (word && !host)
                bytes = KIND == kKindMixed && ((word >> 17) & 3u) != kFmtBf16 ? kRecordFp8 : static_cast<uint32_t>(p.record_bytes);
            uint32_t four = bytes + __shfl_xor_sync(kFull, bytes, 1);
            four += __shfl_xor_sync(kFull, four, 2);
            const int n = min(8, g.t1 - tb);
            for (int i = 0; i < n; ++i, ++k) {
                const uint32_t st = k % kRaw;
                ok = wait_bar(s, &s.raw_empty[st], k / kRaw + 1);
                if (!ok) break;
                const bool mine = (lane >> 2) == i;
                if (mine) s.word[st][lane & 3] = word;
                if (p.host_direct) {   // records in host memory: copied by the load path, the whole warp
                    unsigned hosts = __ballot_sync(kFull, mine && host);
                    fence_proxy_async_shared();
                    while (hosts) {
                        const int l = __ffs(hosts) - 1;
                        hosts &= hosts - 1;
                        const uint8_t* src = reinterpret_cast<const uint8_t*>(
                            __shfl_sync(kFull, reinterpret_cast<unsigned long long>(rec), l));
                        for (int c = lane; c < p.record_bytes / 16; c += 32)
                            cp_async16_g2s(s.raw[st][l & 3] + 16 * c, src + 16 * c);
                    }
                    cp_async_mbar_arrive(&s.raw_full[st]);
                }
                __syncwarp();
                if (lane == 4 * i) {
                    if (four) mbar_arrive_expect_tx(&s.raw_full[st], four);
                    else mbar_arrive(&s.raw_full[st]);
                }
                __syncwarp();
                if (mine && bytes) bulk_copy(s.raw[st][lane & 3], rec, bytes, &s.raw_full[st]);
            }
        }
    }
    if (ok && wait_bar(s, &s.raw_empty[k % kRaw], k / kRaw + 1)) {   // the end, for those that do not walk
        if (lane == 0) {
            s.tiles = k;
            s.word[k % kRaw][0] = kStop;
            mbar_arrive(&s.raw_full[k % kRaw]);
        }
    }
    if (!ok) {   // the copies in flight land before the block leaves
        for (uint32_t i = k > kRaw ? k - kRaw : 0; i < k; ++i) mbar_wait(&s.raw_full[i % kRaw], (i / kRaw) & 1u, nullptr, kWaitNs);
    }
}

// K of every tile, a block a warp; with the tile's mask, limits and factors.
template <int KIND>
__device__ __forceinline__ void key_repacker(Smem<KIND>& s, const ChunkParams& p, int warp, int lane) {
    constexpr int kRaw = Smem<KIND>::kRaw, kStages = Smem<KIND>::kStages;
    const Offsets off(warp, lane);
    #pragma unroll 1
    for (uint32_t k = 0;; ++k) {   // to the producer's mark
        const uint32_t st = k % kRaw, ks = k % kStages, in = k % Smem<KIND>::kInfos;
        if (!wait_two(s, &s.raw_full[st], k / kRaw, &s.k_empty[ks], k / kStages + 1)) return;
        if (s.word[st][0] == kStop) return;
        const uint32_t mine = s.word[st][warp];
        if (warp == 0 && lane == 0)
            s.info[in].mask = static_cast<unsigned long long>(s.word[st][0] & 0xffffu) |
                              static_cast<unsigned long long>(s.word[st][1] & 0xffffu) << 16 |
                              static_cast<unsigned long long>(s.word[st][2] & 0xffffu) << 32 |
                              static_cast<unsigned long long>(s.word[st][3] & 0xffffu) << 48;
        if (lane < kBs) s.info[in].limit[column_of(warp, lane)] = mine >> lane & 1u ? INFINITY : -INFINITY;
        const uint8_t* code = s.raw[st][warp];   // this warp's block
        if constexpr (KIND == kKindBf16) {
            repack_k<kFmtBf16>(code, s.k[ks], off);
        } else if constexpr (is_lowbit(KIND)) {
            repack_k_low<KIND == kKindInt4 ? 4 : 2>(code, s.k[ks], warp, p.ng, lane);
        } else {
            int f = kFmtE4m3;
            if constexpr (KIND == kKindMixed) f = (mine >> 17) & 3u;
            if (lane < kBs) {
                const float* sc = reinterpret_cast<const float*>(code + 2 * kTileFp8);
                const bool on = mine >> lane & 1u, wide = KIND == kKindMixed && f == kFmtBf16;
                const int n = column_of(warp, lane);
                s.factor[in][0][n] = wide ? 1.f : sc[lane];
                const float v = !on ? 0.f : wide ? 1.f : sc[kBs + lane];
                const unsigned wild = __ballot_sync(0xffffu, !isfinite(v));
                s.factor[in][1][n] = isfinite(v) ? v : 0.f;
                if (lane == 0) reinterpret_cast<uint16_t*>(&s.info[in].wild)[warp] = static_cast<uint16_t>(wild);
            }
            if (KIND == kKindMixed && f == kFmtBf16) repack_k<kFmtBf16>(code, s.k[ks], off);
            else if (KIND == kKindMixed && f == kFmtE5m2) repack_k<kFmtE5m2>(code, s.k[ks], off);
            else repack_k<kFmtE4m3>(code, s.k[ks], off);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&s.k_full[ks]);
            mbar_arrive(&s.raw_empty[st]);
        }
    }
}

// V of every tile, 32 dims a warp.
template <int KIND>
__device__ __forceinline__ void value_repacker(Smem<KIND>& s, const ChunkParams& p, int warp, int lane) {
    constexpr int kRaw = Smem<KIND>::kRaw, kStages = Smem<KIND>::kStages;
    const Offsets off(warp, lane);
    Walk walk(p, s);
    Segment g;
    uint32_t k = 0;
    while (walk.next(p, g)) {
        #pragma unroll 1
        for (int t = g.t0; t < g.t1; ++t, ++k) {
            const uint32_t st = k % kRaw, vs = k % kStages;
            if (!wait_two(s, &s.raw_full[st], k / kRaw, &s.v_empty[vs], k / kStages + 1)) return;
            const bool look = t * kTile + kTile - 1 > g.first;
            const uint32_t word[4] = {s.word[st][0], s.word[st][1], s.word[st][2], s.word[st][3]};
            VPut v(s.v[vs], word, look, lane);
            const uint8_t* pair = s.raw[st][(lane & 4) >> 1];   // lanes take the pair of blocks of their columns
            if constexpr (is_lowbit(KIND)) repack_v_low<KIND, KIND == kKindInt4 ? 4 : 2>(pair, v, p.ng, warp, lane);
            else repack_v<KIND>(pair, word, v, off, warp, lane);
            fence_proxy_async_shared();
            if (look) {
                const uint32_t lo = __reduce_or_sync(kFull, static_cast<uint32_t>(v.bad));
                const uint32_t hi = __reduce_or_sync(kFull, static_cast<uint32_t>(v.bad >> 32));
                v.bad = static_cast<unsigned long long>(hi) << 32 | lo;
            }
            __syncwarp();
            if (lane == 0) {
                s.info[k % Smem<KIND>::kInfos].nonfin[warp] = v.bad;
                mbar_arrive(&s.v_full[vs]);
                mbar_arrive(&s.raw_empty[st]);
            }
        }
    }
}

// What an issuing warp leaves behind when a wait ran out: nothing under way in tensor memory.
template <int KIND>
__device__ __forceinline__ void drain_mma(Smem<KIND>& s, int i) {
    if (elect_one()) mma_commit(smem_u32(&s.drain[i]));
    __syncwarp();
    mbar_wait(&s.drain[i], 0, nullptr, kWaitNs);
}

// S(i) = Q·K(i) of warpgroup W, by one warp: two tiles ahead, into the columns that held S(i−2) and P(i−2); a
// warpgroup finds its next S ready when it is done with one.
template <int KIND>
__device__ __forceinline__ void score_issuer(Smem<KIND>& s, const ChunkParams& p, int warpgroup) {
    constexpr uint32_t kDescS = mma_desc_bf16(kWgRows, kTile);
    constexpr int kStages = Smem<KIND>::kStages;
    const uint32_t W = uniform(warpgroup);
    const uint32_t col_s = uniform(s.tmem + kColS + W * 128);
    const uint32_t k_op = uniform(smem_u32(s.k)), q_op = uniform(smem_u32(s.q));
    Walk walk(p, s);
    Segment g;
    uint32_t base = 0, done = 0;   // tiles before the segment, of both and of this warpgroup
    uint32_t own = 0, ones = 0;    // phases of q_ready and q_one
    bool ok = true;
    while (ok && walk.next(p, g)) {
        const uint32_t n = uniform(g.t1 - g.t0), two = uniform(g.two);
        const uint32_t mine = two ? n : (n + 1 - W) / 2;
        if (mine > 0) ok = two || W == 0 ? wait_bar(s, &s.q_ready[W], own++) : wait_bar(s, &s.q_one, ones++);
        const uint32_t a = uniform(q_op + (two ? W : 0) * 2 * kOpBytes);
        #pragma unroll 1
        for (uint32_t i = 0; ok && i < mine; ++i) {
            const uint32_t x = done + i, buf = x & 1u, k = base + (two ? i : 2 * i + W), st = k % kStages;
            const uint32_t cols = uniform(col_s + buf * 64), b = uniform(k_op + st * op_parts(KIND) * kOpBytes);
            const uint32_t full = uniform(smem_u32(&s.s_full[W][buf])), empty = uniform(smem_u32(&s.k_empty[st]));
            ok = wait_two(s, &s.k_full[st], k / kStages, &s.pv_done[W][buf], (x >> 1) - 1, x >= 2);   // P(i−2) has been read
            if (!ok) break;
            tcgen_fence_after();
            if (elect_one()) {
                #pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_ss(cols, smem_desc_sw128(a + (ks >> 2) * kOpBytes + (ks & 3) * 32),
                           smem_desc_sw128(b + (ks >> 2) * 8192 + (ks & 3) * 32), kDescS, ks > 0);
                if constexpr (op_parts(KIND) == 2) {
                    #pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ss(cols, smem_desc_sw128(a + (ks >> 2) * kOpBytes + (ks & 3) * 32),
                               smem_desc_sw128(b + kOpBytes + (ks >> 2) * 8192 + (ks & 3) * 32), kDescS, 1u);
                }
                mma_commit(full);
                mma_commit(empty);
                if (!two) mbar_arrive(&s.k_empty[st]);
            }
            __syncwarp();
        }
        base += n;
        done += mine;
    }
    if (!ok) drain_mma(s, W);
}

// O += P(i)·V(i) of both warpgroups, by one warp, when P(i) is in tensor memory; W = 0, 1 in turn.
template <int KIND>
__device__ __forceinline__ void out_issuer(Smem<KIND>& s, const ChunkParams& p) {
    constexpr uint32_t kDescO = mma_desc_bf16(kWgRows, kDh);
    constexpr int kStages = Smem<KIND>::kStages;
    const uint32_t tmem = uniform(s.tmem), v_op = uniform(smem_u32(s.v));
    Walk walk(p, s);
    Segment g;
    uint32_t base = 0, done0 = 0, done1 = 0;   // tiles before the segment, of both and of each warpgroup
    bool ok = true;
    while (ok && walk.next(p, g)) {
        const uint32_t n = uniform(g.t1 - g.t0), two = uniform(g.two);
        const uint32_t mine0 = two ? n : (n + 1) / 2, mine1 = two ? n : n / 2;
        #pragma unroll 1
        for (uint32_t j = 0; j < 2 * mine0; ++j) {
            const uint32_t W = j & 1u, i = j >> 1;
            if (W && i >= mine1) continue;
            const uint32_t x = (W ? done1 : done0) + i, buf = x & 1u, k = base + (two ? i : 2 * i + W), st = k % kStages;
            const uint32_t d = uniform(tmem + kColO + W * 128), a = uniform(tmem + kColS + W * 128 + buf * 64);
            const uint32_t b = uniform(v_op + st * op_parts(KIND) * kOpBytes), more = uniform(i > 0);
            const uint32_t full = uniform(smem_u32(&s.pv_done[W][buf])), empty = uniform(smem_u32(&s.v_empty[st]));
            ok = wait_two(s, &s.p_full[W][buf], x >> 1, &s.v_full[st], k / kStages);
            if (!ok) break;
            tcgen_fence_after();
            if (elect_one()) {
                #pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_ts(d, a + ks * 8, smem_desc_sw128(b + ks * 32), kDescO, ks > 0 ? 1u : more);
                #pragma unroll   // the remainders
                for (int ks = 0; ks < 4; ++ks) mma_ts(d, a + 32 + ks * 8, smem_desc_sw128(b + ks * 32), kDescO, 1u);
                if constexpr (op_parts(KIND) == 2) {   // the remainders' own product, 2^-15 at most, is left out
                    #pragma unroll
                    for (int ks = 0; ks < 4; ++ks) mma_ts(d, a + ks * 8, smem_desc_sw128(b + kOpBytes + ks * 32), kDescO, 1u);
                }
                mma_commit(full);
                mma_commit(empty);
                if (!two) mbar_arrive(&s.v_empty[st]);
            }
            __syncwarp();
        }
        base += n;
        done0 += mine0;
        done1 += mine1;
    }
    if (!ok) drain_mma(s, 2);
}

// The E4M3 value nearest to x.
__device__ __forceinline__ float e4m3_value(float x) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3), __NV_E4M3)));
}

// A warp's 32 rows of q as the A operand, in the dim order of the K operand.  base: the unit's first token; rel: the
// lane's row counted from there, −1 for none.  Eight lanes read half a row: dims 8c .. 8c+7 are words c & 3 of four
// 16-byte pieces.  Returns what multiplies the row's logits (angle keys; 1 else).
template <int KIND>
__device__ __forceinline__ float load_query(const uint16_t* base, int rel, bool store, bool flip, uint8_t* op, int warp, int lane) {
    float factor = 1.f;
    if (!store && KIND != kKindAngle) return factor;
    const int c = lane & 7;
    uint32_t e[2][8][4];
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = __shfl_sync(kFull, rel, 4 * i + (lane >> 3));
        #pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (at >= 0) v = ld16(reinterpret_cast<const uint8_t*>(base + static_cast<int64_t>(at) * kDh + 64 * half + 8 * c));
            e[half][i][0] = flip ? v.x ^ 0x80008000u : v.x;
            e[half][i][1] = flip ? v.y ^ 0x80008000u : v.y;
            e[half][i][2] = flip ? v.z ^ 0x80008000u : v.z;
            e[half][i][3] = flip ? v.w ^ 0x80008000u : v.w;
        }
    }
    if constexpr (KIND == kKindAngle) {   // the E4M3 code of the row at its absmax scale, ||q||/||d_q||
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            float top = 0.f;
            #pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float2 f = unpack_bf16(e[x >> 2][i][x & 3]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            #pragma unroll
            for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            const float sc = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
            float r2 = 0.f, d2 = 0.f;
            #pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float2 f = unpack_bf16(e[x >> 2][i][x & 3]);
                const float a = __fdiv_rn(f.x, sc), b = __fdiv_rn(f.y, sc);
                const float da = e4m3_value(a), db = e4m3_value(b);
                r2 += a * a + b * b;
                d2 += da * da + db * db;
                e[x >> 2][i][x & 3] = pack_bf16(da, db);
            }
            #pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                r2 += __shfl_xor_sync(kFull, r2, o);
                d2 += __shfl_xor_sync(kFull, d2, o);
            }
            const float f = __shfl_sync(kFull, d2 == 0.f ? 0.f : sc * sqrtf(r2 / d2), (lane & 3) << 3);
            if ((lane >> 2) == i) factor = f;
        }
        if (!store) return factor;
    }
    #pragma unroll
    for (int half = 0; half < 2; ++half) {
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 32 * warp + 4 * i + (lane >> 3);
            uint8_t* to = op + half * kOpBytes + row * 128 + (c & 3) * 4;
            #pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint32_t*>(to + (((4 * (c >> 2) + x) ^ (row & 7)) << 4)) = e[half][i][x];
        }
    }
    fence_proxy_async_shared();
    return factor;
}

template <int KIND>
__device__ __forceinline__ void softmax_group(Smem<KIND>& s, const ChunkParams& p, int w, int tid, int lane) {
    const uint32_t lanes = static_cast<uint32_t>((tid >> 5) & 3) << 21;   // this warp's 32 tensor memory lanes
    constexpr int kStages = Smem<KIND>::kStages;
    const uint32_t tmem = s.tmem + lanes;
    const uint32_t col_s = tmem + kColS + w * 128, col_o = tmem + kColO + w * 128;
    // the scale's sign goes into q; a zero scale becomes one that leaves every finite logit at zero
    const bool flip = p.scale_log2 < 0.f;
    const float scale = fmaxf(fabsf(p.scale_log2), 1e-30f);
    WalkState& state = s.walks[threadIdx.x >> 5];
    {
        const Walk walk(p, s);
        if (lane == 0) state = walk;
        __syncwarp();
    }
    Segment g;
    uint32_t base = 0, done = 0, ones = 0;   // tiles before the segment, of both and of this warpgroup; segments of one row group
    bool merge_pending = false;
    int seg_index = 0;
    while (true) {
        {
            Walk walk(state);
            __syncwarp();
            if (!walk.next(p, g)) return;
            if (lane == 0) state = walk;
            __syncwarp();
        }
        const int n = g.t1 - g.t0;
        const int mine = g.two ? n : (n + 1 - w) / 2;   // tiles of this warpgroup
        const int row = g.two ? w * kWgRows + tid : tid;
        const bool live = row < g.rows;
        const int token = g.tok0 + row / p.g;
        const int64_t first_row = (static_cast<int64_t>(g.s0) + g.tok0) * p.n_q;   // row of q and out; rel: the thread's from there
        const int rel = live ? row / p.g * p.n_q + g.h * p.g + row % p.g : -1;
        const int pos = g.len < 0 ? -1 : g.len - g.T + token;
        if (merge_pending) {   // WG 0 has read the last unit's O and sums of this warpgroup
            if (!wait_bar(s, &s.merge_empty, ones - 1)) return;
            merge_pending = false;
        }
        float rs = load_query<KIND>(p.q + first_row * kDh, rel, g.two || w == 0, flip, s.q[g.two ? w : 0], tid >> 5, lane) * scale;
        rs = fmaxf(rs, 1e-30f);   // a NaN or zero factor: the codes carry it
        __syncwarp();
        if (lane == 0) {
            if (g.two || w == 0) mbar_arrive(&s.q_ready[w]);
            if (!g.two && w == 0 && n > 1) mbar_arrive(&s.q_one);
        }
        float m = -INFINITY, l = 0.f;
        unsigned flagged = 0;                     // tiles with noted V, from the first token's
        float poison = 0.f;                       // NaN where a position with a wild V factor is attended
        const int tile0 = max(g.first, 0) / kTile;
        for (int i = 0; i < mine; ++i) {
            const uint32_t k = base + (g.two ? i : 2 * i + w);
            const int in = k % Smem<KIND>::kInfos;
            const int t = g.t0 + (g.two ? i : 2 * i + w);
            const uint32_t x_at = done + i, cols = col_s + (x_at & 1) * 64;   // S(i), later P(i)
            if (!wait_bar(s, &s.s_full[w][x_at & 1], x_at >> 1)) return;      // and with S the tile's mask and factors
            tcgen_fence_after();
            uint32_t raw[2][32];
            tmem_ld32(cols, raw[0]);
            tmem_ld32(cols + 32, raw[1]);
            unsigned long long may = s.info[in].mask;
            tmem_wait_ld(raw[0]);
            tmem_wait_ld(raw[1]);
            float x[kTile];
            #pragma unroll
            for (int c = 0; c < kTile; ++c) x[c] = __uint_as_float(raw[c >> 5][c & 31]);
            if constexpr (has_factors(KIND)) {
                #pragma unroll
                for (int c = 0; c < kTile; c += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&s.factor[in][0][c]);
                    set2(&x[c], mul2(make_float2(x[c], x[c + 1]), make_float2(f.x, f.y)));
                    set2(&x[c + 2], mul2(make_float2(x[c + 2], x[c + 3]), make_float2(f.z, f.w)));
                }
            }
            const int t_end = t * kTile + kTile - 1;
            if (t_end > g.first) {
                const int left = pos - t * kTile;   // the row attends places 0 .. left
                if (left < kTile - 1) may &= left < 0 ? 0ull : (2ull << left) - 1ull;
                const uint32_t lo = static_cast<uint32_t>(may), hi = static_cast<uint32_t>(may >> 32);
                #pragma unroll
                for (int c = 0; c < kTile; ++c) {
                    const int at = place_of(c);
                    if (!((at < 32 ? lo >> at : hi >> (at - 32)) & 1u)) x[c] = -INFINITY;
                }
            } else if (may != ~0ull) {   // whatever a masked slot holds, the minimum with −inf is −inf
                #pragma unroll
                for (int c = 0; c < kTile; c += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&s.info[in].limit[c]);
                    x[c] = fminf(x[c], f.x);
                    x[c + 1] = fminf(x[c + 1], f.y);
                    x[c + 2] = fminf(x[c + 2], f.z);
                    x[c + 3] = fminf(x[c + 3], f.w);
                }
            }
            if constexpr (has_factors(KIND)) {
                if (s.info[in].wild & may) poison = NAN;
            }
            float part[4];   // four chains
            #pragma unroll
            for (int e = 0; e < 4; ++e) part[e] = max3(x[e], x[e + 4], x[e + 8]);
            #pragma unroll
            for (int c = 12; c < kTile - 4; c += 8)
                #pragma unroll
                for (int e = 0; e < 4; ++e) part[e] = max3(part[e], x[c + e], x[c + e + 4]);
            #pragma unroll
            for (int e = 0; e < 4; ++e) part[e] = fmaxf(part[e], x[kTile - 4 + e]);
            const float top = fmaxf(max3(part[0], part[1], part[2]), part[3]) * rs;
            if (__any_sync(kFull, top > m + kLazy)) {
                if (i > 0) {   // O of the tiles before is complete
                    if (!wait_bar(s, &s.pv_done[w][(x_at - 1) & 1], (x_at - 1) >> 1)) return;
                    tcgen_fence_after();
                }
                const float nm = fmaxf(m, top);
                const float f = m == nm ? 1.f : ex2(m - nm);
                m = nm;
                l *= f;
                if (i > 0) {
                    #pragma unroll 1
                    for (int c = 0; c < kDh; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(col_o + c, o);
                        tmem_wait_ld(o);
                        #pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(col_o + c, o);
                    }
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 rs2 = make_float2(rs, rs), ref2 = make_float2(-ref, -ref);
            uint32_t pw[16];   // in two halves: fewer registers
            #pragma unroll
            for (int c = 0; c < kTile; c += 4) {
                #pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 y = fma2(make_float2(x[c + e], x[c + e + 1]), rs2, ref2);
                    x[c + e] = ex2(y.x);
                    x[c + e + 1] = ex2(y.y);
                    sum[e / 2] = add2(sum[e / 2], make_float2(x[c + e], x[c + e + 1]));
                }
                if constexpr (has_factors(KIND)) {
                    const float4 f = *reinterpret_cast<const float4*>(&s.factor[in][1][c]);
                    set2(&x[c], mul2(make_float2(x[c], x[c + 1]), make_float2(f.x, f.y)));
                    set2(&x[c + 2], mul2(make_float2(x[c + 2], x[c + 3]), make_float2(f.z, f.w)));
                }
                #pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int at = ((c + e) / 2) & 15;
                    const float2 v = make_float2(x[c + e], x[c + e + 1]);
                    const float2 under = mul2(v, make_float2(kBelow, kBelow));
                    const uint32_t a = __float_as_uint(under.x), b = __float_as_uint(under.y);
                    pw[at] = __byte_perm(a, b, 0x7632);
                    set2(&x[c + e], add2(v, make_float2(-__uint_as_float(a & 0xffff0000u), -__uint_as_float(b & 0xffff0000u))));
                }
                if ((c & 31) == 28) {
                    tmem_st16(cols + (c >> 5) * 16, pw);
                    #pragma unroll   // the remainders, in the columns behind
                    for (int e = 0; e < 16; ++e) pw[e] = pack_bf16(x[(c & 32) + 2 * e], x[(c & 32) + 2 * e + 1]);
                    tmem_st16(cols + 32 + (c >> 5) * 16, pw);
                }
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_wait_st();
            if (t_end > g.first) {   // non-finite V that only some rows attend (v_full: the repack has looked)
                // once the tile before it in its stage has been read (this warpgroup may be ahead of both by then)
                if (i > 0 && !wait_bar(s, &s.pv_done[w][(x_at - 1) & 1], (x_at - 1) >> 1)) return;
                if (!wait_bar(s, &s.v_full[k % kStages], k / kStages)) return;
                const unsigned long long* nf = s.info[in].nonfin;
                const unsigned long long bad = nf[0] | nf[1] | nf[2] | nf[3];
                if (bad) {
                    flagged |= 1u << (t - tile0);
                    if (lane == 0) s.flags[threadIdx.x >> 5][t - tile0] = bad;
                }
            }
            tcgen_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.p_full[w][x_at & 1]);
        }
        if (mine > 0) {
            done += mine;
            if (mine > 1 && !wait_bar(s, &s.pv_done[w][done & 1], (done - 2) >> 1)) return;
            if (!wait_bar(s, &s.pv_done[w][(done - 1) & 1], (done - 1) >> 1)) return;
            tcgen_fence_after();
        }
        if constexpr (has_factors(KIND)) {
            if (__any_sync(kFull, poison != 0.f)) {
                #pragma unroll 1
                for (int c = 0; c < kDh; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(col_o + c, o);
                    tmem_wait_ld(o);
                    #pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + poison);
                    tmem_st16(col_o + c, o);
                }
                tmem_wait_st();
            }
        }
        base += n;
        const bool merging = !g.two && n > 1;   // both warpgroups hold a part of the rows
        if (merging && w == 1) {
            // O stays in tensor memory: the lanes are the same rows in both warpgroups
            s.ml()[tid] = m;
            s.ml()[kWgRows + tid] = l;
        }
        float f0 = 1.f, f1 = 0.f;
        if (merging) {
            if (w == 1) {
                // non-finite values noted by this warpgroup are added to its own O below
                for (unsigned e = flagged; e; e &= e - 1) {
                    const int tile = __ffs(e) - 1;
                    #pragma unroll 1
                    for (int c = 0; c < kDh; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(col_o + c, o);
                        tmem_wait_ld(o);
                        #pragma unroll
                        for (int d = 0; d < 32; ++d) {
                            for (unsigned long long bits = s.flags[threadIdx.x >> 5][tile]; bits; bits &= bits - 1) {
                                const int at = (tile0 + tile) * kTile + place_of(__ffsll(bits) - 1);
                                if (!live || at > pos) continue;
                                const float v = pool_value<KIND>(p, g.b, g.h, at, c + d);
                                if (!isfinite(v)) o[d] = __float_as_uint(__uint_as_float(o[d]) + v);
                            }
                        }
                        __syncwarp();
                        tmem_st32(col_o + c, o);
                    }
                    tmem_wait_st();   // the next tile reads these columns again
                }
                tcgen_fence_before();
                __syncwarp();
            }
        }
        if (!g.two && w == 1) {   // (without tiles too: the warpgroups stay within a segment of each other)
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.merge_full);
            ++ones;
            merge_pending = true;
            ++seg_index;
            continue;
        }
        if (!g.two) {
            if (!wait_bar(s, &s.merge_full, ones)) return;
            ++ones;
            tcgen_fence_after();
        }
        if (merging) {
            const float m1 = s.ml()[tid], l1 = s.ml()[kWgRows + tid];
            const float M = fmaxf(m, m1);
            f0 = m == -INFINITY ? 0.f : ex2(m - M);
            f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
            if (m == M) f0 = M == -INFINITY ? f0 : 1.f;
            if (m1 == M) f1 = M == -INFINITY ? f1 : 1.f;
            l = (m == -INFINITY && l == 0.f ? 0.f : l * f0) + (m1 == -INFINITY && l1 == 0.f ? 0.f : l1 * f1);
            m = M;
        }
        const bool whole = g.t0 == 0 && g.t1 == g.tiles;
        const int slot = 2 * blockIdx.x + (seg_index > 0);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint8_t* stage = s.q[g.two ? w : 0];
        #pragma unroll 1
        for (int c = 0; c < kDh; c += 32) {
            uint32_t o[32];
            tmem_ld32(col_o + c, o);
            tmem_wait_ld(o);
            float y[32];
            #pragma unroll
            for (int d = 0; d < 32; ++d) y[d] = __uint_as_float(o[d]);
            if (merging) {
                tmem_ld32(tmem + kColO + 128 + c, o);
                tmem_wait_ld(o);
                #pragma unroll
                for (int d = 0; d < 32; ++d) y[d] = y[d] * f0 + __uint_as_float(o[d]) * f1;
            }
            for (unsigned e = flagged; e; e &= e - 1) {
                const int tile = __ffs(e) - 1;
                for (unsigned long long bits = s.flags[threadIdx.x >> 5][tile]; bits; bits &= bits - 1) {
                    const int at = (tile0 + tile) * kTile + place_of(__ffsll(bits) - 1);
                    if (!live || at > pos) continue;
                    #pragma unroll
                    for (int d = 0; d < 32; ++d) {
                        const float v = pool_value<KIND>(p, g.b, g.h, at, c + d);
                        if (!isfinite(v)) y[d] += v;
                    }
                }
            }
            __syncwarp();
            if (!whole) {
                float* part = p.part + static_cast<int64_t>(slot) * kDh * kUnitRows + row;
                #pragma unroll
                for (int d = 0; d < 32; ++d)
                    if (live) part[(c + d) * kUnitRows] = y[d];
                continue;
            }
            // rows through shared memory (Q's, which no MMA reads any more; the warp's own rows): whole lines out
            #pragma unroll
            for (int d = 0; d < 32; d += 8) {
                if (p.out_f32) {
                    put16(stage, tid, d / 4, __float_as_uint(y[d] * inv), __float_as_uint(y[d + 1] * inv),
                          __float_as_uint(y[d + 2] * inv), __float_as_uint(y[d + 3] * inv));
                    put16(stage, tid, d / 4 + 1, __float_as_uint(y[d + 4] * inv), __float_as_uint(y[d + 5] * inv),
                          __float_as_uint(y[d + 6] * inv), __float_as_uint(y[d + 7] * inv));
                } else {
                    put16(stage, tid, (c & 32) / 8 + d / 8, pack_bf16(y[d] * inv, y[d + 1] * inv),
                          pack_bf16(y[d + 2] * inv, y[d + 3] * inv), pack_bf16(y[d + 4] * inv, y[d + 5] * inv),
                          pack_bf16(y[d + 6] * inv, y[d + 7] * inv));
                }
            }
            if (p.out_f32 || (c & 32)) {   // 128 bytes of each row are there
                __syncwarp();
                const int64_t pitch = kDh * (p.out_f32 ? 4 : 2);
                uint8_t* out = static_cast<uint8_t*>(p.out) + first_row * pitch + (p.out_f32 ? 4 * c : 2 * (c - 32)) + (lane & 7) * 16;
                #pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int src = 4 * e + (lane >> 3), at = __shfl_sync(kFull, rel, src), row128 = (tid & ~31) + src;
                    const uint4 v = ld16(stage + row128 * 128 + (((lane & 7) ^ (row128 & 7)) << 4));
                    if (at >= 0) *reinterpret_cast<uint4*>(out + at * pitch) = v;
                }
                __syncwarp();
            }
        }
        if (live) {
            if (!whole) {
                p.part_ml[static_cast<int64_t>(slot) * 2 * kUnitRows + row] = m;
                p.part_ml[static_cast<int64_t>(slot) * 2 * kUnitRows + kUnitRows + row] = l;
            } else if (p.lse_out) {
                p.lse_out[first_row + rel] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
            }
        }
        if (tid == 0 && w == 0 && !whole) p.part_seg[slot] = make_int4(g.b, g.qt, g.h << 1 | (g.t0 > 0), g.t1);
        if (!g.two) {
            tcgen_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.merge_empty);
        }
        ++seg_index;
    }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const ChunkParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<KIND>& s = *reinterpret_cast<Smem<KIND>*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == kScoreWarp) tmem_alloc_all(&s.tmem);
    if (tid == 0) {
        for (int i = 0; i < Smem<KIND>::kRaw; ++i) {
            mbar_init(&s.raw_full[i], 1);
            mbar_init(&s.raw_empty[i], 8);
        }
        for (int i = 0; i < Smem<KIND>::kStages; ++i) {
            mbar_init(&s.k_full[i], 4);
            mbar_init(&s.k_empty[i], 2);
            mbar_init(&s.v_full[i], 4);
            mbar_init(&s.v_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_ready[i], 4);
            mbar_init(&s.drain[i], 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s.s_full[i][b], 1);
                mbar_init(&s.p_full[i][b], 4);
                mbar_init(&s.pv_done[i][b], 1);
            }
        }
        mbar_init(&s.drain[2], 1);
        mbar_init(&s.q_one, 4);
        mbar_init(&s.merge_full, 4);
        mbar_init(&s.merge_empty, 4);
        mbar_fence_init();
        s.abort = 0;
        s.tiles = 0;
        s.remaining = 0;
    }
    pdl_wait();
    pdl_trigger();
    if (tid < 2) p.part_seg[2 * blockIdx.x + tid] = make_int4(-1, 0, 0, 0);
    static_assert(2 * kMaxBatch * sizeof(int64_t) <= sizeof(s.q), "the schedule's scratch");
    make_schedule(p, s, reinterpret_cast<int64_t*>(s.q));
    if (tid == 0 && (smem_u32(smem_raw) & 1023u)) {   // the operands' swizzle wants it (nothing else stands before them)
        report(p.err, KVD_ERR_CUDA);
        s.remaining = 0;
    }
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    // one copy of each role's code: with one per warpgroup the loops outgrow the instruction cache
    // (its misses took 90% of the next level's rate, and every role ran at half speed)
    // Registers: a scheduler has 512 a lane; five of the twenty warps are on each, at 96 at launch, then
    // 2·152 + 48 + 72 + 56 = 480 = 5·96.
    constexpr int kRegs = 96, kSoftmaxRegs = 152, kKeyRegs = 48, kValueRegs = 72, kIssueRegs = 56;
    static_assert(kThreads % 128 == 0 && 2 * kSoftmaxRegs + kKeyRegs + kValueRegs + kIssueRegs <= kThreads / 128 * kRegs &&
                      kThreads / 128 * kRegs <= 512,
                  "a request beyond what the launch has would not return");
    if (warp < 8) {
        take_registers<kSoftmaxRegs>();
        softmax_group<KIND>(s, p, warp >> 2, tid & 127, lane);
    } else if (warp < kValueWarp) {
        give_registers<kKeyRegs>();
        key_repacker<KIND>(s, p, warp - kKeyWarp, lane);
    } else if (warp < kProducerWarp) {
        give_registers<kValueRegs>();
        value_repacker<KIND>(s, p, warp - kValueWarp, lane);
    } else {
        give_registers<kIssueRegs>();
        if (warp == kProducerWarp) producer<KIND>(s, p, lane);
        else if (warp < kOutWarp) score_issuer<KIND>(s, p, warp - kScoreWarp);
        else out_issuer<KIND>(s, p);
    }
    __syncwarp();
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    if (warp == kScoreWarp) {
        // The commits that gave back the last tiles' stages arrive in this block's shared memory: it must still be its
        // own.  (The phases before them are over: those stages have been filled again.)
        constexpr uint32_t kStages = Smem<KIND>::kStages;
        for (uint32_t k = s.tiles > kStages ? s.tiles - kStages : 0; !s.abort && k < s.tiles; ++k)
            if (!wait_two(s, &s.k_empty[k % kStages], k / kStages, &s.v_empty[k % kStages], k / kStages)) break;
        __syncwarp();
        if (lane == 0 && s.abort) report(p.err, KVD_ERR_TIMEOUT);
        tmem_free_all(s.tmem);
    }
}

template <int KIND>
cudaError_t launch_kind(const ChunkParams& p, int grid, cudaStream_t stream) {
    const size_t smem = sizeof(Smem<KIND>);
    static_assert(sizeof(Smem<KIND>) <= 232448, "shared memory of one SM");
    static_assert(max_record(KIND) % 16 == 0 && sizeof(TileInfo) % 16 == 0, "16-byte accesses");
    const cudaError_t e =
        cudaFuncSetAttribute(chunk_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_dependent(chunk_kernel<KIND>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, -1, stream, p);
}

}  // namespace chunk
}  // namespace kvd
