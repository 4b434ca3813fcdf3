// kvd_latent_attn.cu — absorbed latent attention over the paged cache.
//
// Row (token i of the T new tokens of request b, head h), len = seq_lens[b], P = len − T + i:
//   l_t = scale·<q, (c_t, r_t)> over 512 + 64 dims, t ≤ P and retained;  out = Σ_t softmax(l)_t·c_t,  lse = log Σ exp(l_t).
//
// Work.  A unit is (request, 64 rows: some tokens of up to 64 heads), its cost its tiles of 64 positions and a few tiles' time for its
// start and end.  With more than 64 heads a CTA has one block of heads, and neighbours have the same positions of the others at
// nearly the same time, so the cache leaves DRAM once.  The units' costs, laid end to end, are cut into equal shares, one per CTA (one
// CTA per SM); a unit cut by a border leaves fp32 partials that join_kernel joins.
//
// One CTA:
//  * producer warp: follows the block table and bulk-copies (TMA engine) the four records of a tile.  A record is laid out as
//    the 128-byte-swizzled operand that the tensor cores read, so it is used where it lands, and twice: K-major for the logits (groups of
//    eight tokens 9,216 bytes apart), N-major for the product with c.  A block's place is free once its 16 positions' product is done;
//  * fixer warp: zeroes the rows of positions that nobody may attend (evicted, behind the end, unknown blocks);
//  * a warp that issues S = Q·Kᵀ (Q in tensor memory) and one that issues O += P·C (P in shared memory);
//  * four softmax warps, online in fp32 (exp2 domain), the reference maximum moved only when a row's passes it by 8.
// 64 rows, not 128, since 128 rows of 512 fp32 sums are all of tensor memory: M = 64 uses half its lanes, lanes 0 .. 15 of each 32 hold Q and
// S, 16 .. 31 hold O.  An MMA with M = 64 takes as long as one with M = 128 (33 cycles for N = 64, 129 for N = 256), so the matrix rate ends at
// half; that is enough up to 64 heads: a tile's MMAs take 2,240 cycles (1.15 us), its way through HBM 1.65 us.
// Rounding.  K, C and Q enter the products exactly, logits, statistics and sums are fp32.  Where out is bf16 a weight enters as one bf16 (off
// by at most 2^-8 of itself; in 8 bits with its token's scale).  out is divided by the sum of the weights as they were rounded, so that what all
// of a row's weight is on comes out exactly; lse is that of the weights before.  Outputs are 1.1 to 1.35 times as far from 64 bits as an fp32
// form's rounded to bf16 (divided by the sum before: up to 1.8 in 8 bits; 1 to 2 us less a call).  Where out is fp32 (TWO) nothing behind it hides
// that: a weight enters as two bf16, as in the chunk kernel (off by at most 2^-16 of itself); what the first leaves of it lies where the tile's
// rotated dims were, which only S reads.  That makes O's MMAs 2,060 cycles a tile instead of 1,030: 32 x 8,192 positions with 16 heads 69 us
// (bf16 61), with 128 heads 116 (96), 131,072 in 8 bits 52 (47).
// 8 bits: converter warps load the codes (a tile under way while the one before it is converted) and store them as bf16, exactly, in the same
// layout; the token's scale multiplies the logit's first 512 dims (they and the rotated ones are summed apart) and the weight.  The roles share
// 128 registers a thread at launch, and the kernel spills for it (1,012 bytes of stores, 592 of loads); with bf16 records nothing is spilled.
//
// Bound: 32 x 8,192 positions, 16 heads: 60 us, 5.0 TB/s (74% of measured; the tiles alone at 6.9 TB/s, then 8 us of start, 7 of
// partials and join); 128 heads: 96 us, the tensor cores (85% busy in a tile); 131,072 positions in 8 bits, 64 heads: 47 us, of it 10 until the
// first tile is converted, 1.4 us a tile, 8 for 147 parts and their join.
//
// Waits.  Each barrier's waiter is at most one phase behind it.  Every wait gives up after a second or so (a try suspends 3.8 us; not while a
// row is computed again, which ends by itself and takes 0.5 us a position); the kernel then reports it and ends.
#include "kvd_latent.h"
#include "kvd_tcgen.cuh"

namespace kvd {
namespace {

constexpr int kTile = 64;              // positions per tile: four blocks
constexpr int kRows = kLatUnitRows;
constexpr int kStages = 3;
constexpr int kTileBytes = kTile * kLatKey * 2;
constexpr int kGroup = 9216;           // bytes of eight tokens of a tile
constexpr int kRotated = 8192;         // from where on those of their rotated dims stand
constexpr int kProducerWarp = 4, kScoreWarp = 5, kFixWarp = 6, kValueWarp = 7, kConvertWarp = 8, kConvertWarps = 8;
constexpr int threads_of(bool fp8) { return fp8 ? 32 * (kConvertWarp + kConvertWarps) : 256; }
constexpr float kLazy = 8.f;           // log2: how far a row's maximum may pass its reference
constexpr int kTries = 200000;         // tries of a wait, which suspend: a second or so
constexpr uint64_t kWaitNs = 1000000000ull;   // of what must land before the block leaves
// Tensor memory.  M = 64 leaves half of the lanes: 0 .. 15 of each 32 hold Q and S, 16 .. 31 hold O.
constexpr uint32_t kColQ = 0, kColS = 288, kColR = 352, kHalf = 16u << 16;
constexpr int kUnitTiles = 3;          // what a unit costs beside its tiles, in tiles
constexpr int kMinShare = 2;           // tiles of the smallest share: another CTA costs its start and a part to join

__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void unpack8(float* x, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = unpack_bf16(w[i]);
        x[2 * i] = a.x;
        x[2 * i + 1] = a.y;
    }
}

struct Info {
    alignas(16) float scale[kTile];    // 8-bit records: by column
    float by[kTile];                   // 1/scale, or 0 where that is no number
    unsigned long long mask;           // bit 16·block + t: position may be attended by the unit's last row
    int base;                          // position of column 0
    int id[4];                         // physical blocks, −1: none
};

// What is known of a tile.  8-bit records are loaded by the converters, several tiles behind the producer.
constexpr int infos_of(bool fp8) { return fp8 ? 4 : kStages; }

struct Smem {
    uint8_t k[kStages][kTileBytes];
    uint8_t p[kRows * kTile * 2];
    Info info[infos_of(true)];
    uint64_t full[infos_of(true)], free[infos_of(true)], ready[kStages], empty[kStages][4], s_full, s_free, p_full, q_full, drain[2];
    uint32_t tmem;
    volatile int abort;
    int again;   // warps that compute a row again: every other wait may be longer for it
};

struct Request {
    int s0, T, len;   // first row, new tokens, context (−1: bad length, nothing is attended)
};
struct Segment {
    int b, tb, t0, t1, tiles;
    int s0, T, len;
    int tok0, first, end;    // first token, its position, positions that the last row attends
    int64_t start;           // of the unit's tiles in the schedule
    bool multi;              // rows of more than one token
};

__device__ __forceinline__ Request load_request(const LatentAttnParams& p, int b, bool tell) {
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
__device__ __forceinline__ int unit_end(const Request& r, int tb, int tpb) {
    return r.len < 0 ? 0 : r.len - r.T + min((tb + 1) * tpb, r.T);
}
__device__ __forceinline__ int unit_tiles(const Request& r, int tb, int tpb) {
    return r.len < 0 ? 1 : static_cast<int>((static_cast<uint32_t>(unit_end(r, tb, tpb)) + kTile - 1) / kTile);   // (up to 2^31 − 1 positions)
}
// Tiles of units 0 .. k-1: Σ ⌊(c + i·tpb)/64⌋, whose remainders repeat every 64 units.
__device__ inline int64_t tiles_before(const Request& r, int k, int tpb) {
    if (r.len < 0) return k;
    const int n = (r.T + tpb - 1) / tpb;
    const int64_t whole = min(k, n - 1), c = static_cast<int64_t>(r.len) - r.T + tpb + kTile - 1;
    int64_t rest = 0;
    if (whole >= 64) {
        for (int i = 0; i < 64; ++i) rest += (c + static_cast<int64_t>(i) * tpb) & 63;
        rest *= whole / 64;
    }
    for (int64_t i = whole & ~63ll; i < whole; ++i) rest += (c + i * tpb) & 63;
    int64_t s = (tpb * (whole * (whole - 1) / 2) + c * whole - rest) >> 6;
    if (k == n) s += unit_tiles(r, n - 1, tpb);
    return s;
}

struct Heads {
    int blocks, each, tpb, first, n;   // head blocks, heads of one, tokens of a unit; this CTA's heads
    __device__ __forceinline__ Heads(const LatentAttnParams& p, int block) {
        blocks = (p.n_q + kRows - 1) / kRows;
        each = (p.n_q + blocks - 1) / blocks;
        tpb = kRows / each;
        set(p, block);
    }
    __device__ __forceinline__ void set(const LatentAttnParams& p, int block) {
        first = block * each;
        n = min(each, p.n_q - first);
    }
};

// Quotients are of 32 bits where they can be: the long division takes five times as long, and a call waits for it.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// The CTA's segments in order; every role walks them on its own.
struct Walk {
    int64_t at, remaining, share;
    int b, tb, off, extra, tpb;
    Request r;
    __device__ __forceinline__ bool next(const LatentAttnParams& p, Segment& g) {
        while (remaining > 0) {
            g.b = b;
            g.tb = tb;
            g.tiles = unit_tiles(r, tb, tpb);
            g.start = at - off + extra;
            const int take = static_cast<int>(min(static_cast<int64_t>(g.tiles) + extra - off, remaining));
            g.t0 = max(off - extra, 0);
            g.t1 = off + take - extra;
            g.s0 = r.s0;
            g.T = r.T;
            g.len = r.len;
            g.end = unit_end(r, tb, tpb);
            g.tok0 = tb * tpb;
            g.first = r.len < 0 ? -1 : r.len - r.T + g.tok0;
            g.multi = min(tpb, r.T - g.tok0) > 1;
            at += take;
            remaining -= take;
            off = 0;
            if (remaining > 0 && ++tb * tpb >= r.T) {
                tb = 0;
                do {
                    if (++b >= p.B) {
                        remaining = 0;
                        break;
                    }
                    r = load_request(p, b, false);
                } while (r.T == 0);
            }
            if (g.t1 > g.t0) return true;
        }
        return false;
    }
    // CTAs that share the unit.
    __device__ __forceinline__ int parts(const Segment& g) const {
        return static_cast<int>(quotient(g.start + g.tiles - 1, share) - quotient(g.start, share)) + 1;
    }
};

// The CTA's share, found by each warp.  Requests cost tiles + units·extra; their units are searched by the same sums.
struct Cost {
    int64_t tiles;
    int units;
};
__device__ __forceinline__ Cost cost_of(const Request& r, int tpb) {
    const int units = (r.T + tpb - 1) / tpb;
    return {units <= 1 ? (r.T ? unit_tiles(r, 0, tpb) : 0) : tiles_before(r, units, tpb), units};
}
template <class T>
__device__ __forceinline__ T scan(T x, int lane) {
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T v = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += v;
    }
    return x;
}
// False: nothing for this CTA.
__device__ __forceinline__ bool set_share(Walk& w, int64_t tiles, int64_t units, const Heads& hd) {
    const int lanes = gridDim.x / hd.blocks, me = blockIdx.x / hd.blocks;
    // a small call is cut into its smallest shares; there the border must not fall beside the tiles
    w.extra = tiles >= static_cast<int64_t>(8 * kUnitTiles) * lanes ? kUnitTiles : static_cast<int>(tiles) / (8 * lanes);
    const int64_t total = tiles + units * w.extra;
    w.share = max(quotient(total + lanes - 1, lanes), static_cast<int64_t>(kMinShare));
    w.at = min(w.share * me, total);
    w.remaining = me < lanes ? min(w.share, total - w.at) : 0;
    return w.remaining > 0;
}
// The unit of request r that holds what is `in` from the request's start.
__device__ __forceinline__ void find_unit(Walk& w, int64_t in) {
    int a = 0, z = (w.r.T + w.tpb - 1) / w.tpb;   // the last unit of [a, z) that starts at or before `in`
    int64_t from = 0;
    while (z - a > 1) {
        const int mid = a + (z - a) / 2;
        const int64_t x = tiles_before(w.r, mid, w.tpb) + static_cast<int64_t>(mid) * w.extra;
        if (x <= in) {
            a = mid;
            from = x;
        } else {
            z = mid;
        }
    }
    w.tb = a;
    w.off = static_cast<int>(in - from);
}
// Up to 32 requests, a lane each, their tiles' sum below 2^31 (true: found): no barrier, no long sums.
__device__ inline bool find_share_small(const LatentAttnParams& p, const Heads& hd, int lane, Walk& w) {
    w = Walk{};
    w.tpb = hd.tpb;
    const Request r = lane < p.B ? load_request(p, lane, blockIdx.x == 0 && threadIdx.x < 32) : Request{0, 0, -1};
    const Cost c = cost_of(r, hd.tpb);
    if (__any_sync(kFull, c.tiles >> 25 || c.units >> 23)) return false;
    if (!__any_sync(kFull, c.units > 1)) {
        // Whole shares for every unit, if that makes them no longer than another unit's start and end would: 3 x 16,384 positions,
        // 64 heads 32 us (36 with shares of the sum), 4 x 4,000, 16 heads 16.3 (19.1).
        const int lanes = gridDim.x / hd.blocks, me = blockIdx.x / hd.blocks, n = static_cast<int>(c.tiles);
        const int least = max((static_cast<int>(__reduce_add_sync(kFull, n)) + lanes - 1) / lanes, kMinShare);
        auto ctas_of = [&](int share) { return (n + share - 1) / share; };
        if (static_cast<int>(__reduce_add_sync(kFull, ctas_of(least + kUnitTiles))) <= lanes) {
            int share = least;
            while (static_cast<int>(__reduce_add_sync(kFull, ctas_of(share))) > lanes) ++share;
            const int up = scan(ctas_of(share), lane);
            const unsigned at = __ballot_sync(kFull, me < up);
            if (at == 0) return true;
            const int src = __ffs(at) - 1;
            w.share = share;
            w.at = static_cast<int64_t>(share) * me;
            w.b = src;
            w.r = {__shfl_sync(kFull, r.s0, src), __shfl_sync(kFull, r.T, src), __shfl_sync(kFull, r.len, src)};
            w.off = (me - __shfl_sync(kFull, up - ctas_of(share), src)) * share;
            w.remaining = min(share, __shfl_sync(kFull, n, src) - w.off);
            return true;
        }
    }
    const int tiles = scan(static_cast<int>(c.tiles), lane), units = scan(c.units, lane);
    if (!set_share(w, __shfl_sync(kFull, tiles, 31), __shfl_sync(kFull, units, 31), hd)) return true;
    const int64_t up = tiles + static_cast<int64_t>(units) * w.extra;
    const unsigned at = __ballot_sync(kFull, w.at < up);
    const int src = __ffs(at) - 1;   // (the share starts in some request)
    w.b = src;
    w.r = {__shfl_sync(kFull, r.s0, src), __shfl_sync(kFull, r.T, src), __shfl_sync(kFull, r.len, src)};
    find_unit(w, w.at - __shfl_sync(kFull, up - c.tiles - static_cast<int64_t>(c.units) * w.extra, src));
    return true;
}
// Any number of them: scratch holds 2·p.B int64, filled before by all threads.
__device__ inline void fill_scratch(const LatentAttnParams& p, int64_t* scratch, int tpb, int threads) {
    for (int b = threadIdx.x; b < p.B; b += threads) {
        const Cost c = cost_of(load_request(p, b, blockIdx.x == 0 && p.B > 32), tpb);
        scratch[2 * b] = c.tiles;
        scratch[2 * b + 1] = c.units;
    }
}
__device__ inline Walk find_share(const LatentAttnParams& p, const int64_t* scratch, const Heads& hd, int lane) {
    Walk w{};
    w.tpb = hd.tpb;
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
    if (!set_share(w, tiles, units, hd)) return w;
    int64_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int64_t c = b0 + lane < p.B ? scratch[2 * (b0 + lane)] + w.extra * scratch[2 * (b0 + lane) + 1] : 0;
        const int64_t up = before + scan(c, lane);
        const unsigned at = __ballot_sync(kFull, w.at < up);
        if (at) {
            const int src = __ffs(at) - 1;
            w.b = b0 + src;
            w.r = load_request(p, w.b, false);
            find_unit(w, w.at - __shfl_sync(kFull, up - c, src));
            return w;
        }
        before = __shfl_sync(kFull, up, 31);
    }
    w.remaining = 0;
    return w;
}

__device__ __forceinline__ bool wait_bar(Smem& s, uint64_t* bar, uint32_t phase) {
    #pragma unroll 1
    for (int i = 0; i < kTries; ++i) {
        if (__all_sync(kFull, mbar_try_wait(bar, phase & 1u))) return true;
        if (__any_sync(kFull, s.abort)) return false;
        if (i == kTries - 1 && __any_sync(kFull, *static_cast<volatile int*>(&s.again) > 0)) i = 0;
    }
    s.abort = 1;   // reported at the kernel's end
    return false;
}

// ------------------------------------------------------------- one row, plainly
// A warp a row, of which it writes dims from .. to − 1 (and lse with the first): a lane has dims 8·lane .. +7 and 256 + 8·lane .. +7 of the latent, lanes 0 .. 7 the rotated ones.
template <bool FP8>
__device__ __noinline__ void plain_row(const LatentAttnParams& p, int b, int64_t row, int end, int from, int to) {
    const int lane = threadIdx.x & 31;
    const uint16_t* qr = p.q + row * kLatKey;
    float q[24], acc[16], m = -INFINITY, sum = 0.f;
    unpack8(q, ld16(qr + lane * 8));
    unpack8(q + 8, ld16(qr + 256 + lane * 8));
    unpack8(q + 16, lane < 8 ? ld16(qr + kLatDim + lane * 8) : make_uint4(0, 0, 0, 0));
    #pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    for (int pos = 0; pos < end; ++pos) {
        const int64_t block = p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kBs];
        const int t = pos % kBs;
        if (block < 0 || block >= p.num_blocks || (p.retain && !((p.retain[block] >> t) & 1))) continue;
        const uint8_t* record = p.mem + block * latent_record_bytes(FP8);
        float k[24];
        if constexpr (FP8) {
            const float s = *reinterpret_cast<const float*>(record + kLatScales + 4 * t);
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint2 c = *reinterpret_cast<const uint2*>(record + latent_code(t, lane + 32 * i));
                uint32_t h[4];
                e4m3x4_to_f16x2x2(c.x, h[0], h[1]);
                e4m3x4_to_f16x2x2(c.y, h[2], h[3]);
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = unpack_f16(h[j]);
                    k[8 * i + 2 * j] = v.x * s;
                    k[8 * i + 2 * j + 1] = v.y * s;
                }
            }
            unpack8(k + 16, lane < 8 ? ld16(record + latent_rope_piece(t, lane)) : make_uint4(0, 0, 0, 0));
        } else {
            unpack8(k, ld16(record + latent_piece(t, lane)));
            unpack8(k + 8, ld16(record + latent_piece(t, 32 + lane)));
            unpack8(k + 16, lane < 8 ? ld16(record + latent_piece(t, 64 + lane)) : make_uint4(0, 0, 0, 0));
        }
        float dot = 0.f;
        #pragma unroll
        for (int i = 0; i < 24; ++i) dot = fmaf(q[i], k[i], dot);
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
        const float l = dot * p.scale_log2, top = fmaxf(m, l);
        const float ref = top == -INFINITY ? 0.f : top;
        const float f = exp2f(m - ref), w = exp2f(l - ref);
        m = top;
        sum = sum * f + w;
        #pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, k[i], acc[i] * f);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    #pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int d = (i >> 3) * 256 + lane * 8 + (i & 7);
        if (d < from || d >= to) continue;
        const int64_t at = row * kLatDim + d;
        if (p.out_f32) static_cast<float*>(p.out)[at] = acc[i] * inv;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(acc[i] * inv);
    }
    if (lane == 0 && from == 0 && p.lse_out) p.lse_out[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// Whether a retained token of positions from .. to − 1 has a latent that is not finite; by a warp.
template <bool FP8>
__device__ __noinline__ bool odd_tokens(const LatentAttnParams& p, int b, int from, int to) {
    const int lane = threadIdx.x & 31;
    bool odd = false;
    #pragma unroll 1
    for (int pos = from; pos < to; ++pos) {
        const int64_t block = p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kBs];
        const int t = pos % kBs;
        if (block < 0 || block >= p.num_blocks || (p.retain && !((p.retain[block] >> t) & 1))) continue;
        const uint8_t* record = p.mem + block * latent_record_bytes(FP8);
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (FP8) {   // (a code that is NaN, or a scale that makes it one)
                const uint2 c = *reinterpret_cast<const uint2*>(record + latent_code(t, lane + 32 * i));
                const auto nan = [](uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
                odd |= (nan(c.x) | nan(c.y)) != 0 || !isfinite(*reinterpret_cast<const float*>(record + kLatScales + 4 * t));
            } else {
                const uint4 c = ld16(record + latent_piece(t, lane + 32 * i));
                const auto nan = [](uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                odd |= (nan(c.x) | nan(c.y) | nan(c.z) | nan(c.w)) != 0;
            }
        }
    }
    return __any_sync(kFull, odd);
}
// A token that some rows of a unit attend and others do not may hold what is not finite: its weight is 0 for those, and 0·NaN
// is NaN.  A row that came out as NaN is computed again, plainly, if such a token stands behind what it attends
// (else it is NaN by right).  end: positions that the row attends; unit_end: that the unit's last row does.
template <bool FP8>
__device__ __forceinline__ void again(const LatentAttnParams& p, int b, int64_t row, int end, int unit_end, int from, int to) {
    if (odd_tokens<FP8>(p, b, end, unit_end)) plain_row<FP8>(p, b, row, end, from, to);
}

// ------------------------------------------------------------------ producer
// Follows the block table, eight tiles of ids at a time and the next eight under way; bf16 records are copied as they are,
// 8-bit ones fetched to L2.
struct Ids {
    int id;            // of the lane's block, −1: none
    uint32_t bits;     // its slots that may be attended
};
__device__ __forceinline__ Ids load_ids(const LatentAttnParams& p, const int32_t* table, int t, const Segment& g, int lane) {
    Ids x{-1, 0};
    const int pos = t * kTile + lane * kBs;
    if (pos < g.end && t + (lane >> 2) < g.t1) x.id = table[pos / kBs];
    return x;
}
__device__ __forceinline__ void check_ids(const LatentAttnParams& p, Ids& x, int t, const Segment& g, int lane) {
    const int pos = t * kTile + lane * kBs;
    if (!(pos < g.end && t + (lane >> 2) < g.t1)) return;
    if (x.id < 0 || x.id >= p.num_blocks) {
        report(p.err, KVD_ERR_OOB);
        x.id = -1;
    } else {
        x.bits = p.retain ? p.retain[x.id] : 0xffffu;
        if (g.end - pos < kBs) x.bits &= (1u << (g.end - pos)) - 1u;
    }
}

template <bool FP8>
__device__ __forceinline__ void producer(Smem& s, const LatentAttnParams& p, Walk walk, int lane) {
    constexpr int kInfos = infos_of(FP8);
    constexpr uint32_t kRecord = latent_record_bytes(FP8);
    // The cache passes through L2 once (or by neighbours at nearly the same time): what else is there stays, the kernels' code too.
    const uint64_t policy = policy_evict_first();
    Segment g;
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(p, g)) {
        const int32_t* table = p.block_table + static_cast<int64_t>(g.b) * p.max_blocks;
        Ids ids = load_ids(p, table, g.t0, g, lane);
        #pragma unroll 1
        for (int t = g.t0; ok && t < g.t1; t += 8) {
            check_ids(p, ids, t, g, lane);
            const Ids next = load_ids(p, table, t + 8, g, lane);
            #pragma unroll 1
            for (int u = 0; ok && u < 8 && t + u < g.t1; ++u, ++n) {
                const uint32_t at = n % kInfos;
                if (n >= kInfos) ok = wait_bar(s, FP8 ? &s.free[at] : &s.empty[at][0], n / kInfos - 1);   // (a stage's blocks come free in order)
                if (!ok) break;
                unsigned long long mask = 0;
                int block[4], copies = 0;
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    block[k] = __shfl_sync(kFull, ids.id, 4 * u + k);
                    mask |= static_cast<unsigned long long>(__shfl_sync(kFull, ids.bits, 4 * u + k)) << (16 * k);
                    copies += block[k] >= 0;
                }
                if (lane == 0) {
                    Info& info = s.info[at];
                    info.mask = mask;
                    info.base = (t + u) * kTile;
                    if constexpr (FP8) {
                        #pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            info.id[k] = block[k];
                            if (n >= 2 && block[k] >= 0)   // (the first two are loaded at once)
                                asm volatile("cp.async.bulk.prefetch.L2.global.L2::cache_hint [%0], %1, %2;" ::"l"(p.mem + static_cast<int64_t>(block[k]) * kRecord), "r"(kRecord), "l"(policy) : "memory");
                        }
                        mbar_arrive(&s.full[at]);
                    } else {
                        if (copies) mbar_arrive_expect_tx(&s.full[at], copies * kRecord);
                        else mbar_arrive(&s.full[at]);
                    }
                }
                __syncwarp();
                if constexpr (!FP8) {
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k > 0 && n >= kInfos) ok = ok && wait_bar(s, &s.empty[at][k], n / kInfos - 1);
                        // (a tile begun is copied whole: its barrier counts all its bytes)
                        if (lane == 0 && block[k] >= 0) bulk_g2s(s.k[at] + k * kRecord, p.mem + static_cast<int64_t>(block[k]) * kRecord, kRecord, &s.full[at], policy);
                        __syncwarp();
                    }
                }
            }
            ids = next;
        }
    }
    if (!FP8 && s.abort) {   // copies under way must land in memory that is still this block's
        for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k) mbar_wait(&s.full[k % kStages], (k / kStages) & 1u, nullptr, kWaitNs);
    }
}

// ----------------------------------------------------------------------- fix
// Rows that nobody may attend are zeroed: their weight is 0, and 0·NaN would be NaN.
__device__ __forceinline__ void fixer(Smem& s, const LatentAttnParams& p, Walk walk, int lane) {
    Segment g;
    uint32_t n = 0;
    while (walk.next(p, g)) {
        #pragma unroll 1
        for (int t = g.t0; t < g.t1; ++t, ++n) {
            const uint32_t st = n % kStages;
            if (!wait_bar(s, &s.full[st], n / kStages)) return;
            for (unsigned long long todo = ~s.info[st].mask; todo; todo &= todo - 1) {
                const int c = __ffsll(todo) - 1;
                uint8_t* row = s.k[st] + (c >> 3) * kGroup + (c & 7) * 128 + (lane >> 3) * 1024 + (lane & 7) * 16;
                *reinterpret_cast<uint4*>(row) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(row + 4096) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.ready[st]);
        }
    }
}

// ------------------------------------------------------------------- convert
// 8-bit records become bf16 operands: codes exactly (every e4m3 value is a bf16 value), the scale stays outside.  A warp
// takes eight tokens of a tile: 64 codes of each of them, 512 bytes, a load.  A tile's loads are under way while the one
// before it is converted.
__device__ __forceinline__ uint4 ld16_once(const void* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}
struct Raw {
    uint4 code[8], rot[2];
    float scale;
};
__device__ __forceinline__ bool load_raw(Smem& s, const LatentAttnParams& p, Raw& x, uint32_t n, int warp, int lane) {
    const uint32_t at = n % infos_of(true);
    if (!wait_bar(s, &s.full[at], n / infos_of(true))) return false;
    const int r = lane >> 2, j = lane & 3;
    const Info& info = s.info[at];
    const bool on = info.mask >> (warp * 8 + r) & 1;
    const uint8_t* record = p.mem + static_cast<int64_t>(max(info.id[warp >> 1], 0)) * latent_record_bytes(true);
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint64_t policy = policy_evict_first();
    #pragma unroll
    for (int i = 0; i < 8; ++i) x.code[i] = on ? ld16_once(record + (warp & 1) * 4096 + i * 512 + r * 64 + j * 16, policy) : none;
    #pragma unroll
    for (int i = 0; i < 2; ++i) x.rot[i] = on ? ld16_once(record + kLatCodes + (warp & 1) * 1024 + r * 128 + (2 * j + i) * 16, policy) : none;
    x.scale = on ? *reinterpret_cast<const float*>(record + kLatScales + 4 * ((warp & 1) * 8 + r)) : 0.f;
    return true;
}
__device__ __forceinline__ bool store_raw(Smem& s, const Raw& x, uint32_t n, int warp, int lane) {
    const uint32_t st = n % kStages;
    if (n >= kStages && !wait_bar(s, &s.empty[st][warp >> 1], n / kStages - 1)) return false;
    const int r = lane >> 2, j = lane & 3;
    uint8_t* group = s.k[st] + warp * kGroup + r * 128;
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {x.code[i].x, x.code[i].y, x.code[i].z, x.code[i].w};
        uint32_t o[8];
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(w[k], lo, hi);
            const float2 a = unpack_f16(lo), b = unpack_f16(hi);
            o[2 * k] = pack_bf16(a.x, a.y);
            o[2 * k + 1] = pack_bf16(b.x, b.y);
        }
        *reinterpret_cast<uint4*>(group + i * 1024 + (((2 * j) ^ r) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(group + i * 1024 + (((2 * j + 1) ^ r) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    #pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(group + 8192 + (2 * j + i) * 16) = x.rot[i];   // (in its order already)
    if (j == 0) {
        Info& info = s.info[n % infos_of(true)];
        const float by = 1.f / x.scale;
        info.scale[warp * 8 + r] = x.scale;
        info.by[warp * 8 + r] = isfinite(by) ? by : 0.f;
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.ready[st]);
    return true;
}
__device__ __forceinline__ void converter(Smem& s, const LatentAttnParams& p, Walk walk, int warp, int lane) {
    Segment g;
    uint32_t tiles = 0;
    while (walk.next(p, g)) tiles += g.t1 - g.t0;
    Raw a, b;
    if (tiles == 0 || !load_raw(s, p, a, 0, warp, lane)) return;
    #pragma unroll 1
    for (uint32_t n = 0; n < tiles; n += 2) {
        if (n + 1 < tiles && !load_raw(s, p, b, n + 1, warp, lane)) return;
        if (!store_raw(s, a, n, warp, lane)) return;
        if (n + 1 >= tiles) return;
        if (n + 2 < tiles && !load_raw(s, p, a, n + 2, warp, lane)) return;
        if (!store_raw(s, b, n + 1, warp, lane)) return;
    }
}

// --------------------------------------------------------------------- issue
// Operands with groups of eight rows `group` bytes apart: rows along M or N (K-major), or along K, where 64 columns of N
// stand 1,024 bytes apart (N-major).
__device__ __forceinline__ uint64_t desc_k(uint32_t addr, uint32_t group) {
    return static_cast<uint64_t>(addr >> 4) | (1ull << 16) | (static_cast<uint64_t>(group >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_n(uint32_t addr) {
    return static_cast<uint64_t>(addr >> 4) | (64ull << 16) | (static_cast<uint64_t>(kGroup >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Nothing under way in tensor memory when a warp that issued leaves.
__device__ __forceinline__ void drain_mma(Smem& s, int i) {
    const uint32_t bar = uniform(smem_u32(&s.drain[i]));
    if (elect_one()) mma_commit(bar);
    __syncwarp();
    mbar_wait(&s.drain[i], 0, nullptr, kWaitNs);
}

// A warp for each product: what stands between two runs of MMAs (waits, commits) would leave the tensor cores idle if one
// warp had both.  S(t) = Q·K(t)ᵀ, when S(t − 1) has been read:
template <bool FP8>
__device__ __forceinline__ void score_issuer(Smem& s, const LatentAttnParams& p, Walk walk) {
    constexpr uint32_t kDescS = mma_desc_bf16(64, kTile);
    const uint32_t tmem = uniform(s.tmem), k_op = uniform(smem_u32(s.k)), s_full = uniform(smem_u32(&s.s_full));
    Segment g;
    uint32_t n = 0, segs = 0;
    bool ok = true;
    while (ok && walk.next(p, g)) {
        const uint32_t end = uniform(n + g.t1 - g.t0);
        ok = wait_bar(s, &s.q_full, segs++);
        #pragma unroll 1
        for (; ok && n < end; ++n) {
            const uint32_t st = n % kStages, op = uniform(k_op + st * kTileBytes);
            ok = wait_bar(s, &s.ready[st], n / kStages) && (n == 0 || wait_bar(s, &s.s_free, n - 1));
            if (!ok) break;
            tcgen_fence_after();
            if (elect_one()) {
                #pragma unroll 1   // (less code to fetch: the first tile waits for it)
                for (uint32_t c = 0; c < 9; ++c)
                    #pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        mma_ts(tmem + (FP8 && c == 8 ? kColR : kColS), tmem + kColQ + c * 32 + k * 8, desc_k(op + c * 1024 + k * 32, kGroup),
                               kDescS, (FP8 && c == 8 ? k : (c | k)) != 0);
                mma_commit(s_full);
            }
            __syncwarp();
        }
    }
    drain_mma(s, 0);
}
// O += P(t)·C(t):
template <bool TWO>
__device__ __forceinline__ void value_issuer(Smem& s, const LatentAttnParams& p, Walk walk) {
    constexpr uint32_t kDescO = mma_desc_bf16(64, 256) | (1u << 16);
    const uint32_t tmem = uniform(s.tmem), k_op = uniform(smem_u32(s.k)), p_op = uniform(smem_u32(s.p));
    Segment g;
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(p, g)) {
        const uint32_t first = uniform(n), end = uniform(n + g.t1 - g.t0);
        #pragma unroll 1
        for (; ok && n < end; ++n) {
            const uint32_t st = n % kStages, op = uniform(k_op + st * kTileBytes), empty = uniform(smem_u32(&s.empty[st][0]));
            const uint32_t add = uniform(n > first);
            ok = wait_bar(s, &s.p_full, n);
            if (!ok) break;
            tcgen_fence_after();
            if (elect_one()) {
                if constexpr (TWO) {   // the weights' rests first: they lie in all of the tile's blocks
                    #pragma unroll
                    for (int k = 0; k < 4; ++k)
                        #pragma unroll
                        for (int h = 0; h < 2; ++h)
                            mma_ss(tmem + kHalf + h * 256, desc_k(op + kRotated + k * 32, kGroup), desc_n(op + h * 4096 + k * 2 * kGroup), kDescO,
                                   k > 0 ? 1u : add);
                }
                #pragma unroll
                for (int k = 0; k < 4; ++k) {   // a block at a time, which is free then
                    #pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mma_ss(tmem + kHalf + h * 256, desc_k(p_op + k * 32, 1024), desc_n(op + h * 4096 + k * 2 * kGroup), kDescO,
                               TWO || k > 0 ? 1u : add);
                    mma_commit(empty + 8 * k);
                }
            }
            __syncwarp();
        }
    }
    drain_mma(s, 1);
    // the last commits arrive in this block's shared memory: it must still be its own
    if (!s.abort)
        for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k)
            for (int i = 0; i < 4; ++i)
                if (!wait_bar(s, &s.empty[k % kStages][i], k / kStages)) return;
}

// Four lanes side by side have a pair of dims each of four groups of eight: lane i gets group i whole.
__device__ __forceinline__ uint4 whole_group(const uint32_t* t, int lane) {
    const bool odd = lane & 1, high = lane & 2;
    const uint32_t a = __shfl_xor_sync(kFull, odd ? t[0] : t[1], 1), b = __shfl_xor_sync(kFull, odd ? t[2] : t[3], 1);
    const uint32_t x[4] = {odd ? a : t[0], odd ? t[1] : a, odd ? b : t[2], odd ? t[3] : b};
    const uint32_t c = __shfl_xor_sync(kFull, high ? x[0] : x[2], 2), d = __shfl_xor_sync(kFull, high ? x[1] : x[3], 2);
    return high ? make_uint4(c, d, x[2], x[3]) : make_uint4(x[0], x[1], c, d);
}

// Partials: four values a lane (of rows lane/4 and lane/4 + 8 of a group of 16 two dims each), 32 lanes for eight dims.
__device__ __forceinline__ int64_t part_at(int64_t slot, int group, int eight, int lane) {
    return ((slot * (kRows / 16) + group) * (kLatDim / 8) + eight) * 32 + lane;
}

// ------------------------------------------------------------------- softmax
// 16 lanes × 64 columns: a thread has rows lane/4 and lane/4 + 8, of each column group of eight the two at 2·(lane%4):
// v[4k], v[4k+1] of the first row, v[4k+2], v[4k+3] of the second.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st_16x64(uint32_t addr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_16x32(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Row of q and out of row r of a unit (token r / each, head r % each), or −1.
__device__ __forceinline__ int64_t row_of(const LatentAttnParams& p, const Heads& hd, const Segment& g, int r) {
    const int tok = r / hd.each, h = r - tok * hd.each;
    return tok < hd.tpb && g.tok0 + tok < g.T && h < hd.n ? (static_cast<int64_t>(g.s0) + g.tok0 + tok) * p.n_q + hd.first + h : -1;
}

// A unit's queries to tensor memory: column j holds dims 2j, 2j + 1 of a row.
__device__ __forceinline__ void load_q(Smem& s, const LatentAttnParams& p, const Heads& hd, const Segment& g, uint32_t mine, int warp, int lane) {
    const uint16_t* src[2];
    bool on[2];
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t row = row_of(p, hd, g, warp * 16 + (lane >> 2) + 8 * h);
        on[h] = row >= 0;
        src[h] = p.q + max(row, static_cast<int64_t>(0)) * kLatKey + 4 * (lane & 3);
    }
    // all loads at once: behind the first tiles' copies each round of them would wait its turn (2.3 us)
    uint32_t v[5][32];
    #pragma unroll
    for (int c = 0; c < 5; ++c)   // 64 columns, 128 dims; 32 columns at the end
        #pragma unroll
        for (int k = 0; k < (c < 4 ? 8 : 4); ++k)
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 x = on[h] ? *reinterpret_cast<const uint2*>(src[h] + c * 128 + k * 16) : make_uint2(0, 0);
                v[c][4 * k + 2 * h] = x.x;
                v[c][4 * k + 2 * h + 1] = x.y;
            }
    #pragma unroll
    for (int c = 0; c < 4; ++c) tmem_st_16x64(mine + kColQ + c * 64, v[c]);
    tmem_st_16x32(mine + kColQ + 256, v[4]);
    tmem_wait_st();
    tcgen_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.q_full);
}

template <bool FP8, bool TWO>
__device__ __forceinline__ void softmax(Smem& s, const LatentAttnParams& p, const Heads& hd, Walk walk, int warp, int lane) {
    const uint32_t mine = s.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int quad = lane & 3;
    Segment g;
    uint32_t n = 0;
    bool ok = true;
    bool more = walk.next(p, g);
    if (more) load_q(s, p, hd, g, mine, warp, lane);
    while (ok && more) {
        const int r0 = warp * 16 + (lane >> 2);
        const int limit[2] = {g.first + r0 / hd.each, g.first + (r0 + 8) / hd.each};   // positions that the rows attend, at most
        float ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, cut[2] = {0.f, 0.f};   // sums of weights, of rounded weights
        #pragma unroll 1
        for (int t = g.t0; t < g.t1; ++t, ++n) {
            const uint32_t st = n % kStages;
            uint32_t v[32];
            float x[32];
            ok = wait_bar(s, &s.ready[st], n / kStages) && wait_bar(s, &s.s_full, n);   // (what is known of the tile, and its S)
            if (!ok) break;
            tcgen_fence_after();
            tmem_ld_16x64(mine + kColS, v);
            const Info& info = s.info[n % infos_of(FP8)];
            if constexpr (FP8) {
                uint32_t r[32];
                tmem_ld_16x64(mine + kColR, r);
                tmem_wait_ld(v);
                tmem_wait_ld(r);
                #pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 f = *reinterpret_cast<const float2*>(&info.scale[8 * k + 2 * quad]);
                    x[4 * k] = fmaf(__uint_as_float(v[4 * k]), f.x, __uint_as_float(r[4 * k])) * p.scale_log2;
                    x[4 * k + 1] = fmaf(__uint_as_float(v[4 * k + 1]), f.y, __uint_as_float(r[4 * k + 1])) * p.scale_log2;
                    x[4 * k + 2] = fmaf(__uint_as_float(v[4 * k + 2]), f.x, __uint_as_float(r[4 * k + 2])) * p.scale_log2;
                    x[4 * k + 3] = fmaf(__uint_as_float(v[4 * k + 3]), f.y, __uint_as_float(r[4 * k + 3])) * p.scale_log2;
                }
            } else {
                tmem_wait_ld(v);
                #pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i]) * p.scale_log2;
            }
            tcgen_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.s_free);
            const unsigned long long mask = info.mask;
            const int base = info.base;
            if (mask != ~0ull || (g.multi && base + kTile > g.first + 1)) {
                #pragma unroll
                for (int k = 0; k < 8; ++k)
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = 8 * k + 2 * quad + e;
                        const bool on = mask >> c & 1;
                        if (!on || base + c > limit[0]) x[4 * k + e] = -INFINITY;
                        if (!on || base + c > limit[1]) x[4 * k + 2 + e] = -INFINITY;
                    }
            }
            float top[2] = {x[0], x[2]};
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                top[0] = fmaxf(top[0], fmaxf(x[4 * k], x[4 * k + 1]));
                top[1] = fmaxf(top[1], fmaxf(x[4 * k + 2], x[4 * k + 3]));
            }
            float factor[2] = {1.f, 1.f};
            bool moved = false;
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
                if (top[h] > ref[h] + kLazy) {
                    factor[h] = ex2(ref[h] - top[h]);
                    sum[h] *= factor[h];
                    cut[h] *= factor[h];
                    ref[h] = top[h];
                    moved = true;
                }
            }
            const float z0 = ref[0] == -INFINITY ? 0.f : ref[0], z1 = ref[1] == -INFINITY ? 0.f : ref[1];
            uint32_t w[16];
            uint8_t* rest = s.k[st] + 2 * warp * kGroup + kRotated + (lane >> 2) * 128 + quad * 4;   // (of row r0; S has been read)
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float a = ex2(x[4 * k] - z0), b = ex2(x[4 * k + 1] - z0), c = ex2(x[4 * k + 2] - z1), d = ex2(x[4 * k + 3] - z1);
                sum[0] += a + b;
                sum[1] += c + d;
                const float2 f = FP8 ? *reinterpret_cast<const float2*>(&info.scale[8 * k + 2 * quad]) : make_float2(1.f, 1.f);
                w[2 * k] = FP8 ? pack_bf16(a * f.x, b * f.y) : pack_bf16(a, b);
                w[2 * k + 1] = FP8 ? pack_bf16(c * f.x, d * f.y) : pack_bf16(c, d);
                float2 p0 = unpack_bf16(w[2 * k]), p1 = unpack_bf16(w[2 * k + 1]);
                if constexpr (TWO) {
                    const uint32_t l0 = FP8 ? pack_bf16(a * f.x - p0.x, b * f.y - p0.y) : pack_bf16(a - p0.x, b - p0.y);
                    const uint32_t l1 = FP8 ? pack_bf16(c * f.x - p1.x, d * f.y - p1.y) : pack_bf16(c - p1.x, d - p1.y);
                    *reinterpret_cast<uint32_t*>(rest + ((k ^ (r0 & 7)) << 4)) = l0;
                    *reinterpret_cast<uint32_t*>(rest + kGroup + ((k ^ (r0 & 7)) << 4)) = l1;
                    p0 = add2(p0, unpack_bf16(l0));
                    p1 = add2(p1, unpack_bf16(l1));
                }
                if constexpr (FP8) {   // (without a factor of a normal size the weight itself)
                    const float2 by = *reinterpret_cast<const float2*>(&info.by[8 * k + 2 * quad]);
                    cut[0] += (by.x != 0.f ? p0.x * by.x : a) + (by.y != 0.f ? p0.y * by.y : b);
                    cut[1] += (by.x != 0.f ? p1.x * by.x : c) + (by.y != 0.f ? p1.y * by.y : d);
                } else {
                    cut[0] += p0.x + p0.y;
                    cut[1] += p1.x + p1.y;
                }
            }
            if (n > 0) ok = wait_bar(s, &s.empty[(n - 1) % kStages][3], (n - 1) / kStages);   // P and O are free
            if (!ok) break;
            if (t > g.t0 && __any_sync(kFull, moved)) {
                tcgen_fence_after();
                #pragma unroll 1
                for (int c = 0; c < 512; c += 64) {
                    tmem_ld_16x64(mine + kHalf + c, v);
                    tmem_wait_ld(v);
                    #pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * factor[i >> 1 & 1]);
                    tmem_st_16x64(mine + kHalf + c, v);
                }
                tmem_wait_st();
                tcgen_fence_before();
            }
            uint8_t* pr = s.p + r0 * 128 + quad * 4;
            #pragma unroll
            for (int k = 0; k < 8; ++k) {
                *reinterpret_cast<uint32_t*>(pr + ((k ^ (r0 & 7)) << 4)) = w[2 * k];
                *reinterpret_cast<uint32_t*>(pr + 1024 + ((k ^ (r0 & 7)) << 4)) = w[2 * k + 1];
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.p_full);
                if (FP8) mbar_arrive(&s.free[n % infos_of(true)]);
            }
        }
        // the next unit's queries take the place of this one's, whose logits are all there: S goes on during what follows
        Segment after;
        more = ok && walk.next(p, after);
        if (more) load_q(s, p, hd, after, mine, warp, lane);
        if (ok) ok = wait_bar(s, &s.empty[(n - 1) % kStages][3], (n - 1) / kStages);
        if (!ok) break;
        tcgen_fence_after();
        const bool whole = g.t0 == 0 && g.t1 == g.tiles;
        const int slot = 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0);
        const int64_t row[2] = {row_of(p, hd, g, r0), row_of(p, hd, g, r0 + 8)};
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(kFull, sum[h], 1);
            sum[h] += __shfl_xor_sync(kFull, sum[h], 2);
            cut[h] += __shfl_xor_sync(kFull, cut[h], 1);
            cut[h] += __shfl_xor_sync(kFull, cut[h], 2);
        }
        if (!whole) {
            if (warp == 0 && lane == 0) p.part_seg[slot] = make_int4(g.b, g.s0 + g.tok0, min(hd.tpb, g.T - g.tok0) * hd.each, walk.parts(g));
            #pragma unroll
            for (int h = 0; h < 2; ++h)
                if (quad == 0) {
                    float* ml = p.part_ml + static_cast<int64_t>(slot) * 3 * kRows + r0 + 8 * h;
                    ml[0] = ref[h];
                    ml[kRows] = sum[h];
                    ml[2 * kRows] = cut[h];
                }
        } else if (quad == 0 && p.lse_out) {
            #pragma unroll
            for (int h = 0; h < 2; ++h)
                if (row[h] >= 0) p.lse_out[row[h]] = sum[h] == 0.f ? -INFINITY : (ref[h] + log2f(sum[h])) * kLn2;
        }
        const float inv[2] = {cut[0] == 0.f ? 0.f : 1.f / cut[0], cut[1] == 0.f ? 0.f : 1.f / cut[1]};
        float odd[2] = {0.f, 0.f};
        if (__any_sync(kFull, row[0] >= 0 || row[1] >= 0)) {
            if (!whole) {
                // sums as they are to the partials, in this order: each store is 512 bytes in a row (as rows, in pieces of 32 bytes,
                // 64 of them took 3.0 us)
                float4* dst = reinterpret_cast<float4*>(p.part) + part_at(slot, warp, 0, lane);
                #pragma unroll 1
                for (int c = 0; c < 512; c += 64) {
                    uint32_t v[32];
                    tmem_ld_16x64(mine + kHalf + c, v);
                    tmem_wait_ld(v);
                    #pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[(c / 8 + k) * 32] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]), __uint_as_float(v[4 * k + 2]),
                                                            __uint_as_float(v[4 * k + 3]));
                }
            } else {
                // rows to out: a thread has a pair of every eight dims of two rows
                uint8_t* dst[2];
                #pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t at = max(row[h], static_cast<int64_t>(0)) * kLatDim;
                    dst[h] = static_cast<uint8_t*>(p.out) + (p.out_f32 ? (at + 2 * quad) * 4 : (at + 8 * quad) * 2);
                }
                #pragma unroll 1
                for (int c = 0; c < 512; c += 64) {
                    uint32_t v[32];
                    tmem_ld_16x64(mine + kHalf + c, v);
                    tmem_wait_ld(v);
                    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2 y[8];
                        #pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            y[k] = make_float2(__uint_as_float(v[4 * k + 2 * h]) * inv[h], __uint_as_float(v[4 * k + 2 * h + 1]) * inv[h]);
                            odd[h] += y[k].x + y[k].y;
                        }
                        if (p.out_f32) {
                            #pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (row[h] >= 0) *reinterpret_cast<float2*>(dst[h] + 4 * (c + 8 * k)) = y[k];
                        } else {
                            #pragma unroll
                            for (int k = 0; k < 8; k += 4) {
                                uint32_t t[4];
                                #pragma unroll
                                for (int i = 0; i < 4; ++i) t[i] = pack_bf16(y[k + i].x, y[k + i].y);
                                const uint4 g8 = whole_group(t, lane);
                                if (row[h] >= 0) *reinterpret_cast<uint4*>(dst[h] + 2 * (c + 8 * k)) = g8;
                            }
                        }
                    }
                }
            }
        }
        tcgen_fence_before();
        if (whole && g.multi) {
            #pragma unroll
            for (int h = 0; h < 2; ++h)
                for (unsigned todo = __ballot_sync(kFull, row[h] >= 0 && odd[h] != odd[h]); todo;) {
                    const int i = (__ffs(todo) - 1) >> 2, r = warp * 16 + 8 * h + i;
                    todo &= ~(15u << 4 * i);
                    __syncwarp();
                    if (g.len < 0) continue;
                    if (lane == 0) atomicAdd(&s.again, 1);
                    again<FP8>(p, g.b, row_of(p, hd, g, r), g.first + r / hd.each + 1, g.end, 0, kLatDim);
                    if (lane == 0) atomicSub(&s.again, 1);
                }
        }
        g = after;
    }
}

template <bool FP8, bool TWO>
__global__ void __launch_bounds__(threads_of(FP8), 1) attn_kernel(const LatentAttnParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& s = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == kScoreWarp) tmem_alloc_all(&s.tmem);
    if (tid == 0) {
        for (int i = 0; i < infos_of(FP8); ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.free[i], 4);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.ready[i], FP8 ? kConvertWarps : 1);
            for (int k = 0; k < 4; ++k) mbar_init(&s.empty[i][k], 1);
        }
        mbar_init(&s.s_full, 1);
        mbar_init(&s.s_free, 4);
        mbar_init(&s.p_full, 4);
        mbar_init(&s.q_full, 4);
        mbar_init(&s.drain[0], 1);
        mbar_init(&s.drain[1], 1);
        mbar_fence_init();
        s.abort = 0;
        s.again = 0;
    }
    pdl_wait();
    pdl_trigger();
    const Heads hd(p, blockIdx.x % ((p.n_q + kRows - 1) / kRows));
    if (tid < 2) p.part_seg[2 * blockIdx.x + tid] = make_int4(-1, 0, 0, 0);
    // q of up to 16 MB to L2, a part by each CTA: the queries are read behind the first tiles' copies
    const int64_t q_bytes = static_cast<int64_t>(p.n_tokens) * p.n_q * kLatKey * 2, part = (q_bytes / gridDim.x + 16) & ~15ll;
    if (tid == 0 && q_bytes <= (16 << 20) && part * blockIdx.x < q_bytes)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<const uint8_t*>(p.q) + part * blockIdx.x),
                     "r"(static_cast<uint32_t>(min(part, q_bytes - part * blockIdx.x)))
                     : "memory");
    Walk walk;
    const bool found = p.B <= 32 && find_share_small(p, hd, lane, walk);   // (every warp finds the same)
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    if (!found) {
        static_assert(2 * kMaxBatch * sizeof(int64_t) <= sizeof(s.k[kStages - 1]), "the schedule's scratch");
        int64_t* scratch = reinterpret_cast<int64_t*>(s.k[kStages - 1]);
        fill_scratch(p, scratch, hd.tpb, threads_of(FP8));
        __syncthreads();
        walk = find_share(p, scratch, hd, lane);
        fence_proxy_async_shared();
        __syncthreads();   // the scratch has been read: copies may overwrite it
    }
    if (smem_u32(smem_raw) & 1023u) {   // the operands' swizzle wants it (nothing else stands before them)
        if (tid == 0) report(p.err, KVD_ERR_CUDA);
        walk.remaining = 0;
    }
    // 8 bits: a thread has 128 registers at launch: 200 + 72 + 2·120 = 4·128
    if (warp < 4) {
        if (FP8) take_registers<200>();
        softmax<FP8, TWO>(s, p, hd, walk, warp, lane);
    } else if (warp < kConvertWarp) {
        if (FP8) give_registers<72>();
        if (warp == kProducerWarp) producer<FP8>(s, p, walk, lane);
        else if (warp == kScoreWarp) score_issuer<FP8>(s, p, walk);
        else if (warp == kValueWarp) value_issuer<TWO>(s, p, walk);
        else if (!FP8 && warp == kFixWarp) fixer(s, p, walk, lane);
    } else if constexpr (FP8) {
        give_registers<120>();
        converter(s, p, walk, warp - kConvertWarp, lane);
    }
    __syncwarp();
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    if (warp == kScoreWarp) {
        if (lane == 0 && s.abort) report(p.err, KVD_ERR_TIMEOUT);
        tmem_free_all(s.tmem);
    }
}

// Joins the parts of units that the schedule cut.  A CTA of the schedule starts at most one of them, as its last; the
// others' parts are the following CTAs' first.  Units of few parts are joined 16 rows and 32 dims a warp, those of many 16 rows and
// eight dims a CTA, whose warps share the parts.  Many are more than eight; where the rows are enough for the warps, more than an
// eighth of the rows, up to 32: 768 rows of 13 parts by warps 61 us (the call), by CTAs 78; 64 of 32 parts 32 and 22.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kMaxCtas = 512, kJoinDims = 32;
struct Join {
    int4 start[kMaxCtas];            // (request, first token, rows, parts) of the unit that the CTA starts
    uint32_t groups[kMaxCtas];       // running counts of groups of 16 rows: of few parts, of many << 16
    float4 part[kJoinWarps][32];
    float top[kJoinWarps][16], sum[kJoinWarps][16], cut[kJoinWarps][16];
};
__device__ __forceinline__ void put2(const LatentAttnParams& p, int64_t row, int d, float x, float y, float inv) {
    if (p.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + row * kLatDim + d) = make_float2(x * inv, y * inv);
    else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * kLatDim + d) = pack_bf16(x * inv, y * inv);
}
// A CTA's k-th part of the unit that it starts: in its own second place, or in the first of the k-th CTA behind it.
__device__ __forceinline__ int64_t slot_of(int cta, int k, int blocks) { return k == 0 ? 2 * cta + 1 : 2 * (cta + k * blocks); }
// Parts from, from + step, .. of a group's dims 8·eight .. + 8·N − 1: sums, maximum and sums of weights of a lane's two rows, BATCH parts'
// loads under way at a time.
template <int N, int BATCH>
__device__ __forceinline__ void join_parts(const LatentAttnParams& p, int cta, int blocks, int parts, int from, int step, int group, int eight,
                                           int lane, float4 (&acc)[N], float (&top)[2], float (&sum)[2], float (&cut)[2]) {
    #pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    top[0] = top[1] = -INFINITY;
    sum[0] = sum[1] = cut[0] = cut[1] = 0.f;
    #pragma unroll 1
    for (int k = from; k < parts; k += BATCH * step) {
        float4 x[BATCH][N];
        float m[BATCH][2], l[BATCH][2], c[BATCH][2];
        #pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const bool on = k + b * step < parts;
            const int64_t slot = slot_of(cta, on ? k + b * step : k, blocks);
            const float* ml = p.part_ml + slot * 3 * kRows + group * 16 + (lane >> 2);
            const float4* src = reinterpret_cast<const float4*>(p.part) + part_at(slot, group, eight, lane);
            #pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[b][h] = on ? ml[8 * h] : -INFINITY;
                l[b][h] = on ? ml[kRows + 8 * h] : 0.f;
                c[b][h] = on ? ml[2 * kRows + 8 * h] : 0.f;
            }
            #pragma unroll
            for (int j = 0; j < N; ++j) x[b][j] = on ? src[32 * j] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float z[2];
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float was = top[h];
            #pragma unroll
            for (int b = 0; b < BATCH; ++b) top[h] = fmaxf(top[h], m[b][h]);
            z[h] = top[h] == -INFINITY ? 0.f : top[h];
            const float f = ex2(was - z[h]);
            sum[h] *= f;
            cut[h] *= f;
            #pragma unroll
            for (int j = 0; j < N; ++j)
                if (h == 0) acc[j].x *= f, acc[j].y *= f;
                else acc[j].z *= f, acc[j].w *= f;
        }
        #pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const float f0 = ex2(m[b][0] - z[0]), f1 = ex2(m[b][1] - z[1]);
            sum[0] = fmaf(f0, l[b][0], sum[0]);
            sum[1] = fmaf(f1, l[b][1], sum[1]);
            cut[0] = fmaf(f0, c[b][0], cut[0]);
            cut[1] = fmaf(f1, c[b][1], cut[1]);
            #pragma unroll
            for (int j = 0; j < N; ++j)
                acc[j] = make_float4(fmaf(f0, x[b][j].x, acc[j].x), fmaf(f0, x[b][j].y, acc[j].y), fmaf(f1, x[b][j].z, acc[j].z), fmaf(f1, x[b][j].w, acc[j].w));
        }
    }
}
template <bool FP8>
__device__ __noinline__ void join_again(const LatentAttnParams& p, const int4& g, const Heads& hd, int r, int64_t row, int from, int to) {
    const Request q = load_request(p, g.x, false);
    const int tok0 = g.y - q.s0, first = q.len - q.T;
    if (q.len >= 0) again<FP8>(p, g.x, row, first + tok0 + r / hd.each + 1, first + min(tok0 + hd.tpb, q.T), from, to);
}

// Row of out of row r of the unit, or −1.  by_each: ⌈2^16/heads of a token⌉, whose product with r < 64 has r/heads above bit 16.
__device__ __forceinline__ int64_t join_row(const LatentAttnParams& p, const int4& g, const Heads& hd, int by_each, int r) {
    const int tok = r * by_each >> 16, h = r - tok * hd.each;
    return r < g.z && h < hd.n ? (static_cast<int64_t>(g.y) + tok) * p.n_q + hd.first + h : -1;
}
// 16 rows and 32 dims, by a warp.
template <bool FP8>
__device__ __forceinline__ void join_few(const LatentAttnParams& p, const int4& g, const Heads& hd, int by_each, int cta, int group, int chunk) {
    constexpr int kN = kJoinDims / 8;
    static_assert(kN == 4, "whole_group's");
    const int lane = threadIdx.x & 31, quad = lane & 3, r0 = group * 16 + (lane >> 2);
    float4 acc[kN];
    float top[2], sum[2], cut[2];
    join_parts<kN, 2>(p, cta, hd.blocks, g.w, 0, 1, group, kN * chunk, lane, acc, top, sum, cut);
    const int64_t row[2] = {join_row(p, g, hd, by_each, r0), join_row(p, g, hd, by_each, r0 + 8)};
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float inv = cut[h] == 0.f ? 0.f : 1.f / cut[h];
        float odd = 0.f;
        uint32_t t[kN];
        #pragma unroll
        for (int j = 0; j < kN; ++j) {
            const float a = h ? acc[j].z : acc[j].x, b = h ? acc[j].w : acc[j].y;
            odd += a + b;
            t[j] = pack_bf16(a * inv, b * inv);
            if (p.out_f32 && row[h] >= 0) put2(p, row[h], kJoinDims * chunk + 8 * j + 2 * quad, a, b, inv);
        }
        if (!p.out_f32) {
            const uint4 g8 = whole_group(t, lane);
            if (row[h] >= 0) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row[h] * kLatDim + kJoinDims * chunk + 8 * quad) = g8;
        }
        if (row[h] >= 0 && chunk == 0 && quad == 0 && p.lse_out) p.lse_out[row[h]] = sum[h] == 0.f ? -INFINITY : (top[h] + log2f(sum[h])) * kLn2;
        for (unsigned todo = __ballot_sync(kFull, row[h] >= 0 && odd != odd); todo;) {
            const int i = (__ffs(todo) - 1) >> 2, r = group * 16 + 8 * h + i;
            todo &= ~(15u << 4 * i);
            __syncwarp();
            join_again<FP8>(p, g, hd, r, join_row(p, g, hd, by_each, r), kJoinDims * chunk, kJoinDims * (chunk + 1));
        }
    }
}
// 16 rows and eight dims, by a CTA.
template <bool FP8>
__device__ __forceinline__ void join_many(Join& s, const LatentAttnParams& p, const int4& g, const Heads& hd, int by_each, int cta, int group, int eight) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3, i0 = lane >> 2;
    float4 acc[1];
    float top[2], sum[2], cut[2];
    join_parts<1, 8>(p, cta, hd.blocks, g.w, warp, kJoinWarps, group, eight, lane, acc, top, sum, cut);
    __syncthreads();   // what the one before left has been read
    s.part[warp][lane] = acc[0];
    if (quad == 0) {
        s.top[warp][i0] = top[0];
        s.top[warp][i0 + 8] = top[1];
        s.sum[warp][i0] = sum[0];
        s.sum[warp][i0 + 8] = sum[1];
        s.cut[warp][i0] = cut[0];
        s.cut[warp][i0 + 8] = cut[1];
    }
    __syncthreads();
    // a warp (of the first eight) writes rows `warp` and `warp` + 8 of the group, eight lanes the eight dims of both
    float odd = 0.f;
    if (lane < 8 && warp < 8) {
        const int h = lane >> 2, i = warp + 8 * h;
        float a = 0.f, b = 0.f, l = 0.f, c = 0.f, m = s.top[0][i];
        #pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) m = fmaxf(m, s.top[k][i]);
        #pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) {
            const float4 x = s.part[k][4 * warp + quad];
            const float f = ex2(s.top[k][i] - (m == -INFINITY ? 0.f : m));
            a = fmaf(f, h ? x.z : x.x, a);
            b = fmaf(f, h ? x.w : x.y, b);
            l = fmaf(f, s.sum[k][i], l);
            c = fmaf(f, s.cut[k][i], c);
        }
        const int64_t row = join_row(p, g, hd, by_each, group * 16 + i);
        if (row >= 0) {
            put2(p, row, 8 * eight + 2 * quad, a, b, c == 0.f ? 0.f : 1.f / c);
            if (eight == 0 && quad == 0 && p.lse_out) p.lse_out[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            odd = a + b;
        }
    }
    for (unsigned todo = __ballot_sync(kFull, odd != odd); todo;) {
        const int h = (__ffs(todo) - 1) >> 2, r = group * 16 + warp + 8 * h;
        todo &= ~(15u << 4 * h);
        __syncwarp();
        join_again<FP8>(p, g, hd, r, join_row(p, g, hd, by_each, r), 8 * eight, 8 * eight + 8);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kJoinThreads, 2) join_kernel(const LatentAttnParams p, int ctas) {
    __shared__ Join s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Heads hd(p, 0);
    const int by_each = ((1 << 16) + hd.each - 1) / hd.each;
    pdl_wait();
    pdl_trigger();
    const int few = static_cast<int>(min(max(static_cast<int64_t>(p.n_tokens) * p.n_q / 8, static_cast<int64_t>(8)), static_cast<int64_t>(32)));
    for (int i = tid; i < ctas; i += kJoinThreads) {
        const int4 g = p.part_seg[2 * i + 1];
        const uint32_t n = static_cast<uint32_t>(g.z + 15) / 16;
        s.start[i] = g;
        s.groups[i] = g.x < 0 ? 0u : g.w <= few ? n : n << 16;
    }
    __syncthreads();
    if (warp == 0) {
        uint32_t before = 0;
        for (int i = lane; i - lane < ctas; i += 32) {
            const uint32_t up = before + scan(i < ctas ? s.groups[i] : 0u, lane);
            if (i < ctas) s.groups[i] = up;
            before = __shfl_sync(kFull, up, 31);
        }
    }
    __syncthreads();
    const uint32_t total = s.groups[ctas - 1];
    auto unit_of = [&](int n, int shift, int& group) {   // the CTA that starts group n's unit, and the group in it
        int a = 0, z = ctas - 1;
        while (a < z) {
            const int mid = (a + z) >> 1;
            if (static_cast<int>(s.groups[mid] >> shift & 0xffffu) > n) z = mid;
            else a = mid + 1;
        }
        group = n - (a > 0 ? static_cast<int>(s.groups[a - 1] >> shift & 0xffffu) : 0);
        return a;
    };
    constexpr int kChunks = kLatDim / kJoinDims, kEights = kLatDim / 8;
    for (int item = blockIdx.x * kJoinWarps + warp; item < kChunks * static_cast<int>(total & 0xffffu); item += gridDim.x * kJoinWarps) {
        int group;
        const int cta = unit_of(item / kChunks, 0, group);
        if (hd.blocks > 1) hd.set(p, cta % hd.blocks);
        join_few<FP8>(p, s.start[cta], hd, by_each, cta, group, item % kChunks);
    }
    for (int item = blockIdx.x; item < kEights * static_cast<int>(total >> 16); item += gridDim.x) {
        int group;
        const int cta = unit_of(item / kEights, 16, group);
        if (hd.blocks > 1) hd.set(p, cta % hd.blocks);
        join_many<FP8>(s, p, s.start[cta], hd, by_each, cta, group, item % kEights);
    }
}

template <bool FP8>
cudaError_t launch(const LatentAttnParams& p, int ctas, cudaStream_t stream) {
    static_assert(sizeof(Smem) <= 232448, "shared memory of one SM");
    auto* kernel = p.out_f32 ? attn_kernel<FP8, true> : attn_kernel<FP8, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Smem)));
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), dim3(threads_of(FP8)), sizeof(Smem), -1, stream, p);
    if (e != cudaSuccess) return e;
    return launch_dependent(join_kernel<FP8>, dim3(static_cast<unsigned>(2 * ctas)), dim3(kJoinThreads), 0, -1, stream, p, ctas);
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnParams& p, bool fp8, int num_sms, cudaStream_t stream) {
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    return fp8 ? launch<true>(p, ctas, stream) : launch<false>(p, ctas, stream);
}

}  // namespace kvd
