// kvd_rope.cu — rotary positions of a chunk's queries and keys, fused with the append of its K and V.
//
// Pair j of a head, (x_j, x_{j + rot/2}) or (x_2j, x_{2j+1}), is turned by the angle pos·θ_j:
//   y_a = m·(x_a cos − x_b sin),  y_b = m·(x_a sin + x_b cos);  dims past rot pass through.
// The queries go to q_out; the keys, rounded to bf16, and the values go to their pool slots as
// the plain append writes them, so rope + append is bit for bit the two steps in a row.
//
// Angles: θ_j is given in turns per position as an fp32 pair hi + lo (48 bits).  p = pos·hi has
// its rounding error in one fma, so frac(p) + error + pos·lo is the position's place in the turn to
// about 2^-25 for every pos < 2^24, where a single fp32 product is off by up to pos·θ·2^-24 radians
// (0.008 at position 131,072).  cos and sin come once per (token, pair) of a CTA and serve its heads: two or eight query
// heads, or K of one or four KV heads.
//
// Bound: HBM, 4·128 B per query row and 8·128 B per (token, KV head) against a few FMAs per element: 8,192 tokens
// of 32 + 8 heads take 45 us (4.5 TB/s, 67% of the measured bandwidth: a CTA's loads, its angles and its stores follow
// one another, and three CTAs an SM do not cover all of it; the angles of a token are made in six CTAs), 4,099 tokens of
// 64 + 8 heads, half rotated, 30.5 us (83%).  At 80 registers some 28 bytes a thread are spilled.
#include "kvd_chunk.h"
#include "kvd_common.cuh"

namespace kvd {
namespace {

constexpr int kTok = 16;               // tokens per CTA: the most that share a block
constexpr int kRopeThreads = 256;
constexpr int kRowPad = kDh + 8;       // bf16 elements per staged row (bank spread)
constexpr int kRows = 8;               // rows a thread holds: query heads, or K and V of half as many KV heads

struct RopeSmem {
    float2 cs[kTok][kDh / 2];                              // (cos, sin)·m per (token, pair)
    __align__(16) uint16_t krow[2][kTok][kRowPad];         // rotated K rows of one head, then its V rows
    int64_t slot[kTok];
    uint8_t* record[kTok];                                 // of the token's K and V (the first head's), or null
    int pos[kTok];
    int src[kBs];                                          // the token that goes to slot offset t, or -1
    int ok[kTok];                                          // the token takes part
    int shared_offset;                                     // two tokens want the same slot offset
};

// (cos, sin)·m of a lane's 8 consecutive dims (lane16 = lane % 16): by pair if neighbours are paired, else by dim, where
// the sine has the sign with which it multiplies the partner.
template <bool INTERLEAVED>
__device__ __forceinline__ void lane_factors(float2 (&f)[8], const float2* cs, int rot, int lane16) {
    const int half = rot >> 1;
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = lane16 * 8 + e;
        f[e] = make_float2(1.f, 0.f);
        const int pair = INTERLEAVED ? lane16 * 4 + e : d < half ? d : d - half;
        if (INTERLEAVED ? e < 4 && pair < half : d < rot) f[e] = cs[pair];
        if (!INTERLEAVED && d < half) f[e].y = -f[e].y;
    }
}

// One row of 128 values by 16 lanes, 8 consecutive dims each, rotated in fp32 and rounded to bf16.
template <bool INTERLEAVED>
__device__ __forceinline__ uint4 rotate_row(uint4 raw, const float2 (&f)[8], int rot, int lane16) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t out[4];
    if constexpr (INTERLEAVED) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack_bf16(w[i]), c = f[i];
            const uint32_t v = pack_bf16(x.x * c.x - x.y * c.y, x.x * c.y + x.y * c.x);
            out[i] = lane16 * 8 + 2 * i < rot ? v : w[i];
        }
        return make_uint4(out[0], out[1], out[2], out[3]);
    }
    const int half = rot >> 1;
    float x[8], y[8];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_bf16(w[i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
    }
    const int lane = threadIdx.x & 31;
    // The partner of dim d is d + half (d < half) or d − half.  Its lane and word are fetched by
    // shuffles: with half = 8·hl + hr the element at offset e has its partner at offset e ± hr, one
    // lane further when that leaves the lane's eight.
    const int hl = half >> 3, hr = half & 7;
    const int base = lane & 16;
    if (hr == 0) {
        const bool low = lane16 < hl;
        const int other = base | ((low ? lane16 + hl : lane16 - hl) & 15);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 pv = unpack_bf16(__shfl_sync(kFull, w[i], other));
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int e = 2 * i + k;
                const float b = k ? pv.y : pv.x;
                y[e] = fmaf(b, f[e].y, x[e] * f[e].x);
            }
        }
    } else {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = lane16 * 8 + e;
            const bool low = d < half;
            const int pd = (low ? d + half : d - half) & (kDh - 1);
            // every lane reads the wanted word of its partner lane: four shuffles, one selected
            uint32_t pw = 0;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = __shfl_sync(kFull, w[i], base | (pd >> 3));
                if (((pd & 7) >> 1) == i) pw = v;
            }
            const float2 pv = unpack_bf16(pw);
            const float b = (pd & 1) ? pv.y : pv.x;
            y[e] = fmaf(b, f[e].y, x[e] * f[e].x);
        }
    }
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        // dims past rot keep their bits (a NaN's payload too)
        const int d = lane16 * 8 + 2 * i;
        const uint32_t v = pack_bf16(y[2 * i], y[2 * i + 1]);
        out[i] = d < rot ? v : w[i];   // (rot is even)
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int KIND, int NG>
__device__ __forceinline__ int64_t record_size() {
    constexpr int kBits = KIND == kKindInt4 ? 4 : 2;
    return KIND == kKindFp8 || KIND == kKindAngle ? kRecordFp8
           : is_lowbit(KIND)                      ? lowbit_record_bytes(kBits, NG)
                                                  : kRecordBf16;
}

// The K and V rows of one token of one head, from shared memory, into its record: as the append.
template <int KIND, int NG>
__device__ __forceinline__ void put_token(const RopeParams& p, uint8_t* record, int64_t blk, int t,
                                          const uint16_t* k, const uint16_t* v, int lane) {
    if constexpr (is_lowbit(KIND)) {
        write_token_lowbit<KIND == kKindInt4 ? 4 : 2, NG>(record, t, k, v, lane);
    } else if constexpr (KIND == kKindAngle) {
        write_token<kFmtE4m3, true>(record, t, k, v, lane);
    } else if constexpr (KIND == kKindMixed) {
        const int fmt = block_format(p.block_fmt[blk]);
        if (fmt == kFmtBf16) write_token<kFmtBf16>(record, t, k, v, lane);
        else if (fmt == kFmtE4m3) write_token<kFmtE4m3>(record, t, k, v, lane);
        else if (fmt == kFmtE5m2) write_token<kFmtE5m2>(record, t, k, v, lane);
        else if (lane == 0) report(p.err, KVD_ERR_OOB);
    } else {
        write_token<KIND == kKindFp8 ? kFmtE4m3 : kFmtBf16>(record, t, k, v, lane);
    }
}

// CTA (tile of 16 tokens, group of query heads or one KV head).  A thread has all its rows' loads under way
// before the angles are there.  A KV head's tiles start at a multiple of 16 slots behind the first token's block start, so a
// chunk of one request fills whole blocks (a record's 16-byte pieces hold two or four of its tokens).
template <int KIND, int NG, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_append_kernel(const RopeParams p) {
    __shared__ RopeSmem s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int groups = (p.n_q + p.heads_per_cta - 1) / p.heads_per_cta;
    const bool query = static_cast<int>(blockIdx.y) < groups;
    int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTok;
    if (!query) {
        const int64_t first = p.slot_mapping[0];
        n0 -= first > 0 ? first % kBs : 0;
    }
    const int h0 = query ? blockIdx.y * p.heads_per_cta : (blockIdx.y - groups) * p.kv_heads_per_cta;
    const int heads = query ? min(p.heads_per_cta, p.n_q - h0) : min(p.kv_heads_per_cta, p.n_kv - h0);
    const int half_id = tid >> 4, lane16 = tid & 15;   // 16 half-warps, a token each
    const int64_t row = n0 + half_id;
    uint4 x[kRows];
    #pragma unroll
    for (int i = 0; i < kRows; ++i) x[i] = make_uint4(0, 0, 0, 0);
    if (row >= 0 && row < p.n_tokens) {
        if (query) {
            #pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (i < heads) x[i] = *reinterpret_cast<const uint4*>(p.q + row * p.q_stride + (h0 + i) * kDh + lane16 * 8);
        } else {
            #pragma unroll
            for (int i = 0; i < kRows; i += 2) {
                if (i / 2 >= heads) continue;
                x[i] = *reinterpret_cast<const uint4*>(p.k + row * p.k_stride + (h0 + i / 2) * kDh + lane16 * 8);
                x[i + 1] = *reinterpret_cast<const uint4*>(p.v + row * p.v_stride + (h0 + i / 2) * kDh + lane16 * 8);
            }
        }
    }
    if (tid < kTok) {
        const int64_t n = n0 + tid;
        int ok = n >= 0 && n < p.n_tokens;
        int64_t slot = -1;
        int pos = 0;
        if (ok) {
            pos = p.positions[n];
            if (!query) slot = p.slot_mapping[n];
            if (pos < 0 || pos >= kMaxRopePos) {
                if (blockIdx.y == 0) report(p.err, KVD_ERR_OOB);
                ok = 0;
                slot = -1;
            } else if (slot >= 0 && slot / kBs >= p.num_blocks + p.host_blocks) {
                if (h0 == 0) report(p.err, KVD_ERR_OOB);
                slot = -1;
            }
        }
        const int64_t blk = slot / kBs;
        s.ok[tid] = ok;
        s.pos[tid] = pos;
        s.slot[tid] = slot;
        s.record[tid] = slot < 0 || query ? nullptr
                        : blk < p.num_blocks ? p.kv + (blk * p.n_kv + h0) * record_size<KIND, NG>()
                                             : p.host_kv + ((blk - p.num_blocks) * p.n_kv + h0) * record_size<KIND, NG>();
    }
    __syncthreads();
    if (!query && tid < kBs) {   // slot offset -> token
        int found = -1, twice = 0;
        for (int i = 0; i < kTok; ++i) {
            if (s.slot[i] >= 0 && s.slot[i] % kBs == tid) {
                twice |= found >= 0;
                found = i;
            }
        }
        s.src[tid] = found;
        const unsigned any = __ballot_sync(0xffffu, twice);
        if (tid == 0) s.shared_offset = any != 0;
    }
    const int pairs = p.rot >> 1;
    const float pos = static_cast<float>(s.pos[half_id]);
    for (int j = lane16; j < pairs; j += 16) {
        const float2 f = p.turns[j];
        const float a = __fmul_rn(pos, f.x);
        const float rest = __fmaf_rn(pos, f.x, -a);
        const float turn = __fadd_rn(__fsub_rn(a, rintf(a)), __fmaf_rn(pos, f.y, rest));
        float sn, cn;
        sincospif(2.f * turn, &sn, &cn);
        s.cs[half_id][j] = make_float2(cn * p.mscale, sn * p.mscale);
    }
    __syncthreads();
    float2 factor[8];
    lane_factors<INTERLEAVED>(factor, s.cs[half_id], p.rot, lane16);
    if (query) {
        #pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i >= heads) break;
            const uint4 y = rotate_row<INTERLEAVED>(x[i], factor, p.rot, lane16);
            if (s.ok[half_id]) *reinterpret_cast<uint4*>(p.q_out + row * p.q_out_stride + (h0 + i) * kDh + lane16 * 8) = y;
        }
        return;
    }
    #pragma unroll
    for (int h = 0; h < kRows / 2; ++h) {
        if (h >= heads) break;
        if (h) __syncthreads();   // the head before has been written out
        *reinterpret_cast<uint4*>(&s.krow[0][half_id][lane16 * 8]) = rotate_row<INTERLEAVED>(x[2 * h], factor, p.rot, lane16);
        *reinterpret_cast<uint4*>(&s.krow[1][half_id][lane16 * 8]) = x[2 * h + 1];
        __syncthreads();
        auto record = [&](int tk) -> uint8_t* { return s.record[tk] ? s.record[tk] + h * record_size<KIND, NG>() : nullptr; };
        if (KIND == kKindBf16 && !s.shared_offset) {
            // 16-byte pieces of the two tiles: a K piece holds dims (2x, 2x+1, 2x+8, 2x+9) of tokens
            // t and t + 8, a V piece tokens (2x, 2x+1, 2x+8, 2x+9) of dims r and r + 8.  Whole
            // pieces where their tokens go to the same record, smaller stores where they do not.
            for (int c = tid; c < 512; c += kRopeThreads) {
                const int i = (c >> 5) & 7, l = c & 31, x4 = l & 3, r = l >> 2;
                if (c < 256) {
                    const int ta = s.src[r], tb = s.src[r + 8];
                    const int d = 16 * i + 2 * x4;
                    uint32_t a0 = 0, a1 = 0, b0 = 0, b1 = 0;
                    if (ta >= 0) {
                        a0 = *reinterpret_cast<const uint32_t*>(&s.krow[0][ta][d]);
                        a1 = *reinterpret_cast<const uint32_t*>(&s.krow[0][ta][d + 8]);
                    }
                    if (tb >= 0) {
                        b0 = *reinterpret_cast<const uint32_t*>(&s.krow[0][tb][d]);
                        b1 = *reinterpret_cast<const uint32_t*>(&s.krow[0][tb][d + 8]);
                    }
                    uint8_t* pa = ta >= 0 ? record(ta) : nullptr;
                    uint8_t* pb = tb >= 0 ? record(tb) : nullptr;
                    if (pa == pb) {
                        if (pa) *reinterpret_cast<uint4*>(pa + c * 16) = make_uint4(a0, b0, a1, b1);
                    } else {
                        if (pa) {
                            *reinterpret_cast<uint32_t*>(pa + c * 16) = a0;
                            *reinterpret_cast<uint32_t*>(pa + c * 16 + 8) = a1;
                        }
                        if (pb) {
                            *reinterpret_cast<uint32_t*>(pb + c * 16 + 4) = b0;
                            *reinterpret_cast<uint32_t*>(pb + c * 16 + 12) = b1;
                        }
                    }
                } else {
                    const int d = 16 * i + r;
                    uint16_t lo[4], hi[4];
                    uint8_t* rec[4];
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tk = s.src[2 * x4 + (k & 1) + 8 * (k >> 1)];
                        rec[k] = tk >= 0 ? record(tk) : nullptr;
                        lo[k] = tk >= 0 ? s.krow[1][tk][d] : 0;
                        hi[k] = tk >= 0 ? s.krow[1][tk][d + 8] : 0;
                    }
                    const int off = c * 16;   // the V tile follows the K tile: pieces 256 .. 511
                    auto two = [](uint16_t a, uint16_t b) { return a | (static_cast<uint32_t>(b) << 16); };
                    if (rec[0] == rec[1] && rec[0] == rec[2] && rec[0] == rec[3]) {
                        if (rec[0])
                            *reinterpret_cast<uint4*>(rec[0] + off) =
                                make_uint4(two(lo[0], lo[1]), two(hi[0], hi[1]), two(lo[2], lo[3]), two(hi[2], hi[3]));
                    } else {
                        #pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (!rec[k]) continue;
                            const int at = off + (k & 1) * 2 + (k >> 1) * 8;
                            *reinterpret_cast<uint16_t*>(rec[k] + at) = lo[k];
                            *reinterpret_cast<uint16_t*>(rec[k] + at + 4) = hi[k];
                        }
                    }
                }
            }
        } else {
            for (int tk = warp; tk < kTok; tk += kRopeThreads / 32) {
                if (s.slot[tk] < 0) continue;
                put_token<KIND, NG>(p, record(tk), s.slot[tk] / kBs, static_cast<int>(s.slot[tk] % kBs), s.krow[0][tk],
                                    s.krow[1][tk], lane);
            }
        }
    }
}

template <int KIND, int NG>
cudaError_t launch(const RopeParams& p, dim3 grid, cudaStream_t stream) {
    return p.interleaved ? launch_dependent(rope_append_kernel<KIND, NG, true>, grid, dim3(kRopeThreads), 0, -1, stream, p)
                         : launch_dependent(rope_append_kernel<KIND, NG, false>, grid, dim3(kRopeThreads), 0, -1, stream, p);
}

}  // namespace

cudaError_t launch_rope_append(RopeParams p, int kind, int num_sms, cudaStream_t stream) {
    const int64_t tiles = (p.n_tokens + kTok - 1) / kTok + 1;   // one more: the first tile may start before token 0
    // Eight query heads (four KV heads) a CTA where that leaves four CTAs an SM: the angles are computed once for
    // them; else two (one).  8,192 tokens of 32 + 8 heads take 45 us so, 87 us the other way; a step of 32 tokens takes
    // 4.7 us the other way, 11.1 us so.
    const bool many = tiles * ((p.n_q + 7) / 8) >= 4 * num_sms;
    p.heads_per_cta = many ? 8 : 2;
    p.kv_heads_per_cta = many ? 4 : 1;
    const int groups = (p.n_q + p.heads_per_cta - 1) / p.heads_per_cta;
    const int kv_groups = (p.n_kv + p.kv_heads_per_cta - 1) / p.kv_heads_per_cta;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(groups + kv_groups));
    switch (kind) {
        case kKindFp8: return launch<kKindFp8, 1>(p, grid, stream);
        case kKindMixed: return launch<kKindMixed, 1>(p, grid, stream);
        case kKindAngle: return launch<kKindAngle, 1>(p, grid, stream);
        case kKindInt4:
            return p.ng == 4   ? launch<kKindInt4, 4>(p, grid, stream)
                   : p.ng == 2 ? launch<kKindInt4, 2>(p, grid, stream)
                               : launch<kKindInt4, 1>(p, grid, stream);
        case kKindInt2:
            return p.ng == 4   ? launch<kKindInt2, 4>(p, grid, stream)
                   : p.ng == 2 ? launch<kKindInt2, 2>(p, grid, stream)
                               : launch<kKindInt2, 1>(p, grid, stream);
        default: return launch<kKindBf16, 1>(p, grid, stream);
    }
}

}  // namespace kvd
