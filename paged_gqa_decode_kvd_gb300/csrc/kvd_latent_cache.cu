// kvd_latent_cache.cu — the latent cache is written (norm, rotation, quantisation) and read back.
//
// Append, token n with latent x, key part k and position p:
//   y = x·w / sqrt(mean(x²) + eps)      (w: the norm's weights; without them y = x)
//   r = R(p)·k, and for every query head q' = R(p)·q, R the rotation of kvd_rope_append over 64 dims
//   bf16 record: y and r rounded to bf16; 8-bit record: s = fp32(max|y|/448) (1 where that is 0), codes e4m3(y/s),
//   rounded once from fp32, and r in bf16.
// Read back: y (code·s, rounded to bf16) and r, side by side.
//
// Bound: HBM.  4,099 tokens into 8 bits with 128 heads' queries: 26.6 us, 5.3 TB/s (78% of measured: 67 MB of queries are read and written in
// pieces of 128 bytes); with halves paired 32.4 us (every dim's partner and angle come from other lanes); a decode step of 32 tokens: 2.6 us in a graph, 11 with the host call.  226,000 rows of 24 requests from 8 bits: 64 us,
// 6.3 TB/s (93%).
#include "kvd_common.cuh"
#include "kvd_latent.h"

namespace kvd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPos = 1 << 24;       // positions a float holds exactly

__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(void* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// cos and sin (times m) of a lane's 8 dims of a rotated vector of 64: by pair if neighbours are paired, else by dim,
// where the sine has the sign with which it multiplies the partner.  Angles as in kvd_rope_append: turns per position as
// hi + lo, the rounding error of pos·hi from one fma.  A lane makes one pair's, and the warp hands them round.
template <bool INTERLEAVED>
__device__ __forceinline__ void lane_turns(float2 (&f)[8], const LatentAppendParams& p, float pos, int lane) {
    const int half = p.rot >> 1, lane8 = lane & 7;
    float2 mine = make_float2(1.f, 0.f);
    if (lane < half) {
        const float2 t = p.turns[lane];
        const float a = __fmul_rn(pos, t.x);
        const float rest = __fmaf_rn(pos, t.x, -a);
        const float turn = __fadd_rn(__fsub_rn(a, rintf(a)), __fmaf_rn(pos, t.y, rest));
        float sn, cn;
        sincospif(2.f * turn, &sn, &cn);
        mine = make_float2(cn * p.mscale, sn * p.mscale);
    }
    #pragma unroll
    for (int e = 0; e < (INTERLEAVED ? 4 : 8); ++e) {
        const int d = lane8 * 8 + e;
        const int pair = INTERLEAVED ? lane8 * 4 + e : d < half ? d : d - half;
        f[e] = make_float2(__shfl_sync(kFull, mine.x, pair & 31), __shfl_sync(kFull, mine.y, pair & 31));
        if (!INTERLEAVED && d < half) f[e].y = -f[e].y;
    }
}

// Eight dims of a vector of 64 by each of 8 lanes, rotated in fp32 and rounded to bf16; dims past rot keep their bits.
// row: the vector in memory, for partners that do not stand in one lane's piece.
template <bool INTERLEAVED>
__device__ __forceinline__ uint4 rotate8(uint4 raw, const float2 (&f)[8], int rot, int lane8, const uint16_t* row, bool on) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t o[4];
    if constexpr (INTERLEAVED) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack_bf16(w[i]), c = f[i];
            const uint32_t v = pack_bf16(x.x * c.x - x.y * c.y, x.x * c.y + x.y * c.x);
            o[i] = lane8 * 8 + 2 * i < rot ? v : w[i];
        }
    } else {
        const int half = rot >> 1, lanes = half >> 3, lane = threadIdx.x & 31;
        const bool whole = (half & 7) == 0;   // partners stand half/8 lanes apart, at the same place
        const int other = (lane & 24) | ((lane8 < lanes ? lane8 + lanes : lane8 - lanes) & 7);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack_bf16(w[i]);
            float2 y = unpack_bf16(__shfl_sync(kFull, w[i], other));
            if (!whole && on) {
                const int d = lane8 * 8 + 2 * i;
                const int a = d < half ? d + half : d - half, b = d + 1 < half ? d + 1 + half : d + 1 - half;
                if (d < rot) {   // (rot is even)
                    y.x = __uint_as_float(static_cast<uint32_t>(row[a]) << 16);
                    y.y = __uint_as_float(static_cast<uint32_t>(row[b]) << 16);
                }
            }
            const uint32_t v = pack_bf16(fmaf(y.x, f[2 * i].y, x.x * f[2 * i].x), fmaf(y.y, f[2 * i + 1].y, x.y * f[2 * i + 1].x));
            o[i] = lane8 * 8 + 2 * i < rot ? v : w[i];
        }
        __syncwarp();   // every partner is read before any lane's result is written over it
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void unpack8(float* x, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = unpack_bf16(w[i]);
        x[2 * i] = a.x;
        x[2 * i + 1] = a.y;
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint32_t codes4(const float* x, float s) {
    const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[0], s), __fdiv_rn(x[1], s)), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2], s), __fdiv_rn(x[3], s)), __NV_SATFINITE, __NV_E4M3);
    return static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 16);
}

// A warp takes one token's latent and key part, or p.heads of its query heads, four at a time.  Neighbours paired: five CTAs an SM (48
// registers, 4 to 8 bytes spilled) take 26.2 us for the prompt above, four 27.5, six 26.4.  Halves paired, a lane has eight dims' cos and sin
// in place of four pairs': at five 100 bytes are spilled and more loaded again, in the queries' path too: 34.9 us, with four 32.4, with three
// 38.9; 7,700 tokens of 32 heads in BF16 23.4, 21.3 and 25.8.
template <bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, INTERLEAVED ? 5 : 4) append_kernel(const LatentAppendParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, lane8 = lane & 7;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int groups = (p.n_q + p.heads - 1) / p.heads;
    if (task >= p.n_tokens * (1 + groups)) return;
    const bool query = task >= p.n_tokens;
    const int64_t n = query ? (task - p.n_tokens) / groups : task;
    int pos = 0;
    if (p.turns) {
        pos = p.positions[n];
        if (pos < 0 || pos >= kMaxPos) {
            if (lane == 0) report(p.err, KVD_ERR_OOB);
            return;
        }
    }
    float2 f[8];
    if (query) {
        const int h0 = static_cast<int>((task - p.n_tokens) % groups) * p.heads, h1 = min(h0 + p.heads, p.n_q);
        lane_turns<INTERLEAVED>(f, p, static_cast<float>(pos), lane);
        const uint16_t* src = p.q_rope + n * p.q_stride;
        uint16_t* dst = p.q_out + n * p.out_stride;
        #pragma unroll 1
        for (int h = h0 + (lane >> 3); h - (lane >> 3) < h1; h += 16) {
            uint4 x[4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = h + 4 * i < h1 ? ld16(src + (h + 4 * i) * p.q_head + lane8 * 8) : make_uint4(0, 0, 0, 0);
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (h + 4 * i - (lane >> 3) >= h1) break;
                const bool on = h + 4 * i < h1;
                const uint4 y = rotate8<INTERLEAVED>(x[i], f, p.rot, lane8, src + (h + 4 * i) * p.q_head, on);
                if (on) st16(dst + (h + 4 * i) * p.out_head + lane8 * 8, y);
            }
        }
        return;
    }
    const int64_t slot = p.slot_mapping[n];
    if (slot < 0) return;
    if (slot >= p.num_blocks * kBs) {
        if (lane == 0) report(p.err, KVD_ERR_OOB);
        return;
    }
    uint8_t* record = p.mem + (slot / kBs) * latent_record_bytes(FP8);
    const int t = static_cast<int>(slot % kBs);
    const uint16_t* row = p.latent + n * p.latent_stride;
    const uint16_t* key = p.k_rope + n * p.k_stride;
    uint4 raw[2] = {ld16(row + lane * 8), ld16(row + 256 + lane * 8)};
    uint4 rot = lane < 8 ? ld16(key + lane8 * 8) : make_uint4(0, 0, 0, 0);
    if (p.turns) {
        lane_turns<INTERLEAVED>(f, p, static_cast<float>(pos), lane);
        rot = rotate8<INTERLEAVED>(rot, f, p.rot, lane8, key, lane < 8);
    }
    float x[16];
    if (FP8 || p.norm) {
        unpack8(x, raw[0]);
        unpack8(x + 8, raw[1]);
    }
    if (p.norm) {
        float w[16], sum = 0.f;
        unpack8(w, ld16(p.norm + lane * 8));
        unpack8(w + 8, ld16(p.norm + 256 + lane * 8));
        #pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        const float r = __frcp_rn(__fsqrt_rn(fmaf(sum, 1.f / kLatDim, p.eps)));
        #pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
        raw[0] = pack8(x);
        raw[1] = pack8(x + 8);
    }
    if constexpr (FP8) {
        float top = 0.f;
        #pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        float s = __fdiv_rn(top, 448.f);
        if (s == 0.f) s = 1.f;   // (a row of zeros, or of a few times fp32's smallest value)
        #pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint2*>(record + latent_code(t, lane + 32 * i)) = make_uint2(codes4(x + 8 * i, s), codes4(x + 8 * i + 4, s));
        if (lane < 8) st16(record + latent_rope_piece(t, lane), rot);
        if (lane == 0) *reinterpret_cast<float*>(record + kLatScales + 4 * t) = s;
    } else {
        #pragma unroll
        for (int i = 0; i < 2; ++i) st16(record + latent_piece(t, lane + 32 * i), raw[i]);
        if (lane < 8) st16(record + latent_piece(t, 64 + lane), rot);
    }
}

// Rows in chunks of eight, one a warp; a CTA takes every gridDim-th chunk of all requests.  226,000 rows of 24 requests from
// 8 bits take 64.5 us so, at eight CTAs an SM; with four rows a warp, all loads under way, and four CTAs 76 us, with two 75 us.
constexpr int kChunkRows = kThreads / 32, kGatherCtas = 8;
// Pairs that are sound by themselves may overlap where others are not, and add up to more than 32 bits.  Counts stop here, far above
// what rows that are apart can be, and the requests behind are skipped (64 bits: the prefix of 8,192 4.6 us instead of 4.3, the
// 226,000 rows 65.6 instead of 64.4).
constexpr int kMostChunks = (1 << 30) - 1;
template <bool FP8>
__global__ void __launch_bounds__(kThreads, kGatherCtas) gather_kernel(const LatentGatherParams p) {
    __shared__ int chunks[kMaxBatch];   // up to and with the request
    __shared__ int warp_sum[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        int up = 0;
        if (b < p.B) {
            const int64_t r0 = p.row_start[b], r1 = p.row_start[b + 1], first = p.first ? p.first[b] : 0;
            if (r0 < 0 || r1 < r0 || r1 > p.n_rows || first < 0 || first + (r1 - r0) > static_cast<int64_t>(p.max_blocks) * kBs) {
                if (blockIdx.x == 0) report(p.err, KVD_ERR_OOB);
            } else {
                up = static_cast<int>((r1 - r0 + kChunkRows - 1) / kChunkRows);
            }
        }
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, up, o);
            if (lane >= o) up = min(up + v, kMostChunks);
        }
        if (lane == 31) warp_sum[warp] = up;
        __syncthreads();
        int all = before;
        #pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) up = min(up + warp_sum[w], kMostChunks);
            all = min(all + warp_sum[w], kMostChunks);
        }
        if (b < p.B) chunks[b] = min(before + up, kMostChunks);
        before = all;
        __syncthreads();
    }
    for (int c = blockIdx.x; c < before; c += gridDim.x) {
        int b = 0, z = p.B - 1;
        while (b < z) {   // the first request with more than c chunks up to it
            const int mid = (b + z) >> 1;
            if (chunks[mid] > c) z = mid;
            else b = mid + 1;
        }
        const int64_t r0 = p.row_start[b], r1 = p.row_start[b + 1], first = p.first ? p.first[b] : 0;
        const int64_t row = r0 + static_cast<int64_t>(c - (b > 0 ? chunks[b - 1] : 0)) * kChunkRows + warp, pos = first + (row - r0);
        if (row >= r1) continue;
        const int64_t block = p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kBs];
        if (block < 0 || block >= p.num_blocks) {
            if (lane == 0) report(p.err, KVD_ERR_OOB);
            continue;
        }
        const int t = static_cast<int>(pos % kBs);
        const uint8_t* record = p.mem + block * latent_record_bytes(FP8);
        uint16_t* out = p.out + row * p.out_stride;
        const uint4 rope = lane >= 8 ? make_uint4(0, 0, 0, 0) : ld16(record + (FP8 ? latent_rope_piece(t, lane) : latent_piece(t, 64 + lane)));
        if constexpr (FP8) {
            const uint2 code[2] = {*reinterpret_cast<const uint2*>(record + latent_code(t, lane)),
                                   *reinterpret_cast<const uint2*>(record + latent_code(t, lane + 32))};
            const float s = *reinterpret_cast<const float*>(record + kLatScales + 4 * t);
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t h[4], o[4];
                e4m3x4_to_f16x2x2(code[k].x, h[0], h[1]);
                e4m3x4_to_f16x2x2(code[k].y, h[2], h[3]);
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = unpack_f16(h[j]);
                    o[j] = pack_bf16(v.x * s, v.y * s);
                }
                st16(out + (lane + 32 * k) * 8, make_uint4(o[0], o[1], o[2], o[3]));
            }
        } else {
            const uint4 x[2] = {ld16(record + latent_piece(t, lane)), ld16(record + latent_piece(t, lane + 32))};
            st16(out + lane * 8, x[0]);
            st16(out + (lane + 32) * 8, x[1]);
        }
        if (lane < 8) st16(out + kLatDim + lane * 8, rope);
    }
}

}  // namespace

cudaError_t launch_latent_append(LatentAppendParams p, bool fp8, int num_sms, cudaStream_t stream) {
    // A warp makes a token's cos and sin for its heads: 32 of them where that leaves four warps a scheduler.
    p.heads = p.n_tokens * ((p.n_q + 31) / 32) >= 16 * num_sms ? 32 : 4;
    const int64_t tasks = p.n_tokens * (1 + (p.n_q + p.heads - 1) / p.heads);
    const dim3 grid(static_cast<unsigned>((tasks + kThreads / 32 - 1) / (kThreads / 32)));
    auto* kernel = fp8 ? (p.interleaved ? append_kernel<true, true> : append_kernel<true, false>)
                       : (p.interleaved ? append_kernel<false, true> : append_kernel<false, false>);
    return launch_dependent(kernel, grid, dim3(kThreads), 0, -1, stream, p);
}

cudaError_t launch_latent_gather(const LatentGatherParams& p, bool fp8, int num_sms, cudaStream_t stream) {
    const int64_t most = p.n_rows / kChunkRows + p.B, full = static_cast<int64_t>(kGatherCtas) * num_sms;
    const dim3 grid(static_cast<unsigned>(most < full ? most : full));
    return launch_dependent(fp8 ? gather_kernel<true> : gather_kernel<false>, grid, dim3(kThreads), 0, -1, stream, p);
}

}  // namespace kvd
