// kvd_latent_attn.cu — absorbed latent attention over the paged cache.
//
// Row (token i of the T new tokens of request b, head h), len = seq_lens[b], P = len − T + i:
//   l_t = scale·<q, (c_t, r_t)> over 512 + 64 dims, t ≤ P and retained;  out = Σ_t softmax(l)_t·c_t,  lse = log Σ exp(l_t).
// A warp a row: a lane has dims 8·lane .. +7 and 256 + 8·lane .. +7 of the latent, lanes 0 .. 7 the rotated ones.
#include "kvd_common.cuh"
#include "kvd_latent.h"

namespace kvd {
namespace {

constexpr int kThreads = 256;

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

template <bool FP8>
__global__ void __launch_bounds__(kThreads) attn_kernel(const LatentAttnParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int s0 = p.q_start[b], s1 = p.q_start[b + 1], len = p.seq_lens[b];
    if (s0 < 0 || s1 < s0 || s1 > p.n_tokens) {
        if (threadIdx.x == 0) report(p.err, KVD_ERR_OOB);
        return;
    }
    const int T = s1 - s0;
    if (T == 0) return;
    const bool good = len >= T && static_cast<int64_t>(len) <= static_cast<int64_t>(p.max_blocks) * kBs;
    if (!good && threadIdx.x == 0) report(p.err, KVD_ERR_OOB);
    const int64_t rows = static_cast<int64_t>(T) * p.n_q, warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
        const int64_t row = static_cast<int64_t>(s0) * p.n_q + r;
        const uint16_t* qr = p.q + row * kLatKey;
        float q[24], acc[16], m = -INFINITY, sum = 0.f;
        unpack8(q, ld16(qr + lane * 8));
        unpack8(q + 8, ld16(qr + 256 + lane * 8));
        unpack8(q + 16, lane < 8 ? ld16(qr + kLatDim + lane * 8) : make_uint4(0, 0, 0, 0));
        #pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        const int end = good ? len - T + static_cast<int>(r / p.n_q) + 1 : 0;
        for (int pos = 0; pos < end; ++pos) {
            const int64_t block = p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kBs];
            const int t = pos % kBs;
            if (block < 0 || block >= p.num_blocks) {
                if (lane == 0 && t == 0) report(p.err, KVD_ERR_OOB);
                continue;
            }
            if (p.retain && !((p.retain[block] >> t) & 1)) continue;
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
            const int64_t at = row * kLatDim + (i >> 3) * 256 + lane * 8 + (i & 7);
            if (p.out_f32) static_cast<float*>(p.out)[at] = acc[i] * inv;
            else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(acc[i] * inv);
        }
        if (lane == 0 && p.lse_out) p.lse_out[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
    }
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnParams& p, bool fp8, int num_sms, cudaStream_t stream) {
    const int64_t most = (static_cast<int64_t>(p.n_tokens) * p.n_q + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t share = (16 * num_sms + p.B - 1) / p.B;
    const dim3 grid(static_cast<unsigned>(most < share ? most : share), static_cast<unsigned>(p.B));
    return launch_dependent(fp8 ? attn_kernel<true> : attn_kernel<false>, grid, dim3(kThreads), 0, -1, stream, p);
}

}  // namespace kvd
