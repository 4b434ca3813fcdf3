// kvd_latent_prefill.cu — expanded latent attention: every head has its own 128 dims of key and of value, the 64
// rotated dims of the key are one vector a token.
//
// Row (token i of the T rows of request b, head h) over its N keys, causal: t ≤ N − T + i:
//   l_t = scale·(<q[:128], k_t,h> + <q[128:], r_t>),  out = Σ_t softmax(l)_t·v_t,h,  lse = log Σ exp(l_t).
// A warp a row: a lane has four dims of k and v and two rotated ones.
#include "kvd_common.cuh"
#include "kvd_latent.h"

namespace kvd {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack4(float* x, const uint16_t* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack_bf16(v.x), c = unpack_bf16(v.y);
    x[0] = a.x;
    x[1] = a.y;
    x[2] = c.x;
    x[3] = c.y;
}

__global__ void __launch_bounds__(kThreads) prefill_kernel(const LatentPrefillParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int s0 = p.q_start[b], s1 = p.q_start[b + 1], k0 = p.kv_start[b], k1 = p.kv_start[b + 1];
    if (s0 < 0 || s1 < s0 || s1 > p.n_tokens || k0 < 0 || k1 < k0 || k1 > p.n_keys) {
        if (threadIdx.x == 0) report(p.err, KVD_ERR_OOB);
        return;
    }
    const int T = s1 - s0, N = k1 - k0;
    const int64_t rows = static_cast<int64_t>(T) * p.n_q, warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
        const int64_t row = static_cast<int64_t>(s0) * p.n_q + r;
        const int h = static_cast<int>(r % p.n_q), i = static_cast<int>(r / p.n_q);
        float q[6], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, sum = 0.f;
        unpack4(q, p.q + row * kExpKey + lane * 4);
        const float2 qr = unpack_bf16(*reinterpret_cast<const uint32_t*>(p.q + row * kExpKey + kNope + lane * 2));
        q[4] = qr.x;
        q[5] = qr.y;
        const int end = p.causal ? max(0, N - T + i + 1) : N;
        for (int64_t n = k0; n < k0 + end; ++n) {
            float k[4], v[4];
            unpack4(k, p.k_nope + n * p.k_stride + h * p.k_head + lane * 4);
            unpack4(v, p.v + n * p.v_stride + h * p.v_head + lane * 4);
            const float2 rot = unpack_bf16(*reinterpret_cast<const uint32_t*>(p.k_rope + n * p.rope_stride + lane * 2));
            float dot = fmaf(q[4], rot.x, q[5] * rot.y);
            #pragma unroll
            for (int j = 0; j < 4; ++j) dot = fmaf(q[j], k[j], dot);
            #pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
            const float l = dot * p.scale_log2, top = fmaxf(m, l);
            const float ref = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m - ref), w = exp2f(l - ref);
            m = top;
            sum = sum * f + w;
            #pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = fmaf(w, v[j], acc[j] * f);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = row * kExpVal + lane * 4 + j;
            if (p.out_f32) static_cast<float*>(p.out)[at] = acc[j] * inv;
            else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(acc[j] * inv);
        }
        if (lane == 0 && p.lse_out) p.lse_out[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
    }
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, int num_sms, cudaStream_t stream) {
    const int64_t most = (static_cast<int64_t>(p.n_tokens) * p.n_q + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t share = (16 * num_sms + p.B - 1) / p.B;
    const dim3 grid(static_cast<unsigned>(most < share ? most : share), static_cast<unsigned>(p.B));
    return launch_dependent(prefill_kernel, grid, dim3(kThreads), 0, -1, stream, p);
}

}  // namespace kvd
