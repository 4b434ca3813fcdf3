// kvd_chunk.cu — causal attention of a chunk of new tokens over the paged cache.
//
// Row (token i of the T new tokens of request b, query head h): with len = seq_lens[b] and
// position P = len − T + i,
//   l_t = softmax_scale · q·K_t for t ≤ P (−inf where slot t is evicted),
//   out = Σ_t softmax(l)_t · V_t,  lse = log Σ_t exp(l_t).
//
// One warp per (new token, query head): lane l holds dims 4l .. 4l+3 of q and of the sum; one pass
// over the positions with a running maximum and sum in fp32.
#include "kvd_chunk.h"
#include "kvd_common.cuh"

namespace kvd {
namespace {

struct Row4 {
    float k[4], v[4];
};

// Dims 4·lane .. 4·lane+3 of the token at offset t of a record, as attention reads them.
template <int KIND, int NG>
__device__ __forceinline__ Row4 read_row(const uint8_t* rec, int fmt, int t, int lane) {
    Row4 r;
    if constexpr (is_lowbit(KIND)) {
        constexpr int kBits = KIND == kKindInt4 ? 4 : 2;
        constexpr int kTile = lowbit_tile_bytes(kBits);
        const uint32_t* meta = reinterpret_cast<const uint32_t*>(rec + 2 * kTile);
        const int gi = lane / (32 / NG);
        const float2 ks = unpack_f16(meta[t * NG + gi]), vs = unpack_f16(meta[kBs * NG + t * NG + gi]);
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = 4 * lane + j, sh = kBits * ((d / 16) % (8 / kBits));
            r.k[j] = static_cast<float>((rec[lowbit_k_byte(kBits, t, d)] >> sh) & ((1 << kBits) - 1)) * ks.x + ks.y;
            r.v[j] = static_cast<float>((rec[kTile + lowbit_v_byte(kBits, t, d)] >> sh) & ((1 << kBits) - 1)) * vs.x + vs.y;
        }
        return r;
    }
    const bool wide = fmt == kFmtBf16;
    float ks = 1.f, vs = 1.f;
    if (!wide) {
        const float* sc = reinterpret_cast<const float*>(rec + 2 * kTileFp8);
        ks = sc[t];
        vs = sc[kBs + t];
    }
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
        int fl, fe;
        const int d = 4 * lane + j;
        const int ki = k_frag_i(t, d, &fl, &fe), kl = fl, ke = fe;
        const int vi = v_frag_i(t, d, &fl, &fe);
        if (wide) {
            const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(rec);
            r.k[j] = __bfloat162float(e[bf16_tile_index(ki, kl, ke)]);
            r.v[j] = __bfloat162float(e[kBs * kDh + bf16_tile_index(vi, fl, fe)]);
        } else {
            const __nv_fp8_interpretation_t in = fmt == kFmtE5m2 ? __NV_E5M2 : __NV_E4M3;
            r.k[j] = ks * __half2float(__half(__nv_cvt_fp8_to_halfraw(rec[fp8_tile_index(ki, kl, ke)], in)));
            r.v[j] = vs * __half2float(__half(__nv_cvt_fp8_to_halfraw(rec[kTileFp8 + fp8_tile_index(vi, fl, fe)], in)));
        }
    }
    return r;
}

__device__ __forceinline__ float warp_sum(float x) {
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

template <int KIND, int NG>
__global__ void __launch_bounds__(256) chunk_kernel(const ChunkParams p) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int row = static_cast<int>(w / p.n_q), hq = static_cast<int>(w % p.n_q);
    if (row >= p.n_tokens) return;
    int b = -1, s0 = 0, s1 = 0;
    for (int b0 = 0; b0 < p.B && b < 0; b0 += 32) {
        const int c = b0 + lane;
        int lo = 0, hi = -1;
        if (c < p.B) {
            lo = p.q_start[c];
            hi = p.q_start[c + 1];
            if (lo < 0 || hi < lo || hi > p.n_tokens) {
                report(p.err, KVD_ERR_OOB);
                hi = lo;
            }
        }
        const unsigned m = __ballot_sync(kFull, row >= lo && row < hi);
        if (m) {
            const int l = __ffs(m) - 1;
            b = b0 + l;
            s0 = __shfl_sync(kFull, lo, l);
            s1 = __shfl_sync(kFull, hi, l);
        }
    }
    if (b < 0) return;
    const int T = s1 - s0;
    int len = p.seq_lens[b];
    if (len < T || static_cast<int64_t>(len) > static_cast<int64_t>(p.max_blocks) * kBs) {
        report(p.err, KVD_ERR_OOB);
        len = 0;
    }
    const int last = len ? len - T + (row - s0) : -1;
    const int h = hq / p.g;
    const int64_t at = (static_cast<int64_t>(row) * p.n_q + hq) * kDh + lane * 4;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = __bfloat162float(__ushort_as_bfloat16(p.q[at + j]));
    float qf = 1.f;
    if constexpr (KIND == kKindAngle) {   // the head's direction code and ||q|| / ||d_q||
        float mx = 0.f;
        #pragma unroll
        for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fabsf(q[j]));
        #pragma unroll
        for (int of = 16; of > 0; of >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, of));
        const float s = mx == 0.f ? 1.f : __fdiv_rn(mx, 448.f);
        float r2 = 0.f, d2 = 0.f;
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float c = __half2float(__half(__nv_cvt_fp8_to_halfraw(
                __nv_cvt_float_to_fp8(__fdiv_rn(q[j], s), __NV_SATFINITE, __NV_E4M3), __NV_E4M3)));
            r2 += q[j] * q[j];
            d2 += c * c;
            q[j] = c;
        }
        r2 = warp_sum(r2);
        d2 = warp_sum(d2);
        qf = d2 > 0.f ? sqrtf(r2 / d2) : 0.f;
    }
    const int64_t kRec = p.record_bytes;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j * kBs <= last; ++j) {
        const int ph = p.block_table[static_cast<int64_t>(b) * p.max_blocks + j];
        if (ph < 0 || ph >= p.num_blocks + p.host_blocks) {
            report(p.err, KVD_ERR_OOB);
            continue;
        }
        const uint32_t keep = p.retain ? p.retain[ph] : 0xffffu;
        int fmt = KIND == kKindBf16 ? kFmtBf16 : kFmtE4m3;
        if constexpr (KIND == kKindMixed) {
            fmt = block_format(p.block_fmt[ph]);
            if (fmt < 0) {
                report(p.err, KVD_ERR_OOB);
                continue;
            }
        }
        const uint8_t* rec = ph < p.num_blocks ? p.kv + (static_cast<int64_t>(ph) * p.n_kv + h) * kRec
                                               : p.stage + ((ph - p.num_blocks) * p.n_kv + h) * kRec;
        for (int t = 0; t < kBs && j * kBs + t <= last; ++t) {
            if (!((keep >> t) & 1u)) continue;
            const Row4 r = read_row<KIND, NG>(rec, fmt, t, lane);
            const float s =
                warp_sum(q[0] * r.k[0] + q[1] * r.k[1] + q[2] * r.k[2] + q[3] * r.k[3]) * qf * p.scale_log2;
            const float mn = fmaxf(m, s);
            const float a = m == -INFINITY ? 0.f : exp2f(m - mn), e = s == -INFINITY ? 0.f : exp2f(s - mn);
            l = l * a + e;
            #pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = o[k] * a + e * r.v[k];
            m = mn;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (p.out_f32) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) static_cast<float*>(p.out)[at + j] = o[j] * inv;
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    }
    if (p.lse_out && lane == 0)
        p.lse_out[static_cast<int64_t>(row) * p.n_q + hq] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace

cudaError_t launch_chunk(const ChunkParams& p, int kind, cudaStream_t stream) {
    const int64_t warps = static_cast<int64_t>(p.n_tokens) * p.n_q;
    const dim3 grid(static_cast<unsigned>((warps + 7) / 8)), block(256);
    switch (kind) {
        case kKindFp8: return launch_dependent(chunk_kernel<kKindFp8, 1>, grid, block, 0, -1, stream, p);
        case kKindMixed: return launch_dependent(chunk_kernel<kKindMixed, 1>, grid, block, 0, -1, stream, p);
        case kKindAngle: return launch_dependent(chunk_kernel<kKindAngle, 1>, grid, block, 0, -1, stream, p);
        case kKindInt4:
            return p.ng == 4   ? launch_dependent(chunk_kernel<kKindInt4, 4>, grid, block, 0, -1, stream, p)
                   : p.ng == 2 ? launch_dependent(chunk_kernel<kKindInt4, 2>, grid, block, 0, -1, stream, p)
                               : launch_dependent(chunk_kernel<kKindInt4, 1>, grid, block, 0, -1, stream, p);
        case kKindInt2:
            return p.ng == 4   ? launch_dependent(chunk_kernel<kKindInt2, 4>, grid, block, 0, -1, stream, p)
                   : p.ng == 2 ? launch_dependent(chunk_kernel<kKindInt2, 2>, grid, block, 0, -1, stream, p)
                               : launch_dependent(chunk_kernel<kKindInt2, 1>, grid, block, 0, -1, stream, p);
        default: return launch_dependent(chunk_kernel<kKindBf16, 1>, grid, block, 0, -1, stream, p);
    }
}

}  // namespace kvd
