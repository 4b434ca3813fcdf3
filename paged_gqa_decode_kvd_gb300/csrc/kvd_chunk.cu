// kvd_chunk.cu — chunk attention (kvd_chunk_kernel.cuh): the 16- and 8-bit pools, the join of cut units.
#include "kvd_chunk_kernel.cuh"

namespace kvd {
namespace chunk {

constexpr int kJoinThreads = 256, kJoinRows = 32;

// Joins the partials of a unit that range borders cut: out = Σ_k 2^(m_k − M)·o_k / Σ_k 2^(m_k − M)·l_k, in
// the order of the CTAs.  CTA (x, y): rows 32y .. of the unit whose first part is CTA x's last one; a
// lane is a row, a warp takes 16 dims.
__global__ void __launch_bounds__(kJoinThreads) chunk_combine_kernel(const ChunkParams p) {
    pdl_wait();
    pdl_trigger();
    int slot = 2 * blockIdx.x;
    int4 seg = p.part_seg[slot];
    if (seg.x < 0 || (seg.z & 1)) {   // not the first part of a unit
        seg = p.part_seg[++slot];
        if (seg.x < 0 || (seg.z & 1)) return;
    }
    const int tq = kUnitRows / p.g;
    const int b = seg.x, h = seg.z >> 1, qt = seg.y;
    const Request r = load_request(p, b, false);
    const int tiles = unit_tiles(r, qt, tq);
    const int rows = min(tq, r.T - qt * tq) * p.g;
    const int row = blockIdx.y * kJoinRows + (threadIdx.x & 31);
    if (blockIdx.y * kJoinRows >= rows) return;
    const int first = slot;
    const int d0 = (threadIdx.x >> 5) * 16;
    // the parts: slot `first`, then the first slot of each following CTA
    int parts = 1;
    for (int end = seg.w; end < tiles && blockIdx.x + parts < gridDim.x; ++parts) end = p.part_seg[2 * (blockIdx.x + parts)].w;
    auto slot_of = [&](int k) { return k == 0 ? first : 2 * static_cast<int>(blockIdx.x + k); };
    float M = -INFINITY;
    for (int k = 0; k < parts; ++k) M = fmaxf(M, p.part_ml[static_cast<int64_t>(slot_of(k)) * 2 * kUnitRows + row]);
    float L = 0.f, o[16];
    #pragma unroll
    for (int d = 0; d < 16; ++d) o[d] = 0.f;
    for (int k = 0; k < parts; ++k) {
        const int64_t s = slot_of(k);
        const float m = p.part_ml[s * 2 * kUnitRows + row], l = p.part_ml[s * 2 * kUnitRows + kUnitRows + row];
        if (m == -INFINITY && l == 0.f) continue;   // no position of the part is attended
        const float f = m == M ? 1.f : ex2(m - M);
        L += l * f;
        const float* part = p.part + (s * kDh + d0) * kUnitRows + row;
        #pragma unroll
        for (int d = 0; d < 16; ++d) o[d] += part[d * kUnitRows] * f;
    }
    if (row >= rows) return;
    const int64_t at = (static_cast<int64_t>(r.s0) + qt * tq + row / p.g) * p.n_q + h * p.g + row % p.g;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (p.out_f32) {
        float4* y = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * kDh + d0);
        #pragma unroll
        for (int d = 0; d < 16; d += 4) y[d / 4] = make_float4(o[d] * inv, o[d + 1] * inv, o[d + 2] * inv, o[d + 3] * inv);
    } else {
        uint4* y = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * kDh + d0);
        #pragma unroll
        for (int d = 0; d < 16; d += 8)
            y[d / 8] = make_uint4(pack_bf16(o[d] * inv, o[d + 1] * inv), pack_bf16(o[d + 2] * inv, o[d + 3] * inv),
                                  pack_bf16(o[d + 4] * inv, o[d + 5] * inv), pack_bf16(o[d + 6] * inv, o[d + 7] * inv));
    }
    if (p.lse_out && d0 == 0) p.lse_out[at] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
}

}  // namespace chunk

cudaError_t launch_chunk(const ChunkParams& p, int kind, int ctas, cudaStream_t stream) {
    cudaError_t e;
    switch (kind) {
        case kKindFp8: e = chunk::launch_kind<kKindFp8>(p, ctas, stream); break;
        case kKindMixed: e = chunk::launch_kind<kKindMixed>(p, ctas, stream); break;
        case kKindAngle: e = chunk::launch_kind<kKindAngle>(p, ctas, stream); break;
        case kKindInt4:
        case kKindInt2: e = launch_chunk_lowbit(p, kind, ctas, stream); break;
        default: e = chunk::launch_kind<kKindBf16>(p, ctas, stream); break;
    }
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(ctas), kChunkUnitRows / chunk::kJoinRows);
    return launch_dependent(chunk::chunk_combine_kernel, grid, dim3(chunk::kJoinThreads), 0, -1, stream, p);
}

}  // namespace kvd
