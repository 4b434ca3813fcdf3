// kvd_chunk_lowbit.cu — chunk attention over INT4 / INT2 pools (kvd_chunk_kernel.cuh).
#include "kvd_chunk_kernel.cuh"

namespace kvd {

cudaError_t launch_chunk_lowbit(const ChunkParams& p, int kind, int ctas, cudaStream_t stream) {
    return kind == kKindInt4 ? chunk::launch_kind<kKindInt4>(p, ctas, stream) : chunk::launch_kind<kKindInt2>(p, ctas, stream);
}

}  // namespace kvd
