// Decode family of a batch whose groups of sequences share a prefix: the positions behind what is shared.  The parts are
// joined with those of the shared positions (dense_shared.cu).
#include "dense_decode.cuh"

namespace msa {

template <int H>
static cudaError_t launch_own(const DenseArgs& a, int grid, cudaStream_t stream) {
    if (a.kv_int8)
        return a.out_bf16 ? launch_dense_decode_kernel<H, true, 1, true>(a, grid, stream)
                          : launch_dense_decode_kernel<H, true, 2, true>(a, grid, stream);
    return a.out_bf16 ? launch_dense_decode_kernel<H, false, 2, true>(a, grid, stream)
                      : launch_dense_decode_kernel<H, false, 3, true>(a, grid, stream);
}

cudaError_t run_dense_decode_own(const DenseArgs& a, int grid, cudaStream_t stream) {
    switch (a.H) {
        case 1: return launch_own<1>(a, grid, stream);
        case 2: return launch_own<2>(a, grid, stream);
        case 4: return launch_own<4>(a, grid, stream);
        case 8: return launch_own<8>(a, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace msa
