// attend_window_bf16.cu -- the attention kernel with a sliding window for bf16 caches, 32 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_window_bf16(int n, const AttParams& p, cudaStream_t s) {
    switch (n) {
        case 32: return launch_dim<32, false, true>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
