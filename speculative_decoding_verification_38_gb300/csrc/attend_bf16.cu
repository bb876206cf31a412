// attend_bf16.cu -- the attention kernel for bf16 caches, 16 and 32 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_bf16(int n, const AttParams& p, cudaStream_t s) {
    switch (n) {
        case 16: return launch_dim<16, false>(p, s);
        case 32: return launch_dim<32, false>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
