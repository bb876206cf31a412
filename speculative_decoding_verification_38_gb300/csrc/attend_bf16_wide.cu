// attend_bf16_wide.cu -- the attention kernel for bf16 caches, 48 to 128 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_bf16_wide(int nc, const AttParams& p, cudaStream_t s) {
    switch (nc) {
        case 24: return launch_dim<24, false>(p, s);
        case 40: return launch_dim<40, false>(p, s);
        case 64: return launch_dim<64, false>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
