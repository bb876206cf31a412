// attend_e4m3_wide.cu -- the attention kernel for e4m3 caches, 48 to 128 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_e4m3_wide(int nc, const AttParams& p, cudaStream_t s) {
    switch (nc) {
        case 24: return launch_dim<24, true>(p, s);
        case 40: return launch_dim<40, true>(p, s);
        case 64: return launch_dim<64, true>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
