// attend_e4m3_wide.cu -- the attention kernel for e4m3 caches, 48 to 128 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_e4m3_wide(int n, const AttParams& p, cudaStream_t s) {
    switch (n) {
        case 48: return launch_dim<48, true>(p, s);
        case 80: return launch_dim<80, true>(p, s);
        case 128: return launch_dim<128, true>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
