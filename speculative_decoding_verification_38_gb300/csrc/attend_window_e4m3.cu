// attend_window_e4m3.cu -- the attention kernel with a sliding window for e4m3 caches, 16 to 128 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_window_e4m3(int n, const AttParams& p, cudaStream_t s) {
    switch (n) {
        case 16: return launch_dim<16, true, true>(p, s);
        case 48: return launch_dim<48, true, true>(p, s);
        case 80: return launch_dim<80, true, true>(p, s);
        case 128: return launch_dim<128, true, true>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
