// attend_window_bf16.cu -- the attention kernel with a sliding window for bf16 caches, 16 to 128 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_window_bf16(int n, const AttParams& p, cudaStream_t s) {
    switch (n) {
        case 16: return launch_dim<16, false, true>(p, s);
        case 48: return launch_dim<48, false, true>(p, s);
        case 80: return launch_dim<80, false, true>(p, s);
        case 128: return launch_dim<128, false, true>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
