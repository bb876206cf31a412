// attend_e4m3.cu -- the attention kernel for e4m3 caches, 16 and 32 query rows to a tile.
#include "attend.cuh"

namespace specv {

cudaError_t attend_e4m3(int n, const AttParams& p, cudaStream_t s) {
    switch (n) {
        case 16: return launch_dim<16, true>(p, s);
        case 32: return launch_dim<32, true>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace specv
