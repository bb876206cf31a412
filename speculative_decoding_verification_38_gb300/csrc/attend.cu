// attend.cu -- the host side of the attention on the tensor cores: which row
// tile a call takes, its workspace, its grid.
#include <algorithm>
#include <atomic>

#include "attend.cuh"

namespace specv {

namespace {

// Rows of a row tile: the fewest that hold the rows in as few row tiles as
// 128 rows would.
int tile_rows(int64_t rows) {
    const int64_t tiles = (rows + 127) / 128, each = (rows + tiles - 1) / tiles;
    for (int n : {16, 32, 48, 80})
        if (each <= n) return n;
    return 128;
}

constexpr size_t kPartAlign = 256;

}  // namespace

bool attend_takes(int32_t head_dim) { return head_dim <= 128; }

size_t attend_workspace(int64_t rows) {
    const size_t n = (size_t)kAttMaxGrid * 2 * tile_rows(rows);
    return kHeaderBytes + (n * 128 * 4 + n * 8 + kPartAlign - 1) / kPartAlign * kPartAlign;
}

cudaError_t launch_attend(const KvAttend& a, void* workspace, cudaStream_t s) {
    static std::atomic<int> sms[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int grid = dev < 64 ? sms[dev].load() : 0;
    if (!grid) {
        if ((e = cudaDeviceGetAttribute(&grid, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if (dev < 64) sms[dev].store(grid);
    }
    grid = std::min(grid, kAttMaxGrid);
    AttParams p;
    p.a = a;
    p.grid = grid;
    const int n = tile_rows((int64_t)a.t_max * a.G);
    char* ws = (char*)workspace;
    p.arrive = (uint32_t*)ws;
    p.err = (uint32_t*)(ws + kErrWordOffset);
    p.part_o = (float*)(ws + kHeaderBytes);
    p.part_ml = (float2*)(ws + kHeaderBytes + (size_t)grid * 2 * n * 128 * 4);
    if (a.c.esz == 1) return n < 48 ? attend_e4m3(n, p, s) : attend_e4m3_wide(n, p, s);
    return n < 48 ? attend_bf16(n, p, s) : attend_bf16_wide(n, p, s);
}

}  // namespace specv
