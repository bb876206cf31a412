// attend.cu -- the host side of the attention on the tensor cores: which row
// tile a call takes, its workspace, its grid.
#include <algorithm>
#include <atomic>

#include "attend.cuh"

namespace specv {

namespace {

// Rows of a row tile: the fewest that hold the rows in as few row tiles as
// 128 rows would (each further tile reads the cache again), of five sizes that
// there are kernels for: a product's time grows with its columns from 64 on,
// and a softmax group's with its rows (36 rows of 64 sequences, bf16, in tiles
// of 48: 119 us; 116 in tiles of 128: 180). Sizes between them, 64 or 96, have
// not been measured.
int tile_rows(int64_t rows) {
    const int64_t tiles = (rows + 127) / 128, each = (rows + tiles - 1) / tiles;
    for (int n : {16, 32, 48, 80})
        if (each <= n) return n;
    return 128;
}

constexpr size_t kPartAlign = 256;

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's encoder, looked up once (the library does not link the driver).
EncodeTiled encoder() {
    static const EncodeTiled f = [] {
        void* at = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            at = nullptr;
        return (EncodeTiled)at;
    }();
    return f;
}

// One layer of K or V as (elements, slots, heads, pages), read in boxes of 128
// bytes of a row (past head_dim: zeros) by `box` slots.
cudaError_t box_map(CUtensorMap& m, const KvView& c, void* base, int32_t box) {
    const EncodeTiled f = encoder();
    if (!f) return cudaErrorNotSupported;
    const bool q8 = c.esz == 1;
    const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.bs, (cuuint64_t)c.H, (cuuint64_t)c.num_blocks};
    // an axis of one element is never stepped along, but its stride must pass the encoder
    auto stride = [&](int64_t bytes, cuuint64_t n) { return (cuuint64_t)(n > 1 ? bytes : 16); };
    const cuuint64_t strides[3] = {stride(c.token_bytes, dims[1]), stride(c.head_bytes, dims[2]),
                                   stride(c.block_bytes, dims[3])};
    const cuuint32_t boxes[4] = {q8 ? 128u : 64u, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
    // L2 fetches no further than the bytes that lie together: past an entry of 128 bytes lies another head's, and with
    // 256-byte fetches one e4m3 token of 64 sequences read 458 MB for its 310 (107 us; 105 without).
    const int64_t run = c.token_bytes == (int64_t)c.D * c.esz ? 256 : (int64_t)c.D * c.esz;
    const CUtensorMapL2promotion fetch = run >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : run >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                      : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    const CUresult r =
        f(&m, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, boxes, steps,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

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
    p.device = dev;
    p.box = 1;
    p.box_log = 0;
    while (p.box < kTileTok && a.c.bs % (2 * p.box) == 0) p.box *= 2, ++p.box_log;
    if ((e = box_map(p.k_map, a.c, a.c.k, p.box)) != cudaSuccess) return e;
    if ((e = box_map(p.v_map, a.c, a.c.v, p.box)) != cudaSuccess) return e;
    const int n = tile_rows((int64_t)a.t_max * a.G);
    char* ws = (char*)workspace;
    p.arrive = (uint32_t*)ws;
    p.err = (uint32_t*)(ws + kErrWordOffset);
    p.left = (uint32_t*)(ws + kLeftOffset);
    p.late = (int32_t*)(ws + kLateOffset);
    p.part_o = (float*)(ws + kHeaderBytes);
    p.part_ml = (float2*)(ws + kHeaderBytes + (size_t)grid * 2 * n * 128 * 4);
    if (a.c.esz == 1) return n < 48 ? attend_e4m3(n, p, s) : attend_e4m3_wide(n, p, s);
    return n < 48 ? attend_bf16(n, p, s) : attend_bf16_wide(n, p, s);
}

}  // namespace specv
