// kv.h -- parameter blocks and launch entry points of the paged key-value
// cache's kernels (kv.cu, attend.cu). Not installed.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace specv {

constexpr int kKvMaxQueries = 128;  // new tokens of one sequence in the attention
constexpr int kKvMaxDim = 256;

// Division of 0 <= n < 2^31 by a number the launch knows: with s = ceil(log2 d) and m = floor(2^(31+s) / d) + 1 the
// error n (m - 2^(31+s) / d) / 2^(31+s) stays below 1 / d, so n / d = n m >> (31 + s) exactly. A multiply and a shift
// where the device's own division is some twenty instructions at each of its many places.
struct KvDiv {
    uint32_t m;
    int32_t shift;
    KvDiv() = default;
    explicit KvDiv(uint32_t d) {
        int s = 0;
        while ((1ull << s) < d) ++s;
        m = (uint32_t)((1ull << (31 + s)) / d + (d > 1 ? 1 : 0));
        shift = 31 + s;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int32_t of(int32_t n) const { return (int32_t)(((uint64_t)(uint32_t)n * m) >> shift); }
#endif
};

enum KvType : int32_t { kKvF32 = 0, kKvBf16 = 1, kKvE4m3 = 2 };  // the API's dtype codes
enum KvSeqStatus : int32_t { kKvOk = 0, kKvBadKv = 2, kKvBadLayout = 4, kKvTimeout = 6 };

// One layer of a cache (k, v and the scales already point at the layer), or
// the whole of it for the compaction.
struct KvView {
    unsigned char* k;
    unsigned char* v;
    float* ks;  // [num_blocks, kv_heads, block_size], or null
    float* vs;
    const int32_t* table;  // [B, max_blocks]
    int64_t block_bytes, token_bytes, head_bytes, layer_bytes;
    int64_t scale_layer;  // scales of a layer
    int32_t B, H, D, bs, num_blocks, max_blocks, layers;
    KvDiv by_bs, by_H;
    int32_t esz;  // bytes of an element: 2 or 1
};

struct KvNew {
    const unsigned char* k;
    const unsigned char* v;
    int32_t dtype;
    int64_t row_bytes;
    int64_t rows;
    const int64_t* row_off;  // [B+1] or null: t_max rows each
    int32_t t_max;
    const int32_t* kv_lens;
    int32_t* seq_status;
};

struct KvRead {
    unsigned char* k;
    unsigned char* v;
    int32_t dtype;
    int64_t rows;
    const int64_t* out_off;
    const int32_t* kv_lens;
    int32_t* seq_status;
};

enum KvMovePart : int32_t { kMoveAll = 0, kMoveEntries = 1, kMoveLengths = 2 };  // what a compaction's launch does

struct KvMove {
    int32_t part;  // KvMovePart, set by launch_kv_compact
    const int64_t* node_off;
    int64_t nodes;
    const int32_t* path;
    const int32_t* accepted;
    const int32_t* kv_in;
    int32_t* kv_out;
    int32_t* out_blocks;
    int32_t* seq_status;
};

struct KvAttend {
    KvView c;
    int32_t Hq, G, t_max;  // G = Hq / H
    KvDiv by_G;
    int64_t rows;
    const int64_t* row_off;
    const int32_t* kv_lens;
    const int32_t* parent;
    const unsigned char* q;
    int64_t q_row_bytes;
    float scale;
    unsigned char* out;
    float* lse;
    int32_t* seq_status;
    int32_t window, sinks;  // of a sliding window; window 0: every position before a token's own
};

// Rotary positions (rope.cu).
constexpr int kRopeMaxAxes = 4;
struct Rope {
    const float* inv_freq;     // [half]
    const int32_t* positions;  // [axes, rows], or null: the cache's own
    int64_t rows;
    int32_t rd, half;          // elements that turn, pairs of them
    int32_t adjacent, one_axis;
    float factor;
    KvDiv by_heads;            // of the queries
    uint32_t axis[kKvMaxDim / 2 / 16];  // two bits for each pair
    __host__ __device__ int32_t axis_of(int32_t pair) const { return axis[pair >> 4] >> 2 * (pair & 15) & 3; }
};

// Rows of queries beside the cache's, or alone.
struct RopeRows {
    const unsigned char* x;
    unsigned char* out;
    int64_t x_row_bytes, out_row_bytes;
    int32_t heads, D;
    int32_t dtype, out_dtype;
};

// CTAs that a compaction gives each sequence: a thread for each 16-byte column, and each scale, of a token in all layers.
constexpr int kKvThreads = 256;
inline int64_t kv_compact_ctas(int64_t layers, int64_t kv_heads, int64_t entry_bytes, bool scales) {
    return (layers * kv_heads * 2 * (entry_bytes / 16 + (scales ? 1 : 0)) + kKvThreads - 1) / kKvThreads;
}
constexpr int64_t kKvCompactMaxCtas = 65535;  // a grid's second axis
cudaError_t launch_kv_append(const KvView& c, const KvNew& n, cudaStream_t s);
cudaError_t launch_kv_gather(const KvView& c, const KvRead& r, cudaStream_t s);
cudaError_t launch_kv_compact(const KvView& c, const KvMove& m, cudaStream_t s);
// New tokens into the cache with their keys rotated, and q's rows (heads 0: none). parent: trees, or null.
cudaError_t launch_kv_append_rope(const KvView& c, const KvNew& n, const Rope& r, const RopeRows& q, const int32_t* parent,
                                  cudaStream_t s);
cudaError_t launch_rope(const Rope& r, const RopeRows& q, int64_t rows, cudaStream_t s);
// The attention on the tensor cores (attend.cu), for head_dim up to 128;
// rows = t_max * query heads of a key-value head sets the workspace.
bool attend_takes(int32_t head_dim);
size_t attend_workspace(int64_t rows, bool window);
cudaError_t launch_attend(const KvAttend& a, void* workspace, cudaStream_t s);
// Through a window, for rows up to 16 where no piece of an entry can be long (attend_few.cu).
bool attend_few_takes(const KvAttend& a);
size_t attend_few_workspace(int64_t rows);  // 0: more rows than it takes
cudaError_t launch_attend_few(const KvAttend& a, void* workspace, cudaStream_t s);
// A CTA for each query row, for the rest.
cudaError_t launch_kv_attend_plain(const KvAttend& p, cudaStream_t s);

}  // namespace specv
