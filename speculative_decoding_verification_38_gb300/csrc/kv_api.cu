// kv_api.cu -- the extern "C" entry points of the paged key-value cache:
// argument validation and the launches.
#include <algorithm>

#include "internal.h"
#include "kv.h"
#include "spec_verify.h"

using namespace specv;

namespace {

static_assert(SPEC_E4M3 == kKvE4m3 && SPEC_BF16 == kKvBf16 && SPEC_F32 == kKvF32, "dtype codes");
static_assert(SPEC_KV_MAX_QUERIES == kKvMaxQueries, "query limit");
static_assert(SPEC_ROPE_MAX_AXES == kRopeMaxAxes && kRopeMaxAxes == 4, "two bits for a pair's axis");
static_assert(SPEC_SEQ_BAD_KV == kKvBadKv && SPEC_SEQ_BAD_LAYOUT == kKvBadLayout && SPEC_SEQ_TIMEOUT == kKvTimeout,
              "status codes");

constexpr int64_t kMaxPositions = (int64_t)1 << 30;  // positions are 32-bit in the kernels
constexpr int64_t kMaxEntries = ((int64_t)1 << 31) - 65536;  // (row, head) of one launch: 32-bit in the kernels
constexpr int32_t kMaxBlockSize = 65536;
constexpr int32_t kMaxHeads = 65535;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

spec_status_t check_cache(const spec_kv_cache_t* c, bool scales) {
    if (!c || c->struct_size != sizeof(spec_kv_cache_t)) return SPEC_ERR_INVALID_ARG;
    if (c->batch < 1 || c->batch > kMaxBatch) return SPEC_ERR_INVALID_ARG;
    if (c->kv_heads < 1 || c->head_dim < 1 || c->block_size < 1 || c->num_blocks < 1 || c->max_blocks < 1 ||
        c->layers < 1)
        return SPEC_ERR_INVALID_ARG;
    if (c->dtype != SPEC_BF16 && c->dtype != SPEC_E4M3) return SPEC_ERR_INVALID_ARG;
    if (!c->k || !c->v || !c->block_table) return SPEC_ERR_INVALID_ARG;
    if (c->layer_stride < 0 || c->block_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
        return SPEC_ERR_INVALID_ARG;
    if (c->kv_heads > kMaxHeads || c->head_dim > kKvMaxDim || c->block_size > kMaxBlockSize ||
        (int64_t)c->max_blocks * c->block_size > kMaxPositions)
        return SPEC_ERR_UNSUPPORTED;
    if (scales && c->dtype == SPEC_E4M3 && (!c->k_scale || !c->v_scale)) return SPEC_ERR_INVALID_ARG;
    const int64_t per16 = c->dtype == SPEC_BF16 ? 8 : 16;  // elements of 16 bytes
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->block_table, 4)) return SPEC_ERR_ALIGNMENT;
    if (c->dtype == SPEC_E4M3 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))) return SPEC_ERR_ALIGNMENT;
    for (int64_t x : {(int64_t)c->head_dim, c->layer_stride, c->block_stride, c->token_stride, c->head_stride})
        if (x % per16) return SPEC_ERR_ALIGNMENT;
    return SPEC_OK;
}

// layer < 0: the whole cache.
KvView view(const spec_kv_cache_t* c, int32_t layer) {
    KvView v;
    const int64_t esz = c->dtype == SPEC_BF16 ? 2 : 1;
    const int64_t l = layer < 0 ? 0 : layer;
    const bool q8 = c->dtype == SPEC_E4M3;
    v.scale_layer = (int64_t)c->num_blocks * c->kv_heads * c->block_size;
    v.k = (unsigned char*)c->k + l * c->layer_stride * esz;
    v.v = (unsigned char*)c->v + l * c->layer_stride * esz;
    v.ks = q8 ? c->k_scale + l * v.scale_layer : nullptr;
    v.vs = q8 ? c->v_scale + l * v.scale_layer : nullptr;
    v.table = c->block_table;
    v.block_bytes = c->block_stride * esz;
    v.token_bytes = c->token_stride * esz;
    v.head_bytes = c->head_stride * esz;
    v.layer_bytes = c->layer_stride * esz;
    v.B = c->batch;
    v.H = c->kv_heads;
    v.D = c->head_dim;
    v.bs = c->block_size;
    v.by_bs = KvDiv((uint32_t)c->block_size);
    v.by_H = KvDiv((uint32_t)c->kv_heads);
    v.num_blocks = c->num_blocks;
    v.max_blocks = c->max_blocks;
    v.layers = c->layers;
    v.esz = (int32_t)esz;
    return v;
}

spec_status_t launched(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

// Host fields of an attention call (no pointers).
spec_status_t check_attend_shape(const spec_kv_cache_t* c, const spec_kv_attend_args_t* a) {
    if (!c || c->struct_size != sizeof(spec_kv_cache_t)) return SPEC_ERR_INVALID_ARG;
    if (!a || a->struct_size != sizeof(spec_kv_attend_args_t)) return SPEC_ERR_INVALID_ARG;
    if (c->batch < 1 || c->batch > kMaxBatch || c->kv_heads < 1 || c->head_dim < 1) return SPEC_ERR_INVALID_ARG;
    if (c->dtype != SPEC_BF16 && c->dtype != SPEC_E4M3) return SPEC_ERR_INVALID_ARG;
    if (a->q_heads < 1 || a->q_heads % c->kv_heads || a->t_max < 1) return SPEC_ERR_INVALID_ARG;
    if (a->t_max > SPEC_KV_MAX_QUERIES || c->kv_heads > kMaxHeads || a->q_heads > kMaxHeads ||
        c->head_dim > kKvMaxDim)
        return SPEC_ERR_UNSUPPORTED;
    if (a->rows < 0 || a->rows > (int64_t)c->batch * a->t_max) return SPEC_ERR_INVALID_ARG;
    return SPEC_OK;
}

// The new rows of an append.
spec_status_t new_rows(KvNew& n, const spec_kv_cache_t* c, int32_t layer, const void* k_new, const void* v_new, int32_t new_dtype,
                       int64_t new_token_stride, int64_t rows, const int64_t* row_off, int32_t t_max, const int32_t* kv_lens,
                       int32_t* seq_status) {
    if (layer < 0 || layer >= c->layers || rows < 0 || !kv_lens) return SPEC_ERR_INVALID_ARG;
    if (rows > 0 && (!k_new || !v_new)) return SPEC_ERR_INVALID_ARG;
    if (new_dtype != SPEC_BF16 && new_dtype != SPEC_F32) return SPEC_ERR_INVALID_ARG;
    if (!row_off && (t_max < 1 || rows != (int64_t)c->batch * t_max)) return SPEC_ERR_INVALID_ARG;
    if (new_token_stride < 0) return SPEC_ERR_INVALID_ARG;
    const int64_t esz = new_dtype == SPEC_BF16 ? 2 : 4;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || new_token_stride * esz % 16 || (int64_t)c->head_dim * esz % 16)
        return SPEC_ERR_ALIGNMENT;
    if ((row_off && !aligned(row_off, 8)) || !aligned(kv_lens, 4) || (seq_status && !aligned(seq_status, 4)))
        return SPEC_ERR_ALIGNMENT;
    if (rows > kMaxEntries / c->kv_heads) return SPEC_ERR_UNSUPPORTED;
    n.k = (const unsigned char*)k_new;
    n.v = (const unsigned char*)v_new;
    n.dtype = new_dtype;
    n.row_bytes = new_token_stride * esz;
    n.rows = rows;
    n.row_off = row_off;
    n.t_max = t_max;
    n.kv_lens = kv_lens;
    n.seq_status = seq_status;
    return SPEC_OK;
}

spec_status_t check_rope(const spec_rope_t* r, int32_t head_dim) {
    if (!r || r->struct_size != sizeof(spec_rope_t) || !r->inv_freq) return SPEC_ERR_INVALID_ARG;
    if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > head_dim) return SPEC_ERR_INVALID_ARG;
    if ((r->adjacent & ~1) || (r->alternating & ~1) || !(r->factor > -3.0e38f && r->factor < 3.0e38f)) return SPEC_ERR_INVALID_ARG;
    if (r->axes < 1 || r->axes > SPEC_ROPE_MAX_AXES) return SPEC_ERR_INVALID_ARG;
    if (r->axes > 1) {
        const int32_t half = r->rotary_dim / 2;
        int64_t all = 0;
        for (int a = 0; a < r->axes; ++a) {
            if (r->sections[a] < 0) return SPEC_ERR_INVALID_ARG;
            if (r->alternating && a > 0 && (int64_t)r->axes * r->sections[a] > half) return SPEC_ERR_INVALID_ARG;
            all += r->sections[a];
        }
        if (all != half) return SPEC_ERR_INVALID_ARG;
    }
    if (!aligned(r->inv_freq, 4)) return SPEC_ERR_ALIGNMENT;
    return SPEC_OK;
}

Rope rope_of(const spec_rope_t* r, const int32_t* positions, int64_t rows, int32_t heads) {
    Rope p = {};
    p.inv_freq = r->inv_freq;
    p.positions = positions;
    p.rows = rows;
    p.rd = r->rotary_dim;
    p.half = r->rotary_dim / 2;
    p.adjacent = r->adjacent;
    p.one_axis = r->axes == 1 || !positions;
    p.factor = r->factor;
    p.by_heads = KvDiv((uint32_t)(heads > 0 ? heads : 1));
    int32_t block = 0, left = r->axes > 1 ? r->sections[0] : p.half;
    for (int32_t i = 0; i < p.half && r->axes > 1; ++i) {
        int32_t a = i % r->axes;
        if (r->alternating) {
            if (i >= r->axes * r->sections[a]) a = 0;
        } else {
            while (left == 0) left = r->sections[++block];
            --left;
            a = block;
        }
        p.axis[i >> 4] |= (uint32_t)a << 2 * (i & 15);
    }
    return p;
}

spec_status_t rope_rows(RopeRows& q, const void* x, int32_t x_dtype, int64_t x_stride, void* out, int32_t out_dtype,
                        int64_t out_stride, int64_t rows, int32_t heads, int32_t head_dim) {
    for (int32_t t : {x_dtype, out_dtype})
        if (t != SPEC_BF16 && t != SPEC_F32) return SPEC_ERR_INVALID_ARG;
    if (x_stride < 0 || out_stride < 0) return SPEC_ERR_INVALID_ARG;
    if (x == out && x && (x_dtype != out_dtype || x_stride != out_stride)) return SPEC_ERR_INVALID_ARG;
    const int64_t xsz = x_dtype == SPEC_BF16 ? 2 : 4, osz = out_dtype == SPEC_BF16 ? 2 : 4;
    if (!aligned(x, 16) || !aligned(out, 16) || x_stride * xsz % 16 || out_stride * osz % 16 || head_dim * xsz % 16 ||
        head_dim * osz % 16)
        return SPEC_ERR_ALIGNMENT;
    if (head_dim % 8) return SPEC_ERR_ALIGNMENT;
    if (rows > 1 && out_stride < (int64_t)heads * head_dim) return SPEC_ERR_INVALID_ARG;  // rows of out would overlap
    q.x = (const unsigned char*)x;
    q.out = (unsigned char*)out;
    q.x_row_bytes = x_stride * xsz;
    q.out_row_bytes = out_stride * osz;
    q.heads = heads;
    q.D = head_dim;
    q.dtype = x_dtype;
    q.out_dtype = out_dtype;
    return SPEC_OK;
}

// Bytes that a call works on, with a window (of any length: either kernel) or without.
size_t workspace_of(const spec_kv_cache_t* c, const spec_kv_attend_args_t* a, bool window) {
    const int64_t rows = (int64_t)a->t_max * (a->q_heads / c->kv_heads);
    if (!attend_takes(c->head_dim)) return kHeaderBytes;
    return std::max(attend_workspace(rows, window), window ? attend_few_workspace(rows) : 0);
}

// window 0: none.
spec_status_t attend(const spec_kv_cache_t* c, const spec_kv_attend_args_t* a, int32_t window, int32_t sinks,
                     spec_stream_t stream) {
    spec_status_t st = check_attend_shape(c, a);
    if (st) return st;
    st = check_cache(c, true);
    if (st) return st;
    if (a->layer < 0 || a->layer >= c->layers || !a->kv_lens) return SPEC_ERR_INVALID_ARG;
    if (!a->row_off && a->rows != (int64_t)c->batch * a->t_max) return SPEC_ERR_INVALID_ARG;
    if (a->rows > 0 && (!a->q || !a->out)) return SPEC_ERR_INVALID_ARG;
    if (!(a->scale > 0.f && a->scale < 3.0e38f) || a->q_token_stride < 0) return SPEC_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || a->q_token_stride % 8 || c->head_dim % 8 || !aligned(a->out, 16))
        return SPEC_ERR_ALIGNMENT;
    if ((a->row_off && !aligned(a->row_off, 8)) || !aligned(a->kv_lens, 4) || !aligned(a->parent, 4) ||
        !aligned(a->lse, 4) || !aligned(a->seq_status, 4))
        return SPEC_ERR_ALIGNMENT;
    if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < workspace_of(c, a, window > 0)) return SPEC_ERR_WORKSPACE;
    KvAttend p;
    p.c = view(c, a->layer);
    p.Hq = a->q_heads;
    p.G = a->q_heads / c->kv_heads;
    p.by_G = KvDiv((uint32_t)p.G);
    p.t_max = a->t_max;
    p.rows = a->rows;
    p.row_off = a->row_off;
    p.kv_lens = a->kv_lens;
    p.parent = a->parent;
    p.q = (const unsigned char*)a->q;
    p.q_row_bytes = a->q_token_stride * 2;
    p.scale = a->scale;
    p.out = (unsigned char*)a->out;
    p.lse = a->lse;
    p.seq_status = a->seq_status;
    p.window = (int32_t)std::min<int64_t>(window, kMaxPositions);  // (so that sums with positions stay in range)
    p.sinks = (int32_t)std::min<int64_t>(sinks, kMaxPositions);
    if (window && attend_few_takes(p)) {
        if ((int64_t)c->batch * c->kv_heads > kMaxEntries) return SPEC_ERR_UNSUPPORTED;  // a CTA for each
        return launched(launch_attend_few(p, a->workspace, (cudaStream_t)stream));
    }
    return launched(attend_takes(c->head_dim) ? launch_attend(p, a->workspace, (cudaStream_t)stream)
                                              : launch_kv_attend_plain(p, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

SPEC_API spec_status_t spec_kv_append(const spec_kv_cache_t* c, int32_t layer, const void* k_new, const void* v_new,
                                      int32_t new_dtype, int64_t new_token_stride, int64_t rows,
                                      const int64_t* row_off, int32_t t_max, const int32_t* kv_lens,
                                      int32_t* seq_status, spec_stream_t stream) {
    spec_status_t st = check_cache(c, true);
    if (st) return st;
    KvNew n;
    st = new_rows(n, c, layer, k_new, v_new, new_dtype, new_token_stride, rows, row_off, t_max, kv_lens, seq_status);
    if (st) return st;
    return launched(launch_kv_append(view(c, layer), n, (cudaStream_t)stream));
}

SPEC_API spec_status_t spec_kv_gather(const spec_kv_cache_t* c, int32_t layer, const int32_t* kv_lens,
                                      const int64_t* out_off, int64_t rows, void* k_out, void* v_out,
                                      int32_t out_dtype, int32_t* seq_status, spec_stream_t stream) {
    spec_status_t st = check_cache(c, true);
    if (st) return st;
    if (layer < 0 || layer >= c->layers || rows < 0 || !kv_lens || !out_off) return SPEC_ERR_INVALID_ARG;
    if (rows > 0 && (!k_out || !v_out)) return SPEC_ERR_INVALID_ARG;
    if (out_dtype != SPEC_BF16 && out_dtype != SPEC_F32) return SPEC_ERR_INVALID_ARG;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(out_off, 8) || !aligned(kv_lens, 4) ||
        (seq_status && !aligned(seq_status, 4)))
        return SPEC_ERR_ALIGNMENT;
    if (rows > kMaxEntries / c->kv_heads) return SPEC_ERR_UNSUPPORTED;
    KvRead g;
    g.k = (unsigned char*)k_out;
    g.v = (unsigned char*)v_out;
    g.dtype = out_dtype;
    g.rows = rows;
    g.out_off = out_off;
    g.kv_lens = kv_lens;
    g.seq_status = seq_status;
    return launched(launch_kv_gather(view(c, layer), g, (cudaStream_t)stream));
}

SPEC_API spec_status_t spec_kv_compact(const spec_kv_cache_t* c, const int64_t* node_off, int64_t nodes,
                                       const int32_t* path, const int32_t* accepted, const int32_t* kv_lens_in,
                                       int32_t* kv_lens_out, int32_t* out_num_blocks, int32_t* seq_status,
                                       spec_stream_t stream) {
    spec_status_t st = check_cache(c, true);
    if (st) return st;
    if (!node_off || !path || !accepted || !kv_lens_in || !kv_lens_out) return SPEC_ERR_INVALID_ARG;
    if (nodes < c->batch || nodes > INT32_MAX) return SPEC_ERR_INVALID_ARG;
    if (!aligned(node_off, 8)) return SPEC_ERR_ALIGNMENT;
    for (const void* p : {(const void*)path, (const void*)accepted, (const void*)kv_lens_in, (const void*)kv_lens_out,
                          (const void*)out_num_blocks, (const void*)seq_status})
        if (!aligned(p, 4)) return SPEC_ERR_ALIGNMENT;
    const bool q8 = c->dtype == SPEC_E4M3;
    if (kv_compact_ctas(c->layers, c->kv_heads, c->head_dim * (q8 ? 1 : 2), q8) > kKvCompactMaxCtas)
        return SPEC_ERR_UNSUPPORTED;
    KvMove m;
    m.node_off = node_off;
    m.nodes = nodes;
    m.path = path;
    m.accepted = accepted;
    m.kv_in = kv_lens_in;
    m.kv_out = kv_lens_out;
    m.out_blocks = out_num_blocks;
    m.seq_status = seq_status;
    return launched(launch_kv_compact(view(c, -1), m, (cudaStream_t)stream));
}

SPEC_API size_t spec_kv_attend_workspace_size(const spec_kv_cache_t* c, const spec_kv_attend_args_t* a) {
    if (check_attend_shape(c, a) != SPEC_OK) return 0;
    return std::max(workspace_of(c, a, false), workspace_of(c, a, true));  // (one size, whether the call has a window or not)
}

SPEC_API spec_status_t spec_kv_attend(const spec_kv_cache_t* c, const spec_kv_attend_args_t* a, spec_stream_t stream) {
    return attend(c, a, 0, 0, stream);
}

SPEC_API spec_status_t spec_kv_attend_window(const spec_kv_cache_t* c, const spec_kv_attend_args_t* a, int32_t window,
                                             int32_t sinks, spec_stream_t stream) {
    if (window < 1 || sinks < 0) return SPEC_ERR_INVALID_ARG;
    return attend(c, a, window, sinks, stream);
}

SPEC_API spec_status_t spec_rope(const spec_rope_t* rope, const void* x, int32_t x_dtype, int64_t x_token_stride, void* out,
                                 int32_t out_dtype, int64_t out_token_stride, int64_t rows, int32_t heads, int32_t head_dim,
                                 const int32_t* positions, spec_stream_t stream) {
    if (heads < 1 || head_dim < 1 || rows < 0) return SPEC_ERR_INVALID_ARG;
    if (heads > kMaxHeads || head_dim > kKvMaxDim) return SPEC_ERR_UNSUPPORTED;
    spec_status_t st = check_rope(rope, head_dim);
    if (st) return st;
    if (rows > 0 && (!x || !out || !positions)) return SPEC_ERR_INVALID_ARG;
    if (!aligned(positions, 4)) return SPEC_ERR_ALIGNMENT;
    if (rows > kMaxEntries / heads) return SPEC_ERR_UNSUPPORTED;
    RopeRows q;
    st = rope_rows(q, x, x_dtype, x_token_stride, out, out_dtype, out_token_stride, rows, heads, head_dim);
    if (st) return st;
    return launched(launch_rope(rope_of(rope, positions, rows, heads), q, rows, (cudaStream_t)stream));
}

SPEC_API spec_status_t spec_kv_append_rope(const spec_kv_cache_t* c, const spec_rope_t* rope,
                                           const spec_kv_append_rope_args_t* a, spec_stream_t stream) {
    spec_status_t st = check_cache(c, true);
    if (st) return st;
    if (!a || a->struct_size != sizeof(spec_kv_append_rope_args_t)) return SPEC_ERR_INVALID_ARG;
    st = check_rope(rope, c->head_dim);
    if (st) return st;
    KvNew n;
    st = new_rows(n, c, a->layer, a->k_new, a->v_new, a->new_dtype, a->new_token_stride, a->rows, a->row_off, a->t_max, a->kv_lens,
                  a->seq_status);
    if (st) return st;
    if (a->parent && a->positions) return SPEC_ERR_INVALID_ARG;
    if (!aligned(a->parent, 4) || !aligned(a->positions, 4)) return SPEC_ERR_ALIGNMENT;
    if (a->q_heads < 0 || (a->q_heads > 0 && a->rows > 0 && (!a->q || !a->q_out))) return SPEC_ERR_INVALID_ARG;
    if (a->q_heads > kMaxHeads) return SPEC_ERR_UNSUPPORTED;
    if (a->q_heads > 0 && a->rows > kMaxEntries / a->q_heads) return SPEC_ERR_UNSUPPORTED;
    RopeRows q = {};
    if (a->q_heads > 0) {
        st = rope_rows(q, a->q, a->new_dtype, a->q_token_stride, a->q_out, SPEC_BF16, a->q_out_token_stride, a->rows, a->q_heads,
                       c->head_dim);
        if (st) return st;
    }
    if (a->rows == 0) n.k = (const unsigned char*)c->k;  // (not read: null would mean rows without a cache)
    return launched(launch_kv_append_rope(view(c, a->layer), n, rope_of(rope, a->positions, a->rows, a->q_heads), q, a->parent,
                                          (cudaStream_t)stream));
}

}  // extern "C"
