// kv.cu -- the paged key-value cache: writing new tokens (with quantisation),
// reading back, keeping a tree's accepted path, and the plain attention that
// takes the shapes attend.cu does not.
#include <algorithm>

#include "kv.cuh"

namespace specv {

namespace {

constexpr int kThreads = kKvThreads;

// Status of each sequence, one warp each: the offsets and length by `st`,
// then every page of positions [p0, L).
__device__ __forceinline__ int32_t check_pages(const KvView& c, int32_t b, int64_t p0, int64_t L) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    if (L > p0)
        for (int64_t j = p0 / c.bs + lane; j <= (L - 1) / c.bs; j += 32) {
            const int32_t pg = c.table[(int64_t)b * c.max_blocks + j];
            bad |= pg < 0 || pg >= c.num_blocks;
        }
    return __any_sync(0xFFFFFFFFu, bad) ? kKvBadLayout : kKvOk;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// The smallest power of two s >= 2^-126 with a / s <= 448 = 1.75 * 2^8, as
// exponents: s = 2^e (a finite and >= 0; a = 0 gives 2^0).
__device__ __forceinline__ int32_t scale_exponent(float a) {
    const uint32_t w = __float_as_uint(a);
    if (w == 0) return 0;
    const int32_t e = (int32_t)(w >> 23) - 127 - 8 + ((w & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(e, -126);
}
__device__ __forceinline__ float pow2(int32_t e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127

// The eight values of lane `i` of an entry, as floats.
template <int DT>
__device__ __forceinline__ void load8(const unsigned char* row, int i, float (&x)[8]) {
    if (DT == kKvBf16) {
        const uint4 w = *(const uint4*)(row + 16 * i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_lo(u[j]);
            x[2 * j + 1] = bf16_hi(u[j]);
        }
    } else {
        const float4 a = *(const float4*)(row + 32 * i), b = *(const float4*)(row + 32 * i + 16);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

// One entry (token, head) of K or V, `lanes` (a power of two, 8 values each)
// threads together: scale from the largest finite value, codes, stores.
template <int DT, bool Q8>
__device__ __forceinline__ void write_entry(const float (&x)[8], bool live, unsigned char* dst, float* scale, int i,
                                            int lanes) {
    if (!Q8) {
        if (live) {
            uint4 w;
            w.x = pack_bf16(x[0], x[1]);
            w.y = pack_bf16(x[2], x[3]);
            w.z = pack_bf16(x[4], x[5]);
            w.w = pack_bf16(x[6], x[7]);
            *(uint4*)(dst + 16 * i) = w;
        }
        return;
    }
    float a = 0.f;
    if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fabsf(x[j]);
            a = m < __uint_as_float(0x7F800000u) ? fmaxf(a, m) : a;  // a NaN or an infinity is left out
        }
    }
    for (int o = lanes >> 1; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    if (!live) return;
    const int32_t e = scale_exponent(a);
    const float f = pow2(-e);  // e lies in [-126, 120]: x * 2^-e is exact down to what e4m3 rounds to zero
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const bool fin = fabsf(x[j]) < __uint_as_float(0x7F800000u);
        y[j] = fin ? x[j] * f : __uint_as_float(0x7FC00000u);
    }
    uint2 w;
    w.x = pack_e4m3(y[0], y[1]) | (pack_e4m3(y[2], y[3]) << 16);
    w.y = pack_e4m3(y[4], y[5]) | (pack_e4m3(y[6], y[7]) << 16);
    *(uint2*)(dst + 8 * i) = w;
    if (i == 0) *scale = pow2(e);
}

// Entries (row, head) of a thread: their loads are under way together. Append of 130,238 e4m3 prompt tokens and gather
// of 146,153 tokens: two 178 and 142 us, four 184 and 145.
constexpr int kRows = 2;

// The same for eight bf16 values as they come (w), where all of the warp's are
// finite: their magnitudes compare as 16-bit integers, two at a time, and a
// power of two scales them exactly in bf16 (what falls below its normal range
// is zero in e4m3 too). A third of write_entry's instructions, which were what
// bounded the append of a prompt.
__device__ __forceinline__ void write_codes(const uint32_t (&w)[4], bool live, unsigned char* dst, float* scale, int i,
                                            int lanes) {
    constexpr uint32_t mag = 0x7FFF7FFFu;
    uint32_t m = live ? __vmaxu2(__vmaxu2(w[0] & mag, w[1] & mag), __vmaxu2(w[2] & mag, w[3] & mag)) : 0u;
    for (int o = lanes >> 1; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const uint32_t top = max(m & 0xFFFFu, m >> 16);
    if (__any_sync(0xFFFFFFFFu, top >= 0x7F80u)) {  // a NaN or an infinity somewhere
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_lo(w[j]);
            x[2 * j + 1] = bf16_hi(w[j]);
        }
        write_entry<kKvBf16, true>(x, live, dst, scale, i, lanes);
        return;
    }
    if (!live) return;
    const int32_t e = scale_exponent(__uint_as_float(top << 16));
    const uint32_t f = (uint32_t)(127 - e) << 7, f2 = f | f << 16;
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t y;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w[j]), "r"(f2));
        c[j] = pack_e4m3(bf16_lo(y), bf16_hi(y));
    }
    *(uint2*)(dst + 8 * i) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (i == 0) *scale = pow2(e);
}

// New tokens into the cache. A flat range of entries (row, head), 2^lanes_log
// threads each; a CTA finds its first row's sequence by a warp search over the
// offsets and steps on from there. A thread asks for its values first, so that
// the offsets, lengths and page numbers, each needing the last, come in their
// shadow. The grid's last CTAs write the statuses, one warp for each sequence.
// Issue bounds it to e4m3 (active in 83 % of cycles: conversion, and a look-up
// for each entry): 130,238 tokens of 8 heads in 178 us, 4.5 TB/s (0.67 of the
// copy bandwidth). bf16 to bf16 210 us, 5.1 TB/s (0.75); float32 to bf16
// 228 us, 7.0 TB/s, HBM. A round's 576 tokens: 3.6 us of latency (offsets,
// length, page, store).
template <int DT, bool Q8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvView c, const KvNew n, int lanes_log, int64_t ctas) {
    __shared__ int32_t b_first;
    const int warp = threadIdx.x >> 5;
    if ((int64_t)blockIdx.x >= ctas) {
        const int64_t b = ((int64_t)blockIdx.x - ctas) * (kThreads / 32) + warp;
        if (b >= c.B) return;
        const KvSeq s = kv_seq((int32_t)b, n.row_off, n.t_max, n.rows, n.kv_lens, c.bs, c.max_blocks, false);
        int32_t st = s.st;
        if (st == kKvOk) st = check_pages(c, (int32_t)b, s.L - s.T, s.L);
        if ((threadIdx.x & 31) == 0) n.seq_status[b] = st;
        return;
    }
    const int lanes = 1 << lanes_log, per = kThreads >> lanes_log;  // entries of a round
    const int32_t first = blockIdx.x * (per * kRows);               // entries of a launch: fewer than 2^31
    const int i = threadIdx.x & (lanes - 1);
    const bool column = i * 8 < c.D;
    constexpr bool packed = DT == kKvBf16 && Q8;
    int32_t r[kRows], h[kRows];
    float xk[packed ? 1 : kRows][8], xv[packed ? 1 : kRows][8];
    uint32_t wk[packed ? kRows : 1][4], wv[packed ? kRows : 1][4];
    bool live[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int32_t e = first + u * per + (int)(threadIdx.x >> lanes_log);
        r[u] = c.by_H.of(e);
        h[u] = e - r[u] * c.H;
        live[u] = r[u] < n.rows && column;
        if (live[u]) {
            const int64_t src = r[u] * n.row_bytes + (int64_t)h[u] * c.D * (DT == kKvBf16 ? 2 : 4);
            if constexpr (packed) {
                *(uint4*)wk[u] = *(const uint4*)(n.k + src + 16 * i);
                *(uint4*)wv[u] = *(const uint4*)(n.v + src + 16 * i);
            } else {
                load8<DT>(n.k + src, i, xk[u]);
                load8<DT>(n.v + src, i, xv[u]);
            }
        }
    }
    int32_t b = 0;
    if (n.row_off) {
        if (warp == 0) {
            const int32_t x = kv_find(n.row_off, c.B, c.by_H.of(first));
            if (threadIdx.x == 0) b_first = x;
        }
        __syncthreads();
        b = b_first;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        int64_t at = 0, sc = 0;
        if (r[u] < n.rows) {
            if (n.row_off)
                while (b < c.B && n.row_off[b + 1] <= r[u]) ++b;
            else
                b = r[u] / n.t_max;
            bool ok = false;
            if (b < c.B) {
                const KvSeq s = kv_seq(b, n.row_off, n.t_max, n.rows, n.kv_lens, c.bs, c.max_blocks, false);
                if (s.st == kKvOk && r[u] >= s.lo) {
                    const int32_t pos = s.L - s.T + (int32_t)(r[u] - s.lo);
                    const int32_t j = c.by_bs.of(pos), sl = pos - j * c.bs;
                    const int32_t pg = c.table[(int64_t)b * c.max_blocks + j];
                    ok = pg >= 0 && pg < c.num_blocks;
                    at = pg * c.block_bytes + sl * c.token_bytes + h[u] * c.head_bytes;
                    sc = ((int64_t)pg * c.H + h[u]) * c.bs + sl;
                }
            }
            live[u] = live[u] && ok;
        }
        if constexpr (packed) {
            write_codes(wk[u], live[u], c.k + at, c.ks + sc, i, lanes);
            write_codes(wv[u], live[u], c.v + at, c.vs + sc, i, lanes);
        } else {
            write_entry<DT, Q8>(xk[u], live[u], c.k + at, Q8 ? c.ks + sc : nullptr, i, lanes);
            write_entry<DT, Q8>(xv[u], live[u], c.v + at, Q8 ? c.vs + sc : nullptr, i, lanes);
        }
    }
}

// The cache back as rows: value = code * scale. Threads and entries as above;
// a thread's entries are all looked up, then all asked for, then written.
// Bound by HBM: 146,153 tokens of 8 heads from e4m3 in 143 us, 6.3 TB/s (0.93);
// to float32 265 us, 5.7 TB/s.
template <bool Q8, int ODT>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const KvView c, const KvRead g, int lanes_log, int64_t ctas) {
    __shared__ int32_t b_first;
    const int warp = threadIdx.x >> 5;
    if ((int64_t)blockIdx.x >= ctas) {
        const int64_t b = ((int64_t)blockIdx.x - ctas) * (kThreads / 32) + warp;
        if (b >= c.B) return;
        const int64_t lo = g.out_off[b], hi = g.out_off[b + 1];
        const int32_t L = g.kv_lens[b];
        int32_t st = kKvOk;
        if (lo < 0 || hi > g.rows || hi - lo != L)
            st = kKvBadLayout;
        else if (L < 0 || L > (int64_t)c.bs * c.max_blocks)
            st = kKvBadKv;
        else
            st = check_pages(c, (int32_t)b, 0, L);
        if ((threadIdx.x & 31) == 0) g.seq_status[b] = st;
        return;
    }
    const int lanes = 1 << lanes_log, per = kThreads >> lanes_log;
    const int32_t first = blockIdx.x * (per * kRows);
    if (warp == 0) {
        const int32_t x = kv_find(g.out_off, c.B, c.by_H.of(first));
        if (threadIdx.x == 0) b_first = x;
    }
    __syncthreads();
    const int i = threadIdx.x & (lanes - 1);
    if (i * 8 >= c.D) return;
    int32_t b = b_first;
    int64_t at[kRows], sc[kRows];  // at: -1 no row of a sequence, -2 a page outside the pool
    int32_t e[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        e[u] = first + u * per + (int)(threadIdx.x >> lanes_log);
        at[u] = -1;
        sc[u] = 0;
        const int32_t r = c.by_H.of(e[u]), h = e[u] - r * c.H;
        if (r >= g.rows) continue;
        while (b < c.B && g.out_off[b + 1] <= r) ++b;
        if (b >= c.B) continue;
        const int64_t lo = g.out_off[b], hi = g.out_off[b + 1];
        const int32_t L = g.kv_lens[b];
        if (lo < 0 || hi > g.rows || hi - lo != L || r < lo || L > (int64_t)c.bs * c.max_blocks) continue;
        const int32_t pos = (int32_t)(r - lo);
        const int32_t j = c.by_bs.of(pos), sl = pos - j * c.bs;
        const int32_t pg = c.table[(int64_t)b * c.max_blocks + j];
        at[u] = -2;
        if (pg < 0 || pg >= c.num_blocks) continue;
        at[u] = pg * c.block_bytes + sl * c.token_bytes + h * c.head_bytes;
        sc[u] = ((int64_t)pg * c.H + h) * c.bs + sl;
    }
    uint4 w[kRows][2];
    float s[kRows][2];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            w[u][kv] = make_uint4(0, 0, 0, 0);
            s[u][kv] = 0.f;
            if (at[u] < 0) continue;
            const unsigned char* src = (kv ? c.v : c.k) + at[u];
            if (Q8) {
                const uint2 x = *(const uint2*)(src + 8 * i);
                w[u][kv].x = x.x;
                w[u][kv].y = x.y;
                s[u][kv] = (kv ? c.vs : c.ks)[sc[u]];
            } else {
                w[u][kv] = *(const uint4*)(src + 16 * i);
            }
        }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        if (at[u] == -1) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            unsigned char* dst = (kv ? g.v : g.k) + e[u] * ((int64_t)c.D * (ODT == kKvBf16 ? 2 : 4));
            const uint4 y = w[u][kv];
            if (!Q8 && ODT == kKvBf16) {
                *(uint4*)(dst + 16 * i) = y;
                continue;
            }
            float x[8];
            if (Q8) {
                const uint32_t h2[4] = {e4m3_f16x2(y.x & 0xFFFF), e4m3_f16x2(y.x >> 16), e4m3_f16x2(y.y & 0xFFFF),
                                        e4m3_f16x2(y.y >> 16)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = __half22float2(*(const __half2*)&h2[j]);
                    x[2 * j] = f.x * s[u][kv];
                    x[2 * j + 1] = f.y * s[u][kv];
                }
            } else {
                const uint32_t q[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[2 * j] = bf16_lo(q[j]);
                    x[2 * j + 1] = bf16_hi(q[j]);
                }
            }
            if (ODT == kKvBf16) {
                *(uint4*)(dst + 16 * i) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                     pack_bf16(x[6], x[7]));
            } else {
                *(float4*)(dst + 32 * i) = make_float4(x[0], x[1], x[2], x[3]);
                *(float4*)(dst + 32 * i + 16) = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

// The accepted path's entries to the front of the tree's slots. Path nodes
// rise (path[i] >= i + 1), so entry i's target, slot 1 + i, is read by no
// later entry: taken in order, each thread's column moves in place. A thread
// owns one 16-byte column (or one scale) of one layer and head, and takes the
// path kMove entries at a time: loads together, then stores (of 64 trees in 32
// layers 8.5 us; one at a time 12.3). Bound by latency: path, pages, entries.
// Each CTA of a sequence reads its old length; the first writes the new one
// (m.part says whether that is this launch's to do, see launch_kv_compact).
constexpr int kMove = 4;
__global__ void __launch_bounds__(kThreads, 6) kv_compact_kernel(const KvView c, const KvMove m) {
    __shared__ int64_t from[kMove], to[kMove];    // page * block + slot * token, bytes
    __shared__ int64_t sfrom[kMove], sto[kMove];  // scales: page * H * bs + slot
    const int32_t b = blockIdx.x;
    const int64_t lo = m.node_off[b], hi = m.node_off[b + 1];
    const int32_t L = m.kv_in[b], a = m.accepted[b];
    int32_t st = kKvOk;
    if (lo < 0 || hi > m.nodes || hi <= lo || a < 0 || a >= hi - lo)
        st = kKvBadLayout;
    else if (L < hi - lo || L > (int64_t)c.bs * c.max_blocks)
        st = kKvBadKv;
    const int32_t N = (int32_t)(hi - lo);
    const int32_t base = L - N;
    const int32_t* table = c.table + (int64_t)b * c.max_blocks;
    bool moves = false;
    if (st == kKvOk) {
        bool bad = false;
        for (int32_t i = threadIdx.x; i < a; i += kThreads) {
            const int32_t v = m.path[lo + i], u = i ? m.path[lo + i - 1] : 0;
            moves |= v != i + 1;
            if (v <= u || v >= N) {
                bad = true;
            } else {
                const int32_t ps = table[c.by_bs.of(base + v)], pd = table[c.by_bs.of(base + 1 + i)];
                bad |= ps < 0 || ps >= c.num_blocks || pd < 0 || pd >= c.num_blocks;
            }
        }
        if (__syncthreads_or(bad)) st = kKvBadLayout;
        moves = __syncthreads_or(moves);
    }
    if (m.part != kMoveEntries && blockIdx.y == 0 && threadIdx.x == 0) {
        const int32_t out = st == kKvOk ? L - (N - 1 - a) : L;
        m.kv_out[b] = out;
        if (m.out_blocks) m.out_blocks[b] = (int32_t)(((int64_t)out + c.bs - 1) / c.bs);
        if (m.seq_status) m.seq_status[b] = st;
    }
    if (st != kKvOk || !moves || m.part == kMoveLengths) return;  // the first children all the way: every entry is in its place
    const int32_t cols = c.D * c.esz / 16 + (c.ks ? 1 : 0);  // 16-byte columns of an entry, and its scale
    const uint32_t all = (uint32_t)c.layers * c.H * 2 * cols;  // the host keeps it below 2^31
    const uint32_t t = blockIdx.y * kThreads + threadIdx.x;
    const bool live = t < all;
    uint32_t x = t / cols;
    const uint32_t col = t - x * cols;
    const uint32_t kv = x & 1;
    x >>= 1;
    const int64_t layer = x / c.H;
    const uint32_t h = x - (uint32_t)layer * c.H;
    unsigned char* p = (kv ? c.v : c.k) + layer * c.layer_bytes + h * c.head_bytes + 16 * col;
    const bool scale = c.ks && col == cols - 1;
    float* sp = scale && live ? (kv ? c.vs : c.ks) + layer * c.scale_layer + (int64_t)h * c.bs : nullptr;
    for (int32_t i0 = 0; i0 < a; i0 += kMove) {
        const int32_t k = min(kMove, a - i0);
        __syncthreads();
        if (threadIdx.x < k) {
            const int32_t i = i0 + threadIdx.x;
            const int32_t s = base + m.path[lo + i], d = base + 1 + i;
            const int32_t js = c.by_bs.of(s), jd = c.by_bs.of(d);
            const int64_t ps = table[js], pd = table[jd];
            from[threadIdx.x] = ps * c.block_bytes + (s - js * c.bs) * c.token_bytes;
            to[threadIdx.x] = pd * c.block_bytes + (d - jd * c.bs) * c.token_bytes;
            sfrom[threadIdx.x] = ps * c.H * c.bs + s - js * c.bs;
            sto[threadIdx.x] = pd * c.H * c.bs + d - jd * c.bs;
        }
        __syncthreads();
        if (!live) continue;
        if (scale) {
            float y[kMove];
#pragma unroll
            for (int j = 0; j < kMove; ++j)
                if (j < k) y[j] = sp[sfrom[j]];
#pragma unroll
            for (int j = 0; j < kMove; ++j)
                if (j < k && sfrom[j] != sto[j]) sp[sto[j]] = y[j];
        } else {
            uint4 y[kMove];
#pragma unroll
            for (int j = 0; j < kMove; ++j)
                if (j < k && from[j] != to[j]) y[j] = *(const uint4*)(p + from[j]);
#pragma unroll
            for (int j = 0; j < kMove; ++j)
                if (j < k && from[j] != to[j]) *(uint4*)(p + to[j]) = y[j];
        }
    }
}

// ------------------------------------------------------------ plain attention
// For head_dim above 128. A CTA for each query row (token, query head), float32
// throughout: its warps take 32 positions at a time in turn, a lane's
// position's product with the query in shared memory, the running maximum and
// sum over the warp, then the weighted values with eight of the head's columns
// to a lane; the warps' sums are joined at the end. Bound by its 16-byte loads'
// latency and by every query row reading the cache for itself: 64 x 9 tokens
// over 2,048 positions, 2 x 4 heads of 256, 1.67 ms for bytes of 40 us (e4m3 the
// same time); one token over 4,096 positions 204 us.
constexpr int kPlainWarps = 8;

// Eight elements of an entry from `d` on.
__device__ __forceinline__ void entry_at(const KvView& c, const unsigned char* row, int d, float (&x)[8]) {
    if (c.esz == 2) {
        load8<kKvBf16>(row, d / 8, x);
        return;
    }
    const uint2 w = *(const uint2*)(row + d);
    const uint32_t h2[4] = {e4m3_f16x2(w.x & 0xFFFF), e4m3_f16x2(w.x >> 16), e4m3_f16x2(w.y & 0xFFFF), e4m3_f16x2(w.y >> 16)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*(const __half2*)&h2[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}

__global__ void __launch_bounds__(kPlainWarps * 32) kv_attend_plain_kernel(const KvAttend p) {
    __shared__ __align__(16) float q_sh[kKvMaxDim];
    __shared__ float o_sh[kPlainWarps][kKvMaxDim], m_sh[kPlainWarps], l_sh[kPlainWarps];
    __shared__ uint32_t anc[kKvMaxQueries / 32];
    static_assert(kKvMaxDim == 256 && kPlainWarps * 32 == kKvMaxDim, "eight columns to a lane, one to a thread");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const KvView& c = p.c;
    const int32_t b = blockIdx.x;
    const KvSeq s = kv_seq(b, p.row_off, p.t_max, p.rows, p.kv_lens, c.bs, c.max_blocks, true);
    int32_t st = s.st;
    if (st == kKvOk && p.parent) {
        bool bad = false;
        for (int32_t v = lane; v < s.T; v += 32) {
            const int32_t u = p.parent[s.lo + v];
            bad |= v == 0 ? u != -1 : (u < 0 || u >= v);
        }
        if (__any_sync(0xFFFFFFFFu, bad)) st = kKvBadLayout;
    }
    if (blockIdx.y == 0 && warp == 0 && p.seq_status) {
        const int32_t st2 = st == kKvOk ? check_pages(c, b, 0, s.T ? s.L : 0) : st;
        if (lane == 0) p.seq_status[b] = st2;
    }
    if (s.lo < 0) return;
    const float none = __uint_as_float(0xFF800000u);
    const bool column = lane * 8 < c.D;
    const int32_t ctx = s.L - s.T;
    const float k2 = p.scale * kLog2e;
    for (int64_t w = blockIdx.y; w < (int64_t)s.T * p.Hq; w += gridDim.y) {
        const int32_t t = (int32_t)(w / p.Hq), hq = (int32_t)(w % p.Hq), h = hq / p.G;
        const int64_t row = s.lo + t;
        unsigned char* out = p.out + (row * p.Hq + hq) * (int64_t)c.D * 2;
        if (st != kKvOk) {
            if (tid < c.D) *(uint16_t*)(out + 2 * tid) = 0;
            if (p.lse && tid == 0) p.lse[row * p.Hq + hq] = none;
            continue;
        }
        const unsigned char* q = p.q + row * p.q_row_bytes + (int64_t)hq * c.D * 2;
        __syncthreads();  // the last row is done
        if (tid < c.D) q_sh[tid] = bf16_lo(*(const uint16_t*)(q + 2 * tid));
        if (tid < kKvMaxQueries / 32) anc[tid] = 0;
        __syncthreads();
        if (p.parent && tid == 0)
            for (int32_t v = t; v >= 0; v = p.parent[s.lo + v]) anc[v >> 5] |= 1u << (v & 31);
        __syncthreads();
        float m = none, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const int32_t last = p.parent ? s.L : ctx + t + 1;  // positions past it are not seen
        for (int32_t j0 = warp * 32; j0 < last; j0 += kPlainWarps * 32) {
            const int32_t j = j0 + lane;
            float x = none, vscale = 1.f;
            int64_t at = -1;
            if (j < last && (!p.parent || j < ctx || (anc[(j - ctx) >> 5] >> ((j - ctx) & 31) & 1))) {
                const int32_t pg = c.table[(int64_t)b * c.max_blocks + c.by_bs.of(j)];
                const int32_t sl = j - c.by_bs.of(j) * c.bs;
                if (pg >= 0 && pg < c.num_blocks) {
                    at = pg * c.block_bytes + sl * c.token_bytes + h * c.head_bytes;
                    float acc = 0.f;
#pragma unroll 4
                    for (int d = 0; d < c.D; d += 8) {
                        float e[8];
                        entry_at(c, c.k + at, d, e);
                        const float4 q0 = *(const float4*)(q_sh + d), q1 = *(const float4*)(q_sh + d + 4);
                        const float f[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
                        for (int k = 0; k < 8; ++k) acc = fmaf(f[k], e[k], acc);
                    }
                    if (c.ks) {
                        const int64_t sc = ((int64_t)pg * c.H + h) * c.bs + sl;
                        acc *= c.ks[sc];
                        vscale = c.vs[sc];
                    }
                    x = acc * k2;
                }
            }
            float mt = x;
            for (int sh = 16; sh; sh >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, sh));
            const float mn = fmaxf(m, mt);
            const float mr = mn == none ? 0.f : mn;
            const float f = exp2f(m - mr);
            const float w2 = at >= 0 ? exp2f(x - mr) : 0.f;
            float lt = w2;
            for (int sh = 16; sh; sh >>= 1) lt += __shfl_xor_sync(0xFFFFFFFFu, lt, sh);
            l = l * f + lt;
            m = mn;
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] *= f;
            const float wv = w2 * vscale;
#pragma unroll 4
            for (int src = 0; src < 32; ++src) {
                const int64_t a = __shfl_sync(0xFFFFFFFFu, at, src);
                const float wt = __shfl_sync(0xFFFFFFFFu, wv, src);
                if (a < 0 || !column) continue;
                float e[8];
                entry_at(c, c.v + a, lane * 8, e);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = fmaf(wt, e[k], o[k]);
            }
        }
        // the warps' sums, in their order
#pragma unroll
        for (int k = 0; k < 8; ++k) o_sh[warp][lane * 8 + k] = o[k];
        if (lane == 0) m_sh[warp] = m, l_sh[warp] = l;
        __syncthreads();
        m = none;
        for (int i = 0; i < kPlainWarps; ++i) m = fmaxf(m, m_sh[i]);
        const float mr = m == none ? 0.f : m;
        float sum = 0.f, x = 0.f;
        for (int i = 0; i < kPlainWarps; ++i) {
            const float f = exp2f(m_sh[i] - mr);
            sum += f * l_sh[i];
            x = fmaf(f, o_sh[i][tid], x);
        }
        if (tid < c.D) *(uint16_t*)(out + 2 * tid) = (uint16_t)pack_bf16(sum == 0.f ? 0.f : x / sum, 0.f);
        if (p.lse && tid == 0) p.lse[row * p.Hq + hq] = sum == 0.f ? none : (m + log2f(sum)) * 0.69314718055994531f;
    }
}

int lanes_log_of(int32_t D) {
    int n = 0;
    while ((8 << n) < D) ++n;
    return n;  // D <= 256: at most a warp
}

}  // namespace

cudaError_t launch_kv_append(const KvView& c, const KvNew& n, cudaStream_t s) {
    const int lanes = lanes_log_of(c.D);
    const int per = (kThreads >> lanes) * kRows;
    const int64_t ctas = (n.rows * c.H + per - 1) / per;
    const int64_t grid = ctas + (n.seq_status ? (c.B + kThreads / 32 - 1) / (kThreads / 32) : 0);
    if (grid == 0) return cudaSuccess;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const bool q8 = c.esz == 1;
    auto* f = n.dtype == kKvBf16 ? (q8 ? kv_append_kernel<kKvBf16, true> : kv_append_kernel<kKvBf16, false>)
                                 : (q8 ? kv_append_kernel<kKvF32, true> : kv_append_kernel<kKvF32, false>);
    f<<<(unsigned)grid, kThreads, 0, s>>>(c, n, lanes, ctas);
    return cudaGetLastError();
}

cudaError_t launch_kv_gather(const KvView& c, const KvRead& g, cudaStream_t s) {
    const int lanes = lanes_log_of(c.D);
    const int per = (kThreads >> lanes) * kRows;
    const int64_t ctas = (g.rows * c.H + per - 1) / per;
    const int64_t grid = ctas + (g.seq_status ? (c.B + kThreads / 32 - 1) / (kThreads / 32) : 0);
    if (grid == 0) return cudaSuccess;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const bool q8 = c.esz == 1;
    auto* f = g.dtype == kKvBf16 ? (q8 ? kv_gather_kernel<true, kKvBf16> : kv_gather_kernel<false, kKvBf16>)
                                 : (q8 ? kv_gather_kernel<true, kKvF32> : kv_gather_kernel<false, kKvF32>);
    f<<<(unsigned)grid, kThreads, 0, s>>>(c, g, lanes, ctas);
    return cudaGetLastError();
}

cudaError_t launch_kv_compact(const KvView& c, const KvMove& m, cudaStream_t s) {
    const int64_t y = kv_compact_ctas(c.layers, c.H, c.D * c.esz, c.ks != nullptr);
    if (y > kKvCompactMaxCtas) return cudaErrorInvalidValue;  // (refused by the caller)
    // Lengths cut in place: a CTA of the sequence that starts after the new length is written would take it for the old
    // one and move other entries. With several CTAs to a sequence a launch of its own writes them, behind the moves.
    const bool apart = y > 1 && m.kv_out == m.kv_in;
    KvMove w = m;
    w.part = apart ? kMoveEntries : kMoveAll;
    kv_compact_kernel<<<dim3((unsigned)c.B, (unsigned)y), kThreads, 0, s>>>(c, w);
    if (apart) {
        w.part = kMoveLengths;
        kv_compact_kernel<<<dim3((unsigned)c.B, 1), kThreads, 0, s>>>(c, w);
    }
    return cudaGetLastError();
}

cudaError_t launch_kv_attend_plain(const KvAttend& p, cudaStream_t s) {
    const int64_t y = std::min<int64_t>((int64_t)p.t_max * p.Hq, 65535);
    kv_attend_plain_kernel<<<dim3((unsigned)p.c.B, (unsigned)y), kPlainWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace specv
