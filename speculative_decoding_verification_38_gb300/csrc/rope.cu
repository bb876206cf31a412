// rope.cu -- rotary positions: new keys on their way into the paged cache with
// the pass's queries beside them, and rows without a cache.
#include <algorithm>

#include "kv.cuh"

namespace specv {

namespace {

constexpr int kThreads = kKvThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 8;               // most tokens of a CTA
constexpr int kPairs = kKvMaxDim / 2;

// inv_freq / (2 pi) as a fraction of a turn in units of 2^-64, so that the angle of any integer position is one wrapping
// product: round(2^64 / (2 pi)) times the float's significand, shifted by its exponent. The constant's half unit and
// the shift's one come to two units at most for inv_freq up to 2, 2^-32 of a turn at the furthest position.
constexpr uint64_t kTurn = 0x28BE60DB9391054Aull;
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
    const uint32_t w = __float_as_uint(inv_freq);
    const int e = (int)(w >> 23 & 255);
    const uint64_t m = (w & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);  // 86 bits
    const int right = 150 - max(e, 1);                        // the value is the product / 2^right
    uint64_t f;
    if (right <= 0)
        f = right > -64 ? lo << -right : 0;
    else if (right < 64)
        f = lo >> right | hi << (64 - right);
    else
        f = right < 128 ? hi >> (right - 64) : 0;
    return w >> 31 ? 0 - f : f;
}

// Cosine and sine of a number of turns in units of 2^-64: the quarter turn by its top bits, what is left of it, at most an
// eighth, by the Taylor series (sine to x^9, cosine to x^10: 2e-9 and 2e-10 at pi / 4).
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
    const uint64_t q = (turns + (1ull << 61)) >> 62;
    const float v = __ll2float_rn((int64_t)(turns - (q << 62)));
    constexpr float hi = 0x1.921fb6p-62f, lo = -0x1.777a5cp-87f;  // 2 pi / 2^64, two parts
    const float x = fmaf(v, hi, v * lo), y = x * x;
    float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(s, y, 1.f / 120.f);
    s = fmaf(s, y, -1.f / 6.f);
    s = fmaf(s * y, x, x);
    float c = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(c, y, -1.f / 720.f);
    c = fmaf(c, y, 1.f / 24.f);
    c = fmaf(c, y, -0.5f);
    c = fmaf(c, y, 1.f);
    const bool odd = q & 1;
    const float a = odd ? s : c, b = odd ? c : s;
    return make_float2((q + 1) & 2 ? -a : a, q & 2 ? -b : b);
}

// Where a pair's cosine and sine lie in shared memory. Halves: a thread takes eight pairs in a row, the first four of each
// in one half of the array and the last four in the other, so that 16-byte reads of neighbours meet no bank twice.
__device__ __forceinline__ int place_of(int pair, bool adjacent) {
    return adjacent ? pair : (pair & 4 ? kPairs / 2 : 0) + (pair >> 3) * 4 + (pair & 3);
}

constexpr int kResident = 4;             // CTAs on an SM: 64 registers a thread (3, 4, 5 and 6 of them: prompts 542, 490, 486
                                         // and 606 us; a round 5.1, 5.1, 5.6 and 6.8)
constexpr int kDeepest = kKvMaxQueries - 1;  // of a tree's nodes: a way to the root is one load after another (without a limit a
                                             // chain of 65,536 given as a tree took 25 ms, each token its whole way)
struct Token {
    int64_t at, scale;  // its entry in the cache: bytes, scales
    bool known, cached; // it has a position; its page is there
};

// The elements of a head that a thread takes: chunks c0 and c1, eight each (a chunk past the head: none).
struct Chunks {
    int c0, c1;
    bool has0, has1, turns;
};

// A thread's chunks as they lie in memory.
template <int DT>
struct Raw {
    uint4 w[DT == kKvBf16 ? 2 : 4];
    __device__ __forceinline__ void load(const unsigned char* row, const Chunks& k, bool live) {
        constexpr int per = DT == kKvBf16 ? 1 : 2;  // 16-byte words of a chunk
#pragma unroll
        for (int i = 0; i < 2 * per; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (live && (i < per ? k.has0 : k.has1)) w[i] = *((const uint4*)row + (i < per ? k.c0 : k.c1) * per + i % per);
        }
    }
    __device__ __forceinline__ void floats(float (&x)[2][8]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (DT == kKvBf16) {
                const uint32_t u[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[h][2 * j] = bf16_lo(u[j]);
                    x[h][2 * j + 1] = bf16_hi(u[j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 u = w[(2 * h + i) % (DT == kKvBf16 ? 2 : 4)];
                    x[h][4 * i] = __uint_as_float(u.x), x[h][4 * i + 1] = __uint_as_float(u.y);
                    x[h][4 * i + 2] = __uint_as_float(u.z), x[h][4 * i + 3] = __uint_as_float(u.w);
                }
            }
        }
    }
};

// Both chunks of a row's head (at `row`), turned. VEC: the rotary part is a multiple of 16 elements, so that pairs of
// halves lie in the two chunks of one thread; otherwise an element's other half is fetched by itself.
template <int DT, bool VEC>
__device__ __forceinline__ void turn(const unsigned char* row, const Chunks& k, const Rope& r, const float* cs, const float* sn,
                                     float (&x)[2][8]) {
    if (VEC && !r.adjacent) {
        const int l = k.c0 * 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 c4 = *(const float4*)(cs + h * (kPairs / 2) + l), s4 = *(const float4*)(sn + h * (kPairs / 2) + l);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = x[0][4 * h + j], b = x[1][4 * h + j];
                x[0][4 * h + j] = fmaf(a, c[j], -(b * s[j]));
                x[1][4 * h + j] = fmaf(b, c[j], a * s[j]);
            }
        }
    } else if (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int p = (h ? k.c1 : k.c0) * 4;
            const float4 c4 = *(const float4*)(cs + p), s4 = *(const float4*)(sn + p);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = x[h][2 * j], b = x[h][2 * j + 1];
                x[h][2 * j] = fmaf(a, c[j], -(b * s[j]));
                x[h][2 * j + 1] = fmaf(b, c[j], a * s[j]);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int d0 = (h ? k.c1 : k.c0) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int d = d0 + j;
                if (d >= r.rd) continue;
                const bool second = r.adjacent ? d & 1 : d >= r.half;
                const int pair = r.adjacent ? d >> 1 : second ? d - r.half : d;
                const int other = r.adjacent ? d ^ 1 : second ? d - r.half : d + r.half;
                const float o = DT == kKvBf16 ? bf16_lo(((const uint16_t*)row)[other]) : ((const float*)row)[other];
                const int p = place_of(pair, r.adjacent);
                x[h][j] = second ? fmaf(x[h][j], cs[p], o * sn[p]) : fmaf(x[h][j], cs[p], -(o * sn[p]));
            }
        }
    }
}

template <int ODT>
__device__ __forceinline__ void store8(unsigned char* row, int c, const float (&x)[8]) {
    if (ODT == kKvBf16) {
        *(uint4*)(row + 16 * c) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        *(float4*)(row + 32 * c) = make_float4(x[0], x[1], x[2], x[3]);
        *(float4*)(row + 32 * c + 16) = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// An entry into the cache, by `lanes` threads together.
template <bool Q8>
__device__ __forceinline__ void store_entry(const float (&x)[2][8], const Chunks& k, bool live, unsigned char* dst, float* scale,
                                            bool first, int lanes) {
    if (!Q8) {
        if (live && k.has0) store8<kKvBf16>(dst, k.c0, x[0]);
        if (live && k.has1) store8<kKvBf16>(dst, k.c1, x[1]);
        return;
    }
    float a = 0.f;  // (chunks that are not there hold zeros)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fabsf(x[h][j]);
            a = m < __uint_as_float(0x7F800000u) ? fmaxf(a, m) : a;  // a NaN or an infinity is left out
        }
    for (int o = lanes >> 1; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    if (!live) return;
    const int32_t e = scale_exponent(a);
    const float f = pow2(-e);  // e lies in [-126, 120]: x * 2^-e is exact down to what e4m3 rounds to zero
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!(h ? k.has1 : k.has0)) continue;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = fabsf(x[h][j]) < __uint_as_float(0x7F800000u) ? x[h][j] * f : __uint_as_float(0x7FC00000u);
        *(uint2*)(dst + 8 * (h ? k.c1 : k.c0)) = make_uint2(pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16,
                                                          pack_e4m3(y[4], y[5]) | pack_e4m3(y[6], y[7]) << 16);
    }
    if (first) *scale = pow2(e);
}

// `tb` tokens to a CTA. Their sequences, entries and positions are looked up by a lane each; sines and cosines are made
// once for a token by all threads; then the warps take keys, values and queries, 2^lanes_log threads to a head. What a
// warp takes first is asked for before the look-ups, and the next before the last is done with. n.k null: rows without a
// cache, at q.x.
// Bounds (8 key-value and 32 query heads of 128): HBM for many tokens, 130,238 with their queries bf16 to bf16 490 us, 6.5
// TB/s (0.96 of the copy bandwidth), 131,072 rows of queries 333 us, 6.5 TB/s; latency for a round, 576 tokens 5.1 us
// (offsets, length, page, store), 576 rows of queries alone 3.5.
template <int DT, bool Q8, int ODT, bool VEC>
__global__ void __launch_bounds__(kThreads, kResident) rope_kernel(const __grid_constant__ KvView c, const __grid_constant__ KvNew n,
                                                                   const __grid_constant__ Rope r,
                                                                   const __grid_constant__ RopeRows q, const int32_t* parent,
                                                                   int lanes_log, int tb, int64_t ctas) {
    __shared__ __align__(16) float cs[kTokens][kPairs], sn[kTokens][kPairs];
    __shared__ Token tok[kTokens];
    __shared__ int32_t pos[kTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool cache = n.k != nullptr;
    if ((int64_t)blockIdx.x >= ctas) {
        const int64_t b = ((int64_t)blockIdx.x - ctas) * kWarps + warp;
        if (b >= c.B) return;
        const KvSeq s = kv_seq((int32_t)b, n.row_off, n.t_max, n.rows, n.kv_lens, c.bs, c.max_blocks, false);
        int32_t st = s.st;
        if (st == kKvOk && parent) {
            bool bad = false;
            for (int32_t v = lane; v < s.T; v += 32) {
                const int32_t u = parent[s.lo + v];
                bad |= v == 0 ? u != -1 : (u < 0 || u >= v);
            }
            if (__any_sync(0xFFFFFFFFu, bad)) st = kKvBadLayout;
            // (a smaller tree has no node that deep; every parent is before its child here)
            for (int32_t v0 = 0; s.T > kKvMaxQueries && st == kKvOk && v0 < s.T; v0 += 32) {
                int32_t v = min(v0 + lane, s.T - 1);
                for (int i = 0; v > 0 && i < kDeepest; ++i) v = parent[s.lo + v];
                if (__any_sync(0xFFFFFFFFu, v > 0)) st = kKvBadLayout;
            }
        }
        if (st == kKvOk) st = check_pages(c, (int32_t)b, s.L - s.T, s.L);
        if (lane == 0) n.seq_status[b] = st;
        return;
    }
    const int64_t first = (int64_t)blockIdx.x * tb;
    const int nt = (int)min((int64_t)tb, n.rows - first);

    // this thread's part of a head
    const int lanes = 1 << lanes_log, l = lane & (lanes - 1), groups_log = 5 - lanes_log, sub = lane >> lanes_log;
    Chunks k;
    const int D = cache ? c.D : q.D;
    if (VEC) {
        const int turning = r.rd >> 4;
        k.turns = l < turning;
        k.c0 = k.turns ? l : 2 * l;  // (2 turning + 2 (l - turning))
        k.c1 = k.turns ? l + turning : k.c0 + 1;
    } else {
        k.c0 = 2 * l;
        k.c1 = k.c0 + 1;
        k.turns = k.c0 * 8 < r.rd;
    }
    k.has0 = k.c0 * 8 < D;
    k.has1 = k.c1 * 8 < D;
    // the CTA's heads, 2^groups_log to a warp at a time: [0, u_v) keys, [u_v, u_q) values, [u_q, u_end) queries
    constexpr int isz = DT == kKvBf16 ? 2 : 4, osz = ODT == kKvBf16 ? 2 : 4;
    const int entries = cache ? nt * c.H : 0, heads = nt * q.heads, more = (1 << groups_log) - 1;
    const int u_v = (entries + more) >> groups_log, u_q = 2 * u_v, u_end = u_q + ((heads + more) >> groups_log);
    int t = 0, h = 0;
    bool live = false;
    Raw<DT> raw;
    const unsigned char* row = nullptr;
    auto ask = [&](int u) {
        const bool query = u >= u_q;
        const int e = ((u - (query ? u_q : u >= u_v ? u_v : 0)) << groups_log) + sub;
        live = e < (query ? heads : entries);
        t = live ? (query ? r.by_heads.of(e) : c.by_H.of(e)) : 0;
        h = e - t * (query ? q.heads : c.H);
        row = (query ? q.x : u >= u_v ? n.v : n.k) + (first + t) * (query ? q.x_row_bytes : n.row_bytes) + (int64_t)h * D * isz;
        raw.load(row, k, live);
    };
    if (warp < u_end) ask(warp);

    // a thread's pair, and of how many tokens at a time
    int wide = 5;  // log2 of the threads to a token
    while ((1 << wide) < r.half) ++wide;
    const int pair = threadIdx.x & ((1 << wide) - 1);
    const float freq = pair < r.half ? r.inv_freq[pair] : 0.f;
    if (cache) {
        if (warp == 0) {
            int32_t b = n.row_off ? kv_find(n.row_off, c.B, first) : (int32_t)(first / n.t_max);
            if (lane < nt) {
                const int64_t at_row = first + lane;
                Token k;
                k.at = k.scale = 0;
                k.known = k.cached = false;
                int32_t p = 0;
                if (n.row_off)
                    while (b < c.B && n.row_off[b + 1] <= at_row) ++b;
                else
                    b = (int32_t)(at_row / n.t_max);
                if (b < c.B) {
                    const KvSeq s = kv_seq(b, n.row_off, n.t_max, n.rows, n.kv_lens, c.bs, c.max_blocks, false);
                    if (s.st == kKvOk && at_row >= s.lo) {
                        const int32_t t = (int32_t)(at_row - s.lo), at = s.L - s.T + t;
                        const int32_t j = c.by_bs.of(at), sl = at - j * c.bs;
                        const int32_t pg = c.table[(int64_t)b * c.max_blocks + j];
                        p = at;
                        k.known = true;
                        if (parent) {  // its depth
                            p = s.L - s.T;
                            int32_t v = t;
                            for (int i = 0; v > 0 && i < kDeepest; ++i) {
                                const int32_t u = parent[s.lo + v];
                                if (u < 0 || u >= v) break;
                                v = u;
                                ++p;
                            }
                            k.known = v == 0 && parent[s.lo] == -1;
                        }
                        k.cached = k.known && pg >= 0 && pg < c.num_blocks;
                        k.at = pg * c.block_bytes + sl * c.token_bytes;
                        k.scale = (int64_t)pg * c.H * c.bs + sl;
                    }
                }
                tok[lane] = k;
                pos[lane] = p;
            }
        }
        __syncthreads();
    }
    if (pair < r.half) {
        const uint64_t turn_of = turns_of(freq);
        const bool sound = fabsf(freq) <= 0x1p20f;
        const int axis = r.one_axis ? 0 : r.axis_of(pair), to = place_of(pair, r.adjacent);
        for (int i = threadIdx.x >> wide; i < nt; i += kThreads >> wide) {
            const int32_t p = r.positions ? r.positions[axis * r.rows + first + i] : pos[i];
            const float2 y = cos_sin((uint64_t)(int64_t)p * turn_of);
            cs[i][to] = sound ? y.x * r.factor : __uint_as_float(0x7FC00000u);
            sn[i][to] = sound ? y.y * r.factor : __uint_as_float(0x7FC00000u);
        }
    }
    __syncthreads();

    for (int u = warp; u < u_end; u += kWarps) {
        const int now_t = t, now_h = h;
        const unsigned char* const now_row = row;
        const bool query = u >= u_q, key = u < u_v;
        const bool now_live = live && (!cache || (query ? tok[t].known : tok[t].cached));
        float x[2][8];
        raw.floats(x);
        if (u + kWarps < u_end) ask(u + kWarps);
        if ((key || query) && k.turns && now_live) turn<DT, VEC>(now_row, k, r, cs[now_t], sn[now_t], x);
        if (query) {
            if (!VEC) __syncwarp();  // in place: a head's elements are all read before one is written
            unsigned char* const out = q.out + (first + now_t) * q.out_row_bytes + (int64_t)now_h * D * osz;
            if (now_live && k.has0) store8<ODT>(out, k.c0, x[0]);
            if (now_live && k.has1) store8<ODT>(out, k.c1, x[1]);
        } else {
            const int64_t at = tok[now_t].at + now_h * c.head_bytes, sc = tok[now_t].scale + (int64_t)now_h * c.bs;
            store_entry<Q8>(x, k, now_live, (key ? c.k : c.v) + at, Q8 ? (key ? c.ks : c.vs) + sc : nullptr, l == 0, lanes);
        }
    }
}

template <int DT, bool Q8, int ODT>
cudaError_t launch(const KvView& c, const KvNew& n, const Rope& r, const RopeRows& q, const int32_t* parent, cudaStream_t s) {
    const int D = n.k ? c.D : q.D;
    int lanes_log = 0;
    while ((16 << lanes_log) < D) ++lanes_log;  // D <= 256: at most 16 lanes
    const int64_t slots = 152 * kResident;  // few tokens, one to a CTA; then as many as make one wave (trees of 64: 16 to 11 us)
    const int tb = (int)std::min<int64_t>(kTokens, (n.rows + slots - 1) / slots);
    const int64_t ctas = tb ? (n.rows + tb - 1) / tb : 0;
    const int64_t grid = ctas + (n.seq_status ? (c.B + kWarps - 1) / kWarps : 0);
    if (grid == 0) return cudaSuccess;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto* f = r.rd % 16 ? rope_kernel<DT, Q8, ODT, false> : rope_kernel<DT, Q8, ODT, true>;
    f<<<(unsigned)grid, kThreads, 0, s>>>(c, n, r, q, parent, lanes_log, tb, ctas);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append_rope(const KvView& c, const KvNew& n, const Rope& r, const RopeRows& q, const int32_t* parent,
                                  cudaStream_t s) {
    if (n.dtype == kKvBf16)
        return c.esz == 1 ? launch<kKvBf16, true, kKvBf16>(c, n, r, q, parent, s) : launch<kKvBf16, false, kKvBf16>(c, n, r, q, parent, s);
    return c.esz == 1 ? launch<kKvF32, true, kKvBf16>(c, n, r, q, parent, s) : launch<kKvF32, false, kKvBf16>(c, n, r, q, parent, s);
}

cudaError_t launch_rope(const Rope& r, const RopeRows& q, int64_t rows, cudaStream_t s) {
    KvView c = {};
    KvNew n = {};
    n.rows = rows;
    if (q.dtype == kKvBf16)
        return q.out_dtype == kKvBf16 ? launch<kKvBf16, false, kKvBf16>(c, n, r, q, nullptr, s)
                                      : launch<kKvBf16, false, kKvF32>(c, n, r, q, nullptr, s);
    return q.out_dtype == kKvBf16 ? launch<kKvF32, false, kKvBf16>(c, n, r, q, nullptr, s)
                                  : launch<kKvF32, false, kKvF32>(c, n, r, q, nullptr, s);
}

}  // namespace specv
