// attend_few.cu -- attention through a sliding window for up to 16 query rows
// to a key-value head (new tokens times query heads): single tokens, short
// drafts.
//
// A CTA takes one (sequence, key-value head), or one of `splits` equal pieces
// of what its tokens see; each of its eight, four or two warps goes through
// every eighth, fourth or second run of 16 positions (32 of e4m3 or of heads up
// to 64) by itself: its own ring in shared memory, filled by asynchronous
// copies, its own running maxima, sums and outputs in registers. Nothing is
// waited for but the warp's own copies, and several CTAs on an SM are at
// different places, so that one's start and end (lengths, pages, the join)
// hide behind the others' loads. The products are warp-wide m16n8k16 matrix
// instructions: scores S = Q K^T with the query rows as the instruction's rows,
// O^T += V^T P^T with the rows as its 8 columns, as S's accumulators are that
// operand as they lie. Windows so long that one CTA's piece would outlast a
// call that is shared out evenly take attend.cuh (attend_few_takes).
//
// Bounds (8 heads of 128, pages of 16; us in a graph). bf16 tokens of 16
// sequences through a window of 4,096: 44 us for 269 MB, 0.90 of the copy
// bandwidth; of 64, 159 us, 1.0. e4m3 tokens of 64 sequences through 1,024:
// 30.5 us for 138 MB, 0.67: latency with few warps to hide it, 1.65 to a
// scheduler that issues in 40 % of cycles (209 registers a thread and 25.7 KB of
// ring a warp leave room for no more; a warp turns codes to f16 between its
// loads and its products). One sequence through 4,096: 8.5 us, latency: launch,
// length, page, run, the warps' join, the pieces'. One or two entries, in 32
// pieces at most, leave SMs empty: one key-value head through 65,536 21 us,
// through 131,072 34 (floors 5 and 10). On the tensor cores' asynchronous path
// (attend.cuh, rows in tiles of 16) these took 62, 197, 73 and 14.6 us: there an
// entry's end waits for the last of its tiles, and a window's entry has few. From
// 17 rows on it is the faster one: rows of 16 to a warp, three warps to a run,
// 9 tokens x 4 query heads of 64 sequences took 115 us, there 74.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "kv.cuh"
#include "sight.cuh"

namespace specv {

namespace {

struct FewParams {
    KvAttend a;
    int64_t ctas;       // entries times splits
    int32_t splits;     // pieces of an entry
    int32_t box_log;    // of the positions that lie together
    int32_t rows_max;   // of an entry
    float* part_o;      // [entry][split][rows_max][DP] sums of the pieces
    float4* part_s;     // [entry][split][rows_max] their maxima, weights' sums and units
    uint32_t* arrive;   // [entry] pieces done, zero between calls
};

constexpr int kMaxWarps = 8;
constexpr int kBoxLog = 4;        // log2 of the most positions that the list keeps together
constexpr int64_t kLeast = 32;    // positions of a warp, at least, where an entry is in pieces
constexpr int64_t kParts = 152;   // most pieces where entries are split: an SM for each
constexpr int64_t kMostRows = 16; // query rows of an entry
constexpr int64_t kLongest = 16384;  // positions of a piece, times bytes of an element
constexpr float kNone = -INFINITY;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {  // not there: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4u : 0u) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {  // a in the low half
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two codes each, the low and the high half of a word, exact as f16.
__device__ __forceinline__ void codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

template <int NR, int DP, bool Q8>
struct Few {
    static constexpr int run = Q8 || DP <= 64 ? 32 : 16;            // positions of a run
    static constexpr int sets = NR / 8;                             // rows 8 at a time
    static constexpr uint32_t row = Q8 ? (DP <= 64 ? 64 : 128) : DP * 2;  // bytes of a position in shared memory
    static constexpr uint32_t half = run * row;                     // K, or V, of a run
    static constexpr uint32_t stage = 2 * half + (Q8 ? 384 : 128);  // and (e4m3) their scales [2][run], which positions are there
    static constexpr int stages = 3;
    static constexpr uint32_t warp_bytes = stages * stage > NR * DP * 4 ? stages * stage : NR * DP * 4;  // and its outputs at the end
    static constexpr uint32_t per_warp = warp_bytes + NR * 16;
    // where a 16-byte unit of a position lies: eight positions' same unit in different banks
    static __device__ __forceinline__ uint32_t at(uint32_t pos, uint32_t unit) {
        return pos * row + (unit ^ (row == 64 ? pos >> 1 & 3 : pos & 7)) * 16;
    }
};

template <int NR, int DP, bool Q8>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) attend_few_kernel(const __grid_constant__ FewParams p) {
    using X = Few<NR, DP, Q8>;
    constexpr int sets = X::sets, kRun = X::run, NT = kRun / 8;
    extern __shared__ __align__(128) unsigned char smem[];
    const KvAttend& a = p.a;
    const KvView& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    if ((int64_t)blockIdx.x >= p.ctas) {
        // ------------------------------------------------------ statuses, a warp for each sequence
        const int64_t b = ((int64_t)blockIdx.x - p.ctas) * warps + warp;
        if (b >= c.B) return;
        const KvSeq s = kv_seq((int32_t)b, a.row_off, a.t_max, a.rows, a.kv_lens, c.bs, c.max_blocks, true);
        int32_t st = s.st;
        if (st == kKvOk && a.parent) {
            bool bad = false;
            for (int32_t v = lane; v < s.T; v += 32) {
                const int32_t u = a.parent[s.lo + v];
                bad |= v == 0 ? u != -1 : (u < 0 || u >= v);
            }
            if (__any_sync(0xFFFFFFFFu, bad)) st = kKvBadLayout;
        }
        if (st != kKvOk && s.lo >= 0) {  // its rows are zeros
            const int64_t m = (int64_t)s.T * a.Hq * c.D, o = s.lo * a.Hq * c.D;
            for (int64_t i = (int64_t)lane * 8; i < m; i += 256) *(uint4*)(a.out + (o + i) * 2) = make_uint4(0, 0, 0, 0);
            if (a.lse)
                for (int64_t i = lane; i < (int64_t)s.T * a.Hq; i += 32) a.lse[s.lo * a.Hq + i] = kNone;
        }
        if (a.seq_status) {
            if (st == kKvOk) st = check_pages(c, (int32_t)b, max(0, s.L - s.T + 1 - a.window), s.T ? s.L : 0);
            if (st == kKvOk) st = check_pages(c, (int32_t)b, 0, s.T ? min(a.sinks, s.L) : 0);
            if (lane == 0) a.seq_status[b] = st;
        }
        return;
    }
    // ---------------------------------------------------------- the CTA's piece
    const int32_t entry = (int32_t)(blockIdx.x / (uint32_t)p.splits), split = (int32_t)(blockIdx.x - (uint32_t)entry * p.splits);
    const int32_t b = c.by_H.of(entry), h = entry - b * c.H;
    const KvSeq s = kv_seq(b, a.row_off, a.t_max, a.rows, a.kv_lens, c.bs, c.max_blocks, true);
    if (s.st != kKvOk || s.T == 0) return;
    const int32_t T = s.T, L = s.L, ctx = L - T, rows = T * a.G;
    // ancestors of token `lane` (itself with them) as bits, and its depth: by doubling
    uint32_t anc = lane < 16 ? 2u << lane : 0u;
    anc = a.parent ? anc >> 1 : anc - 1;
    int32_t depth = lane;
    if (a.parent) {
        int32_t up = lane < T ? a.parent[s.lo + lane] : -1;
        if (__any_sync(0xFFFFFFFFu, lane < T && (lane == 0 ? up != -1 : (up < 0 || up >= lane)))) return;  // (zeros, see above)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t more = __shfl_sync(0xFFFFFFFFu, anc, max(up, 0));
            const int32_t far = __shfl_sync(0xFFFFFFFFu, up, max(up, 0));
            if (up >= 0) anc |= more, up = far;
        }
        depth = __popc(anc) - 1;
    }
    const Sight sight(T, L, a.window, a.sinks, p.box_log);
    const int32_t runs = (sight.end + kRun - 1) / kRun;
    const int32_t run0 = (int32_t)((int64_t)runs * split / p.splits), run1 = (int32_t)((int64_t)runs * (split + 1) / p.splits);
    const int32_t* const table = c.table + (int64_t)b * c.max_blocks;

    // this lane's rows: lane / 4 and (sets = 2) 8 more
    const int j = lane & 3;
    uint32_t q[DP / 16][2 * sets];
    uint32_t see[sets];   // new tokens that the row's token sees, as far as the window lets it
    int32_t deep[sets];   // its depth
    float arow[sets];     // scale * log2(e), times what the row's queries were divided by
    const float k2 = a.scale * kLog2e;
#pragma unroll
    for (int t = 0; t < sets; ++t) {
        const int r = (lane >> 2) + 8 * t, tk = r < rows ? a.by_G.of(r) : 0;
        see[t] = __shfl_sync(0xFFFFFFFFu, anc, tk);
        deep[t] = __shfl_sync(0xFFFFFFFFu, depth, tk);
        const unsigned char* const at = a.q + (s.lo + tk) * a.q_row_bytes + ((int64_t)h * a.G + (r - tk * a.G)) * c.D * 2;
        uint32_t top = 0;  // Q8: magnitudes as integers; what is not finite does not count
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // the instruction's element 2j of this half; e4m3: of 16 in a row, 4 to a lane, as their codes lie
                const int d = k * 16 + (Q8 ? 4 * j + 2 * i : 2 * j + 8 * i);
                const uint32_t w = r < rows && d < c.D ? *(const uint32_t*)(at + d * 2) : 0u;
                q[k][2 * t + i] = w;
                const uint32_t lo = w & 0x7FFFu, hi = w >> 16 & 0x7FFFu;
                top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
        arow[t] = k2;
        if (Q8) {
            // in f16, times a power of two that brings the row's largest element to [2^14, 2^15): all 8 bits of what is 2^-31
            // of it or more
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const int e = top ? max(-126, min(113, (int)(top >> 7) - 127 - 14)) : 0;
            const float f = pow2(-e);
            arow[t] = k2 * pow2(e);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w = q[k][2 * t + i];
                    q[k][2 * t + i] = pack_f16(bf16_lo(w) * f, bf16_hi(w) * f);
                }
        }
    }

    // ---------------------------------------------------------- loads
    unsigned char* const ring = smem + warp * X::warp_bytes;
    const uint32_t ring_at = smem_addr(ring);
    constexpr int chunks = X::row / 16, per = 32 / chunks;  // 16-byte units of a position; positions of one copy instruction
    const int chunk = lane % chunks, sub = lane / chunks;
    const bool inside = chunk * 16 < c.D * c.esz;
    // lane i (and, of 16, i + 16): position i of a run, its page
    auto pos_of = [&](int32_t run) { return sight.at(run * kRun + (lane & (kRun - 1))); };
    auto page_of = [&](int32_t run, int32_t pos) {
        return run < run1 && sight.seen(pos, L, a.sinks) ? table[c.by_bs.of(pos)] : -1;
    };
    auto load = [&](int32_t pos, int32_t pg, int st) {
        const bool there = pg >= 0 && pg < c.num_blocks;
        const int32_t pb = there ? c.by_bs.of(pos) : 0, sl = there ? pos - pb * c.bs : 0;
        const int64_t base = there ? pg * c.block_bytes + sl * c.token_bytes + h * c.head_bytes : -1;
        const uint32_t to = ring_at + st * X::stage;
#pragma unroll
        for (int i = 0; i < kRun / per; ++i) {
            const int row = i * per + sub;
            const int64_t at = __shfl_sync(0xFFFFFFFFu, base, row);
            const bool on = at >= 0 && inside;
            const int64_t off = on ? at + chunk * 16 : 0;
            const uint32_t dst = to + X::at(row, chunk);
            cp16(dst, c.k + off, on);
            cp16(dst + X::half, c.v + off, on);
        }
        if (Q8) {
            const int64_t i = there ? ((int64_t)pg * c.H + h) * c.bs + sl : 0;
            cp4(to + 2 * X::half + lane * 4, c.ks + i, there);
            cp4(to + 2 * X::half + 128 + lane * 4, c.vs + i, there);
        }
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, there);
        if (lane == 0) *(uint32_t*)(ring + st * X::stage + X::stage - 16) = bits;
    };

    float m[sets], l[sets], unit[sets], o[DP / 16][sets][4];
#pragma unroll
    for (int t = 0; t < sets; ++t) {
        m[t] = kNone, l[t] = 0.f, unit[t] = 0x1p115f;  // (Q8: 2^(15 - e), e = -100 before any scale)
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[k][t][i] = 0.f;
    }
    // ---------------------------------------------------------- the runs
    constexpr int S = X::stages;
    int32_t next = run0 + warp, next_pos = pos_of(next), next_pg = page_of(next, next_pos);
    auto fetch = [&](int st) {
        const int32_t pos = next_pos, pg = next_pg;
        const bool any = next < run1;
        next += warps;
        next_pos = pos_of(next);
        next_pg = page_of(next, next_pos);
        if (any) load(pos, pg, st);
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
    auto one = [&](int32_t run, int st) {
        fetch((st + S - 1) % S);
        cp_wait<S - 1>();
        __syncwarp();
        const uint32_t k_at = ring_at + st * X::stage, v_at = k_at + X::half;
        const float* const scales = (const float*)(ring + st * X::stage + 2 * X::half);
        const uint32_t live = *(const uint32_t*)(ring + st * X::stage + X::stage - 16);
        const int32_t place0 = run * kRun;
        constexpr uint32_t every = kRun == 32 ? ~0u : (1u << (kRun & 31)) - 1;
        const bool masked = (live & every) != every || (T > 1 && place0 + kRun > sight.tail);
        // ---- scores: rows lane / 4 (+ 8), positions 8n + 2j, + 1
        float x[NT][4] = {};
#pragma unroll
        for (int k = 0; k < DP / 16; k += Q8 ? 4 : 2)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t w[4];  // 8 positions by 4 units of 16 bytes
                ldsm(k_at + X::at(n * 8 + (lane & 7), (Q8 ? k : 2 * k) + (lane >> 3)), w);
#pragma unroll
                for (int i = 0; i < (Q8 ? 4 : 2); ++i) {
                    uint32_t b0 = w[(2 * i) & 3], b1 = w[(2 * i + 1) & 3];
                    if (Q8) codes(w[i], b0, b1);
                    mma<Q8>(x[n], q[k + i][0], sets > 1 ? q[k + i][sets > 1 ? 2 : 0] : 0u, q[k + i][1],
                            sets > 1 ? q[k + i][sets > 1 ? 3 : 1] : 0u, b0, b1);
                }
            }
        float2 vs[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float2 ks = make_float2(1.f, 1.f);
            if (Q8) {
                ks = *(const float2*)(scales + n * 8 + 2 * j);
                vs[n] = *(const float2*)(scales + 32 + n * 8 + 2 * j);
            }
#pragma unroll
            for (int t = 0; t < sets; ++t) {
                x[n][2 * t] *= Q8 ? arow[t] * ks.x : k2;
                x[n][2 * t + 1] *= Q8 ? arow[t] * ks.y : k2;
            }
        }
        uint32_t vis[sets];  // of the row's positions, this lane's: bit 8n + 2j + i
        if (masked) {
#pragma unroll
            for (int t = 0; t < sets; ++t) vis[t] = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = n * 8 + 2 * j + i;
                    const int32_t pos = sight.at(place0 + at), u = pos - ctx;
                    const int32_t du = __shfl_sync(0xFFFFFFFFu, depth, u & 31);
#pragma unroll
                    for (int t = 0; t < sets; ++t) {
                        const bool near = pos < a.sinks || deep[t] - (u >= 0 ? du : u) < a.window;
                        const bool on = (live >> at & 1) && near && (u < 0 || (see[t] >> (u & 31) & 1));
                        vis[t] |= (uint32_t)on << at;
                        x[n][2 * t + i] = on ? x[n][2 * t + i] : kNone;
                    }
                }
        }
        // ---- the rows' maxima, and (Q8) the units by the scales they see
        float f[sets], fo[sets];
        bool change = false;
#pragma unroll
        for (int t = 0; t < sets; ++t) {
            float top = kNone;
#pragma unroll
            for (int n = 0; n < NT; ++n) top = max3(top, x[n][2 * t], x[n][2 * t + 1]);
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const float mn = fmaxf(m[t], top);
            f[t] = mn == kNone ? 1.f : ex2(m[t] - mn);
            change |= mn != m[t];
            m[t] = mn;
            fo[t] = f[t];
            if (Q8) {
                // the largest scale's magnitude, as an integer; of the smallest power of two not below it the exponent as it
                // is held, 0 to 253 (no scale, 2^126 or more)
                uint32_t w = 0;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t lo = __float_as_uint(vs[n].x) & 0x7FFFFFFFu, hi = __float_as_uint(vs[n].y) & 0x7FFFFFFFu;
                    w = max(w, !masked || (vis[t] >> (n * 8 + 2 * j) & 1) ? lo : 0u);
                    w = max(w, !masked || (vis[t] >> (n * 8 + 2 * j + 1) & 1) ? hi : 0u);
                }
                w = max(w, __shfl_xor_sync(0xFFFFFFFFu, w, 1));
                w = max(w, __shfl_xor_sync(0xFFFFFFFFu, w, 2));
                const uint32_t e = min(253u, (w + 0x7FFFFFu) >> 23);
                // the unit is 2^(15 - e), held as 127 + 15 - (e - 127)
                const uint32_t was = 269 - (__float_as_uint(unit[t]) >> 23), now = max(was, max(e, 16u));
                unit[t] = __uint_as_float((269 - now) << 23);
                fo[t] *= now - was > 126 ? 0.f : __uint_as_float((127 - (now - was)) << 23);
                change |= now != was;
            }
        }
        if (__any_sync(0xFFFFFFFFu, change)) {
#pragma unroll
            for (int t = 0; t < sets; ++t) {
                l[t] *= f[t];
                // the outputs' rows are 2j and 2j + 1
                const float f0 = __shfl_sync(0xFFFFFFFFu, fo[t], 8 * j), f1 = __shfl_sync(0xFFFFFFFFu, fo[t], 8 * j + 4);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    o[k][t][0] *= f0, o[k][t][1] *= f1;
                    o[k][t][2] *= f0, o[k][t][3] *= f1;
                }
            }
        }
        // ---- weights: the second product's operand as they lie
        uint32_t w0[sets][NT], w1[sets][NT];  // bf16: two parts, 16 bits of a weight; e4m3: f16, times V's scale and the unit
#pragma unroll
        for (int t = 0; t < sets; ++t) {
            const float mr = m[t] == kNone ? 0.f : m[t];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[i] = ex2(x[n][2 * t + i] - mr);
                    l[t] += w[i];
                    if (Q8) {
                        w[i] *= (i ? vs[n].y : vs[n].x) * unit[t];
                        if (masked) w[i] = vis[t] >> (n * 8 + 2 * j + i) & 1 ? w[i] : 0.f;
                    }
                }
                if (Q8) {
                    w0[t][n] = pack_f16(w[0], w[1]);
                } else {
                    w0[t][n] = pack_bf16(w[0], w[1]);
                    w1[t][n] = pack_bf16(w[0] - bf16_lo(w0[t][n]), w[1] - bf16_hi(w0[t][n]));
                }
            }
        }
        // ---- O^T += V^T P^T
        // V's operands of 16 elements of the head each, `step` at a time: lanes hold pairs of positions of an element
        constexpr int step = Q8 ? 2 : 1;
        auto values = [&](int part, int k, uint32_t (&v)[step][4]) {  // of positions 16 part ..
            uint32_t w[4];
            if constexpr (Q8) {
                // pairs of codes, of positions 0 .. 7 and 8 .. 15, of this 16 elements and the next
                ldsm_t(v_at + X::at(16 * part + (lane & 15), k + (lane >> 4)), w);
#pragma unroll
                for (int i = 0; i < 4; ++i)  // an element's two positions side by side
                    codes(__byte_perm(w[i], 0, 0x3120), v[i >> 1][2 * (i & 1)], v[i >> 1][2 * (i & 1) + 1]);
            } else {
                ldsm_t(v_at + X::at(16 * part + (lane & 7) + (lane & 16 ? 8 : 0), 2 * k + (lane >> 3 & 1)), v[0]);
            }
        };
        // A value that is not finite, at a position that some rows see and others do not, would reach those too (0 * inf).
        bool poison = false;
        if (masked && T > 1) {
            constexpr uint32_t ex = Q8 ? 0 : 0x7F80u;
            bool found = false;
#pragma unroll 1
            for (uint32_t i = lane * 16; i < X::half; i += 512) {
                const uint4 y = *(const uint4*)(ring + st * X::stage + X::half + i);
                const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (Q8)
                        found |= __vcmpeq4(u[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
                    else
                        found |= (u[k] & ex) == ex || (u[k] >> 16 & ex) == ex;
                }
            }
            poison = __any_sync(0xFFFFFFFFu, found);
        }
        if (!poison) {
#pragma unroll
            for (int part = 0; part < NT / 2; ++part)
#pragma unroll
                for (int k = 0; k < DP / 16; k += step) {
                    uint32_t v[step][4];
                    values(part, k, v);
#pragma unroll
                    for (int i = 0; i < step; ++i)
#pragma unroll
                        for (int t = 0; t < sets; ++t) {
                            mma<Q8>(o[k + i][t], v[i][0], v[i][1], v[i][2], v[i][3], w0[t][2 * part], w0[t][2 * part + 1]);
                            if (!Q8)
                                mma<Q8>(o[k + i][t], v[i][0], v[i][1], v[i][2], v[i][3], w1[t][2 * part], w1[t][2 * part + 1]);
                        }
                }
        } else {
            // a row at a time, from the values it sees
#pragma unroll
            for (int t = 0; t < sets; ++t) {
                uint32_t of_row = vis[t];
                of_row |= __shfl_xor_sync(0xFFFFFFFFu, of_row, 1);
                of_row |= __shfl_xor_sync(0xFFFFFFFFu, of_row, 2);
#pragma unroll 1
                for (int r = 0; r < 8; ++r) {
                    const uint32_t on = __shfl_sync(0xFFFFFFFFu, of_row, 4 * r);
#pragma unroll
                    for (int part = 0; part < NT / 2; ++part) {
                        auto both = [&](int at) { return (on >> at & 1 ? 0xFFFFu : 0u) | (on >> (at + 1) & 1 ? 0xFFFF0000u : 0u); };
                        const uint32_t lo = both(16 * part + 2 * j), hi = both(16 * part + 8 + 2 * j);
#pragma unroll
                        for (int k = 0; k < DP / 16; k += step) {
                            uint32_t v[step][4];
                            values(part, k, v);
#pragma unroll
                            for (int i = 0; i < step; ++i) {
                                float y[4] = {0.f, 0.f, 0.f, 0.f};
                                mma<Q8>(y, v[i][0] & lo, v[i][1] & lo, v[i][2] & hi, v[i][3] & hi, w0[t][2 * part], w0[t][2 * part + 1]);
                                if (!Q8)
                                    mma<Q8>(y, v[i][0] & lo, v[i][1] & lo, v[i][2] & hi, v[i][3] & hi, w1[t][2 * part], w1[t][2 * part + 1]);
                                const bool even = r == 2 * j, odd = r == 2 * j + 1;
                                if (even) o[k + i][t][0] += y[0], o[k + i][t][2] += y[2];
                                if (odd) o[k + i][t][1] += y[1], o[k + i][t][3] += y[3];
                            }
                        }
                    }
                }
            }
        }
        __syncwarp();  // its place is the next load's
    };
    int st = 0;
#pragma unroll 1
    for (int32_t run = run0 + warp; run < run1; run += warps) {
        one(run, st);
        st = st + 1 == S ? 0 : st + 1;
    }
    cp_wait<0>();
    __syncwarp();
    // ---------------------------------------------------------- the warps' sums
    float4* const sums = (float4*)(smem + warps * X::warp_bytes);  // [warps][NR] maximum (log2), weights' sum, unit
    float* const mine = (float*)ring;                               // [NR][DP]
#pragma unroll
    for (int t = 0; t < sets; ++t) {
        l[t] += __shfl_xor_sync(0xFFFFFFFFu, l[t], 1);
        l[t] += __shfl_xor_sync(0xFFFFFFFFu, l[t], 2);
        if (j == 0) sums[warp * NR + (lane >> 2) + 8 * t] = make_float4(m[t], l[t], Q8 ? unit[t] : 1.f, 0.f);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 2 * j + (i & 1) + 8 * t;
                // the instruction's rows: elements lane / 4 and 8 more; e4m3: pairs as their codes lie
                const int d = k * 16 + (Q8 ? 2 * (lane >> 2) + (i >> 1) : (lane >> 2) + 8 * (i >> 1));
                mine[r * DP + d] = o[k][t][i];
            }
    }
    __syncthreads();
    // Joins n parts (32 at most), a row to a warp, in their order: lane w has part w's statistics, then each lane DP / 32
    // elements of the outputs.
    constexpr int E = DP / 32, kAtOnce = 16;
    auto join = [&](int n, int r, auto&& stats, auto&& values, bool all, float4* to_s, float* to_o) {
        const float4 y = lane < n ? stats(lane, r) : make_float4(kNone, 0.f, 0x1p115f, 0.f);
        float M = y.x, U = y.z;
#pragma unroll
        for (int i = 16; i; i >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, i));
            U = fminf(U, __shfl_xor_sync(0xFFFFFFFFu, U, i));
        }
        // (a part whose scores are all NaN has no maximum, and a sum that is NaN)
        const float f = y.x != kNone ? ex2(y.x - M) : y.y == 0.f ? 0.f : 1.f;
        float sum = f * y.y;
#pragma unroll
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
        const float g = f * (U / y.z);  // (units are powers of two)
        float x[E] = {};
#pragma unroll 1
        for (int w0 = 0; w0 < n; w0 += kAtOnce) {
            float z[kAtOnce][E];
#pragma unroll
            for (int w = 0; w < kAtOnce; ++w) values(min(w0 + w, n - 1), r, z[w]);
#pragma unroll
            for (int w = 0; w < kAtOnce; ++w) {
                const float gw = __shfl_sync(0xFFFFFFFFu, g, min(w0 + w, n - 1));
                if (w0 + w >= n) continue;
#pragma unroll
                for (int i = 0; i < E; ++i) x[i] = fmaf(gw, z[w][i], x[i]);
            }
        }
        if (!all) {
#pragma unroll
            for (int i = 0; i < E; ++i) to_o[(int64_t)r * DP + lane * E + i] = x[i];
            if (lane == 0) to_s[r] = make_float4(M, sum, U, 0.f);
            return;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum, down = 1.f / U;
        const int32_t tk = a.by_G.of(r);
        const int64_t row = (s.lo + tk) * a.Hq + (int64_t)h * a.G + (r - tk * a.G);
        if (lane * E < c.D) {
#pragma unroll
            for (int i = 0; i < E; i += 2)
                *(uint32_t*)(a.out + (row * c.D + lane * E + i) * 2) =
                    sum == 0.f ? 0u : pack_bf16(x[i] * inv * down, x[i + 1] * inv * down);
        }
        if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? kNone : (M + log2f(sum)) * 0.69314718055994531f;
    };
    const int64_t part0 = (int64_t)entry * p.splits;
    float4* const to_s = p.part_s + (part0 + split) * p.rows_max;
    float* const to_o = p.part_o + (part0 + split) * p.rows_max * DP;
#pragma unroll 1
    for (int r = warp; r < rows; r += warps)
        join(warps, r, [&](int w, int r) { return sums[w * NR + r]; },
             [&](int w, int r, float (&z)[E]) {
#pragma unroll
                 for (int i = 0; i < E; ++i) z[i] = ((const float*)(smem + w * X::warp_bytes))[r * DP + lane * E + i];
             },
             p.splits == 1, to_s, to_o);
    if (p.splits == 1) return;
    // ---------------------------------------------------------- the pieces', by whoever comes last
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        last = atomicAdd(p.arrive + entry, 1u) == (uint32_t)p.splits - 1;
        if (last) p.arrive[entry] = 0;  // for the next call
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
#pragma unroll 1
    for (int r = warp; r < rows; r += warps)
        join(p.splits, r, [&](int w, int r) { return __ldcg(p.part_s + (part0 + w) * p.rows_max + r); },
             [&](int w, int r, float (&z)[E]) {
                 const float* const at = p.part_o + ((part0 + w) * p.rows_max + r) * DP + lane * E;
                 if constexpr (E == 4)
                     *(float4*)z = __ldcg((const float4*)at);
                 else
                     *(float2*)z = __ldcg((const float2*)at);
             },
             true, nullptr, nullptr);
}

template <int NR, int DP, bool Q8>
cudaError_t launch(const FewParams& p, int warps, cudaStream_t s) {
    using X = Few<NR, DP, Q8>;
    auto* f = attend_few_kernel<NR, DP, Q8>;
    static std::atomic<uint64_t> known{0};  // devices on which the kernel may use that much shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(known.load() & bit) || dev >= 64) {
        if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kMaxWarps * X::per_warp))) != cudaSuccess) return e;
        known.fetch_or(bit);
    }
    const int64_t grid = p.ctas + (p.a.c.B + warps - 1) / warps;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    f<<<(unsigned)grid, warps * 32, warps * X::per_warp, s>>>(p);
    return cudaGetLastError();
}

template <int NR, bool Q8>
cudaError_t launch_dim(const FewParams& p, int warps, cudaStream_t s) {
    return p.a.c.D <= 64 ? launch<NR, 64, Q8>(p, warps, s) : launch<NR, 128, Q8>(p, warps, s);
}

struct Plan {
    int64_t rows, entries, most;  // most: positions that an entry's tokens may see
    int warps;                    // of a CTA
    int64_t splits;
    explicit Plan(const KvAttend& a) : rows((int64_t)a.t_max * a.G), entries((int64_t)a.c.B * a.c.H) {
        // Warps to an entry: with fewer a CTA starts and ends for more positions, but the CTAs of a call should be on the 152
        // SMs at once (rings of 1 x 8, 2 x 4 or 4 x 2 warps fit). One e4m3 token through 1,024 positions, us with 8, 4 and 2
        // warps: of 16 sequences (128 entries) 11.8, 13.9, 16; of 32 22, 17, 22; of 64 46, 36, 31; of 96 66, 52, 57.
        // Pieces only where an entry's warps leave SMs empty, and none shorter than kLeast positions for each warp where the
        // window is full (one sequence through 4,096: 32 positions 8.8 us, 64 10.4).
        most = std::min<int64_t>((int64_t)a.c.max_blocks * a.c.bs, (int64_t)a.window + a.t_max + a.sinks + 16);
        warps = entries <= 152 ? 8 : entries <= 304 ? 4 : entries <= 608 ? 2 : 4;
        splits = std::max<int64_t>(1, std::min<int64_t>({kParts / entries, 32, most / (warps * kLeast)}));
    }
};

}  // namespace

bool attend_few_takes(const KvAttend& a) {
    if (a.c.D > 128 || (int64_t)a.t_max * a.G > kMostRows) return false;
    // A piece is one CTA's, however much shorter the others are, and the host does not know the lengths; attend.cuh shares
    // all tiles out evenly. One token of 20 sequences x 8 heads through 16,384 positions, us here and there, bf16: all that
    // long 216 and 214, lengths up to it 186 and 120, one of them that long and the rest 256 183 and 30. Of 64 sequences
    // through 8,192: 309 and 331, 229 and 197, 184 and 43. e4m3, where a piece of as many bytes is twice as long, 64 through
    // 16,384: 344 and 559, 335 and 320, 245 and 49; through 8,192: 177 and 297, 180 and 196, 127 and 44. So the limit is where
    // lengths that differ a little are even; a single long one below it costs up to five times (e4m3 six) what it would there.
    const Plan plan(a);
    return plan.most * a.c.esz <= kLongest * plan.splits;
}

size_t attend_few_workspace(int64_t rows) {
    return rows > kMostRows ? 0 : kHeaderBytes + ((size_t)kParts * rows * (128 * 4 + 16) + 255) / 256 * 256;
}

cudaError_t launch_attend_few(const KvAttend& a, void* workspace, cudaStream_t s) {
    const Plan plan(a);
    const int64_t rows = plan.rows;
    const int warps = plan.warps;
    FewParams p;
    p.a = a;
    p.splits = (int32_t)plan.splits;
    p.ctas = plan.entries * plan.splits;
    p.rows_max = (int32_t)rows;
    p.box_log = 0;
    while (p.box_log < kBoxLog && a.c.bs % (2 << p.box_log) == 0) ++p.box_log;
    char* const ws = (char*)workspace;
    p.arrive = (uint32_t*)ws;
    p.part_s = (float4*)(ws + kHeaderBytes);
    p.part_o = (float*)(p.part_s + kParts * rows);
    const bool q8 = a.c.esz == 1;
    if (rows <= 8) return q8 ? launch_dim<8, true>(p, warps, s) : launch_dim<8, false>(p, warps, s);
    return q8 ? launch_dim<16, true>(p, warps, s) : launch_dim<16, false>(p, warps, s);
}

}  // namespace specv
