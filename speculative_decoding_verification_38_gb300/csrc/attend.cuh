// attend.cuh -- attention of each sequence's new tokens over the paged cache on
// the tensor cores.
//
// The products run transposed: with the 128 positions of a tile as the rows of
// the matrix instruction, S^T = K Q^T [128 x N] and O^T += V^T P^T [head_dim x
// N], N being the query rows (new tokens times the query heads of a key-value
// head). So the long side fills the instruction whatever the number of query
// rows, one token to a whole tree, and work grows with N only.
//
// The flat list of tiles over (sequence, head, row tile) is cut into one equal
// run for each CTA (one CTA on each SM). A CTA that holds a whole (sequence,
// head, row tile) writes its rows; one that holds a part leaves its sums in the
// workspace, and the last CTA of that list entry to arrive joins the parts in
// their order.
#pragma once

#include "internal.h"
#include "kv.cuh"

namespace specv {

struct AttParams {
    KvAttend a;
    float* part_o;     // [grid * 2][N][128] partial sums
    float2* part_ml;   // [grid * 2][N] their maxima (log2) and weights' sums
    uint32_t* arrive;  // [grid] parts arrived, zero between calls
    uint32_t* err;
    int32_t grid;
};

// Attention with row tiles of n query rows (16, 32, 48, 80 or 128).
cudaError_t attend_bf16(int n, const AttParams& p, cudaStream_t s);
cudaError_t attend_bf16_wide(int n, const AttParams& p, cudaStream_t s);
cudaError_t attend_e4m3(int n, const AttParams& p, cudaStream_t s);
cudaError_t attend_e4m3_wide(int n, const AttParams& p, cudaStream_t s);

constexpr int kAttMaxGrid = 160;  // CTAs (the workspace holds two parts for each)

namespace {

constexpr int kTileTok = 128;   // positions of a tile
constexpr int kGroups = 4;      // softmax groups of four warps; a group takes every fourth 8 query rows
constexpr int kSoftWarps = 4 * kGroups;
constexpr int kFeedWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kFeedWarps;
constexpr int kSegWarp = kMmaWarp + 1;
constexpr int kStatusWarp = kSegWarp + 1;
constexpr int kAttThreads = (kStatusWarp + 2) * 32;  // whole groups of four warps
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMaxSlots = 3;                  // tiles of the K ring, and of the V ring
constexpr int kAuxRing = 8;                   // tiles of masks and scales kept: more than the ring and S can hold
constexpr uint64_t kAttWaitNs = 2000000000;   // a wait that gives up marks the call, which then runs out unwaited
constexpr float kNoMax = -1.0e30f;            // running maximum before any score
constexpr float kGrow = 8.f;                  // a maximum may rise by 2^8 before the sums are rescaled
constexpr size_t kSmemMax = 232448;

// ------------------------------------------------------------ instructions
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void tc_ld8(uint32_t at, float (&x)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st8(uint32_t at, const float (&x)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
                 "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])),
                 "r"(__float_as_uint(x[3])), "r"(__float_as_uint(x[4])), "r"(__float_as_uint(x[5])),
                 "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7]))
                 : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// This group of four warps goes on with R registers a thread.
template <int R>
__device__ __forceinline__ void more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ uint64_t nanoseconds() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int n, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(n), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t dst, uint4 w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {  // a in the low half
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t two) {  // the low 16 bits: two codes
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// Shared-memory operand descriptor: start, leading and stride byte offsets,
// swizzle (0 none, 2 128-byte).
__device__ __forceinline__ uint64_t operand(uint32_t start, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
    return (uint64_t)((start >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | (uint64_t)1 << 46 | (uint64_t)swizzle << 61;
}
// Instruction descriptor: float32 accumulators, A and B both f16 or bf16,
// 128 rows, n columns, operands with their rows or columns contiguous.
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, bool a_mn, bool b_mn, int n) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// A run of tiles of one (sequence, head, row tile).
struct __align__(16) Seg {
    int32_t b, h, rt, tile0, n;  // n tiles from tile0; n = 0: no more
    int32_t tiles;               // of the whole entry
    int32_t T, L;                // new tokens, length
    int64_t first;  // the entry's first tile in the flat list
    int64_t lo;     // the sequence's first query row
};

// ------------------------------------------------------------------ layout
template <int NN, int DP, bool Q8>
struct Shape {
    static constexpr int N = NN;                           // query rows of a row tile
    static constexpr int MC = (N / 8 + kGroups - 1) / kGroups;  // 8-row pieces of a softmax group
    static constexpr int NP = Q8 ? N : 2 * N;              // P's columns: one f16, or two bf16 parts
    static constexpr uint32_t slot_bytes = kTileTok * DP * 2;
    static constexpr uint32_t q_bytes = N * DP * 2;
    static constexpr uint32_t p_bytes = NP * kTileTok * 2;
    static constexpr uint32_t aux_bytes = Q8 ? 1024 + 16 : 16;  // scales of K and V, validity bits
    static constexpr int segs = !Q8 && N == 128 && DP == 128 ? 2 : 4;  // segments known ahead
    static constexpr uint32_t red_bytes = 5 * MC * 8 * 4 + 16;  // a group's scratch
    // after the slots, Q and P: aux ring, running maxima, row factors, ancestors, segments, poison, barriers
    static constexpr uint32_t misc = kAuxRing * aux_bytes + N * 4 + (Q8 ? N * 4 + kGroups * red_bytes : 0) +
                                     kKvMaxQueries * 16 + segs * sizeof(Seg) + 32 +
                                     (4 * kMaxSlots + 8 + kAuxRing + 2 * segs) * 8;
    static constexpr int fit = (int)((kSmemMax - q_bytes - p_bytes - misc) / (2 * slot_bytes));
    static constexpr int slots = fit > kMaxSlots ? kMaxSlots : fit;
    static constexpr uint32_t total = 2 * slots * slot_bytes + q_bytes + p_bytes + misc;
    static constexpr int lag = slots - 1;  // tiles whose copies are in flight when one is handed over
    static_assert(slots >= 2, "a ring needs two tiles");
    // the feed may wait for a new segment with `lag` tiles, each a segment, not handed over
    static_assert(segs > lag, "the oldest known segment must be whole in the ring");
};

template <int N>
struct Walk {
    const KvAttend& a;
    int64_t u, u1, base, units;
    int32_t b;
    KvSeq s;
    int32_t tiles, nrt;

    __device__ __forceinline__ static int64_t count(const KvAttend& a, int32_t b, KvSeq& s, int32_t& tiles,
                                                    int32_t& nrt) {
        s = kv_seq(b, a.row_off, a.t_max, a.rows, a.kv_lens, a.c.bs, a.c.max_blocks, true);
        if (s.st != kKvOk || s.T == 0) return 0;
        tiles = (s.L + kTileTok - 1) / kTileTok;
        nrt = (s.T * a.G + N - 1) / N;
        return (int64_t)tiles * nrt * a.c.H;
    }
    __device__ __forceinline__ Walk(const KvAttend& a_, int64_t u0, int64_t u1_, int32_t b0, int64_t base0)
        : a(a_), u(u0), u1(u1_), base(base0), b(b0) {
        units = u < u1 ? count(a, b, s, tiles, nrt) : 0;
    }
    __device__ __forceinline__ void next(Seg& g) {
        g.n = 0;
        if (u >= u1) return;
        while (u >= base + units) {
            base += units;
            if (++b >= a.c.B) return;  // lengths that change under the call
            units = count(a, b, s, tiles, nrt);
        }
        const int64_t rem = u - base;
        const int64_t e = rem / tiles;
        g.tile0 = (int32_t)(rem - e * tiles);
        g.n = (int32_t)min((int64_t)(tiles - g.tile0), u1 - u);
        g.h = (int32_t)(e / nrt);
        g.rt = (int32_t)(e - (int64_t)g.h * nrt);
        g.first = u - g.tile0;
        g.tiles = tiles;
        g.b = b;
        g.lo = s.lo;
        g.T = s.T;
        g.L = s.L;
        u += g.n;
    }
};

template <int NN, int DP, bool Q8>
__global__ void __launch_bounds__(kAttThreads, 1) attend_kernel(const __grid_constant__ AttParams p) {
    using X = Shape<NN, DP, Q8>;
    constexpr int N = X::N, S = X::slots, MC = X::MC, R = X::segs;
    constexpr uint32_t kLag = X::lag;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const q_sm = smem + 2 * S * X::slot_bytes;
    unsigned char* const p_sm = q_sm + X::q_bytes;
    unsigned char* const aux_sm = p_sm + X::p_bytes;
    float* const mref = (float*)(aux_sm + kAuxRing * X::aux_bytes);
    float* const arow = mref + N;  // Q8: a query row's power of two times scale * log2(e)
    unsigned char* const red_sm = (unsigned char*)(mref + (Q8 ? 2 * N : N));
    uint32_t* const anc = (uint32_t*)(red_sm + (Q8 ? kGroups * X::red_bytes : 0));  // [T][4] ancestors of a tree's tokens
    Seg* const segs = (Seg*)(anc + kKvMaxQueries * 4);
    uint32_t* const poison = (uint32_t*)(segs + R);  // [4] new tokens with non-finite values, then 4 words:
    volatile uint32_t* const aborted = poison + 4;   // a wait gave up
    uint32_t* const tmem_at = poison + 5;
    uint32_t* const last_in = poison + 6;
    uint32_t* const tree_bad = poison + 7;
    uint64_t* const full = (uint64_t*)(poison + 8);  // [2][S]: the K ring, the V ring
    uint64_t* const empty = full + 2 * S;
    uint64_t* const s_full = empty + 2 * S;
    uint64_t* const s_empty = s_full + 2;
    uint64_t* const p_full = s_empty + 2;
    uint64_t* const pv_done = p_full + 1;
    uint64_t* const q_full = pv_done + 1;
    uint64_t* const drain = q_full + 1;
    uint64_t* const aux_full = drain + 1;
    uint64_t* const seg_full = aux_full + kAuxRing;
    uint64_t* const seg_empty = seg_full + R;

    const KvAttend& a = p.a;
    const KvView& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return;
        const uint64_t t0 = nanoseconds();
        do {
            for (int i = 0; i < 16; ++i)
                if (mbar_try_wait(bar, parity)) return;
            if (*aborted) return;
        } while (nanoseconds() - t0 < kAttWaitNs);
        *aborted = 1;
    };
    // Segment s of this CTA, by every warp that works on it; next_seg gives its place back.
    auto get_seg = [&](uint32_t s) {
        wait(seg_full + s % R, (s / R) & 1);
        return segs + s % R;
    };
    auto done_seg = [&](uint32_t s) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + s % R);
    };

    // ------------------------------------------------- this CTA's run of tiles
    if (tid == 0) {
        for (int i = 0; i < 2 * S; ++i) {
            mbar_init(full + i, kFeedWarps / 2);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, kSoftWarps);
        }
        mbar_init(p_full, kSoftWarps);
        mbar_init(pv_done, 1);
        mbar_init(q_full, kSoftWarps);
        mbar_init(drain, 1);
        for (int i = 0; i < kAuxRing; ++i) mbar_init(aux_full + i, kFeedWarps / 2);
        for (int i = 0; i < R; ++i) {
            mbar_init(seg_full + i, 1);
            mbar_init(seg_empty + i, kSoftWarps + kFeedWarps + 1);
        }
        *aborted = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_at)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    int64_t* const scan = (int64_t*)p_sm;  // P is not in use yet: [32] warp sums, start of the run
    const int32_t per_thr = (c.B + kAttThreads - 1) / kAttThreads;
    const int32_t bt0 = min(c.B, tid * per_thr), bt1 = min(c.B, bt0 + per_thr);
    int64_t mine = 0;
    for (int32_t b = bt0; b < bt1; ++b) {
        KvSeq s;
        int32_t tiles, nrt;
        mine += Walk<N>::count(a, b, s, tiles, nrt);
    }
    int64_t incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t before = 0, W = 0;
    for (int w = 0; w < kAttThreads / 32; ++w) {
        const int64_t x = scan[w];
        before += w < warp ? x : 0;
        W += x;
    }
    const int64_t pre = before + incl - mine;
    const int64_t per = (W + p.grid - 1) / p.grid;
    const int64_t u0 = (int64_t)blockIdx.x * per, u1 = min(u0 + per, W);
    if (u0 < u1 && pre <= u0 && u0 < pre + mine) {
        int64_t at = pre;
        for (int32_t b = bt0; b < bt1; ++b) {
            KvSeq s;
            int32_t tiles, nrt;
            const int64_t k = Walk<N>::count(a, b, s, tiles, nrt);
            if (u0 < at + k) {
                scan[32] = b;
                scan[33] = at;
                break;
            }
            at += k;
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    const int32_t b0 = u0 < u1 ? (int32_t)scan[32] : 0;
    const int64_t base0 = u0 < u1 ? scan[33] : 0;
    const uint32_t tmem = *tmem_at;
    __syncthreads();  // P's memory is P's from here on

    // The block starts with 72 registers a thread, 7 groups of four warps. bf16: softmax 88 (4 groups), feed 48 (2),
    // the rest 56 (1); e4m3: 72, 80 and 56. Either adds up to 7 x 72.
    if (warp >= kSoftWarps && warp < kMmaWarp) {
        if constexpr (Q8)
            more_regs<80>();
        else
            fewer_regs<48>();
        // ============================================================ feed
        // Four warps bring the K tiles, four the V tiles, 32 rows each (lane =
        // row where an address is made). A bf16 tile goes straight to shared
        // memory (cp.async); an e4m3 tile passes the registers, where it becomes
        // f16 (exactly), its lines asked into L2 a tile ahead. Rows past the
        // length, on a page outside the pool or past head_dim are zeros.
        const bool is_k = warp < kSoftWarps + 4;
        const int fw = warp & 3;
        const unsigned char* const src = is_k ? c.k : c.v;
        const uint32_t ring = smem_addr(smem) + (is_k ? 0 : S * X::slot_bytes) + fw * 32 * 128;
        uint64_t* const my_full = full + (is_k ? 0 : S);
        uint64_t* const my_empty = empty + (is_k ? 0 : S);
        constexpr int chunks = DP * (Q8 ? 1 : 2) / 16;  // 16-byte pieces of a padded row
        const int my_chunk = lane % chunks, my_row = lane / chunks;
        const bool chunk_in = my_chunk * (Q8 ? 16 : 8) < c.D;
        uint32_t kt = 0;
        constexpr int rpr = 32 / chunks;  // rows of one load of the warp
        // Where this lane writes its piece of row `my_row + r * rpr` (r constant): the swizzle exchanges 16-byte
        // units within a row by its row's number, so the address is an exclusive or and an offset away from row my_row's.
        const int unit = my_chunk * (Q8 ? 2 : 1);  // of eight 16-bit elements
        const uint32_t at0 = ring + (unit >> 3) * (kTileTok * 128) + my_row * 128 + ((unit ^ my_row) & 7) * 16;
        auto swizzled = [&](uint32_t base, int r, int more) { return (base ^ ((((r * rpr) & 7) ^ more) * 16)) + r * rpr * 128; };
        for (uint32_t si = 0;; ++si) {
            const Seg* const g = get_seg(si);
            const int n = g->n;
            if (!n) break;
            const int32_t L = g->L;
            int32_t pos = g->tile0 * kTileTok + fw * 32 + lane;
            const int32_t* const table = c.table + (int64_t)g->b * c.max_blocks;
            const int64_t head = g->h * c.head_bytes, sc_head = (int64_t)g->h * c.bs;
            done_seg(si);
            // byte offset of the row at position pos (-1: no row), and its scales'
            int64_t sc_next = 0;
            auto row_at = [&]() {
                int64_t o = -1;
                if (pos < L) {
                    const int32_t pg = table[pos / c.bs];
                    const int32_t sl = pos % c.bs;
                    if (pg >= 0 && pg < c.num_blocks) {
                        o = pg * c.block_bytes + sl * c.token_bytes + head;
                        if (Q8) {
                            sc_next = (int64_t)pg * c.H * c.bs + sl + sc_head;
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(src + o));
                            if (is_k) {
                                asm volatile("prefetch.global.L2 [%0];" ::"l"(c.ks + sc_next));
                                asm volatile("prefetch.global.L2 [%0];" ::"l"(c.vs + sc_next));
                            }
                        }
                    }
                }
                return o;
            };
            int64_t next = row_at();
            if constexpr (!Q8) {
                for (int t = 0; t < n; ++t, ++kt) {
                    const int64_t off = next;
                    pos += kTileTok;
                    next = t + 1 < n ? row_at() : -1;
                    const uint32_t slot = kt % S, use = kt / S;
                    if (use) wait(my_empty + slot, (use - 1) & 1);
                    if (is_k) {
                        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, off >= 0);
                        if (lane == 0) {
                            ((uint32_t*)(aux_sm + (kt % kAuxRing) * X::aux_bytes))[fw] = bits;
                            mbar_arrive(aux_full + kt % kAuxRing);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < chunks; ++r) {
                        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r * rpr + my_row);
                        const bool live = o >= 0 && chunk_in;
                        cp16(swizzled(at0 + slot * X::slot_bytes, r, 0), live ? src + o + my_chunk * 16 : src, live ? 16u : 0u);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (kt >= kLag) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
                        fence_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(my_full + (kt - kLag) % S);
                    }
                }
            } else {
                // a tile in pieces of 16 rows, two of them on their way in registers
                constexpr int rounds = chunks / 2;
                uint4 d[2][rounds];
                auto issue = [&](uint4 (&w)[rounds], int64_t off, int half) {
#pragma unroll
                    for (int r = 0; r < rounds; ++r) {
                        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, half * 16 + r * rpr + my_row);
                        w[r] = make_uint4(0, 0, 0, 0);
                        if (o >= 0 && chunk_in) w[r] = ld_stream_v4(src + o + my_chunk * 16);
                    }
                };
                auto hand = [&](const uint4 (&w)[rounds], uint32_t base) {
#pragma unroll
                    for (int r = 0; r < rounds; ++r) {
                        sts16(swizzled(base, r, 0),
                              make_uint4(e4m3_f16x2(w[r].x & 0xFFFF), e4m3_f16x2(w[r].x >> 16), e4m3_f16x2(w[r].y & 0xFFFF),
                                         e4m3_f16x2(w[r].y >> 16)));
                        sts16(swizzled(base, r, 1),
                              make_uint4(e4m3_f16x2(w[r].z & 0xFFFF), e4m3_f16x2(w[r].z >> 16), e4m3_f16x2(w[r].w & 0xFFFF),
                                         e4m3_f16x2(w[r].w >> 16)));
                    }
                };
                int64_t off = next;
                float sk = 0.f, sv = 0.f;
                auto scales = [&]() {
                    sk = sv = 0.f;
                    if (is_k && off >= 0) sk = c.ks[sc_next], sv = c.vs[sc_next];
                };
                scales();
                issue(d[0], off, 0);
                issue(d[1], off, 1);
                for (int t = 0; t < n; ++t, ++kt) {
                    pos += kTileTok;
                    next = t + 1 < n ? row_at() : -1;
                    const uint32_t slot = kt % S, use = kt / S;
                    if (use) wait(my_empty + slot, (use - 1) & 1);
                    if (is_k) {
                        unsigned char* const at = aux_sm + (kt % kAuxRing) * X::aux_bytes;
                        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, off >= 0);
                        if (lane == 0) ((uint32_t*)at)[fw] = bits;
                        ((float*)(at + 16))[fw * 32 + lane] = sk;
                        ((float*)(at + 16))[kTileTok + fw * 32 + lane] = sv;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(aux_full + kt % kAuxRing);
                    }
                    off = next;
                    hand(d[0], at0 + slot * X::slot_bytes);
                    if (t + 1 < n) {
                        scales();
                        issue(d[0], off, 0);
                    }
                    hand(d[1], at0 + slot * X::slot_bytes + 16 * 128);
                    if (t + 1 < n) issue(d[1], off, 1);
                    fence_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(my_full + slot);
                }
            }
        }
        if constexpr (!Q8) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            fence_async();
            __syncwarp();
            if (lane == 0)
                for (uint32_t t = kt > kLag ? kt - kLag : 0; t < kt; ++t) mbar_arrive(my_full + t % S);
        }
    } else if (warp >= kMmaWarp) {
        fewer_regs<56>();
        if (warp == kMmaWarp) {
        // ============================================================ products
        constexpr uint32_t id_qk = instr_desc(!Q8, false, false, N);
        constexpr uint32_t id_pv = instr_desc(!Q8, true, true, X::NP);
        const uint64_t k_desc = operand(smem_addr(smem), 16, 1024, 2), q_desc = operand(smem_addr(q_sm), 16, 1024, 2);
        const uint64_t v_desc = operand(smem_addr(smem) + S * X::slot_bytes, DP == 128 ? kTileTok * 128 : 0, 1024, 2);
        const uint64_t p_desc = operand(smem_addr(p_sm), 128, 2048, 0);
        uint32_t gt = 0;
        for (uint32_t si = 0;; ++si) {
            const int n = get_seg(si)->n;
            if (!n) break;
            if (lane == 0) {
                wait(q_full, si & 1);
                auto scores = [&](int i) {
                    const uint32_t t = gt + i, buf = t & 1, slot = t % S;
                    wait(full + slot, (t / S) & 1);
                    if (t >= 2) wait(s_empty + buf, ((t >> 1) - 1) & 1);
                    tc_after();
                    const uint64_t ka = k_desc + slot * (X::slot_bytes >> 4);
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        tc_mma(tmem + buf * N, ka + (((k >> 2) * (kTileTok * 128) + (k & 3) * 32) >> 4),
                               q_desc + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), id_qk, k > 0);
                    tc_commit(empty + slot);
                    tc_commit(s_full + buf);
                };
                scores(0);
                for (int i = 0; i < n; ++i) {
                    if (i + 1 < n) scores(i + 1);
                    const uint32_t t = gt + i, slot = t % S;
                    wait(full + S + slot, (t / S) & 1);
                    wait(p_full, t & 1);
                    tc_after();
                    const uint64_t va = v_desc + slot * (X::slot_bytes >> 4);
#pragma unroll
                    for (int k = 0; k < kTileTok / 16; ++k)
                        tc_mma(tmem + 2 * N, va + ((k * 2048) >> 4), p_desc + ((k * 256) >> 4), id_pv, i > 0 || k > 0);
                    tc_commit(empty + S + slot);
                    tc_commit(pv_done);
                }
            }
            gt += n;
            done_seg(si);
        }
        if (lane == 0) {
            tc_commit(drain);  // everything issued here is done before TMEM is freed
            const uint64_t t0 = nanoseconds();
            while (!mbar_try_wait(drain, 0) && nanoseconds() - t0 < kAttWaitNs) {
            }
        }
        __syncwarp();
    } else if (warp == kSegWarp) {
        // ============================================================ segments
        Walk<N> walk(a, u0, u1, b0, base0);
        for (uint32_t s = 0;; ++s) {
            Seg g;
            walk.next(g);
            if (s >= R) wait(seg_empty + s % R, (s / R - 1) & 1);
            if (lane == 0) {
                segs[s % R] = g;
                mbar_arrive(seg_full + s % R);
            }
            if (!g.n) break;
        }
        __syncwarp();
    } else if (warp == kStatusWarp) {
        // ============================================================ statuses
        // One sequence at a time: its offsets, length, tree and pages; the
        // rows of a sequence with an error become zeros.
        for (int32_t b = blockIdx.x; b < c.B; b += p.grid) {
            const KvSeq s = kv_seq(b, a.row_off, a.t_max, a.rows, a.kv_lens, c.bs, c.max_blocks, true);
            int32_t st = s.st;
            bool bad = false;
            if (st == kKvOk && a.parent)
                for (int32_t v = lane; v < s.T; v += 32) {
                    const int32_t u = a.parent[s.lo + v];
                    bad |= v == 0 ? u != -1 : (u < 0 || u >= v);
                }
            if (__any_sync(0xFFFFFFFFu, bad)) st = kKvBadLayout;
            if (st != kKvOk && s.lo >= 0) {
                const int64_t m = (int64_t)s.T * a.Hq * c.D, o = s.lo * a.Hq * c.D;  // head_dim is a multiple of 8
                for (int64_t i = (int64_t)lane * 8; i < m; i += 256) *(uint4*)(a.out + (o + i) * 2) = make_uint4(0, 0, 0, 0);
                if (a.lse)
                    for (int64_t i = lane; i < (int64_t)s.T * a.Hq; i += 32)
                        a.lse[s.lo * a.Hq + i] = __uint_as_float(0xFF800000u);
            }
            if (a.seq_status) {
                if (st == kKvOk) {
                    bad = false;
                    if (s.T > 0)
                        for (int64_t j = lane; j * c.bs < s.L; j += 32) {
                            const int32_t pg = c.table[(int64_t)b * c.max_blocks + j];
                            bad |= pg < 0 || pg >= c.num_blocks;
                        }
                    if (__any_sync(0xFFFFFFFFu, bad)) st = kKvBadLayout;
                }
                if (lane == 0) a.seq_status[b] = st;
            }
        }
        }
    } else {
        if constexpr (!Q8) more_regs<88>();
        // ============================================================ softmax
        // Thread = one position of the tile; group gr has the 8-row pieces gr,
        // gr + 4, ... of the query rows. A weight is 2^(score - m) with m the
        // row's running maximum, which may lag by kGrow: rescaling is rare.
        const int gr = warp >> 2, wq = warp & 3, wt = tid & 127;
        const int bar_gr = 1 + gr;
        constexpr int bar_all = 1 + kGroups;
        constexpr bool kKeep = MC <= 2;  // few pieces: the scores stay in registers between the two looks at them
        const uint32_t lanes = (uint32_t)wq << 21;  // this warp's 32 TMEM lanes
        const uint32_t o_at = tmem + 2 * N + lanes;
        unsigned char* const pw = p_sm + (wt >> 3) * 128 + (wt & 7) * 16;  // this thread's P, piece 0
        // the group's scratch [5][MC * 8]: its own, or its second part of P while P is free
        float* const red = (float*)(Q8 ? red_sm + gr * X::red_bytes : p_sm + (N / 8 + (gr < N / 8 ? gr : 0)) * 2048);
        const float k2 = a.scale * kLog2e;
        const float none = __uint_as_float(0xFF800000u);
        uint32_t gt = 0;
        for (uint32_t si = 0;; ++si) {
            const Seg* const g = get_seg(si);
            const int n = g->n;
            if (!n) break;
            const int32_t T = g->T, L = g->L, row0 = g->rt * N, ctx = L - T;
            const int32_t rows = min(N, T * a.G - row0);
            const int pieces = (rows + 7) / 8;
            const int live = gr < pieces ? (pieces - gr + kGroups - 1) / kGroups : 0;  // this group's pieces
            // ---- the queries, and per-row state. Q is free: every product
            // with the last segment's queries has been waited for.
            {
                constexpr int qc = DP / 8;  // 16-byte pieces of a row
                constexpr int loads = (N * qc + kSoftThreads - 1) / kSoftThreads;
                uint4 w[loads];
#pragma unroll
                for (int i = 0; i < loads; ++i) {
                    const int r = (tid + i * kSoftThreads) / qc, piece = tid % qc;
                    w[i] = make_uint4(0, 0, 0, 0);
                    if (r < rows && piece * 8 < c.D) {
                        const int32_t rr = row0 + r, t = rr / a.G;
                        w[i] = *(const uint4*)(a.q + (g->lo + t) * a.q_row_bytes +
                                               ((int64_t)g->h * a.G + (rr - t * a.G)) * c.D * 2 + piece * 16);
                    }
                }
#pragma unroll
                for (int i = 0; i < loads; ++i) {
                    const int r = (tid + i * kSoftThreads) / qc, piece = tid % qc;
                    if (Q8) {
                        // bf16 to f16 under a power of two for the row: its largest element goes to [2^14, 2^15),
                        // so that only what is 2^-28 of it or less loses bits
                        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                        float x[8], top = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            x[2 * j] = bf16_lo(u[j]);
                            x[2 * j + 1] = bf16_hi(u[j]);
                            const float m0 = fabsf(x[2 * j]), m1 = fabsf(x[2 * j + 1]);
                            top = m0 < __uint_as_float(0x7F800000u) ? fmaxf(top, m0) : top;
                            top = m1 < __uint_as_float(0x7F800000u) ? fmaxf(top, m1) : top;
                        }
#pragma unroll
                        for (int o = qc / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                        int e = (int)(__float_as_uint(top) >> 23) - 127 - 14;  // x / 2^e
                        e = max(-126, min(113, top == 0.f ? 0 : e));
                        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
                        w[i] = make_uint4(f16x2(x[0] * f, x[1] * f), f16x2(x[2] * f, x[3] * f), f16x2(x[4] * f, x[5] * f),
                                          f16x2(x[6] * f, x[7] * f));
                        if (piece == 0 && r < N) arow[r] = k2 * __uint_as_float((uint32_t)(127 + e) << 23);
                    }
                    if (r < N) sts16(smem_addr(q_sm) + (piece >> 3) * (N * 128) + r * 128 + ((piece ^ r) & 7) * 16, w[i]);
                }
                if (tid < N) mref[tid] = kNoMax;
                if (tid < 4) poison[tid] = 0;
                if (a.parent) {
                    // ancestors by doubling: after k rounds a token knows those up to 2^k - 1 above it
                    int32_t jump = -1;
                    bool bad = false;
                    uint32_t m[4] = {0, 0, 0, 0};
                    uint32_t* const jumps = (uint32_t*)p_sm;  // P is free between segments
                    if (tid < kKvMaxQueries) {
                        if (tid < T) {
                            jump = a.parent[g->lo + tid];
                            bad = tid == 0 ? jump != -1 : (jump < 0 || jump >= tid);
                            if (bad) jump = -1;
                            m[tid >> 5] = 1u << (tid & 31);
                        }
                        *(uint4*)(anc + tid * 4) = make_uint4(m[0], m[1], m[2], m[3]);
                        jumps[tid] = (uint32_t)jump;
                    }
                    const bool any = bar_or(bar_all, kSoftThreads, bad);
                    if (tid == 0) *tree_bad = any;
                    for (int reach = 1; reach < T; reach <<= 1) {
                        uint4 up = make_uint4(0, 0, 0, 0);
                        int32_t far = -1;
                        if (jump >= 0) {
                            up = *(const uint4*)(anc + jump * 4);
                            far = (int32_t)jumps[jump];
                        }
                        bar_sync(bar_all, kSoftThreads);
                        if (jump >= 0) {
                            m[0] |= up.x, m[1] |= up.y, m[2] |= up.z, m[3] |= up.w;
                            *(uint4*)(anc + tid * 4) = make_uint4(m[0], m[1], m[2], m[3]);
                            jumps[tid] = (uint32_t)far;
                        }
                        jump = far;
                        bar_sync(bar_all, kSoftThreads);
                    }
                } else {
                    bar_sync(bar_all, kSoftThreads);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            float l[MC][8];
#pragma unroll
            for (int m = 0; m < MC; ++m)
#pragma unroll
                for (int k = 0; k < 8; ++k) l[m][k] = 0.f;
            int32_t lv = -100;  // Q8: values count in units of 2^lv

            for (int i = 0; i < n; ++i) {
                const uint32_t t = gt + i, buf = t & 1;
                if (live) {
                    wait(aux_full + t % kAuxRing, (t / kAuxRing) & 1);
                    const unsigned char* aux = aux_sm + (t % kAuxRing) * X::aux_bytes;
                    const bool in = ((const uint32_t*)aux)[wq] >> lane & 1;
                    const float ks = Q8 ? ((const float*)(aux + 16))[wt] : 1.f;
                    const float vs = Q8 ? ((const float*)(aux + 16))[kTileTok + wt] : 1.f;
                    const int32_t pos0 = (g->tile0 + i) * kTileTok, pos = pos0 + wt;
                    const uint32_t s_at = tmem + buf * N + lanes;
                    const bool tail = pos0 + kTileTok > ctx;
                    // rows that see this position (a bit for each of the group's rows), where not every row sees
                    // every one; a page outside the pool hides positions anywhere
                    uint32_t vis = in ? ~0u : 0u;
                    if (tail && in && pos >= ctx) {
                        const int32_t u = pos - ctx;
                        vis = 0;
#pragma unroll 1
                        for (int m = 0; m < live; ++m)
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                const int32_t tk = (row0 + (gr + kGroups * m) * 8 + k) / a.G;
                                const bool see = a.parent ? tk < T && (anc[tk * 4 + (u >> 5)] >> (u & 31) & 1) : tk >= u;
                                vis |= (uint32_t)see << (m * 8 + k);
                            }
                    }
                    const bool masked = tail || __any_sync(0xFFFFFFFFu, !in);
                    wait(s_full + buf, (t >> 1) & 1);
                    tc_after();

                    // scores of piece m relative to the running maximum, in units of log2
                    auto relative = [&](int m, float (&z)[8], bool from_zero) {
                        const int r = (gr + kGroups * m) * 8;
                        float f[8], x[8];
                        *(float4*)x = *(const float4*)(mref + r);
                        *(float4*)(x + 4) = *(const float4*)(mref + r + 4);
                        if (Q8) {
                            *(float4*)f = *(const float4*)(arow + r);
                            *(float4*)(f + 4) = *(const float4*)(arow + r + 4);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) z[k] = fmaf(z[k], Q8 ? f[k] * ks : k2, from_zero ? 0.f : -x[k]);
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) z[k] = (vis >> (m * 8 + k) & 1) ? z[k] : none;
                        }
                    };
                    float zk[kKeep ? MC : 1][8];
                    float top = none;
                    if constexpr (kKeep) {
#pragma unroll
                        for (int m = 0; m < MC; ++m)
                            if (m < live) tc_ld8(s_at + (gr + kGroups * m) * 8, zk[m]);
                        tc_wait_ld();
#pragma unroll
                        for (int m = 0; m < MC; ++m)
                            if (m < live) {
                                relative(m, zk[m], false);
#pragma unroll
                                for (int k = 0; k < 8; ++k) top = fmaxf(top, zk[m][k]);
                            }
                    } else {
#pragma unroll
                        for (int m = 0; m < MC; ++m)
                            if (m < live) {
                                float z[8];
                                tc_ld8(s_at + (gr + kGroups * m) * 8, z);
                                tc_wait_ld();
                                relative(m, z, false);
#pragma unroll
                                for (int k = 0; k < 8; ++k) top = fmaxf(top, z[k]);
                            }
                    }
                    const float v_unit = Q8 ? __uint_as_float((uint32_t)(lv + 127) << 23) : 0.f;
                    const bool rise = top > kGrow || i == 0 || (Q8 && fabsf(vs) > v_unit);
                    const bool slow = bar_or(bar_gr, 128, rise);
                    if (t) wait(pv_done, (t - 1) & 1);  // P and O are free
                    tc_after();
                    if (slow) {
                        int32_t up = 0;
                        if (Q8) {
                            // the smallest 2^lv that no scale passes
                            const uint32_t w = __float_as_uint(fabsf(vs));
                            int32_t e = (int32_t)(w >> 23) - 127 + ((w & 0x7FFFFFu) ? 1 : 0);
                            e = __reduce_max_sync(0xFFFFFFFFu, e);
                            if (lane == 0) ((int32_t*)red)[5 * MC * 8 + wq] = e;
                        }
#pragma unroll 1
                        for (int m = 0; m < live; ++m) {
                            float z[8];
                            tc_ld8(s_at + (gr + kGroups * m) * 8, z);
                            tc_wait_ld();
                            relative(m, z, true);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                int32_t x = __float_as_int(z[k]);
                                x ^= (x >> 31) & 0x7FFFFFFF;  // the order of the floats as integers
                                x = __reduce_max_sync(0xFFFFFFFFu, x);
                                if (lane == 0) red[wq * MC * 8 + m * 8 + k] = __int_as_float(x ^ ((x >> 31) & 0x7FFFFFFF));
                            }
                        }
                        bar_sync(bar_gr, 128);
                        if (Q8) {
                            const int32_t* e = (const int32_t*)red + 5 * MC * 8;
                            up = min(126, max(lv, max(max(e[0], e[1]), max(e[2], e[3])))) - lv;
                        }
                        if (wt < live * 8) {
                            const int r = (gr + kGroups * (wt >> 3)) * 8 + (wt & 7);
                            const float old = mref[r];
                            float m = old;
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const float x = red[w * MC * 8 + wt];
                                m = x > m || x != x ? x : m;
                            }
                            red[4 * MC * 8 + wt] = ex2(old - m);
                            mref[r] = m;
                        }
                        bar_sync(bar_gr, 128);
                        lv += up;
                        const float shrink = Q8 ? (up > 126 ? 0.f : __uint_as_float((uint32_t)(127 - up) << 23)) : 1.f;
#pragma unroll
                        for (int m = 0; m < MC; ++m)
                            if (m < live)
#pragma unroll
                                for (int k = 0; k < 8; ++k) l[m][k] *= red[4 * MC * 8 + m * 8 + k];
                        if (i > 0) {
#pragma unroll 1
                            for (int m = 0; m < live; ++m)
#pragma unroll
                                for (int part = 0; part < (Q8 ? 1 : 2); ++part) {
                                    float o[8];
                                    const uint32_t at = o_at + part * N + (gr + kGroups * m) * 8;
                                    tc_ld8(at, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 8; ++k) o[k] *= red[4 * MC * 8 + m * 8 + k] * shrink;
                                    tc_st8(at, o);
                                }
                            tc_wait_st();
                        }
                        bar_sync(bar_gr, 128);  // the scratch may be P again
                        if constexpr (kKeep) {
#pragma unroll
                            for (int m = 0; m < MC; ++m)
                                if (m < live) tc_ld8(s_at + (gr + kGroups * m) * 8, zk[m]);
                            tc_wait_ld();
#pragma unroll
                            for (int m = 0; m < MC; ++m)
                                if (m < live) relative(m, zk[m], false);
                        }
                    }
                    // ---- weights
                    // Q8: f16 in units that bring the largest possible one, 2^kGrow, to 2^14
                    const float wv = Q8 ? vs * __uint_as_float((uint32_t)(127 + 6 - lv) << 23) : 1.f;
#pragma unroll
                    for (int m = 0; m < MC; ++m) {
                        if (m < live) {
                            float z[8];
                            if constexpr (kKeep) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) z[k] = zk[m][k];
                            } else {
                                tc_ld8(s_at + (gr + kGroups * m) * 8, z);
                                tc_wait_ld();
                                relative(m, z, false);
                            }
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                z[k] = ex2(z[k]);
                                l[m][k] += z[k];
                            }
                            const int piece = gr + kGroups * m;
                            uint4 w;
                            if (Q8) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) z[k] *= wv;
                                if (masked) {
#pragma unroll
                                    for (int k = 0; k < 8; ++k) z[k] = (vis >> (m * 8 + k) & 1) ? z[k] : 0.f;
                                }
                                w = make_uint4(f16x2(z[0], z[1]), f16x2(z[2], z[3]), f16x2(z[4], z[5]), f16x2(z[6], z[7]));
                                *(uint4*)(pw + piece * 2048) = w;
                            } else {
                                // two bf16 parts: 16 bits of the weight
                                w = make_uint4(bf16x2(z[0], z[1]), bf16x2(z[2], z[3]), bf16x2(z[4], z[5]), bf16x2(z[6], z[7]));
                                *(uint4*)(pw + piece * 2048) = w;
                                w = make_uint4(bf16x2(z[0] - bf16_lo(w.x), z[1] - bf16_hi(w.x)),
                                               bf16x2(z[2] - bf16_lo(w.y), z[3] - bf16_hi(w.y)),
                                               bf16x2(z[4] - bf16_lo(w.z), z[5] - bf16_hi(w.z)),
                                               bf16x2(z[6] - bf16_lo(w.w), z[7] - bf16_hi(w.w)));
                                *(uint4*)(pw + (N / 8 + piece) * 2048) = w;
                            }
                        }
                    }
                    if (tail && gr == 0 && in && pos >= ctx && T > 1) {
                        // A new token's values that are not finite would reach rows that do not see it (0 * inf):
                        // they leave the tile here and join the rows that do see it at the end.
                        wait(full + S + t % S, (t / S) & 1);
                        unsigned char* const v_row = smem + (S + t % S) * X::slot_bytes + wt * 128;
                        constexpr uint32_t ex = Q8 ? 0x7C00u : 0x7F80u;
                        bool found = false;
#pragma unroll 1
                        for (int k = 0; k < DP / 8; ++k) {
                            uint4* const at = (uint4*)(v_row + (k >> 3) * (kTileTok * 128) + (k & 7) * 16);
                            uint4 v = *at;
                            uint32_t* const w = (uint32_t*)&v;
                            bool here = false;
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                if ((w[m] & ex) == ex) w[m] &= 0xFFFF0000u, here = true;
                                if ((w[m] >> 16 & ex) == ex) w[m] &= 0xFFFFu, here = true;
                            }
                            if (here) *at = v;
                            found |= here;
                        }
                        if (found) atomicOr(poison + ((pos - ctx) >> 5), 1u << ((pos - ctx) & 31));
                    }
                    tc_before();
                    fence_async();
                }
                __syncwarp();
                if (lane == 0) {
                    if (!live) {  // in step with the tiles: one arrival in each phase
                        wait(s_full + buf, (t >> 1) & 1);
                        if (t) wait(pv_done, (t - 1) & 1);
                    }
                    mbar_arrive(s_empty + buf);
                    mbar_arrive(p_full);
                }
            }
            gt += n;

            // ---- the segment's sums
            const bool whole = n == g->tiles;
            const bool skip = a.parent && *tree_bad;  // its rows are zeros, written with the statuses
            const int64_t part = (int64_t)blockIdx.x * 2 + (g->tile0 == 0 ? 1 : 0);
            auto out_row = [&](int r) {
                const int32_t rr = row0 + r, tk = rr / a.G;
                return (g->lo + tk) * a.Hq + (int64_t)g->h * a.G + (rr - tk * a.G);
            };
            wait(pv_done, (gt - 1) & 1);
            tc_after();
            if (live) {
                // each row's weights over the 128 positions: a warp's 32 by halving the rows a lane holds
#pragma unroll
                for (int m = 0; m < MC; ++m)
                    if (m < live) {
                        float x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = l[m][k];
#pragma unroll
                        for (int h = 4; h; h >>= 1) {
                            const bool hi = lane & (4 * h);
#pragma unroll
                            for (int k = 0; k < h; ++k)
                                x[k] = (hi ? x[k + h] : x[k]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? x[k] : x[k + h], 4 * h);
                        }
                        x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], 2);
                        x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], 1);
                        if ((lane & 3) == 0) red[wq * MC * 8 + m * 8 + (lane >> 2)] = x[0];
                    }
                bar_sync(bar_gr, 128);
                if (wt < live * 8) {
                    const float sum = red[wt] + red[MC * 8 + wt] + red[2 * MC * 8 + wt] + red[3 * MC * 8 + wt];
                    const int r = (gr + kGroups * (wt >> 3)) * 8 + (wt & 7);
                    red[4 * MC * 8 + wt] = sum == 0.f ? 0.f : 1.f / sum;
                    if (r < rows) {
                        if (!whole)
                            p.part_ml[part * N + r] = make_float2(mref[r], sum);
                        else if (a.lse && !skip)
                            a.lse[out_row(r)] = sum == 0.f ? none : (mref[r] + log2f(sum)) * 0.69314718055994531f;
                    }
                }
                bar_sync(bar_gr, 128);
                const float back = Q8 ? __uint_as_float((uint32_t)(127 + lv) << 23) * 0.015625f : 1.f;
                const bool any_poison = poison[0] | poison[1] | poison[2] | poison[3];
#pragma unroll 1
                for (int m = 0; m < live; ++m) {
                    const int piece = gr + kGroups * m, r0 = piece * 8;
                    float o[8];
                    tc_ld8(o_at + r0, o);
                    if constexpr (!Q8) {
                        float lo[8];
                        tc_ld8(o_at + N + r0, lo);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] += lo[k];
                    } else {
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] *= back;
                    }
                    if (any_poison && wt < c.D) {
#pragma unroll 1
                        for (int32_t u = 0; u < T; ++u) {
                            if (!(poison[u >> 5] >> (u & 31) & 1)) continue;
                            const int32_t pos = ctx + u;
                            const int32_t pg = c.table[(int64_t)g->b * c.max_blocks + pos / c.bs], sl = pos % c.bs;
                            const unsigned char* v = c.v + pg * c.block_bytes + sl * c.token_bytes + g->h * c.head_bytes;
                            const float x = Q8 ? kv_e4m3(v[wt]) : bf16_lo(*(const uint16_t*)(v + 2 * wt));
                            if (fabsf(x) < __uint_as_float(0x7F800000u)) continue;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int32_t tk = (row0 + r0 + k) / a.G;
                                if (a.parent ? tk < T && (anc[tk * 4 + (u >> 5)] >> (u & 31) & 1) : tk >= u) o[k] += x;
                            }
                        }
                    }
                    if (whole) {
                        // through shared memory (this piece's own P) to 16-byte stores
                        uint16_t* const st = (uint16_t*)(p_sm + piece * 2048);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float f = red[4 * MC * 8 + m * 8 + k];
                            st[k * 128 + wt] = (uint16_t)bf16x2(f == 0.f ? 0.f : o[k] * f, 0.f);
                        }
                        bar_sync(bar_gr, 128);
                        const int k = wt >> 4, ch = wt & 15;
                        if (r0 + k < rows && ch * 8 < c.D && !skip)
                            *(uint4*)(a.out + (out_row(r0 + k) * c.D + ch * 8) * 2) = *(const uint4*)(st + k * 128 + ch * 8);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (r0 + k < rows) p.part_o[(part * N + r0 + k) * 128 + wt] = o[k];
                    }
                }
            }
            if (!whole) {
                // ---- join: the entry's parts lie with CTAs c0 (its second place) and c0 + 1 .. c1 (their first)
                const int32_t c0 = (int32_t)(g->first / per), c1 = (int32_t)((g->first + g->tiles - 1) / per);
                __threadfence();
                bar_sync(bar_all, kSoftThreads);
                if (tid == 0) {
                    const uint32_t k = atomicAdd(p.arrive + c0, 1u);
                    *last_in = k == (uint32_t)(c1 - c0);
                    if (k == (uint32_t)(c1 - c0)) p.arrive[c0] = 0;  // for the next call
                    __threadfence();
                }
                bar_sync(bar_all, kSoftThreads);
                if (*last_in && !skip) {
                    // a warp for each row, four columns to a lane
#pragma unroll 1
                    for (int r = warp; r < rows; r += kSoftWarps) {
                        float M = kNoMax;
                        for (int32_t j = c0 + lane; j <= c1; j += 32) {
                            const float x = __ldcg(&p.part_ml[((int64_t)j * 2 + (j == c0)) * N + r].x);
                            M = x > M || x != x ? x : M;
                        }
#pragma unroll
                        for (int o = 16; o; o >>= 1) {
                            const float x = __shfl_xor_sync(0xFFFFFFFFu, M, o);
                            M = x > M || x != x ? x : M;
                        }
                        float sum = 0.f;
                        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                        for (int32_t j = c0; j <= c1; ++j) {
                            const int64_t at = ((int64_t)j * 2 + (j == c0)) * N + r;
                            const float2 ml = __ldcg(p.part_ml + at);
                            const float4 x = __ldcg((const float4*)(p.part_o + at * 128) + lane);
                            const float f = ex2(ml.x - M);
                            sum = fmaf(f, ml.y, sum);
                            o.x = fmaf(f, x.x, o.x);
                            o.y = fmaf(f, x.y, o.y);
                            o.z = fmaf(f, x.z, o.z);
                            o.w = fmaf(f, x.w, o.w);
                        }
                        const float f = sum == 0.f ? 0.f : 1.f / sum;
                        if (f == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
                        const int64_t out = out_row(r);
                        if (lane * 4 < c.D)
                            *(uint2*)(a.out + (out * c.D + lane * 4) * 2) =
                                make_uint2(bf16x2(o.x * f, o.y * f), bf16x2(o.z * f, o.w * f));
                        if (a.lse && lane == 0) a.lse[out] = sum == 0.f ? none : (M + log2f(sum)) * 0.69314718055994531f;
                    }
                }
            }
            bar_sync(bar_all, kSoftThreads);  // scratch and row state are the next segment's
            done_seg(si);
        }
    }

    // ------------------------------------------------------------------ end
    tc_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    if (*aborted && tid == 0) {
        atomicOr(p.err, 1u);
        if (a.seq_status) {
            Walk<N> walk(a, u0, u1, b0, base0);
            Seg g;
            for (walk.next(g); g.n; walk.next(g)) a.seq_status[g.b] = kKvTimeout;
        }
    }
}

template <int N, int DP, bool Q8>
cudaError_t launch(const AttParams& p, cudaStream_t s) {
    using X = Shape<N, DP, Q8>;
    auto* f = attend_kernel<N, DP, Q8>;
    // more than half of an SM's shared memory, whatever the ring took: one CTA on an SM owns its TMEM
    constexpr int bytes = (int)(X::total > kSmemMax / 2 + 1024 ? X::total : kSmemMax / 2 + 1024);
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    f<<<p.grid, kAttThreads, bytes, s>>>(p);
    return cudaGetLastError();
}

template <int N, bool Q8>
cudaError_t launch_dim(const AttParams& p, cudaStream_t s) {
    return p.a.c.D <= 64 ? launch<N, 64, Q8>(p, s) : launch<N, 128, Q8>(p, s);
}

}  // namespace

}  // namespace specv
