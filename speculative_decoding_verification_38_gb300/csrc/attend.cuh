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

// Attention with row tiles of 2 * nc query rows (nc one of 8, 16, 24, 40, 64).
cudaError_t attend_bf16(int nc, const AttParams& p, cudaStream_t s);
cudaError_t attend_bf16_wide(int nc, const AttParams& p, cudaStream_t s);
cudaError_t attend_e4m3(int nc, const AttParams& p, cudaStream_t s);
cudaError_t attend_e4m3_wide(int nc, const AttParams& p, cudaStream_t s);

constexpr int kAttMaxGrid = 160;  // CTAs (the workspace holds two parts for each)

namespace {

constexpr int kTileTok = 128;                // positions of a tile
constexpr int kSoftWarps = 8;                // two groups of four: each takes half of the query rows
constexpr int kFeedWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kFeedWarps;
constexpr int kAuxWarp = kMmaWarp + 1;
constexpr int kAttThreads = (kAuxWarp + 1) * 32;
constexpr int kMaxSlots = 6;                 // ring slots, one K or V tile each
constexpr int kAuxRing = 8;                  // tiles of masks and scales kept: more than the ring and S can hold
constexpr uint32_t kAttWaitLimit = 1u << 22; // a wait that gives up marks the call, which then runs out unwaited
constexpr float kNoMax = -1.0e30f;           // running maximum before any score
constexpr float kGrow = 8.f;                 // a maximum may rise by 2^8 before the sums are rescaled
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

// ------------------------------------------------------------------ layout
template <int NC, int DP, bool Q8>
struct Shape {
    static constexpr int N = 2 * NC;                       // query rows of a row tile
    static constexpr int NP = Q8 ? N : 2 * N;              // P's columns: one f16, or two bf16 parts
    static constexpr uint32_t slot_bytes = kTileTok * DP * 2;
    static constexpr uint32_t q_bytes = N * DP * 2;
    static constexpr uint32_t p_bytes = NP * kTileTok * 2;
    static constexpr uint32_t aux_bytes = Q8 ? 1024 + 16 : 16;  // scales of K and V, validity bits
    // after the slots, Q and P: aux ring, running maxima, row factors, ancestors, poison, barriers
    static constexpr uint32_t misc = kAuxRing * aux_bytes + N * 4 + (Q8 ? N * 4 : 0) + kKvMaxQueries * 16 + 32 +
                                     (2 * kMaxSlots + 8 + kAuxRing) * 8 + 16;
    static constexpr int fit = (int)((kSmemMax - q_bytes - p_bytes - misc) / slot_bytes);
    static constexpr int slots = fit > kMaxSlots ? kMaxSlots : fit;
    static constexpr uint32_t total = slots * slot_bytes + q_bytes + p_bytes + misc;
    static_assert(slots >= 4, "the ring needs four slots");
};

// A run of tiles of one (sequence, head, row tile).
struct Seg {
    int32_t b, h, rt, tile0, n;  // n tiles from tile0
    int32_t tiles;               // of the whole entry
    int64_t first;               // the entry's first tile in the flat list
    int64_t lo;
    int32_t T, L, rows;          // new tokens, length, live query rows of this row tile
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
    __device__ __forceinline__ bool next(Seg& g) {
        if (u >= u1) return false;
        while (u >= base + units) {
            base += units;
            if (++b >= a.c.B) return false;  // lengths that change under the call
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
        g.rows = min(N, s.T * a.G - g.rt * N);
        u += g.n;
        return true;
    }
};

// Order in which a segment's tiles pass the ring: K0 K1 V0 K2 V1 ... so that a
// tile's scores are under way while the previous tile's weights are made.
__device__ __forceinline__ uint32_t item_k(uint32_t it0, int i) { return it0 + (i ? 2 * i - 1 : 0); }
__device__ __forceinline__ uint32_t item_v(uint32_t it0, int i, int n) { return it0 + (i + 1 < n ? 2 * i + 2 : 2 * n - 1); }

template <int NC, int DP, bool Q8>
__global__ void __launch_bounds__(kAttThreads, 1) attend_kernel(const __grid_constant__ AttParams p) {
    using X = Shape<NC, DP, Q8>;
    constexpr int N = X::N, S = X::slots;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const q_sm = smem + S * X::slot_bytes;
    unsigned char* const p_sm = q_sm + X::q_bytes;
    unsigned char* const aux_sm = p_sm + X::p_bytes;
    float* const mref = (float*)(aux_sm + kAuxRing * X::aux_bytes);
    float* const arow = mref + N;  // Q8: a query row's power of two times scale * log2(e)
    uint32_t* const anc = (uint32_t*)(mref + (Q8 ? 2 * N : N));  // [T][4] ancestors of a tree's tokens
    uint32_t* const poison = anc + kKvMaxQueries * 4;            // [4] new tokens with non-finite values, then 4 words:
    volatile uint32_t* const aborted = poison + 4;               // a wait gave up
    uint32_t* const tmem_at = poison + 5;
    uint32_t* const last_in = poison + 6;
    uint32_t* const tree_bad = poison + 7;
    uint64_t* const full = (uint64_t*)(poison + 8);
    uint64_t* const empty = full + kMaxSlots;
    uint64_t* const s_full = empty + kMaxSlots;
    uint64_t* const s_empty = s_full + 2;
    uint64_t* const p_full = s_empty + 2;
    uint64_t* const pv_done = p_full + 1;
    uint64_t* const q_full = pv_done + 1;
    uint64_t* const drain = q_full + 1;
    uint64_t* const aux_full = drain + 1;

    const KvAttend& a = p.a;
    const KvView& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        for (uint32_t i = 0; i < kAttWaitLimit; ++i) {
            if (mbar_try_wait(bar, parity)) return;
            if (*aborted) return;
        }
        *aborted = 1;
    };

    // ------------------------------------------------- this CTA's run of tiles
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, kFeedWarps);
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
        for (int i = 0; i < kAuxRing; ++i) mbar_init(aux_full + i, kFeedWarps);
        *aborted = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_at)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    int64_t* const scan = (int64_t*)p_sm;  // P is not in use yet: [18] warp sums, start of the run
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
    const float k2 = a.scale * kLog2e;

    if (warp >= kSoftWarps && warp < kMmaWarp) {
        // ============================================================ feed
        // Each warp brings 16 rows of every tile. A bf16 tile goes straight to
        // shared memory (cp.async); an e4m3 tile passes the registers, where it
        // becomes f16 (exactly). Rows past the length, on a page outside the
        // pool or past head_dim are zeros.
        const int fw = warp - kSoftWarps;
        Walk<N> walk(a, u0, u1, b0, base0);
        Seg g;
        bool more = walk.next(g);
        int ki = 0, vi = 0;
        uint32_t idx = 0, kt = 0;
        int64_t off0 = 0, off1 = 0;  // lane < 16: a row's byte offset, by the tile's parity
        bool ok0 = false, ok1 = false;
        float sk = 0.f, sv = 0.f;
        constexpr int chunks = DP * (Q8 ? 1 : 2) / 16;  // 16-byte pieces of a padded row
        constexpr int rounds = 16 * chunks / 32;
        const int my_chunk = lane % chunks, my_row = lane / chunks;
        const bool chunk_in = my_chunk * (Q8 ? 16 : 8) < c.D;

        // the rows of tile ki of the segment: offsets, validity, scales
        auto rows_of = [&](int tile_in_seg) {
            const int32_t pos = (g.tile0 + tile_in_seg) * kTileTok + fw * 16 + (lane & 15);
            bool in = lane < 16 && pos < g.L;
            int64_t o = 0;
            sk = sv = 0.f;
            if (in) {
                const int32_t pg = c.table[(int64_t)g.b * c.max_blocks + pos / c.bs];
                const int32_t sl = pos % c.bs;
                in = pg >= 0 && pg < c.num_blocks;
                if (in) {
                    o = pg * c.block_bytes + sl * c.token_bytes + g.h * c.head_bytes;
                    if (Q8) {
                        const int64_t si = ((int64_t)pg * c.H + g.h) * c.bs + sl;
                        sk = c.ks[si];
                        sv = c.vs[si];
                    }
                }
            }
            if (tile_in_seg & 1)
                off1 = o, ok1 = in;
            else
                off0 = o, ok0 = in;
        };
        // aux of tile kt: validity bits and scales, read by the softmax warps
        auto put_aux = [&](bool in, float k_s, float v_s) {
            unsigned char* at = aux_sm + (kt % kAuxRing) * X::aux_bytes;
            const uint32_t bits = __ballot_sync(0xFFFFFFFFu, in);
            if (lane == 0) ((uint16_t*)at)[fw] = (uint16_t)bits;
            if (Q8 && lane < 16) {
                ((float*)(at + 16))[fw * 16 + lane] = k_s;
                ((float*)(at + 16))[kTileTok + fw * 16 + lane] = v_s;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(aux_full + kt % kAuxRing);
            ++kt;
        };
        auto swizzled = [&](uint32_t slot, int row, int chunk) {  // chunk of 8 sixteen-bit elements
            return smem_addr(smem) + slot * X::slot_bytes + (chunk >> 3) * (kTileTok * 128) + row * 128 +
                   ((chunk ^ row) & 7) * 16;
        };

        if constexpr (!Q8) {
            constexpr uint32_t kLag = 2;  // groups of copies in flight when one is handed over
            auto publish = [&](uint32_t i) {
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + i % S);
            };
            while (more) {
                const bool is_k = ki < g.n && ki <= vi + 1;
                const int t = is_k ? ki : vi;
                if (is_k) rows_of(t);
                const uint32_t slot = idx % S, use = idx / S;
                if (use) wait(empty + slot, (use - 1) & 1);
                const unsigned char* src = is_k ? c.k : c.v;
                const int64_t o64 = t & 1 ? off1 : off0;
                const bool in = t & 1 ? ok1 : ok0;
                if (is_k) put_aux(in, 0.f, 0.f);
#pragma unroll
                for (int r = 0; r < rounds; ++r) {
                    const int row = r * (32 / chunks) + my_row;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, o64, row);
                    const bool live = __shfl_sync(0xFFFFFFFFu, in, row) && chunk_in;
                    cp16(swizzled(slot, fw * 16 + row, my_chunk), live ? src + o + my_chunk * 16 : src, live ? 16u : 0u);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (idx >= kLag) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
                    publish(idx - kLag);
                }
                ++idx;
                if (is_k) {
                    ++ki;
                } else if (++vi == g.n) {
                    more = walk.next(g);
                    ki = vi = 0;
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            for (uint32_t i = idx > kLag ? idx - kLag : 0; i < idx; ++i) publish(i);
        } else {
            // three tiles on their way in registers
            struct Stage {
                uint4 d[rounds];
                float sk, sv;
                bool is_k, in, live;
            };
            auto issue = [&](Stage& st) {
                st.live = more;
                if (!more) return;
                st.is_k = ki < g.n && ki <= vi + 1;
                const int t = st.is_k ? ki : vi;
                if (st.is_k) rows_of(t);
                st.sk = sk;
                st.sv = sv;
                const unsigned char* src = st.is_k ? c.k : c.v;
                const int64_t o64 = t & 1 ? off1 : off0;
                st.in = t & 1 ? ok1 : ok0;
#pragma unroll
                for (int r = 0; r < rounds; ++r) {
                    const int row = r * (32 / chunks) + my_row;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, o64, row);
                    const bool live = __shfl_sync(0xFFFFFFFFu, st.in, row) && chunk_in;
                    st.d[r] = live ? ld_stream_v4(src + o + my_chunk * 16) : make_uint4(0, 0, 0, 0);
                }
                if (st.is_k) {
                    ++ki;
                } else if (++vi == g.n) {
                    more = walk.next(g);
                    ki = vi = 0;
                }
            };
            auto hand = [&](const Stage& st) {
                const uint32_t slot = idx % S, use = idx / S;
                if (use) wait(empty + slot, (use - 1) & 1);
                if (st.is_k) put_aux(st.in, st.sk, st.sv);
#pragma unroll
                for (int r = 0; r < rounds; ++r) {
                    const int row = fw * 16 + r * (32 / chunks) + my_row;
                    const uint4 w = st.d[r];
                    sts16(swizzled(slot, row, 2 * my_chunk),
                          make_uint4(e4m3_f16x2(w.x & 0xFFFF), e4m3_f16x2(w.x >> 16), e4m3_f16x2(w.y & 0xFFFF),
                                     e4m3_f16x2(w.y >> 16)));
                    sts16(swizzled(slot, row, 2 * my_chunk + 1),
                          make_uint4(e4m3_f16x2(w.z & 0xFFFF), e4m3_f16x2(w.z >> 16), e4m3_f16x2(w.w & 0xFFFF),
                                     e4m3_f16x2(w.w >> 16)));
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + slot);
                ++idx;
            };
            Stage s0, s1, s2;
            issue(s0);
            issue(s1);
            issue(s2);
            while (s0.live) {
                hand(s0);
                issue(s0);
                if (s1.live) hand(s1);
                issue(s1);
                if (s2.live) hand(s2);
                issue(s2);
            }
        }
    } else if (warp == kMmaWarp) {
        // ============================================================ products
        if (lane == 0) {
            constexpr uint32_t id_qk = instr_desc(!Q8, false, false, N);
            constexpr uint32_t id_pv = instr_desc(!Q8, true, true, X::NP);
            const uint32_t ring = smem_addr(smem), qa = smem_addr(q_sm), pa = smem_addr(p_sm);
            Walk<N> walk(a, u0, u1, b0, base0);
            Seg g;
            uint32_t it0 = 0, gt = 0, segs = 0;
            while (walk.next(g)) {
                wait(q_full, segs & 1);
                auto scores = [&](int i) {
                    const uint32_t idx = item_k(it0, i), slot = idx % S, t = gt + i, buf = t & 1;
                    wait(full + slot, (idx / S) & 1);
                    if (t >= 2) wait(s_empty + buf, ((t >> 1) - 1) & 1);
                    tc_after();
                    const uint32_t ka = ring + slot * X::slot_bytes;
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        tc_mma(tmem + buf * N, operand(ka + (k >> 2) * (kTileTok * 128) + (k & 3) * 32, 16, 1024, 2),
                               operand(qa + (k >> 2) * (N * 128) + (k & 3) * 32, 16, 1024, 2), id_qk, k > 0);
                    tc_commit(empty + slot);
                    tc_commit(s_full + buf);
                };
                scores(0);
                for (int i = 0; i < g.n; ++i) {
                    if (i + 1 < g.n) scores(i + 1);
                    const uint32_t idx = item_v(it0, i, g.n), slot = idx % S;
                    wait(full + slot, (idx / S) & 1);
                    wait(p_full, (gt + i) & 1);
                    tc_after();
                    const uint32_t va = ring + slot * X::slot_bytes;
#pragma unroll
                    for (int k = 0; k < kTileTok / 16; ++k)
                        tc_mma(tmem + 2 * N, operand(va + k * 2048, DP == 128 ? kTileTok * 128 : 0, 1024, 2),
                               operand(pa + k * 256, 128, 2048, 0), id_pv, i > 0 || k > 0);
                    tc_commit(empty + slot);
                    tc_commit(pv_done);
                }
                it0 += 2 * g.n;
                gt += g.n;
                ++segs;
            }
            tc_commit(drain);  // everything issued here is done before TMEM is freed
            for (uint32_t i = 0; i < kAttWaitLimit && !mbar_try_wait(drain, 0); ++i) {
            }
        }
        __syncwarp();
    } else if (warp == kAuxWarp) {
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
                const int64_t n = (int64_t)s.T * a.Hq * c.D, o = s.lo * a.Hq * c.D;  // head_dim is a multiple of 8
                for (int64_t i = (int64_t)lane * 8; i < n; i += 256) *(uint4*)(a.out + (o + i) * 2) = make_uint4(0, 0, 0, 0);
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
    } else {
        // ============================================================ softmax
        // Thread = one position of the tile; group wg has the query rows
        // [wg * NC, wg * NC + NC). A weight is 2^(score - m) with m the row's
        // running maximum, which may lag by kGrow: rescaling the sums is rare.
        const int wg = warp >> 2, wt = tid & 127, col0 = wg * NC;
        const int bar_wg = 1 + wg;
        constexpr int bar_all = 3;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
        const uint32_t o_at = tmem + 2 * N + lanes + col0;
        unsigned char* const pw = p_sm + (col0 / 8) * 2048 + (wt >> 3) * 128 + (wt & 7) * 16;  // this thread's P
        float* const red = (float*)(p_sm + (col0 / 8) * 2048);  // scratch of the group while P is free: [5][NC]
        Walk<N> walk(a, u0, u1, b0, base0);
        Seg g;
        uint32_t it0 = 0, gt = 0;
        while (walk.next(g)) {
            const int32_t row0 = g.rt * N, ctx = g.L - g.T;
            const int live = max(0, min(NC, g.rows - col0));
            // ---- the queries, and per-row state. Q is free: every product
            // with the last segment's queries has been waited for.
            {
                constexpr int qc = DP / 8;  // 16-byte pieces of a row
                const int piece = lane % qc, sub = lane / qc;
                for (int r = warp * (32 / qc) + sub; r < N; r += kSoftWarps * (32 / qc)) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (r < g.rows && piece * 8 < c.D) {
                        const int32_t rr = row0 + r, t = rr / a.G;
                        w = *(const uint4*)(a.q + (g.lo + t) * a.q_row_bytes +
                                            ((int64_t)g.h * a.G + (rr - t * a.G)) * c.D * 2 + piece * 16);
                    }
                    if (Q8) {
                        // bf16 to f16 under a power of two for the row: its largest element goes to [2^14, 2^15),
                        // so that only what is 2^-28 of it or less loses bits
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
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
                        w = make_uint4(f16x2(x[0] * f, x[1] * f), f16x2(x[2] * f, x[3] * f), f16x2(x[4] * f, x[5] * f),
                                       f16x2(x[6] * f, x[7] * f));
                        if (piece == 0) arow[r] = k2 * __uint_as_float((uint32_t)(127 + e) << 23);
                    }
                    sts16(smem_addr(q_sm) + (piece >> 3) * (N * 128) + r * 128 + ((piece ^ r) & 7) * 16, w);
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
                        if (tid < g.T) {
                            jump = a.parent[g.lo + tid];
                            bad = tid == 0 ? jump != -1 : (jump < 0 || jump >= tid);
                            if (bad) jump = -1;
                            m[tid >> 5] = 1u << (tid & 31);
                        }
                        *(uint4*)(anc + tid * 4) = make_uint4(m[0], m[1], m[2], m[3]);
                        jumps[tid] = (uint32_t)jump;
                    }
                    const bool any = bar_or(bar_all, kSoftWarps * 32, bad);
                    if (tid == 0) *tree_bad = any;
                    for (int k = 0; k < 7; ++k) {
                        uint4 up = make_uint4(0, 0, 0, 0);
                        int32_t far = -1;
                        if (jump >= 0) {
                            up = *(const uint4*)(anc + jump * 4);
                            far = (int32_t)jumps[jump];
                        }
                        bar_sync(bar_all, kSoftWarps * 32);
                        if (jump >= 0) {
                            m[0] |= up.x, m[1] |= up.y, m[2] |= up.z, m[3] |= up.w;
                            *(uint4*)(anc + tid * 4) = make_uint4(m[0], m[1], m[2], m[3]);
                            jumps[tid] = (uint32_t)far;
                        }
                        jump = far;
                        bar_sync(bar_all, kSoftWarps * 32);
                    }
                } else {
                    bar_sync(bar_all, kSoftWarps * 32);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            float l[NC];
#pragma unroll
            for (int j = 0; j < NC; ++j) l[j] = 0.f;
            int32_t lv = -100;  // Q8: values count in units of 2^lv

            for (int i = 0; i < g.n; ++i) {
                const uint32_t t = gt + i, buf = t & 1;
                wait(s_full + buf, (t >> 1) & 1);
                tc_after();
                const unsigned char* aux = aux_sm + (t % kAuxRing) * X::aux_bytes;
                wait(aux_full + t % kAuxRing, (t / kAuxRing) & 1);
                const bool in = ((const uint16_t*)aux)[wt >> 4] >> (wt & 15) & 1;
                const float ks = Q8 ? ((const float*)(aux + 16))[wt] : 1.f;
                const float vs = Q8 ? ((const float*)(aux + 16))[kTileTok + wt] : 1.f;
                const int32_t pos0 = (g.tile0 + i) * kTileTok, pos = pos0 + wt;
                const uint32_t s_at = tmem + buf * N + lanes + col0;
                const bool tail = pos0 + kTileTok > ctx;
                // rows that see this position, where not every row sees every one
                uint64_t vis = in ? ~0ull : 0ull;
                if (tail && in && pos >= ctx) {
                    const int32_t u = pos - ctx;
                    if (a.parent) {
                        vis = 0;
                        for (int j = 0; j < live; ++j)
                            vis |= (uint64_t)(anc[((row0 + col0 + j) / a.G) * 4 + (u >> 5)] >> (u & 31) & 1) << j;
                    } else {
                        const int32_t from = u * a.G - row0 - col0;  // rows of tokens u and later
                        vis = from <= 0 ? ~0ull : from >= 64 ? 0ull : ~0ull << from;
                    }
                }
                // a page outside the pool hides positions anywhere
                const bool masked = tail || __any_sync(0xFFFFFFFFu, !in);
                const float none = __uint_as_float(0xFF800000u);

                // scores relative to the running maximum, in units of log2
                auto load = [&](int j, float (&z)[8]) { tc_ld8(s_at + j, z); };
                auto relative = [&](int j, float (&z)[8], bool from_zero) {
                    const float4 m0 = *(const float4*)(mref + col0 + j), m1 = *(const float4*)(mref + col0 + j + 4);
                    const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
                    float f[8];
                    if (Q8) {
                        const float4 a0 = *(const float4*)(arow + col0 + j), a1 = *(const float4*)(arow + col0 + j + 4);
                        f[0] = a0.x, f[1] = a0.y, f[2] = a0.z, f[3] = a0.w;
                        f[4] = a1.x, f[5] = a1.y, f[6] = a1.z, f[7] = a1.w;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        z[k] = fmaf(z[k], Q8 ? f[k] * ks : k2, from_zero ? 0.f : -m[k]);
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) z[k] = (vis >> (j + k) & 1) ? z[k] : none;
                    }
                };
                float top = none;
#pragma unroll
                for (int j = 0; j < NC; j += 8) {
                    if (j < live) {
                        float z[8];
                        load(j, z);
                        tc_wait_ld();
                        relative(j, z, false);
#pragma unroll
                        for (int k = 0; k < 8; ++k) top = j + k < live ? fmaxf(top, z[k]) : top;
                    }
                }
                const float v_unit = Q8 ? __uint_as_float((uint32_t)(lv + 127) << 23) : 0.f;
                const bool rise = top > kGrow || i == 0 || (Q8 && fabsf(vs) > v_unit);
                const bool slow = bar_or(bar_wg, 128, rise);
                if (t) wait(pv_done, (t - 1) & 1);  // P and O are free
                tc_after();
                if (slow) {
                    int32_t up = 0;
                    if (Q8) {
                        // the smallest 2^lv that no scale passes
                        const uint32_t w = __float_as_uint(fabsf(vs));
                        int32_t e = (int32_t)(w >> 23) - 127 + ((w & 0x7FFFFFu) ? 1 : 0);
                        e = __reduce_max_sync(0xFFFFFFFFu, e);
                        if (lane == 0) ((int32_t*)red)[5 * NC + (warp & 3)] = e;
                    }
#pragma unroll
                    for (int j = 0; j < NC; j += 8) {
                        if (j < live) {
                            float z[8];
                            load(j, z);
                            tc_wait_ld();
                            relative(j, z, true);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                int32_t x = __float_as_int(z[k]);
                                x ^= (x >> 31) & 0x7FFFFFFF;  // the order of the floats as integers
                                x = __reduce_max_sync(0xFFFFFFFFu, x);
                                if (lane == 0) red[(warp & 3) * NC + j + k] = __int_as_float(x ^ ((x >> 31) & 0x7FFFFFFF));
                            }
                        }
                    }
                    bar_sync(bar_wg, 128);
                    if (Q8) {
                        const int32_t* e = (const int32_t*)red + 5 * NC;
                        up = min(126, max(lv, max(max(e[0], e[1]), max(e[2], e[3])))) - lv;
                    }
                    if (wt < live) {
                        const float old = mref[col0 + wt];
                        float m = old;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const float x = red[w * NC + wt];
                            m = x > m || x != x ? x : m;
                        }
                        red[4 * NC + wt] = ex2(old - m);
                        mref[col0 + wt] = m;
                    }
                    bar_sync(bar_wg, 128);
                    lv += up;
                    const float shrink = Q8 ? (up > 126 ? 0.f : __uint_as_float((uint32_t)(127 - up) << 23)) : 1.f;
#pragma unroll
                    for (int j = 0; j < NC; j += 8) {
                        if (j < live) {
                            float f[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                f[k] = red[4 * NC + j + k];
                                l[j + k] *= f[k];
                            }
                            if (i > 0) {
#pragma unroll
                                for (int part = 0; part < (Q8 ? 1 : 2); ++part) {
                                    float o[8];
                                    tc_ld8(o_at + part * N + j, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 8; ++k) o[k] *= f[k] * shrink;
                                    tc_st8(o_at + part * N + j, o);
                                }
                            }
                        }
                    }
                    tc_wait_st();
                    bar_sync(bar_wg, 128);  // the scratch is P again
                }
                // ---- weights
                // Q8: f16 in units that bring the largest possible one, 2^kGrow, to 2^14
                const float wv = Q8 ? vs * __uint_as_float((uint32_t)(127 + 6 - lv) << 23) : 1.f;
#pragma unroll
                for (int j = 0; j < NC; j += 8) {
                    if (j < live) {
                        float z[8];
                        load(j, z);
                        tc_wait_ld();
                        relative(j, z, false);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            z[k] = ex2(z[k]);
                            l[j + k] += z[k];
                        }
                        uint4 w;
                        if (Q8) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) z[k] *= wv;
                            if (masked) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) z[k] = (vis >> (j + k) & 1) ? z[k] : 0.f;
                            }
                            w = make_uint4(f16x2(z[0], z[1]), f16x2(z[2], z[3]), f16x2(z[4], z[5]), f16x2(z[6], z[7]));
                            *(uint4*)(pw + (j / 8) * 2048) = w;
                        } else {
                            // two bf16 parts: 16 bits of the weight
                            w = make_uint4(bf16x2(z[0], z[1]), bf16x2(z[2], z[3]), bf16x2(z[4], z[5]), bf16x2(z[6], z[7]));
                            *(uint4*)(pw + (j / 8) * 2048) = w;
                            w = make_uint4(bf16x2(z[0] - bf16_lo(w.x), z[1] - bf16_hi(w.x)),
                                           bf16x2(z[2] - bf16_lo(w.y), z[3] - bf16_hi(w.y)),
                                           bf16x2(z[4] - bf16_lo(w.z), z[5] - bf16_hi(w.z)),
                                           bf16x2(z[6] - bf16_lo(w.w), z[7] - bf16_hi(w.w)));
                            *(uint4*)(pw + (N / 8 + j / 8) * 2048) = w;
                        }
                    }
                }
                if (tail && wg == 0 && in && pos >= ctx && g.T > 1) {
                    // A new token's values that are not finite would reach rows that do not see it (0 * inf):
                    // they leave the tile here and join the rows that do see it at the end.
                    const uint32_t idx = item_v(it0, i, g.n);
                    wait(full + idx % S, (idx / S) & 1);
                    unsigned char* const v_row = smem + (idx % S) * X::slot_bytes + wt * 128;
                    constexpr uint32_t ex = Q8 ? 0x7C00u : 0x7F80u;
                    bool found = false;
                    for (int k = 0; k < DP / 8; ++k) {
                        uint32_t* const w = (uint32_t*)(v_row + (k >> 3) * (kTileTok * 128) + (k & 7) * 16);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            uint32_t x = w[m];
                            if ((x & ex) == ex || (x >> 16 & ex) == ex) {
                                found = true;
                                if ((x & ex) == ex) x &= 0xFFFF0000u;
                                if ((x >> 16 & ex) == ex) x &= 0xFFFFu;
                                w[m] = x;
                            }
                        }
                    }
                    if (found) atomicOr(poison + ((pos - ctx) >> 5), 1u << ((pos - ctx) & 31));
                }
                tc_before();
                fence_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(s_empty + buf);
                    mbar_arrive(p_full);
                }
            }
            gt += g.n;
            it0 += 2 * g.n;

            // ---- the segment's sums
            wait(pv_done, (gt - 1) & 1);
            tc_after();
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                if (j < live) {
                    float x = l[j];
#pragma unroll
                    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                    if (lane == 0) red[(warp & 3) * NC + j] = x;
                }
            }
            bar_sync(bar_all, kSoftWarps * 32);
            const bool whole = g.n == g.tiles;
            const bool skip = a.parent && *tree_bad;  // its rows are zeros, written with the statuses
            const uint32_t any_poison = poison[0] | poison[1] | poison[2] | poison[3];
            const int64_t part = (int64_t)blockIdx.x * 2 + (g.tile0 == 0 ? 1 : 0);
            const float back = Q8 ? __uint_as_float((uint32_t)(127 + lv) << 23) * 0.015625f : 1.f;
#pragma unroll
            for (int j = 0; j < NC; j += 8) {
                if (j < live) {
                    float o[8];
                    tc_ld8(o_at + j, o);
                    if constexpr (!Q8) {
                        float lo[8];
                        tc_ld8(o_at + N + j, lo);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] += lo[k];
                    } else {
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] *= back;
                    }
                    if (any_poison && wt < c.D) {
                        for (int32_t u = 0; u < g.T; ++u) {
                            if (!(poison[u >> 5] >> (u & 31) & 1)) continue;
                            const int32_t pos = ctx + u;
                            const int32_t pg = c.table[(int64_t)g.b * c.max_blocks + pos / c.bs], sl = pos % c.bs;
                            const unsigned char* v = c.v + pg * c.block_bytes + sl * c.token_bytes + g.h * c.head_bytes;
                            const float x = Q8 ? kv_e4m3(v[wt]) : bf16_lo(*(const uint16_t*)(v + 2 * wt));
                            if (fabsf(x) < __uint_as_float(0x7F800000u)) continue;
                            for (int k = 0; k < 8; ++k) {
                                const int32_t tk = (row0 + col0 + j + k) / a.G;
                                if (a.parent ? tk < g.T && (anc[tk * 4 + (u >> 5)] >> (u & 31) & 1) : tk >= u) o[k] += x;
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int r = col0 + j + k;
                        if (j + k < live) {
                            const float sum = red[j + k] + red[NC + j + k] + red[2 * NC + j + k] + red[3 * NC + j + k];
                            if (whole) {
                                if (!skip) {
                                    const int32_t rr = row0 + r, tk = rr / a.G;
                                    const int64_t out = (g.lo + tk) * a.Hq + (int64_t)g.h * a.G + (rr - tk * a.G);
                                    const float y = sum == 0.f ? 0.f : o[k] / sum;
                                    if (wt < c.D) *(uint16_t*)(a.out + (out * c.D + wt) * 2) = (uint16_t)bf16x2(y, 0.f);
                                    if (a.lse && wt == 0)
                                        a.lse[out] = sum == 0.f ? __uint_as_float(0xFF800000u)
                                                                : (mref[r] + log2f(sum)) * 0.69314718055994531f;
                                }
                            } else {
                                p.part_o[(part * N + r) * 128 + wt] = o[k];
                                if (wt == 0) p.part_ml[part * N + r] = make_float2(mref[r], sum);
                            }
                        }
                    }
                }
            }
            if (!whole) {
                // ---- join: the entry's parts lie with CTAs c0 (its second place) and c0 + 1 .. c1 (their first)
                const int64_t c0 = g.first / per, c1 = (g.first + g.tiles - 1) / per;
                __threadfence();
                bar_sync(bar_all, kSoftWarps * 32);
                if (tid == 0) {
                    const uint32_t n = atomicAdd(p.arrive + c0, 1u);
                    *last_in = n == (uint32_t)(c1 - c0);
                    if (n == (uint32_t)(c1 - c0)) p.arrive[c0] = 0;  // for the next call
                    __threadfence();
                }
                bar_sync(bar_all, kSoftWarps * 32);
                if (*last_in && !skip) {
                    for (int r = wg; r < g.rows; r += 2) {
                        float M = kNoMax;
                        for (int64_t i = c0; i <= c1; ++i)
                            M = fmaxf(M, __ldcg(p.part_ml + (i * 2 + (i == c0)) * N + r).x);
                        float sum = 0.f, o = 0.f;
                        for (int64_t i = c0; i <= c1; ++i) {
                            const float2 ml = __ldcg(p.part_ml + (i * 2 + (i == c0)) * N + r);
                            const float f = ex2(ml.x - M);
                            sum = fmaf(f, ml.y, sum);
                            o = fmaf(f, __ldcg(p.part_o + ((i * 2 + (i == c0)) * N + r) * 128 + wt), o);
                        }
                        const int32_t rr = row0 + r, tk = rr / a.G;
                        const int64_t out = (g.lo + tk) * a.Hq + (int64_t)g.h * a.G + (rr - tk * a.G);
                        if (wt < c.D) *(uint16_t*)(a.out + (out * c.D + wt) * 2) = (uint16_t)bf16x2(sum == 0.f ? 0.f : o / sum, 0.f);
                        if (a.lse && wt == 0)
                            a.lse[out] = sum == 0.f ? __uint_as_float(0xFF800000u) : (M + log2f(sum)) * 0.69314718055994531f;
                    }
                }
            }
            bar_sync(bar_all, kSoftWarps * 32);  // scratch and row state are the next segment's
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
            while (walk.next(g)) a.seq_status[g.b] = kKvTimeout;
        }
    }
}

template <int NC, int DP, bool Q8>
cudaError_t launch(const AttParams& p, cudaStream_t s) {
    using X = Shape<NC, DP, Q8>;
    auto* f = attend_kernel<NC, DP, Q8>;
    // more than half of an SM's shared memory, whatever the ring took: one CTA on an SM owns its TMEM
    constexpr int bytes = (int)(X::total > kSmemMax / 2 + 1024 ? X::total : kSmemMax / 2 + 1024);
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    f<<<p.grid, kAttThreads, bytes, s>>>(p);
    return cudaGetLastError();
}

template <int NC, bool Q8>
cudaError_t launch_dim(const AttParams& p, cudaStream_t s) {
    return p.a.c.D <= 64 ? launch<NC, 64, Q8>(p, s) : launch<NC, 128, Q8>(p, s);
}

}  // namespace

}  // namespace specv
