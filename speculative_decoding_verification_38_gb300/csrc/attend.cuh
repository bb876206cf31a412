// attend.cuh -- attention of each sequence's new tokens over the paged cache on
// the tensor cores.
//
// The products run transposed: with the 128 positions of a tile as the rows of
// the matrix instruction, S^T = K Q^T [128 x N] and O^T += V^T P^T [head_dim x
// N], N being the query rows (new tokens times the query heads of a key-value
// head). So the long side fills the instruction whatever the number of query
// rows, one token to a whole tree, and work grows with N only: 16 rows of one
// token would use an eighth of an instruction that has them as its rows.
//
// The flat list of tiles over (sequence, head, row tile) is cut into one equal
// run for each CTA (one CTA on each SM). A CTA that holds a whole (sequence,
// head, row tile) writes its rows; one that holds a part leaves its sums in the
// workspace, and groups of parts are joined by whoever comes last, in a fixed
// order.
//
// Arithmetic. Scores, maxima, sums and outputs are float32. bf16 caches: a
// weight goes to the second product as two bf16 parts, 16 bits of it, so that
// the result has the output's own rounding and no second one; the second
// product has twice the columns for it. e4m3 caches: K is the first product's
// operand as it is and the queries its equal in three e5m2 parts, which hold
// all 8 bits of a bf16 number; V turns to f16, exactly, in shared memory, and
// weights are f16 (11 bits). Scales of K go to the scores and of V to the
// weights, in units that go by the scales that a row sees.
//
// Bounds (8 heads of 128, pages of 16). Nine bf16 tokens of each of 64
// sequences over 146,153 positions: 119 us for 608 MB, 0.75 of the copy
// bandwidth; of two over 262,142: 182 us, 0.87. The difference is the ends of
// entries, where a CTA's groups wait for the last of its tiles (about 12,000
// cycles, four or five times in a run). Where a tile takes one team longer
// than its loads, the length of its chain of steps bounds it (scores, their
// read from TMEM, weights, their stores, the vote on references, the product),
// with issue slots to spare: trees of 29 (116 rows), 180 us, 0.52, issue
// active in 47 % of cycles, one place for P as two parts of 128 rows take
// 64 KB; ragged e4m3 chains of up to 72 rows, 957 us for 2.2 GB, 0.34, about
// 4,200 cycles a tile, issue active in 55 %, a fifth of the tiles make their
// weights twice. One e4m3 token of each of the 64: 108 us for 310 MB, 0.42,
// issue active in 40 %: the ends of entries. A single sequence of 4,111:
// 15 us, of which launch, start (the list, TMEM) and the chain page number -
// tile - score - weight - product - join are latency. Far from the floor:
// rows over short caches (65 tokens of 64 sequences of 100 to 400, 8 query
// heads to a key-value head: 263 us bf16, 401 e4m3, for 201 and 170 MB), where
// an entry's opening and end outweigh its few tiles.
#pragma once

#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv.cuh"
#include "settle.h"

namespace specv {

struct AttParams {
    CUtensorMap k_map, v_map;  // boxes of `box` slots of a page's head
    KvAttend a;
    int32_t box, box_log;  // the largest power of two that divides a page and a tile
    float* part_o;     // [grid * 2][N][128] partial sums
    float2* part_ml;   // [grid * 2][N] their maxima (log2) and weights' sums
    uint32_t* arrive;  // [grid] parts arrived, zero between calls
    uint32_t* err;
    uint32_t* left;    // CTAs that are done, and whether one of them gave up: zero between calls
    int32_t* late;     // [grid][2] sequences of the CTAs that gave up: zero between calls
    int32_t grid, device;
};

// Attention with row tiles of n query rows (16, 32, 48, 80 or 128).
cudaError_t attend_bf16(int n, const AttParams& p, cudaStream_t s);
cudaError_t attend_bf16_wide(int n, const AttParams& p, cudaStream_t s);
cudaError_t attend_e4m3(int n, const AttParams& p, cudaStream_t s);
cudaError_t attend_e4m3_wide(int n, const AttParams& p, cudaStream_t s);

constexpr int kAttMaxGrid = 160;  // CTAs (the workspace holds two parts for each)

namespace {

constexpr int kTileTok = 128;   // positions of a tile
constexpr int kGroups = 4;      // softmax groups of four warps
constexpr int kSoftWarps = 4 * kGroups;
constexpr int kMmaWarp = kSoftWarps;      // issues the products
constexpr int kSegWarp = kMmaWarp + 1;    // makes the segments, loads K
constexpr int kValueWarp = kSegWarp + 1;  // loads V, checks the sequences
constexpr int kQueryWarp = kValueWarp + 1;
constexpr int kTurnWarp = kQueryWarp + 1; // e4m3: four warps for queries and scales, four turn V tiles to f16
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMaxSlots = 4;                  // tiles of the K ring, and of the V ring
constexpr uint32_t kAttWaitNs = 2000000000;   // a wait that gives up marks the call, which then runs out unwaited
constexpr float kNoMax = -3.402823466e38f;    // running maximum before any score: not above one, whatever it is
constexpr size_t kSmemMax = 232448;

// ------------------------------------------------------------ instructions
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One lane of the warp, the same each time. The warps that issue products run whole, so that descriptors and addresses
// stay in uniform registers: with one lane's own registers an issue took about 160 cycles.
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
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
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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
__device__ __forceinline__ void tc_ld8(uint32_t at, float2 (&x)[4]) {
    float y[8];
    tc_ld8(at, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(y[2 * i], y[2 * i + 1]);
}
__device__ __forceinline__ void tc_st8(uint32_t at, const float (&x)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
                 "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])),
                 "r"(__float_as_uint(x[3])), "r"(__float_as_uint(x[4])), "r"(__float_as_uint(x[5])),
                 "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7]))
                 : "memory");
}
// The loads before it are done; their registers pass through it, so that no use of them moves ahead.
__device__ __forceinline__ void tc_wait_ld(float (&x)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7])::"memory");
}
__device__ __forceinline__ void tc_wait_ld(float2 (&x)[4]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0].x), "+f"(x[0].y), "+f"(x[1].x), "+f"(x[1].y), "+f"(x[2].x), "+f"(x[2].y), "+f"(x[3].x),
                   "+f"(x[3].y)::"memory");
}
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
__device__ __forceinline__ uint32_t nanoseconds() {  // of a clock that comes round every 4.3 s
    uint32_t t;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
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
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// A box of the cache (elements, slots, head, page) into shared memory; past the pool or head_dim: zeros.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int32_t e, int32_t slot, int32_t head,
                                        int32_t page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(e), "r"(slot), "r"(head), "r"(page), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    return w;
}
__device__ __forceinline__ void sts16(uint32_t dst, uint4 w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}
__device__ __forceinline__ float min_nan(float a, float b) {  // a NaN stays one
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float larger3(float a, float b, float c) {  // of the magnitudes; a NaN stays one
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_warp(float x) {  // a NaN wins
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(x));
    return r;
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
__device__ __forceinline__ uint32_t e5m2x2(float a, float b) {  // a in the low byte
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
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
// The same for A of e4m3 and B of e5m2.
__host__ __device__ constexpr uint32_t instr_desc_f8(int n) {
    return 1u << 4 | 1u << 10 | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// A run of tiles of one (sequence, head, row tile).
struct __align__(16) Seg {
    int32_t b, h, rt, tile0, n;  // n tiles from tile0; n = 0: no more
    int32_t tiles;               // of the whole entry
    int32_t T, L;                // new tokens, length
    int64_t lo;                  // the sequence's first query row
    int32_t c0, c1;              // the CTAs that share the entry
};

// ------------------------------------------------------------------ layout
template <int NN, int DP, bool Q8>
struct Shape {
    static constexpr int N = NN;                           // query rows of a row tile
    static constexpr bool tight = !Q8 && N == 128 && DP == 128;  // shared memory and TMEM are full
    // Teams of softmax groups take the tiles in turn, each with sums of its own, so that a tile may take a team as
    // long as `TM` tiles take the loads; the groups of a team share the rows. With few rows a tile is mostly latency
    // (teams took 9 tokens x 64 from 166 to 155 us, one e4m3 token x 64 from 174 to 120); with 80 e4m3 rows two teams
    // of five pieces a thread were slower than one of three (1212 us against 1019), and 80 bf16 rows have no place for
    // two teams' P.
    static constexpr int TM = N <= 32 ? 4 : N == 48 ? 2 : 1;
    static constexpr int GT = kGroups / TM;                // groups of a team
    static constexpr int SB = TM == 1 ? 2 : TM;            // score tiles in TMEM
    static constexpr int PS = Q8 && N == 80 ? 2 : TM;      // P tiles: one for each team, or two to take turns
    static constexpr int MC = (N / 8 + GT - 1) / GT;       // 8-row pieces of a group
    static constexpr int NP = Q8 ? N : 2 * N;              // P's columns: one f16, or two bf16 parts
    static constexpr int O_at = SB * N, columns = O_at + TM * NP;  // TMEM
    static constexpr int QB = N == 128 || (Q8 && N == 80) ? 1 : 2;  // row tiles of queries held
    static constexpr int segs = tight ? 2 : 4;             // segments known ahead
    static constexpr int threads = (kTurnWarp + (Q8 ? 8 : 0)) * 32;
    static constexpr uint32_t slot_bytes = kTileTok * DP * 2;
    static constexpr uint32_t raw_tile = kTileTok * 128;   // an e4m3 tile as it is: rows of 128 bytes, whatever DP
    static constexpr uint32_t k_bytes = Q8 ? raw_tile : slot_bytes;
    static constexpr int RV = N > 16 ? 2 : 3;              // V tiles as they are
    static constexpr uint32_t raw_bytes = Q8 ? RV * raw_tile : 0;
    static constexpr uint32_t q_bytes = Q8 ? 3 * N * 128 : N * DP * 2;  // e4m3: three parts
    static constexpr uint32_t p_bytes = NP * kTileTok * 2;
    static constexpr uint32_t aux_bytes = Q8 ? 1024 + 16 : 16;  // scales of K and V, validity bits
    static constexpr int aux_ring = TM == 4 ? 16 : Q8 && TM == 1 ? 6 : 8;  // tiles of them: more than the K ring and scores can hold
    static constexpr uint32_t red_bytes = 5 * MC * 8 * 4 + (Q8 ? 4 * MC * 8 : 0);  // a group's scratch
    // after the tiles, Q and P: aux ring, per team and row the reference, weight sum, factor and (e4m3) unit, row factors
    // of Q, scratch, ancestors, segments, poison, barriers
    static constexpr uint32_t state = tight ? N * 4 : (Q8 ? 4 : 3) * TM * N * 4;
    static constexpr uint32_t misc = aux_ring * aux_bytes + state + (Q8 ? segs * N * 4 : 0) +
                                     (tight ? 0 : kGroups * red_bytes) + kKvMaxQueries * 16 + segs * sizeof(Seg) + (tight ? 40 : 48) +
                                     (tight ? 8 : 4 * kMaxSlots + (Q8 ? 2 * RV : 0)) * 8 +
                                     (2 * SB + 2 * PS + 5 + aux_ring + 2 * segs) * 8;
    static constexpr int room = (int)(kSmemMax - raw_bytes - QB * q_bytes - PS * p_bytes - misc), fit = room / slot_bytes;
    // tiles of the K ring and of the V ring; a V tile is held longer
    static constexpr int SK = Q8 ? (room - 3 * (int)k_bytes) / (int)slot_bytes >= 2 ? 3 : 2 : fit / 2 > kMaxSlots ? kMaxSlots : fit / 2;
    static constexpr int rest = Q8 ? (room - SK * (int)k_bytes) / (int)slot_bytes : fit - SK;
    static constexpr int SV = rest > kMaxSlots ? kMaxSlots : rest;
    static constexpr uint32_t ring_bytes = SK * k_bytes + SV * slot_bytes;
    static constexpr uint32_t total = ring_bytes + raw_bytes + QB * q_bytes + PS * p_bytes + misc;
    static_assert(SK >= 2 && SV >= 2, "a ring needs two tiles");
    static_assert(2 * (SK + SV) <= (tight ? 8 : 4 * kMaxSlots) && total <= kSmemMax && columns <= 512, "memory");
    // a tile's masks and scales are written while those of the last SK + SB tiles may be in use
    static_assert(aux_ring > SK + SB, "aux ring");
};

// The flat list of tiles. An entry counts kOver more than its tiles, at its front, for what opening and closing it
// costs; CTA i has [i * per, (i + 1) * per). (Counting tiles only: trees of 64 sequences 258 us, with this 199.)
constexpr int kOver = 5;

// Kept out of line: the few places that divide 64-bit numbers do so once in a while, and their code is large.
__device__ __noinline__ int64_t divide(int64_t a, int64_t b) { return a / b; }

template <int N>
struct Walk {
    const KvAttend& a;
    int64_t u, u1, per, first;  // place, end; where the entry at hand begins
    int32_t b, h, rt;           // the entry
    KvSeq s;
    int32_t tiles, nrt;

    __device__ __forceinline__ static int64_t count(const KvAttend& a, int32_t b, KvSeq& s, int32_t& tiles,
                                                    int32_t& nrt) {
        s = kv_seq(b, a.row_off, a.t_max, a.rows, a.kv_lens, a.c.bs, a.c.max_blocks, true);
        tiles = nrt = 0;
        if (s.st != kKvOk || s.T == 0) return 0;
        tiles = (s.L + kTileTok - 1) / kTileTok;
        nrt = (s.T * a.G + N - 1) / N;
        return (int64_t)(tiles + kOver) * nrt * a.c.H;
    }
    // base0: where sequence b0 begins, which has u0 in it
    __device__ __forceinline__ Walk(const KvAttend& a_, int64_t u0, int64_t u1_, int64_t per_, int32_t b0, int64_t base0)
        : a(a_), u(u0), u1(u1_), per(per_), b(b0), h(0), rt(0) {
        if (u >= u1) return;
        count(a, b, s, tiles, nrt);
        const int64_t e = divide(u - base0, tiles + kOver);
        h = (int32_t)divide(e, nrt);
        rt = (int32_t)(e - (int64_t)h * nrt);
        first = base0 + e * (tiles + kOver);
    }
    __device__ __forceinline__ void next(Seg& g) {
        g.n = 0;
        while (u < u1) {
            const int64_t end = first + kOver + tiles;
            const int64_t from = max(u, first + kOver), to = min(end, u1);
            if (from < to) {
                g.tile0 = (int32_t)(from - first - kOver);
                g.n = (int32_t)(to - from);
                g.h = h;
                g.rt = rt;
                g.tiles = tiles;
                g.b = b;
                g.lo = s.lo;
                g.T = s.T;
                g.L = s.L;
                if (g.n != tiles) {
                    g.c0 = (int32_t)divide(first + kOver, per);
                    g.c1 = (int32_t)divide(end - 1, per);
                }
            }
            u = to > from ? to : min(end, u1);
            if (u == end) {  // on to the next entry
                first = end;
                if (++rt >= nrt) rt = 0, ++h;
                if (h >= a.c.H) {
                    h = 0;
                    do {
                        if (++b >= a.c.B) {  // (before u1 only with lengths that change under the call)
                            u = u1;
                            break;
                        }
                    } while (count(a, b, s, tiles, nrt) == 0);
                }
            }
            if (g.n) return;
        }
    }
};

// Parts are joined in groups of kJoin, groups of groups and so on, each by whoever of its group comes last: joined by
// one CTA alone, the 26 parts of 128 rows took it 50 us, as an SM has few bytes under way. Fewer rows, larger groups.
template <int N>
constexpr int kJoinLog = N <= 16 ? 5 : N <= 32 ? 4 : N <= 48 ? 3 : 2;

// For lane r, the largest value (zero: none) among the lanes whose `seen_by` has row r, of `rows`, by a warp: the lanes with
// the largest give it to their rows, then those with the next for the rows still without. Out of line: it is for the
// few tiles whose positions some rows do not see.
__device__ __noinline__ uint32_t seen_max(uint32_t value, uint32_t seen_by, uint32_t rows) {
    uint32_t mine = 0;
    if (!seen_by) value = 0;
#pragma unroll 1
    while (rows) {
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, value);
        if (!top) break;
        const uint32_t to = rows & __reduce_or_sync(0xFFFFFFFFu, value == top ? seen_by : 0u);
        if (to >> (threadIdx.x & 31) & 1) mine = top;
        rows &= ~to;
        if (value == top) value = 0;
    }
    return mine;
}

// The words of settle.h.
struct Settled {
    const AttParams& p;
    __device__ __forceinline__ void put(int32_t i, int32_t v) const { p.late[i] = v; }
    __device__ __forceinline__ int32_t get(int32_t i) const { return __ldcg(p.late + i); }
    __device__ __forceinline__ void raise() const { atomicOr(p.left + 1, 1u); }
    __device__ __forceinline__ bool raised() const { return __ldcg(p.left + 1) != 0; }
    __device__ __forceinline__ void lower() const { p.left[1] = 0; }
    __device__ __forceinline__ void fence() const { __threadfence(); }
    __device__ __forceinline__ int32_t count() const { return (int32_t)atomicAdd(p.left, 1u); }
    __device__ __forceinline__ void clear_count() const { p.left[0] = 0; }
    __device__ __forceinline__ void mark(int32_t b) const { p.a.seq_status[b] = kKvTimeout; }
};

// Joins `n` parts of an entry, CTAs c0 + i, c0 + i + step, .., into the first or (all of them) into the output. By the
// softmax warps, a row each at a time, four columns to a lane. Out of line: its registers are not taken from the loop
// over the tiles. Factors of the parts: with few rows a row's warp makes them beside its first loads (a single
// sequence's call 14.2 us, 16.6 with the other way); with many, all of them are made first, in f_sm [n + 1][N], so that
// the loads of two rows run together (calls of 25 to 55 us with 80 and 128 rows took 2 to 6 us less).
struct Join {
    const AttParams& p;
    int32_t c0, i, step, n;
    bool all;
    int32_t rows, row0;
    int64_t lo;
    int32_t h;
    __device__ __forceinline__ int64_t place(int32_t k, int N) const {
        return ((int64_t)(c0 + i + k * step) * 2 + (i + k * step == 0)) * N;
    }
    __device__ __forceinline__ int64_t out_row(int r) const {
        const int32_t rr = row0 + r, tk = p.a.by_G.of(rr);
        return (lo + tk) * p.a.Hq + (int64_t)h * p.a.G + (rr - tk * p.a.G);
    }
    __device__ __forceinline__ void sums(int r, float M, float sum, int N) const {
        if (!all)
            p.part_ml[place(0, N) + r] = make_float2(M, sum);
        else if (p.a.lse)
            p.a.lse[out_row(r)] = sum == 0.f ? __uint_as_float(0xFF800000u) : (M + log2f(sum)) * 0.69314718055994531f;
    }
    __device__ __forceinline__ void row(int r, int lane, float4 o, float inv, int N) const {
        if (!all) {
            *((float4*)(p.part_o + (place(0, N) + r) * 128) + lane) = o;
            return;
        }
        if (inv == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
        *(uint2*)(p.a.out + (out_row(r) * p.a.c.D + lane * 4) * 2) =
            make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
    }
};
__device__ __forceinline__ float larger(float x, float y) { return x > y || x != x ? x : y; }  // a NaN wins
__device__ __forceinline__ void add(float4& o, float f, float4 x) {
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
}

template <int N, bool Q8>
__device__ __noinline__ void join_few(Join w) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool column = lane * 4 < w.p.a.c.D;
    constexpr int UN = Q8 ? 4 : 8;  // parts at a time
#pragma unroll 1
    for (int r = warp; r < w.rows; r += kSoftWarps) {
        const float2 ml = lane < w.n ? __ldcg(w.p.part_ml + w.place(lane, N) + r) : make_float2(kNoMax, 0.f);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f), x[UN];
        auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < UN; ++k)  // (past the last one: the last again, not counted)
                if (column) x[k] = __ldcg((const float4*)(w.p.part_o + (w.place(min(k0 + k, w.n - 1), N) + r) * 128) + lane);
        };
        load(0);
        float M = ml.x;
#pragma unroll
        for (int b = 16; b; b >>= 1) M = larger(__shfl_xor_sync(0xFFFFFFFFu, M, b), M);
        const float f = ex2(ml.x - M);
        float sum = lane < w.n ? f * ml.y : 0.f;
#pragma unroll
        for (int b = 16; b; b >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, b);
#pragma unroll 1
        for (int k0 = 0;;) {
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                if (k0 + k >= w.n) break;
                add(o, __shfl_sync(0xFFFFFFFFu, f, k0 + k), x[k]);
            }
            if ((k0 += UN) >= w.n) break;
            load(k0);
        }
        if (column) w.row(r, lane, o, sum == 0.f ? 0.f : 1.f / sum, N);
        if (lane == 0) w.sums(r, M, sum, N);
    }
}

template <int N>
__device__ __noinline__ void join_many(Join w, float* f_sm) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    {
        constexpr int lg = kJoinLog<N>;
        static_assert((N << lg) <= kSoftThreads, "a thread for each (row, part)");
        const int row = tid >> lg, r = min(row, w.rows - 1), k = tid & ((1 << lg) - 1);
        const float2 ml = k < w.n ? __ldcg(w.p.part_ml + w.place(k, N) + r) : make_float2(kNoMax, 0.f);
        float M = ml.x;
#pragma unroll
        for (int b = 1 << lg >> 1; b; b >>= 1) M = larger(__shfl_xor_sync(0xFFFFFFFFu, M, b), M);
        const float f = ex2(ml.x - M);
        float sum = k < w.n ? f * ml.y : 0.f;
#pragma unroll
        for (int b = 1 << lg >> 1; b; b >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, b);
        if (row < w.rows) {
            if (k < w.n) f_sm[k * N + r] = f;
            if (k == 0) {
                f_sm[w.n * N + r] = sum == 0.f ? 0.f : 1.f / sum;
                w.sums(r, M, sum, N);
            }
        }
    }
    bar_sync(1 + kGroups, kSoftThreads);
    if (lane * 4 >= w.p.a.c.D) return;
#pragma unroll 2
    for (int r = warp; r < w.rows; r += kSoftWarps) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = 0; k0 < w.n; k0 += 4) {
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)  // (past the last one: the last again, not counted)
                x[k] = __ldcg((const float4*)(w.p.part_o + (w.place(min(k0 + k, w.n - 1), N) + r) * 128) + lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k0 + k >= w.n) break;
                add(o, f_sm[(k0 + k) * N + r], x[k]);
            }
        }
        w.row(r, lane, o, f_sm[w.n * N + r], N);
    }
}

template <int NN, int DP, bool Q8>
__global__ void __launch_bounds__(Shape<NN, DP, Q8>::threads, 1) attend_kernel(const __grid_constant__ AttParams p) {
    using X = Shape<NN, DP, Q8>;
    constexpr int N = X::N, MC = X::MC, R = X::segs, QB = X::QB, TM = X::TM, SB = X::SB, PS = X::PS, kAuxRing = X::aux_ring;
    constexpr uint32_t SK = X::SK, SV = X::SV, RV = X::RV;
    constexpr int kAttThreads = X::threads;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const v_sm = smem + SK * X::k_bytes;                // the V ring, after the K ring
    unsigned char* const raw_sm = smem + X::ring_bytes;                // Q8: [RV] V tiles as they are
    unsigned char* const q_sm = raw_sm + X::raw_bytes;
    unsigned char* const p_sm = q_sm + QB * X::q_bytes;                // [PS]
    unsigned char* const aux_sm = p_sm + PS * X::p_bytes;
    float* const mref_all = (float*)(aux_sm + kAuxRing * X::aux_bytes);  // [TM][N] references
    // [TM][N] each: weight sums and factors of the teams, used between segments (tight: in P, free then)
    float* const lsum = X::tight ? (float*)(p_sm + (N / 8 + 4) * 2048) : mref_all + TM * N;
    float* const fac = lsum + TM * N;
    float* const unit_all = fac + TM * N;  // Q8: [TM][N] what a row's weights times V's scales are multiplied by for f16
    float* const arow_all = mref_all + X::state / 4;  // Q8: [R][N] a query row's power of two times scale * log2(e)
    unsigned char* const red_sm = (unsigned char*)(arow_all + (Q8 ? R * N : 0));
    uint32_t* const seen_by = (uint32_t*)(red_sm + (X::tight ? 0 : kGroups * X::red_bytes));  // [T][4] the tokens that see a tree's token
    Seg* const segs = (Seg*)(seen_by + kKvMaxQueries * 4);
    uint32_t* const poison = (uint32_t*)(segs + R);  // [4] new tokens with non-finite values, then:
    volatile uint32_t* const aborted = poison + 4;   // a wait gave up
    uint32_t* const tmem_at = poison + 5;
    uint32_t* const last_in = poison + 6;
    uint32_t* const tree_bad = poison + 7;
    volatile uint32_t* const lost = poison + 9;      // a segment did not come to one of the softmax warps
    uint32_t* const last_seq = poison + 8;           // the last sequence of the run
    uint64_t* const k_full = (uint64_t*)(poison + (X::tight ? 10 : 12));
    uint64_t* const v_full = k_full + SK;
    uint64_t* const k_empty = v_full + SV;
    uint64_t* const v_empty = k_empty + SK;
    uint64_t* const s_full = v_empty + SV;
    uint64_t* const s_empty = s_full + SB;
    uint64_t* const p_full = s_empty + SB;
    uint64_t* const pv_done = p_full + PS;
    uint64_t* const drain = pv_done + PS;
    uint64_t* const q_full = drain + 1;
    uint64_t* const q_empty = q_full + 2;
    uint64_t* const aux_full = q_empty + 2;
    uint64_t* const seg_full = aux_full + kAuxRing;
    uint64_t* const seg_empty = seg_full + R;
    uint64_t* const raw_full = seg_empty + R;       // Q8: [RV]
    uint64_t* const raw_empty = raw_full + RV;

    const KvAttend& a = p.a;
    const KvView& c = a.c;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;

    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint32_t t0 = nanoseconds();
#pragma unroll 1
        while (!mbar_try_wait(bar, parity)) {
            if (*aborted) return false;
            if (nanoseconds() - t0 > kAttWaitNs) *aborted = 1;
        }
        return true;
    };
    // Once a wait has given up, every wait but those for segments returns at once, so that all roles run out in
    // step: the same segments, the same named barriers, whatever the data. A role whose own wait gave up issues no more
    // loads or products and gives no place of a loads' ring back, so that none goes where an earlier one may still be due.
    auto wait_seg = [&](uint64_t* bar, uint32_t parity) -> bool {
        const uint32_t t0 = nanoseconds();
#pragma unroll 1
        while (!mbar_try_wait(bar, parity))
            if (nanoseconds() - t0 > 2 * kAttWaitNs) {
                *aborted = 1;
                return false;
            }
        return true;
    };
    // Tiles of segment s of this CTA (at segs + s % R), by every warp that works on it; none past the last segment or
    // where it did not come. done_seg gives its place back.
    auto tiles_of = [&](uint32_t s) -> int {
        const bool here = wait_seg(seg_full + s % R, (s / R) & 1);
        return __all_sync(0xFFFFFFFFu, here) ? segs[s % R].n : 0;
    };
    // The last loads of a ring have landed (a load under way must not outlive the CTA).
    auto land = [&](uint64_t* full, uint32_t ring, uint32_t loads) {
        if (elect())
#pragma unroll 1
            for (uint32_t t = loads > ring ? loads - ring : 0; t < loads; ++t) wait_seg(full + t % ring, (t / ring) & 1);
        __syncwarp();
    };
    auto done_seg = [&](uint32_t s) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + s % R);
    };

    // ------------------------------------------------- this CTA's run of tiles
    if (tid == 0) {
        for (uint32_t i = 0; i < SK; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, Q8 ? 5 : 1);
        }
        for (uint32_t i = 0; i < SV; ++i) {
            mbar_init(v_full + i, Q8 ? 4 : 1);
            mbar_init(v_empty + i, 1);
        }
        if (Q8)
            for (uint32_t i = 0; i < RV; ++i) {
                mbar_init(raw_full + i, 1);
                mbar_init(raw_empty + i, 4);
            }
        for (int i = 0; i < SB; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, 4 * X::GT);
        }
        for (int i = 0; i < PS; ++i) {
            mbar_init(p_full + i, 4 * X::GT);
            mbar_init(pv_done + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, Q8 ? 4 : 1);
            mbar_init(q_empty + i, 1);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < kAuxRing; ++i) mbar_init(aux_full + i, Q8 ? 4 : 1);
        for (int i = 0; i < R; ++i) {
            mbar_init(seg_full + i, 1);
            mbar_init(seg_empty + i, kSoftWarps + (Q8 ? 2 + 8 : 3));
        }
        *aborted = 0;
        *lost = 0;
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
#pragma unroll 1
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
    const int32_t holders = (c.B + 32 * per_thr - 1) / (32 * per_thr);  // warps with sequences
#pragma unroll 1
    for (int w = 0; w < holders; ++w) {
        const int64_t x = scan[w];
        before += w < warp ? x : 0;
        W += x;
    }
    const int64_t pre = before + incl - mine;
    const int64_t per = divide(W + p.grid - 1, p.grid);
    const int64_t u0 = (int64_t)blockIdx.x * per, u1 = min(u0 + per, W);
    if (u0 < u1 && pre <= u0 && u0 < pre + mine) {
        int64_t at = pre;
        int32_t b = bt0;
#pragma unroll 1
        for (; b + 1 < bt1; ++b) {
            KvSeq s;
            int32_t tiles, nrt;
            const int64_t k = Walk<N>::count(a, b, s, tiles, nrt);
            if (u0 < at + k) break;
            at += k;
        }
        scan[32] = b;
        scan[33] = at;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const int32_t b0 = u0 < u1 ? (int32_t)scan[32] : 0;
    const int64_t base0 = u0 < u1 ? scan[33] : 0;
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_at, 0);
    __syncthreads();  // P's memory is P's from here on

    // A tile's rows lie in boxes of p.box slots (a whole page's, for pages of 16 to 128). Lane j knows the page of box
    // j; one lane issues the loads, in a loop of the whole warp. Past the length or on a page outside the pool the box
    // is one past the pool: zeros. A page's slots past the length come as they are; softmax hides their scores and
    // clears their values.
    const int boxes = kTileTok >> p.box_log;
    auto page_of = [&](const int32_t* table, int32_t pos, int32_t L) {
        int32_t pg = -1;
        if (pos < L) pg = table[c.by_bs.of(pos)];
        return pg >= 0 && pg < c.num_blocks ? pg : c.num_blocks;
    };
    auto bring = [&](const CUtensorMap* map, uint32_t dst, uint64_t* bar, const int32_t* table, int32_t at, int32_t L,
                     int32_t head, int32_t pages) {  // pages: of boxes 0 .. 31, a lane each
        if (elect()) mbar_arrive_expect_tx(bar, kTileTok * (Q8 || DP == 64 ? 128 : 256));
        __syncwarp();
        int32_t sl = at - c.by_bs.of(at) * c.bs;
#pragma unroll 1
        for (int j = 0; j < boxes; ++j) {
            if (j && (j & 31) == 0) pages = page_of(table, at + (j + lane) * p.box, L);
            const int32_t pg = __shfl_sync(0xFFFFFFFFu, pages, j & 31);
            if (elect()) {
                tma_box(dst, map, 0, sl, head, pg, bar);
                if (!Q8 && DP == 128) tma_box(dst + kTileTok * 128, map, 64, sl, head, pg, bar);
            }
            dst += p.box * 128;
            sl += p.box;
            if (sl >= c.bs) sl = 0;
        }
        __syncwarp();
    };
    auto aux_of = [&](uint32_t tile) { return aux_sm + (tile % kAuxRing) * X::aux_bytes; };

    // Registers by role. bf16: 5 groups of four warps start with 96 a thread; softmax (4 groups) goes on with 104, the
    // rest with 64. e4m3: 7 groups with 72; softmax 80, the turning warps (2) 64, the rest 56.
    if (Q8 && warp >= kTurnWarp) {
        fewer_regs<64>();
        const int fw = warp & 3;
        uint32_t kt = 0;
        if (warp < kTurnWarp + 4) {
            // ======================================================== e4m3: queries, scales
            // A K tile is the scores' first operand as it is; the queries are its equal in three e5m2 parts, each
            // the rest's first three bits. A row counts in a power of two that brings its largest element to [2^14,
            // 2^15): the parts hold all 8 bits of what is 2^-24 of it or more, and the rest to 2^-31 of it.
            const float k2 = a.scale * kLog2e;
            constexpr int qc = DP / 8, rpq = 32 / qc;  // 8-element pieces of a row, rows of one load
            static_assert(N / 4 % rpq == 0, "rows of a warp");
            const int piece = lane % qc, sub = lane / qc;
            bool dead = false;
            for (uint32_t si = 0;; ++si) {
                const int n = tiles_of(si);
                if (!n) break;
                const Seg* const g = segs + si % R;
                const int32_t L = g->L, h = g->h, row0 = g->rt * N, rows = min(N, g->T * a.G - row0);
                int32_t pos = g->tile0 * kTileTok + fw * 32 + lane;
                const int32_t* const table = c.table + (int64_t)g->b * c.max_blocks;
                const unsigned char* const q0 = a.q + g->lo * a.q_row_bytes + (int64_t)h * a.G * c.D * 2 + piece * 16;
                done_seg(si);
                int32_t pg = pos < L ? table[c.by_bs.of(pos)] : -1;
                float sk = 0.f, sv = 0.f;
                bool in = false;
                // scales of the row at pos, its page known; on to the next tile's page
                auto scales = [&]() {
                    in = pg >= 0 && pg < c.num_blocks;
                    sk = sv = 0.f;
                    if (in) {
                        const int64_t i = ((int64_t)pg * c.H + h) * c.bs + (pos - c.by_bs.of(pos) * c.bs);
                        sk = c.ks[i];
                        sv = c.vs[i];
                    }
                    pos += kTileTok;
                    pg = pos < L ? table[c.by_bs.of(pos)] : -1;
                };
                scales();
                const uint32_t q_at = smem_addr(q_sm) + (si % QB) * X::q_bytes + (piece & 1) * 8;
                float* const arow = arow_all + (si % R) * N;
                auto load_q = [&](int r) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (r < rows && piece * 8 < c.D) {
                        const int32_t rr = row0 + r, t = a.by_G.of(rr);
                        w = *(const uint4*)(q0 + t * a.q_row_bytes + (int64_t)(rr - t * a.G) * c.D * 2);
                    }
                    return w;
                };
                const int r_end = (fw + 1) * (N / 4);
                int r = fw * (N / 4) + sub;
                uint4 next = load_q(r);
                if (si >= QB) wait(q_empty + si % QB, (si / QB - 1) & 1);
#pragma unroll 1
                for (; r < r_end; r += rpq) {
                    const uint4 w = next;
                    if (r + rpq < r_end) next = load_q(r + rpq);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                    uint32_t m = 0;  // magnitudes compare as integers; what is not finite does not count
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = u[j] & 0x7FFFu, hi = u[j] >> 16 & 0x7FFFu;
                        m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                    }
#pragma unroll
                    for (int o = qc / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                    const int e = m ? max(-126, min(113, (int)(m >> 7) - 127 - 14)) : 0;  // x / 2^e
                    const float f = __uint_as_float((uint32_t)(127 - e) << 23);
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[2 * j] = bf16_lo(u[j]) * f;
                        x[2 * j + 1] = bf16_hi(u[j]) * f;
                        // (an infinity as NaN, as e5m2 conversions saturate: the row's weights are NaN either way)
                        if ((u[j] & 0x7F80u) == 0x7F80u) x[2 * j] = __uint_as_float(0x7FC00000u);
                        if ((u[j] & 0x7F800000u) == 0x7F800000u) x[2 * j + 1] = __uint_as_float(0x7FC00000u);
                    }
#pragma unroll 1
                    for (int part = 0; part < 3; ++part) {
                        uint32_t b[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            b[j] = e5m2x2(x[2 * j], x[2 * j + 1]);
                            // an e5m2 number is the first byte of the fp16 one
                            x[2 * j] -= __half2float(__ushort_as_half((unsigned short)(b[j] << 8)));
                            x[2 * j + 1] -= __half2float(__ushort_as_half((unsigned short)(b[j] & 0xFF00u)));
                        }
                        asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(q_at + (part * N + r) * 128 + (((piece >> 1) ^ r) & 7) * 16),
                                     "r"(b[0] | b[1] << 16), "r"(b[2] | b[3] << 16)
                                     : "memory");
                    }
                    if (piece == 0) arow[r] = k2 * __uint_as_float((uint32_t)(127 + e) << 23);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full + si % QB);
#pragma unroll 1
                for (int t = 0; t < n; ++t, ++kt) {
                    const uint32_t slot = kt % SK;
                    // in step with the K ring, so that the scales' is not overrun
                    if (!wait(k_full + slot, (kt / SK) & 1)) dead = true;
                    unsigned char* const aux = aux_of(kt);
                    const uint32_t bits = __ballot_sync(0xFFFFFFFFu, in);
                    if (lane == 0) ((uint32_t*)aux)[fw] = bits;
                    ((float*)(aux + 16))[fw * 32 + lane] = sk;
                    ((float*)(aux + 16))[kTileTok + fw * 32 + lane] = sv;
                    __syncwarp();
                    if (lane == 0) {
                        if (!dead) mbar_arrive(k_empty + slot);
                        mbar_arrive(aux_full + kt % kAuxRing);
                    }
                    if (t + 1 < n) scales();
                }
            }
        } else {
            // ======================================================== e4m3: V to f16
            // Exactly, 32 rows to a warp, from a tile as it is to the V ring.
            const uint32_t raw = smem_addr(raw_sm) + fw * 32 * 128;
            constexpr int chunks = DP / 16, rpr = 32 / chunks;  // 16-byte units of a row, rows of a warp's access
            const int my_chunk = lane % chunks, my_row = lane / chunks;
            // where this lane's unit of row `my_row + r * rpr` goes in a V tile: an exclusive or and an offset away from
            // row my_row's, as 16-byte units are exchanged within a row by its row's number
            const uint32_t at0 = smem_addr(v_sm) + fw * 32 * 128 + (my_chunk >> 2) * (kTileTok * 128) + my_row * 128 +
                                 ((2 * my_chunk ^ my_row) & 7) * 16;
            auto swizzled = [&](uint32_t base, int r, int more) { return (base ^ ((((r * rpr) & 7) ^ more) * 16)) + r * rpr * 128; };
            bool dead = false;
            for (uint32_t si = 0;; ++si) {
                const int n = tiles_of(si);
                if (!n) break;
                done_seg(si);
#pragma unroll 1
                for (int t = 0; t < n; ++t, ++kt) {
                    const uint32_t from = kt % RV, slot = kt % SV;
                    if (!wait(raw_full + from, (kt / RV) & 1)) dead = true;
                    const uint32_t base = at0 + slot * X::slot_bytes;
                    auto unit_at = [&](int r) {
                        const int row = r * rpr + my_row;
                        return lds16(raw + from * X::raw_tile + row * 128 + ((my_chunk ^ row) & 7) * 16);
                    };
                    // (a short loop, two units at a time and the next two on their way: straight code of this length
                    // waits for its own instructions)
                    uint4 x = unit_at(0), y = unit_at(1);
                    if (kt >= SV) wait(v_empty + slot, (kt / SV - 1) & 1);
#pragma unroll 1
                    for (int r = 0; r < chunks; r += 2) {
                        const uint4 u[2] = {x, y};
                        if (r + 2 < chunks) {
                            x = unit_at(r + 2);
                            y = unit_at(r + 3);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            sts16(swizzled(base, r + i, 0), make_uint4(e4m3_f16x2(u[i].x & 0xFFFF), e4m3_f16x2(u[i].x >> 16),
                                                                       e4m3_f16x2(u[i].y & 0xFFFF), e4m3_f16x2(u[i].y >> 16)));
                            sts16(swizzled(base, r + i, 1), make_uint4(e4m3_f16x2(u[i].z & 0xFFFF), e4m3_f16x2(u[i].z >> 16),
                                                                       e4m3_f16x2(u[i].w & 0xFFFF), e4m3_f16x2(u[i].w >> 16)));
                        }
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (!dead) mbar_arrive(raw_empty + from);
                        mbar_arrive(v_full + slot);
                    }
                }
            }
        }
    } else if (warp >= kMmaWarp) {
        fewer_regs<Q8 ? 56 : 64>();
        if (warp == kMmaWarp) {
        // ============================================================ products
        constexpr uint32_t id_qk = Q8 ? instr_desc_f8(N) : instr_desc(true, false, false, N);
        constexpr uint32_t id_pv = instr_desc(!Q8, true, true, X::NP);
        const uint64_t k_desc = operand(smem_addr(smem), 16, 1024, 2);
        const uint64_t v_desc = operand(smem_addr(v_sm), DP == 128 ? kTileTok * 128 : 0, 1024, 2);
        const uint64_t p_desc = operand(smem_addr(p_sm), 128, 2048, 0);
        const uint64_t q_desc = operand(smem_addr(q_sm), 16, 1024, 2);
        // Scores run ahead of the weights' products, over segments' ends too, as far as there is room in TMEM: two
        // cursors over the segments.
        uint32_t qs = 0, qt = 0, ks = 0, kr = 0, vs = 0, vr = 0;  // segment, tile, ring places and rounds
        int qi = 0, qn = -1;
        bool dead = false;
        auto count_of = [&](uint32_t seg) { return __shfl_sync(0xFFFFFFFFu, tiles_of(seg), 0); };
        auto scores = [&]() {  // of the next tile, if there is one
            if (qn == 0) return;
            if (qi >= qn) {
                qn = count_of(qs);
                if (!qn) return;
                qi = 0;
                if (!wait(q_full + qs % QB, (qs / QB) & 1)) dead = true;
            }
            const uint32_t buf = qt % SB;
            if (!wait(k_full + ks, kr & 1)) dead = true;
            if (qt >= SB) wait(s_empty + buf, (qt / SB - 1) & 1);
            tc_after();
            ++qi;
            if (elect() && !dead) {
                const uint64_t ka = k_desc + ks * (X::k_bytes >> 4);
                const uint64_t qd = q_desc + (qs % QB) * (X::q_bytes >> 4);
                const uint32_t d = tmem + buf * N;
                if constexpr (Q8) {
#pragma unroll
                    for (int part = 0; part < 3; ++part)
#pragma unroll
                        for (int k = 0; k < DP / 32; ++k)
                            tc_mma_f8(d, ka + (k * 32 >> 4), qd + ((part * N * 128 + k * 32) >> 4), id_qk, part + k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        tc_mma(d, ka + (((k >> 2) * (kTileTok * 128) + (k & 3) * 32) >> 4),
                               qd + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), id_qk, k > 0);
                }
                tc_commit(k_empty + ks);
                tc_commit(s_full + buf);
                if (qi == qn) tc_commit(q_empty + qs % QB);
            }
            __syncwarp();
            if (qi == qn) ++qs;
            ++qt;
            if (++ks == SK) ks = 0, ++kr;
        };
        uint32_t t = 0;
#pragma unroll 1
        for (int i = 0; i < TM; ++i) scores();
        for (uint32_t si = 0;; ++si) {
            const int n = count_of(si);
            if (!n) break;
            done_seg(si);  // at once: the cursor ahead, which has read it, may have to wait for its place
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++t) {
                const uint32_t team = t % TM, ps = t % PS;
                if (TM == 1) scores();
                if (!wait(v_full + vs, vr & 1)) dead = true;
                if (!wait(p_full + ps, (t / PS) & 1)) dead = true;
                tc_after();
                if (elect() && !dead) {
                    const uint64_t va = v_desc + vs * (X::slot_bytes >> 4), pd = p_desc + ps * (X::p_bytes >> 4);
                    const uint32_t d = tmem + X::O_at + team * X::NP;
#pragma unroll
                    for (int k = 0; k < kTileTok / 16; ++k)
                        tc_mma(d, va + ((k * 2048) >> 4), pd + ((k * 256) >> 4), id_pv, k > 0 || i >= TM);
                    tc_commit(v_empty + vs);
                    tc_commit(pv_done + ps);
                }
                __syncwarp();
                if (++vs == SV) vs = 0, ++vr;
                if (TM > 1) scores();
            }
        }
        if (elect()) {
            tc_commit(drain);  // everything issued here is done before TMEM is freed
            wait_seg(drain, 0);
        }
        __syncwarp();
    } else if (warp == kQueryWarp) {
        // ============================================================ queries
        // Row tiles of queries, a segment ahead where there is room for two (e4m3: see above).
        constexpr int qc = DP / 8, rpq = 32 / qc;  // 16-byte pieces of a row, rows of one load
        const int piece = lane % qc, sub = lane / qc;
        for (uint32_t si = 0; !Q8; ++si) {
            if (!tiles_of(si)) break;
            const Seg* const g = segs + si % R;
            const int32_t row0 = g->rt * N, rows = min(N, g->T * a.G - row0);
            const unsigned char* const q0 = a.q + g->lo * a.q_row_bytes + (int64_t)g->h * a.G * c.D * 2 + piece * 16;
            auto row_of = [&](int r) {
                const int32_t rr = row0 + r, t = a.by_G.of(rr);
                return q0 + t * a.q_row_bytes + (int64_t)(rr - t * a.G) * c.D * 2;
            };
            if (QB == 1)  // into L2 while the last products still need the place
#pragma unroll 1
                for (int r = lane; r < rows; r += 32)
#pragma unroll
                    for (int d = 0; d < DP / 64; ++d)
                        if (d * 64 < c.D) asm volatile("prefetch.global.L2 [%0];" ::"l"(row_of(r) + d * 128 - piece * 16));
            if (si >= QB) wait(q_empty + si % QB, (si / QB - 1) & 1);
            const uint32_t q_at = smem_addr(q_sm) + (si % QB) * X::q_bytes + (piece >> 3) * (N * 128);
#pragma unroll 8
            for (int r = sub; r < N; r += rpq) {
                const bool in = r < rows && piece * 8 < c.D;
                cp16(q_at + r * 128 + ((piece ^ r) & 7) * 16, in ? row_of(r) : a.q, in ? 16u : 0u);
            }
            cp_wait_all();
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + si % QB);
            done_seg(si);
        }
    } else if (warp == kSegWarp) {
        // ============================================================ segments, K
        Walk<N> walk(a, u0, u1, per, b0, base0);
        if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&p.k_map) : "memory");
        uint32_t kt = 0, loads = 0;  // (loads: fewer than tiles after a wait that gave up)
        for (uint32_t s = 0;; ++s) {
            Seg g;
            walk.next(g);
            // (a place that does not come free: no more segments, and those who wait for them give up in their turn)
            if (s >= R && !__all_sync(0xFFFFFFFFu, wait_seg(seg_empty + s % R, (s / R - 1) & 1))) {
                if (lane == 0) *last_seq = (uint32_t)(c.B - 1);  // the run's end is not known
                break;
            }
            if (lane == 0) {
                segs[s % R] = g;
                *last_seq = (uint32_t)min(walk.b, c.B - 1);
                mbar_arrive(seg_full + s % R);
            }
            if (!g.n) break;
            const int n = __shfl_sync(0xFFFFFFFFu, g.n, 0);
            const int32_t* const table = c.table + (int64_t)g.b * c.max_blocks;
            int32_t at = g.tile0 * kTileTok;
            int32_t next = page_of(table, at + lane * p.box, g.L);
#pragma unroll 1
            for (int t = 0; t < n; ++t, ++kt, at += kTileTok) {
                const int32_t pages = next;
                if (t + 1 < n) next = page_of(table, at + kTileTok + lane * p.box, g.L);
                const uint32_t slot = kt % SK;
                const bool free = kt < SK || wait(k_empty + slot, (kt / SK - 1) & 1);
                if (__all_sync(0xFFFFFFFFu, free && loads == kt)) {
                    bring(&p.k_map, smem_addr(smem) + slot * X::k_bytes, k_full + slot, table, at, g.L, g.h, pages);
                    ++loads;
                }
                if constexpr (!Q8) {
                    // which positions are there
                    uint32_t* const aux = (uint32_t*)aux_of(kt);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int32_t r = w * 32 + lane;
                        int32_t pg = __shfl_sync(0xFFFFFFFFu, pages, (r >> p.box_log) & 31);
                        if (boxes > 32) pg = page_of(table, at + r, g.L);
                        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, pg < c.num_blocks && at + r < g.L);
                        if (lane == 0) aux[w] = bits;
                    }
                    if (lane == 0) mbar_arrive(aux_full + kt % kAuxRing);
                }
            }
        }
        land(k_full, SK, loads);
    } else if (warp == kValueWarp) {
        // ============================================================ V, statuses
        // A sequence's status: its offsets, length, tree and pages; the rows of
        // a sequence with an error become zeros. One after each segment.
        if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&p.v_map) : "memory");
        int32_t next_b = blockIdx.x;
        auto check_one = [&]() {
            const int32_t b = next_b;
            next_b += p.grid;
            const KvSeq s = kv_seq(b, a.row_off, a.t_max, a.rows, a.kv_lens, c.bs, c.max_blocks, true);
            int32_t st = s.st;
            bool bad = false;
            if (st == kKvOk && a.parent)
#pragma unroll 1
                for (int32_t v = lane; v < s.T; v += 32) {
                    const int32_t u = a.parent[s.lo + v];
                    bad |= v == 0 ? u != -1 : (u < 0 || u >= v);
                }
            if (__any_sync(0xFFFFFFFFu, bad)) st = kKvBadLayout;
            if (st != kKvOk && s.lo >= 0) {
                const int64_t m = (int64_t)s.T * a.Hq * c.D, o = s.lo * a.Hq * c.D;  // head_dim is a multiple of 8
#pragma unroll 1
                for (int64_t i = (int64_t)lane * 8; i < m; i += 256) *(uint4*)(a.out + (o + i) * 2) = make_uint4(0, 0, 0, 0);
                if (a.lse)
#pragma unroll 1
                    for (int64_t i = lane; i < (int64_t)s.T * a.Hq; i += 32)
                        a.lse[s.lo * a.Hq + i] = __uint_as_float(0xFF800000u);
            }
            if (a.seq_status) {
                if (st == kKvOk) {
                    bad = false;
                    if (s.T > 0)
#pragma unroll 1
                        for (int32_t j = lane; j <= c.by_bs.of(s.L - 1); j += 32) {
                            const int32_t pg = c.table[(int64_t)b * c.max_blocks + j];
                            bad |= pg < 0 || pg >= c.num_blocks;
                        }
                    if (__any_sync(0xFFFFFFFFu, bad)) st = kKvBadLayout;
                }
                if (lane == 0) a.seq_status[b] = st;
            }
        };
        uint32_t kt = 0, si = 0, loads = 0;
        for (bool open = true; open || next_b < c.B;) {
            if (open) {
                const Seg* const g = segs + si % R;
                const int n = __shfl_sync(0xFFFFFFFFu, tiles_of(si), 0);
                open = n != 0;
                if (open) {
                    const int32_t L = g->L, h = g->h;
                    int32_t at = g->tile0 * kTileTok;
                    const int32_t* const table = c.table + (int64_t)g->b * c.max_blocks;
                    done_seg(si++);
                    int32_t next = page_of(table, at + lane * p.box, L);
#pragma unroll 1
                    for (int t = 0; t < n; ++t, ++kt, at += kTileTok) {
                        const int32_t pages = next;
                        if (t + 1 < n) next = page_of(table, at + kTileTok + lane * p.box, L);
                        if constexpr (Q8) {
                            const uint32_t slot = kt % RV;
                            const bool free = kt < RV || wait(raw_empty + slot, (kt / RV - 1) & 1);
                            if (__all_sync(0xFFFFFFFFu, free && loads == kt)) {
                                bring(&p.v_map, smem_addr(raw_sm) + slot * X::raw_tile, raw_full + slot, table, at, L, h, pages);
                                ++loads;
                            }
                        } else {
                            const uint32_t slot = kt % SV;
                            const bool free = kt < SV || wait(v_empty + slot, (kt / SV - 1) & 1);
                            if (__all_sync(0xFFFFFFFFu, free && loads == kt)) {
                                bring(&p.v_map, smem_addr(v_sm) + slot * X::slot_bytes, v_full + slot, table, at, L, h, pages);
                                ++loads;
                            }
                        }
                    }
                }
            }
            if (next_b < c.B) check_one();
        }
        if constexpr (Q8)
            land(raw_full, RV, loads);
        else
            land(v_full, SV, loads);
        }
    } else {
        more_regs<Q8 ? 80 : 104>();
        // ============================================================ softmax
        // Thread = one position of the tile; group gr is of team gr % TM and has
        // every GT-th 8-row piece of the query rows. A weight is 2^(score - m) with m a
        // reference that starts as the row's maximum in its first tile and moves
        // only when a later score passes it by 2^grow. bf16: 2^16, as what the weights have above one the sums lose of
        // float32's range to values (with 2^60 values of 2^67 overflowed; moves are as rare, and no case took longer).
        // e4m3: 2^8; a weight goes to f16 times V's scale and the row's unit u = 2^(6 - v), 2^v the smallest power of
        // two that no scale the row has seen passes: at most 2^14 (f16's largest is 2^16), and f16's least is 2^-30 of
        // a weight of one with that scale. The unit is a row's own, so that the scale of a new token that the row does
        // not see leaves no trace in it.
        const int gr = warp >> 2, wq = warp & 3, wt = tid & 127;
        const int bar_gr = 1 + gr;
        constexpr int bar_all = 1 + kGroups;
        constexpr float grow = Q8 ? 8.f : 16.f;
        const uint32_t lanes = (uint32_t)wq << 21;  // this warp's 32 TMEM lanes
        const uint32_t team = gr % TM, sub = gr / TM;
        const uint32_t o_at = tmem + X::O_at + lanes + team * X::NP;
        unsigned char* const pw0 = p_sm + (wt >> 3) * 128 + (wt & 7) * 16;  // this thread's P, piece 0
        float* const mref = mref_all + team * N;
        float* const unit = unit_all + team * N;
        constexpr float first_unit = 0x1p106f;  // v = -100
        // the group's scratch [5][MC * 8]: its own, or in its second part of P while P is free
        float* const red = (float*)(X::tight ? p_sm + (N / 8 + gr) * 2048 : red_sm + gr * X::red_bytes);
        const float k2 = a.scale * kLog2e;
        const float none = __uint_as_float(0xFF800000u);
        // eight sums over the warp, lane's the one of value lane >> 2, by halving what a lane holds
        auto over_warp = [&](float (&x)[8]) {
#pragma unroll
            for (int h = 4; h; h >>= 1) {
                const bool hi = lane & (4 * h);
#pragma unroll
                for (int k = 0; k < h; ++k)
                    x[k] = (hi ? x[k + h] : x[k]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? x[k] : x[k + h], 4 * h);
            }
            x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], 2);
            return x[0] + __shfl_xor_sync(0xFFFFFFFFu, x[0], 1);
        };
        uint32_t gt = 0;
        int32_t tree_of = -1;  // the sequence whose ancestors are known
        for (uint32_t si = 0;; ++si) {
            const bool here = wait_seg(seg_full + si % R, (si / R) & 1);
            // ---- per-row state
            if (tid < TM * N) mref_all[tid] = kNoMax;
            if (!X::tight && tid < TM * N) lsum[tid] = 0.f;  // of a team without a tile here
            if (Q8 && tid < TM * N) unit_all[tid] = first_unit;
            if (tid < 4) poison[tid] = 0;
            // (all of them go on or none does: they meet at barriers)
            if (!here) *lost = 1;
            bar_sync(bar_all, kSoftThreads);
            const Seg* const g = segs + si % R;
            const int n = *lost ? 0 : g->n;
            if (!n) break;
            const int32_t T = g->T, L = g->L, row0 = g->rt * N, ctx = L - T;
            const int32_t rows = min(N, T * a.G - row0);
            const int pieces = (rows + 7) / 8;
            const int live = (int)sub < pieces ? (pieces - (int)sub + X::GT - 1) / X::GT : 0;  // this group's pieces
            const float* const arow = arow_all + (si % R) * N;
            if (a.parent && g->b != tree_of) {
                tree_of = g->b;
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
                    *(uint4*)(seen_by + tid * 4) = make_uint4(m[0], m[1], m[2], m[3]);
                    jumps[tid] = (uint32_t)jump;
                }
                const bool any = bar_or(bar_all, kSoftThreads, bad);
                if (tid == 0) *tree_bad = any;
#pragma unroll 1
                for (int reach = 1; reach < T; reach <<= 1) {
                    uint4 up = make_uint4(0, 0, 0, 0);
                    int32_t far = -1;
                    if (jump >= 0) {
                        up = *(const uint4*)(seen_by + jump * 4);
                        far = (int32_t)jumps[jump];
                    }
                    bar_sync(bar_all, kSoftThreads);
                    if (jump >= 0) {
                        m[0] |= up.x, m[1] |= up.y, m[2] |= up.z, m[3] |= up.w;
                        *(uint4*)(seen_by + tid * 4) = make_uint4(m[0], m[1], m[2], m[3]);
                        jumps[tid] = (uint32_t)far;
                    }
                    jump = far;
                    bar_sync(bar_all, kSoftThreads);
                }
                // and turned round: those that a token's entry is seen by, which is what a position's thread asks for
                if (tid < kKvMaxQueries) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j * 32 >= T) break;
                        uint32_t by = 0;
#pragma unroll 4
                        for (int k = 0; k < 32; ++k) {
                            const uint32_t x = __ballot_sync(0xFFFFFFFFu, m[j] >> k & 1);
                            if (lane == k) by = x;
                        }
                        seen_by[(j * 32 + lane) * 4 + warp] = by;
                    }
                }
                bar_sync(bar_all, kSoftThreads);
            }
            float2 l[MC][4];
#pragma unroll
            for (int m = 0; m < MC; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) l[m][k] = make_float2(0.f, 0.f);

            // Q8: the rows' unit, which is one where every row sees every position: rows part only over new tokens, and no
            // tile without those comes after them
            float u_all = first_unit;
            const int first = (int)((team - gt) & (TM - 1));  // this team's first tile of the segment
#pragma unroll 1
            for (int i = first; i < n; i += TM) {
                const uint32_t t = gt + i, buf = t % SB, ps = t % PS, turn = t / PS;
                unsigned char* const pw = pw0 + ps * X::p_bytes;
                if (live) {
                    wait(aux_full + t % kAuxRing, (t / kAuxRing) & 1);
                    const unsigned char* aux = aux_sm + (t % kAuxRing) * X::aux_bytes;
                    const bool in = ((const uint32_t*)aux)[wq] >> lane & 1;
                    const float ks = Q8 ? ((const float*)(aux + 16))[wt] : 1.f;
                    const float vs = Q8 ? ((const float*)(aux + 16))[kTileTok + wt] : 1.f;
                    const int32_t pos0 = (g->tile0 + i) * kTileTok, pos = pos0 + wt;
                    const uint32_t s_at = tmem + buf * N + lanes + sub * 8;
                    const bool tail = pos0 + kTileTok > ctx;
                    // rows that see this position (a bit for each of the group's rows), where not every row sees
                    // every one; a page outside the pool hides positions anywhere
                    using Rows = typename std::conditional<(MC > 4), uint64_t, uint32_t>::type;  // a bit for each
                    static_assert(MC * 8 <= 8 * (int)sizeof(Rows), "a bit for each row of the group");
                    Rows vis = in ? ~(Rows)0 : (Rows)0;
                    if (tail && in && pos >= ctx) {
                        const int32_t u = pos - ctx;
                        vis = 0;
#pragma unroll 1
                        for (int m = 0; m < live; ++m) {
                            const int32_t r = row0 + (sub + X::GT * m) * 8, tk = a.by_G.of(r), w = tk >> 5;
                            int32_t left = (tk + 1) * a.G - r;  // rows of token tk from here
                            uint32_t see;                       // tokens tk, tk + 1, ..
                            if (a.parent)
                                see = __funnelshift_r(w < 4 ? seen_by[u * 4 + w] : 0, w < 3 ? seen_by[u * 4 + w + 1] : 0, tk & 31);
                            else
                                see = tk >= u ? ~0u : u - tk >= 8 ? 0u : ~0u << (u - tk);
                            uint32_t bits = 0;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                bits |= (see & 1) << k;
                                if (--left == 0) left = a.G, see >>= 1;
                            }
                            vis |= (Rows)bits << (m * 8);
                        }
                    }
                    const bool masked = tail || __any_sync(0xFFFFFFFFu, !in);
                    wait(s_full + buf, (t / SB) & 1);
                    tc_after();

                    // scores of piece m less the reference, in units of log2; from zero, for the reference, rounded down, so
                    // that the largest one's weight is no less than one however far from zero it lies (rounded to nearest,
                    // a row's only weight was 2^-128 and less from scores of 2^31 on)
                    auto relative = [&](int m, float2 (&z)[4], bool from_zero) {
                        const int r = (sub + X::GT * m) * 8;
                        float2 f[4];
                        if (Q8) {
                            const float4 a0 = *(const float4*)(arow + r), a1 = *(const float4*)(arow + r + 4);
                            f[0] = {a0.x, a0.y}, f[1] = {a0.z, a0.w}, f[2] = {a1.x, a1.y}, f[3] = {a1.z, a1.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) f[k] = mul2(f[k], make_float2(ks, ks));
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) f[k] = make_float2(k2, k2);
                        }
                        if (from_zero) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) z[k] = make_float2(__fmul_rd(z[k].x, f[k].x), __fmul_rd(z[k].y, f[k].y));
                        } else {
                            const float4 m0 = *(const float4*)(mref + r), m1 = *(const float4*)(mref + r + 4);
                            const float2 x[4] = {{-m0.x, -m0.y}, {-m0.z, -m0.w}, {-m1.x, -m1.y}, {-m1.z, -m1.w}};
#pragma unroll
                            for (int k = 0; k < 4; ++k) z[k] = fma2(z[k], f[k], x[k]);
                        }
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                z[k].x = (vis >> (m * 8 + 2 * k) & 1) ? z[k].x : none;
                                z[k].y = (vis >> (m * 8 + 2 * k + 1) & 1) ? z[k].y : none;
                            }
                        }
                    };
                    // the references to the maxima of this tile and before, the sums after them
                    // (Q8: and the units to the scales seen)
                    auto refer = [&]() {
                        unsigned char* const seen_e = (unsigned char*)(red + 5 * MC * 8);  // Q8: [4][MC * 8] 127 + exponents
                        static_assert(!Q8 || MC <= 4, "a lane for each row of the group");
                        const uint32_t vw = __float_as_uint(fabsf(vs));
                        // of the smallest power of two not below this position's scale, 0 to 253 (no scale, 2^126 or more)
                        const uint32_t e = min(253u, (vw >> 23) + ((vw & 0x7FFFFFu) ? 1u : 0u));
#pragma unroll 1
                        for (int m = 0; m < live; ++m) {
                            float2 z[4];
                            tc_ld8(s_at + X::GT * m * 8, z);
                            tc_wait_ld(z);
                            relative(m, z, true);
                            const float y[8] = {z[0].x, z[0].y, z[1].x, z[1].y, z[2].x, z[2].y, z[3].x, z[3].y};
                            float x = 0.f;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float top = max_warp(y[k]);
                                x = lane == k ? top : x;
                            }
                            if (lane < 8) red[wq * MC * 8 + m * 8 + lane] = x;
                        }
                        if (Q8) {
                            const uint32_t row_e = masked ? seen_max(e, (uint32_t)vis, ~0u >> (32 - live * 8))
                                                          : __reduce_max_sync(0xFFFFFFFFu, e);
                            if (lane < MC * 8) seen_e[wq * MC * 8 + lane] = (unsigned char)row_e;
                        }
                        bar_sync(bar_gr, 128);
                        if (wt < live * 8) {
                            const int r = (sub + X::GT * (wt >> 3)) * 8 + (wt & 7);
                            const float old = mref[r];
                            float m = old;
#pragma unroll
                            for (int w = 0; w < 4; ++w) m = larger(red[w * MC * 8 + wt], m);
                            const float f = ex2(old - m);
                            red[4 * MC * 8 + wt] = f;
                            mref[r] = m;
                            if (Q8) {
                                // exponents as they are held: the unit's is 127 + 6 - v
                                const uint32_t at = 260 - (__float_as_uint(unit[r]) >> 23);
                                uint32_t to = at;
#pragma unroll
                                for (int w = 0; w < 4; ++w) to = max(to, (uint32_t)seen_e[w * MC * 8 + wt]);
                                unit[r] = __uint_as_float((260 - to) << 23);
                                // the sums shrink with it
                                red[wt] = to - at > 126 ? 0.f : f * __uint_as_float((127 - (to - at)) << 23);
                            }
                        }
                        bar_sync(bar_gr, 128);
                        if (Q8) u_all = unit[sub * 8];
                        if (i != first) {
                            if (PS != TM) {
                                wait(pv_done + (t - 1) % PS, ((t - 1) / PS) & 1);
                                tc_after();
                            }
#pragma unroll
                            for (int m = 0; m < MC; ++m)
                                if (m < live)
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        l[m][k] = mul2(l[m][k], *(const float2*)(red + 4 * MC * 8 + m * 8 + 2 * k));
#pragma unroll 1
                            for (int m = 0; m < live; ++m)
#pragma unroll 1
                                for (int part = 0; part < (Q8 ? 1 : 2); ++part) {
                                    float o[8];
                                    const uint32_t at = o_at + part * N + (sub + X::GT * m) * 8;
                                    tc_ld8(at, o);
                                    tc_wait_ld(o);
#pragma unroll
                                    for (int k = 0; k < 8; ++k) o[k] *= red[(Q8 ? 0 : 4 * MC * 8) + m * 8 + k];
                                    tc_st8(at, o);
                                }
                            tc_wait_st();
                        }
                        bar_sync(bar_gr, 128);  // the scratch may be P again
                    };
                    if (turn) wait(pv_done + ps, (turn - 1) & 1);  // P is free, and O where P is one for each team
                    tc_after();
                    // ---- weights. When a score passes the reference by too much, they leave the row sums again
                    // (exactly enough: what rounding leaves behind is within an ulp of that score's weight), the
                    // reference moves, and they are made anew.
                    bool moved = false, due = i == first;
#pragma unroll 1
                    for (float sign = 1.f;;) {
                        if (due) refer();
                        due = false;
                        float top = none;
                        const float wv = Q8 ? vs * u_all : 1.f;
                        // units have to move where a scale passes the common one, or a weight in its row's unit passes 2^14
                        // or is not a number (zero times a unit times a scale past float32's range)
                        float big = Q8 && !masked && fabsf(wv) > 64.f && u_all > 0x1p-120f ? 65536.f : 0.f;  // (it goes no lower)
                        // two pieces at a time, so that one's latencies hide the other's
#pragma unroll
                        for (int m0 = 0; m0 < MC; m0 += 2) {
                            if (m0 >= live) break;
                            float2 zb[2][4];
#pragma unroll
                            for (int d = 0; d < 2; ++d)
                                if (m0 + d < MC) tc_ld8(s_at + X::GT * (m0 + d < live ? m0 + d : m0) * 8, zb[d]);
#pragma unroll
                            for (int d = 0; d < 2; ++d)
                                if (m0 + d < MC) tc_wait_ld(zb[d]);
#pragma unroll
                            for (int d = 0; d < 2; ++d) {
                                const int m = m0 + d;
                                if (m >= MC) continue;
                                float2(&z)[4] = zb[d];
                                const int piece = sub + X::GT * (m < live ? m : m0);  // (a piece that is not there: the other again)
                                relative(m < live ? m : m0, z, false);
                                float high = max3(z[0].x, z[0].y, z[1].x);
                                high = max3(high, z[1].y, z[2].x);
                                high = max3(high, z[2].y, z[3].x);
                                top = max3(top, high, z[3].y);
                                // sums stay finite until the reference moves
#pragma unroll
                                for (int k = 0; k < 4; ++k) z[k] = make_float2(min_nan(z[k].x, grow), min_nan(z[k].y, grow));
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    z[k] = make_float2(ex2(z[k].x), ex2(z[k].y));
                                    l[m][k] = fma2(make_float2(sign, sign), z[k], l[m][k]);
                                }
                                if (Q8) {
                                    if (!masked) {
#pragma unroll
                                        for (int k = 0; k < 4; ++k) z[k] = mul2(z[k], make_float2(wv, wv));
                                    } else {
                                        const float4 u0 = *(const float4*)(unit + piece * 8), u1 = *(const float4*)(unit + piece * 8 + 4);
                                        const float2 u[4] = {{u0.x, u0.y}, {u0.z, u0.w}, {u1.x, u1.y}, {u1.z, u1.w}};
#pragma unroll
                                        for (int k = 0; k < 4; ++k) {
                                            const int at = (m < live ? m : m0) * 8 + 2 * k;
                                            z[k] = mul2(z[k], mul2(make_float2(vs, vs), u[k]));
                                            z[k].x = (vis >> at & 1) ? z[k].x : 0.f;
                                            z[k].y = (vis >> (at + 1) & 1) ? z[k].y : 0.f;
                                            big = larger3(big, z[k].x, z[k].y);
                                        }
                                    }
                                    *(uint4*)(pw + piece * 2048) = make_uint4(f16x2(z[0].x, z[0].y), f16x2(z[1].x, z[1].y),
                                                                              f16x2(z[2].x, z[2].y), f16x2(z[3].x, z[3].y));
                                } else {
                                    // two bf16 parts: 16 bits of the weight
                                    uint32_t w[4];
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        w[k] = bf16x2(z[k].x, z[k].y);
                                        z[k] = sub2(z[k], make_float2(bf16_lo(w[k]), bf16_hi(w[k])));
                                    }
                                    *(uint4*)(pw + piece * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
                                    *(uint4*)(pw + (N / 8 + piece) * 2048) =
                                        make_uint4(bf16x2(z[0].x, z[0].y), bf16x2(z[1].x, z[1].y), bf16x2(z[2].x, z[2].y),
                                                   bf16x2(z[3].x, z[3].y));
                                }
                            }
                        }
                        if (sign < 0.f) {
                            bar_sync(bar_gr, 128);
                            due = moved = true;
                            sign = 1.f;
                            continue;
                        }
                        // (after a move nothing passes the reference, so that a second one is never due)
                        if (i == first || moved || !bar_or(bar_gr, 128, top > grow || !(big <= 16384.f))) break;
                        sign = -1.f;
                    }
                    if (tail && sub == 0 && (pos >= L || (in && pos >= ctx && T > 1))) {
                        // The values of a page's slots past the length are cleared. A new token's values that are not
                        // finite would reach rows that do not see it (0 * inf): they leave the tile here and join the
                        // rows that do see it at the end.
                        // (The last tile's product first: before it the ring may be two rounds behind, and a round two
                        // behind looks done.)
                        if (TM > 1 && t) wait(pv_done + (t - 1) % PS, ((t - 1) / PS) & 1);
                        wait(v_full + t % SV, (t / SV) & 1);
                        unsigned char* const v_row = v_sm + t % SV * X::slot_bytes + wt * 128;
                        constexpr uint32_t ex = Q8 ? 0x7C00u : 0x7F80u;
                        bool found = false;
#pragma unroll 1
                        for (int k = 0; k < DP / 8; ++k) {
                            uint4* const at = (uint4*)(v_row + (k >> 3) * (kTileTok * 128) + (k & 7) * 16);
                            if (pos >= L) {
                                *at = make_uint4(0, 0, 0, 0);
                                continue;
                            }
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
                        wait(s_full + buf, (t / SB) & 1);
                        if (turn) wait(pv_done + ps, (turn - 1) & 1);
                    }
                    mbar_arrive(s_empty + buf);
                    mbar_arrive(p_full + ps);
                }
            }
            gt += n;

            // ---- the segment's sums
            const bool whole = n == g->tiles;
            const bool skip = a.parent && *tree_bad;  // its rows are zeros, written with the statuses
            const int64_t part = (int64_t)blockIdx.x * 2 + (g->tile0 == 0 ? 1 : 0);
            auto out_row = [&](int r) {
                const int32_t rr = row0 + r, tk = a.by_G.of(rr);
                return (g->lo + tk) * a.Hq + (int64_t)g->h * a.G + (rr - tk * a.G);
            };
            // the last product of a team with a tile here
            auto finished = [&](uint32_t tm) {
                const int f = (int)((tm - (gt - n)) & (TM - 1));
                const uint32_t last = gt - n + f + (n - 1 - f) / TM * TM;
                if (f < n) wait(pv_done + last % PS, (last / PS) & 1);
                return f < n;
            };
            if (X::tight) finished(0);  // the scratch is P's
            if (live && first < n) {
                // each row's weights over the 128 positions: a warp's 32 by halving the rows a lane holds
#pragma unroll
                for (int m = 0; m < MC; ++m)
                    if (m < live) {
                        float x[8] = {l[m][0].x, l[m][0].y, l[m][1].x, l[m][1].y, l[m][2].x, l[m][2].y, l[m][3].x, l[m][3].y};
                        const float sum = over_warp(x);
                        if ((lane & 3) == 0) red[wq * MC * 8 + m * 8 + (lane >> 2)] = sum;
                    }
                bar_sync(bar_gr, 128);
                if (wt < live * 8)
                    lsum[team * N + (sub + X::GT * (wt >> 3)) * 8 + (wt & 7)] =
                        red[wt] + red[MC * 8 + wt] + red[2 * MC * 8 + wt] + red[3 * MC * 8 + wt];
            }
            bar_sync(bar_all, kSoftThreads);
            if (tid < rows) {
                float M = mref_all[tid];
#pragma unroll
                for (int tm = 1; tm < TM; ++tm) M = larger(mref_all[tm * N + tid], M);
                float sum = 0.f, f[TM];
#pragma unroll
                for (int tm = 0; tm < TM; ++tm) {
                    f[tm] = ex2(mref_all[tm * N + tid] - M);
                    sum = fmaf(f[tm], lsum[tm * N + tid], sum);
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                for (int tm = 0; tm < TM; ++tm)
                    fac[tm * N + tid] = f[tm] * (whole ? inv : 1.f) * (Q8 ? __uint_as_float((254u << 23) - __float_as_uint(unit_all[tm * N + tid])) : 1.f);
                if (!whole)
                    p.part_ml[part * N + tid] = make_float2(M, sum);
                else if (a.lse && !skip)
                    a.lse[out_row(tid)] = sum == 0.f ? none : (M + log2f(sum)) * 0.69314718055994531f;
            }
            bool has[TM];
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) has[tm] = finished(tm);
            tc_after();
            bar_sync(bar_all, kSoftThreads);
            const bool any_poison = poison[0] | poison[1] | poison[2] | poison[3];
#pragma unroll 1
            for (int piece = gr; piece < pieces; piece += kGroups) {
                const int r0 = piece * 8;
                float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int tm = 0; tm < TM; ++tm)
                    if (has[tm]) {
                        float x[8], y[8];
                        const uint32_t at = tmem + X::O_at + lanes + tm * X::NP + r0;
                        tc_ld8(at, x);
                        if (!Q8) tc_ld8(at + N, y);
                        tc_wait_ld(x);
                        if (!Q8) tc_wait_ld(y);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float f = fac[tm * N + r0 + k];
                            if (!Q8) x[k] += y[k];
                            o[k] = f == 0.f ? o[k] : fmaf(f, x[k], o[k]);
                        }
                    }
                if (any_poison && wt < c.D) {
#pragma unroll 1
                    for (int32_t u = 0; u < T; ++u) {
                        if (!(poison[u >> 5] >> (u & 31) & 1)) continue;
                        const int32_t pos = ctx + u;
                        const int32_t pg = c.table[(int64_t)g->b * c.max_blocks + c.by_bs.of(pos)], sl = (pos - c.by_bs.of(pos) * c.bs);
                        if (pg < 0 || pg >= c.num_blocks) continue;  // (only after a wait has given up)
                        const unsigned char* v = c.v + pg * c.block_bytes + sl * c.token_bytes + g->h * c.head_bytes;
                        const float x = Q8 ? kv_e4m3(v[wt]) : bf16_lo(*(const uint16_t*)(v + 2 * wt));
                        if (fabsf(x) < __uint_as_float(0x7F800000u)) continue;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int32_t tk = a.by_G.of(row0 + r0 + k);
                            if (a.parent ? tk < T && (seen_by[u * 4 + (tk >> 5)] >> (tk & 31) & 1) : tk >= u) o[k] += x;
                        }
                    }
                }
                if (whole) {
                    // through shared memory (the piece's own P) to 16-byte stores
                    uint16_t* const st = (uint16_t*)(p_sm + piece * 2048);
#pragma unroll
                    for (int k = 0; k < 8; ++k) st[k * 128 + wt] = (uint16_t)bf16x2(o[k], 0.f);
                    bar_sync(bar_gr, 128);
                    const int k = wt >> 4, ch = wt & 15;
                    if (r0 + k < rows && ch * 8 < c.D && !skip)
                        *(uint4*)(a.out + (out_row(r0 + k) * c.D + ch * 8) * 2) = *(const uint4*)(st + k * 128 + ch * 8);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (r0 + k < rows && wt < c.D) p.part_o[(part * N + r0 + k) * 128 + wt] = o[k];
                }
            }
            if (!whole) {
                // ---- join: the entry's parts lie with CTAs c0 (its second place) and c0 + 1 .. c1 (their first). A group
                // counts its arrivals at its second member.
                constexpr int lg = kJoinLog<N>;
                const int32_t c0 = g->c0, parts = g->c1 - c0 + 1;
                int32_t i = (int32_t)blockIdx.x - c0;
#pragma unroll 1
                for (int at = 0; 1 << at < parts; at += lg) {
                    i = i >> (at + lg) << (at + lg);
                    const int32_t k = min(1 << lg, (parts - i + (1 << at) - 1) >> at);
                    if (k == 1) continue;
                    __threadfence();
                    bar_sync(bar_all, kSoftThreads);
                    if (tid == 0) {
                        uint32_t* const arrive = p.arrive + c0 + i + (1 << at);
                        const bool last = atomicAdd(arrive, 1u) == (uint32_t)k - 1;
                        *last_in = last;
                        if (last) *arrive = 0;  // for the next call
                        __threadfence();
                    }
                    bar_sync(bar_all, kSoftThreads);
                    if (!*last_in) break;
                    if (skip) continue;
                    const Join w{p, c0, i, 1 << at, k, 1 << (at + lg) >= parts, rows, row0, g->lo, g->h};
                    if constexpr (N <= 16)
                        join_few<N, Q8>(w);
                    else
                        join_many<N>(w, (float*)p_sm);
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
    if (tid == 0) {
        const bool late = *aborted;
        if (late) atomicOr(p.err, 1u);
        if (a.seq_status) {
            const Settled words{p};
            settle(words, (int32_t)blockIdx.x, p.grid, late && u0 < u1 ? b0 : 0, late && u0 < u1 ? (int32_t)*last_seq + 1 : 0);
        }
    }
}

template <int N, int DP, bool Q8>
cudaError_t launch(const AttParams& p, cudaStream_t s) {
    using X = Shape<N, DP, Q8>;
    auto* f = attend_kernel<N, DP, Q8>;
    // more than half of an SM's shared memory, whatever the ring took: one CTA on an SM owns its TMEM
    constexpr int bytes = (int)(X::total > kSmemMax / 2 + 1024 ? X::total : kSmemMax / 2 + 1024);
    static std::atomic<uint64_t> known{0};  // devices on which the kernel may use that much
    const uint64_t bit = 1ull << (p.device & 63);
    if (!(known.load() & bit) || p.device >= 64) {
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        known.fetch_or(bit);
    }
    f<<<p.grid, X::threads, bytes, s>>>(p);
    return cudaGetLastError();
}

template <int N, bool Q8>
cudaError_t launch_dim(const AttParams& p, cudaStream_t s) {
    return p.a.c.D <= 64 ? launch<N, 64, Q8>(p, s) : launch<N, 128, Q8>(p, s);
}

}  // namespace

}  // namespace specv
