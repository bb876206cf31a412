// kv.cuh -- device helpers shared by the cache's kernels.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "kv.h"

namespace specv {

// A sequence's new tokens: rows [lo, lo + T) and the status of its offsets
// and length. T = 0 for a sequence with an error.
struct KvSeq {
    int64_t lo;
    int32_t T, L, st;
};

__device__ __forceinline__ KvSeq kv_seq(int32_t b, const int64_t* off, int32_t t_max, int64_t rows,
                                        const int32_t* lens, int32_t bs, int32_t max_blocks, bool cap_t) {
    KvSeq s;
    const int64_t lo = off ? off[b] : (int64_t)b * t_max;
    const int64_t hi = off ? off[b + 1] : lo + t_max;
    s.lo = lo;
    s.L = lens[b];
    s.T = 0;
    if (lo < 0 || hi < lo || hi > rows || hi - lo > (cap_t ? (int64_t)t_max : (int64_t)INT32_MAX)) {
        s.st = kKvBadLayout;
        s.lo = -1;  // its rows are not known
    } else if (s.L < hi - lo || s.L > (int64_t)bs * max_blocks) {
        s.st = kKvBadKv;
        s.T = (int32_t)(hi - lo);
    } else {
        s.st = kKvOk;
        s.T = (int32_t)(hi - lo);
    }
    return s;
}

// First index b in [0, n) with off[b + 1] > x, by a warp: each step splits
// the range in 32. off must not fall and off[n] > x.
__device__ __forceinline__ int32_t kv_find(const int64_t* off, int32_t n, int64_t x) {
    const int lane = threadIdx.x & 31;
    int32_t lo = 0, len = n;  // the answer lies in [lo, lo + len)
    while (len > 1) {
        const int32_t step = (len + 31) >> 5;
        const int32_t at = min(lo + (lane + 1) * step, lo + len);  // ranges [lo + lane*step, at)
        const unsigned past = __ballot_sync(0xFFFFFFFFu, off[at] > x);
        const int32_t i = past ? __ffs(past) - 1 : 31;
        const int32_t nlo = min(lo + i * step, lo + len - 1);
        len = min(step, lo + len - nlo);
        lo = nlo;
    }
    return lo;
}

__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t two) {  // the low 16 bits: two codes, exact as f16
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ float kv_e4m3(uint8_t code) {
    __nv_fp8_e4m3 x;
    x.__x = code;
    return (float)x;
}

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

}  // namespace specv
