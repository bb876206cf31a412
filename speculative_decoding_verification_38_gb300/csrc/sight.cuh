// sight.cuh -- which positions of the cache a sequence's new tokens see through a sliding window, as a list.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#ifndef SPECV_HD
#define SPECV_HD __host__ __device__ __forceinline__
#endif
#else  // a test's host code
#include <algorithm>
#ifndef SPECV_HD
#define SPECV_HD inline
#endif
#endif

namespace specv {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

// What the tokens of a sequence see through a window: the tiles hold, box by box, the sinks, then the positions from
// where every token sees them to the end, then those before that only some of them still see. A tile of positions that
// all rows see thus never comes after one that parts them, as the e4m3 units need it, and no box is loaded that no row
// sees a position of. Places [0, s1) are positions as they are, [s1, i1) are di further on, [i1, end) are de further on.
struct Sight {
    int32_t s1, i1, di, de, end;
    int32_t lo;    // the first position that the first token's window holds
    int32_t tail;  // the first place from which rows may part: new tokens, or the window's end
    SPECV_HD Sight() {}
    SPECV_HD Sight(int32_t T, int32_t L, int32_t window, int32_t sinks, int32_t box_log) {
        const int32_t ctx = L - T, more = (1 << box_log) - 1;
        lo = max(0, ctx + 1 - window);
        const int32_t first = min(sinks, L), up = (first + more) & ~more;
        s1 = lo < up ? first & ~more : up;  // (a box that the sinks end in, within the window, is the window's)
        const int32_t last = (L + more) & ~more, e0 = max(s1, lo & ~more);
        const int32_t i0 = min(max((max(0, ctx + T - window) + more) & ~more, e0), last);
        di = i0 - s1;
        i1 = last - di;
        de = e0 - i1;
        end = i1 + (i0 - e0);
        tail = ctx < s1 ? ctx : ctx < i0 ? s1 : ctx - di;
    }
    SPECV_HD int32_t at(int32_t place) const {  // a position past any length where there is none
        return place < s1 ? place : place < i1 ? place + di : place < end ? place + de : INT32_MAX;
    }
    // at once for places of one box; whether some token sees it
    SPECV_HD bool seen(int32_t pos, int32_t L, int32_t sinks) const {
        return pos < L && (pos < sinks || pos >= lo);
    }
};

}  // namespace specv
