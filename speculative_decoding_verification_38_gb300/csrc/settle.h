// settle.h -- how the sequences of a CTA whose wait gave up come to say so.
//
// A sequence's status is written by one CTA, and its rows may be worked on by others. A CTA that wrote "timed out" by
// itself could be overwritten by the one that has found the sequence's arguments in order. So each CTA leaves through
// here once, behind its own statuses; one that gave up names the sequences of its run, and whoever leaves last marks
// them, behind every other status. Words return to zero.
//
// M is the memory: on the device a grid's (attend.cuh), on the host the threads' of a test.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SPECV_HD __host__ __device__ __forceinline__
#else
#define SPECV_HD inline
#endif

namespace specv {

// Sequences [b0, b1) of a CTA that gave up; b1 <= b0: it did not (or had none).
template <class M>
SPECV_HD void settle(M&& m, int32_t cta, int32_t ctas, int32_t b0, int32_t b1) {
    if (b1 > b0) {
        m.put(2 * cta, b0);
        m.put(2 * cta + 1, b1);
        m.raise();
    }
    m.fence();  // the CTA's statuses and words, before it is counted
    if (m.count() != ctas - 1) return;
    m.fence();
    m.clear_count();
    if (!m.raised()) return;
    m.lower();
    for (int32_t i = 0; i < ctas; ++i) {
        const int32_t e = m.get(2 * i + 1);
        for (int32_t b = m.get(2 * i); b < e; ++b) m.mark(b);
        m.put(2 * i, 0);
        m.put(2 * i + 1, 0);
    }
}

}  // namespace specv
