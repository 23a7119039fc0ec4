// w8a8_plan.h -- arithmetic of the W8A8 kernels that needs no GPU: plain C++,
// shared by the kernels and their host side, and compiled alone by the tests.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SVDQ_HD __host__ __device__ __forceinline__
#else
#define SVDQ_HD inline
#endif

namespace svdq {

// The ring of the row quantizer.  A block takes rows first, first + step, ...;
// the copy of its i-th row goes to place i % stages, where it is phase
// i / stages of that place's barrier.  When the wait for `lost` has run out,
// the copies still in flight are those of the rows from lost on that were
// fetched, that is below `ahead` (the next row to fetch, or the number of rows).
// wait(place, parity) is called for each of them and for nothing else: a wait
// for another phase would return at once, or run out without a copy to wait for.
template <typename Wait>
SVDQ_HD void drain_ring(int first, int step, int lost, int ahead, int stages, Wait wait) {
    const int64_t begin = ((int64_t)lost - first) / step, end = ((int64_t)ahead - first + step - 1) / step;
    for (int64_t i = begin; i < end; ++i) wait((int)(i % stages), (uint32_t)(i / stages) & 1u);
}

}  // namespace svdq
