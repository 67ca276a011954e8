// mla_ragged.cuh -- packed (ragged) batches: the start of their kernels, and
// which sequence a packed row belongs to.  Internal to the library; device-only.
//
// A packed batch of B sequences lays their rows out one after another; cu[b]
// is the first row of sequence b and cu[B] the number of rows in use, so rows
// from cu[B] on are padding that belongs to no sequence.
#pragma once

#include <stdint.h>

namespace mla {
namespace {

// The stream's next kernel may be set up, and this one goes on when the previous
// one has finished and its memory is visible (launch_dependent, mla_host.h).
// Whatever an earlier kernel of the stream may have written is read after this
// with ordinary loads: a kernel may be resident while several of its
// predecessors still run, and the non-coherent path (__ldg) is only for memory
// that nothing writes during the kernel's whole life.  What the wait makes
// visible holds for ordinary loads alone.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct RaggedRow {
    int seq;     // -1: the row belongs to no sequence
    int at;      // its place within the sequence
    int start;   // start[seq] (0 without start positions)
};

// Warp-collective: the sequence that holds `row` (the same row in every lane),
// by a 32-way search -- one dependent round of loads for up to 32 sequences,
// two for up to 1,024.  The round that ends the search also fetches
// the lengths and start positions of its candidates, so that they cost no
// further round.  Every index stays inside cu[0..B] and start[0..B) whatever
// the offsets hold; among empty sequences at the same offset the last one
// that starts there (the only one that can hold the row) is found.
__device__ __forceinline__ RaggedRow ragged_find(const int32_t* cu, const int32_t* start, int B, int64_t row,
                                                 int lane) {
    int lo = 0, n = B;  // candidates [lo, lo + n)
    while (n > 32) {
        const int step = (n + 31) >> 5;
        const int off = lane * step;
        const bool le = off < n && cu[lo + off] <= row;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    int32_t c = 0, e = 0, s = 0;
    if (lane < n) {
        c = cu[lo + lane];
        e = cu[lo + lane + 1];
        if (start) s = start[lo + lane];
    }
    const unsigned m = __ballot_sync(0xffffffffu, lane < n && c <= row && row < e);
    if (m == 0) return {-1, 0, 0};
    const int k = 31 - __clz(m);
    return {lo + k, static_cast<int>(row - __shfl_sync(0xffffffffu, c, k)), __shfl_sync(0xffffffffu, s, k)};
}

}  // namespace
}  // namespace mla
