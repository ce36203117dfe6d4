// ring_flight.cuh -- which copies of a ring of stages are on their way, after a wait ran out.
//
// The thread that posts rows into a ring (rows t0, t0 + step, ... below `rows`; the n-th of them into
// stage n % stages, each phase of a stage's mbarrier armed once) keeps this account.  Once a wait ran
// out it posts no more: arming a barrier whose phase is not over would be a second arrival on it.
// Then the copies that may still be on their way are those of `stages` rows in turn, one to a stage,
// and the parity to wait for is known for each.  Plain C++, so that the host can check it.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define BL_RING_FN __host__ __device__ __forceinline__
#else
#define BL_RING_FN inline
#endif

namespace bl {

struct RingFlight {
    int64_t first;   // the row at which the thread found that a wait ran out and posted no more; -1: none

    BL_RING_FN void reset() { first = -1; }
    // Row t is done with and row t + stages * step is not posted.
    BL_RING_FN void stop(int64_t t) {
        if (first < 0) first = t;
    }
    // wait(stage, parity) for every copy that may be on its way (stopped or not).
    template <typename Wait>
    BL_RING_FN void drain(int stages, int64_t t0, int64_t step, int64_t rows, Wait&& wait) const {
        const int64_t all = rows > t0 ? (rows - t0 + step - 1) / step : 0;
        // every row posted: the last ones have the stages
        int64_t n = first >= 0 ? (first - t0) / step : all > stages ? all - stages : 0;
        for (int64_t end = n + stages < all ? n + stages : all; n < end; ++n)
            wait(static_cast<int>(n % stages), static_cast<uint32_t>(n / stages) & 1u);
    }
};

}  // namespace bl
