// How the thread that issued a CTA's copies waits for their end. Plain C++: the CPU tries it too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TIDE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TIDE_HOST_DEVICE inline
#endif

namespace tide {

constexpr uint64_t kLandingNs = 20000000;  // 20 ms: what copies on their way are given to land, once nothing else is waited for

// Waits for the last use of each stage of a ring of `stages`, of `uses` in all: until the products that read it have ended, for `limit` ns, or, of a CTA
// that was stopped before or is meanwhile, or whose limit ran out, until its copies have landed, for kLandingNs. All stages have one such time between
// them. `at` is what it waits on: now() ns, stopped(), ended(stage, parity) and landed(stage, parity).
template <typename At>
TIDE_HOST_DEVICE void wait_for_last_uses(int64_t uses, int stages, bool stopped, uint64_t limit, const At& at) {
    bool products = !stopped && !at.stopped();
    uint64_t end = at.now() + (products ? limit : kLandingNs);
    for (int64_t u = uses > stages ? uses - stages : 0; u < uses; ++u) {
        const int stage = int(u % stages);
        const uint32_t parity = uint32_t(u / stages) & 1;
        while (!(products ? at.ended(stage, parity) : at.landed(stage, parity))) {
            const uint64_t now = at.now();
            if (products ? now >= end || at.stopped() : false) {
                products = false;
                end = now + kLandingNs;
            } else if (now >= end) {
                return;
            }
        }
    }
}

}  // namespace tide
