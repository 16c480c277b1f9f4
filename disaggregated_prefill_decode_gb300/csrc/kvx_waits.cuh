// Waits for barriers in shared memory, with a limit.
#pragma once

#include <cstdint>

namespace kvx {

__device__ __forceinline__ uint32_t shared_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Whether a phase of a barrier is through; the hardware may wait for it a while.
__device__ __forceinline__ bool phase_done(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(shared_addr(bar)), "r"(parity) : "memory");
    return done;
}

// Waits for a phase of a stage's barrier. The clock runs from the first try that fails and is read at every 64th, of which the hardware holds each for
// up to 4 us: a wait that runs out ends at most a quarter of a millisecond after limit_ns. What has to end before a CTA does is waited for with
// kCacheWaitNs.
__device__ __forceinline__ bool wait_full(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (uint32_t tries = 0;; ++tries) {
        if (phase_done(bar, parity)) return true;
        if ((tries & 63) == 0) {
            uint64_t now;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
            if (!t0) t0 = now;
            else if (now - t0 > limit_ns) return false;
        }
    }
}

}  // namespace kvx
