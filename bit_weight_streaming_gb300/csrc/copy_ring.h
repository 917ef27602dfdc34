// Uses of a ring of copy stages, each with an mbarrier that completes a phase
// when the stage's copies have landed. Plain arithmetic, for the host too.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define BWS_RING __host__ __device__ constexpr
#else
#define BWS_RING constexpr
#endif

namespace bws {

// Use `it` (from 0) of a ring: its stage, and the parity of the phase that its landing completes.
BWS_RING uint32_t ring_stage(uint32_t it, uint32_t stages) { return it % stages; }
BWS_RING uint32_t ring_parity(uint32_t it, uint32_t stages) { return it / stages & 1u; }

// The first use that may still be on its way when `started` have been started:
// a stage is written again only after its last use has landed.
BWS_RING uint32_t ring_oldest(uint32_t started, uint32_t stages) { return started > stages ? started - stages : 0u; }

}  // namespace bws
