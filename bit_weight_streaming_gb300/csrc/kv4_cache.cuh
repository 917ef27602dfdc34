// What the 4-bit cache's translation units share.
#pragma once
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/bws.h"

namespace bws {

// a / 6 of a finite BF16 magnitude: a product and Markstein's correction by its remainder,
// the quotient's rounding for every one of them.
__host__ __device__ inline float sixth_of(float a) {
  constexpr float kSixth = 1.0f / 6.0f;
  const float y = a * kSixth;
  return fmaf(fmaf(-6.0f, y, a), kSixth, y);
}

// Argument checks of a cache descriptor (kv4_cache.cu): BWS_OK or a status.
int check_kv4_cache(const bws_kv4_cache* c, const char* name);

}  // namespace bws
