// What the key/value cache's translation units share.
#pragma once
#include <cuda_runtime.h>

#include "../../include/bws.h"

namespace bws {

// Argument checks of a cache descriptor (kv_cache.cu): BWS_OK or a status.
int check_kv_cache(const bws_kv_cache* c, const char* name);

// A launch that may begin while the kernel before it ends: every kernel here
// waits for what came before (pdl_wait) ahead of its first read.
template <typename K, typename P>
cudaError_t launch_pdl(K kernel, dim3 grid, unsigned block, size_t smem, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace bws
