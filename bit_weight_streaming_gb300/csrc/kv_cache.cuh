// What the key/value cache's translation units share.
#pragma once
#include "../../include/bws.h"

namespace bws {

// Argument checks of a cache descriptor (kv_cache.cu): BWS_OK or a status.
int check_kv_cache(const bws_kv_cache* c, const char* name);

}  // namespace bws
