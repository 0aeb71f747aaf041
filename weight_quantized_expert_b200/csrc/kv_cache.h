// A quantised key/value cache as the kernels see it (see kv_cache.cu).
#pragma once

#include <stdint.h>

#include "../../include/focr_moe.h"

namespace focr {

struct KvView {
    uint8_t *k, *v;     // codes, [B][heads][cap][128 or 64 bytes]
    float *ks, *vs;     // scales, [B][heads][cap]
    int type, heads, cap;
};

// Checks a caller's cache and fills the view; `what` names it in the error message.
focr_status check_kv_cache(const focr_kv_cache* c, const char* what, KvView* v);

}  // namespace focr
