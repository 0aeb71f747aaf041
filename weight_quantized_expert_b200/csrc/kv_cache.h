// A quantised key/value cache as the kernels see it (see kv_cache.cu).
#pragma once

#include <stdint.h>

#include "../../include/focr_moe.h"
#include "abi_util.h"

namespace focr {

struct KvView {
    uint8_t *k, *v;     // codes, [B][heads][cap][128 or 64 bytes]
    float *ks, *vs;     // scales, [B][heads][cap]
    int type, heads, cap;
};

// A cache's four buffers.
inline void cache_spans(const focr_kv_cache* c, Span (&s)[4]) {
    const size_t rows = (size_t)c->B * c->heads * c->cap, row = c->type == FOCR_W_INT4 ? FOCR_RSWA_DIM / 2 : FOCR_RSWA_DIM;
    s[0] = {c->k, rows * row}, s[1] = {c->k_scale, rows * 4}, s[2] = {c->v, rows * row}, s[3] = {c->v_scale, rows * 4};
}

// Checks a caller's cache and fills the view; `what` names it in the error message.
focr_status check_kv_cache(const focr_kv_cache* c, const char* what, KvView* v);

}  // namespace focr
