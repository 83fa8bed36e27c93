// rr_cache.cuh -- what the cache's kernels share (include/rr_cache.h).
#pragma once

#include "../../include/rr_cache.h"
#include "rr_frag.cuh"

namespace rr_cache {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int chunk_shift(int chunk) { return chunk == 16 ? 4 : chunk == 32 ? 5 : chunk == 64 ? 6 : 7; }

// Heads are limited so that a pool's page has fewer than 2^31 rows.
inline bool config_ok(const rr_cache_config *c) {
    return c && c->pages >= 0 && c->heads >= 1 && c->heads <= 65535 && (c->dh == 64 || c->dh == 128) &&
           (c->chunk == 16 || c->chunk == 32 || c->chunk == 64 || c->chunk == 128) &&
           (c->format == RR_E4M3 || c->format == RR_E2M1);
}

// The value of a scale byte: 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float power_of_two(unsigned byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

}  // namespace rr_cache
