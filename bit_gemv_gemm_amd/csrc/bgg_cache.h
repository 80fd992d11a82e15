// Argument checks of the calls on a paged cache (bgg_cache.cpp), shared by
// the device sources.
#pragma once
#include "bgg_internal.h"

namespace bgg {

constexpr int64_t kMaxQHeads = 4096;
constexpr int64_t kMaxTokens = int64_t(1) << 23;  // (a workgroup each, in a grid below 2^32 threads)
constexpr int64_t kMaxBatch = 4096;  // (a wave looks through 64 sequences per lane)

// BGG_OK iff `c` is exactly what bgg_cache_describe makes for its fields.
bgg_status check_cache(const bgg_cache_desc* c);
bgg_status check_rotary(const bgg_cache_desc* c, const bgg_rotary_args* a);
// The same, and the positions of several axes.
bgg_status check_rotary_axes(const bgg_cache_desc* c, const bgg_rotary_args* a,
                             const bgg_rotary_axes_args* x);
bgg_status check_assign(const bgg_cache_desc* c, const bgg_assign_args* a);
bgg_status check_attention(const bgg_cache_desc* c, const bgg_attention_args* a);
bgg_status check_shared(const bgg_cache_desc* c, const bgg_attention_args* a, const bgg_shared_args* s);

}  // namespace bgg
