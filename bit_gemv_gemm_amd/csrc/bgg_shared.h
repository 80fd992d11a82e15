// The launch of the shared part of bgg_shared_attention (bgg_shared.hip),
// for the call itself (bgg_attention.hip).
#pragma once
#include "bgg_paged.h"

namespace bgg {

// Floats of the parts that launch_prefix writes at most.
int64_t prefix_part_floats(const bgg_cache_desc* c, int64_t q_heads, int64_t batch, int64_t target);

// Every group's prefix into prefix_parts, every sequence's seqs, and the
// schedule of the sequences' own tokens.
void launch_prefix(const AttnParams& p, int32_t type, bool e4m3, int64_t head_dim, hipStream_t s);

}  // namespace bgg
