// cross.cuh -- arguments and launchers of the attention over another sequence's states.
#pragma once

#include "common.cuh"

namespace pa {

struct CrossArgs {
    PrefillArgs a;              // query_start_loc null: row s belongs to sequence s
    const int32_t *key_ranges;  // [num_tokens][2] first key and one past the last, or null
};

int launch_cross(const CrossArgs &c);
int launch_cross_chunk(const CrossArgs &c);  // 16-bit caches, query_start_loc given
int load_cross_chunk(pa_dtype dtype, int head_dim);

}  // namespace pa
