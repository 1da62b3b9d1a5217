// tables.cuh -- arguments and launchers of the block tables kept on the GPU (tables.cu).
#pragma once

#include "common.cuh"

namespace pa {

struct TablesArgs {
    int32_t *block_tables;  // extend: written; trim: read
    int32_t *context_lens, *query_start_loc, *positions;
    int64_t *slot_mapping;
    int32_t *free_blocks;  // extend: read; trim: written
    int32_t *num_free_out;
    const int32_t *cached_lens, *lens, *num_free;  // lens: new_lens or keep_lens
    int num_seqs, max_blocks_per_seq, num_tokens, free_capacity, block_size, num_blocks;
    int32_t *status;
    cudaStream_t stream;
};

int launch_tables_extend(const TablesArgs &a);
int launch_tables_trim(const TablesArgs &a);

}  // namespace pa
