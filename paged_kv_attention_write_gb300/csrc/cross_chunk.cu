// cross_chunk.cu -- chunks of query rows over another sequence's whole paged context, each row
// within its own range of keys (kernel: prefill_rows.cuh).
#include "cross.cuh"
#include "prefill_rows.cuh"

namespace pa {

int load_cross_chunk(pa_dtype dtype, int head_dim) {
    if (dtype == PA_F16) return head_dim == 64 ? load_typed<F16, 64, true>() : load_typed<F16, 128, true>();
    return head_dim == 64 ? load_typed<BF16, 64, true>() : load_typed<BF16, 128, true>();
}

int launch_cross_chunk(const CrossArgs &c) { return launch_rows<true>(c.a, c.key_ranges); }

}  // namespace pa
