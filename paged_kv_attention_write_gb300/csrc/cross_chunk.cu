// cross_chunk.cu -- chunks of query rows over another sequence's whole paged context, each row
// within its own range of keys (kernel: prefill_rows.cuh).
#include "cross.cuh"
#include "prefill_rows.cuh"

namespace pa {

int launch_cross_chunk(const CrossArgs &c) { return launch_rows<true>(c.a, c.key_ranges); }

}  // namespace pa
