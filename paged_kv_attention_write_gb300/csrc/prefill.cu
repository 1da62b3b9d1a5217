// prefill.cu -- the causal instantiations of chunked prefill (and of its decode rows); the
// kernel and its design are in prefill_kernels.cuh.
#include "prefill_kernels.cuh"

namespace pa {

int launch_prefill(const PrefillArgs &a) { return prepare_and_launch<false>(a); }

}  // namespace pa
