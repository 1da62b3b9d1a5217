// prefill_window.cu -- the instantiations of chunked prefill under a sliding window with
// sinks; the kernel and its design are in prefill_kernels.cuh.
#include "prefill_kernels.cuh"

namespace pa {

int launch_prefill_window(const PrefillArgs &a) { return prepare_and_launch<true>(a); }

}  // namespace pa
