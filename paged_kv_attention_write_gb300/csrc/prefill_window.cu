// prefill_window.cu -- chunked prefill over a sliding window with sinks (kernel: prefill_rows.cuh).
#include "prefill_rows.cuh"

namespace pa {

int launch_prefill_window(const PrefillArgs &a) { return launch_rows<false>(a, nullptr); }

}  // namespace pa
