// attend_bf16_qbf16.cu -- the paged attention's kernels for a bf16 cache and an
// bf16 query (one translation unit per pair of types, compiled in parallel).
#include "attend.cuh"

namespace moe {

int launch_attend_bf16_qbf16(const AttendParams &p, int dp, cudaStream_t st) {
    if (dp == 64) return launch_attend_dp<false, false, 64>(p, st);
    if (dp == 96) return launch_attend_dp<false, false, 96>(p, st);
    if (dp == 128) return launch_attend_dp<false, false, 128>(p, st);
    if (dp == 192) return launch_attend_dp<false, false, 192>(p, st);
    return launch_attend_dp<false, false, 256>(p, st);
}

}  // namespace moe
