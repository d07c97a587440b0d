// attend_e4m3_qbf16.cu -- the paged attention's kernels for a e4m3 cache and an
// bf16 query (one translation unit per pair of types, compiled in parallel).
#include "attend.cuh"

namespace moe {

int launch_attend_e4m3_qbf16(const AttendParams &p, int dp, cudaStream_t st) {
    if (dp == 64) return launch_attend_dp<true, false, 64>(p, st);
    if (dp == 128) return launch_attend_dp<true, false, 128>(p, st);
    return launch_attend_dp<true, false, 256>(p, st);
}

}  // namespace moe
