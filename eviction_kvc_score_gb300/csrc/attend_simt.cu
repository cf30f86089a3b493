// attend_simt.cu -- the CUDA cores' attention over rows of the outputs' type.
#include "attend_simt.cuh"

namespace kvc {

AttendNeeds attend_simt_needs(int sms) { return {kBlocksPerSm * sms, 2, kSlotRows}; }

int launch_attend_simt(AttendParams &p, bool f32, int grid, cudaStream_t st) {
    return launch_all<0>(p, f32, grid, st);
}

}  // namespace kvc
