// attend_simt_quant8.cu -- attention by fp32's accuracy over rows held in 8 bits.
#include "attend_pieces.cuh"

namespace kvc {

int launch_attend_simt_quant8(AttendParams &p, bool f32, int grid, cudaStream_t st) {
    return launch_all<8>(p, f32, grid, st);
}

}  // namespace kvc
