// attend_tc_quant.cu -- the tensor cores' attention over rows held in 4 or 8 bits.
#include "attend_tc.cuh"

namespace kvc {

int launch_attend_tc_quant(AttendParams &p, int rows_above, int grid, cudaStream_t st) {
    if (!shape_units(p, rows_above)) return KVC_ERR_UNSUPPORTED;
    if (p.one_term) {
        if (p.bits == 4) return p.dim == 64 ? launch<1, false, 4>(p, grid, st) : launch<2, false, 4>(p, grid, st);
        return p.dim == 64 ? launch<1, false, 8>(p, grid, st) : launch<2, false, 8>(p, grid, st);
    }
    if (p.bits == 4) return p.dim == 64 ? launch<1, true, 4>(p, grid, st) : launch<2, true, 4>(p, grid, st);
    return p.dim == 64 ? launch<1, true, 8>(p, grid, st) : launch<2, true, 8>(p, grid, st);
}

}  // namespace kvc
