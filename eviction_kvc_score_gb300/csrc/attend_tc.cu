// attend_tc.cu -- the tensor cores' attention over bf16 rows.
#include "attend_tc.cuh"

namespace kvc {

AttendNeeds attend_tc_needs(int sms) { return {sms, kSlotsTc, 2 * kTile}; }

bool attend_tc_takes(int dtype, int dim, int group) {
    return dtype == KVC_BF16 && (dim == 64 || dim == 128) && group <= kTile;
}

int launch_attend_tc(AttendParams &p, int grid, cudaStream_t st) {
    if (!shape_units(p, 0)) return KVC_ERR_UNSUPPORTED;
    if (p.one_term) return p.dim == 64 ? launch<1, false, 0>(p, grid, st) : launch<2, false, 0>(p, grid, st);
    return p.dim == 64 ? launch<1, true, 0>(p, grid, st) : launch<2, true, 0>(p, grid, st);
}

}  // namespace kvc
