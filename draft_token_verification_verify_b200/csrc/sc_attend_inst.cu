// The attention kernels of one type and head size (SC_DT, SC_D): a translation
// unit each, so that they build side by side.
#include "sc_plan.h"

#include "sc_attend_tc.cuh"

namespace sv {

namespace {
template <int DT, int D, int N, bool ALT>
AttendKernel take() {
    return {sc_attend_tc_kernel<DT, D, N, ALT>, TC_NT, TcShape<DT, D, N, ALT>::BYTES, N};
}
}  // namespace

template <int DT, int D>
AttendKernel attend_kernel(int rows) {
    if (rows <= 16) return take<DT, D, 16, true>();
    if (rows <= 32) return take<DT, D, 32, true>();
    if (rows <= 48) return take<DT, D, 48, false>();
    return take<DT, D, 80, false>();
}

template AttendKernel attend_kernel<SC_DT, SC_D>(int rows);

}  // namespace sv
