// The attention kernels of one type and head size (SC_DT, SC_D): a translation
// unit each, so that they build side by side.
#include "sc_plan.h"

#include "sc_attend_tc.cuh"

namespace sv {

namespace {
template <int DT, int D, int MB>
AttendKernel warps() {
    return {sc_attend_kernel<DT, D, MB>, SC_NT, AttendSmem<D, MB>::BYTES, AttendSmem<D, MB>::ROWS, 2, SC_BLOCK};
}
template <int DT, int D, int N, bool ALT>
AttendKernel tensor_memory() {
    return {sc_attend_tc_kernel<DT, D, N, ALT>, TC_NT, TcShape<DT, D, N, ALT>::BYTES, N, 1, TC_TILE};
}
}  // namespace

#ifndef TC_FROM
#define TC_FROM 65
#endif
template <int DT, int D>
AttendKernel attend_kernel(int rows) {
    if (rows < TC_FROM) {
        if (rows <= 16) return warps<DT, D, 1>();
        if (rows <= 32) return warps<DT, D, 2>();
        if (rows <= 64) return warps<DT, D, 4>();
    }
    if (rows <= 48) return tensor_memory<DT, D, 48, false>();
    return tensor_memory<DT, D, 80, false>();
}

template AttendKernel attend_kernel<SC_DT, SC_D>(int rows);

}  // namespace sv
