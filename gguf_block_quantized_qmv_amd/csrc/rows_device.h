// Device helpers of the rows' kernels.
#pragma once

#include "qmv_device.h"

namespace qmv {

template <int CTRL, int ROWS>
__device__ __forceinline__ int add_from(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}

// Inclusive sum over the wave's lanes, by six additions of permuted operands.
__device__ __forceinline__ int wave_upto(int v) {
  v = add_from<0x111, 0xF>(v);   // row_shr:1, within rows of 16 lanes
  v = add_from<0x112, 0xF>(v);
  v = add_from<0x114, 0xF>(v);
  v = add_from<0x118, 0xF>(v);
  v = add_from<0x142, 0xA>(v);   // lane 15 of rows 0 and 2 to the rows behind them
  return add_from<0x143, 0xC>(v);   // lane 31 to rows 2 and 3
}

// LDS that a wave alone uses: its writes before, its lanes' reads of each other's
// values behind. The machine keeps a wave's LDS accesses in order; this keeps the
// compiler to it.
__device__ __forceinline__ void in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace qmv
