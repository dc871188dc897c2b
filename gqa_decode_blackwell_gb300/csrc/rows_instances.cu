// The rows kernel instantiations of one head_dim, selected when compiling:
// -DGQA_INST_HD=<64|128|256>.  The host code reaches them through rows_launch.h.
#include "rows_kernel.cuh"
#include "rows_launch.h"

#if !defined(GQA_INST_HD)
#error "compile with -DGQA_INST_HD=<64|128|256>"
#endif

#define GQA_ROWS_REF_NAME_(hd) rows_kernel_ref_##hd
#define GQA_ROWS_REF_NAME(hd) GQA_ROWS_REF_NAME_(hd)

namespace gqa {

KernelRef GQA_ROWS_REF_NAME(GQA_INST_HD)(bool f16) {
  using Cfg = RowsCfg<GQA_INST_HD>;
  const void* fn = f16 ? reinterpret_cast<const void*>(&gqa_rows_kernel<GQA_INST_HD, true>)
                       : reinterpret_cast<const void*>(&gqa_rows_kernel<GQA_INST_HD, false>);
  return KernelRef{fn, Cfg::kSmemBytes, Cfg::kThreads, Cfg::kMoveRegs ? Cfg::kLaunchRegs : 0};
}

}  // namespace gqa
