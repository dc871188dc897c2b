// The rows kernel instantiations of one head_dim, for dense or paged keys,
// selected when compiling: -DGQA_INST_HD=<64|128|256> -DGQA_INST_PAGED=<0|1>.
// The host code reaches them through rows_launch.h.
#include "rows_kernel.cuh"
#include "rows_launch.h"

#if !defined(GQA_INST_HD) || !defined(GQA_INST_PAGED)
#error "compile with -DGQA_INST_HD=<64|128|256> -DGQA_INST_PAGED=<0|1>"
#endif

#define GQA_ROWS_REF_NAME_(hd, paged) rows_kernel_ref_##hd##_##paged
#define GQA_ROWS_REF_NAME(hd, paged) GQA_ROWS_REF_NAME_(hd, paged)

namespace gqa {

namespace {

template <int TILES>
KernelRef ref(bool f16) {
  constexpr bool kPaged = GQA_INST_PAGED != 0;
  using Cfg = RowsCfg<GQA_INST_HD, TILES>;
  const void* fn = f16 ? reinterpret_cast<const void*>(&gqa_rows_kernel<GQA_INST_HD, TILES, true, kPaged>)
                       : reinterpret_cast<const void*>(&gqa_rows_kernel<GQA_INST_HD, TILES, false, kPaged>);
  return KernelRef{fn, Cfg::kSmemBytes, Cfg::kThreads, Cfg::kMoveRegs ? Cfg::kLaunchRegs : 0};
}

}  // namespace

KernelRef GQA_ROWS_REF_NAME(GQA_INST_HD, GQA_INST_PAGED)(int tiles, bool f16) {
#if GQA_INST_HD == 256
  (void)tiles;
  return ref<1>(f16);
#elif GQA_INST_HD == 128 && GQA_INST_PAGED
  return tiles == 1 ? ref<1>(f16) : ref<2>(f16);
#else
  (void)tiles;
  return ref<2>(f16);
#endif
}

}  // namespace gqa
