// Handles on the rows kernel's instantiations (rows_instances.cu, a translation
// unit per head_dim, so that the library builds in parallel).
#pragma once
#include "decode_launch.h"

namespace gqa {

// f16: fp16 inputs (else bf16).
KernelRef rows_kernel_ref_64(bool f16);
KernelRef rows_kernel_ref_128(bool f16);
KernelRef rows_kernel_ref_256(bool f16);

}  // namespace gqa
