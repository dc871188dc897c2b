// Handles on the rows kernel's instantiations (rows_instances.cu, a translation
// unit per head_dim and place of the keys, so that the library builds in parallel).
#pragma once
#include "decode_launch.h"

namespace gqa {

// f16: fp16 inputs (else bf16).
KernelRef rows_kernel_ref_64_0(bool f16);
KernelRef rows_kernel_ref_128_0(bool f16);
KernelRef rows_kernel_ref_256_0(bool f16);
KernelRef rows_kernel_ref_64_1(bool f16);   // keys in a paged cache
KernelRef rows_kernel_ref_128_1(bool f16);
KernelRef rows_kernel_ref_256_1(bool f16);

}  // namespace gqa
