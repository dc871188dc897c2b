// Handles on the rows kernel's instantiations (rows_instances.cu, a translation
// unit per head_dim and place of the keys, so that the library builds in parallel).
#pragma once
#include "decode_launch.h"

namespace gqa {

// tiles: row tiles of a CTA (1 or 2, where there is a choice); f16: fp16 inputs (else bf16).
KernelRef rows_kernel_ref_64_0(int tiles, bool f16);
KernelRef rows_kernel_ref_128_0(int tiles, bool f16);
KernelRef rows_kernel_ref_256_0(int tiles, bool f16);
KernelRef rows_kernel_ref_64_1(int tiles, bool f16);   // keys in a paged cache
KernelRef rows_kernel_ref_128_1(int tiles, bool f16);
KernelRef rows_kernel_ref_256_1(int tiles, bool f16);

}  // namespace gqa
