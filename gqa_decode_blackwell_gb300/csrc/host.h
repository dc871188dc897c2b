// What the host side of gqa_decode.cu shares with that of gqa_shared_keys.cu:
// device state, argument checks and the encoder of tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/gqa_decode.h"

namespace gqa {

constexpr int kMaxDevices = 64;
constexpr size_t kWsAlign = 256;

struct DeviceState {
  int sm_count = 0;
  unsigned long long attr_done = 0;  // one bit per kernel instantiation (decode: 0..23, rows: 24..39)
  unsigned int* err_word = nullptr;  // device address of the library's error word
};

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

EncodeTiledFn encode_fn();
bool env_flag(const char* name);
unsigned long long wait_timeout_ns();
gqa_status_t current_device(int* dev, DeviceState** st);
gqa_status_t error_word(DeviceState* st, unsigned int** out);
gqa_status_t ensure_smem_attr(DeviceState* st, unsigned bit, const void* fn, int bytes, int regs = 0);
cudaLaunchAttribute pdl_attr(bool on);

// A description for any number of query rows, and one the decode kernel can
// serve (at most GQA_MAX_QROWS per KV head).
gqa_status_t check_desc_any_rows(const gqa_desc_t* d);
gqa_status_t check_desc(const gqa_desc_t* d);
gqa_status_t check_inputs(const void* q, const void* k, const void* v, const int32_t* seqlens);

}  // namespace gqa
