// Argument-check helpers shared by the translation units that define C entry points.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/rkv.h"

namespace rkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline uint32_t* status_ptr(void* ws) { return reinterpret_cast<uint32_t*>(ws); }
inline rkv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RKV_OK : RKV_ERR_CUDA; }
inline bool gqa_ok(int g) { return g == 1 || g == 2 || g == 4 || g == 8; }
constexpr float kLog2e = 1.4426950408889634f;

inline bool paged_ok(const void* table, int num_blocks, int block, int max_blocks) {
  return table && num_blocks > 0 && max_blocks > 0 && pow2(block) && block <= 65536 &&
         (long long)max_blocks * block <= (1ll << 30);
}

}  // namespace rkv
