// Launches of the 8-bit kernels (fp8.hip) for the entry points of an adapted
// linear over an 8-bit W (lora_api.hip).
#pragma once
#include <hip/hip_runtime.h>

#include "common.hpp"

namespace lora {

// The LoRA term added to a product: ls lu lb^T (forward: lu = U [M, r],
// lb = B [N, r]) or ls lu lb, masked (dX: lu = V [M, r], lb = A [r, K]).
struct Fp8Lora {
  const float* lu;
  const float* lb;
  int64_t r;
  float ls;
  DropParams drop;   // dX only
};

size_t fp8_operand_bytes(int64_t rows, int64_t cols);
// Rounds X [rows, cols] (float32, contiguous) into `data` (operand layout).
void fp8_launch_quantize(const float* X, int64_t rows, int64_t cols, void* data, hipStream_t st);
// out = x W^T (or x W) + the LoRA term, float32; out2 (may be NULL) the same.
void fp8_launch_lora_product(const void* x, int64_t rows, const void* W, int64_t N, int64_t K,
                             bool dx, const Fp8Lora& l, float* out, float* out2, hipStream_t st);

}  // namespace lora
