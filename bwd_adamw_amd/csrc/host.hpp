// Host-side helpers of the entry points: argument checks, sizes and the
// status of a launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lora.h"

namespace lora {
namespace host {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t rup(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline int64_t clampi(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : (x > hi ? hi : x); }
inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline int hip_status() { return hipGetLastError() == hipSuccess ? LORA_OK : LORA_E_HIP; }

constexpr int64_t kCUs = 256;

}  // namespace host
}  // namespace lora
