// abi_checks.hpp -- argument checks that the entry points share.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/eqtp.h"

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool valid_c(int C) { return C == 8 || C == 16 || C == 32 || C == 64 || C == 128; }
inline bool dtype_ok(int t) { return t == EQTP_F32 || t == EQTP_BF16; }
inline bool aligned_as(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == EQTP_BF16 ? 1u : 3u)) == 0;
}
inline int status_of(hipError_t e) { return e == hipSuccess ? EQTP_OK : EQTP_EHIP; }
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;

}  // namespace
