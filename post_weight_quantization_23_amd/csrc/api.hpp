// Host-side checks shared by the C entry points (gptq_api.hip, adapter_api.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <climits>
#include <cstddef>
#include <cstdint>
#include <string>

#include "../../include/gptq.h"

namespace gptq {
namespace api {

// Text of the last failure on the calling thread (gptq_last_error).
std::string& last_error();

inline gptq_status fail(gptq_status st, const char* fn, const std::string& what) {
  last_error() = std::string(fn) + ": " + what;
  return st;
}

inline gptq_status ok() {
  last_error().clear();
  return GPTQ_OK;
}

inline gptq_status check_launch(const char* fn) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GPTQ_EHIP, fn, hipGetErrorString(e));
  return ok();
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxRows = INT_MAX / 2; // rows of W, tokens of X
// A launch's grid.x times its 256 threads per workgroup must fit in 32 bits.
constexpr int64_t kMaxGroups256 = ((int64_t(1) << 32) - 1) / 256;

// Workgroups of 256 threads needed for n items at `per` items per workgroup.
inline int64_t groups_for(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Bytes spanned by a rows x cols matrix with row stride ld (elements of
// `elem` bytes), or -1 when that does not fit in 63 bits.
inline int64_t extent_bytes(int64_t rows, int64_t ld, int64_t cols, int64_t elem) {
  int64_t e = 0;
  if (rows <= 0 || cols <= 0) return 0;
  if (__builtin_mul_overflow(rows - 1, ld, &e) || __builtin_add_overflow(e, cols, &e) ||
      __builtin_mul_overflow(e, elem, &e))
    return -1;
  return e;
}

// Whether [p, p + bytes) and [q, q + bytes_q) overlap (extents already known to fit).
inline bool overlaps(const void* p, int64_t bytes, const void* q, int64_t bytes_q) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + (uint64_t)bytes_q && b < a + (uint64_t)bytes;
}

inline size_t elem_size(gptq_dtype t) { return t == GPTQ_F32 ? 4 : 2; }
inline bool valid_dtype(int t) { return t == GPTQ_F32 || t == GPTQ_BF16 || t == GPTQ_F16; }

}  // namespace api
}  // namespace gptq
