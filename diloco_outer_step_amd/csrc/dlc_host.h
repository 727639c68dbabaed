// Host helpers that every file of the C-ABI layer uses (defined in dlc_api.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "dlc.h"

namespace dlc {

constexpr int64_t kMaxTensorNumel = (int64_t(1) << 32) - 1;

inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// Set the calling thread's last error and return the code; ok() clears it.
int32_t fail(int32_t code, const std::string& msg);
int32_t ok();
int32_t hip_fail(hipError_t e, const char* what);
const char* last_error();

// DLC_ERR_WORKSPACE for host memory that ran out; its message fits a string's own storage.
int32_t out_of_memory() noexcept;

// No C++ exception crosses the ABI: running out of host memory is an error code.
template <typename F>
int32_t no_throw(F&& f) noexcept {
  try {
    return f();
  } catch (...) {
    return out_of_memory();
  }
}

// What a call uses of one of its device arrays, from the first byte to the last (an absent
// array has no bytes).
struct Stretch {
  const void* p;
  uint64_t bytes;
  bool written;
};

// No array that is written may share memory with another one: blocks of a launch run in any order.
int32_t check_stretches(const Stretch* s, int32_t n);

// The tensor list's own rules: sizes, alignment, extents within a learner row (with
// need_loffset), no overlap.
int32_t check_tensors(const dlc_tensor* t, int32_t n, int64_t learner_stride, bool need_loffset);

}  // namespace dlc
