// ssd_api_check.h -- checks of arguments that the C-ABI layers share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "ssd.h"

namespace {

inline ssd_status hip_status(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
inline bool scale_ok(float s) { return std::isnormal(s); }  // its reciprocal is taken

// Rows of `width` bytes, `pitch` bytes apart; a null base has none.
struct Span {
  const void* base;
  int64_t rows, pitch, width;
};
inline Span whole(const void* p, int64_t bytes) { return Span{p, 1, bytes, bytes}; }
// Whether a, one row, and b share a byte.
inline bool meet(const Span& a, const Span& b) {
  if (!a.base || !b.base || a.width < 1 || b.width < 1 || b.rows < 1) return false;
  const intptr_t at = (intptr_t)a.base - (intptr_t)b.base, end = at + a.width;   // a, from b's first row on
  if (end <= 0) return false;
  // the first of b's rows that ends behind a's start
  const int64_t first = at < b.width ? 0 : (at - b.width) / b.pitch + 1;
  return first < b.rows && first * b.pitch < end;
}
// Whether one of the outputs shares memory with an input or another output: kernels
// read the one while others write the other.
inline bool overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return true;
    for (const Span* p = outs.begin(); p != o; ++p)
      if (meet(*o, *p)) return true;
  }
  return false;
}

inline ssd_status check_ws(const void* workspace, size_t have, size_t need) {
  if (need == 0) return SSD_OK;
  if (!workspace || ((uintptr_t)workspace & 255)) return SSD_ERR_INVALID_ARGUMENT;
  return have < need ? SSD_ERR_WORKSPACE_TOO_SMALL : SSD_OK;
}

}  // namespace
