// Host-side argument checks shared by the entry points of libaa.so.
#pragma once

#include <stdint.h>

#include <string>

#include "aa_internal.h"

namespace aa {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline aa_status_t check_ptr(const void* p, const char* what, const char* fn) {
  if (!p) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": " + what + " is NULL");
  if (!aligned16(p)) return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": " + what + " is not 16-byte aligned");
  return AA_OK;
}

// For an operand that may be absent.
inline aa_status_t check_opt_ptr(const void* p, const char* what, const char* fn) {
  return p ? check_ptr(p, what, fn) : AA_OK;
}

inline aa_status_t check_dtype(aa_dtype_t t, const char* what, const char* fn) {
  if (t != AA_BF16 && t != AA_F32)
    return fail(AA_ERR_INVALID_ARG, std::string(fn) + ": " + what + " is no aa_dtype_t");
  return AA_OK;
}

inline size_t elem_size(aa_dtype_t t) { return t == AA_F32 ? 4 : 2; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace aa
