// abi_checks.h -- argument checks that the host files of the C ABI share.  Each returns MOE_OK or records the error text
// and returns its status; all of them run before anything is enqueued.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "abi_common.h"
#include "qmoe.h"

namespace qmoe {

// A workgroup addresses at most 256 rows of one matrix, of at most 4 bytes an element, with 31-bit byte
// offsets from its own 64-bit base.
inline constexpr int kMaxWidth = (int)((1LL << 31) / (256 * 4)) - 16;

// Rows that leave room for rounding up to tiles in 32 bits.
inline constexpr int kMaxRows = 0x7FFFFC00;

inline int check_rows(const char *fn, int M) {
  if (M < 0) return abi_fail(MOE_ERR_INVALID_ARG, "%s: M=%d is negative", fn, M);
  if (M > kMaxRows) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: M=%d too large", fn, M);
  return MOE_OK;
}

inline bool misaligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

struct Range {
  const void *p;
  size_t n;
};

inline bool overlaps(const Range &a, const Range &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.n && b.n && x < y + b.n && y < x + a.n;
}

inline int check_out(const char *fn, int out_dtype) {
  if (out_dtype != MOE_OUT_F32 && out_dtype != MOE_OUT_BF16)
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: out_dtype=%d is neither MOE_OUT_F32 nor MOE_OUT_BF16", fn, out_dtype);
  return MOE_OK;
}

inline int check_groups(const char *fn, const int32_t *offsets, const int32_t *counts, int E, int M, int expected_rows) {
  if (!offsets) return abi_fail(MOE_ERR_INVALID_ARG, "%s: offsets is NULL", fn);
  if (E < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: E=%d must be positive", fn, E);
  if (int rc = check_rows(fn, M)) return rc;
  if (E > 1024) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: E=%d > 1024", fn, E);
  if (misaligned(offsets, 4) || misaligned(counts, 4))
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: offsets and counts must be 4-byte aligned", fn);
  if (expected_rows < 0) return abi_fail(MOE_ERR_INVALID_ARG, "%s: expected_rows=%d is negative", fn, expected_rows);
  return MOE_OK;
}

inline int check_inputs(const char *fn, std::initializer_list<Range> in, const Range &out, uintptr_t out_align) {
  for (const Range &r : in) {
    if (!r.n) continue;
    if (!r.p) return abi_fail(MOE_ERR_INVALID_ARG, "%s: NULL operand", fn);
    if (overlaps(r, out)) return abi_fail(MOE_ERR_INVALID_ARG, "%s: an output overlaps an operand", fn);
  }
  if (out.n && !out.p) return abi_fail(MOE_ERR_INVALID_ARG, "%s: NULL output", fn);
  if (misaligned(out.p, out_align))
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: outputs must be %d-byte aligned", fn, (int)out_align);
  return MOE_OK;
}

inline int check_aligned16(const char *fn, std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (misaligned(p, 16)) return abi_fail(MOE_ERR_INVALID_ARG, "%s: operands must be 16-byte aligned", fn);
  return MOE_OK;
}

inline int rows_hint(int expected_rows, int M) { return expected_rows > 0 ? std::min(expected_rows, M) : M; }

}  // namespace qmoe
