// Argument checks shared by the C entry points of the 16-bit operators.
#pragma once

#include "grouped_internal.h"

namespace moe {

// Row and column counts in 32 bits leave room for a tile beyond the last one.
constexpr int32_t kMaxExtent = 1 << 30;

inline bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool is16(int32_t t) { return t == MOE_BF16 || t == MOE_FP16; }
// an output type beside operands of type t: t itself, or fp32
inline bool out_type(int32_t o, int32_t t) { return o == t || o == MOE_FP32; }
inline size_t size_of(int32_t t) { return t == MOE_FP32 ? 4 : 2; }
inline bool typed(const void *p, int32_t t) { return aligned(p, size_of(t)); }
// 16-byte units of rows of `width` 16-bit elements are aligned and whole
inline bool units(const void *p, int64_t ld, int64_t width) { return aligned(p, 16) && ld % 8 == 0 && width % 8 == 0; }
// 16-byte runs of rows of elements of type t are aligned
inline bool runs(const void *p, int32_t t, int64_t ld) { return aligned(p, 16) && ld * size_of(t) % 16 == 0; }

// The wide-tile kernel reads its operands through 31-bit byte offsets: from
// the start of A where rows are gathered, of the tile's rows where they are
// consecutive, of a group's rows for the weight gradient, and of a group's weights.
inline bool wide_tiles(const GroupedArgs &a, GroupedMode mode) {
  const int64_t limit = (int64_t)1 << 30;  // elements
  if (!a.vec || a.a_rows < 1) return false;
  if ((int64_t)a.N * a.K >= limit || 256 * a.ld_rows >= limit) return false;
  if (mode == kWgrad) return a.P * a.ld_w < limit && a.a_rows * a.ld_rows < limit;
  return !a.a_row || a.a_rows * a.ld_rows < limit;
}

// For a single matrix those offsets go from the tile's first row on, and from each step's first of 64 terms where rows are the
// terms; only the columns of a gated product lie apart, in the halves of W.
inline bool wide_tiles_dense(const DenseArgs &a, bool gated) {
  const int64_t limit = (int64_t)1 << 30;  // elements
  if (!a.vec || a.a_rows < 1 || 256 * a.ld_rows >= limit || 256 * a.ld_w >= limit) return false;
  return !gated || (int64_t)a.N * a.K < limit;
}

inline int status(hipError_t e) {
  return e == hipSuccess ? MOE_OK : e == hipErrorInvalidConfiguration ? MOE_EUNSUPPORTED : MOE_EHIP;
}

}  // namespace moe
