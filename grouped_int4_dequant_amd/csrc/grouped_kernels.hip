// Products grouped by expert with 16-bit operands, and their gradients, for
// gfx950.
//
//   forward          C[p][n]  = sum_k A[row(p)][k] W_e[n][k]
//   input gradient   dA[p][k] = sum_n dC[p][n] W_e[n][k]
//   weight gradient  dW_e[n][k] = sum_{p of e} dC[p][n] A[row(p)][k]
//
// All three are out[i][j] = sum_r L[i][r] R[j][r] with another dimension cut by
// the groups and another operand lying across r. Products are exact in fp32 and
// accumulate in fp32; the result is rounded once, to the output's type.
//
// The kernels are in grouped_tiles.h.

#include "grouped_tiles.h"

namespace moe {

hipError_t launch_grouped(const GroupedArgs &a, GroupedMode mode, bool fp16, hipStream_t s) {
  switch (mode) {
    case kFwd: return fp16 ? launch_vec<Fp16, kFwd>(a, s) : launch_vec<Bf16, kFwd>(a, s);
    case kDgrad: return fp16 ? launch_vec<Fp16, kDgrad>(a, s) : launch_vec<Bf16, kDgrad>(a, s);
    default: return fp16 ? launch_vec<Fp16, kWgrad>(a, s) : launch_vec<Bf16, kWgrad>(a, s);
  }
}

}  // namespace moe
