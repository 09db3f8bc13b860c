// Launches of the norms between two blocks (norm_kernel.h), and the kernels of bf16
// streams; those of other types are compiled beside them.
#include "norm_kernel.h"

namespace hr {

hipError_t launch_norm(const NormArgs& args, hipStream_t s) {
  NormArgs a = args;
  constexpr float turns[4] = {0.17677669529663687f, 0.125f, 0.08838834764831845f, 0.0625f};
  a.turn = a.order == 0 ? 1.0f : turns[a.order == 32 ? 0 : a.order == 64 ? 1 : a.order == 128 ? 2 : 3];
  if (a.x_dtype == kDtBf16) launch_length<kDtBf16, kDtBf16>(a, s);
  else if (a.x_dtype == kDtF16) launch_norm_f16(a, s);
  else if (a.dtype == kDtBf16) launch_norm_f32_bf16(a, s);
  else if (a.dtype == kDtF16) launch_norm_f32_f16(a, s);
  else launch_norm_f32(a, s);
  return hipGetLastError();
}

}  // namespace hr
