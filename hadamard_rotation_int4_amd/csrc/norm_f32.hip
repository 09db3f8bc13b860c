// The norms between two blocks of fp32 streams with fp32 blocks (norm_kernel.h).
#include "norm_kernel.h"

namespace hr {

void launch_norm_f32(const NormArgs& a, hipStream_t s) { launch_length<kDtF32, kDtF32>(a, s); }

}  // namespace hr
