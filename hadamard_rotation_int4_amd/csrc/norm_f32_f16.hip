// The norms between two blocks of fp32 streams with fp16 blocks (norm_kernel.h).
#include "norm_kernel.h"

namespace hr {

void launch_norm_f32_f16(const NormArgs& a, hipStream_t s) { launch_length<kDtF32, kDtF16>(a, s); }

}  // namespace hr
