// The norms between two blocks of fp32 streams with bf16 blocks (norm_kernel.h).
#include "norm_kernel.h"

namespace hr {

void launch_norm_f32_bf16(const NormArgs& a, hipStream_t s) { launch_length<kDtF32, kDtBf16>(a, s); }

}  // namespace hr
