// The norms between two blocks of fp16 streams (norm_kernel.h).
#include "norm_kernel.h"

namespace hr {

void launch_norm_f16(const NormArgs& a, hipStream_t s) { launch_length<kDtF16, kDtF16>(a, s); }

}  // namespace hr
