// The passes of linear attention in bf16 (linattn_device.h).

#include "linattn_launch.h"

namespace vimscan_dev {
template void launch_lin_pass<Bf16, kLocal>(const LinPasses&, bool, hipStream_t);
template void launch_lin_pass<Bf16, kForward>(const LinPasses&, bool, hipStream_t);
template void launch_lin_pass<Bf16, kGradient>(const LinPasses&, bool, hipStream_t);
template void launch_lin_pass<Bf16, kGradientDots>(const LinPasses&, bool, hipStream_t);
}  // namespace vimscan_dev
