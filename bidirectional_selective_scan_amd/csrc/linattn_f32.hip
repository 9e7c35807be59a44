// The passes of linear attention in fp32 (linattn_device.h).

#include "linattn_launch.h"

namespace vimscan_dev {
template void launch_lin_pass<float, kLocal>(const LinPasses&, bool, hipStream_t);
template void launch_lin_pass<float, kForward>(const LinPasses&, bool, hipStream_t);
template void launch_lin_pass<float, kGradient>(const LinPasses&, bool, hipStream_t);
template void launch_lin_pass<float, kGradientDots>(const LinPasses&, bool, hipStream_t);
}  // namespace vimscan_dev
