// Launches of the pass of linear attention: the instance for the head's dimensions.
#ifndef VIMSCAN_LINATTN_LAUNCH_H
#define VIMSCAN_LINATTN_LAUNCH_H

#include "linattn_device.h"

namespace vimscan_dev {

template <typename IO, int NK, int NV, bool kVec, int kKind>
void launch_lin_instance(const LinPasses& p, hipStream_t s) {
    hipLaunchKernelGGL((k_lin_pass<IO, NK, NV, kVec, kKind>), dim3(static_cast<unsigned>(p.a[0].waves * p.count)), dim3(64), 0, s, p);
}
template <typename IO, int NK, bool kVec, int kKind>
void launch_lin_outputs(const LinPasses& p, hipStream_t s) {
    // (the instances that lin_output_tiles can ask for)
    constexpr int e = sizeof(IoElem<IO>);
    if constexpr (e == 2 && NK <= 4) {
        if (vimscan_host::lin_output_tiles(e, p.a[0].K, p.a[0].V) == 4) return launch_lin_instance<IO, NK, 4, kVec, kKind>(p, s);
    }
    launch_lin_instance<IO, NK, 2, kVec, kKind>(p, s);
}
template <typename IO, bool kVec, int kKind>
void launch_lin_dims(const LinPasses& p, hipStream_t s) {
    switch (vimscan_host::lin_contract_tiles(p.a[0].K)) {
        case 2: return launch_lin_outputs<IO, 2, kVec, kKind>(p, s);
        case 4: return launch_lin_outputs<IO, 4, kVec, kKind>(p, s);
        default: return launch_lin_outputs<IO, 8, kVec, kKind>(p, s);
    }
}
template <typename IO, int kKind>
void launch_lin_pass(const LinPasses& p, bool vec, hipStream_t s) {
    if (vec) launch_lin_dims<IO, true, kKind>(p, s);
    else launch_lin_dims<IO, false, kKind>(p, s);
}

}  // namespace vimscan_dev

#endif  // VIMSCAN_LINATTN_LAUNCH_H
