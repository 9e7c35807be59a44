// What hand-overs between workgroups of one kernel share: a tag of the dispatch, by which a reader knows that
// what it reads was written by this dispatch. Each kernel describes its own protocol (the chunked scans a tag word
// behind the values, the gated recurrence a tag within every value).
#ifndef VIMSCAN_HANDOVER_H
#define VIMSCAN_HANDOVER_H

#include <hip/hip_runtime.h>

#include <cstdint>

namespace vimscan_dev {

// Reads of a tag word before a wait of the chunked scans gives up (about a second).
constexpr int kSpinLimit = 1 << 20;

// llvm.amdgcn.dispatch.id: the dispatch packet's index in its queue, which the command processor
// writes into two SGPRs of every wave it launches.
extern "C" __device__ uint64_t vimscan_dispatch_id() __asm("llvm.amdgcn.dispatch.id");

// A tag unique to this kernel dispatch: the packet index and the queue's address, through the
// splitmix64 finaliser (a bijection), so that tags of neighbouring dispatches differ in every bit
// position; never zero.
__device__ __forceinline__ uint64_t dispatch_tag() {
    uint64_t v = vimscan_dispatch_id() ^
                 (reinterpret_cast<uint64_t>(__builtin_amdgcn_queue_ptr()) * 0x9E3779B97F4A7C15ull);
    v = (v ^ (v >> 30)) * 0xBF58476D1CE4E5B9ull;
    v = (v ^ (v >> 27)) * 0x94D049BB133111EBull;
    return (v ^ (v >> 31)) | 1u;
}

}  // namespace vimscan_dev

#endif  // VIMSCAN_HANDOVER_H
