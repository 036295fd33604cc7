// Counting the workgroups that have arrived at a meeting, in a word of the caller's
// workspace.
//
// The word needs no initialisation, no memory of the library's own and no launch that
// clears it: its upper 52 bits are the call's tag, a number that the host gives out
// once (next_arrival_tag), its lower 12 the arrivals.  Whatever else the word holds
// (zero, what the workspace held before) means that nobody has arrived.  The last to
// arrive leaves zero, so that a captured call, whose tag is the same at every replay,
// starts anew.  Calls that may run at the same time have workspaces of their own, so
// they cannot meet at one word, however they were enqueued; a count in library memory
// that calls share in turn can be taken by two running calls (a deep queue, a
// captured graph replayed beside other calls).
//
// Memory that happens to hold the tag would pass for arrivals: one of 2^52 values, a
// different one every call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace swiglu {

constexpr int kArrivalBits = 12;   // workgroups of a meeting: fewer than 4096

// In three steps, by one thread of each workgroup.  announce(), early, puts the tag into
// a word that holds zero (what the meeting before left); settle(), before the partial
// results are stored, puts it where announce() met something else.  Both are in flight
// beside other work, and arrive(), behind the stores, is a single addition.  (An
// exchange and an addition at the meeting: the router of M=16384 E=128, 256
// workgroups, with its gradient 31.0 us instead of 28.4.)
struct Arrival {
    uint64_t seen;

    __device__ __forceinline__ void announce(uint64_t *word, uint64_t tag) {
        seen = 0;
        __hip_atomic_compare_exchange_strong(word, &seen, tag, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
    }
    // (No loop: a word without the tag is only changed by an exchange of this call's, so
    // if this one fails, the tag is there.)
    __device__ __forceinline__ void settle(uint64_t *word, uint64_t tag) {
        if (seen != 0 && seen >> kArrivalBits != tag >> kArrivalBits)
            __hip_atomic_compare_exchange_strong(word, &seen, tag, __ATOMIC_RELAXED,
                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};
// Arrivals before this one.
__device__ __forceinline__ unsigned arrive(uint64_t *word) {
    return static_cast<unsigned>(__hip_atomic_fetch_add(word, uint64_t{1}, __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT)) &
           ((1u << kArrivalBits) - 1);
}
// By the last to arrive.
__device__ __forceinline__ void arrivals_done(uint64_t *word) {
    __hip_atomic_store(word, uint64_t{0}, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace swiglu
