// Work items drawn by workgroups: each runs the items of its number and of its number in
// the second round, then those that it draws from a count in the caller's workspace
// (arrivals.hpp: the word needs no initialisation and is zero behind the call; nobody
// waits for anybody).
//
// There is a count for each of the eight XCDs, whose workgroups (numbers equal mod 8)
// draw the items of their residue: the tiles that an XCD works on at a time stay
// neighbours in its L2.  A workgroup draws a whole item before it needs the answer.
#pragma once

#include "arrivals.hpp"

namespace swiglu {

constexpr int kXcds = 8;

// One workgroup's draws; the members marked (one) are its first thread's.
struct Draws {
    uint64_t *word;      // of its XCD
    uint64_t tag;
    int xcd, items;      // the XCD, and its number of items
    int workgroups;      // of all XCDs, a multiple of 8
    Arrival meeting;     // (one)
    bool met;

    // (one) `total` items of all XCDs; the workgroup has one (workgroup < total).
    __device__ __forceinline__ void begin(uint64_t *words, uint64_t tag_, int workgroup,
                                          int workgroups_, int total, bool one) {
        xcd = workgroup % kXcds;
        items = (total - xcd + kXcds - 1) / kXcds;
        word = words + xcd;
        tag = tag_;
        workgroups = workgroups_;
        met = false;
        if (one) meeting.announce(word, tag);
    }
    // (one) Asks; once for each item that the workgroup runs.  So an XCD's workgroups ask
    // as often as it has items, and the last one clears the count.
    __device__ __forceinline__ unsigned ask() {
        if (!met) meeting.settle(word, tag);
        met = true;
        return arrive(word);
    }
    __device__ __forceinline__ void answered(unsigned ticket) {
        if (ticket + 1 == static_cast<unsigned>(items)) arrivals_done(word);
    }
    // The item of a ticket (it may be past the last one).
    __device__ __forceinline__ int item(unsigned ticket) const {
        return xcd + kXcds * static_cast<int>(ticket) + 2 * workgroups;
    }
};

}  // namespace swiglu
