// Where the pieces of a contraction begin that is split along K.
#pragma once

#include <hip/hip_runtime.h>

namespace swiglu {

// First K step of piece p of a contraction of nk steps in `pieces` pieces,
// floor(p nk / pieces); p == pieces gives nk, the last piece's end.  With nk =
// q pieces + r that is p q + floor(p r / pieces), whose products stay below nk and
// pieces^2: p nk itself passes 31 bits where the weights' gradients contract over
// 2^30 rows (2^24 steps in 512 pieces).
__device__ __forceinline__ int piece_begin(int p, int nk, int pieces) {
    return p * (nk / pieces) + p * (nk % pieces) / pieces;
}

}  // namespace swiglu
