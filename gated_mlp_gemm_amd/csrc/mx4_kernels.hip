// 4-bit weights: laying them out (quantize) and reading them back (dequantize).
//
// A number is a code of E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times
// a power of two that 32 consecutive numbers of a row share, 2^(S - 127); S = 255
// makes them NaN.
#include "launch.hpp"

#include "device.hpp"

namespace swiglu {

typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));

// (by value: a bit cast of a vector's element as it stands reads its first)
__device__ __forceinline__ bf16_pair pair_of(uint32_t v) { return __builtin_bit_cast(bf16_pair, v); }

// The largest of the four lanes of a quad (DPP quad_perm [1,0,3,2], then [2,3,0,1]).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true));
    v = v > a ? v : a;
    const uint32_t b = static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true));
    return v > b ? v : b;
}

// S from the largest magnitude's exponent, so that it lies in [4, 8) of 2^(S - 127):
// what is above 6 becomes 6.  (Groups below 2^-124 keep S = 0, and zeros.)  Four lanes
// have a group, 8 numbers each: 16 bytes in, 4 bytes out a lane.
__global__ __launch_bounds__(256) void quantize_mx4_kernel(const uint16_t *__restrict__ x,
                                                           uint32_t *__restrict__ q,
                                                           uint8_t *__restrict__ s,
                                                           int64_t nchunks) {
    // (nchunks is a multiple of 4: the lanes of a quad stay together)
    for (int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; c < nchunks;
         c += (int64_t)gridDim.x * blockDim.x) {
        const u32x4 v = gload16(x + c * 8);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = v[i] & 0x7FFFu, hi = (v[i] >> 16) & 0x7FFFu;
            top = top > lo ? top : lo;
            top = top > hi ? top : hi;
        }
        top = quad_max(top);
        const uint32_t e = top >> 7;
        const uint32_t scale = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
        const float f = __builtin_bit_cast(float, scale << 23);
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[0]), f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[1]), f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[2]), f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[3]), f, 3);
        q[c] = e == 255u ? 0u : w;
        if ((c & 3) == 0) s[c >> 2] = static_cast<uint8_t>(scale);
    }
}

__global__ __launch_bounds__(256) void dequantize_mx4_kernel(const uint32_t *__restrict__ q,
                                                             const uint8_t *__restrict__ s,
                                                             uint16_t *__restrict__ x,
                                                             int64_t nchunks) {
    for (int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; c < nchunks;
         c += (int64_t)gridDim.x * blockDim.x) {
        const uint32_t w = q[c];
        const float f = __builtin_bit_cast(float, static_cast<uint32_t>(s[c >> 2]) << 23);
        u32x4 v;
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1));
        v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2));
        v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3));
        gstore16(x + c * 8, v);
    }
}

static int chunk_grid(int64_t chunks) {
    const int64_t blocks = (chunks + 255) / 256;
    return static_cast<int>(blocks < 65536 ? blocks : 65536);
}

hipError_t launch_quantize_mx4(const uint16_t *x, uint8_t *q, uint8_t *s, int64_t count,
                               hipStream_t stream) {
    const int64_t chunks = count / 8;
    hipLaunchKernelGGL(quantize_mx4_kernel, dim3(chunk_grid(chunks)), dim3(256), 0, stream, x,
                       reinterpret_cast<uint32_t *>(q), s, chunks);
    return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const uint8_t *q, const uint8_t *s, uint16_t *x, int64_t count,
                                 hipStream_t stream) {
    const int64_t chunks = count / 8;
    hipLaunchKernelGGL(dequantize_mx4_kernel, dim3(chunk_grid(chunks)), dim3(256), 0, stream,
                       reinterpret_cast<const uint32_t *>(q), s, x, chunks);
    return hipGetLastError();
}

}  // namespace swiglu
