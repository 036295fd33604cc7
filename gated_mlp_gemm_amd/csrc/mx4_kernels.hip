// 4-bit weights: laying them out (quantize), reading them back (dequantize), and the
// products of few rows with them (mx4_few.hpp).
//
// A number is a code of E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times
// a power of two that 32 consecutive numbers of a row share, 2^(S - 127); S = 255
// makes them NaN.
#include "launch.hpp"

#include "device.hpp"
#include "mx4_few.hpp"

#include <atomic>

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
// what is above 6 becomes 6.  (A group whose largest magnitude is below 2^-124 has S = 0, and
// codes of 2^-127: 2^-124 would be 8 of them, and what is at most 2^-129, a quarter,
// becomes zero.)  Four lanes
// have a group, 8 numbers each: 16 bytes in, 4 bytes out a lane.  Bound by its bytes:
// 37889 x 3616 66 us, 5.2 TB/s; 9728 x 896 5.6 us.
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

// One launch; hipErrorNotSupported where a compute unit's LDS does not hold the scales.
template <bool GATED, int R, int NX, int D, int W>
static hipError_t run_few(const uint16_t *X, const uint8_t *Q, const uint8_t *S, uint16_t *Y, int M,
                          int rows, int K, hipStream_t stream) {
    using P = Mx4Few<GATED, R, NX, D, W>;
    constexpr int kLds = 160 * 1024;
    if (P::lds_bytes(K) > kLds) return hipErrorNotSupported;
    const auto kernel = mx4_few_kernel<GATED, R, NX, D, W>;
    // a device takes more than 64 KiB of LDS a launch once it has been told so
    static std::atomic<uint64_t> told[4];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    std::atomic<uint64_t> &mine = told[(dev >> 6) & 3];
    if (!(mine.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (e != hipSuccess) return e;
        mine.fetch_or(uint64_t{1} << (dev & 63), std::memory_order_release);
    }
    hipLaunchKernelGGL(kernel, dim3((rows + P::kRows - 1) / P::kRows), dim3(P::kThreads),
                       P::lds_bytes(K), stream, X, Q, S, Y, M, rows, K);
    return hipGetLastError();
}

// Rows of the weight a workgroup takes, by the 16-row tiles there are for a compute
// unit: every workgroup reads all the activations, so more where that leaves the
// device enough of them.  Measured, us, activations x weight (R = 1 / 2 / 4):
//   M=16  896 x 4864 4.2 / 5.0 / 6.7, 8192 x 29568 47.1 / 36.5 / 49.6,
//         27648 x 5120 29.0 / 24.7 / 20.9
//   M=64  896 x 4864 8.8 / 9.8 / 14.8, 8192 x 29568 113 / 71 / 94,
//         27648 x 5120 68 / 50 / 41
// With at most 4 rows of activations there is little to share: R = 1 (37888 x 3584 14.0
// against 14.5 us), with 8 waves for 4 where a compute unit has one workgroup (3584 x
// 18944 8.3 against 9.5), R = 2 for long rows of many (59136 x 8192 47.5 against 51.3).
template <bool GATED>
static hipError_t launch_few(const uint16_t *X, const uint8_t *Q, const uint8_t *S, uint16_t *Y,
                             int M, int rows, int K, int cus, hipStream_t stream) {
    const int64_t tiles = (static_cast<int64_t>(rows) + 15) / 16;
    const int r = tiles <= cus ? 1 : tiles < 4 * static_cast<int64_t>(cus) ? 2 : 4;
#define SWIGLU_FEW(R, NX, D, W) run_few<GATED, R, NX, D, W>(X, Q, S, Y, M, rows, K, stream)
    if (M <= 4) {
        if (r == 1) return SWIGLU_FEW(1, 1, 4, 8);
        if (r == 4 && K >= 8192) return SWIGLU_FEW(2, 1, 4, 4);
        return SWIGLU_FEW(1, 1, 4, 4);
    }
    if (M <= 8) return r == 1 ? SWIGLU_FEW(1, 2, 2, 8) : SWIGLU_FEW(2, 2, 2, 4);
    if (M <= 16)
        return r == 1 ? SWIGLU_FEW(1, 4, 2, 4)
                      : r == 2 ? SWIGLU_FEW(2, 4, 2, 4) : SWIGLU_FEW(4, 4, 2, 4);
    if (M <= 32)
        return r == 1 ? SWIGLU_FEW(1, 8, 2, 4)
                      : r == 2 ? SWIGLU_FEW(2, 8, 2, 4) : SWIGLU_FEW(4, 8, 1, 4);
    if (M <= 48)
        return r == 1 ? SWIGLU_FEW(1, 12, 1, 8)
                      : r == 2 ? SWIGLU_FEW(2, 12, 1, 8) : SWIGLU_FEW(4, 12, 1, 4);
    return r == 1 ? SWIGLU_FEW(1, 16, 1, 8)
                  : r == 2 ? SWIGLU_FEW(2, 16, 1, 4) : SWIGLU_FEW(4, 16, 1, 4);
#undef SWIGLU_FEW
}

hipError_t launch_mx4_few(const uint16_t *X, const uint8_t *Q, const uint8_t *S, uint16_t *Y, int M,
                          int rows, int K, bool gated, int cus, hipStream_t stream) {
    return gated ? launch_few<true>(X, Q, S, Y, M, rows, K, cus, stream)
                 : launch_few<false>(X, Q, S, Y, M, rows, K, cus, stream);
}

}  // namespace swiglu
