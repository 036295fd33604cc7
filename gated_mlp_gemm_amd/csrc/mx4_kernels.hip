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
// device enough of them.  Measured, us with the weights streamed from memory (R = 1 / 2 /
// 4); the weights have 56, 224 (one form), 320, 512, 608 (the next), 1728, 2368 and 3696
// tiles:
//   M=8   896 x 4864 3.8 / 4.5 / 6.1, 3584 x 18944 12.3 / 16.4 / 25.1, 5120 x 13824 16.3 / 13.1
//         / 19.5, 8192 x 29568 36.1 / 28.5 / 41.8, 9728 x 896 4.7 / 3.5 / 3.4, 27648 x 5120 22.8
//         / 19.7 / 19.0, 37888 x 3584 21.7 / 17.9 / 17.7, 59136 x 8192 63.9 / 56.0 / 53.9
//   M=16  4.3 / 5.1 / 6.4, 16.0 / 21.6 / 29.4, 22.0 / 17.2 / 21.8, 47.4 / 36.7 / 49.4, 3.7 / 3.7
//         / 3.6, 29.3 / 24.9 / 21.4, 27.5 / 21.8 / 19.9, 85.8 / 67.4 / 59.9
//   M=32  5.8 / 6.6 / 8.6, 23.9 / 27.3 / 38.7, 33.4 / 21.5 / 29.5, 70.8 / 45.3 / 65.3, 5.6 / 6.0
//         / 4.5, 43.1 / 34.2 / 25.8, 41.9 / 32.7 / 24.6, 127.2 / 96.4 / 73.4
//   M=48  7.4 / 8.5 / 11.7, 30.3 / 35.4 / 47.0, 42.6 / 27.3 / 35.9, 93.4 / 59.1 / 74.2, 8.8 /
//         7.2 / 5.4, 63.4 / 44.1 / 30.0, 67.2 / 42.5 / 29.2, 190.7 / 124.7 / 96.1
//   M=64  9.0 / 10.7 / 14.0, 37.0 / 44.3 / 57.6, 52.3 / 33.9 / 44.4, 113.4 / 71.4 / 91.6, 10.2 /
//         6.7 / 6.1, 76.5 / 52.4 / 38.9, 81.3 / 40.8 / 39.3, 231.1 / 159.0 / 118.8
// The rule takes the fastest of the three but at 9728 x 896 (short contractions would take
// R = 4 from fewer tiles on: up to 25 % at M=32 and 48) and, 4 % slower at most, for M <= 8
// and wide weights, which share the form of fewer tiles.  Forms between (R = 3, 5, 6, 8, rings
// of 24 rows) are not offered: at M=24 they are within 5 % at 59136 x 8192, but 19.7 (R = 5)
// against 23.7 at 37888 x 3584 and 21.8 (R = 8) against 24.5 at 27648 x 5120.
// With at most 4 rows of activations there is little to share (8 waves, R = 1 / 4 waves,
// R = 1 / 4 waves, R = 2):
//   M=1  896 x 4864 3.6 / 3.7 / 4.6, 3584 x 18944 8.6 / 9.7 / 11.7, 8192 x 29568 25.5 / 24.7 /
//        24.2, 37888 x 3584 18.2 / 13.8 / 14.7, 27648 x 5120 17.5 / 15.0 / 16.5, 59136 x 8192
//        48.6 / 51.4 / 47.7
//   M=4  3.7 / 3.7 / 4.7, 10.1 / 9.9 / 13.8, 29.7 / 28.8 / 25.6, 18.9 / 16.1 / 15.2, 20.1 /
//        17.9 / 17.4, 52.1 / 54.9 / 48.2
// so R = 1, with 8 waves for 4 where a compute unit has one workgroup, and R = 2 for long
// rows of many; the border K = 8192 lies between the last two weights, where M=1 changes
// sides (M=4 would take R = 2 at the three before, by 3 to 11 %).
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
