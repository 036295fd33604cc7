// The router in front of a table of experts or adapters, and its gradient.
//
// For row m of the logits z [M][E], p = softmax(z[m]); the k largest logits
// (ties: the lowest index) become ids[m][0..k) in descending order, with
// weights p[id], or p[id] / (sum of the row's picked p) when normalised.  A
// row routes if `valid` says so and it has a logit above -inf; an expert whose
// logit is -inf is never picked (id -1, weight 0).  Over the n rows that
// route, with c[e] picks of expert e and C = sum c,
//
//     loss = E sum_e (c[e] / C) (sum_m p[m][e] / n).
//
// Gradient by the logits of (d_weights, d_loss): with c, C and n constant and
// g[e] = d_loss E c[e] / (C n),
//     raw weights    G = g + d_weights at the picked e,  dz = p (G - sum p G)
//     normalised     dz = p (g - sum p g) + w (dw - sum w dw) at the picked e.
//
// A row is spread over LPR lanes, 8 neighbouring logits a lane, so a wave
// works on 64 / LPR rows at once: the k rounds of arg-max are instructions,
// not memory, and bound the larger calls, so every lane has to count in them
// (a row a wave would leave most lanes idle at E <= 64 and run the cross-lane
// steps once a row instead of once for 64 / LPR of them).
#include "launch.hpp"

#include "device.hpp"
#include "gemm_core.hpp"

namespace swiglu {

constexpr int kRouteThreads = 1024;
constexpr int kRouteValues = 8;      // logits a lane
constexpr float kNegInf = -__builtin_inff();

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
// The value of the lane that step STEP of an all-reduce over 2^(STEP+1)
// neighbouring lanes pairs this one with (each half already holds one value).
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
    if constexpr (STEP == 0) return dpp<0xB1>(v);         // quad_perm 1 0 3 2
    else if constexpr (STEP == 1) return dpp<0x4E>(v);    // quad_perm 2 3 0 1
    else if constexpr (STEP == 2) return dpp<0x141>(v);   // mirror within 8
    else if constexpr (STEP == 3) return dpp<0x140>(v);   // mirror within 16
    else return __shfl_xor(v, 1 << STEP);
}
template <int STEP>
__device__ __forceinline__ float partner_f(float v) {
    return __builtin_bit_cast(float, partner<STEP>(__builtin_bit_cast(uint32_t, v)));
}
// The larger of two, or NaN if one is NaN (one instruction): a row with a NaN
// routes, with weights of NaN.
__device__ __forceinline__ float nan_max(float a, float b) {
    return __builtin_elementwise_maximum(a, b);
}
template <int LPR, int STEP = 0>
__device__ __forceinline__ float row_max(float v) {
    if constexpr ((1 << STEP) < LPR) return row_max<LPR, STEP + 1>(nan_max(v, partner_f<STEP>(v)));
    else return v;
}
template <int LPR, int STEP = 0>
__device__ __forceinline__ float row_sum(float v) {
    if constexpr ((1 << STEP) < LPR) return row_sum<LPR, STEP + 1>(v + partner_f<STEP>(v));
    else return v;
}
// The larger key of the row, and of equal keys the lower index.
template <int LPR, int STEP = 0>
__device__ __forceinline__ void row_best(uint32_t &key, uint32_t &idx) {
    if constexpr ((1 << STEP) < LPR) {
        const uint32_t k = partner<STEP>(key), i = partner<STEP>(idx);
        const bool take = k > key || (k == key && i < idx);
        key = take ? k : key;
        idx = take ? i : idx;
        row_best<LPR, STEP + 1>(key, idx);
    }
}
// Unsigned keys in the order of the floats, and back.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);   // (-0 counts as 0)
    return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __builtin_bit_cast(float, k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kNegInfKey = 0x007FFFFFu;   // order_key(-inf)

// Logits 8 li .. 8 li + 7 of a row (-inf past the end).
template <bool kBf16>
__device__ __forceinline__ void load_logits(const void *z, int64_t row, int E, int e0, bool vec,
                                            float (&v)[kRouteValues]) {
    const int64_t at = row * E + e0;
    if constexpr (kBf16) {
        const uint16_t *p = static_cast<const uint16_t *>(z) + at;
        if (vec && e0 < E) {
            const u32x4 c = gload16(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __builtin_bit_cast(float, c[i] << 16);
                v[2 * i + 1] = __builtin_bit_cast(float, c[i] & 0xFFFF0000u);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i)
            v[i] = e0 + i < E ? __builtin_bit_cast(float, static_cast<uint32_t>(p[i]) << 16) : kNegInf;
    } else {
        const float *p = static_cast<const float *>(z) + at;
        if (vec && e0 < E) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i) v[i] = e0 + i < E ? p[i] : kNegInf;
    }
}

// Softmax of the row (v becomes p; zeros where it does not route); returns
// whether it routes, and its maximum and 1 / sum.
template <int LPR>
__device__ __forceinline__ bool row_softmax(float (&v)[kRouteValues], bool wanted, float &top,
                                            float &inv) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < kRouteValues; ++i) m = nan_max(m, v[i]);
    top = row_max<LPR>(m);
    const bool live = wanted && top != kNegInf;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kRouteValues; ++i) {
        v[i] = live ? expf(v[i] - top) : 0.0f;
        s += v[i];
    }
    s = row_sum<LPR>(s);
    inv = live ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < kRouteValues; ++i) v[i] *= inv;
    return live;
}

struct RouteArgs {
    const void *logits;
    const uint8_t *valid;
    int *ids;
    float *weights;
    int *counts;    // [E + 1]: picks of each expert, rows that route
    float *loss;
    int64_t M;
    int E, k;
    int normalize, vec;
    uint64_t *partials;   // [grid][E + 1]: {sum of p, picks}; unused by a grid of one
    unsigned *counter;
};

// The loss and the counts over all rows: workgroup b leaves its sums of p and
// its picks in partials[b] (device-scope stores), and the last to arrive adds
// them up in the order of b (so that the sums do not depend on which one that
// is).
template <bool kBf16, int LPR>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs x) {
    constexpr int kRowsPass = kRouteThreads / LPR;
    constexpr int kMaxE = LPR * kRouteValues;
    constexpr int kWaves = kRouteThreads / 64;
    constexpr int kHeld = (kMaxRouteK + LPR - 1) / LPR;
    __shared__ unsigned hist[kMaxE + 1];
    __shared__ float psum[kWaves][kMaxE];
    __shared__ double terms[kRouteThreads];
    __shared__ unsigned arrived;
    const int tid = threadIdx.x, li = tid % LPR, group = tid / LPR;
    const int e0 = li * kRouteValues;
    for (int e = tid; e <= kMaxE; e += kRouteThreads) hist[e] = 0u;
    __syncthreads();

    float mine[kRouteValues] = {};
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRowsPass; first < x.M;
         first += static_cast<int64_t>(gridDim.x) * kRowsPass) {
        const int64_t row = first + group;
        const bool here = row < x.M;
        float v[kRouteValues];
        load_logits<kBf16>(x.logits, here ? row : 0, x.E, e0, x.vec != 0, v);
        if (x.vec && e0 >= x.E) {
#pragma unroll
            for (int i = 0; i < kRouteValues; ++i) v[i] = kNegInf;
        }
        uint32_t key[kRouteValues];
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i) key[i] = order_key(v[i]);
        float top, inv;
        const bool live =
            row_softmax<LPR>(v, here && (x.valid == nullptr || x.valid[row] != 0), top, inv);
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i) mine[i] += v[i];
        if (live && li == 0) atomicAdd(&hist[kMaxE], 1u);

        int id[kHeld];
        float w[kHeld];
        float total = 0.0f;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            id[h] = -1;
            w[h] = 0.0f;
        }
#pragma nounroll
        for (int j = 0; j < x.k; ++j) {
            uint32_t best = key[0], at = e0;
#pragma unroll
            for (int i = 1; i < kRouteValues; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = e0 + i;
                }
            row_best<LPR>(best, at);
#pragma unroll
            for (int i = 0; i < kRouteValues; ++i)
                if (at == static_cast<uint32_t>(e0 + i)) key[i] = 0u;
            const bool pick = live && best > kNegInfKey;
            const float e = pick ? expf(key_value(best) - top) : 0.0f;
            total += e;
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (j == h * LPR + li) {
                    id[h] = pick ? static_cast<int>(at) : -1;
                    w[h] = e;
                }
            if (pick && li == 0) atomicAdd(&hist[at], 1u);
        }
        const float scale = x.normalize ? (total > 0.0f ? 1.0f / total : 0.0f) : inv;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int j = h * LPR + li;
            if (here && j < x.k) {
                x.ids[row * x.k + j] = id[h];
                x.weights[row * x.k + j] = w[h] * scale;
            }
        }
    }

    // sums of p of the wave's row groups, then of the waves
#pragma unroll
    for (int i = 0; i < kRouteValues; ++i) {
#pragma unroll
        for (int d = LPR; d < 64; d *= 2) mine[i] += __shfl_xor(mine[i], d);
        if ((tid & 63) < LPR) psum[tid / 64][e0 + i] = mine[i];
    }
    __syncthreads();
    auto block_sum = [&](int e) {
        float s = 0.0f;
        for (int w = 0; w < kWaves; ++w) s += psum[w][e];
        return s;
    };

    double term = 0.0;
    if (gridDim.x == 1) {
        for (int e = tid; e < x.E; e += kRouteThreads) {
            x.counts[e] = static_cast<int>(hist[e]);
            term += static_cast<double>(hist[e]) * block_sum(e);
        }
        if (tid == 0) x.counts[x.E] = static_cast<int>(hist[kMaxE]);
    } else {
        const int width = x.E + 1;
        uint64_t *own = x.partials + static_cast<int64_t>(blockIdx.x) * width;
        for (int e = tid; e < width; e += kRouteThreads) {
            const uint64_t c = e < x.E ? hist[e] : hist[kMaxE];
            const uint32_t s = e < x.E ? __builtin_bit_cast(uint32_t, block_sum(e)) : 0u;
            __hip_atomic_store(own + e, (static_cast<uint64_t>(s) << 32) | c, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        }
        wait_vmcnt<0>();   // this wave's sums are visible device-wide
        __syncthreads();   // ... and every wave's
        if (tid == 0)
            arrived = __hip_atomic_fetch_add(x.counter, 1u, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (arrived + 1 != gridDim.x) return;
        if (tid == 0)
            __hip_atomic_store(x.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // `parts` threads an expert, each its own run of workgroups
        constexpr int kParts = kRouteThreads / (2 * kMaxE) > 0 ? kRouteThreads / (2 * kMaxE) : 1;
        __shared__ double part_p[kParts][kMaxE + 1];
        __shared__ unsigned part_c[kParts][kMaxE + 1];
        const int G = gridDim.x;
        for (int i = tid; i < kParts * width; i += kRouteThreads) {
            const int part = i / width, e = i % width;
            const int b0 = part * G / kParts, b1 = (part + 1) * G / kParts;
            double s = 0.0;
            unsigned c = 0;
#pragma unroll 16
            for (int b = b0; b < b1; ++b) {
                const uint64_t q = __hip_atomic_load(x.partials + static_cast<int64_t>(b) * width + e,
                                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s += __builtin_bit_cast(float, static_cast<uint32_t>(q >> 32));
                c += static_cast<uint32_t>(q);
            }
            part_p[part][e] = s;
            part_c[part][e] = c;
        }
        __syncthreads();
        for (int e = tid; e < width; e += kRouteThreads) {
            double s = 0.0;
            unsigned c = 0;
            for (int p = 0; p < kParts; ++p) {
                s += part_p[p][e];
                c += part_c[p][e];
            }
            x.counts[e] = static_cast<int>(c);
            if (e < x.E) term += s * c;
            hist[e < x.E ? e : kMaxE] = c;
        }
    }
    // sum of the terms and the total of the picks, over the threads in a tree
    terms[tid] = term;
    __syncthreads();
    for (int d = kRouteThreads / 2; d > 0; d /= 2) {
        if (tid < d) terms[tid] += terms[tid + d];
        __syncthreads();
    }
    const double sum = terms[0];
    __syncthreads();
    double picks = 0.0;
    for (int e = tid; e < x.E; e += kRouteThreads) picks += hist[e];
    terms[tid] = picks;
    __syncthreads();
    for (int d = kRouteThreads / 2; d > 0; d /= 2) {
        if (tid < d) terms[tid] += terms[tid + d];
        __syncthreads();
    }
    if (tid == 0) {
        const double C = terms[0], n = hist[kMaxE];
        *x.loss = static_cast<float>(C > 0.0 ? x.E * sum / (C * n) : 0.0);
    }
}

struct RouteBackwardArgs {
    const void *logits;
    const uint8_t *valid;
    const int *ids;
    const float *weights;
    const int *counts;
    const float *d_weights;   // null: zeros
    const float *d_loss;      // null: zero
    void *d_logits;
    int64_t M;
    int E, k;
    int normalize, vec;
};

template <bool kBf16, int LPR>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBackwardArgs x) {
    constexpr int kThreads = 256, kRowsPass = kThreads / LPR;
    constexpr int kHeld = (kMaxRouteK + LPR - 1) / LPR;
    __shared__ int total_picks;
    const int tid = threadIdx.x, li = tid % LPR, group = tid / LPR;
    const int e0 = li * kRouteValues;
    if (tid == 0) total_picks = 0;
    __syncthreads();
    int picks = 0;
    for (int e = tid; e < x.E; e += kThreads) picks += x.counts[e];
    if (picks) atomicAdd(&total_picks, picks);
    __syncthreads();
    const float n = static_cast<float>(max(x.counts[x.E], 1));
    const float d_loss = x.d_loss ? *x.d_loss : 0.0f;
    const float each = d_loss * x.E / (static_cast<float>(max(total_picks, 1)) * n);
    float g[kRouteValues];
#pragma unroll
    for (int i = 0; i < kRouteValues; ++i)
        g[i] = e0 + i < x.E ? each * static_cast<float>(x.counts[e0 + i]) : 0.0f;

    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRowsPass; first < x.M;
         first += static_cast<int64_t>(gridDim.x) * kRowsPass) {
        const int64_t row = first + group;
        const bool here = row < x.M;
        const int64_t at = here ? row : 0;
        float p[kRouteValues];
        load_logits<kBf16>(x.logits, at, x.E, e0, x.vec != 0, p);
        if (x.vec && e0 >= x.E) {
#pragma unroll
            for (int i = 0; i < kRouteValues; ++i) p[i] = kNegInf;
        }
        // pick j = h LPR + li of the row
        int id[kHeld];
        float w[kHeld], dw[kHeld];
        float wdw = 0.0f;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int j = h * LPR + li;
            const bool held = j < x.k;
            id[h] = held ? x.ids[at * x.k + j] : -1;
            w[h] = held && id[h] >= 0 ? x.weights[at * x.k + j] : 0.0f;
            dw[h] = held && id[h] >= 0 && x.d_weights ? x.d_weights[at * x.k + j] : 0.0f;
            wdw += w[h] * dw[h];
        }
        float top, inv;
        const bool live =
            row_softmax<LPR>(p, here && (x.valid == nullptr || x.valid[at] != 0), top, inv);
        if (x.normalize) {
            wdw = row_sum<LPR>(wdw);
#pragma unroll
            for (int h = 0; h < kHeld; ++h) dw[h] = w[h] * (dw[h] - wdw);
        }
        // each pick's share, at its expert
        float share[kRouteValues] = {};
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int held = min(LPR, x.k - h * LPR);
#pragma nounroll
            for (int j = 0; j < held; ++j) {
                const int from = (tid & 63) / LPR * LPR + j;
                const int e = __shfl(id[h], from);
                const float d = __shfl(dw[h], from);
#pragma unroll
                for (int i = 0; i < kRouteValues; ++i)
                    if (e == e0 + i) share[i] += d;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i)
            dot += p[i] * (x.normalize ? g[i] : g[i] + share[i]);
        dot = row_sum<LPR>(dot);
        float dz[kRouteValues];
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i) {
            dz[i] = x.normalize ? p[i] * (g[i] - dot) + share[i] : p[i] * (g[i] + share[i] - dot);
            if (!live) dz[i] = 0.0f;
        }
        if (!here || e0 >= x.E) continue;
        const int64_t out = row * x.E + e0;
        if constexpr (kBf16) {
            uint16_t *o = static_cast<uint16_t *>(x.d_logits) + out;
            if (x.vec) {
                gstore16(o, u32x4{pack_bf16x2(dz[0], dz[1]), pack_bf16x2(dz[2], dz[3]),
                                  pack_bf16x2(dz[4], dz[5]), pack_bf16x2(dz[6], dz[7])});
            } else {
#pragma unroll
                for (int i = 0; i < kRouteValues; ++i)
                    if (e0 + i < x.E) o[i] = to_bf16(dz[i]);
            }
        } else {
            float *o = static_cast<float *>(x.d_logits) + out;
            if (x.vec) {
                *reinterpret_cast<f32x4 *>(o) = f32x4{dz[0], dz[1], dz[2], dz[3]};
                *reinterpret_cast<f32x4 *>(o + 4) = f32x4{dz[4], dz[5], dz[6], dz[7]};
            } else {
#pragma unroll
                for (int i = 0; i < kRouteValues; ++i)
                    if (e0 + i < x.E) o[i] = dz[i];
            }
        }
    }
}

// Lanes a row: the smallest of 4, 8, ..., 64 that hold E logits.
static int lanes_per_row(int64_t E) {
    int lpr = 4;
    while (lpr * kRouteValues < E) lpr *= 2;
    return lpr;
}

// Workgroups of the forward kernel: one per pass of rows, at most one a
// compute unit.
static int route_grid(int64_t M, int64_t E, int cus) {
    const int64_t per = kRouteThreads / lanes_per_row(E);
    const int64_t passes = (M + per - 1) / per;
    return static_cast<int>(passes < cus ? passes : cus);
}

uint64_t route_partials_bytes(int64_t M, int64_t E, int cus) {
    const int grid = route_grid(M, E, cus);
    return grid > 1 ? static_cast<uint64_t>(grid) * (E + 1) * 8 : 0;
}

template <bool kBf16>
static void run_route(int lpr, int grid, const RouteArgs &a, hipStream_t stream) {
    const dim3 g(grid), t(kRouteThreads);
    switch (lpr) {
        case 4: hipLaunchKernelGGL((route_kernel<kBf16, 4>), g, t, 0, stream, a); break;
        case 8: hipLaunchKernelGGL((route_kernel<kBf16, 8>), g, t, 0, stream, a); break;
        case 16: hipLaunchKernelGGL((route_kernel<kBf16, 16>), g, t, 0, stream, a); break;
        case 32: hipLaunchKernelGGL((route_kernel<kBf16, 32>), g, t, 0, stream, a); break;
        default: hipLaunchKernelGGL((route_kernel<kBf16, 64>), g, t, 0, stream, a); break;
    }
}
template <bool kBf16>
static void run_route_backward(int lpr, int grid, const RouteBackwardArgs &a, hipStream_t stream) {
    const dim3 g(grid), t(256);
    switch (lpr) {
        case 4: hipLaunchKernelGGL((route_backward_kernel<kBf16, 4>), g, t, 0, stream, a); break;
        case 8: hipLaunchKernelGGL((route_backward_kernel<kBf16, 8>), g, t, 0, stream, a); break;
        case 16: hipLaunchKernelGGL((route_backward_kernel<kBf16, 16>), g, t, 0, stream, a); break;
        case 32: hipLaunchKernelGGL((route_backward_kernel<kBf16, 32>), g, t, 0, stream, a); break;
        default: hipLaunchKernelGGL((route_backward_kernel<kBf16, 64>), g, t, 0, stream, a); break;
    }
}

static bool vector_rows(int64_t E, const void *p, const void *q) {
    return E % kRouteValues == 0 &&
           ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
}

hipError_t launch_route(const void *logits, bool bf16, const uint8_t *valid, int *ids,
                        float *weights, int *counts, float *loss, int64_t M, int E, int k,
                        bool normalize, void *partials, uint64_t partial_bytes, unsigned *counter,
                        int cus, hipStream_t stream) {
    int grid = route_grid(M, E, cus);
    if (grid > 1 && (partials == nullptr || counter == nullptr ||
                     partial_bytes < route_partials_bytes(M, E, cus)))
        grid = 1;
    if (grid < 1) grid = 1;   // M == 0: the counts and the loss are still written
    const RouteArgs a{logits, valid, ids, weights, counts, loss, M, E, k, normalize ? 1 : 0,
                      vector_rows(E, logits, nullptr) ? 1 : 0, static_cast<uint64_t *>(partials),
                      counter};
    if (bf16) run_route<true>(lanes_per_row(E), grid, a, stream);
    else run_route<false>(lanes_per_row(E), grid, a, stream);
    return hipGetLastError();
}

hipError_t launch_route_backward(const void *logits, bool bf16, const uint8_t *valid,
                                 const int *ids, const float *weights, const int *counts,
                                 const float *d_weights, const float *d_loss, void *d_logits,
                                 int64_t M, int E, int k, bool normalize, int cus,
                                 hipStream_t stream) {
    const int lpr = lanes_per_row(E);
    const int64_t per = 256 / lpr, passes = (M + per - 1) / per;
    const int64_t most = static_cast<int64_t>(cus) * 8;
    const int grid = static_cast<int>(passes < most ? passes : most);
    const RouteBackwardArgs a{logits, valid, ids, weights, counts, d_weights, d_loss, d_logits, M, E,
                              k, normalize ? 1 : 0, vector_rows(E, logits, d_logits) ? 1 : 0};
    if (bf16) run_route_backward<true>(lpr, grid, a, stream);
    else run_route_backward<false>(lpr, grid, a, stream);
    return hipGetLastError();
}

}  // namespace swiglu
