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
// steps once a row instead of once for 64 / LPR of them).  A round finds the
// largest key, then the lowest index that has it; bf16 logits and their index
// share one word, so that one maximum does both.  What follows from a pick
// (its exponential, its count, its place in the outputs) is done once, pick j
// in lane j of the row.
#include "launch.hpp"

#include "arrivals.hpp"
#include "device.hpp"
#include "gemm_core.hpp"

namespace swiglu {

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
template <int LPR, int STEP = 0>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
    if constexpr ((1 << STEP) < LPR) return row_max_u32<LPR, STEP + 1>(max(v, partner<STEP>(v)));
    else return v;
}
template <int LPR, int STEP = 0>
__device__ __forceinline__ uint32_t row_min_u32(uint32_t v) {
    if constexpr ((1 << STEP) < LPR) return row_min_u32<LPR, STEP + 1>(min(v, partner<STEP>(v)));
    else return v;
}
// Unsigned keys in the order of the floats, and back.  NaN, of either sign (0 / 0 is a
// negative one on many machines), is above all numbers: its row picks it.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);   // (-0 counts as 0)
    return v != v ? 0xFFFFFFFFu : b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
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
    uint64_t *arrivals, tag;   // (arrivals.hpp)
};

// Sum over the lanes of a wave, in every lane.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// The loss and the counts over all rows: workgroup b leaves its sums of p and
// its picks in partials[b] (device-scope stores), and the last to arrive adds
// them up in the order of b (so that the sums do not depend on which one that
// is).  THREADS: 1024, or 256 where those take all rows at once (7.3 -> 5 us at
// M = 1, E = 8: the launch and three memory latencies).
template <bool kBf16, int LPR, int THREADS>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteArgs x) {
    constexpr int kRowsPass = THREADS / LPR;
    constexpr int kMaxE = LPR * kRouteValues;
    constexpr int kWaves = THREADS / 64;
    constexpr int kHeld = (kMaxRouteK + LPR - 1) / LPR;
    __shared__ unsigned hist[kMaxE + 1];
    __shared__ float psum[kWaves][kMaxE];
    __shared__ double sums[kMaxE];   // of p over all rows
    __shared__ unsigned arrived;
    const int tid = threadIdx.x, li = tid % LPR, group = tid / LPR;
    const int e0 = li * kRouteValues;
    for (int e = tid; e <= kMaxE; e += THREADS) hist[e] = 0u;
    __syncthreads();

    Arrival meeting{};
    float mine[kRouteValues] = {};
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRowsPass; first < x.M;
         first += static_cast<int64_t>(gridDim.x) * kRowsPass) {
        const int64_t row = first + group;
        const bool here = row < x.M;
        const bool wanted = here && (x.valid == nullptr || x.valid[row] != 0);
        float v[kRouteValues];
        load_logits<kBf16>(x.logits, here ? row : 0, x.E, e0, x.vec != 0, v);
        // (bf16: the key above, 0xFFFF minus the index below)
        uint32_t key[kRouteValues];
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i) {
            key[i] = order_key(v[i]);
            if constexpr (kBf16) key[i] = (key[i] & 0xFFFF0000u) | (0xFFFFu - (e0 + i));
        }
        float top, inv;
        const bool live = row_softmax<LPR>(v, wanted, top, inv);
        // (in flight beside the picks, not before the logits)
        if (tid == 0 && gridDim.x > 1 && first == static_cast<int64_t>(blockIdx.x) * kRowsPass)
            meeting.announce(x.arrivals, x.tag);
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i) mine[i] += v[i];
        if (live && li == 0) atomicAdd(&hist[kMaxE], 1u);

        // pick j = h LPR + li of the row
        uint32_t picked[kHeld], at[kHeld];
#pragma unroll
        for (int h = 0; h < kHeld; ++h) picked[h] = at[h] = 0u;
#pragma nounroll
        for (int j = 0; j < x.k; ++j) {
            uint32_t best = key[0];
#pragma unroll
            for (int i = 1; i < kRouteValues; ++i) best = max(best, key[i]);
            best = row_max_u32<LPR>(best);
            uint32_t index;
            if constexpr (kBf16) {
                index = 0xFFFFu - (best & 0xFFFFu);
#pragma unroll
                for (int i = 0; i < kRouteValues; ++i) key[i] = key[i] == best ? 0u : key[i];
            } else {
                index = 0xFFFFu;
#pragma unroll
                for (int i = kRouteValues - 1; i >= 0; --i)
                    index = key[i] == best ? static_cast<uint32_t>(e0 + i) : index;
                index = row_min_u32<LPR>(index);
                const uint32_t d = index - e0;
#pragma unroll
                for (int i = 0; i < kRouteValues; ++i) key[i] = d == static_cast<uint32_t>(i) ? 0u : key[i];
            }
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (j == h * LPR + li) {
                    picked[h] = kBf16 ? best & 0xFFFF0000u : best;
                    at[h] = index;
                }
        }
        float w[kHeld], total = 0.0f;
        bool pick[kHeld];
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            // (a negative logit's key ends in ones)
            if (kBf16 && !(picked[h] >> 31)) picked[h] |= 0xFFFFu;
            pick[h] = live && picked[h] > kNegInfKey;
            w[h] = pick[h] ? expf(key_value(picked[h]) - top) : 0.0f;
            total += w[h];
            if (pick[h]) atomicAdd(&hist[at[h]], 1u);
        }
        total = row_sum<LPR>(total);
        // (a row that routes picks its largest logit: its total is 1 at least, or NaN)
        const float scale = x.normalize ? 1.0f / total : inv;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int j = h * LPR + li;
            if (here && j < x.k) {
                x.ids[row * x.k + j] = pick[h] ? static_cast<int>(at[h]) : -1;
                x.weights[row * x.k + j] = pick[h] ? w[h] * scale : 0.0f;
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
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += psum[w][e];
        return s;
    };

    if (gridDim.x == 1) {
        for (int e = tid; e < x.E; e += THREADS) sums[e] = block_sum(e);
    } else {
        if (tid == 0) meeting.settle(x.arrivals, x.tag);
        const int width = x.E + 1;
        uint64_t *own = x.partials + static_cast<int64_t>(blockIdx.x) * width;
        for (int e = tid; e < width; e += THREADS) {
            const uint64_t c = e < x.E ? hist[e] : hist[kMaxE];
            const uint32_t s = e < x.E ? __builtin_bit_cast(uint32_t, block_sum(e)) : 0u;
            __hip_atomic_store(own + e, (static_cast<uint64_t>(s) << 32) | c, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        }
        wait_vmcnt<0>();   // this wave's sums are visible device-wide
        __syncthreads();   // ... and every wave's
        if (tid == 0) arrived = arrive(x.arrivals);
        __syncthreads();
        if (arrived + 1 != gridDim.x) return;
        if (tid == 0) arrivals_done(x.arrivals);
        // as many threads an expert as there are, each its own run of workgroups
        __shared__ double part_p[THREADS];
        __shared__ unsigned part_c[THREADS];
        static_assert(THREADS > kMaxRouteE || THREADS == 256, "256: one workgroup");
        const int parts = min(32, THREADS / width);
        constexpr int kBatch = 20;
        const int G = gridDim.x;
        if (tid < parts * width) {
            const int part = tid / width, e = tid - part * width;
            const int b0 = part * G / parts, b1 = (part + 1) * G / parts;
            double s = 0.0;
            unsigned c = 0;
            for (int b = b0; b < b1; b += kBatch) {   // kBatch loads in flight
                uint64_t q[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    q[i] = b + i < b1 ? __hip_atomic_load(x.partials + static_cast<int64_t>(b + i) * width + e,
                                                          __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                      : 0u;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    s += __builtin_bit_cast(float, static_cast<uint32_t>(q[i] >> 32));
                    c += static_cast<uint32_t>(q[i]);
                }
            }
            part_p[tid] = s;
            part_c[tid] = c;
        }
        __syncthreads();
        for (int e = tid; e < width; e += THREADS) {
            double s = 0.0;
            unsigned c = 0;
            for (int p = 0; p < parts; ++p) {
                s += part_p[p * width + e];
                c += part_c[p * width + e];
            }
            if (e < x.E) sums[e] = s;
            hist[e < x.E ? e : kMaxE] = c;
        }
    }
    __syncthreads();
    for (int e = tid; e <= x.E; e += THREADS)
        x.counts[e] = static_cast<int>(hist[e < x.E ? e : kMaxE]);
    if (tid < 64) {
        double term = 0.0, picks = 0.0;
        for (int e = tid; e < x.E; e += 64) {
            term += hist[e] * sums[e];
            picks += hist[e];
        }
        term = wave_sum(term);
        picks = wave_sum(picks);
        const double n = hist[kMaxE];
        if (tid == 0) *x.loss = static_cast<float>(picks > 0.0 ? x.E * term / (picks * n) : 0.0);
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
    __shared__ unsigned long long total_picks;   // (up to 16 (2^31 - 1))
    __shared__ __attribute__((aligned(16))) float shares_[kThreads * kRouteValues];
    SWIGLU_LDS float *shares = (SWIGLU_LDS float *)shares_;
    const int tid = threadIdx.x, li = tid % LPR, group = tid / LPR;
    const int e0 = li * kRouteValues;
    if (tid == 0) total_picks = 0u;
    __syncthreads();
    unsigned long long picks = 0u;
    for (int e = tid; e < x.E; e += kThreads) picks += x.counts[e];
    if (picks) atomicAdd(&total_picks, picks);
    __syncthreads();
    const float n = static_cast<float>(max(x.counts[x.E], 1));
    const float d_loss = x.d_loss ? *x.d_loss : 0.0f;
    const float each = d_loss * x.E / (static_cast<float>(max(total_picks, 1ull)) * n);
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
        // pick j = h LPR + li of the row
        int id[kHeld];
        float w[kHeld], dw[kHeld];
        float wdw = 0.0f;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            const int j = h * LPR + li;
            const bool held = j < x.k;
            id[h] = held ? x.ids[at * x.k + j] : -1;
            if (id[h] >= x.E) id[h] = -1;   // (the caller's: not to write past the row)
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
        // each pick's share, at its expert: through the row's own LDS (a wave's LDS
        // accesses are in order, and its rows are its own)
        SWIGLU_LDS float *row_shares = shares + (group * LPR + li) * kRouteValues;
        *reinterpret_cast<SWIGLU_LDS f32x4 *>(row_shares) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        *reinterpret_cast<SWIGLU_LDS f32x4 *>(row_shares + 4) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (id[h] >= 0) shares[group * LPR * kRouteValues + id[h]] = dw[h];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float share[kRouteValues];
#pragma unroll
        for (int i = 0; i < kRouteValues; ++i) share[i] = row_shares[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
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

// Threads of the forward kernel, and its workgroups: one per pass of rows, at
// most one a compute unit.
static int route_threads(int64_t M, int64_t E) { return M * lanes_per_row(E) <= 256 ? 256 : 1024; }
static int route_grid(int64_t M, int64_t E, int cus) {
    const int64_t per = route_threads(M, E) / lanes_per_row(E);
    const int64_t passes = (M + per - 1) / per;
    if (cus >= 1 << kArrivalBits) cus = (1 << kArrivalBits) - 1;
    return static_cast<int>(passes < cus ? passes : cus);
}

// The partials, and behind them (in a cache line of its own) the word that the
// workgroups arrive at.
static uint64_t partials_words(int grid, int64_t E) {
    return (static_cast<uint64_t>(grid) * (E + 1) + 31) & ~uint64_t{31};
}
uint64_t route_workspace_bytes(int64_t M, int64_t E, int cus) {
    const int grid = route_grid(M, E, cus);
    return grid > 1 ? (partials_words(grid, E) + 1) * sizeof(uint64_t) : 0;
}

template <bool kBf16, int THREADS>
static void run_route(int lpr, int grid, const RouteArgs &a, hipStream_t stream) {
    const dim3 g(grid), t(THREADS);
    switch (lpr) {
        case 4: hipLaunchKernelGGL((route_kernel<kBf16, 4, THREADS>), g, t, 0, stream, a); break;
        case 8: hipLaunchKernelGGL((route_kernel<kBf16, 8, THREADS>), g, t, 0, stream, a); break;
        case 16: hipLaunchKernelGGL((route_kernel<kBf16, 16, THREADS>), g, t, 0, stream, a); break;
        case 32: hipLaunchKernelGGL((route_kernel<kBf16, 32, THREADS>), g, t, 0, stream, a); break;
        default: hipLaunchKernelGGL((route_kernel<kBf16, 64, THREADS>), g, t, 0, stream, a); break;
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
                        bool normalize, void *workspace, uint64_t workspace_bytes, uint64_t tag,
                        int cus, hipStream_t stream) {
    int grid = route_grid(M, E, cus);
    if (grid > 1 && (workspace == nullptr || workspace_bytes < route_workspace_bytes(M, E, cus)))
        grid = 1;
    if (grid < 1) grid = 1;   // M == 0: the counts and the loss are still written
    uint64_t *const words = static_cast<uint64_t *>(workspace);
    const RouteArgs a{logits, valid, ids, weights, counts, loss, M, E, k, normalize ? 1 : 0,
                      vector_rows(E, logits, nullptr) ? 1 : 0, words,
                      grid > 1 ? words + partials_words(grid, E) : nullptr, tag};
    const int lpr = lanes_per_row(E);
    if (route_threads(M, E) == 256) {
        if (bf16) run_route<true, 256>(lpr, grid, a, stream);
        else run_route<false, 256>(lpr, grid, a, stream);
    } else {
        if (bf16) run_route<true, 1024>(lpr, grid, a, stream);
        else run_route<false, 1024>(lpr, grid, a, stream);
    }
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
