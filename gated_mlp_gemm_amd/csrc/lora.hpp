// Low-rank adapters beside a shared projection: the shared device code.
//
// A projection D = X . W^T (W [cols][K]) with a table of low-rank adapters
// (A [count][parts * rank][K], B [count][cols][rank], scale [count]) gives row
// m, whose slots j name adapters id = ids[m][j] with weights w = weights[m][j],
//
//     D[m] = X[m] . W^T + sum_j w scale[id] (X[m] . A[id]^T) . B[id]^T.
//
// parts is 2 for the interleaved Gate and Up projection (even columns take
// the first `rank` rows of A, odd columns the other), 1 for the down
// projection.  Two steps:
//
//   shrink   T[m][j] = w scale[id] X[m] . A[id]^T, fp32 sums, kept as the sum of
//            two bf16 numbers (the value rounded, and what that rounding lost:
//            16 bits of the value together), so that the expansion takes it
//            through bf16 MFMAs.  (One bf16 number made the block's output
//            1.6 times further off than the rounding of its outputs alone.)
//   expand   D[m] += T[m][j] . B[id]^T, in the fp32 accumulators of the shared
//            product, before its epilogue: B once, with each half of T.
//
// Ids outside [0, count) name no adapter.  Where two slots of a row name the
// same adapter, the first one's T holds the sum of both weights, and only the
// first is expanded.
//
// The shrink also leaves a plan for each 64 rows, so that the expansion, which
// runs once a tile, starts from the adapters' list instead of from the ids:
//     int n, 3 unused ints
//     int ids[capacity]           the adapters that the rows name, ascending
//     uint16 slots[capacity][16]  bits 4 t .. 4 t + 3: 1 + the first slot of row
//                                 16 t + r that names the adapter, 0: none
// The four entries past the n-th repeat the first adapter and name no row: the
// expansion takes 32 k at a time, up to four adapters.
#pragma once

#include "device.hpp"
#include "gemm_core.hpp"
#include "launch.hpp"

namespace swiglu {

constexpr int kPlanRows = 64;
struct LoraTerm {
    const uint16_t *T;   // [M][slots][parts * rank / 8][2][8]: rounded, then the rest
    const uint16_t *B;   // [count][cols][rank]
    const char *plans;
    int plan_bytes, capacity;
    int M, slots, rank, cols;
};

// e / d for 0 <= e < 2^20 and 1 <= d <= 64 (the rounded quotient is exact).
__device__ __forceinline__ int small_quotient(int e, int d) {
    return static_cast<int>((static_cast<float>(e) + 0.5f) / static_cast<float>(d));
}

// Elements c .. c + 3 (c a multiple of 4) of a row of T.
__device__ __forceinline__ void store_t(uint16_t *row, int c, const f32x4 &v) {
    const u32x2 top = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    float rest[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = i % 2 ? top[i / 2] & 0xFFFF0000u : top[i / 2] << 16;
        // (infinite once rounded: nothing to add)
        rest[i] = (h & 0x7F800000u) == 0x7F800000u ? 0.0f : v[i] - __builtin_bit_cast(float, h);
    }
    uint16_t *p = row + (c & ~7) * 2 + (c & 7);
    *reinterpret_cast<u32x2 *>(p) = top;
    *reinterpret_cast<u32x2 *>(p + 8) =
        u32x2{pack_bf16x2(rest[0], rest[1]), pack_bf16x2(rest[2], rest[3])};
}

// Expand into the accumulators of one wave of an S tile at (m0, n0) (16x16
// MFMAs; the accumulators are settled before and after).  Every lane loads its
// own MFMA operands, T and B rows in 16-byte chunks, straight from memory: T
// is a few KiB a tile and the B rows of a tile are read by its waves only, so
// neither gains from a trip through LDS.  Of 64 rows (a plan) 32 k of one part
// at a time: 32 MFMAs of a 128 x 128 wave for Gate and Up (64 for one part) on
// 8 chunks of T and 4 (8) of B, and as many of the next in flight meanwhile;
// twice as many did not fit the registers beside the accumulators.  Rows that
// do not name the lane's adapter read zeros (an offset past the resource), so
// they add nothing.
template <class S, bool kGated>
__device__ __forceinline__ void lora_expand(const LoraTerm &x, typename S::Acc (&acc)[S::TM][S::TN],
                                            int m0, int n0) {
    static_assert(S::MI == 16, "16x16 MFMAs");
    static_assert(!kGated || S::TN % 2 == 0, "Gate and Up in blocks of their own");
    constexpr int kParts = kGated ? 2 : 1;
    constexpr int kGroups = S::kWaveM > kPlanRows ? S::kWaveM / kPlanRows : 1;
    constexpr int kRowBlocks = S::kWaveM / kGroups / 16;
    constexpr int kColBlocks = S::TN / kParts;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int r16 = lane & 15, g = lane >> 4;
    const int mw = m0 + wm * S::kWaveM;
    const int first_block = (mw % kPlanRows) / 16;   // of the wave's rows in the plan
    const int rank8 = x.rank / 8;
    const int slot_bytes = kParts * x.rank * 4;
    // B's row (column of D) of the lane in block 0 of part 0 (pair_row() of its
    // LDS row for Gate and Up), and how far the last row is from it: past the
    // last column any row does, its results are not stored
    const int lane_col = n0 + wn * S::kWaveN + (kGated ? 2 * r16 : r16);
    const int last = x.cols - 1 - lane_col;

    u32x4 tf[2][kRowBlocks][2];   // [buffer][row block][rounded, rest]
    u32x4 bf[2][kColBlocks][2];   // [buffer][column block][16-column half]
    auto group = [&](auto group_) {
        constexpr int grp = decltype(group_)::value;
        const int mg = mw + grp * kPlanRows;
        if (mg >= x.M) return;
        const char *plan = x.plans + static_cast<int64_t>(mg / kPlanRows) * x.plan_bytes;
        const int *ids = reinterpret_cast<const int *>(plan) + 4;
        const uint16_t *map = reinterpret_cast<const uint16_t *>(ids + x.capacity);
        // the lane's chunk (8 of the 32 k) of step s
        struct {
            int adapter;
            uint32_t slots;
        } next;
        auto look_up = [&](int s) {
            const int i = small_quotient(4 * s + g, rank8);
            next.adapter = ids[i];
            next.slots = map[i * 16 + r16];
        };
        look_up(0);   // (in place even where the plan is empty; unused then)
        const int n = __builtin_amdgcn_readfirstlane(*reinterpret_cast<const int *>(plan));
        const int steps = (n * rank8 + 3) / 4;
        if (steps == 0) return;
        const __amdgpu_buffer_rsrc_t trs = make_rsrc(
            x.T + static_cast<int64_t>(mg) * x.slots * (2 * kParts * x.rank),
            static_cast<uint32_t>(min(16 * kRowBlocks, x.M - mg) * x.slots * slot_bytes));

        uint32_t toff[kRowBlocks];
        const uint16_t *brow;
        auto addresses = [&](int s) {
            const int e = 4 * s + g;
            const int element = (e - small_quotient(e, rank8) * rank8) * 8;
#pragma unroll
            for (int t = 0; t < kRowBlocks; ++t) {
                const int slot = static_cast<int>((next.slots >> (4 * (first_block + t))) & 15u) - 1;
                toff[t] = slot >= 0 ? static_cast<uint32_t>(((16 * t + r16) * x.slots + slot) *
                                                                slot_bytes +
                                                            element * 4)
                                    : kOutOfRange;
            }
            brow = x.B + (static_cast<int64_t>(next.adapter) * x.cols + lane_col) * x.rank + element;
            if (s + 1 < steps) look_up(s + 1);
        };
        auto load = [&](u32x4 (&ft)[kRowBlocks][2], u32x4 (&fb)[kColBlocks][2], int part) {
            int rank = x.rank;
            asm volatile("" : "+s"(rank));   // (the row distances are not kept in registers)
#pragma unroll
            for (int c = 0; c < kColBlocks; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int d = kGated ? 64 * c + 32 * h + part : 32 * c + 16 * h;
                    fb[c][h] = gload16(brow + min(d, last) * rank);
                }
#pragma unroll
            for (int t = 0; t < kRowBlocks; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    ft[t][h] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   trs, static_cast<int>(toff[t]), part * x.rank * 4 + h * 16, 0));
        };
        auto multiply = [&](u32x4 (&ft)[kRowBlocks][2], u32x4 (&fb)[kColBlocks][2], auto part_) {
            constexpr int part = decltype(part_)::value;
            // the loads have landed (the compiler waits for them before these),
            // and two wait states lie between any copy it makes and an MFMA
#pragma unroll
            for (int t = 0; t < kRowBlocks; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(ft[t][h]));
#pragma unroll
            for (int c = 0; c < kColBlocks; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(fb[c][h]));
            asm volatile("s_nop 1");
#pragma unroll
            for (int rest = 0; rest < 2; ++rest)
#pragma unroll
                for (int i = 0; i < kRowBlocks; ++i)
#pragma unroll
                    for (int c = 0; c < kColBlocks; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int t = grp * kRowBlocks + i;
                            mfma_16x16x32_acc(acc[t / 2][kParts * c + part].v[2 * (t % 2) + h],
                                              ft[i][rest], fb[c][h]);
                        }
            __builtin_amdgcn_sched_barrier(0);
        };
        constexpr std::integral_constant<int, 0> k0{};
        constexpr std::integral_constant<int, kParts - 1> k1{};
        addresses(0);
        load(tf[0], bf[0], 0);
        if constexpr (kGated) {
#pragma nounroll
            for (int s = 0; s < steps; ++s) {
                load(tf[1], bf[1], 1);
                multiply(tf[0], bf[0], k0);
                if (s + 1 < steps) {
                    addresses(s + 1);
                    load(tf[0], bf[0], 0);
                }
                multiply(tf[1], bf[1], k1);
            }
        } else {
#pragma nounroll
            for (int s = 0; s < steps; s += 2) {
                if (s + 1 < steps) {
                    addresses(s + 1);
                    load(tf[1], bf[1], 0);
                }
                multiply(tf[0], bf[0], k0);
                if (s + 1 < steps) {
                    if (s + 2 < steps) {
                        addresses(s + 2);
                        load(tf[0], bf[0], 0);
                    }
                    multiply(tf[1], bf[1], k1);
                }
            }
        }
    };
    group(std::integral_constant<int, 0>{});
    if constexpr (kGroups > 1) group(std::integral_constant<int, 1>{});
    static_assert(kGroups <= 2, "one or two plans a wave");
    wait_mfma_results();
#pragma unroll
    for (int a = 0; a < S::TM; ++a)
#pragma unroll
        for (int c = 0; c < S::TN; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) asm volatile("" : "+a"(acc[a][c].v[q]));
}

}  // namespace swiglu
