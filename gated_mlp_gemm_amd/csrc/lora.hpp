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
// The shrink also leaves a plan for each 256 rows, so that the expansion, which
// runs once a tile, starts from the adapters' list instead of from the ids:
//     int n, 3 unused ints
//     uint32 where[4][256]    of row r, slots 2 i (low half) and 2 i + 1: 1 + the
//                             list index of the slot's adapter, 0: none, or one
//                             that an earlier slot of the row names
//     uint16 ids[capacity]    the adapters that the rows name, ascending
#pragma once

#include "device.hpp"
#include "gemm_core.hpp"
#include "launch.hpp"

namespace swiglu {

constexpr int kPlanRows = 256;
constexpr int kPlanWhere = 16;                            // byte offsets in a plan
constexpr int kPlanIds = kPlanWhere + 4 * kPlanRows * 4;

// How an expansion walks T: `slots` slots and 8 rank8 elements of each part's
// rank at a time, as much as fits its LDS.
struct LoraChunks {
    int slots, rank8;
};
struct LoraTerm {
    const uint16_t *T;   // [M][slots][parts * rank / 8][2][8]: rounded, then the rest
    const uint16_t *B;   // [count][cols][rank]
    const char *plans;
    int plan_bytes;
    int M, slots, rank, cols;
    LoraChunks whole, quarter;   // of a tile of the kernel's shape, and of a quarter tile
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

// LDS reads that the compiler does not see (as asm_read_b128): it would wait
// for every direct-to-LDS load in flight first.  wait_lgkmcnt0() and an empty
// "+v" statement stand before the use.
__device__ __forceinline__ uint32_t asm_read_b32(uint32_t addr) {
    uint32_t r;
    asm volatile("ds_read_b32 %0, %1" : "=v"(r) : "v"(addr));
    return r;
}
__device__ __forceinline__ uint32_t asm_read_u16(uint32_t addr) {
    uint32_t r;
    asm volatile("ds_read_u16 %0, %1" : "=v"(r) : "v"(addr));
    return r;
}
__device__ __forceinline__ uint32_t landed(uint32_t v) {
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(v));
    return v;
}
// 16 bytes a lane from any address to LDS (buffer loads reach 4 GiB).
__device__ __forceinline__ void gdma16(const uint16_t *p, SWIGLU_LDS char *lds) {
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void *)p, (SWIGLU_LDS void *)lds, 16, 0, 0);
}

// Expand into the accumulators of an S tile at (m0, n0) (16x16 MFMAs; the
// accumulators are settled before and after, the tile's LDS is idle).
//
// K runs over the adapters of the tile's plan, rank8 chunks of 8 elements each,
// 32 k a step.  LDS holds T of the tile's rows as it is in memory (only the
// slots that there are; a lane whose row does not name the adapter of its 8 k
// reads zeros from beside it) and a ring of B's rows of one step, both by
// direct-to-LDS loads, so that every byte is read once a tile and by the
// waves from LDS: loaded by each wave straight into its MFMA operands (T's
// rows by 2 waves, B's by 2, in 16-byte pieces of many cache lines), the
// expansion was bound by the L1 cache at about 2.5 times its MFMAs' time.
template <class S, bool kGated, bool kQuarter>
struct LoraExpand {
    static_assert(S::MI == 16 && S::kWaves == 4, "16x16 MFMAs, 4 waves");
    static_assert(!kGated || S::TN % 2 == 0, "Gate and Up in blocks of their own");
    static_assert(kPlanRows % S::BM == 0, "a tile's rows in one plan");
    static constexpr int kParts = kGated ? 2 : 1;
    // LDS: where [4][256] | ids | zeros | T ... | ring of B
    static constexpr int kIds = 4 * kPlanRows * 4;
    static constexpr int kZeros = kIds + kPlanRows * kMaxLoraSlots * 2;
    static constexpr int kT = kZeros + 64;
    static constexpr int kStageBytes = S::BN * 64;
    static constexpr int kStages = S::BN <= 64 ? 8 : S::kLdsBytes > 65536 && S::BN <= 128 ? 4 : 2;
    static constexpr int kRing = S::kLdsBytes - kStages * kStageBytes;
    static constexpr int kDma = kStageBytes / 4096;   // loads a wave and stage
    // 16-byte chunks of T a row: an odd count, so that 16 rows lie on 16
    // different banks
    static constexpr int kRowChunks = (((kRing - kT) / (16 * S::BM)) - 1) | 1;
    static_assert(kRowChunks * 16 * S::BM <= kRing - kT && kRowChunks >= 2 * kParts + 1, "T fits");

    static LoraChunks chunks(int slots, int rank) {
        const int rank8 = rank / 8, most = (kRowChunks - 1) / (2 * kParts);
        if (slots > most) return {most, 1};
        const int r = most / slots < rank8 ? most / slots : rank8;
        const int n = (rank8 + r - 1) / r;   // as even as they can be
        return {slots, (rank8 + n - 1) / n};
    }

    __device__ __forceinline__ static int swizzle(int row) { return ((row >> 1) ^ (row >> 3)) & 3; }

    __device__ __forceinline__ static void run(SWIGLU_LDS char *lds, const LoraTerm &x,
                                               typename S::Acc (&acc)[S::TM][S::TN], int m0, int n0) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
        const int wm = wave / S::WN, wn = wave % S::WN;
        const int r16 = lane & 15, g = lane >> 4;
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
        const char *plan = x.plans + static_cast<int64_t>(m0 / kPlanRows) * x.plan_bytes;
        // (uniform: a scalar load)
        const int n = *reinterpret_cast<const __attribute__((address_space(4))) int *>(
            reinterpret_cast<uintptr_t>(plan));
        if (n == 0) return;
        const LoraChunks by = kQuarter ? x.quarter : x.whole;
        const int rank8 = x.rank / 8;
        const int slot_bytes = kParts * x.rank * 4;
        const int rows = min(S::BM, x.M - m0);
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(plan, static_cast<uint32_t>(x.plan_bytes));
        const __amdgpu_buffer_rsrc_t tr =
            make_rsrc(x.T + static_cast<int64_t>(m0) * x.slots * (2 * kParts * x.rank),
                      static_cast<uint32_t>(rows * x.slots * slot_bytes));
        // where of the tile's rows: one of the four planes a wave; ids: 1 KiB a wave
        dma16(pr, lds + wave * 1024, static_cast<uint32_t>(kPlanWhere + (m0 % kPlanRows) * 4) + lane * 16u,
              wave * (kPlanRows * 4));
        dma16(pr, lds + kIds + wave * 1024, kPlanIds + lane * 16u, wave * 1024);
        if (threadIdx.x < 16)
            asm volatile("ds_write_b32 %0, %1" ::"v"(at + kZeros + threadIdx.x * 4u), "v"(0u) : "memory");

        // the lane's row and 16 bytes of a step of B
        const int b_row = wave * 16 + lane / 4, b_chunk = (lane & 3) ^ swizzle(lane / 4);
        const int row0 = wm * S::kWaveM + r16;   // the lane's row of T in row block 0
        constexpr int kRowBlocks = S::kWaveM / 16;
        // row blocks whose T is in registers at once, one such group ahead
        constexpr int kRows = kRowBlocks > 4 ? 4 / kParts : kRowBlocks;
        constexpr int kGroups = kRowBlocks / kRows;
        const uint32_t b_read = at + kRing + (wn * S::kWaveN + r16) * 64u + ((g ^ swizzle(r16)) * 16u);

#pragma nounroll
        for (int j0 = 0; j0 < x.slots; j0 += by.slots)
#pragma nounroll
            for (int r0 = 0; r0 < rank8; r0 += by.rank8) {
                const int per_slot = by.rank8 * 2;   // 16-byte chunks of a slot's part
                const int row_chunks = by.slots * kParts * per_slot + 1;
                const int steps = (n * by.rank8 + 3) / 4;
                // T: chunk i of the rows' chunks, in memory's order
                const int total = S::BM * row_chunks;
#pragma nounroll
                for (int i0 = wave * 64; i0 < total; i0 += 256) {
                    const int i = i0 + lane;
                    const int row = small_quotient(i, row_chunks), c = i - row * row_chunks;
                    const int sp = small_quotient(c, per_slot), k = c - sp * per_slot;
                    const int j = j0 + sp / kParts, part = sp % kParts;
                    const bool in = j < x.slots && sp < by.slots * kParts && r0 + k / 2 < rank8;
                    dma16(tr, lds + kT + i0 * 16,
                          in ? static_cast<uint32_t>((row * x.slots + j) * slot_bytes +
                                                     part * x.rank * 4 + r0 * 32 + k * 16)
                             : kOutOfRange,
                          0);
                }
                if (j0 + r0 == 0) {
                    wait_vmcnt<0>();
                    wait_lgkmcnt0();
                    block_barrier();   // the plan has landed
                }
                auto issue_b = [&](int s) {
                    const int e = 4 * s + b_chunk;
                    const int i = small_quotient(e, by.rank8);
                    // past the end: something there is, multiplied with zeros
                    const int element = 8 * min(r0 + e - i * by.rank8, rank8 - 1);
                    const uint32_t id = landed(asm_read_u16(at + kIds + min(i, n - 1) * 2));
                    const uint16_t *p =
                        x.B + static_cast<int64_t>(id) * x.cols * x.rank + element;
#pragma unroll
                    for (int j = 0; j < kDma; ++j) {
                        const int r = j * 64 + b_row;
                        const int col = min(n0 + (kGated ? pair_row(r) : r), x.cols - 1);
                        gdma16(p + col * x.rank,
                               lds + kRing + (s % kStages) * kStageBytes + (j * 4 + wave) * 1024);
                    }
                };
#pragma unroll
                for (int s = 0; s < kStages - 1; ++s) issue_b(s);
#pragma nounroll
                for (int s = 0; s < steps; ++s) {
                    wait_vmcnt<(kStages - 2) * kDma>();
                    block_barrier();   // T and step s are there, and step s - 1 is read
                    issue_b(s + kStages - 1);
                    const int e = 4 * s + g;
                    const int i = small_quotient(e, by.rank8), k = e - i * by.rank8;
                    // the slots of the lane's rows that name the adapter of its k
                    int slot[kRowBlocks];
#pragma unroll
                    for (int t = 0; t < kRowBlocks; ++t) slot[t] = -1;
#pragma nounroll
                    for (int j = j0 / 2; 2 * j < min(x.slots, j0 + by.slots); ++j) {
                        uint32_t w[kRowBlocks];
#pragma unroll
                        for (int t = 0; t < kRowBlocks; ++t)
                            w[t] = asm_read_b32(at + j * (kPlanRows * 4) + (row0 + 16 * t) * 4u);
                        wait_lgkmcnt0();
#pragma unroll
                        for (int t = 0; t < kRowBlocks; ++t) {
                            asm volatile("" : "+v"(w[t]));
                            if (static_cast<int>(w[t] >> 16) == i + 1) slot[t] = 2 * j + 1;
                            if (static_cast<int>(w[t] & 0xFFFFu) == i + 1) slot[t] = 2 * j;
                        }
                    }
                    uint32_t t_read[kRowBlocks];   // of part 0; 0: the zeros
#pragma unroll
                    for (int t = 0; t < kRowBlocks; ++t) {
                        const int j = slot[t] - j0;
                        t_read[t] = j >= 0 && j < by.slots && r0 + k < rank8
                                        ? at + kT + ((row0 + 16 * t) * row_chunks +
                                                     j * kParts * per_slot + 2 * k) * 16u
                                        : 0u;
                    }
                    const uint32_t b_at = b_read + (s % kStages) * kStageBytes;
                    u32x4 bf[S::TN][2], tf[2][kRows][kParts][2];
                    auto read_t = [&](int group) {
#pragma unroll
                        for (int t = 0; t < kRows; ++t)
#pragma unroll
                            for (int p = 0; p < kParts; ++p) {
                                const uint32_t a = t_read[group * kRows + t];
                                const uint32_t from = a ? a + p * per_slot * 16u : at + kZeros;
                                tf[group % 2][t][p][0] = asm_read_b128<0>(from);
                                tf[group % 2][t][p][1] = asm_read_b128<16>(from);
                            }
                    };
                    auto have_t = [&](int group) {
                        asm volatile("s_waitcnt lgkmcnt(0)");
#pragma unroll
                        for (int t = 0; t < kRows; ++t)
#pragma unroll
                            for (int p = 0; p < kParts; ++p)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    asm volatile("" : "+v"(tf[group % 2][t][p][h]));
                    };
                    read_b<0>(b_at, bf);
                    read_t(0);
#pragma unroll
                    for (int group = 0; group < kGroups; ++group) {
                        have_t(group);
                        if (group == 0)
#pragma unroll
                            for (int c = 0; c < S::TN; ++c)
#pragma unroll
                                for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(bf[c][h]));
                        if (group + 1 < kGroups) read_t(group + 1);
                        asm volatile("s_nop 1");
#pragma unroll
                        for (int rest = 0; rest < 2; ++rest)
#pragma unroll
                            for (int t = 0; t < kRows; ++t)
#pragma unroll
                                for (int c = 0; c < S::TN; ++c)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        const int rb = group * kRows + t;
                                        mfma_16x16x32_acc(acc[rb / 2][c].v[2 * (rb % 2) + h],
                                                          tf[group % 2][t][kGated ? c % 2 : 0][rest],
                                                          bf[c][h]);
                                    }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                wait_vmcnt<0>();
                block_barrier();   // T and the ring are free
            }
        wait_mfma_results();
#pragma unroll
        for (int a = 0; a < S::TM; ++a)
#pragma unroll
            for (int c = 0; c < S::TN; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) asm volatile("" : "+a"(acc[a][c].v[q]));
    }
    template <int I>
    __device__ __forceinline__ static void read_b(uint32_t from, u32x4 (&bf)[S::TN][2]) {
        if constexpr (I < 2 * S::TN) {
            bf[I / 2][I % 2] = asm_read_b128<(I / 2) * 2048 + (I % 2) * 1024>(from);
            read_b<I + 1>(from, bf);
        }
    }
};

}  // namespace swiglu
