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
//   shrink   T[m][j] = bf16(w scale[id] X[m] . A[id]^T), fp32 sums and one
//            rounding.  (T is a projection's operand like X and the output's H:
//            its rounding adds to the output's error what rounding the
//            adapter's share of it to bf16 would.)
//   expand   D[m] += T[m][j] . B[id]^T, in the fp32 accumulators of the shared
//            product, before its epilogue.
//
// Ids outside [0, count) name no adapter.  Where two slots of a row name the
// same adapter, the first one's T holds the sum of both weights, and only the
// first is expanded.
#pragma once

#include "device.hpp"
#include "gemm_core.hpp"
#include "launch.hpp"

namespace swiglu {

struct LoraTerm {
    const uint16_t *T;   // [M][slots][parts * rank]
    const uint16_t *B;   // [count][cols][rank]
    const int *ids;      // [M][slots]
    int M, slots, rank, count, cols;
};

// The adapters that `rows` rows from row m0 on name, as one wave sees them:
// `ids` holds the rows' slots (-1: none) and `list` the different adapters, in
// ascending order.  Built by one wave for itself in its own LDS: a bit per
// adapter, set by the slots, then read back 64 adapters at a time (one ballot
// and one prefix count each, so a table of at most 64 takes one pass).
template <int ROWS>
struct AdapterList {
    static constexpr int kBitsBytes = kMaxLoraCount / 8;
    static constexpr int kIdsBytes = ROWS * kMaxLoraSlots * 4;
    static constexpr int kListBytes = ROWS * kMaxLoraSlots * 2;
    static constexpr int kBytes = kBitsBytes + kIdsBytes + kListBytes;

    SWIGLU_LDS uint32_t *bits;
    SWIGLU_LDS int *ids;         // [row][slot]
    SWIGLU_LDS uint16_t *list;
    int n;                       // uniform

    __device__ __forceinline__ void at(SWIGLU_LDS char *lds) {
        bits = reinterpret_cast<SWIGLU_LDS uint32_t *>(lds);
        ids = reinterpret_cast<SWIGLU_LDS int *>(lds + kBitsBytes);
        list = reinterpret_cast<SWIGLU_LDS uint16_t *>(lds + kBitsBytes + kIdsBytes);
    }
    __device__ __forceinline__ void build(SWIGLU_LDS char *lds, const int *row_ids, int m0, int M,
                                          int slots, int count) {
        at(lds);
        const int lane = threadIdx.x & 63;
        for (int w = lane; w < (count + 31) / 32; w += 64) bits[w] = 0u;
        const int rows = min(ROWS, M - m0);
        const int total = ROWS * slots, valid = max(rows, 0) * slots;
        const int *src = row_ids + static_cast<int64_t>(m0) * slots;
        for (int i = lane; i < total; i += 64) {
            int id = i < valid ? src[i] : -1;
            if (id < 0 || id >= count) id = -1;
            ids[i] = id;
            if (id >= 0) __hip_atomic_fetch_or(bits + (id >> 5), 1u << (id & 31), __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_WAVEFRONT);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        n = 0;
        for (int base = 0; base < count; base += 64) {
            const int a = base + lane;
            const bool named = a < count && ((bits[a >> 5] >> (a & 31)) & 1u);
            const uint64_t all = __ballot(named);
            if (named) list[n + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(all >> 32),
                                                          __builtin_amdgcn_mbcnt_lo(
                                                              static_cast<uint32_t>(all), 0u))] =
                static_cast<uint16_t>(a);
            n += __popcll(all);
        }
        n = __builtin_amdgcn_readfirstlane(n);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // First slot of row `row` that names adapter a, or -1.
    __device__ __forceinline__ int slot_of(int row, int a, int slots) const {
        int found = -1;
        for (int j = slots - 1; j >= 0; --j)
            if (ids[row * slots + j] == a) found = j;
        return found;
    }
};

// Chunk e of the expansion (8 elements of k): adapters in list order, each
// rank / 8 chunks.  A lane's chunk, its adapter (a real one also past the end,
// where `live` is false) and its first element within that adapter's rank.
struct ChunkOf {
    int adapter;
    int element;
    bool live;
};
template <class List>
__device__ __forceinline__ ChunkOf chunk_of(const List &list, int e, int rank8) {
    // e and rank8 are far below 2^20: the rounded quotient is exact
    int idx = static_cast<int>((static_cast<float>(e) + 0.5f) / static_cast<float>(rank8));
    ChunkOf c;
    c.element = (e - idx * rank8) * 8;
    c.live = idx < list.n;
    if (!c.live) {
        idx = 0;
        c.element = 0;
    }
    c.adapter = list.list[idx];
    return c;
}

// Expand into the accumulators of one wave of an S tile at (m0, n0) (16x16
// MFMAs; the accumulators are settled before and after).  Every lane loads its
// own MFMA operands, T and B rows in 16-byte chunks, straight from memory: T
// is a few KiB a tile and the B rows of a tile are read by its waves only, so
// neither gains from a trip through LDS.  Per 32 k of adapters a wave of
// 128 x 128 loads 8 chunks of B and 16 of T (Gate and Up blocks take their own
// T) for 64 MFMAs.  Rows that do not name the lane's adapter read zeros (an
// offset past the resource), so they add nothing.
template <class S, bool kGated>
__device__ __forceinline__ void lora_expand(SWIGLU_LDS char *lds, const LoraTerm &x,
                                            typename S::Acc (&acc)[S::TM][S::TN], int m0, int n0) {
    static_assert(S::MI == 16, "16x16 MFMAs");
    static_assert(!kGated || S::TN % 2 == 0, "Gate and Up in blocks of their own");
    using List = AdapterList<S::kWaveM>;
    static_assert(S::kWaves * List::kBytes <= S::kLdsBytes, "the lists fit the idle rings");
    constexpr int kParts = kGated ? 2 : 1;
    constexpr int kRowBlocks = S::kWaveM / 16;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int r16 = lane & 15, g = lane >> 4;
    const int mw = m0 + wm * S::kWaveM;

    List list;
    list.build(lds + wave * List::kBytes, x.ids, mw, x.M, x.slots, x.count);

    const int rows = max(0, min(S::kWaveM, x.M - mw));
    const int slot_bytes = kParts * x.rank * 2;
    const __amdgpu_buffer_rsrc_t trs =
        make_rsrc(x.T + static_cast<int64_t>(mw) * x.slots * (kParts * x.rank),
                  static_cast<uint32_t>(rows * x.slots * slot_bytes));
    const int rank8 = x.rank / 8;
    const int steps = (list.n * rank8 + 3) / 4;
    const int ncol0 = n0 + wn * S::kWaveN;
#pragma nounroll
    for (int s = 0; s < steps; ++s) {
        const ChunkOf ch = chunk_of(list, 4 * s + g, rank8);
        uint32_t toff[kRowBlocks];
#pragma unroll
        for (int t = 0; t < kRowBlocks; ++t) {
            const int row = 16 * t + r16;
            const int slot = list.slot_of(row, ch.adapter, x.slots);
            toff[t] = ch.live && slot >= 0
                          ? static_cast<uint32_t>((row * x.slots + slot) * slot_bytes + ch.element * 2)
                          : kOutOfRange;
        }
        const uint16_t *brow = x.B + static_cast<int64_t>(ch.adapter) * x.cols * x.rank + ch.element;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            u32x4 tf[kRowBlocks];
#pragma unroll
            for (int t = 0; t < kRowBlocks; ++t)
                tf[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                      trs, static_cast<int>(toff[t]),
                                                      part * x.rank * 2, 0));
            u32x4 bf[S::TN / kParts][2];
#pragma unroll
            for (int c = 0; c < S::TN / kParts; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the row of B (column of D) of block kParts c + part, half h:
                    // pair_row() of its LDS row for Gate and Up
                    const int col = kGated ? 64 * c + 2 * (16 * h + r16) + part
                                           : 32 * c + 16 * h + r16;
                    // past the last column: any row, its results are not stored
                    const int n = min(ncol0 + col, x.cols - 1);
                    bf[c][h] = gload16(brow + static_cast<int64_t>(n) * x.rank);
                }
            // the loads have landed (the compiler waits for them before these),
            // and two wait states lie between any copy it makes and an MFMA
#pragma unroll
            for (int t = 0; t < kRowBlocks; ++t) asm volatile("" : "+v"(tf[t]));
#pragma unroll
            for (int c = 0; c < S::TN / kParts; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(bf[c][h]));
            asm volatile("s_nop 1");
#pragma unroll
            for (int t = 0; t < kRowBlocks; ++t)
#pragma unroll
                for (int c = 0; c < S::TN / kParts; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mfma_16x16x32_acc(acc[t / 2][kParts * c + part].v[2 * (t % 2) + h], tf[t],
                                          bf[c][h]);
        }
    }
    wait_mfma_results();
#pragma unroll
    for (int a = 0; a < S::TM; ++a)
#pragma unroll
        for (int c = 0; c < S::TN; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) asm volatile("" : "+a"(acc[a][c].v[q]));
    // the lists' LDS is free for the next tile's loads
    block_barrier();
}

}  // namespace swiglu
