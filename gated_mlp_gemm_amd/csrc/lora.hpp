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

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int kPlanRows = 256;
constexpr int kPlanWhere = 16;                            // byte offsets in a plan
constexpr int kPlanIds = kPlanWhere + 4 * kPlanRows * 4;

// How an expansion walks T: `slots` slots and 8 << shift elements of each part's
// rank at a time, as much as fits its LDS.  (A power of two: with any count the
// quotients by it were a third of the instructions of a step.)
// `plane`: bytes of a plane of T, 64 for each row there is.
struct LoraChunks {
    int slots, shift, plane;
};
struct LoraTerm {
    const uint16_t *T;   // [M][slots][parts * rank / 8][2][8]: rounded, then the rest
    const uint16_t *B;   // [count][cols][rank]
    const char *plans;
    int plan_bytes;
    int M, slots, rank, cols;
    LoraChunks whole, quarter;   // of a tile of the kernel's shape, and of a quarter tile
};

// Quotients by a small divisor that is the same for all lanes, by its
// reciprocal: exact while e < 2^20, the quotient is below 2^12 and the divisor
// at most 512 (e + 1/2 is at least 1/2 from the next multiple of d, 2^-10 of a
// quotient, and the roundings move a quotient below 2^12 by less than 2^-10:
// three of them, each 2^-24 of it).
struct Divisor {
    int d;
    float inverse;
    __device__ __forceinline__ explicit Divisor(int by)
        : d(by), inverse(1.0f / static_cast<float>(by)) {}
    __device__ __forceinline__ int quotient(int e) const {
        return static_cast<int>((static_cast<float>(e) + 0.5f) * inverse);
    }
};

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

// LDS accesses that the compiler does not see (as asm_read_b128): it would
// wait for every direct-to-LDS load in flight first.  wait_lgkmcnt0() and an
// empty "+v" statement stand before the use of what is read.
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
__device__ __forceinline__ void asm_write_b128(uint32_t addr, const u32x4 &v) {
    asm volatile("ds_write_b128 %0, %1" ::"v"(addr), "v"(v) : "memory");
}
__device__ __forceinline__ void asm_write_b32(uint32_t addr, uint32_t v) {
    asm volatile("ds_write_b32 %0, %1" ::"v"(addr), "v"(v) : "memory");
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
// K runs over the adapters of the tile's plan, 1 << shift chunks of 8 elements each,
// 32 k a step.  LDS holds T of the tile's rows (only the slots that there are;
// a lane whose row does not name the adapter of its 8 k reads zeros from beside
// it) and a ring of B's rows, kSteps steps a stage, both loaded straight to
// LDS; so every byte is read once a tile.  Both lie in planes of 64 bytes a
// row, the 16-byte chunks swizzled by the row (16 rows on 16 different banks).
// One wave a SIMD issues an instruction about every 6 clocks, so what bounds
// the steps is the instructions around the MFMAs, not bytes: the addresses and
// LDS reads of a group of row blocks stand between the MFMAs of the group
// before.  256 x 256 tile, Gate and Up, 2 slots of rank 16, in clocks: T's 64
// KiB 3400 (what a compute unit takes in), B and the wait 1600, a step 3300, of
// which the MFMAs are 2048 (4500 with addresses and MFMAs one after the other).
// Loaded by each wave straight into its MFMA operands, T and B took as long as
// that: 16-byte pieces of many cache lines, each row by two waves.  The first
// stages' adapters are looked up before the tile's K steps (begin).
template <class S, bool kGated, bool kQuarter>
struct LoraExpand {
    static_assert(S::MI == 16 && S::kWaves == 4, "16x16 MFMAs, 4 waves");
    static_assert(!kGated || S::TN % 2 == 0, "Gate and Up in blocks of their own");
    static_assert(kPlanRows % S::BM == 0, "a tile's rows in one plan");
    static constexpr int kParts = kGated ? 2 : 1;
    // LDS: where [4][256] | ids | zeros | T ... | ring of B
    static constexpr int kIds = 4 * kPlanRows * 4;
    static constexpr int kZeros = kIds + kPlanRows * kMaxLoraSlots * 2;
    static constexpr int kRowBlocks = S::kWaveM / 16;
    static constexpr int kT = kZeros + kRowBlocks * 1024;   // (a wave's rows, 64 bytes each)
    // a stage of a small tile takes several steps: its barrier and its latency
    // are most of its time
    static constexpr int kSteps = S::BN <= 64 ? 4 : S::BM <= 64 ? 2 : 1;
    static constexpr int kStages = kSteps > 1 ? 3 : S::kLdsBytes > 65536 && S::BN <= 128 ? 4 : 2;
    static constexpr int kStepBytes = S::BN * 64;
    static constexpr int kRing = S::kLdsBytes - kStages * kSteps * kStepBytes;
    static constexpr int kDma = kStepBytes / 4096;   // loads a wave and step
    static constexpr int kEarly = (kStages - 1) * kSteps;
    // A plane of T: 16 elements (4 chunks, rounded and rest) of a slot's part.  In
    // tiles for few rows, of the rows that there are, so that more of the slots and
    // the rank goes at once (M=8 K=928 N=7112, 3 slots of rank 40: 20.7
    // -> 17.3 us).
    static constexpr int kPlane = S::BM * 64;
    static constexpr bool kFewRows = kSteps > 1;
    static_assert((kRing - kT) / kPlane >= kParts, "T fits");
    __device__ __forceinline__ static int plane(const LoraChunks &by) {
        return kFewRows ? by.plane : kPlane;
    }

    static constexpr int planes(int shift) { return shift > 1 ? 1 << (shift - 1) : 1; }   // of a slot's part
    // All slots and the whole rank (rounded up to a power of two) if they fit,
    // else as much of the rank as does, else one plane and as many slots as do.
    // Where requests of their own adapters make many of them (few rows), less of the
    // rank at a time if that leaves out so much padding that it pays for the further
    // passes, each about 3 steps (M=21 K=536 N=1024, 17 adapters of rank 48, two a row:
    // the tile kernel 20.1 us 16 at a time, 21.4 with all 64).
    static LoraChunks chunks(int M, int slots, int rank, int count) {
        const int plane = kFewRows && M < S::BM ? (M + 15) / 16 * 1024 : kPlane;
        const int most = (kRing - kT) / plane / kParts;
        int shift = 0;
        while ((8 << shift) < rank) ++shift;
        while (shift > 1 && planes(shift) * slots > most) --shift;
        if (kFewRows) {
            const int64_t named = static_cast<int64_t>(M) * slots, n = named < count ? named : count;
            auto steps = [&](int by) { return ceil_div(rank, 8 << by) * (ceil_div(n << by, 4) + 3); };
            for (int by = shift - 1; by >= 0; --by)
                if (steps(by) < steps(shift)) shift = by;
        }
        return {slots < most ? slots : most, shift, plane};
    }

    int n;                 // adapters of the plan
    int first, steps;      // the piece's steps of 32 k
    uint32_t id[kEarly];   // the lane's adapter in each of the first steps

    __device__ __forceinline__ static int swizzle(int row) { return ((row >> 1) ^ (row >> 3)) & 3; }
    // the lane's row of B and its 16 bytes of a step
    __device__ __forceinline__ static int b_row(int tid) { return (tid >> 6) * 16 + (tid & 63) / 4; }
    __device__ __forceinline__ static int b_chunk(int tid) { return (tid & 3) ^ swizzle((tid & 63) / 4); }
    // The thread's number, of which the compiler does not know that it is the
    // same for every tile: what follows from it is computed for each, not kept
    // in registers over the K steps.
    __device__ __forceinline__ static int thread() {
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        return tid;
    }

    // Piece `piece` of `pieces` of a tile split along K takes its share of the steps.
    // (All by the last piece: M=525 K=3360 N=3384, 30 adapters of rank 32, 87 against
    // 60 us; M=99 K=4656 N=1256, 23 of rank 40, 26 against 13.5.)
    __device__ __forceinline__ void begin(const LoraTerm &x, int m0, int piece, int pieces) {
        const int tid = thread();
        const char *plan = x.plans + static_cast<int64_t>(m0 / kPlanRows) * x.plan_bytes;
        // (uniform: a scalar load)
        n = *reinterpret_cast<const __attribute__((address_space(4))) int *>(
            reinterpret_cast<uintptr_t>(plan));
        const int shift = kQuarter ? x.quarter.shift : x.whole.shift;
        const int all = ((n << shift) + 3) / 4;
        first = all * piece / pieces;
        steps = all * (piece + 1) / pieces - first;
        const uint16_t *ids = reinterpret_cast<const uint16_t *>(plan + kPlanIds);
#pragma unroll
        for (int s = 0; s < kEarly; ++s)
            id[s] = n > 0 ? ids[min((4 * (first + s) + b_chunk(tid)) >> shift, n - 1)] : 0u;
    }

    // after MFMA i of 4 kRows S::TN: hook(i); with the first row block, zeros times B
    // onto `met`
    template <int kRows, class Hook>
    __device__ __forceinline__ static void multiply(typename S::Acc (&acc)[S::TM][S::TN], f32x4 &met,
                                                    const u32x4 &nothing, int rb0,
                                                    const u32x4 (&tf)[kRows][kParts][2],
                                                    const u32x4 (&bf)[S::TN][2], const Hook &hook) {
        asm volatile("s_nop 1");
#pragma unroll
        for (int rest = 0; rest < 2; ++rest)
#pragma unroll
            for (int t = 0; t < kRows; ++t)
#pragma unroll
                for (int c = 0; c < S::TN; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int rb = rb0 + t;
                        mfma_16x16x32_acc(acc[rb / 2][c].v[2 * (rb % 2) + h],
                                          tf[t][kGated ? c % 2 : 0][rest], bf[c][h]);
                        if (rb == 0 && rest == 0)
                            asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0"
                                         : "+v"(met)
                                         : "v"(nothing), "v"(bf[c][h]));
                        hook(((rest * kRows + t) * S::TN + c) * 2 + h);
                    }
    }

    // Whether the wave's columns met an infinity or NaN in B: then the accumulators are
    // worthless, and the tile is done again with `clean` (which returns false).  That one
    // makes zeros of them in the LDS (each wave of what it loaded) and adds what they are
    // to the rows that name their adapter (add_broken).
    __device__ __forceinline__ bool run(SWIGLU_LDS char *lds, const LoraTerm &x,
                                        typename S::Acc (&acc)[S::TM][S::TN], int m0, int n0,
                                        bool clean) const {
        const int tid = thread(), lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / S::WN, wn = wave % S::WN;
        const int r16 = lane & 15, g = lane >> 4;
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
        const LoraChunks by = kQuarter ? x.quarter : x.whole;
        const int rank8 = x.rank / 8;
        const int slot_bytes = kParts * x.rank * 4, row_bytes = x.slots * slot_bytes;
        const __amdgpu_buffer_rsrc_t pr =
            make_rsrc(x.plans + static_cast<int64_t>(m0 / kPlanRows) * x.plan_bytes,
                      static_cast<uint32_t>(x.plan_bytes));
        const __amdgpu_buffer_rsrc_t tr =
            make_rsrc(x.T + static_cast<int64_t>(m0) * (row_bytes / 2),
                      static_cast<uint32_t>(min(S::BM, x.M - m0) * row_bytes));
        // where of the tile's rows: one of the four planes a wave; ids: 1 KiB a wave
        if (steps > 0) {
            dma16(pr, lds + wave * 1024,
                  static_cast<uint32_t>(kPlanWhere + (m0 % kPlanRows) * 4) + lane * 16u,
                  wave * (kPlanRows * 4));
            dma16(pr, lds + kIds + wave * 1024, kPlanIds + lane * 16u, wave * 1024);
            for (int i = wave; i < kRowBlocks; i += 4)
                asm_write_b128(at + kZeros + i * 1024 + lane * 16u, u32x4{0u, 0u, 0u, 0u});
        }

        uint32_t col[kDma];   // elements from an adapter's B to the lane's rows
#pragma unroll
        for (int j = 0; j < kDma; ++j) {
            const int r = j * 64 + b_row(tid);
            // past the last column any row does, its results are not stored
            col[j] = static_cast<uint32_t>(min(n0 + (kGated ? pair_row(r) : r), x.cols - 1)) * x.rank;
        }
        const int64_t b_adapter = static_cast<int64_t>(x.cols) * x.rank;
        const int planes_part = planes(by.shift), mask = (1 << by.shift) - 1;

        const int row0 = wm * S::kWaveM + r16;   // the lane's row of T in row block 0
        // row blocks whose T is in registers at once, one such group ahead
        constexpr int kRows = kRowBlocks > 2 ? 2 / kParts : kRowBlocks;
        constexpr int kGroups = kRowBlocks / kRows;
        const uint32_t t_row = at + kT + row0 * 64u;
        const int t_plane = plane(by);
        const uint32_t t_part = static_cast<uint32_t>(planes_part * t_plane);
        // (in vector registers: the accumulators may hold all others)
        f32x4 met = {0.0f, 0.0f, 0.0f, 0.0f};
        u32x4 nothing = {0u, 0u, 0u, 0u};
        asm volatile("" : "+v"(nothing), "+v"(met));
        const uint32_t b_read = at + kRing + (wn * S::kWaveN + r16) * 64u + ((g ^ swizzle(r16)) * 16u);

#pragma nounroll
        // (no steps: nothing to expand; one way out, so that the accumulators stay in place)
        for (int j0 = steps > 0 ? 0 : x.slots; j0 < x.slots; j0 += by.slots)
#pragma nounroll
            for (int r0 = 0; r0 < rank8; r0 += mask + 1) {
                // T: a wave a quarter of the rows, 16 rows of a plane a load.  (Past the
                // last slot: past the row, or zeros; never read.)
                {
                    const int row16 = kFewRows ? wave : wave * (S::BM / 64);   // of the first load
                    const uint32_t from =
                        static_cast<uint32_t>((row16 * 16 + lane / 4) * row_bytes) +
                        ((lane & 3) ^ swizzle(lane / 4)) * 16u;
                    SWIGLU_LDS char *to = lds + kT + row16 * 1024;
#pragma nounroll
                    for (int sp = 0; sp < by.slots * kParts; ++sp)
#pragma nounroll
                        for (int i = 0; i < planes_part; ++i) {
                            const uint32_t soff = static_cast<uint32_t>(
                                (j0 * kParts + sp) * x.rank * 4 + r0 * 32 + i * 64);
                            if constexpr (kFewRows) {
                                for (int t = 0; (row16 + t) * 1024 < t_plane; t += 4)
                                    dma16(tr, to + t * 1024, from, soff + t * 16u * row_bytes);
                            } else {
#pragma unroll
                                for (int t = 0; t < S::BM / 64; ++t)
                                    dma16(tr, to + t * 1024, from, soff + t * 16u * row_bytes);
                            }
                            to += t_plane;
                        }
                }
                // step s of B to its stage, from the adapter `of` of the lane
                auto issue_b = [&](int s, uint32_t of) {
                    const int e = 4 * (first + s) + b_chunk(tid);
                    // past the end: something there is, multiplied with zeros
                    const int element = min(r0 + (e & mask), rank8 - 1);
                    const uint16_t *p = x.B + (of * b_adapter + 8 * element);
                    SWIGLU_LDS char *to =
                        lds + kRing + (s % (kStages * kSteps)) * kStepBytes + wave * 1024;
#pragma unroll
                    for (int j = 0; j < kDma; ++j) gdma16(p + col[j], to + j * 4096);
                };
                auto clear_stage = [&](int stage) {   // (what issue_b of this lane brought)
#pragma nounroll
                    for (int i = 0; i < kSteps * kDma; ++i)
                        clear_lds(at + kRing + (stage % kStages) * (kSteps * kStepBytes) +
                                  i / kDma * kStepBytes + i % kDma * 4096 + wave * 1024 + lane * 16u);
                    wait_lgkmcnt0();
                };
                auto next_stage = [&](int stage) {
                    uint32_t of[kSteps];
#pragma unroll
                    for (int q = 0; q < kSteps; ++q)
                        of[q] = asm_read_u16(
                            at + kIds +
                            min((4 * (first + stage * kSteps + q) + b_chunk(tid)) >> by.shift, n - 1) * 2);
#pragma unroll
                    for (int q = 0; q < kSteps; ++q) issue_b(stage * kSteps + q, landed(of[q]));
                };
#pragma unroll
                for (int s = 0; s < kEarly; ++s) issue_b(s, id[s]);
                wait_vmcnt<(kStages - 2) * kSteps * kDma>();
                if (__builtin_expect(clean, 0)) {
                    const int row16 = kFewRows ? wave : wave * (S::BM / 64);
                    uint32_t to = at + kT + row16 * 1024 + lane * 16u;
#pragma nounroll
                    for (int sp = 0; sp < by.slots * kParts * planes_part; ++sp, to += t_plane)
#pragma nounroll
                        for (int t = 0; kFewRows ? (row16 + t) * 1024 < t_plane : t < S::BM / 64;
                             t += kFewRows ? 4 : 1)
                            clear_lds(to + t * 1024);
                    clear_stage(0);
                }
                wait_lgkmcnt0();
                block_barrier();   // the plan, T and stage 0 are there
                next_stage(kStages - 1);

                // the rows' first two slots of the chunk stay in registers
                const int pair0 = j0 / 2, pairs = (min(x.slots, j0 + by.slots) + 1) / 2;
                uint32_t where[kRowBlocks];
#pragma unroll
                for (int t = 0; t < kRowBlocks; ++t)
                    where[t] = asm_read_b32(at + pair0 * (kPlanRows * 4) + (row0 + 16 * t) * 4u);
                wait_lgkmcnt0();
#pragma unroll
                for (int t = 0; t < kRowBlocks; ++t) asm volatile("" : "+v"(where[t]));

                // Where the lane's k of a step is in T, row block 0 and part 0, for the slots
                // of a pair, and what a row's `where` holds if it names that adapter.
                struct Look {
                    uint32_t at[2], key[2];
                };
                auto look_at = [&](int s, int pair) {
                    const int e = 4 * (first + s) + g;
                    const int i = e >> by.shift, k = e & mask;
                    const uint32_t key = r0 + k < rank8 ? i + 1 : 0xFFFFu;   // (no index is that far)
                    Look l;
                    l.key[0] = 2 * pair >= j0 ? key : 0xFFFFu;
                    l.key[1] = 2 * pair + 1 < j0 + by.slots ? key : 0xFFFFu;
                    l.at[0] = t_row + ((2 * pair - j0) * kParts * planes_part + (k >> 1)) * t_plane +
                              ((2 * (k & 1)) ^ swizzle(r16)) * 16u;
                    l.at[1] = l.at[0] + kParts * t_part;
                    return l;
                };
                const uint32_t zeros = at + kZeros;
                auto match = [&](const Look &l, uint32_t w, uint32_t (&from)[kParts]) {
                    const bool lo = (w & 0xFFFFu) == l.key[0], hi = (w >> 16) == l.key[1];
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
                        from[p] = lo ? l.at[0] + p * t_part : hi ? l.at[1] + p * t_part : from[p];
                };
                // T of row block t for the lane's k, all parts, if the row names its adapter,
                // else zeros
                auto read_t = [&](u32x4 (&f)[kParts][2], const Look &l, int s, int t) {
                    uint32_t from[kParts];
#pragma unroll
                    for (int p = 0; p < kParts; ++p) from[p] = zeros;
                    match(l, where[t], from);
                    if (pair0 + 1 < pairs) {
#pragma nounroll
                        for (int pair = pair0 + 1; pair < pairs; ++pair) {
                            uint32_t w = asm_read_b32(at + pair * (kPlanRows * 4) + (row0 + 16 * t) * 4u);
                            w = landed(w);
                            match(look_at(s, pair), w, from);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        f[p][0] = read_one(from[p], t * 1024);
                        f[p][1] = read_one(from[p] ^ 16u, t * 1024);
                    }
                };
                u32x4 bf[2][S::TN][2], tf[2][kRows][kParts][2];
                auto keep = [&](u32x4 (&ft)[kRows][kParts][2], u32x4 (&fb)[S::TN][2]) {
#pragma unroll
                    for (int t = 0; t < kRows; ++t)
#pragma unroll
                        for (int p = 0; p < kParts; ++p)
#pragma unroll
                            for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(ft[t][p][h]));
#pragma unroll
                    for (int c = 0; c < S::TN; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(fb[c][h]));
                };
                auto have = [&](u32x4 (&ft)[kRows][kParts][2], u32x4 (&fb)[S::TN][2]) {
                    asm volatile("s_waitcnt lgkmcnt(0)");
                    keep(ft, fb);
                };
                // step 0
                Look look = look_at(0, pair0);
#pragma unroll
                for (int w = 0; w < 2 * S::TN; ++w) bf[0][w / 2][w % 2] = read_one(b_read, w * 1024);
#pragma unroll
                for (int t = 0; t < kRows; ++t) read_t(tf[0][t], look, 0, t);

                // one step with B in bf[BUF]; the next step's B goes to the other buffer
                auto step = [&](int s, auto buf_) {
                    constexpr int buf = decltype(buf_)::value;
                    constexpr int kMfma = 4 * kRows * S::TN;
                    // T's buffers alternate over the groups of all steps
                    constexpr int first = kGroups % 2 ? buf : 0;
                    uint32_t b_at = b_read;
                    for_each(std::make_integer_sequence<int, kGroups>{}, [&](auto group_) {
                        constexpr int group = decltype(group_)::value;
                        have(tf[(first + group) % 2], bf[buf]);
                        // Registers that reads are in flight to stay theirs until this wait or
                        // the one behind the loop, on every path of the compiled code (also
                        // on those that no number of steps takes: it joins the two exits).
                        if constexpr (group == 0) keep(tf[(first + 1) % 2], bf[buf ^ 1]);
                        constexpr bool next = group + 1 == kGroups;   // the next reads are the next step's
                        if constexpr (next) {
                            if (s + 1 < steps && (s + 1) % kSteps == 0) {
                                // the next stage is there, and everyone has read this one
                                wait_vmcnt<(kStages - 2) * kSteps * kDma>();
                                if (__builtin_expect(clean, 0)) clear_stage((s + 1) / kSteps);
                                block_barrier();
                                next_stage((s + 1) / kSteps + kStages - 1);
                            }
                            b_at += ((s + 1) % (kStages * kSteps)) * kStepBytes;
                            look = look_at(s + 1, pair0);
                        }
                        // between the MFMAs: T of the next group, B of the next step
                        constexpr int kB = 2 * S::TN;
                        constexpr int all = kRows + (next ? kB : 0);
                        multiply<kRows>(acc, met, nothing, group * kRows, tf[(first + group) % 2], bf[buf], [&](int i) {
#pragma unroll
                            for (int w = 0; w < kB + kRows; ++w) {
                                if (w >= all || w * kMfma / all != i) continue;
                                if (next && w < kB)
                                    bf[buf ^ 1][w / 2][w % 2] = read_one(b_at, w * 1024);
                                else if (next)
                                    read_t(tf[(first + group + 1) % 2][w - kB], look, s + 1, w - kB);
                                else
                                    read_t(tf[(first + group + 1) % 2][w], look, s,
                                           (group + 1) * kRows + w);
                            }
                        });
                        __builtin_amdgcn_sched_barrier(0);
                    });
                };
                constexpr std::integral_constant<int, 0> k0{};
                constexpr std::integral_constant<int, 1> k1{};
#pragma nounroll
                for (int s = 0; s < steps; s += 2) {
                    step(s, k0);
                    if (s + 1 < steps) step(s + 1, k1);
                }
                wait_vmcnt<0>();
                // (the reads of the step behind the last)
#pragma unroll
                for (int i = 0; i < 2; ++i) have(tf[i], bf[i]);
                block_barrier();   // T and the ring are free
            }
        wait_mfma_results();
#pragma unroll
        for (int a = 0; a < S::TM; ++a)
#pragma unroll
            for (int c = 0; c < S::TN; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) asm volatile("" : "+a"(acc[a][c].v[q]));
        asm volatile("" : "+v"(met));
        if (__builtin_expect(clean, 0)) {
            if (steps > 0) add_broken(x, acc, m0, n0);
            return false;
        }
        // (all rows of zeros: one tells of its column)
        return __builtin_amdgcn_ballot_w64(met[0] != met[0]) != 0;
    }

    // Whether run() returned true to any wave of the workgroup, for all of them (whose LDS
    // is idle; a barrier has to stand before its next use).
    __device__ __forceinline__ static bool any_wave(SWIGLU_LDS char *lds, bool mine) {
        if constexpr (S::WN == 1) return mine;   // (all have the same columns)
        const int tid = thread();
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
        if ((tid & 63) == 0) asm_write_b32(at + (tid >> 6) * 4u, mine ? 1u : 0u);
        wait_lgkmcnt0();
        block_barrier();
        u32x4 all = read_one(at, 0);
        asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(all));
        return __builtin_amdgcn_readfirstlane(
                   static_cast<int>(all[0] | all[1] | all[2] | all[3])) != 0;
    }

    // Infinities and NaN become zeros; whether there were any.
    __device__ __forceinline__ static bool clear_broken(u32x4 &v) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool lo = (v[i] & 0x7F80u) == 0x7F80u, hi = (v[i] & 0x7F800000u) == 0x7F800000u;
            v[i] &= (lo ? 0xFFFF0000u : ~0u) & (hi ? 0x0000FFFFu : ~0u);
            any = any || lo || hi;
        }
        return any;
    }

    // The same of 16 bytes of LDS.
    __device__ __forceinline__ static void clear_lds(uint32_t addr) {
        u32x4 v = read_one(addr, 0);
        asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(v));
        clear_broken(v);
        asm_write_b128(addr, v);
    }

    // The terms that a clean expansion left out, of the row's own adapters: those with
    // an infinity or NaN in B or in T.  A lane an element, from memory.
    __device__ __forceinline__ void add_broken(const LoraTerm &x, S::Acc (&acc)[S::TM][S::TN], int m0,
                                               int n0) const {
        constexpr int kQuads = S::TM * S::TN * 4;
        static_assert(kRowBlocks <= 8, "a bit a row");
        const int shift = kQuarter ? x.quarter.shift : x.whole.shift, rank8 = x.rank / 8;
        const int tid = thread(), lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / S::WN, wn = wave % S::WN;
        const char *plan = x.plans + static_cast<int64_t>(m0 / kPlanRows) * x.plan_bytes;
        const uint32_t *where = reinterpret_cast<const uint32_t *>(plan + kPlanWhere);
        const uint16_t *ids = reinterpret_cast<const uint16_t *>(plan + kPlanIds);
        const int row0 = m0 + wm * S::kWaveM + (lane >> 4) * 4;   // of row block 0
        auto adapter = [&](int row, int j) {   // 1 + its list index, 0: none
            return static_cast<int>(where[j / 2 * kPlanRows + row % kPlanRows] >> (16 * (j % 2)) & 0xFFFFu);
        };
        auto t_of = [&](int row, int j, int part) {
            return reinterpret_cast<const u32x4 *>(
                x.T + ((static_cast<int64_t>(row) * x.slots + j) * kParts + part) * x.rank * 2);
        };
        auto column = [&](int i) {   // of 16-column block i
            const int pc = wn * S::kWaveN + i * 16 + (lane & 15);
            return n0 + (kGated ? pair_row(pc) : pc);
        };
        auto b_of = [&](int at, int col) {
            return reinterpret_cast<const u32x4 *>(
                x.B + (static_cast<int64_t>(ids[at]) * x.cols + col) * x.rank);
        };
        uint32_t columns = 0u;   // those in which some adapter of the plan has some, a bit each
#pragma nounroll
        for (int i = 0; i < 2 * S::TN; ++i) {
            const int col = column(i);
            bool any = false;
            for (int at = 0; at < n && col < x.cols; ++at)
#pragma unroll 4
                for (int c = 0; c < rank8; ++c) {
                    u32x4 b = b_of(at, col)[c];
                    any |= clear_broken(b);
                }
            columns |= static_cast<uint32_t>(any) << i;
        }
        uint32_t rows = 0u;   // rows whose T has some, bit 4 (row block) + e
#pragma nounroll
        for (int i = 0; i < kRowBlocks * 4; ++i) {
            const int row = row0 + i / 4 * 16 + i % 4;
            bool any = false;
            for (int j = 0; j < x.slots && row < x.M; ++j)
                for (int c = 0; c < kParts * rank8 && adapter(row, j); ++c) {
                    u32x4 t = t_of(row, j, 0)[2 * c];
                    any |= clear_broken(t);
                }
            rows |= static_cast<uint32_t>(any) << i;
        }
#pragma nounroll
        for (int i = 0; i < kQuads; ++i) {
            const int block = i / 4 % S::TN, rb = i / (4 * S::TN) * 2 + (i >> 1 & 1);
            const int at_col = 2 * block + (i & 1), col = column(at_col);
            const uint32_t wanted = columns >> at_col & 1u ? 15u : rows >> (4 * rb) & 15u;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < kQuads; ++q)
                if (q == i) {
                    v = acc[q / (4 * S::TN)][q / 4 % S::TN].v[q % 4];
                    asm volatile("" : "+v"(v));
                }
#pragma nounroll
            for (int e = 0; e < 4; ++e) {
                const int row = row0 + 16 * rb + e;
                float sum = v[0];
                if ((wanted >> e & 1u) && row < x.M && col < x.cols)
                    for (int j = 0; j < x.slots; ++j) {
                        const int at = adapter(row, j) - 1;
                        if (at < 0) continue;
                        const u32x4 *b = b_of(at, col), *t = t_of(row, j, kGated ? block % 2 : 0);
#pragma unroll 4
                        for (int c = 0; c < rank8; ++c) {
                            // (of the piece's own steps)
                            const int step = (at << shift | (c & ((1 << shift) - 1))) / 4 - first;
                            const u32x4 bv = b[c], hi = t[2 * c], lo = t[2 * c + 1];
                            u32x4 b0 = bv, t0 = hi;
                            const bool any = clear_broken(b0) | clear_broken(t0);
                            if (!any || step < 0 || step >= steps) continue;
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                auto value = [&](const u32x4 &v) {
                                    return __builtin_bit_cast(
                                        float, q % 2 ? v[q / 2] & 0xFFFF0000u : v[q / 2] << 16);
                                };
                                if (value(bv) != value(b0) || value(hi) != value(t0))
                                    sum = fmaf(value(hi) + value(lo), value(bv), sum);
                            }
                        }
                    }
                v = f32x4{v[1], v[2], v[3], sum};
            }
#pragma unroll
            for (int q = 0; q < kQuads; ++q)
                if (q == i) {
                    f32x4 &to = acc[q / (4 * S::TN)][q / 4 % S::TN].v[q % 4];
                    to = v;
                    asm volatile("" : "+a"(to));
                }
        }
    }
    template <int... I, class F>
    __device__ __forceinline__ static void for_each(std::integer_sequence<int, I...>, const F &f) {
        (f(std::integral_constant<int, I>{}), ...);
    }
    // (the offset is a constant once everything is unrolled)
    __device__ __forceinline__ static u32x4 read_one(uint32_t from, int offset) {
        u32x4 r;
        asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(r) : "v"(from), "i"(offset));
        return r;
    }
};

}  // namespace swiglu
