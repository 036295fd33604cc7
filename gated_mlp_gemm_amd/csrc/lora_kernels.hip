// The shrink of the low-rank adapters, T = weight scale X . A^T, and the plans
// of the expansion.  lora.hpp has the mathematics and the layouts.
#include "launch.hpp"

#include "lora.hpp"
#include "split_tail.hpp"

namespace swiglu {

constexpr int kShrinkRows = 64;

// The adapters that 64 rows from row m0 on name: their slots' ids (-1: none)
// and weights, and the list of the different adapters, ascending.  Built by one
// wave: a bit per adapter, set by the slots, then read back 64 adapters at a
// time (one ballot and one prefix count each, so a table of at most 64 takes
// one pass).
struct AdapterList {
    uint32_t bits[kMaxLoraCount / 32];
    int ids[kMaxLoraSlots][kShrinkRows];
    float weights[kMaxLoraSlots][kShrinkRows];
    uint16_t list[kShrinkRows * kMaxLoraSlots];
    int n;
};
__device__ __forceinline__ void build_list(SWIGLU_LDS AdapterList &l, const int *row_ids,
                                           const float *row_weights, int m0, int M, int slots,
                                           int count) {
    const int lane = threadIdx.x & 63;
    for (int w = lane; w < (count + 31) / 32; w += 64) l.bits[w] = 0u;
    const bool here = m0 + lane < M;
    const int64_t at = static_cast<int64_t>(m0 + lane) * slots;
    int id[kMaxLoraSlots];
    float weight[kMaxLoraSlots];
#pragma unroll
    for (int j = 0; j < kMaxLoraSlots; ++j) {
        id[j] = here && j < slots ? row_ids[at + j] : -1;
        weight[j] = here && j < slots && row_weights ? row_weights[at + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < kMaxLoraSlots; ++j) {
        if (j >= slots) continue;
        const bool named = id[j] >= 0 && id[j] < count;
        l.ids[j][lane] = named ? id[j] : -1;
        l.weights[j][lane] = weight[j];
        if (named)
            __hip_atomic_fetch_or(&l.bits[id[j] >> 5], 1u << (id[j] & 31), __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_WAVEFRONT);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    int n = 0;
    for (int base = 0; base < count; base += 64) {
        const int a = base + lane;
        const bool named = a < count && ((l.bits[a >> 5] >> (a & 31)) & 1u);
        const uint64_t all = __ballot(named);
        if (named)
            l.list[n + __builtin_amdgcn_mbcnt_hi(
                           static_cast<uint32_t>(all >> 32),
                           __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(all), 0u))] =
                static_cast<uint16_t>(a);
        n += __popcll(all);
    }
    if (lane == 0) l.n = n;
}

struct ShrinkArgs {
    const uint16_t *X, *A;
    const float *scale, *weights;
    const int *ids;
    uint16_t *T;
    char *plans;
    int plan_bytes, plan_wgs;   // the last workgroups of the grid write the plans
    int M, K, slots, cols, count;   // cols = parts * rank
    float *partials;
    uint64_t *arrivals, tag;   // a word an item of a row block (arrivals.hpp)
    int most_splits, per_rows;   // workgroups a row block
};

// The plan of 256 rows (lora.hpp), a row a thread: a bit per adapter, set by
// the slots; an adapter's list index is the number of bits below its own.
struct PlanLists {
    uint32_t bits[kMaxLoraCount / 32];
    uint16_t before[kMaxLoraCount / 32];   // bits of the words below
    uint16_t wave_bits[4];
};
static_assert(kMaxLoraCount / 32 == kPlanRows, "a word of bits and a row a thread");
__device__ __forceinline__ void write_plan(const ShrinkArgs &x, PlanLists &l, int block) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = static_cast<int64_t>(block) * kPlanRows + tid;
    int id[kMaxLoraSlots];
#pragma unroll
    for (int j = 0; j < kMaxLoraSlots; ++j) {
        id[j] = j < x.slots && row < x.M ? x.ids[row * x.slots + j] : -1;
        if (id[j] < 0 || id[j] >= x.count) id[j] = -1;
    }
    l.bits[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxLoraSlots; ++j)
        if (id[j] >= 0) atomicOr(&l.bits[id[j] >> 5], 1u << (id[j] & 31));
    __syncthreads();
    uint32_t mine = l.bits[tid];
    int upto = __popc(mine);   // over the lanes up to this one, then the waves
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int below = __shfl_up(upto, d);
        if (lane >= d) upto += below;
    }
    if (lane == 63) l.wave_bits[wave] = static_cast<uint16_t>(upto);
    __syncthreads();
    int before = upto - __popc(mine), n = 0;
    for (int w = 0; w < 4; ++w) {
        if (w < wave) before += l.wave_bits[w];
        n += l.wave_bits[w];
    }
    l.before[tid] = static_cast<uint16_t>(before);
    __syncthreads();

    char *plan = x.plans + static_cast<int64_t>(block) * x.plan_bytes;
    if (tid == 0) *reinterpret_cast<int *>(plan) = n;
    uint16_t *ids = reinterpret_cast<uint16_t *>(plan + kPlanIds);
    for (; mine; mine &= mine - 1) ids[before++] = static_cast<uint16_t>(32 * tid + __ffs(mine) - 1);
    uint32_t *where = reinterpret_cast<uint32_t *>(plan + kPlanWhere);
#pragma unroll
    for (int i = 0; i < kMaxLoraSlots / 2; ++i) {
        uint32_t word = 0u;
#pragma unroll
        for (int j = 2 * i; j < 2 * i + 2; ++j) {
            bool first = id[j] >= 0;
#pragma unroll
            for (int e = 0; e < j; ++e) first = first && id[e] != id[j];
            if (first)
                word |= static_cast<uint32_t>(1 + l.before[id[j] >> 5] +
                                              __popc(l.bits[id[j] >> 5] & ((1u << (id[j] & 31)) - 1u)))
                        << (16 * (j & 1));
        }
        where[i * kPlanRows + tid] = word;
    }
}

// Shrink.  A workgroup takes 64 rows of X and lists the adapters that they
// name; the rows of A of those, one after the other, make the columns of
// T^T = A . X^T in items of 64, shared out over per_rows workgroups, which
// split K where there are fewer items than workgroups (their sums meet in the
// workspace as in split_tail.hpp: device-scope stores and arrivals, the last to
// arrive adds them up in order, nobody waits).  Every row of X is
// multiplied with every adapter listed: T takes the ones that it names (the
// products that no row takes cost nothing beside the loads).  Both operands
// stream through LDS (the pipeline of gemm_core.hpp); loaded straight into MFMA
// registers, 64 bytes of a row an instruction, they streamed at half the rate.
//
// What bounds it: where rows are many, the bytes of X and A (M=8192 K=13824,
// one adapter of rank 64: 57 us, X at 4.0 TB/s).  Where they are few, what one
// compute unit takes in, about 26 bytes a clock, and a chain of dependent
// accesses; M=33 K=8960, 16 adapters of rank 8, in clocks: the list 2100, the
// first loads 4700, nine K steps 6100, the store and the arrival 2400, the 15
// others' sums 7900, T 1200 (11.6 us with the launch).  Eight stages instead of
// four, or half the splits, moved that by less than 5 %.
// Four stages, two workgroups a compute unit: one lists its adapters or meets
// the others while the other streams.
using ShapeShrink = TileShape<64, 64, 64, 2, 2, 4, 2, 4, 16>;

// Panel A of the pipeline: 64 of the listed adapters' rows, 8 of which, always
// of one adapter, are one load of one wave.
struct AdapterPanel {
    using S = ShapeShrink;
    static_assert(S::kChunksPerRow == 8, "a wave loads 8 rows");
    __amdgpu_buffer_rsrc_t rsrc[S::kDmaA];
    uint32_t voff;
    int klim, lds_base, last;

    __device__ __forceinline__ void init(const ShrinkArgs &x, const SWIGLU_LDS AdapterList &l,
                                         const Divisor &cols, int first, int total) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
        const int c = (lane % 8) ^ swz<S>(wave * 8 + lane / 8);
        voff = static_cast<uint32_t>(lane / 8) * static_cast<uint32_t>(x.K) * 2u + c * 16u;
        klim = x.K - c * 8;
        last = x.K - S::BK;
        lds_base = wave * 1024;
#pragma unroll
        for (int j = 0; j < S::kDmaA; ++j) {
            const int at = first + 32 * j + 8 * wave;
            const bool in = at < total;
            const int i = in ? cols.quotient(at) : 0, row = in ? at - i * x.cols : 0;
            const int id = __builtin_amdgcn_readfirstlane(static_cast<int>(l.list[i]));
            rsrc[j] = make_rsrc(x.A + (static_cast<int64_t>(id) * x.cols + row) * x.K,
                                in ? 8u * static_cast<uint32_t>(x.K) * 2u : 0u);
        }
    }
    // kEven: K is a multiple of BK (a step past the end loads the last again)
    template <bool kEven>
    __device__ __forceinline__ void issue(int k0, SWIGLU_LDS char *dst, int only) const {
        if constexpr (kEven) k0 = min(k0, last);
        const uint32_t v = kEven || k0 < klim ? voff : kOutOfRange;
#pragma unroll
        for (int j = 0; j < S::kDmaA; ++j)
            if (only < 0 || only == j)
                dma16(rsrc[j], dst + lds_base + j * 4096, v, static_cast<uint32_t>(k0) * 2u);
    }
};

template <bool kEven>
__device__ __forceinline__ void shrink_body(const ShrinkArgs &x, char *smem,
                                            SWIGLU_LDS AdapterList &list, SWIGLU_LDS unsigned &word) {
    using S = ShapeShrink;
    SWIGLU_LDS char *lds = (SWIGLU_LDS char *)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;
    // neighbouring row blocks, which often name the same adapters, on one XCD
    const int G = x.per_rows;
    const int at_ = xcd_order(blockIdx.x, gridDim.x - x.plan_wgs);
    const int rows_at = at_ / G, y = at_ % G;
    const int m0 = rows_at * kShrinkRows;

    if (wave == 0) build_list(list, x.ids, x.weights, m0, x.M, x.slots, x.count);
    __syncthreads();
    const int n = __builtin_amdgcn_readfirstlane(list.n);
    const int total = n * x.cols;
    const Divisor cols(x.cols);
    const int items = (total + S::BM - 1) / S::BM;
    if (items == 0) return;
    const int splits = max(1, min(G / items, x.most_splits));
    const int nk = (x.K + S::BK - 1) / S::BK;

    PanelLoader<S, S::BN, S::kDmaB> xp;
    xp.init(KMajor{x.X, x.M, 1, 0, 0, 0}, m0, x.K);
    for (int job = y; job < items * splits; job += G) {
        const int item = job / splits, split = job % splits;
        const int kb = piece_begin(split, nk, splits), len = piece_begin(split + 1, nk, splits) - kb;
        AdapterPanel ap;
        ap.init(x, list, cols, item * S::BM, total);
        Pipeline<S> pl;
        pl.init(lds);
        // steps past the range load nothing (K step nk is past the end of K)
        auto issue = [&](int s, int part, SWIGLU_LDS char *dst, int j) {
            const int k0 = (s < len ? kb + s : nk) * S::BK;
            if (part == 0) ap.issue<kEven>(k0, dst, j);
            else xp.issue<kEven>(k0, dst, j);
        };
        pl.prologue_issue(issue);
        // quad q of a lane: rows f .. f + 3 of the item's (8 of them are always of
        // one adapter), and one row of X
        int slot[4], c[4];
        float weight[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int f = item * S::BM + 32 * wm + 16 * (q / 2) + 4 * (lane >> 4);
            const int row = 32 * wn + 16 * (q % 2) + (lane & 15);
            const int i = f < total ? cols.quotient(f) : 0;
            const int id = f < total ? list.list[i] : -2;
            c[q] = f - i * x.cols;
            // the weights of every slot that names id, the first one's T holding the sum
            slot[q] = -1;
            weight[q] = 0.0f;
            for (int j = x.slots - 1; j >= 0; --j)
                if (list.ids[j][row] == id) {
                    slot[q] = j;
                    weight[q] += list.weights[j][row];
                }
            weight[q] *= x.scale[max(id, 0)];
        }
        // (two workgroups an item at least: G / 2 items)
        uint64_t *arrivals = x.arrivals + static_cast<int64_t>(rows_at) * (G / 2) + item;
        Arrival meeting{};
        S::Acc acc[S::TM][S::TN];
        pl.prologue_wait();
        if (splits > 1 && tid == 0) meeting.announce(arrivals, x.tag);
        pl.run_init0<kEven>(issue, len, len, acc);
        pl.drain(acc);

        f32x4 sum[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[q][i] = read_acc(acc[0][0].v[q][i]);
        if (splits > 1) {
            if (tid == 0) meeting.settle(arrivals, x.tag);
            constexpr uint32_t kSlot = 4 * S::kThreads * 16;
            const __amdgpu_buffer_rsrc_t pr = make_rsrc(
                x.partials + (static_cast<int64_t>(rows_at) * G + item * splits) * (kSlot / 4),
                splits * kSlot);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                __builtin_amdgcn_raw_buffer_store_b128(
                    __builtin_bit_cast(u32x4, sum[q]), pr,
                    static_cast<int>(split * kSlot + (q * S::kThreads + tid) * 16), 0, kDeviceScope);
            wait_vmcnt<0>();   // this wave's sums are visible device-wide
            __syncthreads();   // ... and every wave's
            if (tid == 0) word = arrive(arrivals);
            __syncthreads();
            // (a workgroup has one job where K is split)
            if (word + 1 != static_cast<unsigned>(splits)) return;
            if (tid == 0) arrivals_done(arrivals);
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (int p = 0; p < splits; ++p)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sum[q] += __builtin_bit_cast(
                        f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   pr, static_cast<int>(p * kSlot + (q * S::kThreads + tid) * 16), 0,
                                   kDeviceScope));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t row = m0 + 32 * wn + 16 * (q % 2) + (lane & 15);
            if (slot[q] >= 0)
                store_t(x.T + (row * x.slots + slot[q]) * (2 * x.cols), c[q], sum[q] * weight[q]);
        }
        __syncthreads();   // the ring and `word` are free
    }
}

__global__ __launch_bounds__(ShapeShrink::kThreads, 2) void lora_shrink_kernel(ShrinkArgs x) {
    __shared__ __attribute__((aligned(16))) char smem[ShapeShrink::kLdsBytes];
    __shared__ AdapterList list;
    __shared__ unsigned word;
    SWIGLU_LDS AdapterList &l = *(SWIGLU_LDS AdapterList *)&list;
    SWIGLU_LDS unsigned &w = *(SWIGLU_LDS unsigned *)&word;
    const int workers = gridDim.x - x.plan_wgs;
    if (static_cast<int>(blockIdx.x) >= workers)
        write_plan(x, *reinterpret_cast<PlanLists *>(smem), blockIdx.x - workers);
    else if (x.K % ShapeShrink::BK == 0) shrink_body<true>(x, smem, l, w);
    else shrink_body<false>(x, smem, l, w);
}

int lora_plan_bytes(int count, int slots) {
    const int named = kPlanRows * slots;
    return kPlanIds + ((count < named ? count : named) + 7) / 8 * 16;
}

hipError_t launch_lora_shrink(const uint16_t *X, const LoraTable &t, const int *ids,
                              const float *weights, int slots, uint16_t *T, char *plans, int M,
                              int K, int parts, const GemmWorkspace &ws, hipStream_t stream) {
    using S = ShapeShrink;
    const int cols = parts * t.rank;
    const int64_t tiles = ceil_div(M, kShrinkRows);
    const int64_t named = static_cast<int64_t>(kShrinkRows) * slots;
    const int64_t items = ceil_div((t.count < named ? t.count : named) * cols, S::BM);
    // a split keeps at least six K steps (meeting costs as much as ten), and the
    // last to arrive has its reads of the others' sums in flight in two goes
    const int64_t nk = ceil_div(K, S::BK);
    int64_t most = nk <= 16 ? 1 : nk / 6;
    if (most > 16) most = 16;
    if (most < 1) most = 1;
    // workgroups a row block: two a compute unit in all (four where that leaves
    // them 24 K steps and more: row blocks that name one adapter more than
    // others would else end last), and no more than there can be work for
    int64_t G = 2 * ws.cus / tiles;
    if (2 * G * 24 <= nk) G = 4 * ws.cus / tiles;
    if (G > items * most) G = items * most;
    if (G < 1) G = 1;
    const uint64_t partials = static_cast<uint64_t>(tiles) * G * (S::BM * S::BN * 4);
    const uint64_t words = static_cast<uint64_t>(tiles) * (G / 2);
    if (ws.base == nullptr || partials + words * sizeof(uint64_t) > ws.bytes) most = 1;
    const int64_t plan_wgs = ceil_div(M, kPlanRows);
    const ShrinkArgs a{X, t.A, t.scale, weights, ids, T, plans, lora_plan_bytes(t.count, slots),
                       static_cast<int>(plan_wgs), M, K, slots, cols, t.count, static_cast<float *>(ws.base),
                       reinterpret_cast<uint64_t *>(static_cast<char *>(ws.base) + partials), ws.tag,
                       static_cast<int>(most), static_cast<int>(G)};
    hipLaunchKernelGGL(lora_shrink_kernel, dim3((unsigned)(tiles * G + plan_wgs)), dim3(S::kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace swiglu
