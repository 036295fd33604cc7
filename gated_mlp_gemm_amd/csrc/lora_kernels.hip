// The low-rank adapter kernels outside the tile kernels: the shrink
// T = weight scale X . A^T, and the projections of at most 128 rows, which
// stream the weight through registers.  lora.hpp has the mathematics.
#include "launch.hpp"

#include "lora.hpp"
#include "split_tail.hpp"

#include <cstdio>

namespace swiglu {

static inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 16x16x32 MFMA through the builtin: the accumulators of these kernels are
// few and short-lived enough for the compiler to place them.
__device__ __forceinline__ f32x4 mfma_16x16x32(const u32x4 &a, const u32x4 &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u32x4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                         r, static_cast<int>(voff), static_cast<int>(soff), 0));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint16_t *base, int64_t row,
                                                            int rows, int K) {
    return make_rsrc(base + row * K, static_cast<uint32_t>(rows) * static_cast<uint32_t>(K) * 2u);
}

// ---------------------------------------------------------------------------
// Shrink.  One workgroup takes 32 rows of X, one of the adapters that they
// name at a time, and 64 of that adapter's rows; its waves split K, and their
// partial sums meet in LDS in wave order.  The adapter's rows are the MFMA's
// first operand, so that a lane ends with four neighbouring elements of T.
// Every operand goes from memory to registers, 16 bytes a lane.
// ---------------------------------------------------------------------------
struct ShrinkArgs {
    const uint16_t *X, *A;
    const float *scale, *weights;
    const int *ids;
    uint16_t *T;
    int M, K, slots, rank, parts, count;
};
constexpr int kShrinkRows = 32;
constexpr int kShrinkCols = 64;
constexpr int kShrinkWaves = 8;

__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(ShrinkArgs x) {
    constexpr int kCB = kShrinkCols / 16, kMB = kShrinkRows / 16;
    using List = AdapterList<kShrinkRows>;
    __shared__ __attribute__((aligned(16))) char list_lds[List::kBytes];
    __shared__ __attribute__((aligned(16))) f32x4 part[kShrinkWaves][kCB * kMB][64];
    __shared__ int list_n;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int r16 = lane & 15, g = lane >> 4;
    const int m0 = blockIdx.x * kShrinkRows;
    const int c0 = blockIdx.z * kShrinkCols;
    const int cols = x.parts * x.rank;

    List list;
    if (wave == 0) {
        list.build((SWIGLU_LDS char *)list_lds, x.ids, m0, x.M, x.slots, x.count);
        if (lane == 0) list_n = list.n;
    }
    __syncthreads();
    list.at((SWIGLU_LDS char *)list_lds);
    list.n = list_n;

    const int rows = min(kShrinkRows, x.M - m0);
    const __amdgpu_buffer_rsrc_t xr = rows_rsrc(x.X, m0, rows, x.K);
    const uint32_t voff = static_cast<uint32_t>(r16) * static_cast<uint32_t>(x.K) * 2u + g * 16u;
    const uint32_t blk = 16u * static_cast<uint32_t>(x.K) * 2u;
    const int units = (x.K + 63) / 64;
    const int u_begin = wave * units / kShrinkWaves, u_end = (wave + 1) * units / kShrinkWaves;

    for (int at = blockIdx.y; at < list.n; at += gridDim.y) {
        const int a = __builtin_amdgcn_readfirstlane(static_cast<int>(list.list[at]));
        const __amdgpu_buffer_rsrc_t ar =
            rows_rsrc(x.A, static_cast<int64_t>(a) * cols + c0, min(kShrinkCols, cols - c0), x.K);
        f32x4 acc[kCB][kMB];
#pragma unroll
        for (int c = 0; c < kCB; ++c)
#pragma unroll
            for (int m = 0; m < kMB; ++m) acc[c][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma nounroll
        for (int u = u_begin; u < u_end; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k0 = u * 64 + h * 32;
                const uint32_t v = k0 + g * 8 < x.K ? voff : kOutOfRange;
                u32x4 af[kCB], xf[kMB];
#pragma unroll
                for (int m = 0; m < kMB; ++m) xf[m] = bload16(xr, v, m * blk + k0 * 2u);
#pragma unroll
                for (int c = 0; c < kCB; ++c) af[c] = bload16(ar, v, c * blk + k0 * 2u);
#pragma unroll
                for (int c = 0; c < kCB; ++c)
#pragma unroll
                    for (int m = 0; m < kMB; ++m) acc[c][m] = mfma_16x16x32(af[c], xf[m], acc[c][m]);
            }
        }
#pragma unroll
        for (int c = 0; c < kCB; ++c)
#pragma unroll
            for (int m = 0; m < kMB; ++m) part[wave][c * kMB + m][lane] = acc[c][m];
        __syncthreads();
        for (int q = wave; q < kCB * kMB; q += kShrinkWaves) {
            f32x4 sum = part[0][q][lane];
#pragma unroll
            for (int w = 1; w < kShrinkWaves; ++w) sum += part[w][q][lane];
            const int c = c0 + 16 * (q / kMB) + 4 * g;
            const int row = 16 * (q % kMB) + r16;
            const int slot = list.slot_of(row, a, x.slots);
            if (slot >= 0 && c < cols) {
                const int64_t at_row = static_cast<int64_t>(m0 + row) * x.slots;
                // the weights of every slot that names a, the first one's T holding the sum
                float w = 0.0f;
                for (int j = slot; j < x.slots; ++j)
                    if (list.ids[row * x.slots + j] == a) w += x.weights ? x.weights[at_row + j] : 1.0f;
                w *= x.scale[a];
                const u32x2 v = {pack_bf16x2(sum[0] * w, sum[1] * w), pack_bf16x2(sum[2] * w, sum[3] * w)};
                *reinterpret_cast<u32x2 *>(x.T + (at_row + slot) * cols + c) = v;
            }
        }
        __syncthreads();
    }
}

hipError_t launch_lora_shrink(const uint16_t *X, const LoraTable &t, const int *ids,
                              const float *weights, int slots, uint16_t *T, int M, int K,
                              int parts, hipStream_t stream) {
    const int64_t tiles = ceil_div(M, kShrinkRows);
    const int64_t most = static_cast<int64_t>(kShrinkRows) * slots;
    int64_t y = t.count < most ? t.count : most;
    // about four workgroups a compute unit: with more rows, a workgroup takes
    // several of its rows' adapters
    const int64_t fill = ceil_div(1024, tiles);
    if (y > fill) y = fill;
    const ShrinkArgs a{X, t.A, t.scale, weights, ids, T, M, K, slots, t.rank, parts, t.count};
    hipLaunchKernelGGL(lora_shrink_kernel,
                       dim3((unsigned)tiles, (unsigned)y,
                            (unsigned)ceil_div(static_cast<int64_t>(parts) * t.rank, kShrinkCols)),
                       dim3(64 * kShrinkWaves), 0, stream, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Projections of at most 128 rows.  Bound by the weight's bytes: each
// workgroup takes 16 RB rows of the weight (columns of D) and all rows of X
// (16 MB of them), its four waves split K, and with few column tiles `splits`
// workgroups split K further.  The weight is the MFMA's first operand, read
// once from memory straight into registers (16 rows by 128 bytes at a time, no
// LDS and no barrier in the loop); X, small enough to stay in L2, is the
// second.  Gate and Up of an output are then neighbouring accumulator
// registers of one lane (the packed weight's rows alternate), so the epilogue
// needs no lane exchange.  The expansion goes on in the same accumulators: B's
// rows as the weight's, T as X, with Gate rows masked out of the Up product
// and the other way round.  The waves' sums meet in LDS, the workgroups' in
// the workspace (device-scope stores and an arrival count, split_tail.hpp),
// each in a fixed order.
// ---------------------------------------------------------------------------
struct StreamArgs {
    const uint16_t *X, *W;
    uint16_t *Y;
    int M, K, cols;    // W [cols][K]
    int splits;
    float *partials;
    unsigned *counters;
    LoraTerm lora;
};
constexpr int kStreamWaves = 4;

template <int MB, int RB, bool kGated>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void lora_stream_kernel(StreamArgs x) {
    constexpr int kParts = kGated ? 2 : 1;
    constexpr int kQuads = RB * MB;
    constexpr int kRows = 16 * MB;
    using List = AdapterList<kRows>;
    constexpr int kSumBytes = kStreamWaves * kQuads * 64 * 16;
    constexpr int kLds = kSumBytes > List::kBytes ? kSumBytes : List::kBytes;
    __shared__ __attribute__((aligned(16))) char smem[kLds];
    __shared__ int shared_word;
    SWIGLU_LDS char *lds = (SWIGLU_LDS char *)smem;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int r16 = lane & 15, g = lane >> 4;
    const int tile = blockIdx.x / x.splits, split = blockIdx.x % x.splits;
    const int n0 = tile * 16 * RB;
    const int rows = min(16 * RB, x.cols - n0);

    const __amdgpu_buffer_rsrc_t wr = rows_rsrc(x.W, n0, rows, x.K);
    const __amdgpu_buffer_rsrc_t xr = rows_rsrc(x.X, 0, x.M, x.K);
    const uint32_t voff = static_cast<uint32_t>(r16) * static_cast<uint32_t>(x.K) * 2u + g * 16u;
    const uint32_t blk = 16u * static_cast<uint32_t>(x.K) * 2u;
    // units of 64 k shared out over the waves of all splits
    const int workers = x.splits * kStreamWaves, worker = split * kStreamWaves + wave;
    const int units = (x.K + 63) / 64;
    const int u_begin = static_cast<int>(static_cast<int64_t>(worker) * units / workers);
    const int u_end = static_cast<int>(static_cast<int64_t>(worker + 1) * units / workers);

    f32x4 acc[RB][MB];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[b][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma nounroll
    for (int u = u_begin; u < u_end; ++u) {
        u32x4 wf[2][RB], xf[2][MB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k0 = u * 64 + h * 32;
            const uint32_t v = k0 + g * 8 < x.K ? voff : kOutOfRange;
#pragma unroll
            for (int b = 0; b < RB; ++b) wf[h][b] = bload16(wr, v, b * blk + k0 * 2u);
#pragma unroll
            for (int m = 0; m < MB; ++m) xf[h][m] = bload16(xr, v, m * blk + k0 * 2u);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    acc[b][m] = mfma_16x16x32(wf[h][b], xf[h][m], acc[b][m]);
    }

    // expansion
    const LoraTerm &lt = x.lora;
    List list;
    if (wave == 0) {
        list.build(lds, lt.ids, 0, lt.M, lt.slots, lt.count);
        if (lane == 0) shared_word = list.n;
    }
    __syncthreads();
    list.at(lds);
    list.n = shared_word;
    const int slot_bytes = kParts * lt.rank * 2;
    const __amdgpu_buffer_rsrc_t tr =
        make_rsrc(lt.T, static_cast<uint32_t>(lt.M * lt.slots * slot_bytes));
    const int rank8 = lt.rank / 8;
    const int steps = (list.n * rank8 + 3) / 4;
    for (int s = worker; s < steps; s += workers) {
        const ChunkOf ch = chunk_of(list, 4 * s + g, rank8);
        u32x4 bf[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            // past the last column: any row, its results are not stored
            const int n = min(n0 + 16 * b + r16, x.cols - 1);
            bf[b] = gload16(lt.B + (static_cast<int64_t>(ch.adapter) * x.cols + n) * lt.rank +
                            ch.element);
        }
        u32x4 tf[kParts][MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int row = 16 * m + r16;
            const int slot = list.slot_of(row, ch.adapter, lt.slots);
            const uint32_t off =
                ch.live && slot >= 0
                    ? static_cast<uint32_t>((row * lt.slots + slot) * slot_bytes + ch.element * 2)
                    : kOutOfRange;
#pragma unroll
            for (int p = 0; p < kParts; ++p) tf[p][m] = bload16(tr, off, p * lt.rank * 2u);
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                u32x4 w = bf[b];
                if constexpr (kGated)
                    if ((lane & 1) != p) w = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (int m = 0; m < MB; ++m) acc[b][m] = mfma_16x16x32(w, tf[p][m], acc[b][m]);
            }
    }
    __syncthreads();   // the list is read; its LDS takes the sums

    SWIGLU_LDS f32x4 *sums = reinterpret_cast<SWIGLU_LDS f32x4 *>(lds);
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m) sums[(wave * kQuads + b * MB + m) * 64 + lane] = acc[b][m];
    __syncthreads();
    constexpr int kMine = (kQuads + kStreamWaves - 1) / kStreamWaves;
    f32x4 d[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int q = i * kStreamWaves + wave;
        if (q < kQuads) {
            d[i] = sums[q * 64 + lane];
#pragma unroll
            for (int w = 1; w < kStreamWaves; ++w) d[i] += sums[(w * kQuads + q) * 64 + lane];
        }
    }
    if (x.splits > 1) {
        // partial sums of quad q of split j of this tile at [(tile, j, q)][lane]
        constexpr uint32_t kSlot = kQuads * 64 * 16;
        float *slots = x.partials + static_cast<int64_t>(tile) * x.splits * (kSlot / 4);
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(slots, x.splits * kSlot);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int q = i * kStreamWaves + wave;
            if (q < kQuads)
                __builtin_amdgcn_raw_buffer_store_b128(
                    __builtin_bit_cast(u32x4, d[i]), pr,
                    static_cast<int>(split * kSlot + (q * 64 + lane) * 16), 0, kDeviceScope);
        }
        wait_vmcnt<0>();
        __syncthreads();
        if (threadIdx.x == 0)
            shared_word = static_cast<int>(__hip_atomic_fetch_add(
                x.counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        __syncthreads();
        if (shared_word + 1 != x.splits) return;
        if (threadIdx.x == 0)
            __hip_atomic_store(x.counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int q = i * kStreamWaves + wave;
            if (q < kQuads) {
                f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int j = 0; j < x.splits; ++j)
                    sum += __builtin_bit_cast(
                        f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   pr, static_cast<int>(j * kSlot + (q * 64 + lane) * 16), 0,
                                   kDeviceScope));
                d[i] = sum;
            }
        }
    }
    // lane (r16, g) of quad (b, m) holds columns n0 + 16 b + 4 g + 0..3 of row 16 m + r16
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int q = i * kStreamWaves + wave;
        const int row = 16 * (q % MB) + r16, col = n0 + 16 * (q / MB) + 4 * g;
        if (q < kQuads && row < x.M && col < x.cols) {
            if constexpr (kGated) {
                const uint32_t v = pack_bf16x2(silu(d[i][0]) * d[i][1], silu(d[i][2]) * d[i][3]);
                *reinterpret_cast<uint32_t *>(x.Y + static_cast<int64_t>(row) * (x.cols / 2) +
                                              col / 2) = v;
            } else {
                const u32x2 v = {pack_bf16x2(d[i][0], d[i][1]), pack_bf16x2(d[i][2], d[i][3])};
                *reinterpret_cast<u32x2 *>(x.Y + static_cast<int64_t>(row) * x.cols + col) = v;
            }
        }
    }
}

template <int MB, int RB, bool kGated>
static hipError_t run_stream(StreamArgs a, int tiles, hipStream_t stream) {
    hipLaunchKernelGGL((lora_stream_kernel<MB, RB, kGated>), dim3(tiles * a.splits),
                       dim3(64 * kStreamWaves), 0, stream, a);
    return hipGetLastError();
}

// Weight rows of a workgroup (16 RB) and its splits along K.  The more rows,
// the fewer times X is read; the fewer, the more workgroups there are to keep
// loads in flight: at least two a compute unit, else K is split (a worker
// keeps at least two 64-k units).
struct StreamPlan {
    int rb, tiles, splits;
};
static StreamPlan stream_plan(int M, int cols, int K, const GemmWorkspace &ws) {
    const int want = 2 * ws.cus;
    StreamPlan p{};
    p.rb = M <= 64 ? 4 : 2;   // (at most 16 accumulator quads a lane: 64 KiB of sums in LDS)
    while (p.rb > 1 && ceil_div(cols, 16 * p.rb) < want) p.rb /= 2;
    p.tiles = static_cast<int>(ceil_div(cols, 16 * p.rb));
    p.splits = 1;
    if (p.tiles < want && ws.base != nullptr && ws.counters != nullptr &&
        p.tiles <= ws.max_counters) {
        int s = want / p.tiles;
        const int most = static_cast<int>(ceil_div(K, 64) / (2 * kStreamWaves));
        if (s > most) s = most;
        const int mb = M <= 16 ? 1 : M <= 32 ? 2 : M <= 64 ? 4 : 8;
        const uint64_t slot = static_cast<uint64_t>(p.rb) * mb * 1024;
        if (s > 1 && static_cast<uint64_t>(p.tiles) * s * slot <= ws.bytes) p.splits = s;
    }
    return p;
}

template <int MB, bool kGated>
static hipError_t stream_rb(const StreamArgs &a, const StreamPlan &p, hipStream_t stream) {
    if constexpr (MB <= 4)
        if (p.rb == 4) return run_stream<MB, 4, kGated>(a, p.tiles, stream);
    if (p.rb == 2) return run_stream<MB, 2, kGated>(a, p.tiles, stream);
    return run_stream<MB, 1, kGated>(a, p.tiles, stream);
}

template <bool kGated>
static hipError_t launch_stream(const uint16_t *X, const uint16_t *W, uint16_t *Y, int M, int cols,
                                int K, const LoraTerm &lora, const GemmWorkspace &ws,
                                hipStream_t stream) {
    const StreamPlan p = stream_plan(M, cols, K, ws);
    const StreamArgs a{X, W, Y, M, K, cols, p.splits, static_cast<float *>(ws.base), ws.counters, lora};
    if (M <= 16) return stream_rb<1, kGated>(a, p, stream);
    if (M <= 32) return stream_rb<2, kGated>(a, p, stream);
    if (M <= 64) return stream_rb<4, kGated>(a, p, stream);
    return stream_rb<8, kGated>(a, p, stream);
}

hipError_t launch_lora_stream(const uint16_t *X, const uint16_t *W, uint16_t *Y, int M, int cols,
                              int K, bool gated, const LoraTable &t, const int *ids, int slots,
                              const uint16_t *T, const GemmWorkspace &ws, hipStream_t stream) {
    const LoraTerm lora{T, t.B, ids, M, slots, t.rank, t.count, cols};
    return gated ? launch_stream<true>(X, W, Y, M, cols, K, lora, ws, stream)
                 : launch_stream<false>(X, W, Y, M, cols, K, lora, ws, stream);
}

}  // namespace swiglu
