// Products of few rows with 4-bit weights: the weights' stream, and little else.
//
// A workgroup has 16 R rows of the weight and all of K; its W waves share K in
// blocks of 128, wave w taking the blocks w, w + W, ...  A wave streams its blocks
// through a ring of D slots of LDS that no other wave touches (no barrier until the
// sums meet): a block's codes, 64 bytes of each row, straight to LDS in pieces of 64
// bytes, which four lanes fetch together, and the same 128 k of the activations.
//
// The weight is the MFMA's row operand: lane l = 16 q + i of v_mfma_f32_16x16x32_bf16
// holds 8 k of row i.  The k of a lane may be any as long as both operands agree: the
// four MFMAs of a block take k = 32 q + 8 j of the block (j = 0..3), so a lane's codes
// are 16 bytes that lie together, and they are one group of 32: one scale a lane.
// The codes become bf16 in registers, exactly.
//
// The scales of the workgroup's rows lie together in memory: they go to LDS first, all
// of them, and a lane reads its byte there (from memory, 4 bytes of each of 16 rows a
// block, they took a fifth of the time: 16.0 against 13.1 us at M=1 K=3584, 37888 rows).
//
// The waves' sums meet in LDS, added in the order of the waves, and the workgroup
// finishes its outputs: SiLU(Gate) Up of adjacent rows, or the sums.
//
// Measured: one row, K=3584, 37888 rows (72 MB): 14.6 us, 4.9 TB/s, the rate of a copy,
// and 12.2 where the caches hold part of the weight.  24 rows: K=8192, 59136 rows (257 MB)
// 69 us, K=29568, 8192 rows (129 MB) 43 us, 3.7 and 3.0 TB/s: every workgroup reads all
// activations, 1.4 and 2.8 bytes a byte of the weight.  At these two weights rings of 1.5
// times the bytes, 6 or 12 waves and rings without the rows past the 24th are within 5 %;
// at 37888 x 3584 and 27648 x 5120 a workgroup of 80 or 128 rows is 17 and 11 % faster
// than the forms there are (launch_few).  LDS is at work in 30 and 17 % of the two launches'
// cycles; of those 73 and 47 % count as bank conflicts.  (The scales of a tile's 16 rows are
// K / 32 bytes apart: at K=8192 all in one bank.  A pitch apart from K's is not built.)
#pragma once

#include "gemm_core.hpp"

namespace swiglu {

// NX: KiB of activations a block and slot, 4 rows each; M <= 4 NX <= 64.
template <bool GATED, int R, int NX, int D, int W>
struct Mx4Few {
    static constexpr int kThreads = 64 * W;
    static constexpr int kRows = 16 * R;
    static constexpr int kSlot = (R + NX) * 1024;
    static constexpr int kRing = D * kSlot;
    static constexpr int MB = (NX + 3) / 4;   // column blocks of 16 activation rows
    static constexpr int kSums = W * R * MB * 1024;
    static constexpr int kRings = W * kRing > kSums ? W * kRing : kSums;   // LDS before the scales
    static constexpr int kVm = R + NX;       // vector memory operations a block
    static_assert(D * kVm < 64, "vmcnt is a 6-bit counter");
    static_assert(NX == 1 || NX == 2 || NX % 4 == 0, "whole blocks of 16 rows, or fewer rows");

    __amdgpu_buffer_rsrc_t codes, scales, x;
    uint32_t vcodes, vx[NX];           // byte offsets of the lane in block 0
    int kc, kx[NX];                    // K minus the lane's first k of each
    uint32_t rcodes, rx[4];            // LDS addresses of the lane's reads in slot 0
    uint32_t rscale;                   // ... of its scale in block 0, tile 0
    int ks;
    SWIGLU_LDS char *ring;
    int tile_codes, tile_scales;       // bytes from a 16-row tile to the next

    // LDS bytes of a launch: the rings, and K / 2 bytes of scales for 16 rows (and what
    // the last load of 16 bytes a lane may clear behind them).
    static constexpr int lds_bytes(int K) { return kRings + R * (K / 2) + kThreads * 16; }

    __device__ __forceinline__ void init(const uint16_t *X, const uint8_t *Q, const uint8_t *S, int M,
                                         int rows, int K, int row0, SWIGLU_LDS char *lds) {
        const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
        const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
        const int pitch = K / 2, spitch = K / 32, here = min(kRows, rows - row0);
        codes = make_rsrc(Q + static_cast<int64_t>(row0) * pitch, static_cast<uint32_t>(here * pitch));
        scales = make_rsrc(S + static_cast<int64_t>(row0) * spitch, static_cast<uint32_t>(here * spitch));
        x = make_rsrc(X, static_cast<uint32_t>(M) * static_cast<uint32_t>(K) * 2u);
        SWIGLU_LDS char *all = lds + kRings;
        for (int o = 0; o < here * spitch; o += kThreads * 16)
            dma16(scales, all + o + wave * 1024, static_cast<uint32_t>(threadIdx.x) * 16u,
                  static_cast<uint32_t>(o));
        rscale = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(all)) + i * spitch +
                 (q < spitch ? q : 0);
        tile_codes = 16 * pitch;
        tile_scales = 16 * spitch;
        // chunk c of row r lies in place c ^ (r / 4): the 16 lanes of one LDS cycle
        // read the same chunk of 16 rows
        const int r = lane >> 2, c = (lane & 3) ^ (r >> 2);
        vcodes = static_cast<uint32_t>(r * pitch + c * 16);
        kc = K - 32 * c;
        ks = K - 32 * q;
        ring = lds + wave * kRing;
        const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(ring));
        rcodes = base + i * 64 + ((q ^ (i >> 2)) * 16);
#pragma unroll
        for (int n = 0; n < NX; ++n) {
            const int m = 4 * n + q, cx = i ^ (m & 15);   // 16 chunks a row
            vx[n] = static_cast<uint32_t>(m) * static_cast<uint32_t>(K) * 2u + cx * 16u;
            kx[n] = K - 8 * cx;
        }
        const int m = NX < 4 ? i % (4 * NX) : i;   // (rows that are not there: any)
#pragma unroll
        for (int j = 0; j < 4; ++j) rx[j] = base + R * 1024 + m * 256 + (((4 * q + j) ^ m) * 16);
    }
    // Block b of K into slot `slot`; blocks and parts of blocks past K are zeros.
    __device__ __forceinline__ void fetch(int b, int slot) const {
        const int k0 = b * 128;
        SWIGLU_LDS char *to = ring + slot * kSlot;
#pragma unroll
        for (int t = 0; t < R; ++t)
            dma16(codes, to + t * 1024, k0 < kc ? vcodes : kOutOfRange,
                  static_cast<uint32_t>(b * 64 + t * tile_codes));
#pragma unroll
        for (int n = 0; n < NX; ++n)
            dma16(x, to + (R + n) * 1024, k0 < kx[n] ? vx[n] : kOutOfRange,
                  static_cast<uint32_t>(b * 256));
    }
    struct Block {
        u32x4 w[R], x[MB][4];
        uint32_t scale[R];
    };
    // (A lane past K reads zeros of codes and a scale of its own row: zeros times a number,
    // or NaN in a row whose sum is NaN by that group already.)
    template <int SLOT, int... T>
    __device__ __forceinline__ void read(Block &f, int b, std::integer_sequence<int, T...>) const {
        const uint32_t at = rscale + static_cast<uint32_t>(b * 128 < ks ? b * 4 : 0);
        ((f.scale[T] = asm_read_u8(at + static_cast<uint32_t>(T * tile_scales))), ...);
        ((f.w[T] = asm_read_b128<SLOT * kSlot + T * 1024>(rcodes)), ...);
        read_x<SLOT, 0>(f);
        asm volatile("s_waitcnt lgkmcnt(0)");
        (landed(f.w[T]), ...);
#pragma unroll
        for (int e = 0; e < R; ++e) asm volatile("" : "+v"(f.scale[e]));
#pragma unroll
        for (int e = 0; e < 4 * MB; ++e) landed(f.x[e / 4][e % 4]);
    }
    template <int SLOT, int B>
    __device__ __forceinline__ void read_x(Block &f) const {
        if constexpr (B < MB) {
            f.x[B][0] = asm_read_b128<SLOT * kSlot + B * 4096>(rx[0]);
            f.x[B][1] = asm_read_b128<SLOT * kSlot + B * 4096>(rx[1]);
            f.x[B][2] = asm_read_b128<SLOT * kSlot + B * 4096>(rx[2]);
            f.x[B][3] = asm_read_b128<SLOT * kSlot + B * 4096>(rx[3]);
            read_x<SLOT, B + 1>(f);
        }
    }
    __device__ __forceinline__ static void multiply(const Block &f, f32x4 (&acc)[R][MB]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int t = 0; t < R; ++t) {
                const uint32_t w = f.w[t][j];
                const float s = __builtin_bit_cast(float, f.scale[t] << 23);
                const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
                const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
                const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
                const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
                const bf16x8 v = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    const u32x4 y = f.x[b][j];
                    acc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        v, __builtin_bit_cast(bf16x8, y), acc[t][b], 0, 0, 0);
                }
            }
        }
    }
    // One round of the ring: blocks of slots 0..D-1, and, unless it is the last, the
    // fetch of the blocks D rounds on into the slots just read.
    template <bool LAST, int... SLOT>
    __device__ __forceinline__ void round(int b, f32x4 (&acc)[R][MB],
                                          std::integer_sequence<int, SLOT...>) const {
        (
            [&] {
                wait_vmcnt<LAST ? (D - 1 - SLOT) * kVm : (D - 1) * kVm>();
                Block f;
                read<SLOT>(f, b + SLOT * W, std::make_integer_sequence<int, R>{});
                if constexpr (!LAST) fetch(b + (D + SLOT) * W, SLOT);
                multiply(f, acc);
            }(),
            ...);
    }
};

// (two waves a SIMD: the compiler then keeps the sums in the first 256 registers)
template <bool GATED, int R, int NX, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void mx4_few_kernel(const uint16_t *__restrict__ X,
                                                            const uint8_t *__restrict__ Q,
                                                            const uint8_t *__restrict__ S,
                                                            uint16_t *__restrict__ Y, int M,
                                                            int rows, int K) {
    using P = Mx4Few<GATED, R, NX, D, W>;
    extern __shared__ __attribute__((aligned(128))) char smem[];   // P::lds_bytes(K)
    P p;
    const int row0 = blockIdx.x * P::kRows;
    p.init(X, Q, S, M, rows, K, row0, (SWIGLU_LDS char *)smem);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    constexpr auto slots = std::make_integer_sequence<int, D>{};
#pragma unroll
    for (int d = 0; d < D; ++d) p.fetch(wave + d * W, d);
    f32x4 acc[R][P::MB];
#pragma unroll
    for (int e = 0; e < R * P::MB; ++e) acc[e / P::MB][e % P::MB] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int rounds = (K + 128 * W * D - 1) / (128 * W * D);
    int b = wave;
    wait_vmcnt<D * P::kVm>();   // this wave's share of the scales
    block_barrier();            // ... and everyone's
    for (int n = 1; n < rounds; ++n, b += D * W) p.template round<false>(b, acc, slots);
    p.template round<true>(b, acc, slots);
    __syncthreads();   // every wave is done with its ring
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);
    constexpr int kBlocks = R * P::MB;
#pragma unroll
    for (int e = 0; e < kBlocks; ++e) sums[(wave * kBlocks + e) * 64 + lane] = acc[e / P::MB][e % P::MB];
    __syncthreads();
    for (int e = threadIdx.x; e < kBlocks * 64; e += P::kThreads) {
        f32x4 v = sums[e];
#pragma unroll
        for (int w = 1; w < W; ++w) v += sums[w * kBlocks * 64 + e];
        // element k of v: row 4 q + k of tile t, activation row m
        const int l = e & 63, t = (e >> 6) / P::MB;
        const int m = ((e >> 6) % P::MB) * 16 + (l & 15);
        const int row = row0 + 16 * t + 4 * (l >> 4);
        if (m >= M || row >= rows) continue;
        if constexpr (GATED) {
            uint16_t *y = Y + static_cast<int64_t>(m) * (rows / 2) + row / 2;
            *reinterpret_cast<uint32_t *>(y) = pack_bf16x2(silu(v[0]) * v[1], silu(v[2]) * v[3]);
        } else {
            uint16_t *y = Y + static_cast<int64_t>(m) * rows + row;
            *reinterpret_cast<u32x2 *>(y) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
    }
}

}  // namespace swiglu
