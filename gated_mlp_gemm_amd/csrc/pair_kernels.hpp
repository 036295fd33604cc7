// Two products of a backward pass in one launch: the gradient by an activation (X) and
// the gradient by a weight (W), which read the same operand and wait for nothing of each
// other.  One after the other, each has a last round that leaves compute units idle, and
// all workgroups' epilogues store at the same time; together the second's tiles fill the
// first's last round, and the tiles' different lengths keep the epilogues apart.
//
// The work items are the first product's tiles, whole or split along K into pieces
// (split_tail.hpp), then the second's, drawn by the workgroups (draws.hpp).  Which
// workgroup runs an item changes nothing in its result.
#pragma once

#include "draws.hpp"
#include "tile_kernels.hpp"

namespace swiglu {

struct PairCounts {
    uint64_t *words;   // one for each XCD
    uint64_t tag;
    int w_first;       // the weight's gradient is the first product
};

// The items of this workgroup: fetch(), by all threads, asks for the item behind the
// next one; next(), behind a tile's last LDS access, gives the next one to all.
struct Draw {
    Draws draws;
    unsigned ticket;
    int ahead;           // the item behind the current one

    __device__ __forceinline__ void init(const PairCounts &c, int total) {
        draws.begin(c.words, c.tag, blockIdx.x, gridDim.x, total, threadIdx.x == 0);
        ahead = static_cast<int>(blockIdx.x + gridDim.x);
    }
    __device__ __forceinline__ void fetch() {
        if (threadIdx.x == 0) ticket = draws.ask();
    }
    __device__ __forceinline__ int next(char *smem) {
        unsigned *shared = reinterpret_cast<unsigned *>(smem);
        if (threadIdx.x == 0) {
            draws.answered(ticket);
            *shared = ticket;
        }
        __syncthreads();
        const unsigned t = __builtin_amdgcn_readfirstlane(*shared);
        __syncthreads();   // read by all before the next item's loads reuse LDS
        const int item = ahead;
        ahead = draws.item(t);
        return item;
    }
};

// The items of one product, from `item` on (numbered from this product's first, which is
// number `base` of all); returns the first item drawn that is not one of them.
template <class S, class Epi, bool kEven>
__device__ __forceinline__ int pair_items(char *smem, const KMajor &A, const KMajor &B, int M, int K,
                                          const Epi &epi, const Schedule &sch, int item, int base,
                                          Draw &draw) {
    SWIGLU_LDS char *lds = (SWIGLU_LDS char *)smem;
    const int nk = sch.nk;
    if (item < sch.dp) {
        Pipeline<S> pl;
        pl.init(lds);
        TileLoader<S> ld;
        int tm, tn;
        tile_coords(xcd_order(item, sch.dp), sch.tiles_m, sch.tiles_n, sch.group_m, tm, tn);
        ld.init(A, tm * S::BM, B, tn * S::BN, K, lds);
        auto issue = [&](int s, int part, SWIGLU_LDS char *dst, int j) {
            ld.template issue<kEven>(s < nk ? s : nk, part, dst, j);
        };
        pl.prologue_issue(issue);
        for (bool more = true; more;) {
            typename S::Acc acc[S::TM][S::TN];
            const int m0 = tm * S::BM, n0 = tn * S::BN;
            pl.prologue_wait();
            draw.fetch();
            run_tile<S, kEven>(pl, issue, nk, acc);
            pl.drain(acc);
            item = draw.next(smem) - base;
            more = item < sch.dp;
            if (more) {
                tile_coords(xcd_order(item, sch.dp), sch.tiles_m, sch.tiles_n, sch.group_m, tm, tn);
                ld.init(A, tm * S::BM, B, tn * S::BN, K, lds);
                pl.prologue_issue(issue);
            }
            epi.template apply<S>(acc, m0, n0, threadIdx.x);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    const int n = sch.dp + sch.split_tiles * sch.pieces;
    while (item < n) {
        const int j = item - sch.dp;
        const int piece = j % sch.pieces;
        const int kb = piece_begin(piece, nk, sch.pieces);
        const int ke = piece_begin(piece + 1, nk, sch.pieces);
        int tm, tn;
        tile_coords(sch.dp + j / sch.pieces, sch.tiles_m, sch.tiles_n, sch.group_m, tm, tn);
        typename S::Acc acc[S::TM][S::TN];
        draw.fetch();
        tile_mainloop<S, kEven>(lds, A, B, M, K, tm * S::BM, tn * S::BN, kb, ke, nk, acc);
        item = draw.next(smem) - base;
        store_partial<S>(sch.partials + static_cast<int64_t>(j) * S::BM * S::BN, acc, threadIdx.x);
    }
    return item + base;
}

template <class SX, class EX, class SW>
__global__ __launch_bounds__(256, 1) void gemm_pair_kernel(KMajor Ax, KMajor Bx, int Mx, int Kx, EX ex,
                                                           Schedule sx, KMajor Aw, KMajor Bw, int Mw,
                                                           int Kw, WeightGradEpilogue ew, Schedule sw,
                                                           PairCounts counts) {
    static_assert(SX::kThreads == 256 && SW::kThreads == 256 && SW::kATr && SW::kBTr, "pairs");
    constexpr int kLds = SX::kLdsBytes > SW::kLdsBytes ? SX::kLdsBytes : SW::kLdsBytes;
    __shared__ __attribute__((aligned(128))) char smem[kLds];
    const int nx = sx.dp + sx.split_tiles * sx.pieces, nw = sw.dp + sw.split_tiles * sw.pieces;
    int item = blockIdx.x;
    if (item >= nx + nw) return;
    Draw draw;
    draw.init(counts, nx + nw);
    int base = 0;
#pragma nounroll
    for (int phase = 0; phase < 2; ++phase) {
        const bool w = (phase == 0) == (counts.w_first != 0);
        if (item < base + (w ? nw : nx)) {
            if (w)
                item = pair_items<SW, WeightGradEpilogue, true>(smem, Aw, Bw, Mw, Kw, ew, sw,
                                                                item - base, base, draw);
            else if (Kx % SX::BK == 0)
                item = pair_items<SX, EX, true>(smem, Ax, Bx, Mx, Kx, ex, sx, item - base, base, draw);
            else
                item = pair_items<SX, EX, false>(smem, Ax, Bx, Mx, Kx, ex, sx, item - base, base, draw);
        }
        base += w ? nw : nx;
    }
}

// gemm_pair_kernel on `grid` workgroups (a multiple of 8)
template <class SX, class EX, class SW>
struct PairLaunch {
    static hipError_t run(int grid, const KMajor &Ax, const KMajor &Bx, int Mx, int Kx, const EX &ex,
                          const Schedule &sx, const KMajor &Aw, const KMajor &Bw, int Mw, int Kw,
                          const WeightGradEpilogue &ew, const Schedule &sw, const PairCounts &counts,
                          hipStream_t stream);
};

}  // namespace swiglu
