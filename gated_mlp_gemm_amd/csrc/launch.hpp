// Host-side launchers of the kernels in kernels.hip.  Arguments are assumed
// validated by the C ABI layer (api.cpp); each launcher enqueues on `stream`
// and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace swiglu {

// Caller-owned scratch for the split-tail schedule (may be empty: base == nullptr).
struct GemmWorkspace {
    void *base;
    uint64_t bytes;
    int cus;          // compute units of the device
    int tile;         // variant I / ablation GEMM tile: 0 = by the cost model, 256 or 128 = forced
    int tail;         // partly idle last round: 0 = by the cost model, else a TailChoice
    uint64_t tag;     // of the meetings of one launch's workgroups (arrivals.hpp)
};
// How the tiles of a partly idle last round run (GemmWorkspace::tail).
enum TailChoice { kTailAuto = 0, kTailWhole = 1, kTailPieces = 2, kTailQuarters = 3, kTailFixup = 4 };
// Scratch that lets the single-accumulator GEMMs split the tiles of a partial
// last round along K (the same for every shape: one fp32 256 x 256 tile slot
// per compute unit).
uint64_t partials_bytes(int cus);
uint64_t workspace_bytes_for(int cus);

// Text naming the kernels (tile shape, schedule) a GEMM over an M x cols
// output would launch (snprintf semantics).
// fused_i: the variant-I GEMM (its M <= 128 tile choice differs from the
// ablation's and the down projection's).
int describe_gemm(int M, int cols, int K, const GemmWorkspace &ws, const char *epi, char *buf,
                  size_t n, bool fused_i = false);
int describe_fused_sequential(int M, int N, int K, const GemmWorkspace &ws, char *buf, size_t n);

hipError_t launch_pack(const uint16_t *W1, const uint16_t *W2, uint16_t *Wf, int64_t K,
                       int64_t N, hipStream_t stream);
// Linear-layer-layout weights W1t, W2t [N][K] -> packed [2N][K] (row interleave).
hipError_t launch_pack_nk(const uint16_t *W1t, const uint16_t *W2t, uint16_t *Wf, int64_t K,
                          int64_t N, hipStream_t stream);
hipError_t launch_silu_mul(const uint16_t *g, const uint16_t *u, uint16_t *y, int64_t count,
                           hipStream_t stream);
// lda / ldy: elements from one row of A / Y to the next (K / N when contiguous).
hipError_t launch_fused_interleaved(const uint16_t *A, int lda, const uint16_t *Wf, uint16_t *Y,
                                    int ldy, int M, int N, int K, const GemmWorkspace &ws,
                                    hipStream_t stream);
// ws: only its compute-unit count (the persistent kernel's grid) and tail
// choice are used
hipError_t launch_fused_sequential(const uint16_t *A, int lda, const uint16_t *Wf, uint16_t *Y,
                                   int ldy, int M, int N, int K, const GemmWorkspace &ws,
                                   hipStream_t stream);
// phase 0: C = A . W1 (Gate columns of W_fused), phase 1: C = A . W2 (Up columns)
hipError_t launch_gemm_store(const uint16_t *A, const uint16_t *Wf, int phase, uint16_t *C,
                             int M, int N, int K, const GemmWorkspace &ws, hipStream_t stream);
// Out [M][D] = bf16(H [M][N] . W3), W3 given K-contiguous as W3t [D][N].
hipError_t launch_down_proj(const uint16_t *H, const uint16_t *W3t, uint16_t *Out, int M, int N,
                            int D, const GemmWorkspace &ws, hipStream_t stream);
// Training.  H and GU [M][2N] (Gate and Up, bf16, interleaved) of one pass over A.
hipError_t launch_fused_train(const uint16_t *A, const uint16_t *Wf, uint16_t *H, uint16_t *GU,
                              int M, int N, int K, const GemmWorkspace &ws, hipStream_t stream);
// launch_down_proj with the training calls' schedules.
hipError_t launch_down_train(const uint16_t *H, const uint16_t *W3t, uint16_t *Out, int M, int N,
                             int D, const GemmWorkspace &ws, hipStream_t stream);
// dGU of a given dH, count = M N (a multiple of 8); dGU may be GU.
hipError_t launch_gate_grad(const uint16_t *dH, const uint16_t *GU, uint16_t *dGU, int64_t count,
                            hipStream_t stream);
// Gradients by an activation (bf16) and by a weight (fp32 or bf16, f32; + add, which may
// be the gradient itself), each unless it is NULL; M == 0: the weight's is zeros (+ add).
//   down projection: dH [M][N] = dOut [M][D] . W3, dW3t [D][N] = dOut^T . H
hipError_t launch_down_backward(const uint16_t *dOut, const uint16_t *H, const uint16_t *W3t,
                                uint16_t *dH, void *dW3t, const void *add, bool f32, int M, int N,
                                int D, const GemmWorkspace &ws, hipStream_t stream);
//   ... with dGU [M][2N] of that dH, which stays in registers (dGU may be GU)
hipError_t launch_gate_backward(const uint16_t *dOut, const uint16_t *H, const uint16_t *W3t,
                                const uint16_t *GU, uint16_t *dGU, void *dW3t, const void *add,
                                bool f32, int M, int N, int D, const GemmWorkspace &ws,
                                hipStream_t stream);
//   SwiGLU stage: dA [M][K] = dGU [M][2N] . W_fused^T, dW_fused [2N][K] = dGU^T . A
hipError_t launch_stage_backward(const uint16_t *dGU, const uint16_t *A, const uint16_t *W_fused,
                                 uint16_t *dA, void *dW, const void *add, bool f32, int M, int N,
                                 int K, const GemmWorkspace &ws, hipStream_t stream);
// What a backward call with all its gradients launches, as text (snprintf semantics); add:
// the weights' gradients are added to sums.
enum BackwardCall { kDownBackward = 0, kStageBackward = 1, kBlockBackward = 2 };
void describe_backward(BackwardCall call, bool f32, bool add, int M, int N, int K,
                       const GemmWorkspace &ws, char *buf, size_t n);
// 4-bit weights: codes [rows][K / 2] and scales [rows][K / 32] of `count` numbers.
hipError_t launch_quantize_mx4(const uint16_t *x, uint8_t *q, uint8_t *s, int64_t count,
                               hipStream_t stream);
hipError_t launch_dequantize_mx4(const uint8_t *q, const uint8_t *s, uint16_t *x, int64_t count,
                                 hipStream_t stream);
// The product of at most kMx4FewRows rows with a weight [rows][K] (gated: the packed
// one, Y [M][rows / 2]); hipErrorNotSupported where K is too long for it, nothing
// launched.  (The kernel has forms for at most 64 rows.  Behind them are 128x64 tiles, up to
// 128 rows, and the step to them is dear, us at 64 / 65 / 128 rows: K=3584 N=18944 Gate/Up
// 39.5 / 58.0 / 59.0, down projection 29.5 / 30.1 / 31.8; K=8192 N=29568 118 / 178 / 184 and
// 71 / 93 / 100; K=896 N=4864 6.6 / 8.0 / 8.3 and 8.1 / 13.6 / 13.8.)
constexpr int kMx4FewRows = 64;
hipError_t launch_mx4_few(const uint16_t *X, const uint8_t *Q, const uint8_t *S, uint16_t *Y, int M,
                          int rows, int K, bool gated, int cus, hipStream_t stream);
hipError_t launch_fused_mx4(const uint16_t *A, const uint8_t *Wq, const uint8_t *Ws, uint16_t *Y,
                            int M, int N, int K, const GemmWorkspace &ws, hipStream_t stream);
hipError_t launch_down_proj_mx4(const uint16_t *H, const uint8_t *W3q, const uint8_t *W3s,
                                uint16_t *Out, int M, int N, int D, const GemmWorkspace &ws,
                                hipStream_t stream);
// FP8 (E4M3) path: q = fp8(x * 2^-scale_exp); variant I on FP8 operands with
// the epilogue scaling Gate and Up by `scale` (= 2^(a_exp + w_exp)).
hipError_t launch_quantize_fp8(const uint16_t *x, uint8_t *q, int64_t count, int scale_exp,
                               hipStream_t stream);
hipError_t launch_fused_interleaved_fp8(const uint8_t *A8, const uint8_t *Wf8, uint16_t *Y,
                                        int M, int N, int K, float scale,
                                        const GemmWorkspace &ws, hipStream_t stream);
hipError_t launch_fused_sequential_fp8(const uint8_t *A8, const uint8_t *Wf8, uint16_t *Y, int M,
                                       int N, int K, float scale, hipStream_t stream);
int describe_gemm_fp8(int M, int cols, int K, const GemmWorkspace &ws, char *buf, size_t n);
// The router and its gradient (route_kernels.hip).
constexpr int kMaxRouteE = 512, kMaxRouteK = 16;
uint64_t route_workspace_bytes(int64_t M, int64_t E, int cus);
// workspace: without it (or too few bytes) one workgroup does it all; tag: of the
// workgroups' meeting (arrivals.hpp).
hipError_t launch_route(const void *logits, bool bf16, const uint8_t *valid, int *ids,
                        float *weights, int *counts, float *loss, int64_t M, int E, int k,
                        bool normalize, void *workspace, uint64_t workspace_bytes, uint64_t tag,
                        int cus, hipStream_t stream);
hipError_t launch_route_backward(const void *logits, bool bf16, const uint8_t *valid,
                                 const int *ids, const float *weights, const int *counts,
                                 const float *d_weights, const float *d_loss, void *d_logits,
                                 int64_t M, int E, int k, bool normalize, int cus,
                                 hipStream_t stream);
// Low-rank adapters (lora.hpp): a table of `count` of them beside a projection.
constexpr int kMaxLoraCount = 8192;   // adapters of a table
constexpr int kMaxLoraSlots = 8;      // adapters of a row
constexpr int kMaxLoraRank = 256;
struct LoraTable {
    const uint16_t *A, *B;   // [count][parts * rank][K], [count][cols][rank]
    const float *scale;      // [count]
    int count, rank;
};
// Bytes of a plan of 256 rows (lora.hpp).
int lora_plan_bytes(int count, int slots);
// T [M][slots][parts * rank] = weight scale X . A^T of each row's adapters, 4 bytes an
// element, and the plans of each 256 rows (lora.hpp).  ws: scratch to split K (may be empty).
hipError_t launch_lora_shrink(const uint16_t *X, const LoraTable &t, const int *ids,
                              const float *weights, int slots, uint16_t *T, char *plans, int M,
                              int K, int parts, const GemmWorkspace &ws, hipStream_t stream);
// The projection of X [M][K] with the expansion of T, and its epilogue: gated,
// W the packed [cols = 2N][K] weight and Y [M][N]; else W [cols][K], Y [M][cols].
hipError_t launch_lora_project(const uint16_t *X, const uint16_t *W, uint16_t *Y, int M, int cols,
                               int K, bool gated, const LoraTable &t, int slots, const uint16_t *T,
                               const char *plans, const GemmWorkspace &ws, hipStream_t stream);
// Largest workgroup count any launcher uses for an M x cols output tile grid.
int64_t max_tiles(int64_t M, int64_t cols);

}  // namespace swiglu
