// Internal declarations shared by the CUDA translation units of libmoe.so.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Rows per expert tile of the grouped GEMMs (the UMMA M dimension).
constexpr int kTileM = 128;
// Largest supported expert count and top-K.
constexpr int kMaxE = 256;
constexpr int kMaxK = 8;
// Rows per token kept in the compact per-token row list of the Token Rounding
// forward (a token with more falls back to its row_map entries).
constexpr int kTokCap = 16;
// Largest Token Rounding tile size accepted.
constexpr int kMaxRoundM = 1 << 16;
// Tokens per grouping chunk (one warp, one bit per token).
constexpr int kChunk = 32;
// One-kernel grouping: at most this many blocks (all resident at once), each of
// at most kGroupMaxCpb chunks; larger T takes the three-kernel grouping.
constexpr int kGroupMaxBlocks = 64;
constexpr int kGroupMaxCpb = 32;

// Byte offsets of the workspace regions for one layer shape (all 256-aligned).
struct WsLayout {
    size_t err;         // uint32 error word + control words (64 B)
    size_t group_flags; // uint32 [kGroupMaxBlocks] one-kernel grouping: block flags (fixed offset)
    size_t group_agg;   // int32 [kGroupMaxBlocks * E] one-kernel grouping: block counts
    size_t counts;      // int32 [E]
    size_t offsets;     // int32 [E+1]
    size_t tile_base;   // int32 [E+1]
    size_t totals;      // int32 [E]   per-expert recount (grouping)
    size_t chunk_base;  // int32 [E * nchunks]
    size_t rank;        // int32 [R]
    size_t perm_token;  // int32 [R]
    size_t perm_slot;   // int32 [R]
    size_t row_of_slot; // int32 [R]
    size_t topk_idx;    // int32 [R]
    size_t topk_w;      // fp32  [R]
    size_t tiles;       // int32 [max_tiles][4]
    size_t num_tiles;   // int32 [1]
    size_t grouping_end;// end of the grouping regions (what moe_permute needs)
    size_t dep;         // uint32 [max_tiles] row-tile counters of the fused expert MLP
    size_t xg;          // bf16  [R, d]  gathered rows (CTA-pair gate/up GEMM)
    size_t h;           // bf16  [R, n]
    size_t z;           // bf16  [R, d]
    size_t logits;      // fp32  [T, E] router logits (moe_forward only)
    size_t counts_round;// int32 [E]    Token Rounding counts (rounded layout only)
    size_t row_map;     // int32 [T, E] Token Rounding rows (rounded layout only)
    size_t row_w;       // fp32  [R]    Token Rounding row weights (rounded layout only)
    size_t round_scratch; // Token Rounding candidate keys (rounded layout only)
    size_t tok_rows;    // int32 [T, kTokCap] compact per-token rows (rounded layout only)
    size_t tok_n;       // int32 [T] (rounded layout only)
    size_t total;
    size_t rows;        // row capacity R of the grouped buffers
    int nchunks;
    int max_tiles;
};

// Control words at the start of the workspace (uint32 each): the error word,
// the grouping scan's ticket, the fused expert MLP's launch epoch and
// ticket (its row-tile counters carry the epoch, so they need no clearing),
// and the router backward's column-sum ticket (zeroed by the kernel before it).
enum : int { kWordErr = 0, kWordDone = 1, kWordEpoch = 2, kWordTicket = 3, kWordGroupEpoch = 4,
             kWordGroupTicket = 5, kWordColTicket = 6 };

WsLayout ws_layout(int T, int d, int E, int K, int n);
// Layout for the Token Rounding forward: grouped buffers sized for the largest
// rounded row count, plus row_map, row_w and the rounding scratch.
WsLayout ws_layout_rounded(int T, int d, int E, int K, int n);
// Most rows Token Rounding with tile size M can produce.
int64_t round_capacity(int T, int E, int K, int M);
// Workspace bytes the rounding kernel needs besides its outputs.
size_t round_scratch_bytes(int T, int E);

// ---- launchers (each returns the CUDA error of its launch) -----------------
cudaError_t launch_route(const __nv_bfloat16 *X, const float *Wr, const float *bias, int T,
                         int d, int E, int K, int renorm, float *logits, int32_t *idx, float *w,
                         int32_t *counts, cudaStream_t s);
// Whether launch_route runs one kernel (logits and selection together) for
// this shape and router-weight alignment; otherwise two.
bool route_is_one_kernel(int d, int E, bool wr16);
cudaError_t launch_router_logits(const __nv_bfloat16 *X, const float *Wr, const float *bias,
                                 int T, int d, int E, float *L, cudaStream_t s);
cudaError_t launch_route_logits(const float *logits, int T, int E, int K, int renorm,
                                int32_t *idx, float *w, int32_t *counts, cudaStream_t s);
// Kernels launch_permute enqueues: 1 for T <= 65536 (the one-kernel grouping),
// else 3.
int permute_launch_count(int T);
cudaError_t launch_permute(const int32_t *idx, const int32_t *counts_in, int T, int E, int K,
                           int32_t *offsets, int32_t *perm_token, int32_t *perm_slot,
                           int32_t *row_of_slot, int32_t *tiles, int32_t *num_tiles,
                           const WsLayout &L, char *ws, cudaStream_t s, bool one_kernel = true);
// Rows p < min(R, *rows_used) (rows_used: device, nullable); a token index out of
// range gives a zero row and sets MOE_DEVERR_BAD_EXPERT in *err.
cudaError_t launch_gather_rows(const __nv_bfloat16 *X, const int32_t *perm_token, int T, int R,
                               const int32_t *rows_used, int d, __nv_bfloat16 *Xg, uint32_t *err,
                               cudaStream_t s);
// xg: scratch [R, d] for the gathered rows (used when the CTA-pair kernel runs)
cudaError_t launch_gemm_gate_up(const __nv_bfloat16 *X, const int32_t *perm_token, int T,
                                const __nv_bfloat16 *W1, const __nv_bfloat16 *W3,
                                const int32_t *offsets, int R, int d, int E, int n,
                                __nv_bfloat16 *H, __nv_bfloat16 *xg, uint32_t *err,
                                cudaStream_t s);
// The gate/up GEMM that also stores the pre-activations A1 = x W1[e] and
// A3 = x W3[e] (fp32 [R, n] each) beside H.
cudaError_t launch_gemm_gate_up_train(const __nv_bfloat16 *X, const int32_t *perm_token, int T,
                                      const __nv_bfloat16 *W1, const __nv_bfloat16 *W3,
                                      const int32_t *offsets, int R, int d, int E, int n,
                                      __nv_bfloat16 *H, float *A1, float *A3,
                                      __nv_bfloat16 *xg, uint32_t *err, cudaStream_t s);
// Backward dH: dA1, dA3 [R, n] bf16 and dS [R] fp32 from dY [T, d], W2 and the
// pre-activations; xg: scratch [R, d] bf16 for the gathered dY rows (CTA-pair
// path), dspart: scratch [R, n/32] fp32 (n % 256 == 0).
cudaError_t launch_backward_dh(const __nv_bfloat16 *dY, const int32_t *perm_token, int T,
                               const __nv_bfloat16 *W2, const float *A1,
                               const float *A3, const float *topk_w,
                               const int32_t *perm_slot, const int32_t *offsets, int R, int d,
                               int E, int n, __nv_bfloat16 *dA1, __nv_bfloat16 *dA3,
                               __nv_bfloat16 *xg, float *dspart, float *dS, uint32_t *err,
                               cudaStream_t s);
// Backward dX: dXg [R, d] = dA1 W1[e]^T + dA3 W3[e]^T (bf16), then
// dX [T, d] = sum over k of dXg[row_of_slot[t*K + k]] (the combine).
cudaError_t launch_backward_dx(const __nv_bfloat16 *dA1, const __nv_bfloat16 *dA3,
                               const __nv_bfloat16 *W1, const __nv_bfloat16 *W3,
                               const int32_t *offsets, const int32_t *row_of_slot, int T, int K,
                               int R, int d, int E, int n, __nv_bfloat16 *dXg,
                               __nv_bfloat16 *dX, uint32_t *err, cudaStream_t s);
// Router backward (backward.cu): dL [T, E], dbias [E], dWr [d, E] (fp32) and
// dX [T, d] = bf16(sum_k dXg[row_of_slot[t*K+k]] + dL Wr^T), with `scratch`
// (T * d floats) for the partial sums of dWr and, on the tensor-core path with
// a second scratch region (nullable), the fp32 router share dL Wr^T.
cudaError_t launch_backward_router(const __nv_bfloat16 *X, const float *Wr, const float *L,
                                   const int32_t *idx, const float *dS,
                                   const int32_t *row_of_slot, int T, int d, int E, int K,
                                   int renorm, const __nv_bfloat16 *dXg, float *dL, float *dWr,
                                   float *dbias, float *scratch, char *scratch2,
                                   size_t scratch2_bytes, __nv_bfloat16 *dX, uint32_t *err,
                                   cudaStream_t s);
// dWr partials on the tensor cores: P[c][j][col] = sum over the tokens t of chunk c
// of X[t][j] dLc[t][col] (fp32 [nchunks*d, 2E]), chunk c = tokens offsets[c] ..
// offsets[c+1] - 1 (multiples of 64); dLc [T, 2E] bf16. E % 128 == 0, d % 128 == 0.
// The router's share dXr [T, d] fp32 = (dLh + dLl)(Wrh + Wrl)^T on the tensor
// cores: dLc = [dLh | dLl] [T, 2E], WrA = [Wrh | Wrh], WrB = [Wrl | Wrl] [d, 2E]
// bf16; offsets = {0, T}. 2E % 64 == 0, d % 256 == 0.
cudaError_t launch_router_dx_tc(const __nv_bfloat16 *dLc, const __nv_bfloat16 *WrA,
                                const __nv_bfloat16 *WrB, const int32_t *offsets, int T, int d,
                                int E, float *dXr, uint32_t *err, cudaStream_t s);
cudaError_t launch_router_dwr_tc(const __nv_bfloat16 *X, const __nv_bfloat16 *dLc,
                                 const int32_t *offsets, int T, int d, int E, int nchunks,
                                 float *P, uint32_t *err, cudaStream_t s);
// Rows of src gathered into the padded grouped layout of the weight gradients
// (each expert's rows from a 64-row boundary, zeros after them), optionally
// scaled by w[perm_slot[p]]; poff [E+1] receives (or, offsets_done, holds) the
// padded offsets. dst: [cap, d] with cap >= R + 64*E.
cudaError_t launch_gather_padded(const __nv_bfloat16 *src, const int32_t *perm_token, int T,
                                 const int32_t *offsets, int E, int d, const float *w,
                                 const int32_t *perm_slot, int64_t R, int64_t cap,
                                 int32_t *poff, __nv_bfloat16 *dst, bool offsets_done,
                                 cudaStream_t s);
// Weight gradients: dW1, dW3 [E, d, n] and dW2 [E, n, d] (fp32). pad: scratch
// [R + 64*E, d] bf16, poff: scratch [E+1].
cudaError_t launch_backward_dw(const __nv_bfloat16 *X, const __nv_bfloat16 *dY,
                               const __nv_bfloat16 *H, const __nv_bfloat16 *dA1,
                               const __nv_bfloat16 *dA3, const float *topk_w,
                               const int32_t *perm_token, const int32_t *perm_slot,
                               const int32_t *offsets, int T, int R, int d, int E, int n,
                               float *dW1, float *dW3, float *dW2, __nv_bfloat16 *pad,
                               int32_t *poff, uint32_t *err, cudaStream_t s);
cudaError_t launch_gemm_down(const __nv_bfloat16 *H, const __nv_bfloat16 *W2,
                             const float *topk_w, const int32_t *perm_slot,
                             const int32_t *offsets, int R, int d, int E, int n,
                             __nv_bfloat16 *Z, uint32_t *err, cudaStream_t s);
// Both expert GEMMs, H then Z. With small n (and the single-CTA variant) one
// persistent kernel runs the units of both (see gemm.cu), which needs the
// workspace's control words (err points at them) and dep [max_tiles];
// otherwise launch_gemm_gate_up then launch_gemm_down.
cudaError_t launch_expert_mlp(const __nv_bfloat16 *X, const int32_t *perm_token, int T,
                              const __nv_bfloat16 *W1, const __nv_bfloat16 *W3,
                              const __nv_bfloat16 *W2, const float *topk_w,
                              const int32_t *perm_slot, const int32_t *offsets, int R, int d,
                              int E, int n, __nv_bfloat16 *H, __nv_bfloat16 *Z,
                              __nv_bfloat16 *xg, uint32_t *dep, uint32_t *err, cudaStream_t s);
// Whether launch_expert_mlp runs the fused kernel for this shape, and whether
// the gate/up GEMM runs on CTA pairs (after a separate row gather).
bool use_fused_mlp(int R, int d, int E, int n);
bool gemm_uses_pair(int R, int E);
cudaError_t launch_combine(const __nv_bfloat16 *Z, const int32_t *row_of_slot, int T, int K,
                           int d, __nv_bfloat16 *Y, cudaStream_t s);

// Token Rounding of a top-K routing (rounding.cu): rounded counts, grouped
// offsets, perm_token, row_map [T,E], row weights and the 128-row tile list.
cudaError_t launch_round(const float *L, const int32_t *idx, const int32_t *counts, int T, int E,
                         int K, int M, int renorm, int32_t *counts_out, int32_t *offsets,
                         int32_t *perm_token, int32_t *row_map, float *row_w, int32_t *tiles,
                         int32_t *num_tiles, int32_t *tok_rows, int32_t *tok_n, void *scratch,
                         uint32_t *err, cudaStream_t s);
// Y[t] = sum of Z[row_map[t,e]] over e ascending (rows >= rows_cap are skipped);
// tok_rows [T][kTokCap] / tok_n [T] (nullable) list each token's rows compactly.
cudaError_t launch_combine_rows(const __nv_bfloat16 *Z, const int32_t *row_map,
                                const int32_t *tok_rows, const int32_t *tok_n, int T, int E,
                                int d, int64_t rows_cap, __nv_bfloat16 *Y, cudaStream_t s);

// Layer norm (norm.cu); w32: gamma, beta and their gradients are fp32, else of
// `type`. part: ln_partials(T) * 2 * d floats of scratch. withheld: a row whose copies are
// never issued (the self-test of the bounded waits), or -1.
constexpr int kLnPartials = 384;
int ln_partials(int64_t T);
cudaError_t launch_layernorm_forward(const void *x, int64_t ldx, const void *gamma, const void *beta,
                                     void *y, int64_t ldy, float *mean, float *rstd, int64_t T,
                                     int d, float eps, moe_dtype_t type, bool w32, int64_t withheld,
                                     cudaStream_t s);
cudaError_t launch_layernorm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                      const void *gamma, const float *mean, const float *rstd,
                                      const void *dres, int64_t lddres, void *dx, int64_t lddx,
                                      void *dgamma, void *dbeta, int64_t T, int d,
                                      moe_dtype_t type, bool w32, float *part, int64_t withheld,
                                      cudaStream_t s);
// Residual dropout (dropout.cu); res may be NULL.
cudaError_t launch_dropout(const void *x, int64_t ldx, const void *res, int64_t ldr, void *y,
                           int64_t ldy, int64_t T, int d, uint32_t thr, uint64_t seed,
                           uint64_t offset, const uint64_t *offset_dev, moe_dtype_t type,
                           cudaStream_t s);

// Dense gated feed-forward block (ffn.cu: tiled products; ffn_small.cu: few tokens,
// which stream the weights). f16: fp16, else bf16. The factors F1, F3 of the gate product
// may be NULL; dX may be NULL, and dW1, dW3, dW2 together.
// The weight-streaming kernel takes up to 48 tokens, and up to 64 where the weights are
// at most 2^27: it reads each token's values with every 128 columns of weights, which
// costs large weights more of the SMs' intake than the tiled products' wider tiles.
// Measured, streaming against tiled, in us: 4096 x 14336 16 tokens 70 / 75, 40: 75 / 77,
// 48: 76.5 / 76.6, 64: 80 / 77; 8192 x 4096 64: 54.4 / 54.9; 7168 x 2048 16: 31 / 37, 64:
// 35 / 38; 1024 x 1024 64: 18.5 / 19.9.
constexpr int kFfnStreamTokens = 64;
inline bool ffn_streams(int T, int d, int n) {
    return T <= 48 || (T <= kFfnStreamTokens && 3ll * d * n <= (1ll << 27));
}
constexpr int kFfnMaxCtas = 192;       // of one weight-streaming launch
constexpr int kFfnMaxWidth = 1 << 20;  // of d and n
constexpr size_t kFfnTicketOffset = 256;  // workspace: control words, then tickets
constexpr size_t kFfnControlBytes =  // a ticket for each warp of each tile of two products
    kFfnTicketOffset + 2 * (size_t)(kFfnMaxWidth / 128) * 4 * sizeof(uint32_t);
size_t ffn_stream_part_bytes(int T, int d, int n);
// Scratch of the tiled products' joins (part; ticket: counters that are zero between
// launches, 16 for each of up to kFfnMaxCtas cut tiles).
size_t ffn_dense_part_bytes();
cudaError_t launch_ffn_stream(const void *X, const void *W1, const void *W3, const void *W2, int T,
                              int d, int n, int act, bool f16, void *H, void *Y, float *part,
                              uint32_t *ticket, uint32_t *err, cudaStream_t s);
cudaError_t launch_ffn_gate(const void *X, const void *W1, const void *W3, int T, int d, int n,
                            int act, bool f16, void *H, float *F1, float *F3, float4 *part,
                            uint32_t *ticket, uint32_t *err, cudaStream_t s);
cudaError_t launch_ffn_down(const void *H, const void *W2, int T, int d, int n, bool f16, void *Y,
                            float4 *part, uint32_t *ticket, uint32_t *err, cudaStream_t s);
cudaError_t launch_ffn_backward(const void *dY, const void *X, const void *W1, const void *W3,
                                const void *W2, const void *H, const float *F1, const float *F3,
                                int T, int d, int n, bool f16, void *dA1, void *dA3,
                                void *dX, void *dW1, void *dW3, void *dW2, float4 *part,
                                uint32_t *ticket, uint32_t *err, cudaStream_t s);

// A projection, Y = act(X W + bias) + residual (ffn.cu, ffn_small.cu), and what its gradients
// take beside the products (linear.cu). bias, res may be NULL; act: moe_act_t. Y may be res.
struct LinearCall {
    const void *X, *W, *bias, *res;
    void *Y;
    int T, k, n, act;
    bool f16, bias32;
};
// Few tokens stream the weights: up to 16, or 64 where n <= 2048 leaves the tiles so few that they
// are cut into many segments. Measured, streaming against tiled, in us: 14336 x 4096 16 tokens
// 28.9 / 30.9, 32: 30.9 / 30.9, 64: 33.1 / 31.3; 4096 x 4096 32: 18.6 / 18.5, 64: 20.8 / 18.6; 4096
// x 8192 32: 24.7 / 23.4; 2048 x 2728 64: 18.2 / 15.7; 7168 x 2048 16: 14.6 / 20.8, 64: 18.8 / 22.7;
// 8192 x 1024 64: 14.9 / 18.6; 4096 x 128 64: 10.3 / 15.2.
inline bool linear_streams(int T, int n) { return T <= 16 || (T <= kFfnStreamTokens && n <= 2048); }
size_t linear_stream_part_bytes(int T, int k, int n);
cudaError_t launch_linear_stream(const LinearCall &c, float *part, uint32_t *ticket, uint32_t *err,
                                 cudaStream_t s);
// F: act'(X W + bias) in blocks of 32 x 32 (moe_ffn_forward_train), or NULL.
cudaError_t launch_linear_tiled(const LinearCall &c, float *F, float4 *part, uint32_t *ticket, uint32_t *err,
                                cudaStream_t s);
// dX = dA W^T, dW = X^T dA; either may be NULL. With dW, dbias may be given: the sums of
// launch_linear_grad's rows, beside the products: up to 320 rows of them. One warp a CTA adds a column's
// rows one after the other, and with more it ends behind the products: launch_linear_bias takes them.
// The whole backward, beside / by a kernel of its own, in us: 4096 x 1024 x 512 (128 rows) 33.1 / 37.1,
// 8192 x 1024 x 256 (256) 37.1 / 40.0, 16384 x 1024 x 1024 (304) 94.5 / 98.2, 11000 x 1024 x 256 (344)
// 47.9 / 49.2 and x 256 x 256 35.5 / 35.2, 13000 x 1024 x 256 (407) 57.1 / 51.7, 16384 x 2048 x 512 (512)
// 100.7 / 87.6, 40000 x 256 x 256 (1216) 121 / 70.
constexpr int kLinearSumsBeside = 320;
cudaError_t launch_linear_products(const void *dA, const void *X, const void *W, int T, int k, int n, bool f16,
                                   void *dX, void *dW, void *dbias, bool bias32, const float *sums,
                                   float4 *part, uint32_t *ticket, uint32_t *err, cudaStream_t s);
// dA = dY F (F NULL: dY itself, nothing is written) and, unless sums is NULL, the column sums of
// dY F over runs of rows: sums [linear_sum_rows(T, n)][n]. And the sums of those rows alone, of the
// 16-bit type or fp32.
int linear_sum_rows(int T, int n);
cudaError_t launch_linear_grad(const void *dY, const float *F, int T, int n, bool f16, void *dA, float *sums,
                               cudaStream_t s);
cudaError_t launch_linear_bias(const float *sums, int T, int n, bool f16, void *dbias, bool bias32,
                               cudaStream_t s);

// The norms around a block (block_norm.cu, block_norm_forward.cuh, block_norm_backward.cuh); w32: post, pre and their
// gradients are fp32. gate_rows: gate and dgate are [T,d] of `type`, else fp32, one a row.
constexpr int kBlockNormMaxWidth = 16384;
struct Matrix {
    const void *p;
    int64_t ld;
};
struct BlockNormCall {
    Matrix x, b, gate, y, u;
    const void *post, *pre;
    float *r_post, *r_pre;
    int64_t T;
    int d;
    moe_dtype_t type;
    bool w32, gate_rows, post_norm, pre_norm;
    float scale, eps;
    // backward (r_post and r_pre are inputs then); part: block_norm_partials(T) * 2 * d floats
    Matrix dy, du, dx, db, dgate;
    void *dpost, *dpre;
    float *part;
};
// Rows of partial weight sums: one of each block, and blocks come by eights where rows start
// anywhere.
int block_norm_partials(int64_t T);
cudaError_t launch_block_norm_forward(const BlockNormCall &c, int64_t withheld, cudaStream_t s);
cudaError_t launch_block_norm_backward(const BlockNormCall &c, int64_t withheld, cudaStream_t s);
// first, second [d] of wtype (each may be NULL) = the sums of P rows of part [P][2][d].
cudaError_t launch_weight_reduce(const float *part, int P, int d, moe_dtype_t wtype, void *first,
                                 void *second, cudaStream_t s);

constexpr int kMaxRowWidth = 1 << 28;
// Token rows and rows sorted by expert (dispatch.cu). x: by token (the dispatch's input, the
// combine's gradient); z: by sorted row; out: by sorted row, or (x NULL) by token; res, w may
// be NULL.
struct RowArgs {
    const void *x, *z, *res;
    const int32_t *row_of_slot;
    const float *w;
    void *out;
    float *dw;
    int64_t ldx, ldz, ldr, ldo;
    int64_t T, rows;
    int K, d;
    int split;  // warps a token
};
cudaError_t launch_dispatch(const RowArgs &a, moe_dtype_t type, cudaStream_t s);
cudaError_t launch_sum_rows(const RowArgs &a, moe_dtype_t type, cudaStream_t s);
cudaError_t launch_combine_backward(const RowArgs &a, moe_dtype_t type, cudaStream_t s);

// One CTA whose pipeline wait on a barrier nothing arrives at runs out after the
// wait limit (about 1 s) and sets MOE_DEVERR_TIMEOUT in *err.
cudaError_t launch_wait_timeout_selftest(uint32_t *err, cudaStream_t s);

// ---- programmatic dependent launch ------------------------------------------
// Kernels of the path are launched so that each may start (and run the setup
// that touches no global memory) while its predecessor on the stream finishes.
// Every such kernel calls pdl_wait() before its first global-memory access, which
// returns once the predecessor grid has completed and its writes are visible
// (at once for a launch without the attribute), then pdl_trigger(), which lets
// its own dependent be scheduled. A dependent launches only after every CTA of
// its predecessor is resident, so waiting CTAs never block their predecessor.
// MOE_PDL=0 in the environment launches them in plain stream order.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
bool pdl_enabled();

template <typename... KArgs, typename... Args>
inline cudaError_t launch_k(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The same in clusters of two CTAs, which are resident together.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pairs(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A launch whose CTAs wait on one another: cooperative, so that they are resident
// together or not launched at all, whatever else runs on the device. (It starts in
// plain stream order: 2 us later than a programmatic dependent launch.)
template <typename... KArgs, typename... Args>
inline cudaError_t launch_together(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                   cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Streaming multiprocessors of the current device (cached per device).
int sm_count();
// Unique id of the CUDA context current on this thread (never reused, unlike a
// context handle); false when there is none yet or the driver cannot say.
bool current_context_id(unsigned long long *id);
// Raises the kernel's dynamic shared-memory limit to `bytes` in the current
// context. Remembered per (kernel, context), so each context gets it once;
// safe to call from several host threads.
cudaError_t ensure_dynamic_smem(const void *kernel, int bytes);
// MOE_OK when the current device is sm_103 (cached per device), MOE_ERR_ARCH
// otherwise, MOE_ERR_CUDA when the device cannot be queried. Clears a CUDA error
// left pending by an earlier, unrelated call first.
moe_status_t check_arch();

}  // namespace moe
