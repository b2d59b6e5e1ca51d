/*
 * fp8bw_layer.h -- C ABI of the operators that stand around the blockwise-FP8
 * linears of a transformer layer (fp8bw.h), for B200 (sm_100a): what produces
 * a linear's E4M3 input codes, and what turns its weight gradient into an
 * orthogonalised update.
 *
 * The conventions of fp8bw.h hold (device pointers owned by the caller, 16-byte
 * aligned; row-major; asynchronous on `stream`; the current device; status
 * codes; argument errors found before anything is launched; bounded waits),
 * with these differences:
 *   - rows is a token count: any number from 0 to 2^30, odd ones included.
 *     bf16 tensors have exactly `rows` rows. Codes and scales have
 *     rp = 16 * ceil(rows / 16) rows (tokens), so that the GEMMs of fp8bw.h
 *     take them as they are; the codes of rows `rows` .. rp-1 are zero and
 *     their row-wise scales 1. Layouts, with rp for rows, are those of the
 *     quantisers:
 *       q   [rp, cols]   s   [ceil(cols/128)][rp]     1x128 groups
 *       q_t [cols, rp]   s_t [ceil(rp/128)][cols]     128x1 groups, transposed
 *   - cols (and f, n, k) are multiples of 16.
 *   - Values are computed in fp32 and rounded once, to E4M3: the codes are
 *     those of the fp32 value, not of its bf16 rounding. The scale rules are
 *     the quantisers' (the *_pow2 forms: power-of-two scales).
 *   - Outputs must overlap neither an input nor one another.
 *   - A workspace is scratch of the given size that the call uses on `stream`
 *     only: calls that may run at the same time (two streams, two graphs that
 *     replay concurrently) need one each.
 */
#ifndef FP8BW_LAYER_H
#define FP8BW_LAYER_H

#include "fp8bw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual addition and root-mean-square norm, to E4M3 codes:
 *   h = bf16(x + residual)            (h = x when residual is NULL)
 *   rstd[i] = 1 / sqrt(mean_j h[i][j]^2 + eps)
 *   v[i][j] = (h[i][j] * rstd[i]) * gamma[j]             fp32
 *   x, residual : bf16 [rows, cols] (residual may be NULL)
 *   gamma       : [cols], fp32 if gamma_is_f32 != 0, else bf16
 *   h           : bf16 [rows, cols] (out); required with a residual, NULL
 *                 without one
 *   rstd        : fp32 [rows] (out) or NULL; required for q_t
 *   y           : bf16 [rows, cols] (out) or NULL: v rounded to bf16
 *   q, s        : row-wise codes of v (out), both or neither
 *   q_t, s_t    : column-wise codes of v, transposed (out), both or neither
 * cols <= 32768; eps >= 0 (else FP8BW_ERR_SHAPE). The sum of a row's squares is
 * fp32: rows whose Euclidean norm is in [2^-50, 2^64) are right to a few roundings,
 * and down to zero rows for eps >= 2^-100. Rows of 2^64 and more (values around
 * 2^58.5 in all of 2048 columns) have rstd 0; smaller ones than 2^-50 lose bits with
 * a smaller eps, and are not finite where all squares vanish (as a row of zeros is
 * with eps == 0, by the formula).
 * The two products are taken in the order above, or with rstd last where nothing
 * leaves fp32's range on the way; a factor that a group's or a column's values share
 * joins their scale's. */
int fp8bw_rmsnorm_quantize(const uint16_t* x, const uint16_t* residual,
                           const void* gamma, int gamma_is_f32, int64_t rows,
                           int64_t cols, float eps, uint16_t* h, float* rstd,
                           uint16_t* y, uint8_t* q, float* s, uint8_t* q_t,
                           float* s_t, void* stream);
int fp8bw_rmsnorm_quantize_pow2(const uint16_t* x, const uint16_t* residual,
                                const void* gamma, int gamma_is_f32,
                                int64_t rows, int64_t cols, float eps,
                                uint16_t* h, float* rstd, uint16_t* y,
                                uint8_t* q, float* s, uint8_t* q_t, float* s_t,
                                void* stream);

/* Its backward pass. dy is the gradient of v, dres (may be NULL) the one that
 * reaches h directly:
 *   dh = bf16(rstd * (dy*gamma - xh * mean_j(dy*gamma*xh)) + dres),
 *   dgamma[j] = sum_i dy * xh,   xh = h * rstd
 * dh is the gradient of both x and residual.
 *   dy, h, dres : bf16 [rows, cols];  rstd : fp32 [rows]
 *   dh          : bf16 [rows, cols] (out);  dgamma : fp32 [cols] (out)
 *   workspace   : at least fp8bw_rmsnorm_backward_workspace(rows, cols) bytes
 * fp32 throughout: rstd^2 has to be a normal number (rstd in 2^-63 .. 2^63).
 * The sum over rows is taken in a fixed order: equal inputs give equal bits.
 * rows == 0 writes dgamma = 0. */
int64_t fp8bw_rmsnorm_backward_workspace(int64_t rows, int64_t cols);
int fp8bw_rmsnorm_backward(const uint16_t* dy, const uint16_t* h,
                           const float* rstd, const void* gamma,
                           int gamma_is_f32, const uint16_t* dres,
                           int64_t rows, int64_t cols, uint16_t* dh,
                           float* dgamma, void* workspace,
                           int64_t workspace_bytes, void* stream);

/* SiLU-gated product of a fused gate/up projection, to E4M3 codes:
 *   gu = [gate | up] : bf16 [rows, 2f];  a = gate * sigmoid(gate) * up
 *   q, s     : row-wise codes of a [rp, f] (out)
 *   q_t, s_t : column-wise codes of a, transposed (out), both or neither
 * f <= 2^22; fewer than 2^31 tiles of 128 x 128 in [rows, 2f]. */
int fp8bw_swiglu_quantize(const uint16_t* gu, int64_t rows, int64_t f,
                          uint8_t* q, float* s, uint8_t* q_t, float* s_t,
                          void* stream);
int fp8bw_swiglu_quantize_pow2(const uint16_t* gu, int64_t rows, int64_t f,
                               uint8_t* q, float* s, uint8_t* q_t, float* s_t,
                               void* stream);

/* Its backward pass, to E4M3 codes of d = [dgate | dup] (rows x 2f):
 *   dgate = da * up * sg * (1 + gate * (1 - sg)),  dup = da * gate * sg,
 *   sg = sigmoid(gate);   da : bf16 [rows, f]
 *   q [rp, 2f], s [ceil(2f/128)][rp], q_t [2f, rp], s_t [ceil(rp/128)][2f]
 * (all required): the operands of the gate/up linear's dgrad and wgrad. */
int fp8bw_swiglu_backward_quantize(const uint16_t* da, const uint16_t* gu,
                                   int64_t rows, int64_t f, uint8_t* q,
                                   float* s, uint8_t* q_t, float* s_t,
                                   void* stream);
int fp8bw_swiglu_backward_quantize_pow2(const uint16_t* da, const uint16_t* gu,
                                        int64_t rows, int64_t f, uint8_t* q,
                                        float* s, uint8_t* q_t, float* s_t,
                                        void* stream);

/* Orthogonalisation of weight updates by Newton-Schulz products (the update
 * rule of the Muon optimiser), for up to FP8BW_NS_MAX_JOBS matrices of any shapes at
 * once:
 *   X = G / (||G||_F + eps), then `steps` times
 *   X <- a X + b (X X^T) X + c (X X^T)^2 X
 * (grouped on the shorter side; two consecutive steps may be taken as one there).
 * The products' operands are fp16 with fp32 accumulation; X itself is held in 32
 * bits, an fp16 pair (entries below 2^-45 are lost). The polynomial must keep the
 * singular values of X below 4 and those of b A + c A^2 (A = X X^T) below 15,
 * as the usual coefficients (3.4445, -4.7750, 2.0315) do: beyond, fp16
 * overflows and the result is not finite.
 *   jobs      : HOST array of `count` (0..FP8BW_NS_MAX_JOBS) descriptions
 *   g_is_f32  : every g is fp32 (!= 0) or bf16 (0)
 *   steps     : 1..64
 *   workspace : at least fp8bw_newton_schulz_workspace(jobs, count) bytes,
 *               128-byte aligned
 * n and k are multiples of 16, at most 2^17; an empty matrix is a no-op. */
#define FP8BW_NS_MAX_JOBS 8

typedef struct fp8bw_ns_job {
    const void* g;       /* [n, k], fp32 or bf16                             */
    int64_t n, k;
    uint16_t* out;       /* bf16 [n, k]                                      */
} fp8bw_ns_job;

int64_t fp8bw_newton_schulz_workspace(const fp8bw_ns_job* jobs, int count);
int fp8bw_newton_schulz(const fp8bw_ns_job* jobs, int count, int g_is_f32,
                        int steps, float a, float b, float c, float eps,
                        void* workspace, int64_t workspace_bytes,
                        void* stream);

/* fp8bw_check_device_error for the operators of this header. */
int fp8bw_layer_check_device_error(void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP8BW_LAYER_H */
