/*
 * ionn.h -- C ABI of the integer-only training-step library for AMD MI355X
 * (gfx950).  Library file: libionn.so.
 *
 * What the calls compute is defined by these pages (cited by title and
 * section):
 *  [TI]   "Integer On-Device Training: Overview" (TI C2000 MCU-AI guide):
 *         section 3 "The NITI Algorithm" -> "The Solution: Dynamic Shifts"
 *         (steps 1-5, delta propagation with target_bits = 7); section 4
 *         (layers fill an activation buffer and a ReLU mask in the forward
 *         pass; the backward pass reads the loss delta and updates weights);
 *         section 7 (Conv2D, Conv2D+ReLU, Linear, Linear+ReLU layers; grouped
 *         and dilated convolutions are refused).
 *  [DFP]  "Mixed Precision Training of Convolutional Neural Networks using
 *         Integer Operations" (source-linked summary): section 3 (DFP-P
 *         tensor = integers + one shared signed 8-bit exponent), 3.1 (product
 *         exponent Ea+Eb; down-conversion by a right shift Rs), 4 "Handling
 *         overflows" (short int32 partial chains).
 *  [APT]  "Adaptive Precision Training for Resource Constrained Devices"
 *         (quantisation underflow, epsilon; the Gavg metric, Equation 4).
 *  [TGR]  "Compilation Pipeline" (TiGrIS): fully-connected weight index
 *         W[oc*IC + ic]; NHWC activations.
 *
 * Conventions for every call:
 *  - Tensors are DEVICE pointers, allocated and owned by the caller; the
 *    library keeps no pointer after a call returns and allocates nothing.
 *  - Row-major layouts.  Linear: X[B][IN], W[OUT][IN], Y[B][OUT].  Conv:
 *    NHWC activations, OHWI weights W[Cout][KH][KW][Cin], cross-correlation.
 *  - int8 x int8 products accumulate in int32 modulo 2^32 (two's-complement
 *    wrap), so results do not depend on summation order.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Every call checks
 *    its arguments on the host, then enqueues its kernels on `stream` and
 *    returns without waiting.  On any error nothing is enqueued.
 *  - absmax arguments are device uint32 scalars that the call MAX-COMBINES
 *    into: *absmax = max(*absmax, max |t|) with |INT32_MIN| = 2^31.  Set them
 *    to 0 first (ionn_fill_u32) when a fresh maximum is wanted.  Several
 *    calls may accumulate into one scalar (e.g. a tensor produced in parts).
 *  - Shifts and exponents produced by a call are written to device memory, so
 *    consecutive calls chain on the stream without a host round trip.
 *  - Return value: IONN_OK (0) or one of the IONN_ERR_* codes below;
 *    ionn_last_error() gives a message for the calling thread's last error.
 */
#ifndef IONN_H
#define IONN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    IONN_OK = 0,
    IONN_ERR_ARG = 1,    /* a required pointer is NULL, or a flag is invalid   */
    IONN_ERR_SHAPE = 2,  /* a size is negative, too large, or inconsistent     */
    IONN_ERR_RANGE = 3,  /* target_bits, mu_weight, chunk ... out of range     */
    IONN_ERR_ALIGN = 4,  /* a pointer lacks the alignment the call documents   */
    IONN_ERR_UNSUPPORTED = 5, /* geometry outside what the library implements */
    IONN_ERR_HIP = 6,    /* a HIP runtime call or kernel launch failed         */
    IONN_ERR_WORKSPACE = 7 /* workspace NULL or smaller than required          */
};

/* Message for a status code (static string). */
const char *ionn_status_str(int status);
/* Message describing the calling thread's most recent error ("" if none). */
const char *ionn_last_error(void);
/* Library version, e.g. "ionn 0.1.0 gfx950". */
const char *ionn_version(void);

/* ------------------------------------------------------------------------ */
/* Small helpers.                                                            */
/* ------------------------------------------------------------------------ */

/* dst[0..n) = value.  A kernel, not hipMemset, so it is safe inside captured
 * HIP graphs.  n >= 0. */
int ionn_fill_u32(uint32_t *dst, int64_t n, uint32_t value, void *stream);

/* [TI] step 1, "max_val = max(|G|)": max-combines max |x[j]| over j < n into
 * *absmax.  n >= 0 (n = 0 leaves *absmax unchanged). */
int ionn_absmax_i32(const int32_t *x, int64_t n, uint32_t *absmax, void *stream);

/* ------------------------------------------------------------------------ */
/* Linear layer contractions (int8 x int8 -> int32).                         */
/* Sizes: B, IN, OUT >= 0 and each < 2^31.                                   */
/* ------------------------------------------------------------------------ */

/* Forward product of a Linear layer ([TI] section 7, [TGR] FC index):
 *   Y[b][o] = sum_i X[b][i] * W[o][i].
 * X: int8 [B][IN]; W: int8 [OUT][IN]; Y: int32 [B][OUT] (written).
 * absmax_Y (nullable): max-combined with max |Y|. */
int int_linear_fwd(const int8_t *X, const int8_t *W, int32_t *Y, int64_t B,
                   int64_t IN, int64_t OUT, uint32_t *absmax_Y, void *stream);

/* Delta propagation (dgrad) of a Linear layer ([TI] section 3, delta
 * propagation; section 4, ReLU mask):
 *   dX[b][i] = sum_o dY[b][o] * W[o][i],
 * then, if relu_act is not NULL, dX[b][i] = 0 wherever relu_act[b][i] <= 0
 * (relu_act is the int8 [B][IN] output of the layer below, whose ReLU mask is
 * "activation > 0").  dY: int8 [B][OUT]; W: int8 [OUT][IN]; dX: int32
 * [B][IN] (written).  absmax_dX (nullable) sees the masked values. */
int int_linear_dgrad(const int8_t *dY, const int8_t *W, const int8_t *relu_act,
                     int32_t *dX, int64_t B, int64_t IN, int64_t OUT,
                     uint32_t *absmax_dX, void *stream);

/* Weight gradient of a Linear layer, the tensor G of [TI] section 3:
 *   G[o][i] = sum_b dY[b][o] * X[b][i].
 * dY: int8 [B][OUT]; X: int8 [B][IN]; G: int32 [OUT][IN] (written).
 * absmax_G (nullable): max-combined with max |G|. */
int int_linear_wgrad(const int8_t *dY, const int8_t *X, int32_t *G, int64_t B,
                     int64_t IN, int64_t OUT, uint32_t *absmax_G, void *stream);

/* The same weight gradient with a caller-provided workspace, for a small G
 * over a long batch (G within 32 blocks of 32 x 32, between 2 and 256 per
 * side, B >= 4096): each range of the batch leaves its partial G in the workspace
 * and one pass sums them (modulo 2^32, so the result is the one above bit
 * for bit) and takes the max, instead of adding into a cleared G with
 * atomics.  int_linear_wgrad_workspace_bytes gives the bytes needed (0 when
 * the shape does not take this path; then, or with dY / X not 4-byte
 * aligned, the call is int_linear_wgrad).  workspace: device, 4-byte
 * aligned, at least that many bytes, else IONN_ERR_WORKSPACE. */
size_t int_linear_wgrad_workspace_bytes(int64_t B, int64_t IN, int64_t OUT);
int int_linear_wgrad_ws(const int8_t *dY, const int8_t *X, int32_t *G, int64_t B,
                        int64_t IN, int64_t OUT, uint32_t *absmax_G, void *workspace,
                        size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------ */
/* NITI quantiser and update ([TI] section 3, steps 1-5).                    */
/* ------------------------------------------------------------------------ */

/* Requantise an int32 tensor to int8 with one dynamic per-tensor shift:
 *   m  = *absmax (device; the caller has max-combined max |acc| into it);
 *   s  = max(0, bitlen(m) - target_bits)            (bitlen = ceil(log2(m+1)))
 *   out[j] = sat8(rhu(acc[j], s)), then max(out, 0) if relu != 0,
 * where rhu(x, s) = floor((x + 2^(s-1)) / 2^s) ("round-half-up", ties toward
 * +infinity) and sat8 clamps to [-128, 127].  target_bits = 7 is the delta
 * propagation setting.  shift_out (nullable, device int32) receives s.
 * n >= 0; target_bits in [1, 31]; relu in {0, 1}. */
int niti_quantize(const int32_t *acc, int64_t n, const uint32_t *absmax,
                  int target_bits, int relu, int8_t *out, int32_t *shift_out,
                  void *stream);

/* NITI weight update, in place on W:
 *   s  = max(0, bitlen(*absmax) - target_bits)
 *   ws = max(0, s - mu_weight)
 *   Gq = rhu(G[j], s)          (int32, not clamped)
 *   d  = rhu(Gq, ws)
 *   W[j] = sat8(W[j] - d)
 * Every W element is rewritten.  shifts_out (nullable, device int32[2])
 * receives {s, ws}.  gq_out (nullable, device int32[n]) receives Gq.
 * n >= 0; target_bits in [1, 31]; mu_weight in [0, 31]. */
int niti_quantize_update(const int32_t *G, int64_t n, const uint32_t *absmax,
                         int target_bits, int mu_weight, int8_t *W,
                         int32_t *shifts_out, int32_t *gq_out, void *stream);

/* One whole NITI step of a small Linear layer in one launch, for layers of
 * microcontroller size ([TI] section 3 "The NITI Algorithm", steps 1-5, and
 * the weight index of the TiGrIS "Compilation Pipeline" page), in this order:
 *   Y[b][o]  = sum_i X[b][i] * W[o][i]                  (int32)
 *   dX[b][i] = sum_o dY[b][o] * W[o][i]                 (int32, W before the update)
 *   delta    = sat8(rhu(dX, s_d)), s_d = max(0, bitlen(max |dX|) - tb_d)
 *   G[o][i]  = sum_b dY[b][o] * X[b][i]                 (int32)
 *   s = max(0, bitlen(max |G|) - tb_w), ws = max(0, s - mu_weight),
 *   Gq = rhu(G, s), W[o][i] = sat8(W[o][i] - rhu(Gq, ws)) (in place).
 * The same results as int_linear_fwd, int_linear_dgrad, niti_quantize,
 * int_linear_wgrad and niti_quantize_update in sequence, from one
 * workgroup.  Device buffers: X int8 [B][IN]; W int8 [OUT][IN] (read, then
 * rewritten); dY int8 [B][OUT]; Y int32 [B][OUT], dX int32 [B][IN], delta
 * int8 [B][IN], G int32 [OUT][IN], gq (nullable) int32 [OUT][IN], all
 * written; maxima uint32[3] receives max |Y|, max |dX|, max |G| (written,
 * not max-combined: nothing needs clearing first); shifts int32[3] receives
 * s_d, s, ws.  Requires int_linear_step_small_fits(B, IN, OUT): X, W and dY
 * together within 32 KiB (IONN_ERR_SHAPE otherwise); tb_w, tb_d in [1, 31];
 * mu_weight in [0, 31]. */
int int_linear_step_small(const int8_t *X, int8_t *W, const int8_t *dY,
                          int64_t B, int64_t IN, int64_t OUT, int tb_w,
                          int mu_weight, int tb_d, int32_t *Y, int32_t *dX,
                          int8_t *delta, int32_t *G, int32_t *gq,
                          uint32_t *maxima, int32_t *shifts, void *stream);

/* 1 when int_linear_step_small takes a layer of this shape (B, IN, OUT >= 1
 * and B*IN + OUT*IN + B*OUT <= 32768), else 0. */
int int_linear_step_small_fits(int64_t B, int64_t IN, int64_t OUT);

/* niti_quantize_update, which also sets clear[0 .. n_clear) to 0 (device
 * uint32, 0 <= n_clear <= 256, must not overlap *absmax).  For a training
 * loop that alternates two sets of max-combined scalars: the update of one
 * step clears the set the next step max-combines into, so no separate fill
 * precedes each step (a HIP graph then captures an even number of steps).
 * Nothing reads clear in the call; the clearing happens before the kernel
 * ends, so the next call on the stream sees zeros. */
int niti_quantize_update_clear(const int32_t *G, int64_t n,
                               const uint32_t *absmax, int target_bits,
                               int mu_weight, int8_t *W, int32_t *shifts_out,
                               int32_t *gq_out, uint32_t *clear,
                               int64_t n_clear, void *stream);

/* Output error of a classifier whose loss pushes the true class toward a
 * target magnitude and the others toward 0 ([TI] sections 4 and 6.2: user
 * loss writes the delta for the backward pass):
 *   e[b][c] = (c == labels[b] ? target_mag : 0) - out[b][c].
 * out: int8 [B][C]; labels: int32 [B] (values outside [0, C) match no class);
 * e: int32 [B][C] (written); absmax_e (nullable) max-combined.
 * target_mag in [-128, 127]. */
int int_output_error(const int8_t *out, const int32_t *labels, int64_t B,
                     int64_t C, int target_mag, int32_t *e, uint32_t *absmax_e,
                     void *stream);

/* ------------------------------------------------------------------------ */
/* Conv2D contractions ([TI] section 7), NHWC / OHWI, cross-correlation.     */
/* Geometry: stride 1, dilation 1, groups 1 (anything else returns           */
/* IONN_ERR_UNSUPPORTED; the page's export refuses grouped and dilated       */
/* convolutions outright); KH, KW in [1, 1024]; zero padding P = pad in     */
/* [0, 1024] (else IONN_ERR_RANGE).  Output Ho = H + 2P - KH + 1,             */
/* Wo = W + 2P - KW + 1.  N, H, W, Cin, Cout >= 0; every tensor must hold    */
/* fewer than 2^31 elements.  3x3 / pad 1 with Cin and Cout multiples of 16  */
/* runs on the matrix cores and needs 16-byte aligned tensors; other         */
/* geometries (e.g. the page's 16 x 2 "valid" filter bank) run on direct     */
/* kernels and need 4-byte aligned int32 tensors only.                       */
/* ------------------------------------------------------------------------ */

typedef struct ionn_conv_desc {
    int64_t N, H, W, Cin, Cout;
    int32_t KH, KW, stride, pad, dilation, groups;
} ionn_conv_desc;

/* Y[n,h,w,co] = sum_{kh,kw,ci} X[n,h+kh-P,w+kw-P,ci] * Wt[co,kh,kw,ci]
 * (zero outside the image).  X: int8 [N][H][W][Cin]; Wt: int8
 * [Cout][KH][KW][Cin]; Y: int32 [N][Ho][Wo][Cout] (written). */
int int_conv_fwd(const int8_t *X, const int8_t *Wt, int32_t *Y,
                 const ionn_conv_desc *desc, uint32_t *absmax_Y, void *stream);

/* dX[n,h,w,ci] = sum_{kh,kw,co} dY[n,h-kh+P,w-kw+P,co] * Wt[co,kh,kw,ci]
 * (terms outside dY dropped).  dY: int8 [N][Ho][Wo][Cout]; dX: int32
 * [N][H][W][Cin] (written). */
int int_conv_dgrad(const int8_t *dY, const int8_t *Wt, int32_t *dX,
                   const ionn_conv_desc *desc, uint32_t *absmax_dX,
                   void *stream);

/* The forward contraction with the NITI requantisation of its result fused
 * in ("Integer On-Device Training: Overview", section 3, steps 1-3 and the
 * ReLU of the Conv2D layer, section 7): Y8 = sat8(rhu(Y, s)), then
 * max(Y8, 0) if relu, with s = max(0, bitlen(max|Y|) - target_bits) and Y
 * the int32 sum of int_conv_fwd.  Y is never stored.
 *  - With a workspace (int_conv_requant_workspace_bytes(desc) bytes, 16-byte
 *    aligned, clobbered; IONN_ERR_WORKSPACE if smaller) and target_bits <= 7:
 *    one contraction pass stores, per block of 32 pixels x 64 channels,
 *    f = asr(Y, s_b) as int8 with the block's own shift s_b (it always fits
 *    int8) and bit s_b - 1 of every Y (its rounding bit) in the workspace;
 *    a streaming pass over Y8 then applies the tensor's shift s >= s_b:
 *    rhu(Y, s) = f + bit when s = s_b, rhu(f, s - s_b) otherwise.  Y8 must
 *    then be 16-byte aligned.
 *  - Without one (workspace NULL), or with target_bits > 7: the contraction
 *    runs twice, first for max|Y| only, then for the int8 output.
 * Same bits either way.  Y8: int8 [N][H][W][Cout] (written).  absmax_Y
 * (device, 4-byte aligned, required): must hold 0 on entry (ionn_fill_u32);
 * receives max|Y|.  shift_out (nullable, device): receives s.  Only 3x3 /
 * stride 1 / pad 1 with 64 input and 64 output channels and a width whose
 * halo fits (as the int32 fast path); other geometries return
 * IONN_ERR_UNSUPPORTED and take int_conv_fwd and niti_quantize.  X and Wt
 * 16-byte aligned, Y8 4-byte aligned. */
size_t int_conv_requant_workspace_bytes(const ionn_conv_desc *desc);
int int_conv_fwd_requant(const int8_t *X, const int8_t *Wt, int8_t *Y8,
                         const ionn_conv_desc *desc, int target_bits, int relu,
                         uint32_t *absmax_Y, int32_t *shift_out,
                         void *workspace, size_t workspace_bytes, void *stream);

/* The same for delta propagation (section 3, the propagated-delta note:
 * target_bits = 7): dX8 = sat8(rhu(dX, s)) with dX the int32 sum of
 * int_conv_dgrad, never stored; one pass plus the streaming pass with a
 * workspace, two contraction passes without. */
int int_conv_dgrad_requant(const int8_t *dY, const int8_t *Wt, int8_t *dX8,
                           const ionn_conv_desc *desc, int target_bits,
                           uint32_t *absmax_dX, int32_t *shift_out,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Device workspace (bytes) that lets int_conv_wgrad take its fast path for
 * this geometry: for 64 input and 64 output channels (3x3, W up to about
 * 100), one partial G per compute unit; for a
 * full-row-window filter (no padding, KW = W, KH*W*Cin a multiple of 4, at
 * most 8 output channels), one partial G per workgroup (at most 1024).  0
 * when the geometry has no fast path (the call then needs no workspace). */
size_t int_conv_wgrad_workspace_bytes(const ionn_conv_desc *desc);

/* G[co,kh,kw,ci] = sum_{n,h,w} dY[n,h,w,co] * X[n,h+kh-P,w+kw-P,ci] over the
 * output positions (h, w) < (Ho, Wo).  G: int32 [Cout][KH][KW][Cin] (written).  workspace (nullable, device,
 * 16-byte aligned, ws_bytes long, owned by the caller, clobbered): with at
 * least int_conv_wgrad_workspace_bytes(desc) bytes, the gradient is
 * computed as per-compute-unit partial sums reduced in two passes; without
 * it, by a split-K product with integer atomics.  Same bits either way. */
int int_conv_wgrad(const int8_t *dY, const int8_t *X, int32_t *G,
                   const ionn_conv_desc *desc, uint32_t *absmax_G,
                   void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------ */
/* DFP-16 shared-exponent contractions ([DFP] sections 3, 3.1, 4).           */
/*                                                                            */
/* A DFP-16 tensor is int16 mantissas I plus one shared exponent E (value     */
/* I * 2^E); E is a device int32 scalar that must lie in [-128, 127].  Each   */
/* contraction multiplies int16 x int16 -> int32 and sums the reduction in    */
/* chunks of `chunk` terms (the last chunk may be shorter).  Overflow         */
/* management: each chunk's int32 partial p_c is shifted down by              */
/* r = ceil(log2(number of chunks)) (0 for one chunk) with round-half-up      */
/* before the chunks are summed, acc = sum_c rhu(p_c, r) (int32).  Adaptive  */
/* down-conversion: Rs = max(0, bitlen(max |acc|) - 15),                      */
/* out = sat16(rhu(acc, Rs)), E_out = Ea + Eb + r + Rs.  If E_out leaves the  */
/* signed 8-bit range the output exponent is still written and the device     */
/* status word (status_out, nullable int32) is set to 1, else 0.              */
/*                                                                            */
/* Sizes: M, K, N >= 1, every tensor below 2^31 elements; chunk must be 64;  */
/* the int16 output must be 16-byte aligned.  `workspace` is device memory of */
/* at least dfp16_workspace_bytes(M, K, N, which) bytes, 256-byte aligned;    */
/* its contents on entry are ignored (it holds the int32 accumulator, the     */
/* max-abs scalar and, for dgrad/wgrad, K-major copies of the operands).      */
/* ------------------------------------------------------------------------ */

enum { IONN_DFP16_FWD = 0, IONN_DFP16_DGRAD = 1, IONN_DFP16_WGRAD = 2 };

size_t dfp16_workspace_bytes(int64_t M, int64_t K, int64_t N, int which);

/* Y[M][N] = X[M][K] . W[N][K]^T, reduced over K. */
int dfp16_gemm_fwd(const int16_t *X, const int32_t *eX, const int16_t *W,
                   const int32_t *eW, int16_t *Y, int32_t *eY, int64_t M,
                   int64_t K, int64_t N, int chunk, void *workspace,
                   size_t workspace_bytes, int32_t *status_out, void *stream);

/* dX[M][K] = dY[M][N] . W[N][K], reduced over N. */
int dfp16_gemm_dgrad(const int16_t *dY, const int32_t *edY, const int16_t *W,
                     const int32_t *eW, int16_t *dX, int32_t *edX, int64_t M,
                     int64_t K, int64_t N, int chunk, void *workspace,
                     size_t workspace_bytes, int32_t *status_out,
                     void *stream);

/* G[N][K] = dY[M][N]^T . X[M][K], reduced over M. */
int dfp16_gemm_wgrad(const int16_t *dY, const int32_t *edY, const int16_t *X,
                     const int32_t *eX, int16_t *G, int32_t *eG, int64_t M,
                     int64_t K, int64_t N, int chunk, void *workspace,
                     size_t workspace_bytes, int32_t *status_out,
                     void *stream);

/* Gavg of a layer ([APT] Equation 4): the mean gradient magnitude over the
 * layer's n parameters relative to the weights' resolution epsilon = 2^eW:
 *   gavg = (sum_j |G[j]| / n) * 2^(eG - eW),
 * the sum exact in int64, the division and scaling in IEEE double.
 * G: int16 [n]; eG, eW: device int32; gavg_out: device double (written).
 * n >= 1. */
int dfp16_gavg(const int16_t *G, const int32_t *eG, const int32_t *eW,
               int64_t n, double *gavg_out, void *stream);

/* ------------------------------------------------------------------------ */
/* DFP as the DFP page runs it ([DFP] 3.1: float -> DFP conversion with the   */
/* shared exponent from the exponent of the absolute maximum; 4 "Handling    */
/* overflows": int32 partials of short chains converted to FP32, scaled by    */
/* 2^(E_inp + E_wt) and accumulated into an FP32 output, the input shifted by */
/* one bit; 3: Blocked-DFP, several exponents per tensor; 4: the operations   */
/* around the integer kernels, the weight update among them, in floating      */
/* point).  Exponents are device int32.                                       */
/* ------------------------------------------------------------------------ */

/* The FP32-partial contractions: the roles and layouts of dfp16_gemm_*, with
 * an FP32 output instead of the down-converted DFP-16 one.  Per output:
 *   A' = rhu(A, input_shift)   (A is the data operand: X for fwd, dY for
 *                               dgrad and wgrad; input_shift 0 or 1)
 *   p_c = the 64-term chunk partials of A' . B   (int32, modulo 2^32)
 *   the chunks fall into S consecutive ranges, range s covering chunks
 *   [floor(n_c s / S), floor(n_c (s + 1) / S)); each range is summed in FP32
 *   in chunk order starting from 0 (every float(p_c) and every addition
 *   rounded to nearest even), the range sums are added in order to 0, and
 *   out = fl(total * 2^(eA + input_shift + eB)) with one rounding.
 * S = nsplit, or dfp16_f32_splits(M, K, N, which) when nsplit = 0 (a
 * function of the shape alone); 1 <= nsplit <= n_c.  The order is part of
 * the result: the same S gives the same bits on any path.  out: float,
 * 16-byte aligned.  workspace: dfp16_f32_workspace_bytes(M, K, N, which,
 * nsplit) bytes, 256-byte aligned (split partials, operand transposes). */
int dfp16_f32_splits(int64_t M, int64_t K, int64_t N, int which);
size_t dfp16_f32_workspace_bytes(int64_t M, int64_t K, int64_t N, int which,
                                 int nsplit);
int dfp16_gemm_fwd_f32(const int16_t *X, const int32_t *eX, const int16_t *W,
                       const int32_t *eW, float *Y, int64_t M, int64_t K,
                       int64_t N, int input_shift, int nsplit, void *workspace,
                       size_t workspace_bytes, void *stream);
int dfp16_gemm_dgrad_f32(const int16_t *dY, const int32_t *edY,
                         const int16_t *W, const int32_t *eW, float *dX,
                         int64_t M, int64_t K, int64_t N, int input_shift,
                         int nsplit, void *workspace, size_t workspace_bytes,
                         void *stream);
int dfp16_gemm_wgrad_f32(const int16_t *dY, const int32_t *edY,
                         const int16_t *X, const int32_t *eX, float *G,
                         int64_t M, int64_t K, int64_t N, int input_shift,
                         int nsplit, void *workspace, size_t workspace_bytes,
                         void *stream);

/* The forward contraction on Blocked-DFP operands whose blocks are the
 * 64-term chunks: X [M][K] with exponents eX[m * nch + c], W [N][K] with
 * eW[n * nch + c] (device int32, nch = ceil(K / 64); dfp_from_f32_blocked
 * with B = 64 writes this layout).  Each chunk's term is scaled on its own,
 * t_c = fl(float(p_c) * 2^(eX[m][c] + input_shift + eW[n][c])) (one
 * rounding), and the terms are summed in the order of dfp16_gemm_fwd_f32;
 * the output is not scaled again.  Workspace as dfp16_gemm_fwd_f32. */
int dfp16_gemm_fwd_f32_blocked(const int16_t *X, const int32_t *eX,
                               const int16_t *W, const int32_t *eW, float *Y,
                               int64_t M, int64_t K, int64_t N, int input_shift,
                               int nsplit, void *workspace,
                               size_t workspace_bytes, void *stream);

/* Workspace bytes of dfp_from_f32 and dfp16_sgd_update (4-byte aligned). */
size_t dfp_convert_workspace_bytes(void);

/* FP32 -> DFP-P, P in [2, 16]: max |x| = f * 2^q (f in [1, 2)) gives
 * E = q - (P - 2) (0 for an all-zero x) and out = sat_P(round_to_nearest_even
 * (x / 2^E)).  x: float [n], 16-byte aligned; out: int16 [n], 8-byte aligned;
 * e_out: device int32; status_out (nullable): 0, 1 when E leaves the signed
 * 8-bit range (E still written), 2 when x holds a NaN or infinity (outputs
 * then unspecified). */
int dfp_from_f32(const float *x, int64_t n, int P, int16_t *out,
                 int32_t *e_out, int32_t *status_out, void *workspace,
                 size_t workspace_bytes, void *stream);

/* DFP -> FP32: out = fl(I * 2^e), one rounding (exact for normal results). */
int dfp_to_f32(const int16_t *I, int64_t n, const int32_t *e, float *out,
               void *stream);

/* Blocked-DFP: x [rows][K] float; every row is cut into blocks of B values
 * (the last one shorter when B does not divide K) and each block is
 * converted as dfp_from_f32 does with its own exponent,
 * e_out[r * ceil(K / B) + b].  status_out (nullable): the largest status of
 * any block. */
int dfp_from_f32_blocked(const float *x, int64_t rows, int64_t K, int B, int P,
                         int16_t *out, int32_t *e_out, int32_t *status_out,
                         void *stream);

/* The weight update of the DFP pipeline: FP32 master weights
 * W32 = fl(W32 - fl(lr * G32)) (two roundings, never fused), then their
 * DFP-16 copy W16 / eW (as dfp_from_f32 with P = 16) for the next forward.
 * W32, G32: float [n], 16-byte aligned; W16: int16 [n], 8-byte aligned. */
int dfp16_sgd_update(float *W32, const float *G32, int64_t n, float lr,
                     int16_t *W16, int32_t *eW, int32_t *status_out,
                     void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------ */
/* Per-channel offsets (bias) and the static OSS requantisation ([TI]        */
/* section 7: every layer carries mutable int32 offsets, updated by the      */
/* backward pass, and per-filter right shifts k with multipliers mult;       */
/* section 8, PC-side Step 2: the chain Add(offset) -> Mul(scale1) ->        */
/* Mul(scale2) -> Floor -> Clip).  Channels are the last dimension: C        */
/* output channels of a Linear layer or of an NHWC convolution output, with  */
/* M = rows (batch, times pixels for a convolution).                         */
/* ------------------------------------------------------------------------ */

/* out[m][c] = clip(floor(t * mult[c] / 2^k[c]), lo, 127),
 *   t = acc[m][c] + offset[c] modulo 2^32 (the int32 accumulator's add),
 *   the product exact in 64 bits, lo = 0 if relu (the *_RELU layer types)
 *   else -128.
 * acc: int32 [M][C]; offset, mult: int32 [C]; k: int8 [C], each in [0, 62]
 * (other values give unspecified outputs, no fault); out: int8 [M][C]
 * (written).  M, C >= 0, M * C < 2^31; relu in {0, 1}. */
int ionn_oss_requant(const int32_t *acc, const int32_t *offset,
                     const int32_t *mult, const int8_t *k, int64_t M,
                     int64_t C, int relu, int8_t *out, void *stream);

/* Forward of a Linear layer with its offsets and static OSS requantisation
 * in one call: Y[b][o] = oss(sum_i X[b][i] * W[o][i]) with the per-output
 * offset, mult and k of ionn_oss_requant (relu selects the *_RELU clip
 * range).  X: int8 [B][IN]; W: int8 [OUT][IN]; Y: int8 [B][OUT] (written).
 * Tile-aligned shapes (B, IN, OUT multiples of 256, IN > 0) with 16-byte
 * aligned X, W, offset, mult and 4-byte aligned k, Y run as one kernel whose
 * epilogue applies the chain to the int32 accumulators (no int32 tensor
 * reaches memory); other shapes or alignments compute the int32 product in
 * `workspace` (16-byte aligned, int_linear_fwd_oss_workspace_bytes bytes;
 * IONN_ERR_WORKSPACE without it) and then run the OSS pass. */
size_t int_linear_fwd_oss_workspace_bytes(int64_t B, int64_t IN, int64_t OUT);
int int_linear_fwd_oss(const int8_t *X, const int8_t *W, const int32_t *offset,
                       const int32_t *mult, const int8_t *k, int relu,
                       int8_t *Y, int64_t B, int64_t IN, int64_t OUT,
                       void *workspace, size_t workspace_bytes, void *stream);

/* Gradient of the offsets: gb[c] = sum_m d[m][c] modulo 2^32, over the int8
 * output error d[M][C] that also feeds dgrad and wgrad.  gb: int32 [C],
 * overwritten.  The row ranges' sums pass through `workspace` (4-byte
 * aligned, ionn_bias_grad_workspace_bytes(M, C) bytes; IONN_ERR_WORKSPACE
 * when NULL or smaller, except for M = 0).  M, C >= 0, M * C < 2^31. */
size_t ionn_bias_grad_workspace_bytes(int64_t M, int64_t C);
int ionn_bias_grad(const int8_t *d, int64_t M, int64_t C, int32_t *gb,
                   void *workspace, size_t workspace_bytes, void *stream);

/* ionn_bias_grad for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same result, with the row-range sums held in a 2 MiB device array of
 * the library instead of a caller workspace.  Allocates nothing and calls
 * no allocating routine; each GPU the library runs on holds one such array
 * until the process ends.  Shapes whose sums need more than 2 MiB
 * (ionn_bias_grad_workspace_bytes(M, C) > 2 MiB) return IONN_ERR_SHAPE and
 * enqueue nothing.  All calls on one GPU share its array: calls that
 * overlap on one GPU (two streams, two threads) race and give unspecified
 * gb; calls ordered on a stream are independent (every entry a call reads
 * it has written first).  The stream's device must be the current device or
 * the stream must belong to it; the array's address is looked up once per
 * device (IONN_ERR_HIP if that lookup fails). */
int ionn_bias_grad_noalloc(const int8_t *d, int64_t M, int64_t C, int32_t *gb,
                           void *stream);

/* NITI update of int32 parameters (the offsets), in place on P: the steps of
 * niti_quantize_update with the last one P[j] = sat32(P[j] - d) (clamped to
 * the int32 range).  *absmax must hold max |G| (e.g. from ionn_absmax_i32).
 * shifts_out (nullable, device int32[2]) receives {s, ws}; gq_out (nullable,
 * device int32[n]) receives Gq.  n >= 0; target_bits in [1, 31]; mu in
 * [0, 31]. */
int niti_quantize_update_i32(const int32_t *G, int64_t n,
                             const uint32_t *absmax, int target_bits, int mu,
                             int32_t *P, int32_t *shifts_out, int32_t *gq_out,
                             void *stream);

/* ------------------------------------------------------------------------ */
/* Model-level driver: the INT_LAYERS forward and backward ([TI] section 7:  */
/* Conv2D, Conv2D+ReLU, Linear and Linear+ReLU layers with int8 weights,     */
/* int32 offsets and per-filter OSS shifts / multipliers; section 8: the OSS */
/* chain and the per-class TARGET_MAG loss; section 3: the NITI updates).    */
/* A sequence of the calls above on one stream; the caller owns the layer    */
/* parameters and one workspace, and the driver allocates nothing.           */
/* ------------------------------------------------------------------------ */

enum {
    IONN_LAYER_CONV2D = 0,
    IONN_LAYER_CONV2D_RELU = 1,
    IONN_LAYER_LINEAR = 2,
    IONN_LAYER_LINEAR_RELU = 3
};
#define IONN_MAX_LAYERS 64

/* One layer.  Per sample it reads H x W x Cin int8 values (NHWC; a Linear
 * layer has H = W = 1 and Cin = its input features) and writes, for a conv,
 * Ho x Wo x Cout (stride 1, zero padding pad, Ho = H + 2 pad - KH + 1,
 * Wo = W + 2 pad - KW + 1), for a Linear, Cout values.  Layer l + 1 must read
 * as many values per sample as layer l writes (a conv output feeds a Linear
 * as one NHWC row).  weight: int8 [Cout][KH][KW][Cin] or [Cout][Cin];
 * offset, mult: int32 [Cout]; k: int8 [Cout] in [0, 62] (the OSS chain of
 * ionn_oss_requant).  weight and offset are device tensors updated in place
 * by ionn_model_backward. */
typedef struct ionn_layer {
    int32_t type;
    int32_t KH, KW, pad;
    int64_t H, W, Cin, Cout;
    int8_t *weight;
    int32_t *offset;
    const int32_t *mult;
    const int8_t *k;
} ionn_layer;

/* Gradient of the MSE loss against per-class target magnitudes ([TI]
 * section 8, PC-side Step 3: TARGET_MAG_CORRECT[c] for the true class,
 * TARGET_MAG_WRONG[c] for the others):
 *   g[b][c] = out[b][c] - (c == labels[b] ? tmc[c] : tmw[c]).
 * out: int8 [B][C]; labels: int32 [B] (values outside [0, C) match no class);
 * tmc, tmw: int8 [C]; g: int32 [B][C] (written); absmax_g (nullable)
 * max-combined. */
int ionn_mse_grad_targets(const int8_t *out, const int32_t *labels, int64_t B,
                          int64_t C, const int8_t *tmc, const int8_t *tmw,
                          int32_t *g, uint32_t *absmax_g, void *stream);

/* d[j] = 0 where act[j] <= 0 (the ReLU mask of [TI] section 4), in place;
 * absmax_d (nullable) is max-combined with the masked values. */
int ionn_relu_mask_i32(int32_t *d, const int8_t *act, int64_t n,
                       uint32_t *absmax_d, void *stream);

/* Device workspace of the driver for this model and batch (0 and an error
 * message on an invalid model).  It holds every layer's activation between
 * ionn_model_forward and ionn_model_backward. */
size_t ionn_model_workspace_bytes(const ionn_layer *layers, int L, int64_t B);

/* Forward of the L layers over the batch X (int8 [B][H0][W0][Cin0]): per
 * layer the int32 contraction, then the OSS chain (ReLU clip for the *_RELU
 * types) into the layer's int8 activation, kept in `workspace` (256-byte
 * aligned, ionn_model_workspace_bytes bytes).  out (nullable): int8
 * [B][last layer's outputs] receives a copy of the last activation. */
int ionn_model_forward(const ionn_layer *layers, int L, const int8_t *X,
                       int64_t B, int8_t *out, void *workspace,
                       size_t workspace_bytes, void *stream);

/* Backward of the last ionn_model_forward on the same X and workspace, and
 * the updates: g = the MSE gradient of the last activation against the
 * per-class targets (ionn_mse_grad_targets), delta = niti_quantize(g,
 * tb_delta); for l = L..1: the offset gradient (ionn_bias_grad over the
 * batch and, for a conv, its output pixels), wgrad, and for l > 1 dgrad with
 * the pre-update weights, masked by layer l-1's activation > 0 when layer
 * l-1 has a ReLU, requantised with tb_delta; then niti_quantize_update of the
 * weights and niti_quantize_update_i32 of the offsets (tb_weight, mu).
 * shifts_out (nullable, device int32[1 + 5 L]): [0] the error's shift, then
 * per layer l at 1 + 5 l: the shift of the delta it propagates (-1 for the
 * first layer, which propagates none), {s, ws} of its weight update and
 * {s, ws} of its offset update.
 * Models of at most 8 layers and 2^22 multiply-adds per step whose layers'
 * operands fit in LDS run the forward and the backward as one workgroup each
 * (same bits); others run the sequence above as separate launches.  Either
 * way the calls are stream-ordered and allocate nothing. */
int ionn_model_backward(const ionn_layer *layers, int L, const int8_t *X,
                        int64_t B, const int32_t *labels, const int8_t *tmc,
                        const int8_t *tmw, int tb_delta, int tb_weight, int mu,
                        void *workspace, size_t workspace_bytes,
                        int32_t *shifts_out, void *stream);

/* ------------------------------------------------------------------------ */
/* Adaptive per-layer precision ([APT]: the weight resolution epsilon of a   */
/* k-bit tensor, Equation 2; the update of Equation 1 on that grid,          */
/* Equation 3; Gavg, Equation 4; the policy of Algorithm 1 applied between   */
/* epochs as Algorithm 2 lays out).                                          */
/*                                                                          */
/* Layer l holds k[l]-bit signed weight mantissas W[l] (int16 storage, or   */
/* int8 through the _mixed calls; the k-bit range [-2^(k-1), 2^(k-1) - 1]) */
/* with one shared exponent e_w[l]: a                                       */
/* weight is m * 2^e_w and one grid step is epsilon = 2^e_w.  k, e_w, the   */
/* gradient exponents e_g and the per-epoch Gavg sums are DEVICE int32 /    */
/* double arrays of L entries, so steps and epochs chain on the stream      */
/* without a host synchronisation.  W, G and n are HOST arrays of L device  */
/* pointers and sizes (2-byte aligned; 16-byte aligned tensors take the     */
/* vector path).  1 <= L <= IONN_MAX_LAYERS, 1 <= n[l] <= 2^36.  A k[l]     */
/* outside [2, 16] is read as the nearest bound.                             */
/* ------------------------------------------------------------------------ */

/* Workspace (bytes, 8-byte aligned) a sampling apt_update needs for these
 * layer sizes; 0 on invalid sizes. */
size_t apt_workspace_bytes(int L, const int64_t *n);

/* One step's update of every layer, in place on W:
 *   W[l][j] = sat_k(W[l][j] - c),  c = rhu(G[l][j], sigma) if sigma >= 0,
 *                                  c = G[l][j] * 2^-sigma   otherwise,
 *   sigma = e_w[l] + lr_shift - e_g[l]
 * i.e. W - lr * g with lr = 2^-lr_shift and g = G * 2^e_g, rounded to the
 * layer's grid (a change under half a step is lost: quantisation underflow).
 * G: int16 [n[l]] (a DFP-16 weight gradient, e.g. from dfp16_gemm_wgrad).
 * lr_shift in [0, 62].  Sampling: when gavg_sum (double [L]) and gavg_count
 * (int32 [L]) are given, every layer's Gavg of this gradient,
 * mean(|G|) * 2^(e_g - e_w) (as dfp16_gavg), is added to gavg_sum[l] and
 * gavg_count[l] grows by one; that needs `workspace`
 * (apt_workspace_bytes(L, n) bytes); both NULL: no sampling, no workspace. */
int apt_update(int L, int16_t *const *W, const int16_t *const *G,
               const int64_t *n, const int32_t *k, const int32_t *e_w,
               const int32_t *e_g, int lr_shift, double *gavg_sum,
               int32_t *gavg_count, void *workspace, size_t workspace_bytes,
               void *stream);

/* Between epochs, per layer (Algorithm 1 on the mean of the epoch's
 * samples, gavg_sum[l] / gavg_count[l]; no samples: no change):
 *   mean < t_min and k < k_max:  k += 1, e_w -= 1, m -> 2m
 *   mean > t_max and k > k_min:  k -= 1, e_w += 1, m -> sat_{k-1}(rhu(m, 1))
 * (the range stays, the grid step halves or doubles); then gavg_sum and
 * gavg_count are cleared.  dk_out (nullable, device int32 [L]) receives
 * each layer's change.  2 <= k_min <= k_max <= 16; t_min <= t_max (t_max
 * may be +inf: never lower).  No workspace. */
int apt_adjust(int L, int16_t *const *W, const int64_t *n, int32_t *k,
               int32_t *e_w, double *gavg_sum, int32_t *gavg_count,
               double t_min, double t_max, int k_min, int k_max,
               int32_t *dk_out, void *stream);

/* apt_update and apt_adjust over layers held at their own width, for the
 * memory saving low precision brings ([APT] section on the memory of
 * training): wbytes (HOST int32 [L]) gives each layer's bytes per weight,
 * 2 (int16 mantissas, as above) or 1 (int8 mantissas; W[l] 1-byte aligned,
 * 8-byte aligned for the vector path).  A layer held in int8 reads its k in
 * [2, 8] (a k above 8 as 8) and apt_adjust never raises it past 8, so its
 * mantissas always fit; the arithmetic is that of an int16 layer with the
 * same k, bit for bit.  wbytes NULL: every layer int16.  A wbytes entry other
 * than 1 or 2 is IONN_ERR_ARG. */
int apt_update_mixed(int L, void *const *W, const int32_t *wbytes,
                     const int16_t *const *G, const int64_t *n, const int32_t *k,
                     const int32_t *e_w, const int32_t *e_g, int lr_shift,
                     double *gavg_sum, int32_t *gavg_count, void *workspace,
                     size_t workspace_bytes, void *stream);
int apt_adjust_mixed(int L, void *const *W, const int32_t *wbytes, const int64_t *n,
                     int32_t *k, int32_t *e_w, double *gavg_sum,
                     int32_t *gavg_count, double t_min, double t_max, int k_min,
                     int k_max, int32_t *dk_out, void *stream);

/* ------------------------------------------------------------------------ */
/* The floating-point operations around the integer products ([DFP] section  */
/* 4: the integer kernels do the products, the operations around them run in */
/* floating point): a Linear layer on DFP-8 operands with bias, activation   */
/* and residual in its epilogue, its backward pass, layer norm and AdamW.    */
/*                                                                          */
/* A DFP-8 tensor is int8 mantissas I plus one shared exponent E (a device   */
/* int32 in [-128, 127]): value I * 2^E ([DFP] section 3 with P = 8).        */
/* Floating tensors are of type `dtype` (one of the IONN_F32 ... values) and */
/* row-major; arithmetic is in float32 and a value is rounded to its type    */
/* once, when it is stored.  Every tensor must be aligned to its element     */
/* size; 16-byte aligned tensors whose rows are multiples of 16 bytes take   */
/* the vector paths.                                                         */
/* ------------------------------------------------------------------------ */

enum { IONN_F32 = 0, IONN_BF16 = 1, IONN_F16 = 2 };

/* gelu: z * Phi(z), Phi the normal distribution function; gelu_tanh: its
 * approximation z / 2 * (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))); silu:
 * z / (1 + exp(-z)). */
enum {
    IONN_ACT_NONE = 0,
    IONN_ACT_RELU = 1,
    IONN_ACT_GELU = 2,
    IONN_ACT_GELU_TANH = 3,
    IONN_ACT_SILU = 4
};

/* Longest reduction of the DFP-8 products: the int32 sum of this many
 * products of int8 values cannot overflow. */
#define IONN_DFP8_MAX_REDUCTION 131071

/* Floating point -> DFP-8: max |x| = f * 2^q (f in [1, 2)) gives E = q - 6
 * (0 for an all-zero x) and out = sat8(round_to_nearest_even(x / 2^E)).
 * x: dtype [n]; out: int8 [n]; e_out: device int32; status_out (nullable,
 * device int32): 0, 1 when E leaves the signed 8-bit range (E still
 * written), 2 when x holds a NaN or infinity (outputs then unspecified).
 * absmax (nullable): device uint32 that holds the float32 bits of max |x|, of
 * x itself or as it was before it was rounded to its type (as the absmax
 * arguments below leave them: the call rounds it); the maximum is then not
 * taken again.  Without it the call takes it, in `workspace` (4-byte aligned,
 * dfp8_from_float_workspace_bytes() bytes).  n >= 1. */
size_t dfp8_from_float_workspace_bytes(void);
int dfp8_from_float(const void *x, int dtype, int64_t n, const uint32_t *absmax,
                    int8_t *out, int32_t *e_out, int32_t *status_out,
                    void *workspace, size_t workspace_bytes, void *stream);

/* Forward of a Linear layer on DFP-8 operands:
 *   z[b][o] = fl(sum_i X[b][i] * W[o][i]) * 2^(eX + eW) + bias[o]
 *   Y[b][o] = act(z[b][o]) + residual[b][o]
 * with the sum exact in int32.  X: int8 [B][IN]; W: int8 [OUT][IN]; bias
 * (nullable): float [OUT]; act: IONN_ACT_*; residual (nullable), Y: dtype
 * [B][OUT] (Y may be the residual itself); Z (nullable): dtype [B][OUT],
 * receives z for the backward pass.  absmax_Y (nullable): device uint32,
 * max-combined with the float32 bits of |Y| before its rounding (a NaN counts
 * above every number), to be rounded by dfp8_from_float.  B, OUT in
 * [0, 2^30], of fewer than 2^24 tiles of 64 x 64 where the output is cut into
 * them; 0 <= IN <= IONN_DFP8_MAX_REDUCTION (IN = 0: the sum is 0).
 * workspace: 16-byte aligned, dfp8_linear_fwd_workspace_bytes(B, IN, OUT)
 * bytes (may be 0). */
size_t dfp8_linear_fwd_workspace_bytes(int64_t B, int64_t IN, int64_t OUT);
int dfp8_linear_fwd(const int8_t *X, const int32_t *eX, const int8_t *W,
                    const int32_t *eW, const float *bias, int act,
                    const void *residual, void *Z, void *Y, int dtype,
                    int64_t B, int64_t IN, int64_t OUT, uint32_t *absmax_Y,
                    void *workspace, size_t workspace_bytes, void *stream);

/* Backward of that layer, for the error dY of Y:
 *   dZ = dY * act'(Z)                       (float32, not stored)
 *   gb[o] = sum_b dZ[b][o]                  (float32, a fixed order)
 *   dZ8, edZ = DFP-8 of dZ, as dfp8_from_float converts
 *   dX = fl(dZ8 . W) * 2^(edZ + eW),  G = fl(dZ8^T . X) * 2^(edZ + eX)
 * (the residual's gradient is dY itself).  dY: dtype [B][OUT]; Z: dtype
 * [B][OUT] as the forward stored it (may be NULL for IONN_ACT_NONE); dZ8:
 * int8 [B][OUT] and edZ: device int32 (written); dX (nullable): dtype
 * [B][IN]; G (nullable): dtype [OUT][IN]; gb (nullable): float [OUT].
 * status_out (nullable, device int32): as in dfp8_from_float, for dZ.
 * B, IN, OUT in [0, 2^30]; OUT <= IONN_DFP8_MAX_REDUCTION with dX, B <= it
 * with G; the gradients, together, of fewer than 2^24 tiles of 64 x 64 where
 * they are cut into them.
 * B = 0 writes G = 0 and gb = 0; OUT = 0 writes dX = 0; edZ = 0 either way.
 * workspace: 16-byte aligned, dfp8_linear_bwd_workspace_bytes(B, IN, OUT)
 * bytes. */
size_t dfp8_linear_bwd_workspace_bytes(int64_t B, int64_t IN, int64_t OUT);
int dfp8_linear_bwd(const void *dY, const void *Z, int act, int dtype,
                    const int8_t *X, const int32_t *eX, const int8_t *W,
                    const int32_t *eW, int8_t *dZ8, int32_t *edZ, void *dX,
                    void *G, float *gb, int64_t B, int64_t IN, int64_t OUT,
                    int32_t *status_out, void *workspace,
                    size_t workspace_bytes, void *stream);

/* The gated layer of a feed-forward block.  W: int8 [2 H][IN], the gate's rows
 * and then the up projection's, one DFP-8 tensor; with (g | u) the two halves of
 *   z[b][o] = fl(sum_i X[b][i] * W[o][i]) * 2^(eX + eW) + bias[o],
 *   Y[b][h] = act(g[b][h]) * u[b][h]
 * (act IONN_ACT_NONE: g * u).  bias (nullable): float [2 H]; Y: dtype [B][H];
 * Z (nullable): dtype [B][2 H], receives z for the backward pass (apart from Y).
 * absmax_Y and the rest as in dfp8_linear_fwd with OUT = 2 H: H in [0, 2^29],
 * 0 <= IN <= IONN_DFP8_MAX_REDUCTION.  workspace: 16-byte aligned,
 * dfp8_gated_fwd_workspace_bytes(B, IN, H) bytes (may be 0; of large products
 * whose rows are not whole 16-byte pieces, X and W once more). */
size_t dfp8_gated_fwd_workspace_bytes(int64_t B, int64_t IN, int64_t H);
int dfp8_gated_fwd(const int8_t *X, const int32_t *eX, const int8_t *W,
                   const int32_t *eW, const float *bias, int act, void *Z,
                   void *Y, int dtype, int64_t B, int64_t IN, int64_t H,
                   uint32_t *absmax_Y, void *workspace, size_t workspace_bytes,
                   void *stream);

/* Its backward pass, for the error dY of Y:
 *   dZ = (dY * u * act'(g) | dY * act(g))   (not stored; float32, and float64
 *     for dtype IONN_F32 with IONN_ACT_NONE or IONN_ACT_RELU, where a value
 *     that float32 would round to infinity counts as that)
 *   gb[o] = sum_b dZ[b][o]                  (float32, a fixed order)
 *   dZ8, edZ = DFP-8 of dZ, one exponent for both halves
 *   dX = fl(dZ8 . W) * 2^(edZ + eW),  G = fl(dZ8^T . X) * 2^(edZ + eX)
 * Z: dtype [B][2 H] as the forward stored it (for every act); dZ8: int8
 * [B][2 H] and edZ: device int32 (written); dX (nullable): dtype [B][IN]; G
 * (nullable): dtype [2 H][IN]; gb (nullable): float [2 H]; the rest as in
 * dfp8_linear_bwd with OUT = 2 H. */
size_t dfp8_gated_bwd_workspace_bytes(int64_t B, int64_t IN, int64_t H);
int dfp8_gated_bwd(const void *dY, const void *Z, int act, int dtype,
                   const int8_t *X, const int32_t *eX, const int8_t *W,
                   const int32_t *eW, int8_t *dZ8, int32_t *edZ, void *dX,
                   void *G, float *gb, int64_t B, int64_t IN, int64_t H,
                   int32_t *status_out, void *workspace,
                   size_t workspace_bytes, void *stream);

/* How a product of the Linear layer is cut, by its sizes: the forward product, dX or
 * G (product 0, 1 or 2), IONN_DFP8_ROWS: small tiles, the reduction cut among
 * a workgroup's wavefronts; _TILES_256, _TILES_128: tiles of that side, of
 * operands whose addresses are multiples of 16 (others take _TILES);
 * _TILES: tiles of 64, in ranges of the reduction where there are few;
 * _NARROW: the same for contiguous sides below 16.  -1: sizes out of range. */
enum {
    IONN_DFP8_ROWS = 0,
    IONN_DFP8_TILES_256 = 1,
    IONN_DFP8_TILES_128 = 2,
    IONN_DFP8_TILES = 3,
    IONN_DFP8_NARROW = 4
};
int dfp8_linear_path(int product, int64_t B, int64_t IN, int64_t OUT);

/* Layer norm over the rows of x:
 *   mean[r] = sum_c x[r][c] / cols, rstd[r] = 1 / sqrt(sum_c (x[r][c] -
 *   mean[r])^2 / cols + eps),
 *   y[r][c] = (x[r][c] - mean[r]) * rstd[r] * gamma[c] + beta[c].
 * x, y: dtype [rows][cols] (y may be x); gamma (nullable: 1), beta
 * (nullable: 0): float [cols]; mean, rstd (nullable): float [rows], written
 * for the backward pass.  absmax_y as in dfp8_linear_fwd.  rows, cols >= 0
 * and below 2^31; eps >= 0. */
int ionn_layer_norm_fwd(const void *x, const float *gamma, const float *beta,
                        double eps, void *y, float *mean, float *rstd,
                        int dtype, int64_t rows, int64_t cols,
                        uint32_t *absmax_y, void *stream);

/* Its gradient, for the error dy of y, with h = (x - mean) * rstd and
 * d = dy * gamma:
 *   dx = rstd * (d - mean_c(d) - h * mean_c(d * h)) + dres
 *   dgamma[c] = sum_r dy[r][c] * h[r][c],  dbeta[c] = sum_r dy[r][c].
 * dres (nullable): dtype [rows][cols], the gradient that reaches x past the
 * norm (the residual branch); dx may be dy or dres.  dgamma, dbeta
 * (nullable): float [cols], summed in an order that the sizes fix (0 for
 * rows = 0).  workspace: 16-byte aligned,
 * ionn_layer_norm_bwd_workspace_bytes(rows, cols) bytes (needed where dgamma
 * or dbeta is asked for). */
size_t ionn_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t cols);
int ionn_layer_norm_bwd(const void *dy, const void *x, const float *mean,
                        const float *rstd, const float *gamma, const void *dres,
                        void *dx, float *dgamma, float *dbeta, int dtype,
                        int64_t rows, int64_t cols, void *workspace,
                        size_t workspace_bytes, void *stream);

/* What lies between two blocks of a residual stream: the norm after a block's
 * output a, its gate, the scaled residual, and the norm before the next block,
 *   p = N_a(a),  y[r][c] = alpha * x[r][c] + gate[r / gate_rows][c] * p[r][c],
 *   n = N_y(y)
 * with the statistics of y and n taken from y before it is rounded.  norm_a,
 * norm_y: IONN_NORM_NONE (the row itself), _LAYER (as ionn_layer_norm_fwd) or
 * _RMS: N(v)[c] = v[c] * rstd * gamma[c], rstd = 1 / sqrt(sum_c v[c]^2 / cols +
 * eps).  a, x, y, n: dtype [rows][cols]; gamma_* (nullable: 1), beta_* (nullable:
 * 0; layer norms only): float [cols]; gate (nullable: 1): float
 * [ceil(rows / gate_rows)][cols], gate_rows rows share a gate (0, or rows and
 * more: all); mean_* (layer norms only), rstd_* (nullable): float [rows], written
 * for the backward pass.  a NULL: y = alpha * x (the norm before the first
 * block).  y NULL or n NULL: not written (without n nor are its norm's other
 * results); n NULL where norm_y is IONN_NORM_NONE.  y and n may be a or x.
 * absmax_n as in dfp8_linear_fwd.  rows >= 0 and below 2^31, 0 <= cols <= 16384;
 * eps >= 0; alpha finite. */
enum { IONN_NORM_NONE = 0, IONN_NORM_LAYER = 1, IONN_NORM_RMS = 2 };
int ionn_residual_norm_fwd(const void *a, const void *x, int norm_a,
                           const float *gamma_a, const float *beta_a,
                           const float *gate, int64_t gate_rows, double alpha,
                           int norm_y, const float *gamma_y,
                           const float *beta_y, double eps, void *y, void *n,
                           float *mean_a, float *rstd_a, float *mean_y,
                           float *rstd_y, int dtype, int64_t rows, int64_t cols,
                           uint32_t *absmax_n, void *stream);

/* Its gradient, for the errors dy of y (nullable: 0) and dn of n, with h_a, h_y
 * the normalised rows ((v - mean) * rstd; without a norm v itself):
 *   t  = dy + N_y'(dn)      (float32, not stored; N_y' as dx in
 *                            ionn_layer_norm_bwd, without mean_c(d) for _RMS)
 *   dx = alpha * t,  da = N_a'(gate * t)
 *   dgate[g][c] = sum over the rows of g of t * p
 *   dgamma_a[c] = sum_r gate * t * h_a,  dbeta_a[c] = sum_r gate * t
 *   dgamma_y[c] = sum_r dn * h_y,        dbeta_y[c] = sum_r dn
 * y: as the forward stored it; the statistics: as it left them.  Every output is
 * nullable; da and dx may be dy, dn, a or y, but not each other.  The vectors'
 * gradients are float32, summed in an order that the sizes fix (rows = 0: zeros,
 * dgate's for the one gate of all rows); beta_a is read for dgate.  workspace:
 * 16-byte aligned, ionn_residual_norm_bwd_workspace_bytes(rows, cols, gate_rows)
 * bytes (needed where a vector's gradient is asked for; gate_rows = 0 without a
 * gate). */
size_t ionn_residual_norm_bwd_workspace_bytes(int64_t rows, int64_t cols,
                                              int64_t gate_rows);
int ionn_residual_norm_bwd(const void *dy, const void *dn, const void *a,
                           const void *y, int norm_a, const float *gamma_a,
                           const float *beta_a, const float *gate,
                           int64_t gate_rows, double alpha, int norm_y,
                           const float *gamma_y, const float *mean_a,
                           const float *rstd_a, const float *mean_y,
                           const float *rstd_y, void *da, void *dx,
                           float *dgamma_a, float *dbeta_a, float *dgate,
                           float *dgamma_y, float *dbeta_y, int dtype,
                           int64_t rows, int64_t cols, void *workspace,
                           size_t workspace_bytes, void *stream);

/* One AdamW step of L tensors, in place.  Per element, each operation
 * rounded to float32 on its own (none fused):
 *   g = G * grad_scale
 *   m = beta1 * m + (1 - beta1) * g,  v = beta2 * v + ((1 - beta2) * g) * g
 *   u = m / (sqrt(v) * (1 / sqrt(1 - beta2^t)) + eps)
 *   P = P * (1 - lr * weight_decay) - (lr / (1 - beta1^t)) * u
 * (the scalar factors computed in double and rounded once).  P: float32
 * [n[l]] master weights; G: [n[l]] of type g_dtype.
 * state_bits 32: M, V float32 [n[l]] hold m and v; S NULL.
 * state_bits 8: blocks of IONN_ADAMW_BLOCK elements (the last one shorter).
 * M and V hold 8-bit floating codes of OCP E4M3 (1-4-3, bias 7, largest
 * 448), of m and of r = sqrt(v): m = code * 2^S[l][2 b], r = code *
 * 2^S[l][2 b + 1] in block b, S[l]: int8 [2 * blocks].  The step works on
 * the float32 m and v and stores both again: for a block's largest finite
 * magnitude f * 2^q (f in [1, 2)) the exponent is q - 8 where f <= 1.75,
 * q - 7 otherwise, at least -126 (0 for an all-zero block).
 *   m rounds to the nearest code (even) where beta1 <= 15/16.  Above, a step
 * changes it by less than a code's half step, and it goes to the code on either
 * side of it, the farther from 0 with probability (|s| - lo) / (hi - lo), s =
 * m / 2^exponent.
 *   r, which a step changes by less than a code's half step, goes to the code
 * below or above, lo or hi: with s = r / 2^exponent to hi where (s - lo) * (s +
 * lo) > d * (hi^2 - lo^2) in float32, d in (0, 1) a hash of t and the element's
 * index (draw4() in csrc/adamw.hip), so that the expectation of v is kept.  Over
 * many steps v is right on average, and r scatters by about 15% around the
 * 32-bit state's (25% where beta2 = 0.95 and the gradients fall);
 * ionn_adamw_step_carried follows it closely.  A positive r never becomes 0 (the
 * smallest code, 2^-18 of the block's largest, takes its place, so that no later
 * step divides by a vanished r).
 *   A value that is not finite becomes the NaN code 0x7f; the block's others are
 * unaffected.
 * t: the number of this step, from 1.  For a captured graph, step (nullable,
 * device int32) gives t and lr_dev (nullable, device float) gives lr when the
 * kernel runs; the caller advances them.  grad_scale (nullable, device
 * float): 1.  absmax_P (nullable, device uint32 [L]): max-combined with the
 * float32 bits of |P| after the step, for dfp8_from_float.
 * L >= 1; P, G, M, V, S, n are HOST arrays; 1 <= n[l] <= 2^35 - 2^11 (8-bit
 * states; twice that in 32 bits).
 * 0 <= beta1, beta2 < 1; eps >= 0; lr and weight_decay finite. */
#define IONN_ADAMW_BLOCK 256
int ionn_adamw_step(int L, float *const *P, const void *const *G, int g_dtype,
                    void *const *M, void *const *V, int8_t *const *S,
                    int state_bits, const int64_t *n, int64_t t, double lr,
                    double beta1, double beta2, double eps, double weight_decay,
                    const int32_t *step, const float *lr_dev,
                    const float *grad_scale, uint32_t *absmax_P, void *stream);

/* The same step of 8-bit states whose roots carry a remainder, so that the
 * second moment follows its definition over any number of steps.  P and M are
 * the step's above.  R[l], int8 [n[l]], holds q of the whole root w /
 * 2^exponent = value(code) + q * step / 254, step the distance from the code's
 * value to the next; w steps as the root of v does, V's codes are the nearest
 * ones to it (even; at least the smallest for a positive w), and q is the whole
 * number below or above, by the same hash (floor(x + d)), from -127 to 127.  w
 * stays within about 2% of the 32-bit state's root, 0.5% in the mean square.
 * R = 0 to begin with. */
int ionn_adamw_step_carried(int L, float *const *P, const void *const *G,
                            int g_dtype, void *const *M, void *const *V,
                            int8_t *const *S, int8_t *const *R,
                            const int64_t *n, int64_t t, double lr,
                            double beta1, double beta2, double eps,
                            double weight_decay, const int32_t *step,
                            const float *lr_dev, const float *grad_scale,
                            uint32_t *absmax_P, void *stream);

/* One Muon step of L matrices, in place:
 *   g = G * grad_scale,  M = momentum * M + g
 *   u = g + momentum * M (nesterov) or M
 *   X = u / (|u| + eps), |u| the root of the sum of squares (in float64)
 *   ns_steps times:  A = X X^T,  X = a X + (b A + c A A) X
 *     (a, b, c = 3.4445, -4.7750, 2.0315; of a matrix of more rows than columns,
 *     X^T in the place of X)
 *   P = P * (1 - lr * weight_decay) - lr * scale[l] * X
 * P, M: float32 [rows[l]][cols[l]]; G: the same of type g_dtype.  The products'
 * operands are held as pairs of float16 terms (22 bits, steps of 2^-36 at
 * least) and summed in float32, so X is right to about 1e-6 of its size; where
 * |u| is below eps / 1000 the steps show, and below 2^-37 an element of u /
 * (|u| + eps) counts as 0.  A u of zeros leaves X = 0; one that is not finite
 * everywhere makes the whole of P not a number.  scale (nullable, HOST [L]):
 * sqrt(max(1, rows / cols)).  lr_dev (nullable, device float) gives lr when the
 * kernels run; grad_scale (nullable, device float): 1.  absmax_P (nullable,
 * device uint32 [L]): max-combined with the float32 bits of |P| after the step,
 * for dfp8_from_float.  L >= 1; P, G, M, rows, cols are HOST arrays; rows, cols
 * >= 1, their product as multiples of 256 at most 2^28; no P or M overlaps
 * another of them or a G (gradients may be one tensor); 0 <= momentum < 1; eps
 * >= 0; lr and weight_decay finite; ns_steps in [1, 32].  workspace: 256-byte
 * aligned, ionn_muon_workspace_bytes(L, rows, cols) bytes (0 on invalid sizes). */
size_t ionn_muon_workspace_bytes(int L, const int64_t *rows, const int64_t *cols);
/* The side of the tiles that matrix l is worked in, with those that share its
 * launches: 32, 64, 128 or 256; -1: sizes out of range.  (Which one decides how
 * sums are rounded and nothing else.) */
int ionn_muon_tile(int L, const int64_t *rows, const int64_t *cols, int l);
int ionn_muon_step(int L, float *const *P, const void *const *G, int g_dtype,
                   float *const *M, const int64_t *rows, const int64_t *cols,
                   double lr, double momentum, int nesterov, double eps,
                   double weight_decay, int ns_steps, const double *scale,
                   const float *lr_dev, const float *grad_scale,
                   uint32_t *absmax_P, void *workspace, size_t workspace_bytes,
                   void *stream);

#ifdef __cplusplus
}
#endif
#endif /* IONN_H */
