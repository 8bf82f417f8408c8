/*
 * qb.h -- C ABI of libqb: block-wise dynamic quantization, nested quantization
 * of the block constants, the fused 8-bit AdamW step and its sibling 8-bit
 * optimizers (with paged states), user codes, the product of a 4-bit layer, the
 * stable embedding layer (embedding lookup, layer norm, their gradients), and the
 * training step around a 4-bit layer (linear and gated layers with their
 * gradients, the global gradient norm), for AMD Instinct MI355X (gfx950).
 *
 * The method: a tensor is cut into blocks of `blocksize` consecutive elements;
 * every block is scaled by its own absolute maximum and each scaled value is
 * replaced by the index of the nearest entry of a fixed code, so blocks are
 * quantized independently and in parallel (abstract of "8-bit Optimizers via
 * Block-wise Quantization", quoted on the page "Py之bitsandbytes：bitsandbytes的
 * 简介、安装、使用方法之详细攻略", section 2; page "bitsandbytes深度解析",
 * section 核心量化原理与实现机制).
 *
 * Codes (QB_DYN8, QB_NF4, QB_FP4, QB_UDYN8) -- see qb_codebook() for the exact
 * tables:
 *   QB_DYN8  256-entry signed dynamic code (decimal exponent + linear fraction),
 *            one byte per element; index 127 is 0.0, 255 is +1.0.
 *   QB_UDYN8 256-entry unsigned dynamic code for an optimizer state that is
 *            never negative (see qb_optim_hparams.v_code): the sign bit of
 *            QB_DYN8 spent on one more fraction bit, so each of the same seven
 *            decades holds twice as many values; index 0 is 0.0, 255 is +1.0.
 *            The pages name only the signed code; this is its plainest
 *            unsigned form.
 *   QB_NF4   16 normal-quantile values in [-1, 1], two codes per byte.
 *   QB_FP4   E2M1 minifloat / 6, sign-magnitude nibble, two codes per byte.
 * 4-bit packing: element 2k is the high nibble of byte k, element 2k+1 the low
 * nibble; an odd count leaves the last low nibble 0.
 * Encoding: nearest entry of value/absmax, a tie going to the entry of smaller
 * magnitude; a block whose absmax is 0 gets the code of 0.0.
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers unless marked "host".  The caller
 *     owns every buffer: libqb never allocates device memory and keeps no state
 *     between calls except its constant tables (and the one scratch array of
 *     qb_multi_tensor_step_noalloc).  Every entry point is safe to
 *     call from several host threads at once, with two exceptions whose
 *     calls on one device must not overlap in time (see their descriptions):
 *     qb_multi_tensor_step_noalloc, whose calls on one device share its
 *     scratch array, and qb_paged_optimizer_step, whose calls on one device
 *     share internal copy streams and events.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Work is enqueued
 *     asynchronously on it; no entry point synchronizes the device.
 *   - Arguments are validated before anything is enqueued; on any error
 *     nothing runs and nothing is written.  A failed launch returns QB_EHIP.
 *     No C++ exception crosses this interface.
 *   - Device pointers must be 16-byte aligned (QB_EALIGN otherwise).
 *   - n == 0 is a no-op returning QB_OK.
 *   - Inputs must be finite; NaN/Inf inputs give unspecified codes.
 *   - blocksize is a power of two in [64, 4096]; the number of blocks must be
 *     below 2^31.
 */
#ifndef QB_H
#define QB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QB_OK = 0,
    QB_EINVAL = 1,        /* a null pointer, bad size, bad enum or bad hyperparameter */
    QB_EALIGN = 2,        /* a device pointer is not 16-byte aligned */
    QB_EUNSUPPORTED = 3,  /* a valid but unsupported combination */
    QB_EHIP = 4,          /* a HIP runtime call or kernel launch failed */
    QB_EWORKSPACE = 5,    /* the workspace is too small */
    QB_EINIT = 6          /* the constant tables could not be built or uploaded */
} qb_status;

typedef enum { QB_F32 = 0, QB_F16 = 1, QB_BF16 = 2 } qb_dtype;

/* Type of token ids (the row-wise layers below). */
typedef enum { QB_I32 = 0, QB_I64 = 1 } qb_index;

typedef enum { QB_DYN8 = 0, QB_NF4 = 1, QB_FP4 = 2, QB_UDYN8 = 3 } qb_code;

/*
 * Nested ("double") quantization state of the per-block absmax (page
 * "Bitsandbytes" (Transformers docs), section İç içe nicelleştirme: a second
 * quantization of the constants of the first, about 0.4 bit per parameter).
 * The nb = ceil(n / blocksize) fp32 absmax values a_j are centred on their mean
 *   offset = the exact mean of a_j, rounded once to fp32,
 * and d_j = a_j - offset (fp32) is quantized with QB_DYN8 in blocks of
 * blocksize2.  The decoded constant is dyn8[codes_j] * absmax2[j / blocksize2]
 * + offset (two rounded fp32 operations).
 */
typedef struct {
    uint8_t* codes;      /* [nb] QB_DYN8 codes of a_j - offset */
    float*   absmax2;    /* [ceil(nb / blocksize2)] */
    float*   offset;     /* [1] */
    int32_t  blocksize2; /* power of two in [64, 4096]; 256 is the usual value */
    void*    ws;         /* workspace of qb_dq_workspace_bytes(n, blocksize) bytes; used by qb_quantize only */
    size_t   ws_bytes;
} qb_dq;

/*
 * Hyperparameters of one AdamW step (pages: "bitsandbytes - Quantização de
 * LLM", section Workflow 3, where the 8-bit optimizer replaces AdamW with the
 * same lr, betas and eps; "Py之bitsandbytes", section 使用8位优化器).  They are
 * real numbers: every per-element scalar (beta1, 1-beta1, beta2, 1-beta2,
 * lr/(1-beta1^t), 1/sqrt(1-beta2^t), 1-lr*weight_decay, eps) is computed in
 * binary64 and rounded once to binary32.  step is the 1-based step t.
 * Requirements: 0 <= beta1, beta2 < 1; eps > 0; lr, weight_decay finite, >= 0;
 * step >= 1.
 */
typedef struct {
    double  lr;
    double  beta1;
    double  beta2;
    double  eps;
    double  weight_decay;
    int32_t step;
} qb_adamw_hparams;

/*
 * The fused 8-bit optimizers.  The pages list 8-bit Adam, AdamW, SGD, RMSprop
 * and Lion as drop-in replacements that keep their optimizer's
 * hyperparameters (page "bitsandbytes深度解析", section 优化器模块深度分析; page
 * "Py之bitsandbytes", sections 1 and 使用8位优化器).  Each follows its usual
 * definition, every state tensor held as block-wise QB_DYN8 codes with one fp32
 * absmax per block (state 1; state 2 for the two-state kinds):
 *   QB_ADAMW    state 1 = m, state 2 = v; decoupled weight decay (as
 *               qb_adamw8bit_step).
 *   QB_ADAM     state 1 = m, state 2 = v; L2 decay: g <- g + wd*p, then the
 *               bias-corrected Adam update.
 *   QB_LION     state 1 = m:  c = b1*m + (1-b1)*g;  p <- p*(1-lr*wd) - lr*sign(c);
 *               m <- b2*m + (1-b2)*g.
 *   QB_SGD      state 1 = momentum buffer (beta1 = momentum, in (0, 1)):
 *               g <- g + wd*p; buf <- g at step 1, else momentum*buf +
 *               (1-dampening)*g; p <- p - lr*(nesterov ? g + momentum*buf : buf).
 *   QB_RMSPROP  state 1 = v (beta2 = alpha):  g <- g + wd*p;
 *               v <- alpha*v + (1-alpha)*g*g;  p <- p - lr*g/(sqrt(v) + eps).
 * The layer-wise kinds (8-bit LARS and LAMB are listed beside them on page
 * "Py之bitsandbytes", section 1; the pages give no formulas, so these follow
 * the published definitions) scale each tensor's step by a ratio of norms over
 * that whole tensor, one tensor being one layer:
 *   QB_LAMB     state 1 = m, state 2 = v (You et al., 2019):  Adam's moments,
 *               r = (m/(1-b1^t)) / (sqrt(v/(1-b2^t)) + eps),  u = r + wd*p,
 *               p <- p - lr*ratio*u  with ratio = |p| / |u|.
 *   QB_LARS     state 1 = momentum buffer (beta1 = momentum, in [0, 1);
 *               You, Gitman and Ginsburg, 2017):
 *               ratio = trust_coefficient*|p| / (|g| + wd*|p|),
 *               buf <- momentum*buf + lr*ratio*(g + wd*p),  p <- p - buf.
 *   The norms (of p, and of u or g) and the ratio are binary64, a zero norm
 *   makes the ratio 1, and the step takes S = (float)(lr*ratio) as one
 *   binary32 scalar.  They need a workspace for the norms: only
 *   qb_multi_tensor_optimizer_step runs them (one tensor is a call with
 *   count 1).
 * The never-negative state (v of QB_ADAMW, QB_ADAM and QB_LAMB; the state of
 * QB_RMSPROP) may be held in QB_UDYN8 instead (hp->v_code): the same bytes,
 * with twice the resolution in every decade, which halves its worst
 * quantization error relative to the block absmax (0.0035 against 0.0070).
 * Its fresh state is code 0 (0.0).  A state written with one code must be
 * stepped with the same code.
 * The states and their codes are bit-exact against an IEEE binary32 evaluation
 * of these formulas (each operation rounded on its own, IEEE square root and
 * division).  So is p' for every kind but AdamW and LAMB, whose states never
 * read p: there p' takes hardware square root and reciprocal and is within
 * 1e-6 relative.  The layer-wise kinds add their norms in a fixed order of
 * their own (run to run the same bits); an evaluation that adds in another
 * order can differ in the last bits of the binary64 sums, which changes S only
 * when the ratio lies that close to a binary32 rounding boundary.
 */
typedef enum { QB_ADAMW = 0, QB_ADAM = 1, QB_LION = 2, QB_SGD = 3, QB_RMSPROP = 4, QB_LAMB = 5, QB_LARS = 6 } qb_optimizer;

/* Hyperparameters of one step of any kind (unused fields are ignored). */
typedef struct {
    qb_optimizer kind;
    double  lr;
    double  beta1;         /* Adam(W), Lion: beta1; SGD: momentum */
    double  beta2;         /* Adam(W), Lion: beta2; RMSprop: alpha */
    double  eps;           /* Adam(W), RMSprop */
    double  weight_decay;
    double  dampening;     /* SGD */
    int32_t nesterov;      /* SGD: 0 or 1 (1 needs dampening 0) */
    int32_t step;          /* t >= 1 */
    double  trust_coefficient;   /* LARS: eta > 0 */
    qb_code v_code;        /* code of the never-negative state: QB_DYN8 (0, the
                              default) or QB_UDYN8 (QB_ADAMW, QB_ADAM, QB_LAMB,
                              QB_RMSPROP only) */
} qb_optim_hparams;

/* One tensor of a multi-tensor step; the fields are those of qb_adamw8bit_step
 * (m, absmax_m: state 1; v, absmax_v: state 2, ignored by one-state kinds).
 * p holds n values of the call's parameter dtype (fp32 for qb_multi_tensor_step). */
typedef struct {
    void*       p;
    const void* g;
    uint8_t*    m;
    uint8_t*    v;
    float*      absmax_m;
    float*      absmax_v;
    int64_t     n;
} qb_tensor;

/*
 * One tensor of a grouped quantization; the fields are those of qb_quantize.
 * A plain tensor gives absmax and leaves c2, absmax2, offset NULL; a nested
 * one gives c2, absmax2, offset (the outputs of qb_dq) and absmax NULL.
 */
typedef struct {
    const void* x;
    uint8_t*    codes;
    float*      absmax;
    uint8_t*    c2;
    float*      absmax2;
    float*      offset;
    int64_t     n;
} qb_quant_tensor;

/*
 * One tensor of a grouped dequantization; the fields are those of
 * qb_dequantize.  A plain tensor gives absmax and leaves c2, absmax2, offset
 * NULL; a nested one gives c2, absmax2, offset (the qb_dq fields) and absmax
 * NULL.
 */
typedef struct {
    const uint8_t* codes;
    const float*   absmax;
    const uint8_t* c2;
    const float*   absmax2;
    const float*   offset;
    void*          y;
    int64_t        n;
} qb_dequant_tensor;

/*
 * qb_quantize -- block-wise quantization (pages cited at the top; NF4: page
 * "Bitsandbytes", section Normal Float 4 (NF4); FP4: page "Quantize 🤗
 * Transformers models", section FP4 quantization).
 *   x       [n] input of dtype xdt (fp32, fp16 or bf16).
 *   code    QB_DYN8 (codes: n bytes) or QB_NF4 / QB_FP4 (codes: ceil(n/2) bytes);
 *           QB_UDYN8 serves only the optimizer states (QB_EINVAL here).
 *   absmax  [ceil(n/blocksize)] fp32 block absmax out; must be NULL when dq is given.
 *   dq      NULL, or the nested state to fill (codes, absmax2, offset; the
 *           workspace holds the fp32 absmax while the call runs).
 * Outputs are fully overwritten.  One kernel, or four with dq (clear the
 * workspace's exponent bins, quantize, exact mean of the absmax, quantize
 * absmax - mean), all on `stream`.
 */
qb_status qb_quantize(const void* x, qb_dtype xdt, int64_t n, qb_code code, int32_t blocksize,
                      uint8_t* codes, float* absmax, const qb_dq* dq, void* stream);

/*
 * qb_normalize -- the normalized values of block-wise quantization, the step
 * between the block absmax and the encoding (each block is scaled by its own
 * absmax: "8-bit Optimizers via Block-wise Quantization" abstract, quoted on
 * page "Py之bitsandbytes", section 2), computed by the quantize kernels' own
 * quotient: out[i] = RN(x[i] / absmax[i / blocksize]) in binary32, equal to
 * IEEE division bit for bit (a zero x keeps its sign), and +0 where that
 * absmax is 0.  For inspection, e.g. counting values that lie within an ulp
 * of a code midpoint.
 *   x          [n] of dtype xdt.
 *   absmax     [ceil(n/blocksize)] fp32, finite, >= 0, with |x[i]| <=
 *              absmax[i / blocksize] (as qb_quantize writes it); other values
 *              give unspecified results.
 *   blocksize  any value >= 1 (1: one absmax per element).
 *   out        [n] fp32, fully overwritten.
 * One kernel.  QB_EINVAL for n < 0, blocksize < 1 or a NULL pointer with n > 0.
 */
qb_status qb_normalize(const void* x, qb_dtype xdt, int64_t n, const float* absmax, int32_t blocksize, float* out,
                       void* stream);

/*
 * qb_multi_tensor_quantize -- qb_quantize on `count` tensors (same input
 * dtype, code, block size and nested block size for all) in one kernel launch,
 * or four with nesting; the result equals a loop of single-tensor calls, bit
 * for bit.  Quantizing all weights of a model at load time (page
 * "Bitsandbytes", sections Normal Float 4 (NF4) and İç içe nicelleştirme) this
 * way avoids one launch ramp per tensor.
 *   tensors     host array of `count` descriptors (read during the call only);
 *               either every tensor is nested or none (else QB_EUNSUPPORTED).
 *   blocksize2  block size of the nested level (ignored without nesting).
 *   ws          device workspace of
 *               qb_multi_tensor_quantize_workspace_bytes(tensors, count,
 *               blocksize) bytes: tables of the tensors, copied in on
 *               `stream`, and with nesting the exponent bins and the fp32
 *               absmax of every tensor (4 bytes per block) while the call runs.
 * Tensors with n == 0 are skipped.  count == 0 is a no-op.
 */
qb_status qb_multi_tensor_quantize(const qb_quant_tensor* tensors, int32_t count, qb_dtype xdt, qb_code code,
                                   int32_t blocksize, int32_t blocksize2, void* ws, size_t ws_bytes,
                                   void* stream);
size_t qb_multi_tensor_quantize_workspace_bytes(const qb_quant_tensor* tensors, int32_t count,
                                                int32_t blocksize);

/*
 * qb_dequantize -- y_i = ydt(table[c_i] * s_b), one fp32 multiply then a
 * round-to-nearest-even conversion (page "Bitsandbytes", section on
 * dequantizing a model; compute dtype: page "Quantize 🤗 Transformers models",
 * section Change the compute dtype).  s_b is absmax[b], or with dq the decoded
 * nested constant of block b (dq->ws is not used).
 *   codes  [n] (DYN8) or [ceil(n/2)] (NF4/FP4);  y [n] of dtype ydt.
 */
qb_status qb_dequantize(const uint8_t* codes, const float* absmax, const qb_dq* dq, qb_code code,
                        int32_t blocksize, int64_t n, void* y, qb_dtype ydt, void* stream);

/*
 * qb_dequant_matmul -- y = x W^T with the weights W held in 4 bits: the
 * product of a 4-bit layer in its compute dtype (page "Bitsandbytes",
 * section QLoRA: Hesaplama veri türü; page "Quantize 🤗 Transformers models",
 * sections Change the compute dtype and Using NF4).  Every weight is first
 * dequantized exactly as by qb_dequantize into the compute dtype xdt, then the
 * products are summed in binary32 (fused in one kernel: the dequantized matrix
 * is never written to memory).
 *   x       [M, K] row-major, dtype xdt (QB_F32, QB_F16 or QB_BF16), 16-byte aligned.
 *   codes   W [N, K] row-major (a layer's [out, in] weight), NF4 or FP4 codes,
 *           two per byte as qb_quantize writes them; 16-byte aligned.
 *   absmax  [ceil(N*K / blocksize)] fp32, or NULL with dq (nested constants:
 *           dq->codes, absmax2, offset, blocksize2; dq->ws is not used).
 *   y       [M, N] row-major, dtype xdt, 16-byte aligned; each output is the
 *           binary32 sum rounded once to xdt.
 * Requirements: K a positive multiple of 32 below 2^24; M, N >= 0 (either 0: no-op).
 * Performance: up to 64 rows of x one wave per 16 weight rows streams W once
 * (up to 8 16-bit rows of at most 64 KiB in all are staged in LDS first);
 * from 65 rows (xdt 16-bit, K a multiple of 128) an LDS-tiled kernel shares x
 * across 64- or 128-row tiles and dequantizes W once per tile.  qb_dequant_linear
 * without an epilogue is the same product (other last bits), faster up to 64 rows and
 * from 512 on, with a workspace beyond 64 rows (K, N < 2^21 there).
 * Accuracy: each product of two xdt values is exact in binary32; the K-term
 * sums are added in an order of the kernel's own (fixed: the same bits on
 * every run), so y is within (K+2) 2^-23 sum_k |x_mk w_nk| of the exact
 * product before its final rounding.
 */
qb_status qb_dequant_matmul(const void* x, qb_dtype xdt, int64_t M, int64_t K, const uint8_t* codes,
                            const float* absmax, const qb_dq* dq, qb_code code, int32_t blocksize, int64_t N,
                            void* y, void* stream);

/*
 * One weight of qb_dequant_matmul_grouped: codes, absmax / nested constants
 * and y as for qb_dequant_matmul; N its rows (the layer's output features).
 * A plain weight gives absmax and leaves c2, absmax2, offset NULL; a nested
 * one gives c2, absmax2, offset (the qb_dq fields) and absmax NULL.
 */
typedef struct {
    const uint8_t* codes;
    const float*   absmax;
    const uint8_t* c2;
    const float*   absmax2;
    const float*   offset;
    void*          y;
    int64_t        N;
} qb_matmul_weight;

#define QB_MATMUL_GROUP_MAX 8

/*
 * qb_dequant_matmul_grouped -- qb_dequant_matmul for up to QB_MATMUL_GROUP_MAX
 * weights that multiply the same activations (a layer's query, key and value
 * projections; its gate and up projections): y_i = x W_i^T, each y_i bit for
 * bit the y of a qb_dequant_matmul call on weight i.  Same page citations as
 * qb_dequant_matmul.
 *   x, xdt, M, K         as for qb_dequant_matmul (one x for all weights).
 *   weights              host array of `count` descriptors (read during the
 *                        call only); every weight is plain or every one is
 *                        nested (else QB_EUNSUPPORTED); code, blocksize and
 *                        blocksize2 (nested only) are shared.
 * Weights with N == 0 are skipped (their pointers are not looked at);
 * count == 0 or M == 0 is a no-op;
 * count > QB_MATMUL_GROUP_MAX is QB_EINVAL.  Up to 64 rows of x (and for
 * binary32 x, or K not a multiple of 128, at any M) the column tiles of all
 * weights are one kernel launch, so small-batch projections fill the GPU
 * together; in the LDS-tiled regime it launches once per weight.
 */
qb_status qb_dequant_matmul_grouped(const void* x, qb_dtype xdt, int64_t M, int64_t K,
                                    const qb_matmul_weight* weights, int32_t count, qb_code code,
                                    int32_t blocksize, int32_t blocksize2, void* stream);

/*
 * qb_multi_tensor_dequantize -- qb_dequantize on `count` tensors in ONE kernel
 * launch (same code, block size, nested block size and output dtype for all;
 * the result equals a loop of single-tensor calls, bit for bit).  Dequantizing
 * the weights of many layers at once (page "Bitsandbytes", section on
 * dequantizing a model) this way avoids one launch ramp per tensor.
 *   tensors     host array of `count` descriptors (read during the call only);
 *               either every tensor is nested or none (else QB_EUNSUPPORTED).
 *   blocksize2  block size of the nested level (ignored without nesting).
 *   ws          device workspace of qb_multi_tensor_workspace_bytes(count)
 *               bytes, filled with a table of the tensors on `stream` (so it
 *               must not be reused by another stream until the call has run).
 * Tensors with n == 0 are skipped.  count == 0 is a no-op.
 */
qb_status qb_multi_tensor_dequantize(const qb_dequant_tensor* tensors, int32_t count, qb_code code,
                                     int32_t blocksize, int32_t blocksize2, qb_dtype ydt, void* ws,
                                     size_t ws_bytes, void* stream);

/*
 * qb_adamw8bit_step -- one fused AdamW step with both moments held as block-wise
 * QB_DYN8 codes (abstract quoted on "Py之bitsandbytes", section 2: 8-bit
 * optimizer state with block-wise dynamic quantization; "bitsandbytes -
 * Quantização de LLM", section Workflow 3: 2 bytes of state per parameter).
 * Per block of `blocksize` elements, in one kernel:
 *   m = dyn8[m_i]*absmax_m[b], v = dyn8[v_i]*absmax_v[b]
 *   m' = b1*m + (1-b1)*g,  v' = b2*v + (1-b2)*g*g
 *   p' = p*(1-lr*wd) - lr/(1-b1^t) * m' / (sqrt(v')/sqrt(1-b2^t) + eps)
 *   absmax_m[b] = max|m'|, absmax_v[b] = max|v'|, m_i, v_i = codes of m', v'.
 *   p          [n] fp32, in place.     g [n] of dtype gdt, read only; must not alias p.
 *   m, v       [n] uint8 codes, in place.  Fresh state: every code 127 (0.0), absmax 0.
 *   absmax_*   [ceil(n/blocksize)] fp32, in place.
 * The state codes and absmax are bit-exact against an IEEE binary32 evaluation
 * of the formulas above; p' uses hardware square root and reciprocal and is
 * within 1e-6 relative of it.
 */
qb_status qb_adamw8bit_step(float* p, const void* g, qb_dtype gdt, int64_t n, uint8_t* m, uint8_t* v,
                            float* absmax_m, float* absmax_v, int32_t blocksize,
                            const qb_adamw_hparams* hp, void* stream);

/*
 * qb_multi_tensor_step -- qb_adamw8bit_step on `count` tensors in ONE kernel
 * launch (blocks never span tensors; the result equals a loop of single-tensor
 * calls, bit for bit).
 *   tensors   host array of `count` descriptors (read during the call only).
 *   ws        device workspace of qb_multi_tensor_workspace_bytes(count) bytes;
 *             the call copies a table of the tensors (pointers, sizes, first
 *             tile numbers, and a coarse index from tile ranges to tensors)
 *             into it on `stream`, so ws must not be reused by another stream
 *             until the step has run.
 * Tensors with n == 0 are skipped.  count == 0 is a no-op.
 * Under graph capture (this call and every other one that uploads a table: the
 * other multi-tensor and grouped calls, qb_prepare_code) the table goes into the
 * graph itself, as arguments of small kernels (3.5 KB each) that write it into ws,
 * so a replay reads no host memory; hp is the capture's as well.  Make one call on
 * the device before: the first one uploads the library's constant tables.
 */
qb_status qb_multi_tensor_step(const qb_tensor* tensors, int32_t count, qb_dtype gdt, int32_t blocksize,
                               const qb_adamw_hparams* hp, void* ws, size_t ws_bytes, void* stream);

/*
 * qb_multi_tensor_step_noalloc -- qb_multi_tensor_step without a workspace
 * argument, for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation).  The
 * tensor table goes into the library's own scratch: a device array of 384 KiB
 * that every GPU the library runs on holds until the process ends.  No device
 * memory is allocated or freed (no hipMalloc, hipFree or allocating library
 * call); host-side staging reuses per-thread buffers of the library.
 *   count     at most 4096 (QB_EWORKSPACE beyond).
 * Other arguments, the result (bit for bit) and the errors are those of
 * qb_multi_tensor_step.  Every call on one GPU shares that GPU's scratch,
 * which keeps the last call's table: calls that overlap in time on one GPU
 * (other streams, other host threads) race and must not be made; calls on
 * one stream are ordered and safe.
 */
qb_status qb_multi_tensor_step_noalloc(const qb_tensor* tensors, int32_t count, qb_dtype gdt, int32_t blocksize,
                                       const qb_adamw_hparams* hp, void* stream);

/*
 * qb_optimizer8bit_step -- one fused 8-bit step of optimizer hp->kind (see
 * qb_optimizer above) on one tensor.  Arguments as qb_adamw8bit_step, with
 * state1/absmax1 in place of m/absmax_m and state2/absmax2 in place of
 * v/absmax_v; state2 and absmax2 are ignored (may be NULL) for the one-state
 * kinds.
 * Parameter dtype pdt: QB_F32 (any gdt), or QB_F16 / QB_BF16 with gdt equal
 * to it (16-bit training without binary32 master weights, e.g. fp16 mixed
 * precision next to the 8-bit optimizer: "bitsandbytes - Quantização de LLM",
 * section Workflow 3).  A 16-bit parameter is widened to binary32 (exactly),
 * updated by the same binary32 formulas and rounded once, to nearest even,
 * back to its dtype; other pairs give QB_EUNSUPPORTED.  Fresh state: every code of 0.0 (127; 0 for a state in
 * QB_UDYN8), absmax 0.  A v_code other than QB_DYN8 or QB_UDYN8, or QB_UDYN8 for a kind without a never-negative
 * state, gives QB_EINVAL.  Invalid
 * hyperparameters for the kind (ranges above; lr, weight_decay >= 0) give
 * QB_EINVAL before anything is launched; the layer-wise kinds give
 * QB_EUNSUPPORTED (they run through qb_multi_tensor_optimizer_step).
 * 32-bit fallback: with absmax1 == NULL (and absmax2 == NULL) the states stay
 * binary32: state1 / state2 are float[n] arrays updated in place by the same
 * formulas, with no quantization.  This is the pages' policy for small or
 * chosen tensors (page "Py之bitsandbytes", sections 如果需要高精度的参数 and
 * 更改单个参数的位数: tensors under min_8bit_size elements, or marked 32-bit,
 * keep 32-bit state).  The multi-tensor step takes the same per tensor, so one
 * launch can mix 8-bit and 32-bit tensors.
 */
qb_status qb_optimizer8bit_step(const qb_optim_hparams* hp, void* p, qb_dtype pdt, const void* g, qb_dtype gdt,
                                int64_t n, uint8_t* state1, uint8_t* state2, float* absmax1, float* absmax2,
                                int32_t blocksize, void* stream);

/*
 * qb_multi_tensor_optimizer_step -- qb_optimizer8bit_step on `count` tensors in
 * one kernel launch (one parameter dtype pdt and gradient dtype gdt for all);
 * tensors, ws as for qb_multi_tensor_step, except that ws
 * holds qb_optimizer_workspace_bytes(hp, tensors, count, blocksize) bytes.
 * The layer-wise kinds (QB_LAMB, QB_LARS) take three launches on `stream`:
 * partial sums of the squared norms per group of optimizer tiles, one
 * workgroup per tensor that adds them in a fixed order and forms S, then the
 * fused step; the partial sums and the S of every tensor live in ws.
 */
qb_status qb_multi_tensor_optimizer_step(const qb_optim_hparams* hp, const qb_tensor* tensors, int32_t count,
                                         qb_dtype pdt, qb_dtype gdt, int32_t blocksize, void* ws, size_t ws_bytes,
                                         void* stream);

/*
 * qb_paged_optimizer_step -- the multi-tensor 8-bit step with the optimizer
 * states held in host memory: the paged 8-bit optimizer of page
 * "bitsandbytes - Quantização de LLM", section Workflow 3 (optimizer
 * "paged_adamw_8bit"), for models whose states do not fit beside the weights.
 * Each tensor is cut into pages of page_params parameters; per page the
 * state codes and absmax are copied to a device staging slot, the fused step
 * runs on the page, and the states are copied back.  Two staging slots and
 * two internal copy streams (host to device, device to host; default priority)
 * overlap the copies of neighbouring pages with the step of the current one.
 * The result equals qb_multi_tensor_optimizer_step on device-resident states,
 * bit for bit (the same kernel per block).
 *   tensors      as for qb_multi_tensor_optimizer_step, with p and g in device
 *                memory and m, v, absmax_m, absmax_v in pinned host memory
 *                (hipHostMalloc, or torch's pin_memory); 8-bit states only.
 *   page_params  parameters per page: a positive multiple of blocksize.
 *   ws           device staging of qb_paged_workspace_bytes(page_params,
 *                blocksize) bytes, 16-byte aligned.
 * Kinds: every element-wise kind (QB_ADAMW .. QB_RMSPROP); the layer-wise ones
 * give QB_EUNSUPPORTED (their norms need a whole tensor before any page moves).
 * Ordering: the call's work starts after the work already on `stream` and
 * `stream` waits for the last copy back, so later work on `stream` sees the
 * updated parameters and states.  Calls on one device share the internal
 * streams and events, so they must not be made from several host threads at
 * once; the states of a call must not be touched by the host until `stream`
 * has passed the call, and consecutive calls on the same states should use
 * the same `stream`.
 */
qb_status qb_paged_optimizer_step(const qb_optim_hparams* hp, const qb_tensor* tensors, int32_t count, qb_dtype pdt,
                                  qb_dtype gdt, int32_t blocksize, int64_t page_params, void* ws, size_t ws_bytes,
                                  void* stream);

/* Device staging bytes of qb_paged_optimizer_step: two slots, each with two
 * code pages of page_params bytes and two absmax pages, 256-byte aligned.
 * 0 if page_params is not a positive multiple of a valid blocksize. */
size_t qb_paged_workspace_bytes(int64_t page_params, int32_t blocksize);

/*
 * User codes.  The pages list three 8-bit quantization types, quantile,
 * linear and dynamic, and a fast quantile estimation (page "Py之bitsandbytes",
 * section 1).  Besides the built-in dynamic code, a block-wise 8-bit
 * quantization can use any 256-entry code held in a device table of
 * qb_code_table_bytes() bytes (16-byte aligned): the entries (256 floats at
 * the start), their exact decision thresholds (nearest entry; the midpoint of
 * two entries is taken in binary64; a tie goes to the entry of smaller
 * magnitude, between equal magnitudes to the upper one), and an index of the
 * thresholds by 2^-11-wide bucket of the normalized value, so the encoder
 * searches only its value's bucket.  Write tables only through the two calls
 * below.
 *   qb_linear_code      host: the linear code k/127, k = -128..127 (returns 256).
 *   qb_prepare_code     host values[256] (finite, non-decreasing; else
 *                       QB_EINVAL) -> device table, copied on `stream`.
 *   qb_estimate_quantiles
 *                       device: the quantile code of x[n] straight into a
 *                       device table.  The quantiles at j/257 (j = 0..256) are
 *                       estimated over chunks of 4096 consecutive values, each
 *                       sorted on its own (the chunk's order statistic at
 *                       floor(j L / 257), L its length; -0 counts as +0): A_j is
 *                       the exact mean of the chunks' statistics, rounded once
 *                       to nearest-even binary64.  Entries = binary32 of
 *                       q_i / max|q| with q_i = (A_i + A_{i+1}) / 2 (binary64).
 *                       Deterministic, and independent of the order of the
 *                       chunks' additions.  averages: NULL, or device double[257]
 *                       (16-byte aligned) that receives A.  ws:
 *                       qb_quantile_workspace_bytes(n) bytes.  Three kernels.
 *   qb_quantize_code / qb_dequantize_code
 *                       as qb_quantize / qb_dequantize with 8-bit codes (codes:
 *                       n bytes) and no nesting, the code given by `table`.
 */
size_t    qb_code_table_bytes(void);
int32_t   qb_linear_code(float* out);
qb_status qb_prepare_code(const float* values, void* table, void* stream);
size_t    qb_quantile_workspace_bytes(int64_t n);
qb_status qb_estimate_quantiles(const void* x, qb_dtype xdt, int64_t n, void* table, double* averages, void* ws,
                                size_t ws_bytes, void* stream);
qb_status qb_quantize_code(const void* x, qb_dtype xdt, int64_t n, const void* table, int32_t blocksize,
                           uint8_t* codes, float* absmax, void* stream);
qb_status qb_dequantize_code(const uint8_t* codes, const float* absmax, const void* table, int32_t blocksize,
                             int64_t n, void* y, qb_dtype ydt, void* stream);

/* Workspace sizes (bytes) for qb_quantize with nesting, and for
 * qb_multi_tensor_step, qb_multi_tensor_optimizer_step and qb_multi_tensor_dequantize. */
size_t qb_dq_workspace_bytes(int64_t n, int32_t blocksize);
size_t qb_multi_tensor_workspace_bytes(int32_t count);

/* Workspace bytes of qb_multi_tensor_optimizer_step: qb_multi_tensor_workspace_bytes(count)
 * for the element-wise kinds; for the layer-wise kinds two tables of the
 * tensors (by optimizer tile and by norm group), 16 bytes per norm group (32
 * optimizer tiles of max(blocksize, 1024) elements of one tensor) and 4 bytes
 * per tensor.  0 when hp, tensors or a size is invalid. */
size_t qb_optimizer_workspace_bytes(const qb_optim_hparams* hp, const qb_tensor* tensors, int32_t count,
                                    int32_t blocksize);

/*
 * The row-wise layers: embedding lookup, layer norm, and the stable embedding
 * that joins them (page "Py之bitsandbytes", section 1, lists a stable embedding
 * layer next to the 8-bit optimizers: an embedding followed by layer norm, whose
 * table keeps 32-bit optimizer state).  Common to these calls:
 *   - Matrices are row-major and dense: a table [rows, dim], tokens [n, dim].
 *     Rows may begin at any element (dim may be odd); the arrays themselves are
 *     16-byte aligned.
 *   - Token ids: n int32 or int64 values (idt).  An id outside [0, rows) names
 *     no row: its output row is zero and it takes no gradient.  This serves
 *     padded batches (id -1) and shards of a vocabulary (ids shifted by the
 *     shard's first row).  With rows == 0 the table may be NULL.
 *   - Arithmetic, sums and statistics are binary32; each output is rounded once
 *     to its dtype.  Every sum is added in a fixed order: the same inputs give
 *     the same bits on every run.  NaN and infinities propagate as in the
 *     formulas: into the rows (and, for the sums over rows, columns) that they
 *     enter, into no others.
 *   - n == 0: the forward calls do nothing; the backward calls write the
 *     gradient of no tokens (zeros) unless they accumulate.
 *   - Outputs must not overlap inputs or each other.
 *   - accumulate (0 or 1): add the gradient to what the outputs hold (read in
 *     their dtype, added in binary32, rounded once) instead of overwriting them.
 *   - Workspaces: a *_workspace_bytes result never shrinks when n, rows or dim
 *     grows, so a workspace for the largest call serves every smaller one.
 *   - Limits: n, rows < 2^31; dim < 2^24; a table's gradient takes at most 2^30
 *     tokens and 2^26 rows.
 */

/*
 * qb_embedding -- y[t] = ydt(scale * table[ids[t]]): one binary32 multiply, one
 * rounding.
 *   table   [rows, dim] of dtype tdt.     ids  [n] of type idt.
 *   scale   finite (in binary32 too).     y    [n, dim] of dtype ydt.
 * One kernel.
 */
qb_status qb_embedding(const void* table, qb_dtype tdt, int64_t rows, int64_t dim, const void* ids, qb_index idt,
                       int64_t n, double scale, void* y, qb_dtype ydt, void* stream);

/*
 * qb_dequant_embedding -- qb_embedding with the table [rows, dim] held as
 * block-wise codes, as qb_quantize writes them for its rows * dim elements
 * (blocks may span rows; an odd dim begins every other row inside a byte):
 * y[t] = ydt(scale * w) with w the binary32 value of qb_dequantize, two rounded
 * multiplies.  Only the rows that ids name are decoded (the embedding of a
 * 4-bit model: page "Bitsandbytes", section Normal Float 4 (NF4)).
 *   codes, absmax, dq, code, blocksize   as for qb_dequantize (dq->ws is not used);
 *           the table has fewer than 2^31 blocks.
 * One kernel.  The first call on a device that needs the library's constant
 * tables uploads them: make one before capturing a graph.
 */
qb_status qb_dequant_embedding(const uint8_t* codes, const float* absmax, const qb_dq* dq, qb_code code,
                               int32_t blocksize, int64_t rows, int64_t dim, const void* ids, qb_index idt, int64_t n,
                               double scale, void* y, qb_dtype ydt, void* stream);

/*
 * qb_embedding_backward -- the gradient of the table,
 *   dtable[v] = scale * (sum of dy[t] over the tokens t with ids[t] = v),
 * zero for an id without tokens.  The tokens are sorted by id first, and each
 * row's sum runs over them in order.
 *   dy          [n, dim] of dtype gdt.
 *   padding_id  an id that takes no gradient (its row is zero, or left as it is
 *               with accumulate); -1 for none.
 *   dtable      [rows, dim] of dtype ddt, every row written (with accumulate:
 *               only the rows of ids that have tokens are read and written).
 *   ws          device workspace of qb_embedding_workspace_bytes(n, rows, dim)
 *               bytes, 16-byte aligned; holds nothing between calls, and must not
 *               be shared by calls that may overlap in time.
 * Up to three kernels on `stream` (one for up to 128 tokens, four for many
 * tokens of a table of over 256000 rows); no memory operations, so it may be
 * captured.  Every id is read by 256 workgroups or more: 2^20 tokens of rows of 8
 * elements take 0.6 ms, of which the time grows with the tokens.
 */
qb_status qb_embedding_backward(const void* dy, qb_dtype gdt, const void* ids, qb_index idt, int64_t n, int64_t rows,
                                int64_t dim, double scale, int64_t padding_id, int32_t accumulate, void* dtable,
                                qb_dtype ddt, void* ws, size_t ws_bytes, void* stream);
size_t qb_embedding_workspace_bytes(int64_t n, int64_t rows, int64_t dim);

/*
 * qb_layer_norm -- per row x of n rows of dim elements
 *   mean = sum x / dim,  var = sum (x - mean)^2 / dim,  rstd = 1 / sqrt(var + eps),
 *   y = xdt((x - mean) * rstd * gamma + beta).
 *   x, y         [n, dim] of dtype xdt.
 *   gamma, beta  [dim] of dtype wdt, each may be NULL (ones, zeros).  wdt is
 *                QB_F32 or xdt (else QB_EUNSUPPORTED).
 *   eps          finite and positive, a normal number in binary32 too (at least 2^-126).
 *   mean, rstd   [n] fp32 out, each may be NULL; qb_layer_norm_backward takes them.
 * One kernel.
 */
qb_status qb_layer_norm(const void* x, qb_dtype xdt, int64_t n, int64_t dim, const void* gamma, const void* beta,
                        qb_dtype wdt, double eps, void* y, float* mean, float* rstd, void* stream);

/*
 * qb_layer_norm_backward -- with h = (x - mean) * rstd and g = dy * gamma:
 *   dx = rstd * (g - (sum g) / dim - h * (sum g h) / dim)   per row,
 *   dgamma = sum over rows of dy * h,  dbeta = sum over rows of dy.
 *   dy, x, dx      [n, dim] of dtype xdt.      mean, rstd  [n] as qb_layer_norm wrote them.
 *   gamma          [dim] of dtype wdt, or NULL (ones).
 *   dx, dgamma, dbeta   each may be NULL (not wanted); dgamma, dbeta [dim] of
 *                  dtype wdt.
 *   accumulate     applies to dgamma and dbeta; dx is overwritten.
 *   ws             device workspace of qb_layer_norm_workspace_bytes(n, dim)
 *                  bytes, 16-byte aligned; needed for dgamma or dbeta only.
 * Two kernels (dx alone: one; rows over 16384 elements: three).
 */
qb_status qb_layer_norm_backward(const void* dy, const void* x, qb_dtype xdt, int64_t n, int64_t dim,
                                 const void* gamma, qb_dtype wdt, const float* mean, const float* rstd, void* dx,
                                 void* dgamma, void* dbeta, int32_t accumulate, void* ws, size_t ws_bytes,
                                 void* stream);
size_t qb_layer_norm_workspace_bytes(int64_t n, int64_t dim);

/*
 * qb_stable_embedding -- layer norm of an embedding's rows in one kernel:
 * y[t] = ydt(layer_norm(scale * table[ids[t]])), the lookup in binary32 (not
 * rounded in between).  Arguments as qb_embedding and qb_layer_norm; wdt is
 * QB_F32 or tdt, and dim at most 16384 (else QB_EUNSUPPORTED).  The row of an id
 * outside the table is zero (beta is not added).
 */
qb_status qb_stable_embedding(const void* table, qb_dtype tdt, int64_t rows, int64_t dim, const void* ids,
                              qb_index idt, int64_t n, double scale, const void* gamma, const void* beta, qb_dtype wdt,
                              double eps, void* y, qb_dtype ydt, void* stream);

/*
 * qb_stable_embedding_backward -- the gradients of qb_stable_embedding.  The
 * tokens of an id v share their row and its statistics, so with S_v = sum of
 * dy[t] over them, h the normalized row and g = S_v * gamma:
 *   dtable[v] = scale * rstd * (g - (sum g) / dim - h * (sum g h) / dim),
 *   dgamma = sum over ids of S_v * h,  dbeta = sum over ids of S_v.
 * The statistics are taken anew from the table, which must hold what the
 * forward call read.
 *   padding_id   an id whose table row takes no gradient (its tokens still
 *                count in dgamma and dbeta); -1 for none.
 *   dgamma, dbeta   [dim] of dtype wdt, each may be NULL.
 *   ws           device workspace of qb_stable_embedding_workspace_bytes(n, rows,
 *                dim) bytes, as for qb_embedding_backward.
 * Other arguments as qb_embedding_backward and qb_stable_embedding.  Up to five
 * kernels (two for up to 128 tokens, six where qb_embedding_backward takes four).
 */
qb_status qb_stable_embedding_backward(const void* dy, qb_dtype gdt, const void* table, qb_dtype tdt, int64_t rows,
                                       int64_t dim, const void* ids, qb_index idt, int64_t n, double scale,
                                       const void* gamma, qb_dtype wdt, double eps, int64_t padding_id,
                                       int32_t accumulate, void* dtable, qb_dtype ddt, void* dgamma, void* dbeta,
                                       void* ws, size_t ws_bytes, void* stream);
size_t qb_stable_embedding_workspace_bytes(int64_t n, int64_t rows, int64_t dim);

/*
 * The 4-bit layers: the product of qb_dequant_matmul with what a layer does to it in its
 * epilogue (the layers whose weights the pages hold in 4 bits: page "Quantize 🤗 Transformers
 * models", section Using NF4), and the gradients that fine-tuning through
 * frozen 4-bit weights takes (page "bitsandbytes - Quantização de LLM", section on QLoRA;
 * page "Bitsandbytes", section QLoRA: Hesaplama veri türü).  Common to these calls:
 *   - W is the weight [N, K] as qb_dequantize gives it in the compute dtype xdt; codes,
 *     absmax, dq, code, blocksize as for qb_dequant_matmul.  x, y and every other [M, .]
 *     array is row-major and dense, of dtype xdt, 16-byte aligned.
 *   - K is a positive multiple of 32; K, N < 2^21; M < 2^31.  M == 0 is a no-op (but see the
 *     bias's gradient).
 *   - Products of two xdt values are summed in binary32, in an order of the kernel's own that
 *     depends on the sizes alone (the same bits on every run); bias, activation, product and
 *     residual are binary32 too, and each output is rounded once.  NaN and infinities
 *     propagate as in the formulas, into the rows that they enter; activations and their
 *     derivatives are their limits at the infinities, and NaN at NaN.
 *   - Outputs must not overlap inputs or each other, unless said otherwise.
 *   - ws: device workspace, 16-byte aligned, of the *_workspace_bytes size (0: none, ws may be
 *     NULL), which never shrinks when M, K or N grows: the weights in the compute dtype (none for
 *     a gradient of up to 48 rows in a 16-bit type, 32 MiB or little more up to 64), a gradient's
 *     dz, and up to 80 MiB for partial sums of products split over their length.  It holds nothing
 *     between calls and must not be shared by calls that may overlap in time (two captured
 *     graphs that run at once among them).
 *   - No memory operations, so the calls may be captured; the first call on a device that
 *     needs the library's constant tables uploads them: make one before.
 */
typedef enum {
    QB_ACT_NONE = 0,
    QB_ACT_RELU = 1,          /* max(z, 0), derivative 0 at 0 */
    QB_ACT_GELU = 2,          /* z P(z), P the normal distribution */
    QB_ACT_GELU_TANH = 3,     /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    QB_ACT_SILU = 4           /* z / (1 + e^-z) */
} qb_act;

/* A 4-bit weight of a gated block: a plain one gives absmax and leaves c2, absmax2, offset
 * NULL; a nested one gives these (the qb_dq fields) and absmax NULL. */
typedef struct {
    const uint8_t* codes;
    const float*   absmax;
    const uint8_t* c2;
    const float*   absmax2;
    const float*   offset;
} qb_weight;

/*
 * qb_dequant_linear -- z = x W^T + bias,  y = act(z) + residual.
 *   x         [M, K].
 *   bias      [N] of dtype bdt (QB_F32 or xdt, else QB_EUNSUPPORTED), or NULL.
 *   residual  [M, N], or NULL; may be y itself.
 *   z         [M, N] out, or NULL: the pre-activation, which the gradient takes.
 *   y         [M, N] out.
 * Up to 64 rows (any number with K = 32) one kernel reads the codes and no workspace is needed.
 * Beyond, the workspace is needed, and one kernel does it all where an estimate from the sizes
 * favours it; else the weights are dequantized into ws and multiplied from there (two to four
 * kernels).  N == 0 is a no-op.
 * Without bias, activation and residual it is the product of qb_dequant_matmul, by other kernels and
 * with other last bits: faster up to 64 rows (16 rows of 4096 inputs and 11008 outputs in bf16 13 us
 * and 20) and from 512 on (4096 rows 315 and 503); in between qb_dequant_matmul, which never needs a
 * workspace, is mostly as fast or faster (128 rows 49 and 31).
 */
qb_status qb_dequant_linear(const void* x, qb_dtype xdt, int64_t M, int64_t K, const uint8_t* codes,
                            const float* absmax, const qb_dq* dq, qb_code code, int32_t blocksize, int64_t N,
                            const void* bias, qb_dtype bdt, qb_act act, const void* residual, void* z, void* y,
                            void* ws, size_t ws_bytes, void* stream);
size_t qb_dequant_linear_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N);

/*
 * qb_dequant_linear_backward -- dz = dy act'(z),  dx = dz W,  dbias = sum over rows of dz.
 *   dy      [M, N] (the residual's gradient is dy itself).
 *   z       [M, N] as qb_dequant_linear wrote it; not looked at for QB_ACT_NONE.
 *   dx      [M, K] out, dz [M, N] out (the gradient that an adapter beside W takes), dbias [N]
 *           of dtype bdt (QB_F32 or xdt) out: each may be NULL (not wanted).
 *   accumulate   dbias is added to what it holds (in binary32, rounded once); with M == 0 it
 *           is left as it is, and zero otherwise.
 * dz is rounded to xdt before it is multiplied by W (the matrix instructions take
 * that type; for binary32 nothing is rounded); dbias sums the unrounded dz.  N >= 1.
 * The workspace is needed for dx and dbias.  Up to four kernels: dz and the weights
 * transposed, the product in one or two launches, its pieces joined or dbias.  Few rows are
 * multiplied by weights transposed on the way, without a copy of them.
 */
qb_status qb_dequant_linear_backward(const void* dy, const void* z, qb_dtype xdt, int64_t M, int64_t K,
                                     const uint8_t* codes, const float* absmax, const qb_dq* dq, qb_code code,
                                     int32_t blocksize, int64_t N, qb_act act, void* dx, void* dz, void* dbias,
                                     qb_dtype bdt, int32_t accumulate, void* ws, size_t ws_bytes, void* stream);
size_t qb_dequant_linear_backward_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N);

/*
 * qb_dequant_gated -- the gated feed-forward block's two projections, activation and product:
 *   g = x Wg^T,  u = x Wu^T,  y = act(g) u.
 *   gate, up           host: the weights Wg, Wu [N, K]; both plain or both nested (else
 *                      QB_EUNSUPPORTED); code, blocksize and blocksize2 (nested only) are shared.
 *   gate_out, up_out   [M, N] out, each may be NULL: g and u, which the gradient takes.
 *   y                  [M, N] out.
 * Kernels and workspace as for qb_dequant_linear.  N == 0 is a no-op.
 */
qb_status qb_dequant_gated(const void* x, qb_dtype xdt, int64_t M, int64_t K, const qb_weight* gate,
                           const qb_weight* up, qb_code code, int32_t blocksize, int32_t blocksize2, int64_t N,
                           qb_act act, void* gate_out, void* up_out, void* y, void* ws, size_t ws_bytes, void* stream);
size_t qb_dequant_gated_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N);

/*
 * qb_dequant_gated_backward -- dg = dy u act'(g),  du = dy act(g),  dx = dg Wg + du Wu.
 *   dy, gate_out, up_out   [M, N]: the gradient of y; g and u as qb_dequant_gated wrote them.
 *   dx          [M, K] out, dgate, dup [M, N] out: each may be NULL (not wanted).
 * dg and du are rounded to xdt before they are multiplied.  N >= 1.  The workspace is needed
 * for dx.  Up to four kernels: dg, du and the weights transposed, the product in one or two
 * launches, its pieces joined.
 */
qb_status qb_dequant_gated_backward(const void* dy, const void* gate_out, const void* up_out, qb_dtype xdt, int64_t M,
                                    int64_t K, const qb_weight* gate, const qb_weight* up, qb_code code,
                                    int32_t blocksize, int32_t blocksize2, int64_t N, qb_act act, void* dx,
                                    void* dgate, void* dup, void* ws, size_t ws_bytes, void* stream);
size_t qb_dequant_gated_backward_workspace_bytes(qb_dtype xdt, int64_t M, int64_t K, int64_t N);

/*
 * The global gradient norm, and clipping by it, before an optimizer step (the 8-bit
 * optimizers are drop-in replacements in a training loop: page "bitsandbytes - Quantização de
 * LLM", section Workflow 3).
 * One gradient: n values of its own dtype at g and (clipping) out, which is g or overlaps no
 * gradient.  Both may begin at any element, as views of a bucket do.  n < 2^33; n == 0 is
 * skipped.
 */
typedef struct {
    const void* g;
    void*       out;
    int64_t     n;
    qb_dtype    dtype;
} qb_grad;

/*
 * qb_multi_tensor_grad_norm -- norm[0] = sqrt(sum over gradients and elements of g^2): squares
 * and sums in binary64, rounded once to binary32.
 *   grads   host array of `count` descriptors (read during the call only).
 *   norm    [1] fp32 out, 16-byte aligned; 0 without gradients.
 *   ws      device workspace of qb_multi_tensor_grad_norm_workspace_bytes(count) bytes, 16-byte
 *           aligned; holds nothing between calls.
 * The same bits on every run.  One launch per 224 gradients (neighbours in memory, of one
 * type and in order, count as one) and one more (a few small gradients: one in all); no memory
 * operations, so the call may be captured.  Several ranks' norms of their own gradients make the
 * global one as sqrt(sum of norm^2).
 */
qb_status qb_multi_tensor_grad_norm(const qb_grad* grads, int32_t count, float* norm, void* ws, size_t ws_bytes,
                                    void* stream);
size_t qb_multi_tensor_grad_norm_workspace_bytes(int32_t count);

/*
 * qb_multi_tensor_clip_grads -- out = g * s with s = min(1, max_norm / (norm[0] + 1e-6)), in
 * binary64 and rounded to binary32; one binary32 product, rounded once.
 *   max_norm   finite, >= 0.
 *   norm       device [1] fp32, 16-byte aligned: what qb_multi_tensor_grad_norm wrote, or a
 *              norm over several ranks.  An infinite norm makes s 0, a NaN s NaN.
 * With s = 1 and out = g a gradient is left as it is (not read).  Gradients must not overlap
 * each other, nor appear twice.  One launch per 150 gradients (neighbours count as
 * one); may be captured.
 */
qb_status qb_multi_tensor_clip_grads(const qb_grad* grads, int32_t count, double max_norm, const float* norm,
                                     void* stream);

/*
 * qb_codebook -- host: copy the decode table of `code` (indexed by stored code)
 * into out (256 floats for DYN8 and UDYN8, 16 for NF4/FP4).  Returns the entry
 * count, or -1 for a bad code or a failed table build.
 */
int32_t qb_codebook(qb_code code, float* out);

/*
 * qb_encoder_table -- host: the encoder's bucket table, for inspection and
 * tests.  Each entry is two uint32 words {threshold bits, payload}:
 *   DYN8: 2 x 1409 entries, those of n >= 0 and then those of n < 0; bucket
 *         b = (clamp(bits(|n|), 2^-22, 1.0) >> 17) - (bits(2^-22) >> 17), plus
 *         1409 for n < 0; the code is payload + (n >= threshold).
 *   UDYN8: 2817 entries, n >= 0; bucket b = (clamp(bits(n), 2^-22, 1.0) >> 16)
 *         - (bits(2^-22) >> 16); the code is payload + (n >= threshold).
 *   NF4/FP4: bucket b = n*16 + 16 rounded once to the nearest integer, ties
 *         to even (0..32); NF4: the code is payload + (n >= threshold); FP4:
 *         byte 0 of payload if n < threshold, else byte 1.
 * Copies at most `capacity` entries (2*capacity words) into out and returns the
 * table's entry count, or -1 on error.
 */
int32_t qb_encoder_table(qb_code code, uint32_t* out, int32_t capacity);

/* Static text for a status code. */
const char* qb_status_string(qb_status s);

#ifdef __cplusplus
}
#endif

#endif /* QB_H */
