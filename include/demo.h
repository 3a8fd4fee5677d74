/*
 * demo.h -- C ABI of libdemo: the DeMo / FlexDeMo optimizer step on one
 * accelerator's parameter shard, for AMD Instinct MI355X (gfx950).
 *
 * The operations follow the DeToNATION paper notes (AAAI 2026), section
 * "FlexDeMo optimizer", Algorithm 1, steps 3-7:
 *   3. momentum accumulation      m <- beta*m + g
 *   4. extract fast components    q  (DCT-II + top-k, or another scheme)
 *   5. error feedback             m <- m - q
 *   6. synchronise q over the replication group R (the payload exchange)
 *   7. parameter update           theta <- theta - lr*Q
 * and the same notes' "Replication schemes" table (DeMo, Random, Striding,
 * DiLoCo) and "Sign function" section (sign before sync: ternary values,
 * chunk size 32).  The DeMo abstract ("DeMo: Decoupled Momentum
 * Optimization") fixes the transform as a fast orthonormal DCT with top-k.
 *
 * Conventions shared by every entry point
 *  - All tensors are flat fp32 arrays of n_elems elements in device memory
 *    (hipMalloc / PyTorch allocations), 16-byte aligned, with
 *    1 <= n_elems <= DEMO_MAX_ELEMS (2^36, 256 GB per array; larger shards
 *    are split by the caller, for instance at tensor boundaries, each part
 *    with its own chunk_offset).  The caller owns all memory; the library
 *    never allocates, frees or keeps pointers.
 *  - A chunk is 32 consecutive elements; C = ceil(n_elems/32) chunks; the last
 *    chunk is zero-padded inside the kernels and padded outputs are dropped.
 *  - Calls are asynchronous on the given HIP stream (hipStream_t passed as
 *    void*, NULL = the default stream).  A configuration or argument error is
 *    returned synchronously as a negative code and nothing is launched; a
 *    launch failure returns DEMO_EHIP; device faults surface at the caller's
 *    next synchronisation.  No C++ exception crosses the ABI.
 *  - Buffers passed to one call must not overlap.  Calls on distinct buffers
 *    may be made from several threads.
 *  - Values are not checked: NaN or infinity in an input propagates into that
 *    chunk's outputs (which slots a DCT chunk with a NaN transform selects is
 *    unspecified); every memory access stays inside the buffers described.
 */
#ifndef DEMO_H
#define DEMO_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DEMO_ABI_VERSION 1
#define DEMO_CHUNK 32
#define DEMO_MAX_ELEMS ((uint64_t)1 << 36)

/* Replication schemes ("Replication schemes" table of the DeToNATION notes). */
enum {
    DEMO_SCHEME_DCT = 0,    /* DeMo: DCT-II per chunk, top-k, indices sent      */
    DEMO_SCHEME_RANDOM = 1, /* k random positions from a shared seed, no indices */
    DEMO_SCHEME_STRIDE = 2, /* every (32/k)-th position, offset = step mod 32/k  */
    DEMO_SCHEME_DILOCO = 3  /* everything once every `period` steps, else nothing */
};

/* Wire format of the slot values.  Sign before sync makes every value
 * ternary (-1, 0, +1); TERNARY packs it into two bit-planes, F16 / F32 store
 * it as a number (the notes compare fp16 and fp32 communication). */
enum { DEMO_VAL_TERNARY = 0, DEMO_VAL_F16 = 1, DEMO_VAL_F32 = 2 };

enum {
    DEMO_OK = 0,
    DEMO_EINVAL = -1,       /* bad configuration value, size or null pointer */
    DEMO_EALIGN = -2,       /* pointer or stride not aligned as required      */
    DEMO_EUNSUPPORTED = -3, /* valid request this library does not implement  */
    DEMO_EHIP = -4,         /* HIP launch / runtime error                     */
    DEMO_EABI = -5          /* cfg->abi_version != DEMO_ABI_VERSION           */
};

typedef struct demo_cfg {
    uint32_t abi_version;  /* must be DEMO_ABI_VERSION */
    uint32_t scheme;       /* DEMO_SCHEME_* */
    uint32_t chunk;        /* must be 32 ("chunk size = 32", notes' hyper-parameters) */
    uint32_t k;            /* DCT: top-k in [1,32]; RANDOM: n in [1,32];
                              STRIDE: n with 32 % n == 0; DILOCO: ignored (32) */
    uint32_t period;       /* DILOCO: sync when step % period == period-1; >= 1 */
    uint32_t sign;         /* 1 = sign before sync: every slot carries sign(value)
                              in {-1, 0, +1} ("Sign function" section).
                              0 = slots carry the selected values themselves:
                              the DCT coefficient (DCT) or u (others), stored
                              as fp32 or as fp16 rounded to nearest even with
                              subnormals kept; needs value_fmt F16 or F32
                              (TERNARY with sign 0 is DEMO_EINVAL). */
    uint32_t value_fmt;    /* DEMO_VAL_* */
    float beta;            /* momentum decay, finite (offset 28) */
    float lr;              /* learning rate eta, finite (offset 32) */
    uint32_t reserved;     /* must be 0; keeps seed at its natural offset 40 */
    uint64_t seed;         /* shared selection seed (RANDOM) */
    uint64_t step;         /* optimizer step t, from 0 (hashed mod 2^32) */
    uint64_t chunk_offset; /* global chunk index of this shard's element 0 */
} demo_cfg;

/*
 * Payload of one replica for one step: one byte buffer whose regions start at
 * multiples of 256 bytes, in the order IDX, NZ, NEG (TERNARY) or IDX, VAL
 * (F16/F32); its size is rounded up to 256 bytes.  With k slots per chunk
 * (k = 32 for DILOCO) and G = ceil(C/64):
 *   IDX  uint8 [C][k]   DCT scheme only: chunk-local position of slot s of
 *                       chunk c at byte c*k+s; the k positions ascend.
 *   NZ   uint64 [G][k]  TERNARY: bit b of word g*k+s is set iff slot s of chunk
 *   NEG  uint64 [G][k]  64g+b is nonzero / negative.  Value = NZ ? (NEG ? -1 :
 *                       +1) : 0.  NEG without NZ and bits of chunks >= C are 0
 *                       (the encoder never sets them; the decoder reads a NEG
 *                       bit without its NZ bit as 0 and index bytes mod 32).
 *   VAL  fp16|fp32 [C][k] F16/F32: value of slot s of chunk c at entry c*k+s:
 *                       +-1 or 0 with sign 1, the value itself with sign 0.
 * RANDOM, STRIDE and DILOCO carry no IDX: every replica recomputes the slot
 * positions from (seed, step, chunk) and slots follow ascending position.
 */
typedef struct demo_layout {
    uint64_t idx_off, idx_bytes;
    uint64_t nz_off, neg_off, plane_bytes;
    uint64_t val_off, val_bytes;
    uint64_t total_bytes; /* minimum stride between replicas */
} demo_layout;

/*
 * Decoupled AdamW (DeToNATION notes, "Decoupled AdamW": an AdamW variant whose
 * first and second moments are not synchronised).  The notes give no formula;
 * the reading implemented: both moments stay local and are never exchanged;
 * the first moment m = beta1*m + (1-beta1)*g (beta1 = demo_cfg.beta) takes the
 * momentum's place in the extraction, the payload and the error feedback of
 * demo_encode; v = beta2*v + (1-beta2)*g^2; the decode applies the exchanged
 * mean Q as AdamW applies its first moment:
 *   theta -= lr * ((Q / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *                  + weight_decay * theta),   t = demo_cfg.step + 1.
 * The slots carry the selected values (demo_cfg.sign 0, value_fmt F16 or
 * F32): with the sign before sync ("Sign function" section) Q is a mean of
 * ternary values that has lost the first moment's magnitude, and dividing it
 * by sqrt(v) would scale the step by 1/|g|, so demo_cfg.sign 1 is DEMO_EINVAL
 * for both AdamW calls.  beta1 (demo_cfg.beta) and beta2 in [0, 1); eps >= 0
 * and weight_decay finite; reserved must be 0.
 */
typedef struct demo_adamw {
    float beta2;
    float eps;
    float weight_decay;
    uint32_t reserved;
} demo_adamw;

/* Library version; equals DEMO_ABI_VERSION. */
int demo_abi_version(void);

/* Static string for a DEMO_* code (never NULL). */
const char *demo_strerror(int code);

/* Payload layout of one replica for n_elems >= 1 elements under cfg.
 * Host-only (touches no device).  Returns DEMO_OK or a negative code. */
int demo_payload_layout(const demo_cfg *cfg, uint64_t n_elems, demo_layout *out);

/*
 * Encoder side of one optimizer step (Algorithm 1 steps 3-5 and the sender
 * half of step 6):
 *   u = beta*momentum + grad; per chunk select slots (DCT: the k largest |DCT-II
 *   coefficients|, equal magnitudes to the lower index; RANDOM / STRIDE: the
 *   shared positions; DILOCO: all 32 on a sync step, none otherwise);
 *   q = inverse DCT of the selected coefficients (DCT) or u on the selected
 *   positions (others); momentum <- u - q; payload <- the slot values, as
 *   ternary signs or (sign 0) the values themselves, and positions for DCT.
 * grad      [n_elems] read-only.
 * momentum  [n_elems] updated in place.
 * payload_out  >= demo_payload_layout(...).total_bytes bytes, 16-byte aligned.
 *           On a DILOCO non-sync step it is not written.
 * q_out     [n_elems] or NULL: receives q (diagnostics; costs 4 bytes/element).
 */
int demo_encode(const demo_cfg *cfg, uint64_t n_elems, const float *grad, float *momentum,
                void *payload_out, float *q_out, void *hip_stream);

/*
 * Receiver side (Algorithm 1 steps 6-7): payloads holds R >= 1 replicas'
 * payloads for this step, replica r at payloads + r*stride (own payload among
 * them; the layout an all-gather produces).  Per chunk the slot values are
 * summed over replicas into the slot positions, divided by R, taken back
 * through the inverse DCT (DCT scheme) and applied as params -= lr*Q.
 * On a DILOCO non-sync step nothing is read or written.
 * stride >= total_bytes and a multiple of 16.
 */
int demo_decode_apply(const demo_cfg *cfg, uint64_t n_elems, float *params, const void *payloads,
                      uint64_t stride, uint32_t R, void *hip_stream);

/*
 * demo_encode for Decoupled AdamW (see demo_adamw): moment1 [n_elems] is the
 * first moment (extracted from and updated in place like demo_encode's
 * momentum), moment2 [n_elems] the second moment, updated in place (also on
 * DiLoCo steps without a payload).  16-byte aligned; no argument may alias
 * another.  Same payload, codes and asynchrony as demo_encode.
 */
int demo_encode_adamw(const demo_cfg *cfg, const demo_adamw *adamw, uint64_t n_elems, const float *grad,
                      float *moment1, float *moment2, void *payload_out, float *q_out, void *hip_stream);

/*
 * demo_decode_apply for Decoupled AdamW: the same Q, applied with this
 * replica's second moment moment2 [n_elems] (read-only, 16-byte aligned, not
 * aliasing params) and weight decay, as stated at demo_adamw.  On a DILOCO
 * non-sync step nothing is read or written.
 */
int demo_decode_apply_adamw(const demo_cfg *cfg, const demo_adamw *adamw, uint64_t n_elems, float *params,
                            const float *moment2, const void *payloads, uint64_t stride, uint32_t R,
                            void *hip_stream);

/*
 * Receiver-side check of one replica's payload before demo_decode_apply: the
 * payload comes from another replica (the exchange of Algorithm 1 step 6 in
 * the DeToNATION notes), and this call counts, into *violations_out, every
 * violation of the format stated at demo_layout for this cfg and n_elems:
 * a NEG bit without its NZ bit (chunks c < C); each NZ or NEG bit of a chunk
 * c >= C; an IDX byte above 31; an IDX byte not above the previous slot's
 * (positions must ascend strictly); with cfg->sign 1 an F16/F32 value other
 * than -1, 0 or +1 (the ternary values of sign before sync); with cfg->sign 0
 * a value that is not finite.  0 means well formed.  A DILOCO step that sends
 * nothing has no payload: payload may be NULL and the count is 0.
 * payload: device buffer of at least demo_payload_layout's total_bytes,
 * 16-byte aligned, read-only.  violations_out: device uint64, 8-byte aligned,
 * written asynchronously on hip_stream (read it after synchronising); it must
 * not overlap the payload.  The count is cleared by a kernel, not a memset.
 */
int demo_payload_validate(const demo_cfg *cfg, uint64_t n_elems, const void *payload, uint64_t *violations_out,
                          void *hip_stream);

/*
 * Shared-seed slot positions of n_chunks chunks (global ids chunk_offset +
 * c, c < n_chunks): masks_out[c] bit j set iff chunk-local position j is
 * selected.  cfg->scheme RANDOM: k positions drawn without replacement by
 * Philox4x32-10 (Salmon et al., SC'11) keyed by `seed`, counter (chunk_lo,
 * chunk_hi, step_lo, (1 << 24) | i/4), draw i taking word i%4 w and picking
 * free position number floor(w*(32-i)/2^32) counted from bit 0.  STRIDE:
 * positions j % (32/k) == step % (32/k).  `seed` and `step` override
 * cfg->seed and cfg->step.  masks_out: device uint32 [n_chunks], 4-byte aligned;
 * 1 <= n_chunks <= DEMO_MAX_ELEMS / 32.
 */
int demo_random_select(const demo_cfg *cfg, uint64_t seed, uint64_t step, uint64_t n_chunks,
                       uint32_t *masks_out, void *hip_stream);

/*
 * The low-precision linear layer beside the optimizer step: a layer whose fp32
 * master weight is a piece of the shard, whose products run on 8-bit operands
 * with a scale for each block of 128 along the sum, and whose weight gradient
 * is added in fp32 to the gradient that demo_encode reads.
 *
 * Types of matrices that are not operands.
 */
enum { DEMO_DTYPE_F32 = 0, DEMO_DTYPE_F16 = 1, DEMO_DTYPE_BF16 = 2 };

/* 8-bit formats (OCP): e4m3 reaches 448 and has no infinity, e5m2 reaches
 * 57344. */
enum { DEMO_FMT_E4M3 = 0, DEMO_FMT_E5M2 = 1 };

#define DEMO_BLOCK 128
#define DEMO_BLOCK_MAX_K ((uint64_t)1 << 22) /* longest sum of a product */
#define DEMO_BLOCK_MAX_WORKSPACE ((uint64_t)64 << 20) /* no product needs more */

/*
 * Dropout from a counter: element e = 32*chunk_offset + i takes the 16-bit
 * half e % 2 of word (e % 8)/2 of Philox4x32-10 with key `seed` and counter
 * (e/8 mod 2^32, e/8 div 2^32, step mod 2^32, 2*2^24 + site), and is kept iff
 * that number is at least T = floor(65536 p + 1/2); kept values are scaled by
 * 65536/(65536 - T) in fp32 (0 for T = 65536).  A shard that starts at
 * chunk_offset draws what the whole tensor draws there, and no draw of
 * demo_random_select with the same seed coincides with one of these.  The
 * configuration is read when the call is made: a call captured in a graph draws
 * the numbers of that step at every replay, so a graph that is replayed for
 * step after step has its dropouts outside, or is captured anew.
 */
typedef struct demo_dropout_cfg {
    uint32_t abi_version;  /* must be DEMO_ABI_VERSION */
    float p;               /* probability of dropping, in [0, 1], taken to the nearest multiple of 2^-16 */
    uint32_t site;         /* which dropout of the model, below 2^24 */
    uint32_t reserved;     /* must be 0 */
    uint64_t seed;
    uint64_t step;
    uint64_t chunk_offset; /* global chunk index of element 0 */
} demo_dropout_cfg;

/*
 * An operand of the product: `rows` rows of codes with a pitch of the next
 * multiple of 128 bytes (codes behind the last column are 0), then at
 * scale_off one byte e + 127 for each row and block of 128 columns, with a
 * pitch of the next multiple of 4 bytes.  A code c of that block stands for
 * c * 2^e.  Operands are 16-byte aligned.
 */
typedef struct demo_operand {
    uint64_t pitch;
    uint64_t scale_off;
    uint64_t scale_pitch;
    uint64_t total_bytes;
} demo_operand;

typedef struct demo_block_cfg {
    uint32_t abi_version;
    uint32_t fmt;   /* DEMO_FMT_* of the codes */
    uint32_t tile;  /* 0: a scale for 128 values of a row; 1: for a square of 128 x 128 */
    uint32_t dtype; /* DEMO_DTYPE_* of src */
} demo_block_cfg;

typedef struct demo_product_cfg {
    uint32_t abi_version;
    uint32_t fmt_a, fmt_b; /* DEMO_FMT_* of the operands */
    uint32_t dtype;        /* DEMO_DTYPE_* of c and addend */
} demo_product_cfg;

/*
 * y = residual + (kept ? x*scale : 0), in fp32 and rounded once to the
 * tensors' common type; residual may be NULL.  1 <= n_elems <= DEMO_MAX_ELEMS;
 * 16-byte aligned.  y may be x or residual themselves, else it overlaps
 * neither.  A dropped NaN or infinity leaves nothing.
 */
int demo_dropout(const demo_dropout_cfg *cfg, uint32_t dtype, uint64_t n_elems, const void *x, const void *residual,
                 void *y, void *hip_stream);

/*
 * The gradient of demo_dropout for x under the same cfg: dx = kept ? dy*scale
 * : 0, the mask drawn again (the residual's gradient is dy itself).  dx may be
 * dy.
 */
int demo_dropout_backward(const demo_dropout_cfg *cfg, uint32_t dtype, uint64_t n_elems, const void *dy, void *dx,
                          void *hip_stream);

/* Layout of an operand of rows x cols (cols is the summed axis); host-only.
 * Both sides at most 2^30, their product at most DEMO_MAX_ELEMS. */
int demo_block_layout(uint64_t rows, uint64_t cols, demo_operand *out);

/*
 * Quantises src [rows][cols] (row pitch ld elements, (rows - 1)*ld at most
 * 2^40, aligned to its element) into operand (rows x cols, blocks along the
 * columns) and into operand_t (cols x rows: the transposed matrix, blocks along
 * the rows) in one pass; one of the two may be NULL.  A block's scale is 2^e with the smallest e >=
 * -127 that keeps its largest finite magnitude within the format; codes are
 * rounded to nearest even; infinities and NaN become NaN codes.  With dropout
 * the values are first multiplied as demo_dropout_backward does (element i =
 * row*cols + column), in fp32 without a rounding between.
 */
int demo_block_quantize(const demo_block_cfg *cfg, uint64_t rows, uint64_t cols, const void *src, uint64_t ld,
                        const demo_dropout_cfg *dropout, void *operand, void *operand_t, void *hip_stream);

/* Bytes of workspace demo_block_matmul needs for these sizes (0 for most, at
 * most DEMO_BLOCK_MAX_WORKSPACE); host-only. */
int demo_block_workspace(const demo_product_cfg *cfg, uint64_t m, uint64_t n, uint64_t k, uint64_t *bytes);

/*
 * c[i][j] = addend[i][j] + drop(sum over k of a[i][k]*b[j][k]) for operands a
 * (m x k) and b (n x k): with X, W and dY the matrices of a layer Y = X W^T,
 *   Y  = product of X's operand and W's,
 *   dX = product of dY's operand and W's operand_t,
 *   dW = product of dY's operand_t and X's operand_t.
 * Sums are held in fp32 and the result is rounded once; the order of the sums
 * depends on the sizes only.  For an fp32 result products and sums have fp32's
 * precision for operand values between 2^-126 and 2^128; for 16-bit results
 * the hardware lines up eight neighbouring products of the sum at the largest
 * of them and keeps 13 binary places below it.  Root mean square, relative to
 * the result's, that is 1.5e-5 on normal values and up to 4.7e-5 where a few
 * channels are 20 times larger: at most 1/35 of the rounding to bf16, but 1/14
 * to 1/4 of the rounding to fp16.  An fp32 result is the way to have it exact.
 * addend may be NULL, or c itself with the same pitch (to add to a gradient);
 * dropout (NULL: none) applies to the product as demo_dropout does, element
 * i*n + j.  c and addend [m][n] with row pitches ldc and ld_addend in elements,
 * aligned to their element, (m - 1)*ldc and (m - 1)*ld_addend at most 2^40.
 * m, n at most 2^30, k at most DEMO_BLOCK_MAX_K (DEMO_EUNSUPPORTED beyond), each
 * of m*n, m*k and n*k at most DEMO_MAX_ELEMS.  c, from its first element to its
 * last with what lies between its rows, may overlap no other buffer of the
 * call, so neighbouring column slices of one matrix cannot be c and addend;
 * the workspace neither.  The workspace is written by the call and free again
 * when it has run: calls that may run at the same time (other streams, other
 * graphs) need one each.
 */
int demo_block_matmul(const demo_product_cfg *cfg, uint64_t m, uint64_t n, uint64_t k, const void *a, const void *b,
                      void *c, uint64_t ldc, const void *addend, uint64_t ld_addend,
                      const demo_dropout_cfg *dropout, void *workspace, uint64_t workspace_bytes, void *hip_stream);

/*
 * Root-mean-square norm in front of a linear layer, with the residual's
 * addition before it and the layer's 8-bit operand behind it:
 *   h = residual + x            in fp32, rounded to the tensors' type dtype,
 *   r = 1 / sqrt(mean over the row of h^2 + eps),
 *   y = (h * r) * weight        in fp32.
 */
#define DEMO_NORM_MAX_COLS 16384

typedef struct demo_norm_cfg {
    uint32_t abi_version; /* must be DEMO_ABI_VERSION */
    uint32_t dtype;       /* DEMO_DTYPE_* of x, residual, h and y, or of the gradients */
    uint32_t fmt;         /* DEMO_FMT_* of the operands' codes */
    float eps;            /* finite, at least 0 */
} demo_norm_cfg;

/*
 * x, residual, h, y: [rows][cols] with row pitches in elements, aligned to
 * their element ((rows - 1) * pitch at most 2^40); weight fp32 [cols], rstd
 * fp32 [rows], 4-byte aligned.  Each output may be NULL, not all of them:
 * h, y (rounded to dtype), rstd (r, which the backward pass reads), operand
 * (y as demo_block_quantize quantises an fp32 y: rows x cols, blocks along the
 * columns) and operand_t (cols x rows, blocks along the rows).  residual may be
 * NULL (h = x).  operand_t is made from h and r, so it needs rstd, and h where
 * there is a residual.  h and y may each be x or residual, in the same place
 * with the same pitch (y not x where operand_t is made from x); otherwise what
 * is written meets no other buffer of the call.  A row whose sum of squares
 * passes fp32's range has r = 0; with eps = 0 a row of zeros gives NaN.  The
 * squares are fp32's at the lower end too, which shows where eps is below 2^-126:
 * magnitudes below 2^-63 lose digits of r, and a row of 2^-75 or less has r
 * infinite.  1 <= cols <= DEMO_NORM_MAX_COLS (DEMO_EUNSUPPORTED beyond), rows at most
 * 2^30, rows * cols at most DEMO_MAX_ELEMS.
 */
int demo_rms_norm(const demo_norm_cfg *cfg, uint64_t rows, uint64_t cols, const void *x, uint64_t ld_x,
                  const void *residual, uint64_t ld_residual, const float *weight, void *h, uint64_t ld_h, void *y,
                  uint64_t ld_y, float *rstd, void *operand, void *operand_t, void *hip_stream);

/* Bytes of workspace demo_rms_norm_backward needs for these sizes where
 * dweight is wanted (at most DEMO_BLOCK_MAX_WORKSPACE); host-only. */
int demo_rms_norm_workspace(const demo_norm_cfg *cfg, uint64_t rows, uint64_t cols, uint64_t *bytes);

/*
 * The gradients, from dy (of y), the forward pass' h and rstd, and dresidual
 * (what reaches h from the residual's side; NULL: nothing): with n = h*r and g =
 * dy*weight
 *   dx      = r * (g - n * mean over the row of g*n) + dresidual,
 *   dweight = addend + sum over the rows of dy*n,
 * dx being the gradient of x and of residual alike.  Sums in an order that the
 * sizes fix: dx's in fp32, and it is rounded once to dtype; dweight's in fp32 over the
 * rows of a workgroup, then in fp64.  dweight is within 2^-24 * ((R + 9) sum |dy*n| +
 * |addend| + |dweight|), R = rows / 4096 up to 512 columns, / 2048 up to 1024, / 1024
 * up to 2048, / 512 up to 4096 and / 256 beyond, rounded up.  dweight fp32 [cols] (NULL:
 * not wanted, and no workspace is needed); addend fp32 [cols], NULL or dweight
 * itself (to add to a gradient) among others.  dx may be dy, h or dresidual, in
 * the same place with the same pitch.  cfg->fmt and cfg->eps are not used.  The
 * workspace is one call's at a time, as demo_block_matmul's.
 */
int demo_rms_norm_backward(const demo_norm_cfg *cfg, uint64_t rows, uint64_t cols, const void *dy, uint64_t ld_dy,
                           const void *h, uint64_t ld_h, const float *weight, const float *rstd,
                           const void *dresidual, uint64_t ld_dresidual, void *dx, uint64_t ld_dx, float *dweight,
                           const float *addend, void *workspace, uint64_t workspace_bytes, void *hip_stream);

/*
 * Between the backward pass and demo_encode: the norm of the whole gradient,
 * and its clipped copy.  The gradient is a list of tensors, each contiguous,
 * of one of the types, aligned to its element, possibly empty (data may then be
 * NULL).  The list is host memory, read when the call is made.
 */
#define DEMO_MAX_TENSORS 65536

typedef struct demo_tensor {
    void *data;
    uint64_t n_elems;  /* at most DEMO_MAX_ELEMS */
    uint32_t dtype;    /* DEMO_DTYPE_* */
    uint32_t reserved; /* must be 0 */
} demo_tensor;

/* Bytes of workspace demo_grad_norm needs for this list (0 for small ones, at
 * most DEMO_BLOCK_MAX_WORKSPACE); host-only. */
int demo_grad_workspace(uint32_t count, const demo_tensor *tensors, uint64_t *bytes);

/*
 * *sumsq = sum of the squares of all elements, in fp64 in an order that the
 * list fixes (a tensor that stands in it twice counts twice; 0 for nothing).
 * sumsq: device double, 8-byte aligned.  Where the gradient is spread over
 * shards, add the shards' sums up before demo_grad_clip.
 */
int demo_grad_norm(uint32_t count, const demo_tensor *tensors, double *sumsq, void *workspace,
                   uint64_t workspace_bytes, void *hip_stream);

/*
 * dst = c * src tensor by tensor, in fp32 and rounded once, with
 *   c = min(1, max_norm / (sqrt(*sumsq) + 1e-6)),
 * in fp64 and rounded once to fp32,
 * and *norm = sqrt(*sumsq) (device float; NULL: not wanted).  dst holds as many
 * tensors of the same sizes, each of src's type or fp32: pieces of the flat fp32
 * gradient that demo_encode reads, for instance.  dst NULL: in place, and then
 * a gradient within max_norm is neither read nor written.  A tensor of dst may
 * be the same one of src (type too); otherwise what is written meets nothing
 * else.  max_norm >= 0; at infinity c is 1 for every norm but NaN.  At any other
 * limit infinities in the gradient make c 0 (and 0 * infinity is NaN); a NaN makes
 * all of it NaN at every limit: a caller that skips such steps reads *norm.
 */
int demo_grad_clip(uint32_t count, const demo_tensor *src, const demo_tensor *dst, const double *sumsq,
                   double max_norm, float *norm, void *hip_stream);

/*
 * The same linear layer on 4-bit operands: e2m1 codes (OCP microscaling; 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 and their negatives) with a power of two for each block of
 * 32 along the sum.
 */
#define DEMO_MX_BLOCK 32

typedef struct demo_mx_cfg {
    uint32_t abi_version; /* must be DEMO_ABI_VERSION */
    uint32_t tile;  /* quantiser: 0: a scale for 32 values of a row; 1: for a square of 32 x 32; else 0 */
    uint32_t dtype; /* DEMO_DTYPE_* of src, dst, or c and addend */
    uint32_t reserved; /* must be 0 */
} demo_mx_cfg;

/*
 * Layout of a 4-bit operand of rows x cols (cols is the summed axis);
 * host-only: rows of codes with a pitch of the next multiple of 256 codes, two
 * in a byte, the even column in the low half (codes behind the last column are
 * 0), then at scale_off one byte e + 127 for each row and block of 32 columns,
 * with a pitch of the next multiple of 16 bytes.  A code c of that block stands
 * for c * 2^e, whatever the code for NaN where the byte is 255.  Operands are
 * 16-byte aligned.  Sizes as for demo_block_layout.
 */
int demo_mx_layout(uint64_t rows, uint64_t cols, demo_operand *out);

/*
 * demo_block_quantize to 4-bit operands: src [rows][cols] into operand and its
 * transposed matrix into operand_t, in one pass; one of the two may be NULL.
 * A block's scale is 2^e with the smallest e >= -127 that keeps its largest
 * magnitude within 6 * 2^e; codes are rounded to nearest even.  The format has
 * neither infinity nor NaN: a block with one of them has the scale byte 255 and
 * stands for NaN as a whole.  With dropout the values are first multiplied as
 * demo_dropout_backward does, in fp32 without a rounding between.  At most 2^24
 * - 1 squares of 128 x 128, padding counted (DEMO_EUNSUPPORTED beyond).
 */
int demo_mx_quantize(const demo_mx_cfg *cfg, uint64_t rows, uint64_t cols, const void *src, uint64_t ld,
                     const demo_dropout_cfg *dropout, void *operand, void *operand_t, void *hip_stream);

/* The values that an operand stands for, rounded once to dst's type: dst
 * [rows][cols], row pitch ld elements, aligned to its element. */
int demo_mx_dequantize(const demo_mx_cfg *cfg, uint64_t rows, uint64_t cols, const void *operand, void *dst,
                       uint64_t ld, void *hip_stream);

/* Bytes of workspace demo_mx_matmul needs for these sizes (0 for most, at most
 * DEMO_BLOCK_MAX_WORKSPACE); host-only. */
int demo_mx_workspace(const demo_mx_cfg *cfg, uint64_t m, uint64_t n, uint64_t k, uint64_t *bytes);

/*
 * demo_block_matmul on 4-bit operands a (m x k) and b (n x k):
 *   c[i][j] = addend[i][j] + drop(sum over k of a[i][k]*b[j][k]),
 * with its rules for addend, dropout, pitches, overlaps, sizes and workspace.
 * Products are exact and sums are held in fp32 for every type of the result, with
 * subnormal numbers.  A part of a sum that passes fp32's range is infinite, and a
 * result NaN where such parts have both signs; what reaches below 2^-149 is lost.
 */
int demo_mx_matmul(const demo_mx_cfg *cfg, uint64_t m, uint64_t n, uint64_t k, const void *a, const void *b, void *c,
                   uint64_t ldc, const void *addend, uint64_t ld_addend, const demo_dropout_cfg *dropout,
                   void *workspace, uint64_t workspace_bytes, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* DEMO_H */
