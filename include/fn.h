/*
 * fn.h -- FusedNormalization on AMD Instinct MI355X (gfx950): the C ABI of libfn.so.
 *
 * One memory pass turns a batch of uint8 NHWC images into per-channel
 * normalized (x/255 - mean)/std tensors in fp32 or fp16, with a per-sample
 * random horizontal flip and a per-sample RandomErasing rectangle applied in
 * the same pass.  The operation is the FusedNormalization step of the page
 * "(11) FusedNormalization: fusing the last steps of data augmentation into one
 * memory pass" (tech-renaissance.cn/blog/?p=487):
 *   - section 5: ToTensor (x/255), RandomHorizontalFlip, Normalize
 *     ((v - mean)/std) and RandomErasing fused into one execute() call; the
 *     flip is drawn first, then the rectangle;
 *   - section 6: fp32 output or fp16 output (round to nearest even);
 *   - section 10: every random number is a pure function of (seed, offset)
 *     through the Philox counter-based generator;
 *   - section 12: the rectangle sampler (gate, up to 10 attempts of area
 *     fraction and log aspect ratio, rounding, acceptance, corner).
 * The page runs this per image on CPU threads; here one call processes a
 * whole batch on one GPU.  The operators of a model's 8-bit linear layer
 * follow: a norm that quantises, row quantisation, the product of the codes and
 * the norm's gradients.  Then those of a network in training: dropout, layer norm
 * and the softmax cross entropy of a linear head, each with its gradients.
 *
 * Conventions for every entry point:
 *   - Pointers named *_dev are device memory (hipMalloc or a PyTorch CUDA
 *     tensor); pointers without the suffix are host memory.  All memory is
 *     owned by the caller; the library keeps no pointer after returning and
 *     allocates nothing.
 *   - `stream` is a hipStream_t cast to void* (NULL = the null stream).  Work
 *     is enqueued asynchronously on it; the call does not synchronize.  The
 *     caller keeps the buffers alive until the stream has finished the work.
 *   - Return value: FN_OK (0) on success, or a negative FN_E* code.  On an
 *     error nothing is enqueued and no output byte is written; the message is
 *     available from fn_last_error() on the calling thread.
 *   - All entry points are thread-safe and reentrant (no global state beyond
 *     the thread-local error message).
 */
#ifndef FN_H
#define FN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FN_OK 0
#define FN_EINVAL (-1)    /* an argument is out of its documented domain           */
#define FN_EOVERFLOW (-2) /* a size does not fit the index arithmetic              */
#define FN_EHIP (-3)      /* the HIP runtime reported an error (message kept)      */

/* Output element type. */
#define FN_OUT_FP32 0 /* 4-byte IEEE binary32                                       */
#define FN_OUT_FP16 1 /* 2-byte IEEE binary16, rounded to nearest even (page sec. 6) */
#define FN_OUT_FP16_PAD4 2 /* binary16 with 4 channels per pixel: channels c < C as
                              FN_OUT_FP16, channels C..3 are +0 -- the page's
                              mixed-precision layout (page sec. 8) */
#define FN_OUT_BF16 3 /* 2-byte bfloat16, rounded to nearest even: the row and
                         product operators below, not the pixel operations     */

/* One sample's random decisions (32 bytes, all int32):
 *   flip        1 if the image is mirrored left-right, else 0;
 *   erase       1 if the rectangle below is zeroed, else 0;
 *   i, j        row and column of the rectangle's top-left corner, in output
 *               (post-flip) coordinates; 0 when erase is 0;
 *   eh, ew      rectangle height and width in pixels (0 < eh < H, 0 < ew < W
 *               when erase is 1; 0 when erase is 0);
 *   attempt     index 0..9 of the accepted attempt, or -1 when none was;
 *   words_used  generator words the sample consumed (see fn_params). */
typedef struct {
    int32_t flip, erase, i, j, eh, ew, attempt, words_used;
} fn_sample_params;

/*
 * fn_fused_normalize -- the whole operation on a batch (page sec. 5, 6, 10, 12).
 *
 *   in_u8_dev   N*H*W*C bytes, image n at byte offset n*H*W*C, row-major
 *               (h, w, c) inside an image (NHWC, contiguous).  Any alignment.
 *   N           images (N = 0: validate the arguments, enqueue nothing).
 *   H, W, C     image height, width, channels; 1 <= C <= 4; H*W <= 2^24.
 *   mean, std   host arrays of C floats; std[c] > 0, all finite.
 *   flip_p      probability in [0, 1] of mirroring an image (page sec. 5
 *               uses 0.5); 0 draws no flip word.
 *   erase_p     probability in [0, 1] of trying to erase (page sec. 12); 0
 *               draws no gate word.
 *   scale_min/max  area-fraction range, 2^-30 <= scale_min <= scale_max <= 1
 *               (page sec. 4 defaults 0.02, 0.33).
 *   ratio_min/max  aspect-ratio range, 2^-30 <= ratio_min <= ratio_max <= 2^30
 *               (page sec. 4 defaults 0.3, 3.3).
 *   seed        64-bit generator key; sample n draws from the stream keyed by
 *               (seed, n), so the result does not depend on the launch shape.
 *   out_dtype   FN_OUT_FP32, FN_OUT_FP16 or FN_OUT_FP16_PAD4.
 *   out_dev     N*H*W*OC elements of out_dtype in NHWC order, OC = C (no
 *               padding) or 4 for FN_OUT_FP16_PAD4, aligned to the element
 *               size (4 or 2 bytes); must not overlap the input.
 *               Speed only: a 16-byte aligned out_dev whose rows are whole
 *               16-byte vectors (W*OC*element size a multiple of 16) takes
 *               the fastest kernel; other outputs take a flat layout at
 *               about two thirds of its rate; input rows that leave room
 *               for only one tile per compute unit in LDS (about 80 KB on
 *               MI355X) take slower paths.  Results are the same bits.
 *
 * Result, per sample n with P = fn_params(seed, ...)[n]:
 *   out[n,h,w,c] = +0                                 if P.erase and
 *                                                     P.i <= h < P.i+P.eh and P.j <= w < P.j+P.ew
 *                = (x/255 - mean_c)/std_c             otherwise,
 *   x = in[n, h, P.flip ? W-1-w : w, c].  The pixel order is mirrored, the
 *   channel order inside a pixel is kept (page sec. 7).  The value is
 *   computed as page sec. 7 writes it, x*mul_c - sub_c, with mul_c =
 *   1/(255 std_c) and sub_c = mean_c/std_c each carried as a pair of fp32
 *   numbers (their double values split into high and low parts):
 *   fma(x, mul_hi, -sub_hi) + fma(x, mul_lo, -sub_lo).  fp32 output is within
 *   2e-6 of the correctly rounded value for |value| < 8 and within about one
 *   fp32 ulp of it relative to the value; fp16 output is that fp32 value
 *   rounded to nearest even, within one fp16 ulp of the correctly rounded
 *   fp32 value.  With FN_OUT_FP16_PAD4, out[n,h,w,c] for c < C is the fp16
 *   value above and out[n,h,w,c] = +0 for C <= c < 4.
 *
 * Errors: FN_EINVAL for a null pointer (N > 0), a device pointer that is not
 * device memory or whose buffer is shorter than the sizes above, a misaligned
 * out_dev, any scalar outside its domain, an unknown out_dtype, or
 * overlapping in/out;
 * FN_EOVERFLOW for N*H*W*C*4 beyond int64 or H*W > 2^24; FN_EHIP if the
 * launch fails.
 */
int fn_fused_normalize(const uint8_t* in_u8_dev, int64_t N, int32_t H, int32_t W, int32_t C,
                       const float* mean, const float* std, float flip_p, float erase_p,
                       float scale_min, float scale_max, float ratio_min, float ratio_max,
                       uint64_t seed, int32_t out_dtype, void* out_dev, void* stream);

/*
 * fn_params -- the per-sample random decisions alone (page sec. 5 execute(),
 * sec. 10 uniform()/randint(), sec. 12 generate_erase_rect()).
 *
 * Writes params_dev[n] for n in [0, N): exactly the decisions
 * fn_fused_normalize takes with the same (seed, H, W, probabilities, ranges).
 * Arguments as for fn_fused_normalize; params_dev holds N fn_sample_params.
 *
 * Generator: word k of sample n is output k%4 of Philox4x32-10 (Salmon et al.,
 * SC'11) with counter (k/4 low, k/4 high, n low, n high) and key (seed low,
 * seed high).  A word becomes u = (word >> 8) * 2^-24.  Words are consumed in
 * order: the flip word (if flip_p > 0; flip iff u < flip_p), the gate word (if
 * erase_p > 0; try iff u < erase_p), then per attempt an area-fraction word
 * and a log-ratio word, and after an accepted attempt a row word and a column
 * word (randint(lo, hi) = lo + floor(word * (hi-lo+1) / 2^32), inclusive).
 * The attempt arithmetic is fp32 with one rounding per operation; exp, sqrt
 * and division are correctly rounded; sides are rounded half away from zero.
 *
 * Errors: as fn_fused_normalize (params_dev must be device memory of at
 * least N*32 bytes).
 */
int fn_params(uint64_t seed, int64_t N, int32_t H, int32_t W, float flip_p, float erase_p,
              float scale_min, float scale_max, float ratio_min, float ratio_max,
              fn_sample_params* params_dev, void* stream);

/*
 * fn_fused_normalize_ex -- fn_fused_normalize on a strided source, with the
 * sample numbering offset.
 *
 *   in_u8_dev        the first byte read: channel 0 of pixel (0, 0) of image 0.
 *   in_row_stride    bytes from one source row to the next, >= W*C.
 *   in_image_stride  bytes from one source image to the next, >= 0 (images
 *                    may overlap; 0 reads the same image N times).
 *                    Row h of image n starts at
 *                    in_u8_dev + n*in_image_stride + h*in_row_stride and
 *                    holds W*C bytes.  With W*C and H*W*C this is
 *                    fn_fused_normalize's layout.  The page's per-image
 *                    entry point takes such a row stride (page sec. 5,
 *                    execute(input_ptr, width, height, input_stride, ...)),
 *                    and the crop that precedes the fused step in the
 *                    operator chain (page sec. 4) is then a pointer offset:
 *                    pass the window's top-left pixel and the full image's
 *                    strides.
 *   first_sample_id  >= 0; sample n of this call draws from stream
 *                    (seed, first_sample_id + n) (page sec. 10: decisions
 *                    are a function of seed and offset only).  Splitting a
 *                    batch into slices [a, b) called with first_sample_id =
 *                    a reproduces the whole batch's result bit for bit, on
 *                    one device or several.
 *   all other arguments as fn_fused_normalize; the output is compact.
 *
 * Errors: as fn_fused_normalize, plus FN_EINVAL for in_row_stride < W*C,
 * in_image_stride < 0 or first_sample_id < 0, and FN_EOVERFLOW when the
 * input span (N-1)*in_image_stride + (H-1)*in_row_stride + W*C exceeds
 * 2^62.  The whole span must lie in one device allocation.
 */
int fn_fused_normalize_ex(const uint8_t* in_u8_dev, int64_t in_row_stride,
                          int64_t in_image_stride, int64_t N, int32_t H, int32_t W, int32_t C,
                          const float* mean, const float* std, float flip_p, float erase_p,
                          float scale_min, float scale_max, float ratio_min, float ratio_max,
                          uint64_t seed, int64_t first_sample_id, int32_t out_dtype,
                          void* out_dev, void* stream);

/* fn_params_ex -- fn_params for samples first_sample_id .. first_sample_id +
 * N - 1: params_dev[n] is sample first_sample_id + n's record, the decisions
 * fn_fused_normalize_ex takes with the same first_sample_id.  Errors as
 * fn_params, plus FN_EINVAL for first_sample_id < 0. */
int fn_params_ex(uint64_t seed, int64_t first_sample_id, int64_t N, int32_t H, int32_t W,
                 float flip_p, float erase_p, float scale_min, float scale_max, float ratio_min,
                 float ratio_max, fn_sample_params* params_dev, void* stream);

/* ------------------------------------------------------------------------ */
/* The 8-bit linear layer: a norm that quantises, the quantisation of rows,   */
/* the product of the codes, and the norm's gradients for training.           */
/*                                                                            */
/* A matrix is `rows` rows of contiguous elements, a row stride (in elements) */
/* apart.  Bases and strides need the element's own alignment only.  An       */
/* input's stride may be 0 (one row for all) or anything above; an output's   */
/* is at least the row's length.  No output may overlap another buffer of the */
/* call, except as each operator allows; column ranges of one buffer, with    */
/* the same stride, do not overlap.  dtype is FN_OUT_FP32, FN_OUT_FP16 or     */
/* FN_OUT_BF16.  Sums, statistics and scales are fp32 (integer sums 32-bit).  */
/* Speed only: rows that start at multiples of 16 bytes are fastest.          */
/*                                                                            */
/* Errors of all: FN_EINVAL for a null, misaligned, too short or overlapping  */
/* buffer, a negative size or stride, an output stride shorter than a row, an */
/* unknown dtype; FN_EOVERFLOW for width > 2^30, rows > 2^40 or a span beyond */
/* 2^62 bytes; FN_EHIP if a launch fails.  rows = 0 (M = 0 or N = 0) enqueues */
/* nothing and needs no buffers, unless stated.                               */
/* ------------------------------------------------------------------------ */

/*
 * fn_rms_norm -- h = x + residual and its root-mean-square norm, per row:
 *   h     = x + residual, rounded to dtype and stored in sum_dev (h = x and
 *           nothing stored when residual_dev and sum_dev are NULL);
 *   rstd  = 1 / sqrt(mean(h^2) + eps), stored if rstd_dev is not NULL (the
 *           backward pass takes it);
 *   out   = h * rstd * weight, rounded to dtype.
 * weight_dev: `width` elements of dtype.  eps > 0.  sum_dev and out_dev may
 * each be exactly x_dev or residual_dev (same stride), not each other.
 * A row that holds a NaN or an infinity, or whose squares overflow fp32, has
 * rstd = NaN and is NaN throughout.
 */
int fn_rms_norm(const void* x_dev, int64_t x_stride, const void* residual_dev,
                int64_t residual_stride, const void* weight_dev, int64_t rows, int32_t width,
                float eps, int32_t dtype, void* sum_dev, int64_t sum_stride, void* out_dev,
                int64_t out_stride, float* rstd_dev, void* stream);

/*
 * fn_rms_norm_q8 -- the same norm with its output in 8 bits and a scale per
 * row.  With t_j = h_j * weight_j and A = max |t_j|, each operation rounded to
 * fp32:
 *   code_j = rint(t_j * (127 * (1 / A))), ties to even, in -127..127;
 *   scale  = A * rstd / 127,   so that   out_j ~ code_j * scale.
 * rstd is common to a row and cancels in its codes, which therefore depend on
 * no order of summation: they are the same bits on every run and device.
 * A code is the nearest to 127 t_j / A but for the three roundings: a value
 * within 127 * 3 * 2^-24 of half way between two codes may get either.  In
 * 16-bit types many lie exactly half way (normally distributed rows of 768: one
 * code in 3,000 of bf16, one in 11,000 of fp16 is not the one that ties to
 * even of 127 t_j / A would give).
 * (Where A < 2^-100, t and A are scaled by 2^100 first.)  A row of zeros has
 * codes 0 and scale 0; a row without a norm (above), or with a NaN or an
 * infinity among its t_j, has codes 0 and scale NaN.
 * sum_dev may be exactly x_dev or residual_dev.
 */
int fn_rms_norm_q8(const void* x_dev, int64_t x_stride, const void* residual_dev,
                   int64_t residual_stride, const void* weight_dev, int64_t rows, int32_t width,
                   float eps, int32_t dtype, void* sum_dev, int64_t sum_stride,
                   int8_t* codes_dev, int64_t codes_stride, float* scales_dev, float* rstd_dev,
                   void* stream);

/* fn_quantize_rows -- codes and scales of rows as they are: fn_rms_norm_q8's
 * formulas with t = x and scale = A / 127.  For weights (a row per output
 * channel) and for activations that come from no norm. */
int fn_quantize_rows(const void* x_dev, int64_t x_stride, int64_t rows, int32_t width,
                     int32_t dtype, int8_t* codes_dev, int64_t codes_stride, float* scales_dev,
                     void* stream);

/*
 * fn_rms_norm_backward -- the gradients of fn_rms_norm.  dout is the gradient
 * of out; dsum (or NULL) the gradient that reaches the stored sum by another
 * way; h the sum (x if there was no residual) and rstd what the forward pass
 * stored.  With n = h * rstd and g = dout * weight:
 *   dx      = rstd * (g - n * mean(g * n)) + dsum, rounded to dtype: the
 *             gradient of x and of the residual alike;
 *   dweight = sum over the rows of dout * n, fp32, overwritten, joined in an
 *             order that the sizes alone fix (no atomics).  rows = 0 writes
 *             zeros.
 * A row's mean is summed in an order that the width, the type and rows and
 * dout_stride fix, but not the same for every row: 16-bit rows of odd width
 * from 2561 to 16384 at an odd dout_stride are added up from another first
 * element if their number is odd.  There dx of equal rows may differ by the
 * rounding of that sum; dweight does not depend on it.
 * dx_dev may be exactly dout_dev, h_dev or dsum_dev.  workspace_dev: at least
 * fn_rms_norm_backward_workspace(rows, width) bytes, 16-byte aligned, that no
 * other call in flight uses.  For a norm whose output was quantised, dout is
 * the gradient of code * scale, passed straight through the rounding.
 */
int fn_rms_norm_backward(const void* dout_dev, int64_t dout_stride, const void* h_dev,
                         int64_t h_stride, const void* weight_dev, const float* rstd_dev,
                         const void* dsum_dev, int64_t dsum_stride, int64_t rows, int32_t width,
                         int32_t dtype, void* dx_dev, int64_t dx_stride, float* dweight_dev,
                         void* workspace_dev, int64_t workspace_bytes, void* stream);

/* Writes to *bytes (host) the workspace that fn_rms_norm_backward needs. */
int fn_rms_norm_backward_workspace(int64_t rows, int32_t width, int64_t* bytes);

/*
 * fn_matmul_q8 -- the product of two matrices of codes:
 *   out[m, n] = a_scales[m] * b_scales[n] * sum_k a[m, k] * b[n, k] + bias[n]
 * a is M x K (tokens), b is N x K (output channels), out M x N of out_dtype.
 * The sum is exact (32-bit integers; K <= 131071, else FN_EOVERFLOW; codes may
 * be -128..127); the rest is ((sum * a_scale) * b_scale) + bias in fp32, one
 * rounding per operation, then one rounding to out_dtype.  bias_dev may be
 * NULL.  K = 0 gives bias (or 0), and needs no a_dev and b_dev.
 */
int fn_matmul_q8(const int8_t* a_dev, int64_t a_stride, const float* a_scales_dev,
                 const int8_t* b_dev, int64_t b_stride, const float* b_scales_dev,
                 const float* bias_dev, int64_t M, int64_t N, int32_t K, int32_t out_dtype,
                 void* out_dev, int64_t out_stride, void* stream);

/* ------------------------------------------------------------------------ */
/* Dropout and layer norm, with their gradients: what stands between the     */
/* linear layers of a network in training.  Matrices, strides, types,         */
/* overlaps and errors as for the 8-bit linear layer.                         */
/* ------------------------------------------------------------------------ */

/*
 * fn_dropout -- out = residual + dropout(x), or dropout(x) if residual_dev is
 * NULL, in fp32 with one rounding to dtype at the end.  The mask is never
 * stored: it is a function of (seed, first_row + row, column), so the gradient
 * of x is the same call on the gradient of out (without a residual, or with
 * another gradient of x to add), and a batch split into calls with matching
 * first_row gives the bits of the whole one.
 *   dropout_p   the probability of an element's loss, in [0, 1]; it counts in
 *               steps of 1/65536: D = rint(65536 dropout_p) in 65536 are lost,
 *               and the others multiplied by 65536 / (65536 - D), rounded to
 *               fp32, so that the expectation is exact.
 *   first_row   >= 0; row r draws from stream (seed, first_row + r).  Give
 *               every use of a step rows, or a seed, of its own.
 * Column j of a row has 16 bits of block j / 8 of the row's stream: half j % 2
 * (the low one first) of output (j % 8) / 2 of Philox4x32-10 with counter
 * (j / 8, 2^31, row low, row high) and key (seed low, seed high).  It is lost
 * if they are below D.  fn_params' words have counters below these, so the
 * streams have none in common.  A lost element is +0 (plus the residual)
 * whatever x holds there, NaN included.
 * out_dev may be exactly x_dev or residual_dev (same stride).
 * Errors: also FN_EINVAL for dropout_p outside [0, 1] or first_row < 0,
 * FN_EOVERFLOW for first_row + rows beyond 2^63 - 1.
 */
int fn_dropout(const void* x_dev, int64_t x_stride, const void* residual_dev,
               int64_t residual_stride, int64_t rows, int32_t width, float dropout_p, uint64_t seed,
               int64_t first_row, int32_t dtype, void* out_dev, int64_t out_stride, void* stream);

/*
 * fn_layer_norm -- h = residual + dropout(x) and its layer norm, per row:
 *   h    = fn_dropout's result (x + residual for dropout_p = 0), rounded to
 *          dtype and stored in sum_dev; h = x and sum_dev = NULL without a
 *          residual and dropout;
 *   mean = sum(h) / width,  rstd = 1 / sqrt(sum((h - mean)^2) / width + eps),
 *          stored if mean_dev and rstd_dev are not NULL (the backward pass
 *          takes both);
 *   out  = (h - mean) * rstd * weight + bias, rounded to dtype.
 * weight_dev and bias_dev: `width` elements of dtype, or NULL for ones and
 * zeros.  eps > 0.  sum_dev and out_dev may each be exactly x_dev or
 * residual_dev, not each other.  A row that holds a NaN or an infinity, or
 * whose sum or squares overflow fp32, is NaN throughout, with rstd = NaN.
 */
int fn_layer_norm(const void* x_dev, int64_t x_stride, const void* residual_dev,
                  int64_t residual_stride, const void* weight_dev, const void* bias_dev,
                  int64_t rows, int32_t width, float eps, float dropout_p, uint64_t seed,
                  int64_t first_row, int32_t dtype, void* sum_dev, int64_t sum_stride,
                  void* out_dev, int64_t out_stride, float* mean_dev, float* rstd_dev,
                  void* stream);

/*
 * fn_layer_norm_backward -- the gradients of fn_layer_norm.  dout is the
 * gradient of out; dsum (or NULL) the gradient that reaches h by another way;
 * h the sum (x if there was none), mean and rstd what the forward pass stored.
 * With n = (h - mean) * rstd and g = dout * weight:
 *   dh      = rstd * (g - mean(g) - n * mean(g * n)) + dsum: the gradient of h
 *             and of the residual, rounded to dtype;
 *   dx      = dropout(dh) with the forward pass's mask, from dh in fp32 and
 *             rounded once.  dx_dev is NULL for dropout_p = 0, where dh is the
 *             gradient of x too;
 *   dweight = sum over the rows of dout * n,  dbias = sum over the rows of
 *             dout: fp32, overwritten, joined in an order that the sizes alone
 *             fix (no atomics); either may be NULL.  rows = 0 writes zeros.
 * dh_dev and dx_dev may each be exactly dout_dev, h_dev or dsum_dev, not each
 * other.  workspace_dev: at least fn_layer_norm_backward_workspace(rows, width)
 * bytes, 16-byte aligned, that no other call in flight uses.
 */
int fn_layer_norm_backward(const void* dout_dev, int64_t dout_stride, const void* h_dev,
                           int64_t h_stride, const void* weight_dev, const float* mean_dev,
                           const float* rstd_dev, const void* dsum_dev, int64_t dsum_stride,
                           int64_t rows, int32_t width, float dropout_p, uint64_t seed,
                           int64_t first_row, int32_t dtype, void* dh_dev, int64_t dh_stride,
                           void* dx_dev, int64_t dx_stride, float* dweight_dev, float* dbias_dev,
                           void* workspace_dev, int64_t workspace_bytes, void* stream);

/* Writes to *bytes (host) the workspace that fn_layer_norm_backward needs. */
int fn_layer_norm_backward_workspace(int64_t rows, int32_t width, int64_t* bytes);

/* ------------------------------------------------------------------------ */
/* The softmax cross entropy of a linear head over many classes, whose logits */
/* are never kept, and its gradients.                                         */
/*                                                                            */
/* x is rows x width (features), weight classes x width, both of dtype with   */
/* any row stride; bias `classes` fp32 numbers or NULL.  With                 */
/*   z[t, v] = sum_k x[t, k] weight[v, k] + bias[v]                           */
/* in fp32:                                                                   */
/*   lse[t]  = log(sum_v exp(z[t, v])),                                       */
/*   loss[t] = lse[t] - (1 - smoothing) z[t, y_t] - smoothing mean_v z[t, v]. */
/* targets are 64-bit; a row whose target y_t lies outside 0..classes-1 (-100, */
/* say) is ignored: its loss and its gradients are zero, whatever its logits   */
/* (but its features still meet dweight's zeros, so they have to be finite).   */
/* smoothing lies in [0, 1].  A class of bias -infinity is left out:           */
/* probability 0, and a loss of +infinity for rows that want it (with smoothing */
/* every row does).  A row with a NaN or +infinity among its logits, or all     */
/* classes left out, has a NaN loss.                                           */
/*                                                                            */
/* In large fp32 products an operand is taken as three bf16 numbers, which     */
/* hold all of its digits if it is 2^-100 or more; one that is infinite, or    */
/* that bf16 rounds to infinity, gives NaN logits.                             */
/*                                                                            */
/* Operands are read in place if in_place(x), which is that the base, the      */
/* stride and the width are multiples of 16 bytes and the stride is at least   */
/* the width and below 2^23 bytes; others are copied to the workspace first.   */
/* For x this is a matter of speed only.  A weight that is copied may be taken */
/* in other pieces than one in place, and the sums in another order: the       */
/* results then differ by the rounding of the sums.                            */
/*                                                                            */
/* Errors: FN_EINVAL as for the other matrices, for classes or width < 1,      */
/* smoothing outside [0, 1] or a workspace that is too short; FN_EOVERFLOW     */
/* for rows or classes > 2^28, width > 2^20, or a product of two of the three  */
/* > 2^36.                                                                     */
/* ------------------------------------------------------------------------ */

/*
 * fn_linear_cross_entropy -- the losses and lse (which the backward pass takes),
 * `rows` fp32 numbers each.  A loss is computed from differences from the largest
 * logit, not from lse, and keeps digits that a number of the logits' size has not.
 * Sums are fp32, in an order that the sizes, the type and whether weight is read
 * in place fix.  workspace_dev: at least fn_linear_cross_entropy_workspace(...)
 * bytes, 16-byte aligned, that no other call in flight uses.
 */
int fn_linear_cross_entropy(const void* x_dev, int64_t x_stride, const void* weight_dev,
                            int64_t weight_stride, const float* bias_dev,
                            const int64_t* targets_dev, int64_t rows, int64_t classes,
                            int32_t width, float smoothing, int32_t dtype, float* losses_dev,
                            float* lse_dev, void* workspace_dev, int64_t workspace_bytes,
                            void* stream);

/*
 * fn_linear_cross_entropy_backward -- the gradients.  dlosses are the gradients
 * of the losses, dlosses_stride apart: 1, or 0 for one number for all rows.  With
 *   g[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - (1 - smoothing) [v = y_t]
 *                       - smoothing / classes)     (0 in an ignored row):
 *   dx = g weight, dweight = g^T x, rounded to dtype; dbias[v] = sum_t g[t, v]
 * in fp32.  All are overwritten; each may be NULL.  The logits are computed
 * again, a piece of the classes at a time, and g is rounded to dtype before its
 * products, as the matrix instructions take it (dbias comes before that); the
 * sums are fp32, in an order that the sizes, the type, whether weight is read in
 * place and whether both dx and dweight are wanted fix (no atomics).  In 16-bit
 * types g is scaled so that the largest finite |dloss| of a row that counts is 1
 * (bf16) or 2^14 (fp16, where probabilities down to 2^-28 then keep all their
 * digits in rows of that dloss), and its products back; an ignored row's dloss may
 * be anything.  rows = 0 writes zeros.
 */
int fn_linear_cross_entropy_backward(
    const float* dlosses_dev, int64_t dlosses_stride, const void* x_dev, int64_t x_stride,
    const void* weight_dev, int64_t weight_stride, const float* bias_dev,
    const int64_t* targets_dev, const float* lse_dev, int64_t rows, int64_t classes, int32_t width,
    float smoothing, int32_t dtype, void* dx_dev, int64_t dx_stride, void* dweight_dev,
    int64_t dweight_stride, float* dbias_dev, void* workspace_dev, int64_t workspace_bytes,
    void* stream);

/* Writes to *bytes (host) the workspace that fn_linear_cross_entropy
 * (backward_pass 0) or its gradients (1) need.  in_place_x, in_place_weight:
 * nonzero if the operand can be read in place, as above; 0 is always enough. */
int fn_linear_cross_entropy_workspace(int64_t rows, int64_t classes, int32_t width, int32_t dtype,
                                      int32_t in_place_x, int32_t in_place_weight,
                                      int32_t backward_pass, int64_t* bytes);

/* The message of the last nonzero return on the calling thread ("" if none).
 * The pointer stays valid until the next call on the same thread. */
const char* fn_last_error(void);

/* ------------------------------------------------------------------------ */
/* Test and measurement hooks.  Not part of the operation; exposed so tests  */
/* can check the building blocks exhaustively and the benchmark can measure  */
/* the operation's traffic alone.  Same conventions as above.                */
/* ------------------------------------------------------------------------ */

/* One erase attempt (page sec. 12) per index s in [0, count): from the area
 * word w_scale_dev[s] and the log-ratio word w_ratio_dev[s], writes the rounded
 * sides eh_dev[s], ew_dev[s] (-1 if beyond int32) and accepted_dev[s] (1 if
 * 0 < eh < H and 0 < ew < W).  Same domains as fn_params. */
int fn_test_erase_dims(const uint32_t* w_scale_dev, const uint32_t* w_ratio_dev, int64_t count,
                       int32_t H, int32_t W, float scale_min, float scale_max, float ratio_min,
                       float ratio_max, int32_t* eh_dev, int32_t* ew_dev, uint8_t* accepted_dev,
                       void* stream);

/* The correctly rounded fp32 operations the sampler uses, per index s:
 *   op 0: out[s] = RN32(exp(a[s]))   for |a[s]| <= 80;
 *   op 1: out[s] = RN32(sqrt(a[s]))  for positive normal a[s];
 *   op 2: out[s] = RN32(a[s] / b[s]) for positive normal a[s], b[s] whose
 *         quotient is a normal float.
 * Outside those domains the output is unspecified (but written, and the
 * kernel still ends normally).  b_dev may be NULL for ops 0 and 1. */
int fn_test_cr_ops(int32_t op, const float* a_dev, const float* b_dev, int64_t count,
                   float* out_dev, void* stream);

/* The operation's traffic without its arithmetic, as the practical bandwidth
 * roof of the fused kernels: reads in_bytes from src_dev and writes every
 * byte zero-extended to `widen` bytes, in_bytes * widen bytes in all, as
 * 16-byte streaming stores.
 *   widen 2 (the fp16 operation's 1:2 read:write mix): the output is the
 *     input widened to 16 bits, in order.
 *   widen 4 (the fp32 one's 1:4 mix): per block of 256 input vectors of 16
 *     bytes starting at vector b (m = min(256, in_bytes/16 - b) vectors in
 *     the block), dword k of vector v, widened to four 32-bit values, is
 *     output vector 4b + k*m + (v - b).
 * in_bytes a multiple of 16; both pointers 16-byte aligned; no overlap.
 * Errors as above (FN_EINVAL for any other widen). */
int fn_test_stream(const void* src_dev, void* dst_dev, int64_t in_bytes, int32_t widen,
                   void* stream);

/* Measurement hook of the instrumented build libfn_timeline.so (the same
 * sources compiled with FN_TIMELINE=1): every later fused call whose tiles
 * kernel runs records, for each tile t < tiles, four 64-bit stamps of the
 * GPU's 100 MHz real-time clock at stamps_dev + 4 t: its work-group's start,
 * the end of staging (tile loaded and decisions drawn), its stores issued
 * (first wavefront) and its stores acknowledged (all wavefronts).  The
 * tile order is the kernel's own (tile t covers the t-th range of rows).
 * stamps_dev is a caller-owned device buffer of tiles * 32 bytes that must
 * outlive those calls; tiles = 0 stops recording.  Not thread-safe: one
 * setting per process.  The product library libfn.so returns FN_EINVAL. */
int fn_test_timeline(void* stamps_dev, int64_t tiles);

#ifdef __cplusplus
}
#endif

#endif /* FN_H */
