/*
 * mmq_q4g.h -- C ABI of the matrix-vector products of libmmq.so with 4-bit weights that carry one
 * scale, and optionally one zero, per group of values (q4_G), for 1 to 16 tokens: decoding with
 * weights of the plain group-scaled kind, beside the q4_K products of mmq.h.
 *
 *   w_jk = s_jg (v_jk - z_jg),  g = k / group,  v in 0..15,  z = 8 where the weights have no zeros
 *   y[i][j] = act( sum_k x_ik w_jk + bias_j ) + residual_ij
 *
 * Activations are float32, float16 or bfloat16 and are not quantized: every product x v is exact in
 * float32, all sums are float32, and a result is rounded once, to the output's type. No sum over 128
 * values overflows, whatever finite values x has, for zeros in 0..16, and none over a row while its
 * partial sums are below 2^128 (float32 and bfloat16 x: 2^140). Products and sums below 2^-114 s are
 * exact to 2^-137 s each, s being the scale.
 *
 * The conventions of mmq.h hold: DEVICE pointers owned by the caller, 16-byte aligned, not
 * overlapping (but for a residual that is the output); `stream` is a hipStream_t; every argument is
 * validated on the host before anything is launched; nothing is allocated and nothing synchronizes;
 * results are deterministic; return values are mmq_status codes.
 */
#ifndef MMQ_Q4G_H
#define MMQ_Q4G_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum mmq_type { MMQ_F32 = 0, MMQ_F16 = 1, MMQ_BF16 = 2 };

#define MMQ_Q4G_MAX_TOKENS 16

typedef struct mmq_q4G_format {
  int32_t group;      /* values that share a scale: a multiple of 32, or K or more (one per row) */
  int32_t scale_type; /* enum mmq_type of scales and zeros: MMQ_F16 or MMQ_BF16 */
  int32_t zeros;      /* 1: zeros are given; 0: z = 8 */
  int32_t reserved;   /* must be 0 */
} mmq_q4G_format;

/* Bytes of repacked weights N x K: about N*K/2 and 2 (with zeros 4) per row and group. K % 32 == 0,
 * K <= 2^24, N <= 2^25, ceil(N/16) * ceil(K/128) < 2^24. Host only. */
int mmq_q4G_repacked_bytes(int64_t N, int64_t K, const mmq_q4G_format* format, size_t* bytes);

/*
 * repack_q4_G: w uint8 [N][K/2], value 2i of a row in the low and 2i + 1 in the high four bits of its
 * byte i; scales and zeros [N][ceil(K/group)] of scale_type (the last group of a row may be short;
 * zeros NULL without zeros; a zero need not be a whole number) -> the kernels' layout. Run once per
 * weight matrix. Precondition of the products: finite scales and zeros.
 */
int repack_q4_G(const void* w, const void* scales, const void* zeros, int64_t N, int64_t K,
                const mmq_q4G_format* format, void* w_rep, void* stream);

typedef struct mmq_q4G_epilogue {
  const float* bias;    /* [N], added before the activation, or NULL */
  const void* residual; /* [M][N] of y's type, added after it, or NULL; may be y itself */
  int32_t act;          /* enum mmq_act (mmq_layer.h) */
  int32_t reserved;     /* must be 0 */
} mmq_q4G_epilogue;

/*
 * mmq_q4G: y[M][N] of y_type from x[M][K] of x_type (row-major, any two of enum mmq_type) and w_rep
 * from repack_q4_G with the same N, K and format; epi may be NULL. 1 <= M <= 16. Precondition:
 * finite x (a token with an infinity or NaN gets unspecified values in its own row only).
 * Errors: MMQ_E_ARG (null or misaligned pointer, a type, format or epilogue out of range),
 *         MMQ_E_SHAPE (K % 32, M > 16, sizes too large, a group that is neither a multiple of 32 nor
 *         K or more), MMQ_E_LDS, MMQ_E_DEVICE, MMQ_E_HIP.
 */
int mmq_q4G(int64_t M, int64_t N, int64_t K, int32_t x_type, const void* x, const void* w_rep,
            const mmq_q4G_format* format, int32_t y_type, void* y, const mmq_q4G_epilogue* epi,
            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MMQ_Q4G_H */
