/*
 * saga_q4.h -- the decode step over a KV cache held in 4 bits.
 *
 * The calls of saga.h with the caches K and V replaced by a saga_q4_cache:
 * rows are quantised as they are written (saga_q4_append_kv), can be read
 * back (saga_q4_read_kv), and are attended in place by full attention
 * (saga_q4_dense_decode), the Atop-N step (saga_q4_decode_step) and its
 * refresh (saga_q4_refresh_threshold). The paper stores its caches in 16
 * bits and has no counterpart to these entry points; the attention they
 * compute is that of saga.h (Eq. 2-4, Eq. 6 and 7) over the stored values.
 *
 * What a row stores. The d values of a row are held in blocks of 16: a 4-bit
 * code per value and an 8-bit scale per block, 4.5 bits a value, and an
 * optional fp32 scale g per head:
 *   value = code (e2m1) * scale (e4m3) * g.
 *   e2m1: sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4,
 *   6 and their negatives. e4m3: sign (ignored: a scale is taken as
 *   non-negative), four exponent bits (bias 7), three mantissa bits; the byte
 *   0x7f, never written here, is read as 480.
 * Quantisation of a block x[0..15] (fp32 arithmetic, each operation rounded
 * to nearest even):
 *   scale = e4m3(min(448, max|x| / (6 g))),  t = scale * g,
 *   code  = e2m1(x / t) with |x / t| > 6 stored as 6;
 *   every code is zero where the scale rounds to zero.
 * NaN counts as zero; an infinity makes the block's scale 448 and is stored
 * as 6.
 *
 * Conventions (streams, ownership, host checks, device error word) are those
 * of saga.h. `shape` describes the problem as there, with these readings:
 *   dtype                the type of q, k_new, v_new and of the rows read back;
 *   k_stride_*, v_stride_*  strides of the 4-bit caches in values: element
 *                        (b,h,t,i) has its code in byte
 *                        (b*stride_b + h*stride_h + t*d + i) / 2 of the codes
 *                        (low half for even i) and its scale in byte
 *                        (b*stride_b + h*stride_h + t*d + i) / 16 of the scales.
 *                        They must be multiples of 256.
 *   cap                  a multiple of 4.
 * saga_shape_contiguous gives such strides for every cap that is a multiple of 4.
 * A shape that is valid in saga.h but breaks the last two, or has B (h_k + h_v)
 * above 65535 or max_l_kv above 2^31 - 4097, gets SAGA_ERR_UNSUPPORTED.
 */
#ifndef SAGA_Q4_H_
#define SAGA_Q4_H_

#include "saga.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A 4-bit cache: device pointers, owned by the caller.
 *   k_codes  [B][h_k][cap][d/2]  bytes, 16-byte aligned
 *   k_scales [B][h_k][cap][d/16] bytes, 16-byte aligned
 *   v_codes, v_scales            as above with h_v heads
 *   k_g [h_k], v_g [h_v]         nullable fp32 scale of each head, positive and
 *                                finite (1 where NULL)
 * Bytes of positions at or behind l_kv[b] may hold anything.
 */
typedef struct saga_q4_cache {
  void *k_codes, *k_scales;
  void *v_codes, *v_scales;
  const float *k_g, *v_g;
} saga_q4_cache;

/*
 * Bytes of device workspace that the calls below need for `shape`; 0 if the
 * shape is invalid. To be initialised with saga_workspace_init, as in saga.h;
 * saga_read_device_error reads its error word.
 */
size_t saga_q4_workspace_size(const saga_shape *shape);

/*
 * Quantise new rows and append them: for every sequence b, rows
 * k_new[b][i][0..h_k-1][0..d-1] and v_new[b][i][0..h_v-1][0..d-1], i < n, are
 * written at position l_kv[b] + i of every head, then l_kv[b] grows by n, in
 * stream order.
 *   k_new, v_new  [B][T][h_k][d] and [B][T][h_v][d], contiguous, the shape's
 *                 dtype; T >= 1. T = 1 is one decoded token per sequence.
 *   n_new         nullable [B] int32: n = n_new[b], in [0, T]; NULL: n = T.
 *   l_kv          [B] int32, read and written.
 *   ws            a workspace (only its error word is used; >= 256 bytes).
 * A sequence that is left as it is, with the error word's bit set: l_kv[b]
 * < 0 or n < 0 (SAGA_DEVERR_LKV_NEGATIVE), n > T or l_kv[b] + n above cap or
 * 2^31 - 1 (SAGA_DEVERR_LKV_TOO_LONG).
 */
saga_status saga_q4_append_kv(const saga_shape *shape, const saga_q4_cache *cache,
                              const void *k_new, const void *v_new, int32_t T,
                              const int32_t *n_new, int32_t *l_kv, void *ws,
                              size_t ws_bytes, saga_stream_t stream);

/*
 * Read a window back: K[b][h][i] = row start[b] + i of key head h, and V
 * likewise, for i < n and start[b] + i < min(l_kv[b], cap); rows at or behind
 * the sequence's end (and every row of a sequence whose start[b] is negative,
 * which sets SAGA_DEVERR_LKV_NEGATIVE) are left as they were in K and V. A
 * length above cap sets SAGA_DEVERR_LKV_TOO_LONG.
 *   n        rows per head, 1 <= n.
 *   start    nullable [B] int32 (NULL: 0).
 *   K, V     [B][h_k][n][d] and [B][h_v][n][d], contiguous, the shape's dtype,
 *            16-byte aligned: the value code * scale * g rounded to fp32 and,
 *            for SAGA_BF16, then to bfloat16 (to nearest even; without g the
 *            value is exact in both).
 *   ws       a workspace (only its error word is used; >= 256 bytes).
 */
saga_status saga_q4_read_kv(const saga_shape *shape, const saga_q4_cache *cache,
                            const int32_t *start, int64_t n, const int32_t *l_kv,
                            void *K, void *V, void *ws, size_t ws_bytes,
                            saga_stream_t stream);

/*
 * Full-attention decode over a 4-bit cache: saga_dense_decode with the key
 * and value heads of `shape` (gqa_dense_decode's result when h_k == h_v).
 *   q    [B][h_q][d] as in saga.h, the shape's dtype.
 *   out  [B][h_q][d] fp32, written; zero for an empty sequence.
 * Head layouts supported: those of saga_dense_decode; others return
 * SAGA_ERR_UNSUPPORTED.
 */
saga_status saga_q4_dense_decode(const saga_shape *shape, const saga_q4_cache *cache,
                                 const void *q, const int32_t *l_kv, float *out,
                                 void *ws, size_t ws_bytes, saga_stream_t stream);

/*
 * One Atop-N step with stored thresholds over a 4-bit cache: arguments and
 * results as for saga_decode_step.
 */
saga_status saga_q4_decode_step(const saga_shape *shape, const saga_q4_cache *cache,
                                const void *q, const int32_t *l_kv, const float *tau,
                                float *out, int32_t *sel_count, uint8_t *sel_mask,
                                void *ws, size_t ws_bytes, saga_stream_t stream);

/*
 * Refresh over a 4-bit cache: tau[b][j] = the exact N-th largest score of row
 * (b, j), or -inf when N >= l_kv[b], as saga_refresh_threshold; N >= 1.
 * Where a bounded wait gave up (SAGA_DEVERR_TIMEOUT), tau is NaN in place of a
 * score, and out and sel_count are as in saga_q4_decode_step then: NaN and -1.
 *   out      nullable: with it, the same call then runs this step's selection
 *            and PV with the fresh tau (out, sel_count and sel_mask as in
 *            saga_q4_decode_step). Without it sel_count and sel_mask must be NULL.
 *   scores   nullable [B][h_q][max_l_kv] fp32: receives the score rows.
 */
saga_status saga_q4_refresh_threshold(const saga_shape *shape, const saga_q4_cache *cache,
                                      const void *q, const int32_t *l_kv, int32_t N,
                                      float *tau, float *out, int32_t *sel_count,
                                      uint8_t *sel_mask, float *scores, void *ws,
                                      size_t ws_bytes, saga_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SAGA_Q4_H_ */
