// C ABI of the 4-bit cache calls (saga_q4.h): argument checks, the work plan
// and the kernel launches. Nothing here allocates device memory or
// synchronises.
#include <cmath>

#include "plan.h"
#include "q4.cuh"
#include "q4_kernels.h"
#include "saga_q4.h"

namespace saga {
namespace {

saga_status check_q4_shape(const saga_shape *shape) {
  const saga_status r = check_shape(shape);
  if (r != SAGA_OK) return r;
  const saga_shape &s = *shape;
  // 16-byte aligned rows of scales and codes, whole groups of four rows
  if (s.k_stride_b % 256 != 0 || s.k_stride_h % 256 != 0 || s.v_stride_b % 256 != 0 ||
      s.v_stride_h % 256 != 0 || s.cap % 4 != 0)
    return SAGA_ERR_UNSUPPORTED;
  // positions and the ends of the last chunk fit an int
  if (s.max_l_kv > INT32_MAX - 4096) return SAGA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s.B) * (s.h_k + s.h_v) > 65535) return SAGA_ERR_UNSUPPORTED;
  return SAGA_OK;
}

saga_status check_cache(const saga_q4_cache *c) {
  if (c == nullptr) return SAGA_ERR_INVALID_ARG;
  for (const void *x : {c->k_codes, c->k_scales, c->v_codes, c->v_scales})
    if (x == nullptr || !aligned(x, 16)) return SAGA_ERR_INVALID_ARG;
  if (!aligned(c->k_g, 4) || !aligned(c->v_g, 4)) return SAGA_ERR_INVALID_ARG;
  return SAGA_OK;
}

// CTAs that share the rows: as many as fit on the GPU at once, and no more than
// there can be chunks.
int ctas_for(const saga_shape &s, int64_t chunk, int64_t ctas_per_sm) {
  const int64_t chunks = static_cast<int64_t>(s.B) * s.h_k * std::max<int64_t>(1, ceil_div(s.max_l_kv, chunk));
  return static_cast<int>(std::min(chunks, kSms * ctas_per_sm));
}

// The blocks of a row that a CTA of the gather has at least, so that a warp has
// several batches of rows to overlap and a row few records to merge (batch 1, 128K,
// d 128: 15.7 us for the step, 17.0 with 64). As many CTAs as fit at once otherwise: more
// leave a second wave half empty (d 128, batch 8: 43.5 us, 49.6 with four per SM).
constexpr int64_t kGatherBlocks = 128;

// Workspace: error and abort words, the records of the dense call or of the
// gather, the kept lists, the gather's tickets, and for the refresh the group
// maxima and the lower bounds.
struct Q4Plan {
  int dense, scan;     // CTAs of the dense kernel and of a score pass
  int SB;              // gather splits of a row
  int64_t blk_per_split, nblk;
  size_t off_records, off_lmask, off_lscore, off_tickets, off_gmax, off_bound, total;
};
Q4Plan q4_plan(const saga_shape &s) {
  Q4Plan p;
  const int64_t items = static_cast<int64_t>(s.B) * s.h_q;
  p.nblk = std::max<int64_t>(1, ceil_div(s.max_l_kv, 32));
  p.scan = ctas_for(s, kQ4ScanChunk, kQ4ScanCtasPerSm);
  const int64_t sb = std::min(std::max<int64_t>(1, p.nblk / kGatherBlocks),
                              std::max<int64_t>(1, q4_gather_ctas_per_sm(s.d) * kSms / items));
  p.blk_per_split = ceil_div(p.nblk, sb);
  p.SB = static_cast<int>(ceil_div(p.nblk, p.blk_per_split));
  p.dense = 0;
  if (dense_supports(s.h_q, s.h_k, s.h_v))
    p.dense = ctas_for(s, q4_dense_chunk(s.d, s.h_q, s.h_k, s.h_v), kQ4DenseCtasPerSm);
  const size_t rec = static_cast<size_t>(s.d + kRecPad) * sizeof(float);
  const size_t rows = items, lists = rows * p.nblk;
  // a dense CTA leaves a record for each query head of a row it shares: at most
  // one row more than there are CTAs between two rows' ends
  const size_t dense_recs = (p.dense + static_cast<size_t>(s.B) * s.h_k) * (s.h_q / s.h_k);
  p.off_records = kAlign;
  p.off_lmask = align_up(p.off_records + std::max(dense_recs, rows * p.SB) * rec);
  p.off_lscore = align_up(p.off_lmask + lists * sizeof(uint32_t));
  p.off_tickets = align_up(p.off_lscore + lists * 32 * sizeof(float));
  p.off_gmax = align_up(p.off_tickets + (rows + 1) * sizeof(int32_t));
  p.off_bound = align_up(p.off_gmax + lists * 4 * sizeof(uint16_t));
  p.total = align_up(p.off_bound + rows * sizeof(float));
  return p;
}

saga_status check_q4_ws(const Q4Plan &pl, void *ws, size_t ws_bytes) {
  if (ws == nullptr || !aligned(ws, kAlign) || ws_bytes < pl.total) return SAGA_ERR_WORKSPACE;
  return SAGA_OK;
}

saga_status check_q4_inputs(const saga_q4_cache *cache, const void *q, const int32_t *l_kv) {
  const saga_status r = check_cache(cache);
  if (r != SAGA_OK) return r;
  if (q == nullptr || l_kv == nullptr || !aligned(q, 16) || !aligned(l_kv, 4))
    return SAGA_ERR_INVALID_ARG;
  return SAGA_OK;
}

Q4Params base_params(const saga_shape &s, const Q4Plan &pl, const saga_q4_cache &c, const void *q,
                     const int32_t *l_kv, void *ws) {
  Q4Params p{};
  char *wsb = static_cast<char *>(ws);
  p.q = q;
  p.kc = static_cast<const uint8_t *>(c.k_codes);
  p.ks = static_cast<const uint8_t *>(c.k_scales);
  p.vc = static_cast<const uint8_t *>(c.v_codes);
  p.vs = static_cast<const uint8_t *>(c.v_scales);
  p.k_g = c.k_g;
  p.v_g = c.v_g;
  p.l_kv = l_kv;
  p.partials = reinterpret_cast<float *>(wsb + pl.off_records);
  p.lmask = reinterpret_cast<uint32_t *>(wsb + pl.off_lmask);
  p.lscore = reinterpret_cast<float *>(wsb + pl.off_lscore);
  p.group_max = reinterpret_cast<uint16_t *>(wsb + pl.off_gmax);
  p.tickets = reinterpret_cast<int32_t *>(wsb + pl.off_tickets);
  p.nblk = pl.nblk;
  p.err = static_cast<int32_t *>(ws);
  p.abort = static_cast<int32_t *>(ws) + 1;
  p.q_sb = s.q_stride_b; p.q_sh = s.q_stride_h;
  p.kc_sb = s.k_stride_b / 2; p.kc_sh = s.k_stride_h / 2;
  p.vc_sb = s.v_stride_b / 2; p.vc_sh = s.v_stride_h / 2;
  p.cap = s.cap; p.max_l_kv = s.max_l_kv; p.row_stride = s.max_l_kv;
  p.B = s.B; p.h_q = s.h_q; p.h_k = s.h_k; p.h_v = s.h_v;
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(s.d)));
  return p;
}

// The V half of a step, from the kept lists.
saga_status run_gather(const saga_shape &s, const Q4Plan &pl, const Q4Params &p, float *out,
                       int32_t *sel_count, cudaStream_t st) {
  Q4Gather g{};
  g.vc = p.vc; g.vs = p.vs; g.v_g = p.v_g;
  g.vc_sb = p.vc_sb; g.vc_sh = p.vc_sh;
  g.l_kv = p.l_kv; g.cap = p.cap; g.max_l_kv = p.max_l_kv;
  g.lmask = p.lmask; g.lscore = p.lscore; g.nblk = p.nblk;
  g.partials = p.partials; g.out = out; g.sel_count = sel_count;
  g.tickets = p.tickets; g.abort = p.abort; g.err = p.err;
  g.B = s.B; g.h_q = s.h_q; g.hpv = s.h_q / s.h_v;
  g.SB = pl.SB; g.blk_per_split = static_cast<int32_t>(pl.blk_per_split);
  return cuda_check(launch_q4_gather(g, s.d, st), "gather kernel (4-bit)");
}

}  // namespace
}  // namespace saga

using namespace saga;

extern "C" {

size_t saga_q4_workspace_size(const saga_shape *shape) {
  if (check_q4_shape(shape) != SAGA_OK) return 0;
  return q4_plan(*shape).total;
}

saga_status saga_q4_append_kv(const saga_shape *shape, const saga_q4_cache *cache, const void *k_new,
                              const void *v_new, int32_t T, const int32_t *n_new, int32_t *l_kv,
                              void *ws, size_t ws_bytes, saga_stream_t stream) {
  saga_status r = check_q4_shape(shape);
  if (r != SAGA_OK) return r;
  const saga_shape &s = *shape;
  if ((r = check_cache(cache)) != SAGA_OK) return r;
  if (T < 1 || k_new == nullptr || v_new == nullptr || l_kv == nullptr) return SAGA_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(l_kv, 4) || !aligned(n_new, 4))
    return SAGA_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, kAlign) || ws_bytes < kAlign) return SAGA_ERR_WORKSPACE;
  Q4Append p{};
  p.k_new = k_new; p.v_new = v_new; p.n_new = n_new; p.l_kv = l_kv;
  p.kc = static_cast<uint8_t *>(cache->k_codes); p.ks = static_cast<uint8_t *>(cache->k_scales);
  p.vc = static_cast<uint8_t *>(cache->v_codes); p.vs = static_cast<uint8_t *>(cache->v_scales);
  p.k_g = cache->k_g; p.v_g = cache->v_g;
  p.err = static_cast<int32_t *>(ws);
  p.kb_sb = s.k_stride_b / 16; p.kb_sh = s.k_stride_h / 16;
  p.vb_sb = s.v_stride_b / 16; p.vb_sh = s.v_stride_h / 16;
  p.cap = s.cap; p.B = s.B; p.T = T; p.h_k = s.h_k; p.h_v = s.h_v; p.d = s.d;
  return cuda_check(launch_q4_append(p, s.dtype, reinterpret_cast<cudaStream_t>(stream)),
                    "append kernel (4-bit)");
}

saga_status saga_q4_read_kv(const saga_shape *shape, const saga_q4_cache *cache, const int32_t *start,
                            int64_t n, const int32_t *l_kv, void *K, void *V, void *ws,
                            size_t ws_bytes, saga_stream_t stream) {
  saga_status r = check_q4_shape(shape);
  if (r != SAGA_OK) return r;
  const saga_shape &s = *shape;
  if ((r = check_cache(cache)) != SAGA_OK) return r;
  if (n < 1 || l_kv == nullptr || K == nullptr || V == nullptr) return SAGA_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(l_kv, 4) || !aligned(start, 4))
    return SAGA_ERR_INVALID_ARG;
  if (n > INT32_MAX) return SAGA_ERR_UNSUPPORTED;
  if (ws == nullptr || !aligned(ws, kAlign) || ws_bytes < kAlign) return SAGA_ERR_WORKSPACE;
  Q4Read p{};
  p.kc = static_cast<const uint8_t *>(cache->k_codes); p.ks = static_cast<const uint8_t *>(cache->k_scales);
  p.vc = static_cast<const uint8_t *>(cache->v_codes); p.vs = static_cast<const uint8_t *>(cache->v_scales);
  p.k_g = cache->k_g; p.v_g = cache->v_g;
  p.start = start; p.l_kv = l_kv; p.K = K; p.V = V;
  p.err = static_cast<int32_t *>(ws);
  p.kb_sb = s.k_stride_b / 16; p.kb_sh = s.k_stride_h / 16;
  p.vb_sb = s.v_stride_b / 16; p.vb_sh = s.v_stride_h / 16;
  p.cap = s.cap; p.n = n; p.B = s.B; p.h_k = s.h_k; p.h_v = s.h_v; p.d = s.d;
  return cuda_check(launch_q4_read(p, s.dtype, reinterpret_cast<cudaStream_t>(stream)),
                    "read kernel (4-bit)");
}

saga_status saga_q4_dense_decode(const saga_shape *shape, const saga_q4_cache *cache, const void *q,
                                 const int32_t *l_kv, float *out, void *ws, size_t ws_bytes,
                                 saga_stream_t stream) {
  saga_status r = check_q4_shape(shape);
  if (r != SAGA_OK) return r;
  const saga_shape &s = *shape;
  if (!dense_supports(s.h_q, s.h_k, s.h_v)) return SAGA_ERR_UNSUPPORTED;
  if ((r = check_q4_inputs(cache, q, l_kv)) != SAGA_OK) return r;
  if (out == nullptr || !aligned(out, 16)) return SAGA_ERR_INVALID_ARG;
  const Q4Plan pl = q4_plan(s);
  if ((r = check_q4_ws(pl, ws, ws_bytes)) != SAGA_OK) return r;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Q4Params p = base_params(s, pl, *cache, q, l_kv, ws);
  p.S = pl.dense;
  p.out = out;
  return cuda_check(launch_q4_dense(p, s.dtype, s.d, st), "dense kernel (4-bit)");
}

saga_status saga_q4_decode_step(const saga_shape *shape, const saga_q4_cache *cache, const void *q,
                                const int32_t *l_kv, const float *tau, float *out, int32_t *sel_count,
                                uint8_t *sel_mask, void *ws, size_t ws_bytes, saga_stream_t stream) {
  saga_status r = check_q4_shape(shape);
  if (r != SAGA_OK) return r;
  const saga_shape &s = *shape;
  if ((r = check_q4_inputs(cache, q, l_kv)) != SAGA_OK) return r;
  if (tau == nullptr || out == nullptr || !aligned(tau, 4) || !aligned(out, 16) || !aligned(sel_count, 4))
    return SAGA_ERR_INVALID_ARG;
  const Q4Plan pl = q4_plan(s);
  if ((r = check_q4_ws(pl, ws, ws_bytes)) != SAGA_OK) return r;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Q4Params p = base_params(s, pl, *cache, q, l_kv, ws);
  p.S = pl.scan;
  p.tau = tau;
  p.sel_mask = sel_mask;
  const cudaError_t e = launch_q4_scan(p, kQ4Step, s.dtype, s.d, st);
  if (e != cudaSuccess) return cuda_fail(e, "scan kernel (4-bit)");
  return run_gather(s, pl, p, out, sel_count, st);
}

saga_status saga_q4_refresh_threshold(const saga_shape *shape, const saga_q4_cache *cache, const void *q,
                                      const int32_t *l_kv, int32_t N, float *tau, float *out,
                                      int32_t *sel_count, uint8_t *sel_mask, float *scores, void *ws,
                                      size_t ws_bytes, saga_stream_t stream) {
  saga_status r = check_q4_shape(shape);
  if (r != SAGA_OK) return r;
  const saga_shape &s = *shape;
  if ((r = check_q4_inputs(cache, q, l_kv)) != SAGA_OK) return r;
  if (N < 1 || tau == nullptr || !aligned(tau, 4) || !aligned(out, 16) || !aligned(sel_count, 4) ||
      !aligned(scores, 4))
    return SAGA_ERR_INVALID_ARG;
  if (out == nullptr && (sel_count != nullptr || sel_mask != nullptr)) return SAGA_ERR_INVALID_ARG;
  const Q4Plan pl = q4_plan(s);
  if ((r = check_q4_ws(pl, ws, ws_bytes)) != SAGA_OK) return r;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Q4Params p = base_params(s, pl, *cache, q, l_kv, ws);
  p.S = pl.scan;
  cudaError_t e;
  if (scores != nullptr) {
    p.scores_out = scores;
    if ((e = launch_q4_scan(p, kQ4Dump, s.dtype, s.d, st)) != cudaSuccess)
      return cuda_fail(e, "score dump kernel (4-bit)");
  }
  // 1. the largest score of every eight positions, and the N-th largest of those:
  // a lower bound of the threshold (-inf with N groups or fewer)
  float *bound = nullptr;
  if (s.max_l_kv > kQ4NoBound) {
    bound = reinterpret_cast<float *>(static_cast<char *>(ws) + pl.off_bound);
    if ((e = launch_q4_scan(p, kQ4Max, s.dtype, s.d, st)) != cudaSuccess)
      return cuda_fail(e, "group maximum kernel (4-bit)");
    if ((e = launch_q4_bound(p, N, bound, st)) != cudaSuccess) return cuda_fail(e, "bound kernel (4-bit)");
  }
  // 2. the scores that reach it
  p.tau = bound;
  if ((e = launch_q4_scan(p, kQ4Step, s.dtype, s.d, st)) != cudaSuccess)
    return cuda_fail(e, "scan kernel (4-bit)");
  // 3. their N-th largest; for the step, the lists cut down to it
  if ((e = launch_q4_select(p, N, bound, tau, out != nullptr, sel_mask, st)) != cudaSuccess)
    return cuda_fail(e, "select kernel (4-bit)");
  return out == nullptr ? SAGA_OK : run_gather(s, pl, p, out, sel_count, st);
}

}  // extern "C"
