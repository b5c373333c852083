// The work plan (split of l_kv across CTAs, workspace carve-up) and the host
// checks shared by the C entry points.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "saga.h"

namespace saga {

constexpr int64_t kSms = 148;              // B200 SMs: the persistent grid
constexpr int64_t kTileKeys = 128;         // split lengths are multiples of a K tile
constexpr int64_t kUnitTiles = 32;         // grid-per-split kernels: at most about this many tiles per split
constexpr int64_t kPersistTiles = 128;     // persistent kernel: at most about this many tiles per unit
constexpr int64_t kGridCtasPerSm = 4;      // grid-per-split kernels: at least this many units per SM
constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  int S;                    // scan / split-kernel units per (b, key head)
  int64_t split_len;        // positions per unit
  // tensor-core path: the gather kernel's own splits of a row
  bool lists;               // the scan writes per-head kept lists
  int SB;                   // gather splits per (b, query head)
  int64_t blk_per_split;    // 32-position blocks per gather split
  int64_t nblk;             // 32-position blocks per row
  // the records the combine merges: comb_S per (b, j), comb_split_len positions each
  int comb_S;
  int64_t comb_split_len;
  // radix select: per row, the list of the top-byte bucket (gcap keys at most)
  int gcap;
  size_t off_partials, off_lmask, off_lscore, off_scores, off_hist, off_gcount, off_hist1,
      off_gcand, off_tau, off_tie, total;
};

// Keys per row in the radix select's bucket list: half the row (the top-byte
// bucket of a score row can hold a third of it), at least 16384, a multiple
// of 4.
inline int select_list_cap(int64_t max_l_kv) {
  const int64_t c = std::max<int64_t>(16384, (max_l_kv / 2 + 3) / 4 * 4);
  return static_cast<int>(c);
}

// Splits of equal length, a multiple of the K tile.
// Grid-per-split kernels (SIMT, dense): the (b, kh, split) units number about a
// whole multiple of the SM count, with at most about kUnitTiles tiles each and,
// where the sequence is long enough, at least as many per SM as fit on one
// (`ctas_per_sm`, at most kGridCtasPerSm, which sizes the workspace): those
// kernels hide their load latency only with every resident slot filled, and
// more splits than slots only add waves and combine work.
// Persistent tensor-core scan: at most one unit per SM and wave, units of up
// to about kPersistTiles tiles. Its gather kernel splits each (b, query head)
// row on its own, into at most kGatherCtas CTAs in all (about four waves of
// eight resident per SM, so that heads that keep more rows than others are
// balanced out by the block scheduler) where the rows allow, each at least
// kGatherMinBlocks blocks of 32 positions long; the combine merges the
// gather's records.
constexpr int64_t kGatherCtas = 32 * kSms;
constexpr int64_t kGatherMinBlocks = 64;

inline Plan make_plan(const saga_shape &s, bool persistent, int64_t ctas_per_sm = kGridCtasPerSm) {
  Plan p{};
  const int64_t rows = static_cast<int64_t>(s.B) * s.h_k;
  const int64_t L = std::max<int64_t>(1, s.max_l_kv);
  const int64_t tiles = rows * ceil_div(L, kTileKeys);
  int64_t s_target;
  if (persistent) {
    const int64_t waves = std::max<int64_t>(1, ceil_div(tiles, kSms * kPersistTiles));
    s_target = std::max<int64_t>(1, kSms * waves / rows);
  } else {
    const int64_t waves = std::max<int64_t>(1, ceil_div(tiles, kSms * kUnitTiles));
    const int64_t slots = std::min(std::max<int64_t>(1, ctas_per_sm), kGridCtasPerSm);
    s_target = std::max<int64_t>(1, ceil_div(kSms * std::max(waves, slots), rows));
  }
  p.split_len = ceil_div(ceil_div(L, s_target), kTileKeys) * kTileKeys;
  p.S = static_cast<int>(ceil_div(L, p.split_len));
  p.comb_S = p.S;
  p.comb_split_len = p.split_len;
  p.nblk = ceil_div(L, 32);
  if (persistent && saga_tc_supports(s.dtype, s.d, s.h_q, s.h_k, s.h_v)) {
    p.lists = true;
    const int64_t items = static_cast<int64_t>(s.B) * s.h_q;
    const int64_t max_sb = std::max<int64_t>(1, p.nblk / kGatherMinBlocks);
    const int64_t sb = std::min(max_sb, std::max<int64_t>(1, kGatherCtas / items));
    p.blk_per_split = ceil_div(p.nblk, sb);
    p.SB = static_cast<int>(ceil_div(p.nblk, p.blk_per_split));
    p.comb_S = p.SB;
    p.comb_split_len = p.blk_per_split * 32;
  }
  const size_t rec = static_cast<size_t>(s.d + kRecPad) * sizeof(float);
  const size_t lists = p.lists ? static_cast<size_t>(s.B) * s.h_q * p.nblk : 0;
  p.off_partials = kAlign;   // [0, 256): device error word, then the step's abort word
  p.off_lmask = align_up(p.off_partials + static_cast<size_t>(s.B) * s.h_q * p.comb_S * rec);
  p.off_lscore = align_up(p.off_lmask + lists * sizeof(uint32_t));
  p.off_scores = align_up(p.off_lscore + lists * 32 * sizeof(float));
  p.off_hist = align_up(p.off_scores + static_cast<size_t>(s.B) * s.h_q * s.max_l_kv * sizeof(float));
  // the bucket counts, the digit-1 histograms and the select's counter of rows follow
  // the top-byte histograms directly: one memset clears all four
  p.gcap = select_list_cap(s.max_l_kv);
  p.off_gcount = p.off_hist + static_cast<size_t>(s.B) * s.h_q * 256 * sizeof(uint32_t);
  p.off_hist1 = p.off_gcount + static_cast<size_t>(s.B) * s.h_q * sizeof(uint32_t);
  p.off_gcand = align_up(p.off_hist1 + (static_cast<size_t>(s.B) * s.h_q * 256 + 1) * sizeof(uint32_t));
  p.off_tau = align_up(p.off_gcand + static_cast<size_t>(s.B) * s.h_q * p.gcap * sizeof(uint32_t));
  p.off_tie = align_up(p.off_tau + static_cast<size_t>(s.B) * s.h_q * sizeof(float));
  p.total = align_up(p.off_tie + static_cast<size_t>(s.B) * s.h_q * sizeof(int32_t));
  return p;
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline saga_status check_shape(const saga_shape *s) {
  if (s == nullptr) return SAGA_ERR_INVALID_ARG;
  if (s->B < 1 || s->h_q < 1 || s->h_k < 1 || s->h_v < 1 || s->d < 1) return SAGA_ERR_INVALID_ARG;
  if (s->h_k > s->h_v || s->h_v > s->h_q) return SAGA_ERR_INVALID_ARG;
  if (s->dtype != SAGA_F32 && s->dtype != SAGA_BF16) return SAGA_ERR_INVALID_ARG;
  if (s->max_l_kv < 0 || s->cap < s->max_l_kv) return SAGA_ERR_INVALID_ARG;
  if (s->h_q % s->h_v != 0 || s->h_v % s->h_k != 0) return SAGA_ERR_UNSUPPORTED;
  if (s->h_q / s->h_k > kMaxGroup) return SAGA_ERR_UNSUPPORTED;
  if (s->d != 64 && s->d != 128) return SAGA_ERR_UNSUPPORTED;
  if (s->max_l_kv > INT32_MAX) return SAGA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->B) * s->h_k > 65535) return SAGA_ERR_UNSUPPORTED;
  const int64_t esz = s->dtype == SAGA_F32 ? 4 : 2;
  const int64_t st[6] = {s->q_stride_b, s->q_stride_h, s->k_stride_b,
                         s->k_stride_h, s->v_stride_b, s->v_stride_h};
  for (int64_t x : st)
    if (x <= 0 || (x * esz) % 16 != 0) return SAGA_ERR_INVALID_ARG;
  if (s->q_stride_h < s->d || s->k_stride_h < s->cap * s->d || s->v_stride_h < s->cap * s->d)
    return SAGA_ERR_INVALID_ARG;
  return SAGA_OK;
}

}  // namespace saga
