// Launchers of the 4-bit cache kernels (host side, internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "saga.h"

namespace saga {

struct Q4Params;

// Strides kb_*, vb_* in blocks of 16 values (8 bytes of codes, 1 of scales).
struct Q4Append {
  const void *k_new, *v_new;       // [B][T][h_k][d], [B][T][h_v][d]
  const int32_t *n_new;            // nullable [B]
  int32_t *l_kv;
  uint8_t *kc, *ks, *vc, *vs;
  const float *k_g, *v_g;
  int32_t *err;
  int64_t kb_sb, kb_sh, vb_sb, vb_sh, cap;
  int32_t B, T, h_k, h_v, d;
};
struct Q4Read {
  const uint8_t *kc, *ks, *vc, *vs;
  const float *k_g, *v_g;
  const int32_t *start, *l_kv;     // start nullable
  void *K, *V;                     // [B][h_k][n][d], [B][h_v][n][d]
  int32_t *err;
  int64_t kb_sb, kb_sh, vb_sb, vb_sh, cap, n;
  int32_t B, h_k, h_v, d;
};

cudaError_t launch_q4_append(const Q4Append &p, int dtype, cudaStream_t st);
cudaError_t launch_q4_read(const Q4Read &p, int dtype, cudaStream_t st);

// Full attention by p.S CTAs, then the combine. Head layouts as dense_supports.
cudaError_t launch_q4_dense(const Q4Params &p, int dtype, int d, cudaStream_t st);
// The dense kernel's chunk of positions.
int q4_dense_chunk(int d, int h_q, int h_k, int h_v);
constexpr int kQ4DenseCtasPerSm = 1;

// Score pass by p.S CTAs: the kept lists of p.tau (step; -inf where it is null), the group maxima
// (max), or the score rows (dump).
enum { kQ4Step = 0, kQ4Max = 1, kQ4Dump = 2 };
cudaError_t launch_q4_scan(const Q4Params &p, int mode, int dtype, int d, cudaStream_t st);
constexpr int kQ4ScanChunk = 256;      // the shortest chunk of a pass
constexpr int kQ4ScanCtasPerSm = 2;

// bound[b][j]: a lower bound of the N-th largest score of row (b, j), from the
// group maxima (-inf with N groups or fewer).
cudaError_t launch_q4_bound(const Q4Params &p, int32_t N, float *bound, cudaStream_t st);

// tau[b][j] = the N-th largest of row (b, j)'s listed scores, all of them at
// least bound[b][j] (-inf where bound is null), or -inf when N >= l_kv[b]; NaN instead
// of the former when a score pass of the call gave up. With `keep`, the lists (and a given
// sel_mask) are cut down to it, and a gather has to follow; without it this ends the call.
constexpr int kQ4SelectKeys = 10240;   // scores of a row that it holds on chip
// Rows up to this long go to the select whole: without the maximum pass and the
// bound a refresh of 4096 positions takes 13.0 us instead of 18.2 (batch 8: 21.7
// instead of 26.2), one of 8192 17.2 instead of 16.8 (29.4 instead of 24.4).
constexpr int kQ4NoBound = 6144;
cudaError_t launch_q4_select(const Q4Params &p, int32_t N, const float *bound, float *tau, bool keep,
                             uint8_t *sel_mask, cudaStream_t st);

// The V half of a step from the kept lists, SB CTAs of blk_per_split blocks a row.
struct Q4Gather {
  const uint8_t *vc, *vs;
  const float *v_g;
  const int32_t *l_kv;
  const uint32_t *lmask;
  const float *lscore;
  float *partials;                 // [B * h_q][SB][d + kRecPad]
  float *out;
  int32_t *sel_count;              // nullable
  int32_t *tickets, *abort, *err;
  int64_t vc_sb, vc_sh, nblk, cap, max_l_kv;
  int32_t B, h_q, hpv, SB, blk_per_split;
};
constexpr int q4_gather_ctas_per_sm(int d) { return d == 64 ? 4 : 3; }   // that fit at once
cudaError_t launch_q4_gather(const Q4Gather &p, int d, cudaStream_t st);

}  // namespace saga
