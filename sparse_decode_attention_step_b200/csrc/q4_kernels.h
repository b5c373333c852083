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
// The dense kernel's chunk of positions and CTAs per SM.
int q4_dense_chunk(int d, int h_q, int h_k, int h_v);
int q4_dense_ctas_per_sm(int d, int h_q, int h_k, int h_v);

// Score pass by p.S CTAs: the kept lists of p.tau (step), the group
// maxima and group counts (max), or the score rows (dump).
enum { kQ4Step = 0, kQ4Max = 1, kQ4Dump = 2 };
cudaError_t launch_q4_scan(const Q4Params &p, int mode, int dtype, int d, cudaStream_t st);
constexpr int kQ4ScanChunk = 256;
constexpr int kQ4ScanCtasPerSm = 3;

// tau[b][j] = the N-th largest of row (b, j)'s listed scores, or -inf when
// N >= l_kv[b]; with `keep`, the lists (and a given sel_mask) are cut down to it.
cudaError_t launch_q4_select(const Q4Params &p, int32_t N, float *tau, bool keep, uint8_t *sel_mask,
                             cudaStream_t st);

}  // namespace saga
