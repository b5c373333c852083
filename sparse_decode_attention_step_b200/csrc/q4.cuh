// What the 4-bit cache kernels share: the row format, its conversion to fp16
// MMA operands, and the score tile.
//
// A row of D values is D/2 bytes of e2m1 codes and D/16 e4m3 scales. In fp16
// both factors and their product are exact: a code has 2 significant bits, a
// scale 4, and code * scale has at most 6 and lies between 2^-10 and 2688. The
// scale byte moved to bits 7..14 of a half is the scale times 2^-8 (subnormal
// scales become subnormal halves), so one integer multiply converts it, and
// operands built this way carry a common factor 2^-8 that the kernels take out
// in fp32. Any byte therefore reads as a finite value, stale ones included.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100.cuh"

namespace saga {

// Strides of the code arrays in bytes; the scale arrays have an eighth of them
// (D/2 code bytes to D/16 scale bytes a row).
struct Q4Params {
  const void *q;
  const uint8_t *kc, *ks, *vc, *vs;
  const float *k_g, *v_g;      // nullable [h_k], [h_v]
  const int32_t *l_kv;
  const float *tau;
  float *partials;             // dense: [S + B * h_k][h_q / h_k][d + kRecPad]
  float *out;                  // dense: [B][h_q][d]
  float *scores_out;           // dump: [B][h_q][row_stride]
  uint16_t *group_max;         // max: [B * h_q][nblk * 4], largest scores of 8-position groups:
                               // the upper halves of their order keys
  int32_t *tickets;            // step: [B * h_q + 1] counters of the gather (the last one of the
                               // select where no gather follows), cleared here
  uint8_t *sel_mask;           // nullable [B][h_q][row_stride]
  uint32_t *lmask;             // step: [B * h_q][nblk] kept positions of every 32-position block
  float *lscore;               // [B * h_q][nblk * 32] kept scores, each at its position
  int64_t nblk;
  int32_t *err, *abort;
  int64_t q_sb, q_sh;          // elements
  int64_t kc_sb, kc_sh, vc_sb, vc_sh;
  int64_t cap, max_l_kv, row_stride;
  int32_t B, h_q, h_k, h_v;
  int32_t S;                   // CTAs that share the rows
  float scale;                 // 1 / sqrt(d)
};

constexpr float kQ4Unit = 256.f;   // what the fp16 operands are scaled down by

namespace q4 {

// Four bytes of codes: their eight values as four f16x2, in order.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// A scale byte in both halves, times 2^-8.
__device__ __forceinline__ uint32_t scale_f16(uint32_t byte) { return (byte & 0x7fu) * 0x00800080u; }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// {lo, hi} as f16x2
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// the same cut off
__device__ __forceinline__ uint32_t pack_f16_rz(float lo, float hi) {
  uint32_t d;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d (+)= a [16 x 16] * b [16 x 8], fp16 operands, fp32 sums
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = a * b: the first step of a sum, without registers of zeros
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// A query row's share of this lane: dims tq * D/4 .. + D/4 - 1 as fp32.
template <int D>
__device__ __forceinline__ void load_q(const float *row, int tq, float (&v)[D / 4]) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const float4 x = __ldg(reinterpret_cast<const float4 *>(row + tq * (D / 4)) + i);
    v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
  }
}
template <int D>
__device__ __forceinline__ void load_q(const uint16_t *row, int tq, float (&v)[D / 4]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float x[8];
    load8(row + tq * (D / 4) + 8 * i, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[8 * i + e] = x[e];
  }
}

// The query operand. MMA column k of k-step s is dim tq * D/4 + 4 s + {0, 1}
// (k = 2 tq, 2 tq + 1) and + {2, 3} (k = 2 tq + 8, + 9): a lane's operands of a
// key row are then D/4 consecutive values, one or two whole scale blocks.
//
// Rows are brought to fp16 by a power of two that puts their largest magnitude
// into [2^14, 2^15): bf16 queries are then exact down to 2^-24 / 2^15 of the
// row's maximum, and fp32 queries keep 22 bits in a high and a low half (Q2).
// A row that is not `live` is one of zeros. Returns the inverse of the power of two.
template <int D, typename T, bool Q2, int HALF>
__device__ __forceinline__ float q_frag(const T *q, bool live, int tq, uint32_t (&hi)[D / 16][4],
                                        uint32_t (&lo)[Q2 ? D / 16 : 1][4]) {
  float v[D / 4];
  if (live) {
    load_q<D>(q, tq, v);
  } else {
#pragma unroll
    for (int i = 0; i < D / 4; ++i) v[i] = 0.f;
  }
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(v[i]));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const int e = max(1, static_cast<int>(__float_as_uint(mx) >> 23));
  const int k = min(126, 141 - e);                   // mx * 2^k in [2^14, 2^15)
  const float f = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = v[4 * s + 2 * i] * f, b = v[4 * s + 2 * i + 1] * f;
      const uint32_t h = pack_f16(a, b);
      hi[s][2 * i + HALF] = h;
      if constexpr (Q2) {
        const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        lo[s][2 * i + HALF] = pack_f16(a - r.x, b - r.y);
      }
    }
  return __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
}

// What turns a raw score (fp16 operands' units) into a score times `unit`; `inv` is the
// power of two from q_frag, g the key head's scale. g comes last, so that a large one
// overflows nothing that a small query row would bring back. The result stays between the
// smallest and the largest fp32 value: positions behind a row's end are -inf and keys of
// zeros 0 before they are multiplied, and a factor of 0 or infinity would make them NaN.
// (A factor under 2^-126 has fewer bits: of scores under 2^-100, which no softmax sees. One
// that the largest value bounds belongs to scores past 2^120, or of 0.)
__device__ __forceinline__ float score_factor(float unit, float inv, float g) {
  return fminf(fmaxf(unit * kQ4Unit * inv * g, 0x1p-149f), 0x1.fffffep127f);
}

// Eight codes of two value rows (keys k and k + 1 of an MMA step) into A operands:
// register `half` * 2 of tile n holds dim 2 n of both rows, the next one dim 2 n + 1.
// The rows' codes are interleaved by nibble before they are converted, so that
// each converted pair holds one dim of both.
__device__ __forceinline__ void value_pair(uint32_t wa, uint32_t wb, uint32_t sa, uint32_t sb, int half,
                                           uint32_t (&a)[4][4]) {
  const uint32_t sc = ((sa + (sb << 16)) & 0x007f007fu) * 0x80u;
  const uint32_t even = (wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u);
  const uint32_t odd = ((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u);
  uint32_t t[4];
  codes_f16(even, t);
#pragma unroll
  for (int n = 0; n < 4; ++n) a[n][2 * half] = mul_f16x2(t[n], sc);
  codes_f16(odd, t);
#pragma unroll
  for (int n = 0; n < 4; ++n) a[n][2 * half + 1] = mul_f16x2(t[n], sc);
}

// Where a warp stands in its CTA's ring.
template <int ST>
struct Stage {
  int st = 0;
  uint32_t phase = 0;          // parity of the stage's current use
  __device__ __forceinline__ void advance() {
    if (++st == ST) { st = 0; phase ^= 1u; }
  }
  // the stage to refill, and the parity of its last use's end
  static constexpr int kBack = ST >= 3 ? 2 : 1;
  __device__ __forceinline__ int refill() const { return st >= kBack ? st - kBack : st + ST - kBack; }
  __device__ __forceinline__ uint32_t refill_parity() const { return st >= kBack ? phase : phase ^ 1u; }
};

// Raw scores (fp16 operands' units) of 16 MT query rows against 8 NT keys: this
// lane's key row of the first tile starts at `codes` and `scales` in shared
// memory, those of the others eight rows apart; column c of a tile is the key of
// the lanes with lane / 4 == c. The tiles' MMAs alternate: each depends on the
// one before it in its own tile only.
template <int D, int MT, int NT, bool Q2>
__device__ __forceinline__ void score_tiles(const uint8_t *codes, const uint8_t *scales, int tq,
                                            const uint32_t (&hi)[MT][D / 16][4],
                                            const uint32_t (&lo)[Q2 ? MT : 1][Q2 ? D / 16 : 1][4],
                                            float (&c)[NT][MT][4]) {
  uint32_t w[NT][D / 32], sb[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if constexpr (D == 64) {
      const uint2 x = *reinterpret_cast<const uint2 *>(codes + t * 8 * (D / 2) + tq * 8);
      w[t][0] = x.x; w[t][1] = x.y;
      sb[t] = scales[t * 8 * (D / 16) + tq];
    } else {
      const uint4 x = *reinterpret_cast<const uint4 *>(codes + t * 8 * (D / 2) + tq * 16);
      w[t][0] = x.x; w[t][1] = x.y; w[t][2] = x.z; w[t][3] = x.w;
      sb[t] = *reinterpret_cast<const uint16_t *>(scales + t * 8 * (D / 16) + tq * 2);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t h[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t sc = scale_f16(i < 2 ? sb[t] : sb[t] >> 8);
      codes_f16(w[t][i], h[t]);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[t][e] = mul_f16x2(h[t][e], sc);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < (Q2 ? 2 : 1); ++q)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (i == 0 && k == 0 && q == 0) mma_first(c[t][m], hi[m][0], h[t][0], h[t][1]);
            else mma(c[t][m], q == 0 ? hi[m][2 * i + k] : lo[Q2 ? m : 0][Q2 ? 2 * i + k : 0], h[t][2 * k], h[t][2 * k + 1]);
          }
  }
}

// Untiled asynchronous copy (a multiple of 16 bytes, both ends 16-byte
// aligned) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(sm100::smem_u32(bar))
      : "memory");
}

// The same for data that is read once: first out of L2.
__device__ __forceinline__ void bulk_load_once(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(sm100::smem_u32(bar)), "l"(policy)
      : "memory");
}

// Bounded wait of every lane of a warp, given up early when *abort is set. The short-wait
// build (-DSAGA_SHORT_WAITS) gives up at once where there is anything to wait for, which
// runs what follows a give-up: the poisoned results, and the wait for copies in flight.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const int *abort) {
#ifdef SAGA_SHORT_WAITS
  return sm100::mbar_test_wait(bar, parity);
#else
  if (sm100::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = sm100::global_ns();
  for (;;) {
    if (sm100::mbar_try_wait_sleep(bar, parity, sm100::kSuspendHintNs)) return true;
    if (*reinterpret_cast<const volatile int *>(abort) != 0) return false;
    if (sm100::global_ns() - t0 > sm100::kWaitLimitNs) return false;
  }
#endif
}

// A sequence's length in [0, min(cap, max_l_kv)]; a violation is recorded where
// `report` is set.
__device__ __forceinline__ int length(const Q4Params &p, int b, bool report) {
  int L = p.l_kv[b];
  const int hi = static_cast<int>(p.cap < p.max_l_kv ? p.cap : p.max_l_kv);   // max_l_kv fits an int
  if (L < 0 || L > hi) {
    if (report) atomicOr(p.err, L < 0 ? SAGA_DEVERR_LKV_NEGATIVE : SAGA_DEVERR_LKV_TOO_LONG);
    L = L < 0 ? 0 : hi;
  }
  return L;
}

// How the rows (b, key head) are shared among CTAs: every row is a run of chunks
// of CH positions, the rows follow one another, and CTA i of n takes the chunks
// from floor(i T / n) to floor((i + 1) T / n) of all T. The lengths are read on the
// device, so the CTAs have equal work whatever the lengths and whatever bound
// max_l_kv gives. n <= T, so every CTA has a chunk. Called by whole warps.
struct Work {
  int64_t total;
  int n;
  __device__ __forceinline__ int64_t begin(int i) const { return total * i / n; }
  // the CTA that has chunk x
  __device__ __forceinline__ int cta_of(int64_t x) const {
    return static_cast<int>(((x + 1) * n - 1) / total);
  }
};

template <int CH>
__device__ __forceinline__ int chunks_of(int L) { return L / CH + (L % CH != 0); }

template <int CH>
__device__ __forceinline__ Work work_of(const Q4Params &p, int lane, bool report) {
  int64_t t = 0;
  for (int b = lane; b < p.B; b += 32) t += static_cast<int64_t>(chunks_of<CH>(length(p, b, report))) * p.h_k;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return {t, static_cast<int>(t < p.S ? t : p.S)};
}

// The sequence that holds chunk x: its first chunk is `start`, each of its rows
// has nb.
struct Seq {
  int64_t start;
  int b, L, nb;
};

template <int CH>
__device__ __forceinline__ Seq seq_at(const Q4Params &p, int lane, int64_t x) {
  int64_t start = 0;
  for (int b0 = 0;; b0 += 32) {
    const int L = b0 + lane < p.B ? length(p, b0 + lane, false) : 0;
    const int64_t mine = static_cast<int64_t>(chunks_of<CH>(L)) * p.h_k;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, start + incl > x);
    if (past != 0u || b0 + 32 >= p.B) {
      const int at = past != 0u ? __ffs(past) - 1 : 0;
      Seq s;
      s.b = b0 + at;
      s.L = __shfl_sync(0xffffffffu, L, at);
      s.start = start + __shfl_sync(0xffffffffu, incl - mine, at);
      s.nb = chunks_of<CH>(s.L);
      return s;
    }
    start += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The pieces of rows in a CTA's chunks [x, end), one after the other.
struct Piece {
  int b, kh, L, c0, c1;         // chunks [c0, c1) of row (b, kh)
};

template <int CH>
__device__ __forceinline__ Piece next_piece(const Q4Params &p, Seq &s, int64_t &x, int64_t end) {
  while (x >= s.start + static_cast<int64_t>(s.nb) * p.h_k && s.b + 1 < p.B) {   // sequences without a chunk fall out
    s.start += static_cast<int64_t>(s.nb) * p.h_k;
    s.L = length(p, ++s.b, false);
    s.nb = chunks_of<CH>(s.L);
  }
  const int64_t at = x - s.start;
  Piece q;
  q.L = s.L;
  q.b = s.b;
  q.kh = static_cast<int>(at / s.nb);
  q.c0 = static_cast<int>(at % s.nb);
  const int64_t n = end - x < s.nb - q.c0 ? end - x : s.nb - q.c0;
  q.c1 = q.c0 + static_cast<int>(n);
  x += n;
  return q;
}

// A CTA's ring of ST stages. Chunk i (counted over all of the CTA's pieces) goes
// into stage i % ST; kAhead chunks are issued before the first is computed and
// one more before each, by a lane of warp i % kWarps, so that no warp is slower
// than the others (a warp of its own for the copies would cost every thread an
// eighth of its registers). A stage is refilled when the chunk two before the
// current one has been read by all warps (with two stages, the chunk before it).
template <int CH, int ST>
struct Ring {
  static constexpr int kAhead = ST >= 3 ? ST - 2 : 1;
  static_assert(ST >= 2, "a stage to fill and a stage to read");
  uint64_t full[ST], empty[ST];
  int abort;

  __device__ __forceinline__ void init(int warps) {
    for (int i = 0; i < ST; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], warps);
    }
    abort = 0;
    sm100::fence_mbar_init();
  }
  __device__ __forceinline__ bool gave_up() const { return *reinterpret_cast<const volatile int *>(&abort) != 0; }
  __device__ __forceinline__ void give_up(int32_t *err) {
    atomicOr(err, SAGA_DEVERR_TIMEOUT);
    *reinterpret_cast<volatile int *>(&abort) = 1;
  }
  // Issue into stage st, whose last use had `parity`, the chunk that is `ahead`
  // chunks behind chunk c of piece pc, if the CTA has it: load(b, kh, L, chunk
  // of the row, stage). (seq, x, end) is the walk after pc. A stage that does not
  // become free in time is a give-up, which the waits for its chunk see.
  template <typename F>
  __device__ __forceinline__ void issue(const Q4Params &p, int st, uint32_t parity, Piece pc, int c, int ahead,
                                        Seq seq, int64_t x, int64_t end, F load) {
    c += ahead;
    while (c >= pc.c1) {
      if (x >= end) return;
      c -= pc.c1;
      pc = next_piece<CH>(p, seq, x, end);
      c += pc.c0;
    }
    if (wait_bar(&empty[st], parity, &abort)) load(pc.b, pc.kh, pc.L, c, st);
    else give_up(p.err);
  }
  // After a give-up, before the CTA can exit: any copies in flight have landed
  // (the wait for one that was never issued ends by its limit).
  __device__ __forceinline__ void drain(int st, uint32_t phase) {
    for (int k = 0; k < ST; ++k) {
      sm100::mbar_wait(&full[st], phase);
      if (++st == ST) { st = 0; phase ^= 1u; }
    }
  }
};

}  // namespace q4
}  // namespace saga
