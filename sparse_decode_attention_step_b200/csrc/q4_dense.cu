// Full-attention decode over a 4-bit cache: Eq. (2-4) over every position, for
// GQA (h_k == h_v) and SAGA heads (VPG = h_v / h_k value heads per key head).
//
// As many CTAs as fit on the GPU share the rows (b, key head) in equal runs of
// chunks, whatever the lengths (see Work in q4.cuh); a row that several CTAs
// share leaves a record per CTA for the combine kernel below. Chunks of positions
// (codes and scales of the key head and its VPG value heads, each a contiguous
// range) come through a ring of shared-memory stages with untiled bulk copies
// (see Ring). Eight warps each own a run of a chunk's positions (and, with four
// value heads, two of them) and keep their own running softmax,
// so they meet only at the ring and at the end of a row. A warp works in
// registers throughout:
//
//   scores   S[rows x keys] = Q K^T, mma.sync m16n8k16 with the query rows on M
//            and eight keys on N: a lane converts the consecutive codes of one
//            key row into the B operand;
//   softmax  per row (a row's scores sit in the four lanes of a quad);
//   output   O^T[dims x rows] += V^T P^T with the dims on M and the score rows on
//            N: the scores' accumulators have the layout of the B operand, and
//            a lane converts the same dims of four keys into the A operand. The
//            operand pairs two keys per register, so the codes of two rows are
//            interleaved by nibble before they are converted.
//
// Probabilities are split into a high and a low fp16 half (22 bits; fp16 alone
// would cost the fp32 output its precision), relative to the largest score of the
// warp's positions of one chunk and scaled by 2^7: a probability loses bits when it
// lies more than 2^9 under that maximum, and then at most 2^-30 of it. (2^15, as far
// up as fp16 goes, would move that to 2^-38, but the exponents' arguments would reach
// 15 instead of 7, and their rounding took the error of ordinary rows from 2.2e-7 to
// 3.4e-7 of the norm.) The chunk's sums are brought to the row's running maximum when
// they are added to its own, by the factor that the addition takes anyway; the running
// maximum follows lazily, and a row is rescaled when its maximum has grown by more than
// 2^8 of weight. (P relative to the running maximum lost the bits of every key far
// under a dominating one: with keys of value 0 that outweigh the others 2^20 times
// each, 1.6e-4 of the output.) The tensor cores cut their fp32 sums off instead of
// rounding them, so a sum runs over a warp's positions of one chunk there and over
// chunks in rounded fp32 additions.
//
// Rows of the score tile (each 8-row tile belongs to one value head):
//   S    at most 4 query heads per value head: rows 0-3 the heads, rows 4-7 the
//        same heads again; rows 0-3 put the high half of P into the product,
//        rows 4-7 the low half, and the sums are added at the end: one MMA
//        where a high and a low one would each leave half the tile empty;
//   L8   5 to 8 heads: one tile, a high and a low MMA into the same sums;
//   L16  9 to 16 heads (one value head): two such tiles.
//
// Bound by instruction issue: about 310 per 32 positions of a key head and a value
// head of 64 (64 conversions, 64 scale products, 32 MMAs, the softmax, the nibbles)
// at 2.3-2.7 a cycle and SM. 8 x 128K positions of 8 + 8 heads of 64 (604 MB): 144
// us, 4.2 TB/s; 16 sequences of up to 64K, 1 + 4 heads of 128 (201 MB): 70 us, 2.9
// TB/s, where four value heads share each key row's scores. The factors of the chunks
// cost 0.4% of the instructions in the first case, and up to 4% of the time at d 128.
#include <atomic>

#include "kernels.h"
#include "plan.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 7.f;                  // P is scaled by 2^kPShift
constexpr float kLazy = 8.f;                    // log2 growth of a row's maximum that rescales it
constexpr int kMaxDevices = 64;

enum { kRowsS = 0, kRowsL8 = 1, kRowsL16 = 2 };

// VPW value heads per warp, NG groups of warps: VPG = VPW * NG.
template <int D, int VPW, int MODE, int NG>
struct QD {
  static constexpr int VPG = VPW * NG;
  static constexpr int SL = kWarps / NG;                        // position slabs of a chunk
  static constexpr int NRT = MODE == kRowsL16 ? 2 : VPW;        // 8-row score tiles per warp
  static constexpr int MT = (NRT + 1) / 2;                      // 16-row MMA tiles
  static constexpr int NM = D / 16;                             // 16-dim MMA tiles of the output
  // Positions per warp and chunk. One CTA per SM, whose eight warps have up to 255
  // registers each, is as fast as two with half of that or as 12 and 16 warps, and
  // long runs of positions spread a chunk's fixed work (waits, the running maximum,
  // addresses: a hundred instructions): 8 x 128K positions of 8 + 8 heads of 64 took
  // 161 us with 32 at a time, 147 with 48 and 142 with 128. As many as leave two or
  // three stages of the ring room and the accumulators their registers: none spill but
  // at d 128 mode L16 (24 bytes a thread, fp32 queries 188) and fp32 queries of two and
  // four value heads (28 to 36).
  static constexpr int kKeys = D == 64 ? (VPG == 1 ? 128 : 80) : (VPG == 1 ? 64 : VPG == 2 ? 32 : 48);
  static constexpr int NT = kKeys / 8, NJ = kKeys / 16;         // key tiles, 16-key steps
  // Row tiles of a product of P and V, and the 16-key steps whose values are converted
  // before it: in mode L16 one or two at a time, whose registers hold the second tile's sums (8 x
  // 128K, one head of 128: 65 us in bf16 and 77 in fp32; 67 and 80 with all steps at once)
  static constexpr int NP = MODE == kRowsL16 ? 2 : 1, JB = MODE != kRowsL16 ? NJ : D == 64 ? 2 : 1;
  static constexpr int KC = SL * kKeys;
  static constexpr int kCodes = KC * D / 2, kScales = KC * D / 16;
  static constexpr int kStage = (kCodes + kScales) * (1 + VPG);
  static constexpr int kState = NRT * (NM * 4 + 2);             // a warp's registers to merge
  static constexpr int kSlot = NG * kState * 32 * 4;            // a slab's states
  static constexpr int kSpace = 230400;                         // shared memory of a CTA, less its barriers
  static constexpr int kStages = (kSpace - kSlot) / kStage < 8 ? (kSpace - kSlot) / kStage : 8;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kSlots = (kSpace - kRing) / kSlot < SL / 2 ? (kSpace - kRing) / kSlot : SL / 2;
  static constexpr int kSmem = kRing + kSlots * kSlot;
  static_assert(kStages >= 2 && kSlots >= 1, "a ring and a slab's states");
};

// Merge a second running softmax state (m2, l2, and acc2 by f(register)) into
// (m, l, acc) of one row tile: rows g of this lane, columns 2 tq and 2 tq + 1.
template <int NM, typename F>
__device__ __forceinline__ void merge_state(float &m, float &l, float (&acc)[NM][4], float m2, float l2, int tq,
                                            F acc2) {
  const float mn = fmaxf(m, m2);
  const float a = m == -INFINITY ? 0.f : q4::ex2(m - mn), c = m2 == -INFINITY ? 0.f : q4::ex2(m2 - mn);
  m = mn;
  l = l * a + l2 * c;
  const float a0 = __shfl_sync(0xffffffffu, a, tq * 8), a1 = __shfl_sync(0xffffffffu, a, tq * 8 + 4);
  const float c0 = __shfl_sync(0xffffffffu, c, tq * 8), c1 = __shfl_sync(0xffffffffu, c, tq * 8 + 4);
#pragma unroll
  for (int n = 0; n < NM; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[n][e] = acc[n][e] * (e % 2 ? a1 : a0) + acc2(n * 4 + e) * (e % 2 ? c1 : c0);
}

template <int D, int VPW, int MODE, int NG, typename T>
__global__ void __launch_bounds__(kThreads, 1)
q4_dense_kernel(const Q4Params p) {
  using C = QD<D, VPW, MODE, NG>;
  constexpr bool Q2 = sizeof(T) == 4;
  constexpr int NRT = C::NRT, MT = C::MT, NM = C::NM, ST = C::kStages, KC = C::KC, NT = C::NT, NJ = C::NJ;
  constexpr int NP = C::NP, JB = C::JB;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ q4::Ring<KC, ST> bars;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.h_q / p.h_k, HPV = G / C::VPG;

  if (tid == 0) bars.init(kWarps);
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int cta = blockIdx.x;
  const q4::Work work = q4::work_of<KC>(p, lane, cta == 0 && warp == 0);
  for (int b = cta; b < p.B; b += gridDim.x)         // an empty sequence: zero rows
    if (q4::length(p, b, false) == 0)
      for (int i = tid; i < p.h_q * D; i += kThreads) p.out[static_cast<int64_t>(b) * p.h_q * D + i] = 0.f;
  if (cta >= work.n) return;
  int64_t x0 = work.begin(cta);
  const int64_t x1 = work.begin(cta + 1);
  q4::Seq seq = q4::seq_at<KC>(p, lane, x0);

  const auto load = [&](int b, int kh, int L, int c, int st) {
    const int64_t kb = b * p.kc_sb + kh * p.kc_sh;
    const int64_t vb = b * p.vc_sb + static_cast<int64_t>(kh) * C::VPG * p.vc_sh;
    const int64_t t = static_cast<int64_t>(c) * KC;
    const int left = L - c * KC;
    // whole groups of four rows: 16 bytes of scales at least (cap is a multiple of 4)
    const uint32_t rows = left < KC ? (left + 3) & ~3 : KC;
    const uint32_t nc = rows * (D / 2), ns = rows * (D / 16);
    uint8_t *dst = ring + st * C::kStage, *dsc = dst + (1 + C::VPG) * C::kCodes;
    if (!saga_in_bounds(b < p.B && kh < p.h_k && left > 0 && t + rows <= p.cap && st < ST, p.err)) {
      sm100::mbar_arrive(&bars.full[st]);
      return;
    }
    sm100::mbar_arrive_expect_tx(&bars.full[st], (nc + ns) * (1 + C::VPG));
    q4::bulk_load(dst, p.kc + kb + t * (D / 2), nc, &bars.full[st]);
    q4::bulk_load(dsc, p.ks + kb / 8 + t * (D / 16), ns, &bars.full[st]);
#pragma unroll
    for (int v = 0; v < C::VPG; ++v) {
      const int64_t vo = vb + v * p.vc_sh;
      q4::bulk_load(dst + (1 + v) * C::kCodes, p.vc + vo + t * (D / 2), nc, &bars.full[st]);
      q4::bulk_load(dsc + (1 + v) * C::kScales, p.vs + vo / 8 + t * (D / 16), ns, &bars.full[st]);
    }
  };
  const int g = lane >> 2, tq = lane & 3;
  const int slab = warp / NG, vg = warp % NG;
  const int key = (g >> 1) + 4 * (g & 1);           // this lane's key of an 8-key tile: column g
  const int row0 = slab * C::kKeys;
  const float lo_row = g < 4 ? 0.f : -1.f;           // mode S: rows 4-7 take the low halves
  float *const merge = reinterpret_cast<float *>(ring + C::kRing);
  q4::Stage<ST> at;
  int turn = 0;                                      // the warp that issues next
  bool first = true, ok = true;

  while (x0 < x1) {
    const q4::Piece pc = q4::next_piece<KC>(p, seq, x0, x1);
    const int b = pc.b, kh = pc.kh;
    if (first && tid == 0)
      for (int i = 0; i < bars.kAhead; ++i) bars.issue(p, i, 1u, pc, pc.c0, i, seq, x0, x1, load);
    first = false;
    __syncwarp();
    float m[NRT], l[NRT], acc[NRT][NM][4];
#pragma unroll
    for (int r = 0; r < NRT; ++r) {
      m[r] = -INFINITY; l[r] = 0.f;
#pragma unroll
      for (int n = 0; n < NM; ++n) acc[r][n][0] = acc[r][n][1] = acc[r][n][2] = acc[r][n][3] = 0.f;
    }

    // ---- query rows ----------------------------------------------------------
    uint32_t qh[MT][D / 16][4], ql[Q2 ? MT : 1][Q2 ? D / 16 : 1][4];
    float fac[2 * MT];                               // raw score -> log2 units, per row tile
    const float unit = p.scale * kLog2e, gk = p.k_g != nullptr ? __ldg(p.k_g + kh) : 1.f;
    const T *qb = static_cast<const T *>(p.q) + b * p.q_sb;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // rows g (the even tile) and g + 8 (the odd one)
      const int r0 = 2 * mt, r1 = 2 * mt + 1;
      const int hd0 = MODE == kRowsS ? (g & 3) : g;
      const int hd1 = MODE == kRowsS ? (g & 3) : (MODE == kRowsL16 ? 8 + g : g);
      const int v0 = MODE == kRowsL16 ? 0 : vg * VPW + r0, v1 = MODE == kRowsL16 ? 0 : vg * VPW + r1;
      fac[r0] = q4::score_factor(
          unit, q4::q_frag<D, T, Q2, 0>(qb + static_cast<int64_t>(kh * G + v0 * HPV + hd0) * p.q_sh, hd0 < HPV, tq,
                                        qh[mt], ql[Q2 ? mt : 0]), gk);
      if constexpr (NRT % 2 == 0) {
        fac[r1] = q4::score_factor(
            unit, q4::q_frag<D, T, Q2, 1>(qb + static_cast<int64_t>(kh * G + v1 * HPV + hd1) * p.q_sh, hd1 < HPV, tq,
                                          qh[mt], ql[Q2 ? mt : 0]), gk);
      } else {
        fac[r1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          qh[mt][i][1] = qh[mt][i][3] = 0u;
          if constexpr (Q2) ql[mt][i][1] = ql[mt][i][3] = 0u;
        }
      }
    }

    for (int c = pc.c0; c < pc.c1; ++c) {
      // a warp that gave up still meets the others at the barriers below
      if (!ok) continue;
      if (warp == turn && lane == 0)
        bars.issue(p, at.refill(), at.refill_parity(), pc, c, bars.kAhead, seq, x0, x1, load);
      turn = (turn + 1) % kWarps;
      __syncwarp();
      ok = __all_sync(0xffffffffu, q4::wait_bar(&bars.full[at.st], at.phase, &bars.abort));
      if (!ok) {
        if (lane == 0) bars.give_up(p.err);
        continue;
      }
      const int left = pc.L - c * KC - row0;
      if (left > 0) {
        const uint8_t *codes = ring + at.st * C::kStage;
        const uint8_t *scales = codes + (1 + C::VPG) * C::kCodes;
        const uint8_t *kc = codes + row0 * (D / 2), *ks = scales + row0 * (D / 16);

        // ---- scores of the warp's keys: x[tile][key tile][2 keys of this lane] -------
        float x[NRT][NT][2];
        {
          float d[NT][MT][4];
          q4::score_tiles<D, MT, NT, Q2>(kc + key * (D / 2), ks + key * (D / 16), tq, qh, ql, d);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < NRT; ++r) {
              x[r][nt][0] = d[nt][r / 2][r % 2 * 2];
              x[r][nt][1] = d[nt][r / 2][r % 2 * 2 + 1];
            }
        }
        if (left < C::kKeys) {                 // columns 2 tq, 2 tq + 1 are keys tq, tq + 4
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < NRT; ++r) {
              if (8 * nt + tq >= left) x[r][nt][0] = -INFINITY;
              if (8 * nt + tq + 4 >= left) x[r][nt][1] = -INFINITY;
            }
        }

        // ---- the chunk's maxima; running maxima, followed lazily --------------
        float cand[NRT];
        bool grow = false;
#pragma unroll
        for (int r = 0; r < NRT; ++r) {
          float mx = fmaxf(x[r][0][0], x[r][0][1]);
#pragma unroll
          for (int nt = 1; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(x[r][nt][0], x[r][nt][1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          cand[r] = mx * fac[r];
          grow |= cand[r] > m[r] + kLazy;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int r = 0; r < NRT; ++r) {
            const float mn = cand[r] > m[r] + kLazy ? cand[r] : m[r];
            const float corr = m[r] == -INFINITY ? 0.f : q4::ex2(m[r] - mn);
            m[r] = mn;
            l[r] *= corr;
            const float c0 = __shfl_sync(0xffffffffu, corr, tq * 8);
            const float c1 = __shfl_sync(0xffffffffu, corr, tq * 8 + 4);
#pragma unroll
            for (int n = 0; n < NM; ++n) {
              acc[r][n][0] *= c0; acc[r][n][1] *= c1;
              acc[r][n][2] *= c0; acc[r][n][3] *= c1;
            }
          }
        }

        // ---- probabilities, as B operands: keys 16 j + .. of row g -------------
        uint32_t ph[NRT][NJ][2], pl[MODE == kRowsS ? 1 : NRT][NJ][2];
        float to_row[NRT];                       // from the chunk's maximum to the row's
#pragma unroll
        for (int r = 0; r < NRT; ++r) {
          const float bias = cand[r] == -INFINITY ? 0.f : kPShift - cand[r];
          to_row[r] = cand[r] == -INFINITY ? 0.f : q4::ex2(cand[r] - m[r]);
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float p0 = q4::ex2(fmaf(x[r][nt][0], fac[r], bias));
            const float p1 = q4::ex2(fmaf(x[r][nt][1], fac[r], bias));
            sum += p0 + p1;
            // the high half is p cut off at fp16's 11 bits, the low one the rest
            const float h0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u);
            const float h1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
            if constexpr (MODE == kRowsS) {
              ph[r][nt / 2][nt % 2] = q4::pack_f16_rz(fmaf(lo_row, h0, p0), fmaf(lo_row, h1, p1));
            } else {
              ph[r][nt / 2][nt % 2] = q4::pack_f16_rz(p0, p1);
              pl[r][nt / 2][nt % 2] = q4::pack_f16(p0 - h0, p1 - h1);
            }
          }
          l[r] = fmaf(to_row[r], sum, l[r]);
        }

        // ---- P V: MMA key k of a 16-key step is row tq (k = 2 tq), tq + 4 (2 tq + 1),
        // tq + 8 (2 tq + 8), tq + 12 (2 tq + 9); this lane's dims: D/8 from g D/8,
        // rows g and g + 8 of output tile n its dims 2 n and 2 n + 1
#pragma unroll
        for (int vw = 0; vw < VPW; ++vw) {
          const int v = vg * VPW + vw;
          // the factors of the tile's rows 2 tq and 2 tq + 1, ahead of the products (mode L16:
          // behind them, where they hold no registers meanwhile)
          float f0, f1;
          const auto columns = [&](int r) {
            f0 = __shfl_sync(0xffffffffu, to_row[r], tq * 8);
            f1 = __shfl_sync(0xffffffffu, to_row[r], tq * 8 + 4);
          };
          if (MODE != kRowsL16) columns(vw);
          const uint8_t *vc = codes + (1 + v) * C::kCodes + (row0 + tq) * (D / 2) + g * (D / 16);
          const uint8_t *vs = scales + (1 + v) * C::kScales + (row0 + tq) * (D / 16) + (D == 64 ? g / 2 : g);
#pragma unroll
          for (int u = 0; u < D / 64; ++u) {         // eight dims at a time
            float t[NP][4][4];                       // of tile vw (mode L16: of both)
#pragma unroll
            for (int j0 = 0; j0 < NJ; j0 += JB) {
              uint32_t a[JB][4][4];
#pragma unroll
              for (int j = 0; j < JB; ++j)
#pragma unroll
                for (int pr = 0; pr < 2; ++pr) {
                  const int r0 = 16 * (j0 + j) + 8 * pr, r1 = r0 + 4;
                  const uint32_t wa = *reinterpret_cast<const uint32_t *>(vc + r0 * (D / 2) + 4 * u);
                  const uint32_t wb = *reinterpret_cast<const uint32_t *>(vc + r1 * (D / 2) + 4 * u);
                  q4::value_pair(wa, wb, vs[r0 * (D / 16)], vs[r1 * (D / 16)], pr, a[j]);
                }
#pragma unroll
              for (int i = 0; i < NP; ++i) {
                const int r = MODE == kRowsL16 ? i : vw;
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                  const int k = j0 + j;
#pragma unroll
                  for (int n = 0; n < 4; ++n) {
                    if (k == 0) q4::mma_first(t[i][n], a[j][n], ph[r][k][0], ph[r][k][1]);
                    else q4::mma(t[i][n], a[j][n], ph[r][k][0], ph[r][k][1]);
                  }
                  if constexpr (MODE != kRowsS) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) q4::mma(t[i][n], a[j][n], pl[r][k][0], pl[r][k][1]);
                  }
                }
              }
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const int r = MODE == kRowsL16 ? i : vw;
              if (MODE == kRowsL16) columns(r);
#pragma unroll
              for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  acc[r][4 * u + n][e] = fmaf(e % 2 ? f1 : f0, t[i][n][e], acc[r][4 * u + n][e]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&bars.empty[at.st]);
      at.advance();
    }

    // ---- the slabs' states, merged pairwise into slab 0 ------------------------
#pragma unroll
    for (int r = 0; r < NRT; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
#pragma unroll
    for (int n = C::SL; n > 1; n = (n + 1) / 2) {    // n slabs left: the upper half joins the lower
      const int h = (n + 1) / 2;
#pragma unroll
      for (int s0 = h; s0 < n; s0 += C::kSlots) {    // as many at a time as there is room for
        sm100::named_bar(1, kWarps * 32);            // the last reads of `merge` are done
        if (slab >= s0 && slab < n && slab < s0 + C::kSlots) {
          float *o = merge + ((slab - s0) * NG + vg) * (C::kState * 32) + lane;
#pragma unroll
          for (int r = 0; r < NRT; ++r) {
#pragma unroll
            for (int e = 0; e < NM * 4; ++e) o[(r * (NM * 4 + 2) + e) * 32] = acc[r][e / 4][e % 4];
            o[(r * (NM * 4 + 2) + NM * 4) * 32] = m[r];
            o[(r * (NM * 4 + 2) + NM * 4 + 1) * 32] = l[r];
          }
        }
        sm100::named_bar(1, kWarps * 32);
        const int from = slab + h;                   // the slab that joins this one
        if (from >= s0 && from < n && from < s0 + C::kSlots) {
          const float *o = merge + ((from - s0) * NG + vg) * (C::kState * 32) + lane;
#pragma unroll
          for (int r = 0; r < NRT; ++r) {
            const float *q = o + r * (NM * 4 + 2) * 32;
            merge_state<NM>(m[r], l[r], acc[r], q[NM * 4 * 32], q[(NM * 4 + 1) * 32], tq,
                            [&](int e) { return q[e * 32]; });
          }
        }
      }
    }
    if (slab != 0) continue;

    // ---- the heads' outputs, or their records ----------------------------------
    const bool whole = pc.c0 == 0 && pc.c1 == q4::chunks_of<KC>(pc.L);
    const bool gave_up = bars.gave_up();
#pragma unroll
    for (int r = 0; r < NRT; ++r) {
      const int v = MODE == kRowsL16 ? 0 : vg * VPW + r;
      const float gv = p.v_g != nullptr ? __ldg(p.v_g + kh * C::VPG + v) : 1.f;
      if constexpr (MODE == kRowsS) {                // the low halves' sums: rows 4-7
#pragma unroll
        for (int n = 0; n < NM; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][n][e] += __shfl_xor_sync(0xffffffffu, acc[r][n][e], 2);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mh = __shfl_sync(0xffffffffu, m[r], tq * 8 + 4 * e);
        const float lh = __shfl_sync(0xffffffffu, l[r], tq * 8 + 4 * e);
        const int hd = (MODE == kRowsL16 ? 8 * r : 0) + 2 * tq + e;
        if (hd >= HPV || (MODE == kRowsS && tq >= 2)) continue;
        const int hg = v * HPV + hd;                 // head of the group
        float f = 1.f, gh = 1.f;                     // the head scale comes last, times values that fit
        float *o;
        if (whole) {
          o = p.out + (static_cast<int64_t>(b) * p.h_q + kh * G + hg) * D;
          f = gave_up ? __int_as_float(0x7fc00000) : kQ4Unit / lh;
          gh = gv;
        } else {
          if (!saga_in_bounds(cta < p.S && hg < G, p.err)) continue;      // q4_plan: S + B h_k records of G
          o = p.partials + (static_cast<int64_t>(cta + b * p.h_k + kh) * G + hg) * (D + kRecPad);
          if (g == 0) *reinterpret_cast<float4 *>(o) = make_float4(mh, lh, gave_up ? 1.f : 0.f, 0.f);
          o += kRecPad;
        }
#pragma unroll
        for (int n = 0; n < NM; ++n)
          *reinterpret_cast<float2 *>(o + g * (D / 8) + 2 * n) =
              make_float2(acc[r][n][e] * f * gh, acc[r][n][2 + e] * f * gh);
      }
    }
  }
  if (tid == 0 && !ok) bars.drain(at.st, at.phase);
}

// Rows that several CTAs share: their records {m, l, gave up, -, acc} (m in log2
// units) merged in CTA order. One CTA per (b, query head): the largest maximum,
// then kCombAt records' weights at a time and their sums, each thread one dim of
// every kPar-th record with several loads under way (a row of batch 1 has a
// record of every CTA).
constexpr int kCombThreads = 256;
constexpr int kCombWarps = kCombThreads / 32;
constexpr int kCombAt = 128;

template <int D, int CH>
__global__ void __launch_bounds__(kCombThreads) q4_combine_kernel(const Q4Params p) {
  constexpr int kPar = kCombThreads / D;
  __shared__ float s_acc[kCombThreads], s_w[kCombAt], s_m[kCombWarps], s_l[kCombWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.h_q / p.h_k;
  const int b = blockIdx.x / p.h_q, j = blockIdx.x % p.h_q, kh = j / G;
  const q4::Work work = q4::work_of<CH>(p, lane, false);
  int64_t start = 0;                                 // chunks of the sequences before b
  for (int i = lane; i < b; i += 32) start += static_cast<int64_t>(q4::chunks_of<CH>(q4::length(p, i, false))) * p.h_k;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) start += __shfl_xor_sync(0xffffffffu, start, o);
  const int nb = q4::chunks_of<CH>(q4::length(p, b, false));
  if (nb == 0) return;
  const int64_t x = start + static_cast<int64_t>(kh) * nb;
  const int i0 = work.cta_of(x), n = work.cta_of(x + nb - 1) - i0 + 1;
  if (n == 1 || !saga_in_bounds(i0 >= 0 && n > 0 && i0 + n <= p.S, p.err)) return;   // written by its one CTA

  // a CTA's record of the next row follows G (D + kRecPad) floats on, and so does
  // the next CTA's of this row
  const int64_t step = static_cast<int64_t>(G) * (D + kRecPad);
  const float *rec = p.partials + (i0 + b * p.h_k + kh) * step + (j % G) * (D + kRecPad);
  float m = -INFINITY;
  for (int i = tid; i < n; i += kCombThreads) {
    const float4 h = *reinterpret_cast<const float4 *>(rec + i * step);
    m = fmaxf(m, h.z != 0.f ? INFINITY : h.x);       // a CTA that gave up: NaN below
  }
  m = warp_max(m);
  if (lane == 0) s_m[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombWarps; ++w) m = fmaxf(m, s_m[w]);
  float a = 0.f, l = 0.f;
  for (int r0 = 0; r0 < n; r0 += kCombAt) {
    const int k = min(kCombAt, n - r0);
    __syncthreads();
    if (tid < k) {
      const float2 h = *reinterpret_cast<const float2 *>(rec + (r0 + tid) * step);
      const float c = h.x == -INFINITY ? 0.f : q4::ex2(h.x - m);
      s_w[tid] = c;
      l = fmaf(c, h.y, l);
    }
    __syncthreads();
#pragma unroll 8
    for (int i = tid / D; i < k; i += kPar) a = fmaf(s_w[i], rec[(r0 + i) * step + kRecPad + tid % D], a);
  }
  l = warp_sum(l);
  if (lane == 0) s_l[warp] = l;
  s_acc[tid] = a;
  __syncthreads();
  if (tid >= D) return;
  l = s_l[0];
#pragma unroll
  for (int w = 1; w < kCombWarps; ++w) l += s_l[w];
#pragma unroll
  for (int i = 1; i < kPar; ++i) a += s_acc[tid + i * D];
  const float gv = p.v_g != nullptr ? __ldg(p.v_g + j / (p.h_q / p.h_v)) : 1.f;
  p.out[static_cast<int64_t>(blockIdx.x) * D + tid] = m == INFINITY ? __int_as_float(0x7fc00000) : a / l * kQ4Unit * gv;
}

template <int D, int VPW, int MODE, int NG, typename T>
cudaError_t launch_cfg(const Q4Params &p, cudaStream_t st) {
  using C = QD<D, VPW, MODE, NG>;
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(q4_dense_kernel<D, VPW, MODE, NG, T>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  e = launch_pdl(q4_dense_kernel<D, VPW, MODE, NG, T>, dim3(p.S), dim3(kThreads), C::kSmem, st, p);
  if (e != cudaSuccess || p.max_l_kv <= C::KC) return e;   // rows of one chunk are never shared
  return launch_pdl(q4_combine_kernel<D, C::KC>, dim3(p.B * p.h_q), dim3(kCombThreads), 0, st, p);
}

// f(cfg) with the configuration of a head layout: S up to 4 query heads per
// value head, L8 up to 8, L16 above (one value head); four value heads are
// shared between two groups of warps, so that a warp's sums stay in registers.
template <int D, typename F>
auto with_cfg(int h_q, int h_k, int h_v, F f) {
  const int vpg = h_v / h_k, hpv = h_q / h_v;
  if (vpg == 4) return f(QD<D, 2, kRowsS, 2>{});
  if (vpg == 2) return hpv <= 4 ? f(QD<D, 2, kRowsS, 1>{}) : f(QD<D, 2, kRowsL8, 1>{});
  return hpv <= 4 ? f(QD<D, 1, kRowsS, 1>{}) : (hpv <= 8 ? f(QD<D, 1, kRowsL8, 1>{}) : f(QD<D, 1, kRowsL16, 1>{}));
}

template <typename T>
struct LaunchQ4 {
  const Q4Params &p;
  cudaStream_t st;
  template <int D, int VPW, int MODE, int NG>
  cudaError_t operator()(QD<D, VPW, MODE, NG>) const {
    return launch_cfg<D, VPW, MODE, NG, T>(p, st);
  }
};

}  // namespace

int q4_dense_chunk(int d, int h_q, int h_k, int h_v) {
  auto chunk = [](auto c) { return decltype(c)::KC; };
  return d == 64 ? with_cfg<64>(h_q, h_k, h_v, chunk) : with_cfg<128>(h_q, h_k, h_v, chunk);
}

cudaError_t launch_q4_dense(const Q4Params &p, int dtype, int d, cudaStream_t st) {
  if (!dense_supports(p.h_q, p.h_k, p.h_v) || (d != 64 && d != 128)) return cudaErrorInvalidValue;
  if (dtype == SAGA_BF16)
    return d == 64 ? with_cfg<64>(p.h_q, p.h_k, p.h_v, LaunchQ4<uint16_t>{p, st})
                   : with_cfg<128>(p.h_q, p.h_k, p.h_v, LaunchQ4<uint16_t>{p, st});
  return d == 64 ? with_cfg<64>(p.h_q, p.h_k, p.h_v, LaunchQ4<float>{p, st})
                 : with_cfg<128>(p.h_q, p.h_k, p.h_v, LaunchQ4<float>{p, st});
}

}  // namespace saga
