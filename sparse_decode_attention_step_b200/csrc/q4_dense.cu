// Full-attention decode over a 4-bit cache: Eq. (2-4) over every position, for
// GQA (h_k == h_v) and SAGA heads (VPG = h_v / h_k value heads per key head).
//
// One CTA per (b, key head, split of l_kv). A producer warp copies chunks of
// positions (codes and scales of the key head and its VPG value heads, each a
// contiguous range) through a ring of shared-memory stages with untiled bulk
// copies. Eight compute warps each own 32 positions of a chunk (and, with four
// value heads, two of them) and keep their own running softmax, so they meet
// only at the ring and at the end. A warp works in registers throughout:
//
//   scores   S[rows x keys] = Q K^T, mma.sync m16n8k16 with the query rows on M
//            and eight keys on N: a lane converts the consecutive codes of one
//            key row into the B operand;
//   softmax  per row (a row's scores sit in the four lanes of a quad);
//   output   O^T[dims x rows] += V^T P^T with the dims on M and the score rows on
//            N: the scores' accumulators have the layout of the B operand, and
//            a lane converts the same dims of four keys into the A operand.
//
// Probabilities are scaled by 2^7 and split into a high and a low fp16 half
// (22 bits; fp16 alone would cost the fp32 output its precision), with fp32
// sums. The running maximum follows the scores lazily: a row is rescaled when
// its maximum has grown by more than 2^8 of weight, so that P stays below 2^15.
//
// Rows of the score tile (each 8-row tile belongs to one value head):
//   S    at most 4 query heads per value head: rows 0-3 the heads, rows 4-7 the
//        same heads again; rows 0-3 put the high half of P into the product,
//        rows 4-7 the low half, and the sums are added at the end: one MMA
//        where a high and a low one would each leave half the tile empty;
//   L8   5 to 8 heads: one tile, a high and a low MMA into the same sums;
//   L16  9 to 16 heads (one value head): two such tiles.
#include <atomic>

#include "kernels.h"
#include "plan.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kWarps = 8;                       // compute warps; one more produces
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kKeysPerWarp = 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 7.f;                  // P is scaled by 2^kPShift
constexpr float kLazy = 8.f;                    // log2 growth of a row's maximum that rescales it
constexpr int kMaxDevices = 64;

enum { kRowsS = 0, kRowsL8 = 1, kRowsL16 = 2 };

// VPW value heads per warp, NG groups of warps: VPG = VPW * NG.
template <int D, int VPW, int MODE, int NG>
struct QD {
  static constexpr int VPG = VPW * NG;
  static constexpr int SL = kWarps / NG;                        // position slabs of a chunk
  static constexpr int KC = SL * kKeysPerWarp;
  static constexpr int NRT = MODE == kRowsL16 ? 2 : VPW;        // 8-row score tiles per warp
  static constexpr int MT = (NRT + 1) / 2;                      // 16-row MMA tiles
  static constexpr int NM = D / 16;                             // 16-dim MMA tiles of the output
  static constexpr int kCodes = KC * D / 2, kScales = KC * D / 16;
  static constexpr int kStage = (kCodes + kScales) * (1 + VPG);
  // two CTAs per SM where the registers allow (the accumulators of a warp are
  // 16 per score tile at d = 64, 32 at d = 128)
  static constexpr int kCtas = NRT * NM <= 8 ? 2 : 1;
  static constexpr int kBudget = kCtas == 2 ? 108 * 1024 : 200 * 1024;
  static constexpr int kStages = kBudget / kStage < 8 ? kBudget / kStage : 8;
  static constexpr int kRows = NRT * 8;
  static constexpr int kAccRow = D + 4;                         // floats of a merged row
  static constexpr int kMerge = kWarps * kRows * kAccRow * 4;
  static constexpr int kRing = kStages * kStage > kMerge ? kStages * kStage : kMerge;
  static_assert(kStages >= 2, "a ring");
  static_assert(kRing <= kBudget + 20 * 1024, "shared memory");
};

template <int D, int VPW, int MODE, int NG, typename T>
__global__ void __launch_bounds__(kThreads, QD<D, VPW, MODE, NG>::kCtas)
q4_dense_kernel(const Q4Params p) {
  using C = QD<D, VPW, MODE, NG>;
  constexpr bool Q2 = sizeof(T) == 4;
  constexpr int NRT = C::NRT, MT = C::MT, NM = C::NM, ST = C::kStages;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t s_full[ST], s_empty[ST];
  __shared__ float s_m[kWarps][C::kRows], s_l[kWarps][C::kRows];
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x;
  const int b = blockIdx.y / p.h_k, kh = blockIdx.y % p.h_k;
  const int G = p.h_q / p.h_k, HPV = G / C::VPG;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&s_empty[i], kWarps);
    }
    s_abort = 0;
    sm100::fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int64_t L = q4::length(p, b, tid == 0 && s == 0);
  const int64_t t_begin = static_cast<int64_t>(s) * p.split_len;
  if (t_begin >= L) return;
  const int64_t t_end = min(t_begin + p.split_len, L);
  const int nchunks = static_cast<int>((t_end - t_begin + C::KC - 1) / C::KC);

  if (warp == kWarps) {
    // ---- producer ----------------------------------------------------------
    if (lane == 0) {
      const int64_t kb = b * p.kc_sb + kh * p.kc_sh;
      const int64_t vb = b * p.vc_sb + static_cast<int64_t>(kh) * C::VPG * p.vc_sh;
      int c = 0;
      for (; c < nchunks; ++c) {
        const int st = c % ST;
        if (!q4::wait_bar(&s_empty[st], ((c / ST) & 1) ^ 1, &s_abort)) break;
        const int64_t t = t_begin + static_cast<int64_t>(c) * C::KC;
        // whole groups of four rows: 16 bytes of scales at least (cap is a multiple of 4)
        const int64_t left = t_end - t;
        const uint32_t rows = left < C::KC ? static_cast<uint32_t>((left + 3) & ~3ll) : C::KC;
        const uint32_t nc = rows * (D / 2), ns = rows * (D / 16);
        uint8_t *dst = ring + st * C::kStage;
        sm100::mbar_arrive_expect_tx(&s_full[st], (nc + ns) * (1 + C::VPG));
        q4::bulk_load(dst, p.kc + kb + t * (D / 2), nc, &s_full[st]);
        uint8_t *dsc = dst + (1 + C::VPG) * C::kCodes;
        q4::bulk_load(dsc, p.ks + kb / 8 + t * (D / 16), ns, &s_full[st]);
#pragma unroll
        for (int v = 0; v < C::VPG; ++v) {
          const int64_t vo = vb + v * p.vc_sh;
          q4::bulk_load(dst + (1 + v) * C::kCodes, p.vc + vo + t * (D / 2), nc, &s_full[st]);
          q4::bulk_load(dsc + (1 + v) * C::kScales, p.vs + vo / 8 + t * (D / 16), ns, &s_full[st]);
        }
      }
      if (c < nchunks) {
        atomicOr(p.err, SAGA_DEVERR_TIMEOUT);
        *reinterpret_cast<volatile int *>(&s_abort) = 1;
      }
      // the copies in flight land before the ring is used again
      for (int i = c > ST ? c - ST : 0; i < c; ++i) sm100::mbar_wait(&s_full[i % ST], (i / ST) & 1);
    }
    __syncwarp();
  }

  const int g = lane >> 2, tq = lane & 3;
  const int slab = warp / NG, vg = warp % NG;
  float m[NRT], l[NRT], acc[NRT][NM][4];
#pragma unroll
  for (int r = 0; r < NRT; ++r) {
    m[r] = -INFINITY; l[r] = 0.f;
#pragma unroll
    for (int n = 0; n < NM; ++n) acc[r][n][0] = acc[r][n][1] = acc[r][n][2] = acc[r][n][3] = 0.f;
  }

  if (warp < kWarps) {
    // ---- query rows ----------------------------------------------------------
    uint32_t qh[MT][D / 16][4], ql[Q2 ? MT : 1][Q2 ? D / 16 : 1][4];
    float fac[2 * MT];                           // raw score -> log2 units, per row tile
    const float unit = p.scale * kLog2e * kQ4Unit * (p.k_g != nullptr ? __ldg(p.k_g + kh) : 1.f);
    const T *qb = static_cast<const T *>(p.q) + b * p.q_sb;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // rows g (the even tile) and g + 8 (the odd one)
      const int r0 = 2 * mt, r1 = 2 * mt + 1;
      const int hd0 = MODE == kRowsS ? (g & 3) : (MODE == kRowsL16 ? g : g);
      const int hd1 = MODE == kRowsS ? (g & 3) : (MODE == kRowsL16 ? 8 + g : g);
      const int v0 = MODE == kRowsL16 ? 0 : vg * VPW + r0, v1 = MODE == kRowsL16 ? 0 : vg * VPW + r1;
      fac[r0] = unit * q4::q_frag<D, T, Q2, 0>(
                           qb + static_cast<int64_t>(kh * G + v0 * HPV + hd0) * p.q_sh, hd0 < HPV, tq,
                           qh[mt], ql[Q2 ? mt : 0]);
      if constexpr (NRT % 2 == 0) {
        fac[r1] = unit * q4::q_frag<D, T, Q2, 1>(
                             qb + static_cast<int64_t>(kh * G + v1 * HPV + hd1) * p.q_sh, hd1 < HPV, tq,
                             qh[mt], ql[Q2 ? mt : 0]);
      } else {
        fac[r1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          qh[mt][i][1] = qh[mt][i][3] = 0u;
          if constexpr (Q2) ql[mt][i][1] = ql[mt][i][3] = 0u;
        }
      }
    }

    const int key = (g >> 1) + 4 * (g & 1);       // this lane's key of an 8-key tile: column g
    bool ok = true;
    for (int c = 0; c < nchunks; ++c) {
      const int st = c % ST;
      if (!q4::wait_bar(&s_full[st], (c / ST) & 1, &s_abort)) { ok = false; break; }
      const int row0 = slab * kKeysPerWarp;
      const int64_t left = t_end - (t_begin + static_cast<int64_t>(c) * C::KC + row0);
      if (left > 0) {
        const uint8_t *codes = ring + st * C::kStage;
        const uint8_t *scales = codes + (1 + C::VPG) * C::kCodes;
        const uint8_t *kc = codes + row0 * (D / 2), *ks = scales + row0 * (D / 16);

        // ---- scores of 32 keys: x[tile][key tile][2 keys of this lane] -------
        float x[NRT][4][2];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          float d[MT][4];
          q4::score_tile<D, MT, Q2>(kc + (8 * nt + key) * (D / 2), ks + (8 * nt + key) * (D / 16), tq,
                                    qh, ql, d);
#pragma unroll
          for (int r = 0; r < NRT; ++r) {
            x[r][nt][0] = d[r / 2][r % 2 * 2];
            x[r][nt][1] = d[r / 2][r % 2 * 2 + 1];
          }
        }
        if (left < kKeysPerWarp) {                 // columns 2 tq, 2 tq + 1 are keys tq, tq + 4
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int r = 0; r < NRT; ++r) {
              if (8 * nt + tq >= left) x[r][nt][0] = -INFINITY;
              if (8 * nt + tq + 4 >= left) x[r][nt][1] = -INFINITY;
            }
        }

        // ---- running maxima, followed lazily ----------------------------------
        float cand[NRT];
        bool grow = false;
#pragma unroll
        for (int r = 0; r < NRT; ++r) {
          float mx = fmaxf(x[r][0][0], x[r][0][1]);
#pragma unroll
          for (int nt = 1; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(x[r][nt][0], x[r][nt][1]));
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
        uint32_t ph[NRT][2][2], pl[MODE == kRowsS ? 1 : NRT][2][2];
#pragma unroll
        for (int r = 0; r < NRT; ++r) {
          const float bias = m[r] == -INFINITY ? 0.f : kPShift - m[r];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const float p0 = q4::ex2(fmaf(x[r][nt][0], fac[r], bias));
            const float p1 = q4::ex2(fmaf(x[r][nt][1], fac[r], bias));
            l[r] += p0 + p1;
            const float h0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u);
            const float h1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
            if constexpr (MODE == kRowsS) {
              ph[r][nt / 2][nt % 2] = q4::pack_f16(g < 4 ? h0 : p0 - h0, g < 4 ? h1 : p1 - h1);
            } else {
              ph[r][nt / 2][nt % 2] = q4::pack_f16(h0, h1);
              pl[r][nt / 2][nt % 2] = q4::pack_f16(p0 - h0, p1 - h1);
            }
          }
        }

        // ---- P V: MMA key k of a 16-key step is row tq (2 tq), tq + 4 (2 tq + 1),
        // tq + 8 (2 tq + 8), tq + 12 (2 tq + 9); this lane's dims: D/8 from g D/8
#pragma unroll
        for (int vw = 0; vw < VPW; ++vw) {
          const int v = vg * VPW + vw;
          const uint8_t *vc = codes + (1 + v) * C::kCodes + row0 * (D / 2) + g * (D / 16);
          const uint8_t *vs = scales + (1 + v) * C::kScales + row0 * (D / 16) + (D == 64 ? g / 2 : g);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t h[4][NM];                     // f16x2 of dims 2 n, 2 n + 1 of key i
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 16 * j + 4 * i + tq;
              const uint32_t sc = q4::scale_f16(vs[row * (D / 16)]);
              uint32_t w[D / 64];
              if constexpr (D == 64) {
                w[0] = *reinterpret_cast<const uint32_t *>(vc + row * (D / 2));
              } else {
                const uint2 y = *reinterpret_cast<const uint2 *>(vc + row * (D / 2));
                w[0] = y.x; w[1] = y.y;
              }
#pragma unroll
              for (int u = 0; u < D / 64; ++u) {
                uint32_t t4[4];
                q4::codes_f16(w[u], t4);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[i][4 * u + e] = q4::mul_f16x2(t4[e], sc);
              }
            }
#pragma unroll
            for (int n = 0; n < NM; ++n) {
              const uint32_t a[4] = {__byte_perm(h[0][n], h[1][n], 0x5410), __byte_perm(h[0][n], h[1][n], 0x7632),
                                     __byte_perm(h[2][n], h[3][n], 0x5410), __byte_perm(h[2][n], h[3][n], 0x7632)};
              if constexpr (MODE == kRowsL16) {
#pragma unroll
                for (int r = 0; r < NRT; ++r) {
                  q4::mma(acc[r][n], a, ph[r][j][0], ph[r][j][1]);
                  q4::mma(acc[r][n], a, pl[r][j][0], pl[r][j][1]);
                }
              } else {
                q4::mma(acc[vw][n], a, ph[vw][j][0], ph[vw][j][1]);
                if constexpr (MODE == kRowsL8) q4::mma(acc[vw][n], a, pl[vw][j][0], pl[vw][j][1]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&s_empty[st]);
    }
    if (!ok) {
      if (lane == 0) atomicOr(p.err, SAGA_DEVERR_TIMEOUT);
      *reinterpret_cast<volatile int *>(&s_abort) = 1;
    }
#pragma unroll
    for (int r = 0; r < NRT; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
  }
  __syncthreads();                                  // every copy has landed and been read

  // ---- the warps' states, merged in slab order into the heads' records ------
  float *red = reinterpret_cast<float *>(ring);     // [kWarps][kRows][kAccRow]
  if (warp < kWarps) {
#pragma unroll
    for (int r = 0; r < NRT; ++r) {
      if (tq == 0) { s_m[warp][8 * r + g] = m[r]; s_l[warp][8 * r + g] = l[r]; }
      float *o = red + (warp * C::kRows + 8 * r + 2 * tq) * C::kAccRow + g * (D / 8);
#pragma unroll
      for (int n = 0; n < NM; ++n) {
        o[2 * n] = acc[r][n][0];
        o[C::kAccRow + 2 * n] = acc[r][n][1];
        o[2 * n + 1] = acc[r][n][2];
        o[C::kAccRow + 2 * n + 1] = acc[r][n][3];
      }
    }
  }
  __syncthreads();
  const bool gave_up = s_abort != 0;
  for (int idx = tid; idx < G * D; idx += kThreads) {
    const int hd = idx / D, e = idx % D;            // head of the group, dim
    const int v = hd / HPV, hv = hd % HPV;
    const int row = MODE == kRowsL16 ? hv : (v % VPW) * 8 + hv;
    float M = -INFINITY;
#pragma unroll
    for (int sl = 0; sl < C::SL; ++sl) M = fmaxf(M, s_m[sl * NG + v / VPW][row]);
    float a = 0.f, ll = 0.f;
#pragma unroll
    for (int sl = 0; sl < C::SL; ++sl) {
      const int w = sl * NG + v / VPW;
      const float mw = s_m[w][row];
      const float wt = mw == -INFINITY ? 0.f : q4::ex2(mw - M);
      const float *o = red + (w * C::kRows + row) * C::kAccRow + e;
      float x = o[0];
      if constexpr (MODE == kRowsS) x += o[4 * C::kAccRow];
      a = fmaf(wt, x, a);
      ll = fmaf(wt, s_l[w][row], ll);
    }
    const int j = kh * G + hd;
    float *rec = p.partials + (static_cast<int64_t>(b * p.h_q + j) * p.S + s) * (D + kRecPad);
    const float vg_ = p.v_g != nullptr ? __ldg(p.v_g + kh * C::VPG + v) : 1.f;
    rec[kRecPad + e] = a * (kQ4Unit * vg_);
    if (e == 0) {
      rec[0] = gave_up ? INFINITY : M * kLn2;
      rec[1] = ll;
      rec[2] = __int_as_float(gave_up ? -1 : static_cast<int>(t_end - t_begin));
      rec[3] = 0.f;
    }
  }
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
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kRing);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(q4_dense_kernel<D, VPW, MODE, NG, T>, dim3(p.S, p.B * p.h_k), dim3(kThreads), C::kRing,
                    st, p);
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

int q4_dense_chunk(int h_k, int h_v) { return h_v / h_k == 4 ? 4 * kKeysPerWarp : 8 * kKeysPerWarp; }

int q4_dense_ctas_per_sm(int d, int h_q, int h_k, int h_v) {
  auto ctas = [](auto c) { return decltype(c)::kCtas; };
  return d == 64 ? with_cfg<64>(h_q, h_k, h_v, ctas) : with_cfg<128>(h_q, h_k, h_v, ctas);
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
