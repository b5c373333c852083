// The score pass of the Atop-N step and its refresh over a 4-bit K cache:
// Eq. 2 scores of every position for the G <= 16 query heads of a key head, then
// either the compare with the thresholds (Atop-N item 1) and the kept lists that
// the gather kernel reads, or the score rows and their top-byte histograms for
// the refresh. The scores of the two modes come from the same instructions and
// are the same bit for bit.
//
// One CTA per (b, key head, split of l_kv). A producer warp copies chunks of 256
// positions (codes and scales, two contiguous ranges) through a ring of
// shared-memory stages with untiled bulk copies; each of eight warps scores
// its 32 positions: mma.sync m16n8k16 with the heads on M and eight keys on N, a
// lane converting consecutive codes of one key row into the B operand. A
// quad of lanes then holds two heads' 32 scores: their masks of kept positions
// come together in two shuffles, and each kept score goes to its key's rank in
// the 32-position block. Fixed places, so the step is deterministic.
#include <atomic>

#include "kernels.h"
#include "plan.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kChunk = kQ4ScanChunk;
constexpr int kMaxDevices = 64;
static_assert(kChunk == kWarps * 32, "a 32-position block per warp");

template <int D>
struct QS {
  static constexpr int kCodes = kChunk * D / 2, kScales = kChunk * D / 16;
  static constexpr int kStage = kCodes + kScales;               // 9 KB (d 64), 18 KB
  static constexpr int kStages = D == 64 ? 6 : 3;
  static constexpr int kRing = kStages * kStage;                // 54 KB: three CTAs per SM
};

template <int D, bool DUMP, typename T>
__global__ void __launch_bounds__(kThreads, kQ4ScanCtasPerSm) q4_scan_kernel(const Q4Params p) {
  using C = QS<D>;
  constexpr bool Q2 = sizeof(T) == 4;
  constexpr int ST = C::kStages;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t s_full[ST], s_empty[ST];
  __shared__ uint32_t s_hist[DUMP ? 16 * 256 : 1];
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x;
  const int b = blockIdx.y / p.h_k, kh = blockIdx.y % p.h_k;
  const int G = p.h_q / p.h_k;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&s_empty[i], kWarps);
    }
    s_abort = 0;
    sm100::fence_mbar_init();
  }
  if (DUMP)
    for (int i = tid; i < 16 * 256; i += kThreads) s_hist[i] = 0u;
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int64_t L = q4::length(p, b, tid == 0 && s == 0);
  const int64_t t_begin = static_cast<int64_t>(s) * p.split_len;
  if (t_begin >= L) return;
  const int64_t t_end = min(t_begin + p.split_len, L);
  const int nchunks = static_cast<int>((t_end - t_begin + kChunk - 1) / kChunk);

  if (warp == kWarps) {
    if (lane == 0) {
      const int64_t kb = b * p.kc_sb + kh * p.kc_sh;
      int c = 0;
      for (; c < nchunks; ++c) {
        const int st = c % ST;
        if (!q4::wait_bar(&s_empty[st], ((c / ST) & 1) ^ 1, &s_abort)) break;
        const int64_t t = t_begin + static_cast<int64_t>(c) * kChunk, left = t_end - t;
        const uint32_t rows = left < kChunk ? static_cast<uint32_t>((left + 3) & ~3ll) : kChunk;
        const uint32_t nc = rows * (D / 2), ns = rows * (D / 16);
        uint8_t *dst = ring + st * C::kStage;
        sm100::mbar_arrive_expect_tx(&s_full[st], nc + ns);
        q4::bulk_load(dst, p.kc + kb + t * (D / 2), nc, &s_full[st]);
        q4::bulk_load(dst + C::kCodes, p.ks + kb / 8 + t * (D / 16), ns, &s_full[st]);
      }
      if (c < nchunks) {
        atomicOr(p.err, SAGA_DEVERR_TIMEOUT);
        atomicExch(p.abort, 1);                    // the gather poisons this step's records
        *reinterpret_cast<volatile int *>(&s_abort) = 1;
        for (int i = c > ST ? c - ST : 0; i < c; ++i) sm100::mbar_wait(&s_full[i % ST], (i / ST) & 1);
      }
    }
    __syncwarp();
  } else {
    const int g = lane >> 2, tq = lane & 3;
    const int j0 = kh * G;
    uint32_t qh[1][D / 16][4], ql[1][Q2 ? D / 16 : 1][4];
    float fac[2], tau[2];
    const float unit = p.scale * kQ4Unit * (p.k_g != nullptr ? __ldg(p.k_g + kh) : 1.f);
    const T *qb = static_cast<const T *>(p.q) + b * p.q_sb + static_cast<int64_t>(j0 + g) * p.q_sh;
    fac[0] = unit * q4::q_frag<D, T, Q2, 0>(qb, g < G, tq, qh[0], ql[0]);
    fac[1] = unit * q4::q_frag<D, T, Q2, 1>(qb + 8 * p.q_sh, g + 8 < G, tq, qh[0], ql[0]);
    if (!DUMP) {
      tau[0] = g < G ? p.tau[b * p.h_q + j0 + g] : INFINITY;
      tau[1] = g + 8 < G ? p.tau[b * p.h_q + j0 + g + 8] : INFINITY;
    }

    bool ok = true;
    for (int c = 0; c < nchunks; ++c) {
      const int st = c % ST;
      if (!q4::wait_bar(&s_full[st], (c / ST) & 1, &s_abort)) { ok = false; break; }
      const int64_t t0 = t_begin + static_cast<int64_t>(c) * kChunk + warp * 32;
      const int left = static_cast<int>(t_end - t0 < 32 ? t_end - t0 : 32);
      float x[2][4][2];
      if (left > 0) {
        const uint8_t *codes = ring + st * C::kStage + warp * 32 * (D / 2);
        const uint8_t *scales = ring + st * C::kStage + C::kCodes + warp * 32 * (D / 16);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          float d[1][4];
          q4::score_tile<D, 1, Q2>(codes + (8 * nt + g) * (D / 2), scales + (8 * nt + g) * (D / 16), tq, qh,
                                   ql, d);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            x[r][nt][0] = d[0][2 * r] * fac[r];
            x[r][nt][1] = d[0][2 * r + 1] * fac[r];
          }
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&s_empty[st]);
      if (left <= 0) continue;

      if constexpr (DUMP) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int hd = g + 8 * r;
          float *row = p.scores_out + (static_cast<int64_t>(b) * p.h_q + j0 + hd) * p.row_stride + t0;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = 8 * nt + 2 * tq + e;
              const bool in = hd < G && k < left;
              if (in && saga_in_bounds(t0 + k < p.row_stride, p.err)) row[k] = x[r][nt][e];
              // top byte of the score's order key, one shared atomic per
              // distinct (head, bin) in the warp
              const uint32_t active = __ballot_sync(0xffffffffu, in);
              if (in) {
                const uint32_t bin = hd * 256 + (order_key(x[r][nt][e]) >> 24);
                const uint32_t peers = __match_any_sync(active, bin);
                if (lane == __ffs(peers) - 1) atomicAdd(&s_hist[bin], static_cast<uint32_t>(__popc(peers)));
              }
            }
        }
      } else {
        const int64_t blk = t0 >> 5;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int hd = g + 8 * r;
          uint32_t mine = 0u;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = 8 * nt + 2 * tq + e;
              mine |= static_cast<uint32_t>(x[r][nt][e] >= tau[r] && k < left) << k;
            }
          uint32_t mask = mine | __shfl_xor_sync(0xffffffffu, mine, 1);
          mask |= __shfl_xor_sync(0xffffffffu, mask, 2);
          const int64_t hrow = (static_cast<int64_t>(b) * p.h_q + j0 + hd) * p.nblk + blk;
          if (hd < G && saga_in_bounds(blk < p.nblk, p.err)) {
            if (tq == 0) p.lmask[hrow] = mask;
            if (mine != 0u) {
#pragma unroll
              for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int k = 8 * nt + 2 * tq + e;
                  if ((mine >> k) & 1u)
                    p.lscore[hrow * 32 + __popc(mask & ((1u << k) - 1u))] = x[r][nt][e];
                }
            }
            if (p.sel_mask != nullptr) {
              uint8_t *sm = p.sel_mask + (static_cast<int64_t>(b) * p.h_q + j0 + hd) * p.row_stride + t0;
              for (int k = tq; k < left; k += 4) sm[k] = static_cast<uint8_t>((mask >> k) & 1u);
            }
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0) {
        atomicOr(p.err, SAGA_DEVERR_TIMEOUT);
        atomicExch(p.abort, 1);
      }
      *reinterpret_cast<volatile int *>(&s_abort) = 1;
    }
  }
  __syncthreads();
  if (DUMP) {
    for (int i = tid; i < G * 256; i += kThreads) {
      const uint32_t n = s_hist[i];
      if (n != 0u) atomicAdd(&p.hist[(static_cast<int64_t>(b) * p.h_q + kh * G) * 256 + i], n);
    }
  }
}

template <int D, bool DUMP, typename T>
cudaError_t launch_scan(const Q4Params &p, cudaStream_t st) {
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(q4_scan_kernel<D, DUMP, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             QS<D>::kRing);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(q4_scan_kernel<D, DUMP, T>, dim3(p.S, p.B * p.h_k), dim3(kThreads), QS<D>::kRing, st, p);
}

template <int D, typename T>
cudaError_t launch_scan_m(const Q4Params &p, bool dump, cudaStream_t st) {
  return dump ? launch_scan<D, true, T>(p, st) : launch_scan<D, false, T>(p, st);
}

}  // namespace

cudaError_t launch_q4_scan(const Q4Params &p, bool dump, int dtype, int d, cudaStream_t st) {
  if (p.h_q / p.h_k > kMaxGroup || (d != 64 && d != 128)) return cudaErrorInvalidValue;
  if (dtype == SAGA_BF16)
    return d == 64 ? launch_scan_m<64, uint16_t>(p, dump, st) : launch_scan_m<128, uint16_t>(p, dump, st);
  return d == 64 ? launch_scan_m<64, float>(p, dump, st) : launch_scan_m<128, float>(p, dump, st);
}

}  // namespace saga
