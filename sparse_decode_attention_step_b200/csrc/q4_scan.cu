// The score passes of the Atop-N step and its refresh over a 4-bit K cache:
// Eq. 2 scores of every position for the G <= 16 query heads of a key head, then
//   step   the compare with the thresholds (Atop-N item 1) and the kept lists that
//          the gather kernel reads,
//   max    the largest score of every group of eight positions (refresh), or
//   dump   the score rows.
// The scores of the three come from the same instructions and are the same bit
// for bit.
//
// The refresh (Atop-N item 2) finds the exact N-th largest of a row without
// storing the row: the N-th largest of its group maxima is a lower bound t0 (N
// groups reach it, so N scores do), and at most 8 N scores, ties aside, reach it
// (they lie in those N groups); when large scores are spread over the row, about
// N (1 + 3.5 N / l_kv). A step pass with t0 lists them, and the select kernel
// below takes the N-th largest of the listed scores and drops the entries under
// it, which leaves the step's own kept lists. The K cache is read twice, at 4.5
// bits a value, where writing and reading the rows would move 8 bytes a score.
//
// As many CTAs as fit on the GPU share the rows (b, key head) in equal runs of
// chunks of 256 positions, whatever the lengths (see Work). The chunks (codes
// and scales, two contiguous ranges) come through a ring of shared-memory stages
// with untiled bulk copies (see Ring); each of eight warps scores its 32
// positions: mma.sync m16n8k16 with the heads on M and eight keys on N, a
// lane converting consecutive codes of one key row into the B operand. A
// quad of lanes then holds two heads' 32 scores: their masks of kept positions
// come together in two shuffles, and a kept score goes to its own place in the
// 32-position block. The step is deterministic.
#include <atomic>

#include "kernels.h"
#include "plan.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = kQ4ScanChunk;
constexpr int kMaxDevices = 64;
static_assert(kChunk == kWarps * 32, "a 32-position block per warp");

template <int D>
struct QS {
  static constexpr int kCodes = kChunk * D / 2, kScales = kChunk * D / 16;
  static constexpr int kStage = kCodes + kScales;               // 9 KB (d 64), 18 KB
  static constexpr int kStages = D == 64 ? 7 : 4;
  static constexpr int kRing = kStages * kStage;                // 63, 72 KB: three CTAs per SM
};

template <int D, int MODE, typename T>
__global__ void __launch_bounds__(kThreads, D == 128 && sizeof(T) == 4 ? 2 : kQ4ScanCtasPerSm)
q4_scan_kernel(const Q4Params p) {
  using C = QS<D>;
  constexpr bool Q2 = sizeof(T) == 4;
  constexpr int ST = C::kStages;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ q4::Ring<kChunk, ST> bars;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.h_q / p.h_k;

  if (tid == 0) bars.init(kWarps);
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int cta = blockIdx.x;
  if (MODE == kQ4Max && cta == 0)
    for (int b = tid; b < p.B; b += kThreads) p.n_groups[b] = static_cast<int32_t>((q4::length(p, b, false) + 31) / 32 * 4);
  const q4::Work work = q4::work_of<kChunk>(p, lane, cta == 0 && warp == 0);
  if (cta >= work.n) return;
  int64_t x0 = work.begin(cta);
  const int64_t x1 = work.begin(cta + 1);
  q4::Seq seq = q4::seq_at<kChunk>(p, lane, x0);

  const auto load = [&](int b, int kh, int64_t L, int c, int st) {
    const int64_t kb = b * p.kc_sb + kh * p.kc_sh;
    const int64_t t = static_cast<int64_t>(c) * kChunk, left = L - t;
    // whole groups of four rows: 16 bytes of scales at least (cap is a multiple of 4)
    const uint32_t rows = left < kChunk ? static_cast<uint32_t>((left + 3) & ~3ll) : kChunk;
    const uint32_t nc = rows * (D / 2), ns = rows * (D / 16);
    uint8_t *dst = ring + st * C::kStage;
    sm100::mbar_arrive_expect_tx(&bars.full[st], nc + ns);
    q4::bulk_load(dst, p.kc + kb + t * (D / 2), nc, &bars.full[st]);
    q4::bulk_load(dst + C::kCodes, p.ks + kb / 8 + t * (D / 16), ns, &bars.full[st]);
  };
  bool ok = true;

  const int g = lane >> 2, tq = lane & 3;
  const bool live[2] = {g < G, g + 8 < G};
  int n_seen = 0;                                    // chunks taken from the ring
  while (x0 < x1) {
  const q4::Piece pc = q4::next_piece<kChunk>(p, seq, x0, x1);
  const int b = pc.b, j0 = pc.kh * G;
  if (n_seen == 0 && tid == 0)
    for (int i = 0; i < bars.kAhead; ++i) ok = ok && bars.issue(p, i, pc, pc.c0, i, seq, x0, x1, load);
  __syncwarp();
  uint32_t qh[1][D / 16][4], ql[1][Q2 ? D / 16 : 1][4];
  float fac[2], thr[2];
  const float unit = p.scale * kQ4Unit * (p.k_g != nullptr ? __ldg(p.k_g + pc.kh) : 1.f);
  const T *qb = static_cast<const T *>(p.q) + b * p.q_sb + static_cast<int64_t>(j0 + g) * p.q_sh;
  fac[0] = unit * q4::q_frag<D, T, Q2, 0>(qb, live[0], tq, qh[0], ql[0]);
  fac[1] = unit * q4::q_frag<D, T, Q2, 1>(qb + 8 * p.q_sh, live[1], tq, qh[0], ql[0]);
  if (MODE == kQ4Step) {
#pragma unroll
    for (int r = 0; r < 2; ++r) thr[r] = live[r] ? p.tau[b * p.h_q + j0 + g + 8 * r] : INFINITY;
  }
  const int64_t row = static_cast<int64_t>(b) * p.h_q + j0 + g;     // this lane's first head

  for (int c = pc.c0; c < pc.c1; ++c, ++n_seen) {
    const int st = n_seen % ST;
    if (warp == n_seen % kWarps && lane == 0)
      ok = ok && bars.issue(p, n_seen + bars.kAhead, pc, c, bars.kAhead, seq, x0, x1, load);
    __syncwarp();
    if (!__all_sync(0xffffffffu, ok && q4::wait_bar(&bars.full[st], (n_seen / ST) & 1, &bars.abort))) {
      if (lane == 0) {
        bars.give_up(p.err);
        atomicExch(p.abort, 1);                    // the gather poisons this step's records
      }
      if (tid == 0) bars.drain(n_seen + ST);
      return;
    }
    const int64_t blk = static_cast<int64_t>(c) * kWarps + warp;    // this warp's 32 positions
    const int64_t rest = pc.L - blk * 32;
    float x[4][4];
    if (rest > 0) {
      const uint8_t *codes = ring + st * C::kStage + (warp * 32 + g) * (D / 2);
      const uint8_t *scales = ring + st * C::kStage + C::kCodes + (warp * 32 + g) * (D / 16);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float d[1][4];
        q4::score_tile<D, 1, Q2>(codes + 8 * nt * (D / 2), scales + 8 * nt * (D / 16), tq, qh, ql, d);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = d[0][e];
      }
    }
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&bars.empty[st]);
    if (rest <= 0) continue;
    if (rest < 32 && MODE != kQ4Dump) {            // positions behind the end: below every score
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * nt + 2 * tq + (e & 1) >= rest) x[nt][e] = MODE == kQ4Step ? __int_as_float(0x7fc00000) : -INFINITY;
    }

#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (MODE == kQ4Max) {
        float mx = fmaxf(x[0][2 * r], x[0][2 * r + 1]);
#pragma unroll
        for (int nt = 1; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(x[nt][2 * r], x[nt][2 * r + 1]));
        if (live[r] && saga_in_bounds(blk < p.nblk, p.err)) p.group_max[((row + 8 * r) * p.nblk + blk) * 4 + tq] = mx * fac[r];
      } else if constexpr (MODE == kQ4Dump) {
        float *o = p.scores_out + (row + 8 * r) * p.row_stride + blk * 32;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 8 * nt + 2 * tq + e;
            if (live[r] && k < rest && saga_in_bounds(blk * 32 + k < p.row_stride, p.err)) o[k] = x[nt][2 * r + e] * fac[r];
          }
      } else {
        // NaN behind the end compares false
        float *o = p.lscore + ((row + 8 * r) * p.nblk + blk) * 32 + 2 * tq;
        uint32_t mask = 0u;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = x[nt][2 * r + e] * fac[r];
            if (a >= thr[r]) {
              mask |= 1u << (8 * nt + e);
              o[8 * nt + e] = a;
            }
          }
        mask <<= 2 * tq;
        mask |= __shfl_xor_sync(0xffffffffu, mask, 1);
        mask |= __shfl_xor_sync(0xffffffffu, mask, 2);
        if (live[r] && saga_in_bounds(blk < p.nblk, p.err)) {
          if (tq == 0) p.lmask[(row + 8 * r) * p.nblk + blk] = mask;
          if (p.sel_mask != nullptr) {
            uint8_t *sm = p.sel_mask + (row + 8 * r) * p.row_stride + blk * 32;
            for (int k = tq; k < 32 && k < rest; k += 4) sm[k] = static_cast<uint8_t>((mask >> k) & 1u);
          }
        }
      }
    }
  }
  }
}

// ---- N-th largest of the listed scores ----------------------------------------
// One CTA per row (b, query head): the listed scores' order keys on chip (in
// no particular order; they are only counted), then four 8-bit digits from the
// top, each a histogram and a scan from the highest bin. Lists too long for the
// chip (ties at the lower bound) are read again for each digit.
constexpr int kSelThreads = 512;
constexpr int kSelKeys = 11264;                 // 44 KB

struct SelParams {
  uint32_t *lmask;
  const float *lscore;
  const int32_t *l_kv;
  float *tau;
  uint8_t *sel_mask;             // nullable
  int64_t nblk, cap, max_l_kv;
  int32_t h_q, N;
  int32_t keep;                  // rewrite the masks with the fresh threshold
};

__global__ void __launch_bounds__(kSelThreads) q4_select_kernel(const SelParams p) {
  extern __shared__ uint32_t keys[];            // [kSelKeys]
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_n, s_digit, s_rem;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t bj = blockIdx.x;
  const int b = static_cast<int>(bj / p.h_q);
  int64_t L = p.l_kv[b];
  const int64_t hi = p.cap < p.max_l_kv ? p.cap : p.max_l_kv;
  L = L < 0 ? 0 : (L > hi ? hi : L);
  const int64_t nb = (L + 31) / 32;
  uint32_t *mask = p.lmask + bj * p.nblk;
  const float *score = p.lscore + bj * p.nblk * 32;

  float tau = -INFINITY;
  if (p.N < L) {
    if (tid == 0) { s_n = 0; s_digit = 0; s_rem = static_cast<uint32_t>(p.N); }
    __syncthreads();
    for (int64_t i = tid; i < nb; i += kSelThreads) {
      uint32_t m = mask[i];
      uint32_t at = m != 0u ? atomicAdd(&s_n, static_cast<uint32_t>(__popc(m))) : 0u;
      for (; m != 0u; m &= m - 1u, ++at)
        if (at < kSelKeys) keys[at] = order_key(score[i * 32 + __ffs(m) - 1]);
    }
    __syncthreads();
    const uint32_t n = s_n;
    uint32_t prefix = 0u, fixed = 0u;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0u;
      __syncthreads();
      auto count = [&](uint32_t k) {
        if ((k & fixed) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      };
      if (n <= kSelKeys) {
        for (uint32_t i = tid; i < n; i += kSelThreads) count(keys[i]);
      } else {
        for (int64_t i = tid; i < nb; i += kSelThreads)
          for (uint32_t m = mask[i]; m != 0u; m &= m - 1u) count(order_key(score[i * 32 + __ffs(m) - 1]));
      }
      __syncthreads();
      // the bin that holds the rank: suffix sums of 256 bins, eight a lane
      if (warp == 0) {
        uint32_t c[8], sum = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) { c[e] = hist[255 - (lane * 8 + e)]; sum += c[e]; }
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        uint32_t before = incl - sum;
        const uint32_t rem = s_rem;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (before < rem && rem <= before + c[e]) {
            s_digit = 255u - (lane * 8 + e);
            s_rem = rem - before;
          }
          before += c[e];
        }
      }
      __syncthreads();
      prefix |= s_digit << shift;
      fixed |= 255u << shift;
      __syncthreads();
    }
    tau = from_order_key(prefix);
  }
  if (tid == 0) p.tau[bj] = tau;
  if (p.keep == 0) return;
  for (int64_t i = tid; i < nb; i += kSelThreads) {
    const uint32_t old = mask[i];
    uint32_t kept = 0u;
    for (uint32_t m = old; m != 0u; m &= m - 1u) {
      const int k = __ffs(m) - 1;
      if (score[i * 32 + k] >= tau) kept |= 1u << k;
    }
    if (kept != old) mask[i] = kept;
    if (p.sel_mask != nullptr)
      for (int k = 0; k < 32 && i * 32 + k < L; ++k)
        p.sel_mask[bj * p.max_l_kv + i * 32 + k] = static_cast<uint8_t>((kept >> k) & 1u);
  }
}

template <int D, int MODE, typename T>
cudaError_t launch_scan(const Q4Params &p, cudaStream_t st) {
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(q4_scan_kernel<D, MODE, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             QS<D>::kRing);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(q4_scan_kernel<D, MODE, T>, dim3(p.S), dim3(kThreads), QS<D>::kRing, st, p);
}

template <int D, typename T>
cudaError_t launch_scan_m(const Q4Params &p, int mode, cudaStream_t st) {
  switch (mode) {
    case kQ4Step: return launch_scan<D, kQ4Step, T>(p, st);
    case kQ4Max: return launch_scan<D, kQ4Max, T>(p, st);
    case kQ4Dump: return launch_scan<D, kQ4Dump, T>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_q4_scan(const Q4Params &p, int mode, int dtype, int d, cudaStream_t st) {
  if (p.h_q / p.h_k > kMaxGroup || (d != 64 && d != 128)) return cudaErrorInvalidValue;
  if (dtype == SAGA_BF16)
    return d == 64 ? launch_scan_m<64, uint16_t>(p, mode, st) : launch_scan_m<128, uint16_t>(p, mode, st);
  return d == 64 ? launch_scan_m<64, float>(p, mode, st) : launch_scan_m<128, float>(p, mode, st);
}

cudaError_t launch_q4_select(const Q4Params &p, int32_t N, float *tau, bool keep, uint8_t *sel_mask,
                             cudaStream_t st) {
  static_assert(kSelKeys * 4 + 2048 <= 48 * 1024, "no opt-in shared memory");
  const SelParams sp{p.lmask, p.lscore, p.l_kv, tau, sel_mask, p.nblk, p.cap, p.max_l_kv, p.h_q, N, keep ? 1 : 0};
  return launch_pdl(q4_select_kernel, dim3(p.B * p.h_q), dim3(kSelThreads), kSelKeys * 4, st, sp);
}

}  // namespace saga
