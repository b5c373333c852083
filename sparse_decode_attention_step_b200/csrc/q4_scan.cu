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
// chunks of 256 or 512 positions, whatever the lengths (see Work). The chunks (codes
// and scales, two contiguous ranges) come through a ring of shared-memory stages
// with untiled bulk copies (see Ring); each of eight warps scores its one or two
// blocks of 32 positions: mma.sync m16n8k16 with the heads on M and eight keys on N, a
// lane converting consecutive codes of one key row into the B operand. A
// quad of lanes then holds two heads' 32 scores: their masks of kept positions
// come together in two shuffles, and a kept score goes to its own place in the
// 32-position block. The step is deterministic.
//
// Bound by instruction issue: about 260 per 32 positions and 16 heads (32
// conversions, 32 scale products, 16 MMAs, and per score a product, a compare and
// a mask bit) at 2.3 a cycle and SM. 8 x 128K positions of 2 heads of 64 (75 MB):
// step 31 us, max 28 us, 2.4-2.7 TB/s, where a copy would take 12.
#include <atomic>

#include "kernels.h"
#include "plan.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxDevices = 64;

template <int D, int MODE, typename T>
struct QS {
  // 32-position blocks per warp and chunk: two spread a chunk's fixed work and give
  // a warp independent MMAs (8 x 128K positions, heads of 64: the step's pass 36 ->
  // 31 us; four, with one CTA per SM, 38), where the registers of two CTAs per SM
  // hold them. At d 128 the step gains (8 x 128K: 51.6 -> 49.8 us with its gather)
  // although it spills 24 bytes a thread; the other modes and fp32 queries would spill so
  // much that they lose (refresh 67 -> 72), and with one block fp32 queries still spill 12
  // bytes in the step and 80 in the maxima.
  static constexpr int kBlocks = D == 64 || (MODE == kQ4Step && sizeof(T) == 2) ? 2 : 1;
  static constexpr int kChunk = kWarps * kBlocks * 32;
  static_assert(kChunk >= kQ4ScanChunk, "the plan counts chunks of at least this");
  static constexpr int kCodes = kChunk * D / 2, kScales = kChunk * D / 16;
  static constexpr int kStage = kCodes + kScales;               // 18 or 36 KB
  // A short ring leaves a step room for the gather's CTAs beside its own (6 stages
  // instead of 4 cost 15 us of 46, 3 instead of 4 gained 1; 8 x 64K, heads of 64);
  // the maxima at d 128 want a longer one (refresh of 8 x 64K: 49 us with 5, 53 with 4)
  static constexpr int kStages = kBlocks == 1 ? 5 : (D == 64 ? 3 : 2);
  static constexpr int kRing = kStages * kStage;
};

template <int D, int MODE, typename T>
__global__ void __launch_bounds__(kThreads, kQ4ScanCtasPerSm) q4_scan_kernel(const Q4Params p) {
  using C = QS<D, MODE, T>;
  constexpr bool Q2 = sizeof(T) == 4;
  constexpr int ST = C::kStages, kChunk = C::kChunk, NB = C::kBlocks;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ q4::Ring<kChunk, ST> bars;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.h_q / p.h_k;

  if (tid == 0) bars.init(kWarps);
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int cta = blockIdx.x;
  if (MODE == kQ4Step && cta == 0)
    for (int i = tid; i <= p.B * p.h_q; i += kThreads) p.tickets[i] = 0;
  const q4::Work work = q4::work_of<kChunk>(p, lane, cta == 0 && warp == 0);
  if (cta >= work.n) return;
  int64_t x0 = work.begin(cta);
  const int64_t x1 = work.begin(cta + 1);
  q4::Seq seq = q4::seq_at<kChunk>(p, lane, x0);

  const auto load = [&](int b, int kh, int L, int c, int st) {
    const int64_t kb = b * p.kc_sb + kh * p.kc_sh;
    const int64_t t = static_cast<int64_t>(c) * kChunk;
    const int left = L - c * kChunk;
    // whole groups of four rows: 16 bytes of scales at least (cap is a multiple of 4)
    const uint32_t rows = left < kChunk ? (left + 3) & ~3 : kChunk;
    const uint32_t nc = rows * (D / 2), ns = rows * (D / 16);
    uint8_t *dst = ring + st * C::kStage;
    if (!saga_in_bounds(b < p.B && kh < p.h_k && left > 0 && t + rows <= p.cap && st < ST, p.err)) {
      sm100::mbar_arrive(&bars.full[st]);
      return;
    }
    sm100::mbar_arrive_expect_tx(&bars.full[st], nc + ns);
    const uint8_t *codes = p.kc + kb + t * (D / 2), *scales = p.ks + kb / 8 + t * (D / 16);
    if (MODE == kQ4Step) {     // a step's K stream leaves its lists in L2 (8 x 128K: 68.6 -> 67 us)
      q4::bulk_load_once(dst, codes, nc, &bars.full[st]);
      q4::bulk_load_once(dst + C::kCodes, scales, ns, &bars.full[st]);
    } else {
      q4::bulk_load(dst, codes, nc, &bars.full[st]);
      q4::bulk_load(dst + C::kCodes, scales, ns, &bars.full[st]);
    }
  };

  const int g = lane >> 2, tq = lane & 3;
  const bool live[2] = {g < G, g + 8 < G};
  q4::Stage<ST> at;
  int turn = 0;                                      // the warp that issues next
  bool first = true;
  while (x0 < x1) {
    const q4::Piece pc = q4::next_piece<kChunk>(p, seq, x0, x1);
    const int b = pc.b, j0 = pc.kh * G;
    if (first && tid == 0)
      for (int i = 0; i < bars.kAhead; ++i) bars.issue(p, i, 1u, pc, pc.c0, i, seq, x0, x1, load);
    first = false;
    __syncwarp();
    uint32_t qh[1][D / 16][4], ql[1][Q2 ? D / 16 : 1][4];
    float fac[2], thr[2];
    const float gk = p.k_g != nullptr ? __ldg(p.k_g + pc.kh) : 1.f;
    const T *qb = static_cast<const T *>(p.q) + b * p.q_sb + static_cast<int64_t>(j0 + g) * p.q_sh;
    fac[0] = q4::score_factor(p.scale, q4::q_frag<D, T, Q2, 0>(qb, live[0], tq, qh[0], ql[0]), gk);
    fac[1] = q4::score_factor(p.scale, q4::q_frag<D, T, Q2, 1>(qb + 8 * p.q_sh, live[1], tq, qh[0], ql[0]), gk);
    if (MODE == kQ4Step) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        thr[r] = live[r] ? (p.tau != nullptr ? p.tau[b * p.h_q + j0 + g + 8 * r] : -INFINITY) : INFINITY;
    }
    // this lane's places in the outputs of its first head, at 32-position block
    // 0; the second is eight heads on
    const int64_t row = static_cast<int64_t>(b) * p.h_q + j0 + g;
    float *const o_score = MODE == kQ4Step ? p.lscore + row * p.nblk * 32 + 2 * tq : nullptr;
    float *const o_dump = MODE == kQ4Dump ? p.scores_out + row * p.row_stride + 2 * tq : nullptr;
    uint16_t *const o_max = MODE == kQ4Max ? p.group_max + row * p.nblk * 4 + tq : nullptr;
    uint32_t *const o_mask = MODE == kQ4Step ? p.lmask + row * p.nblk : nullptr;

    for (int c = pc.c0; c < pc.c1; ++c) {
      if (warp == turn && lane == 0)
        bars.issue(p, at.refill(), at.refill_parity(), pc, c, bars.kAhead, seq, x0, x1, load);
      turn = (turn + 1) % kWarps;
      __syncwarp();
      if (!__all_sync(0xffffffffu, q4::wait_bar(&bars.full[at.st], at.phase, &bars.abort))) {
        if (lane == 0) {
          bars.give_up(p.err);
          atomicExch(p.abort, 1);                  // the gather, or the select, poisons the call's results
        }
        if (tid == 0) bars.drain(at.st, at.phase);
        return;
      }
      const int blk0 = (c * kWarps + warp) * NB;   // this warp's 32-position blocks
      const int rest0 = pc.L - blk0 * 32;
      float x[4 * NB][1][4];
      if (rest0 > 0) {
        const int row = warp * NB * 32 + g;
        q4::score_tiles<D, 1, 4 * NB, Q2>(ring + at.st * C::kStage + row * (D / 2),
                                          ring + at.st * C::kStage + C::kCodes + row * (D / 16), tq, qh, ql, x);
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&bars.empty[at.st]);
      at.advance();
      if (rest0 < 32 * NB && MODE != kQ4Dump) {    // positions behind the end: below every score
#pragma unroll
        for (int nt = 0; nt < 4 * NB; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * nt + 2 * tq + (e & 1) >= rest0)
              x[nt][0][e] = MODE == kQ4Step ? __int_as_float(0x7fc00000) : -INFINITY;
      }

#pragma unroll
      for (int rr = 0; rr < 2 * NB; ++rr) {
        const int r = rr % 2, blk = blk0 + rr / 2, rest = rest0 - 32 * (rr / 2);
        if (rest <= 0 || !saga_in_bounds(blk < p.nblk, p.err)) break;
        const auto score = [&](int nt, int e) { return x[4 * (rr / 2) + nt][0][2 * r + e]; };
        if constexpr (MODE == kQ4Max) {
          float mx = fmaxf(score(0, 0), score(0, 1));
#pragma unroll
          for (int nt = 1; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(score(nt, 0), score(nt, 1)));
          if (live[r]) (o_max + 8 * r * p.nblk * 4)[blk * 4] = static_cast<uint16_t>(order_key(mx * fac[r]) >> 16);
        } else if constexpr (MODE == kQ4Dump) {
          float *o = o_dump + 8 * r * p.row_stride + static_cast<int64_t>(blk) * 32;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (live[r] && 8 * nt + 2 * tq + e < rest) o[8 * nt + e] = score(nt, e) * fac[r];
        } else {
          // NaN behind the end compares false
          float a[8];
          uint32_t mask = 0u;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = score(i / 2, i % 2) * fac[r];
            if (a[i] >= thr[r]) mask |= 1u << (8 * (i / 2) + i % 2);
          }
          mask <<= 2 * tq;
          mask |= __shfl_xor_sync(0xffffffffu, mask, 1);
          mask |= __shfl_xor_sync(0xffffffffu, mask, 2);
          // a quad's eight scores of a key tile are one sector: written whole when
          // one of them is kept, so that reading it back needs no fill from memory
          float2 *o = reinterpret_cast<float2 *>(o_score + 8 * r * p.nblk * 32 + static_cast<int64_t>(blk) * 32);
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
            if (mask & (0xffu << (8 * nt))) o[4 * nt] = make_float2(a[2 * nt], a[2 * nt + 1]);
          if (live[r] && tq == 0) (o_mask + 8 * r * p.nblk)[blk] = mask;
          if (p.sel_mask != nullptr && live[r]) {
            uint8_t *sm = p.sel_mask + (row + 8 * r) * p.row_stride + static_cast<int64_t>(blk) * 32;
            for (int k = tq; k < 32 && k < rest; k += 4) sm[k] = static_cast<uint8_t>((mask >> k) & 1u);
          }
        }
      }
    }
  }
}

// The N-th largest of a CTA's keys, given that all lie in [lo, hi] or, if below
// lo, do not matter, and that N of them reach lo: a histogram of kBins equal
// ranges of [lo, hi], the range that holds the rank, and again within it, ten
// bits at a time. each(f) calls f(key) for every key of the calling thread.
constexpr int kSelThreads = 512;
constexpr int kBins = 1024;
constexpr int kBinsPer = kBins / kSelThreads;

struct Nth {
  uint32_t hist[kBins], wsum[kSelThreads / 32];
  uint32_t bin, rem;
};

template <typename F>
__device__ __forceinline__ uint32_t nth_largest(uint32_t lo, uint32_t hi, uint32_t N, Nth &sh, F each) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) { sh.bin = 0u; sh.rem = N; }
  if (hi < lo) return lo;        // fewer keys than N: scores of NaN, which nothing orders
  for (;;) {                     // every turn leaves hi - lo < 2^shift, ten bits less
    const int shift = hi - lo < kBins ? 0 : 32 - __clz(hi - lo) - 10;
#pragma unroll
    for (int e = 0; e < kBinsPer; ++e) sh.hist[tid + e * kSelThreads] = 0u;
    __syncthreads();
    each([&](uint32_t k) {
      if (k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
    });
    __syncthreads();
    // counts from the highest range down; this thread's kBinsPer ranges
    uint32_t c[kBinsPer], sum = 0u;
#pragma unroll
    for (int e = 0; e < kBinsPer; ++e) { c[e] = sh.hist[kBins - 1 - (tid * kBinsPer + e)]; sum += c[e]; }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sh.wsum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - sum;
    for (int w = 0; w < warp; ++w) before += sh.wsum[w];
    const uint32_t want = N;
#pragma unroll
    for (int e = 0; e < kBinsPer; ++e) {
      if (before < want && want <= before + c[e]) {
        sh.bin = kBins - 1 - (tid * kBinsPer + e);
        sh.rem = want - before;
      }
      before += c[e];
    }
    __syncthreads();
    N = sh.rem;
    lo += sh.bin << shift;
    if (shift == 0) return lo;
    const uint32_t top = lo + (1u << shift) - 1u;
    hi = top < hi ? top : hi;
  }
}

// The largest of `x` over the CTA, in *s (cleared before).
__device__ __forceinline__ uint32_t cta_max(uint32_t x, uint32_t *s) {
  x = __reduce_max_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) atomicMax(s, x);
  __syncthreads();
  return *s;
}

// ---- the lower bound from the group maxima ---------------------------------------
// One CTA per row, the maxima's 16-bit keys in registers (those behind the first
// 128K positions are read again for each histogram). 512 rows of up to 128K: 10 us,
// the latency of one read and two histograms; three CTAs per SM spill 48 bytes a thread,
// four spill more and gain nothing.
// Cutting an order key off rounds the score down,
// so the bound stays one. A row whose rank lies in the eight octaves (1024
// keys) under its maximum takes one histogram.
constexpr int kBoundRegs = 8;                   // 8-byte words of keys a thread: 16384 keys a CTA

struct BoundParams {
  const uint16_t *group_max;
  const int32_t *l_kv;
  float *bound;
  int64_t nblk, cap, max_l_kv;
  int32_t h_q, N;
};

__global__ void __launch_bounds__(kSelThreads, 3) q4_bound_kernel(const BoundParams p) {
  __shared__ Nth sh;
  __shared__ uint32_t s_max, s_near;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t bj = blockIdx.x;
  int L = p.l_kv[bj / p.h_q];
  const int cap = static_cast<int>(p.cap < p.max_l_kv ? p.cap : p.max_l_kv);
  L = L < 0 ? 0 : (L > cap ? cap : L);
  const int n = (L + 31) / 32 * 4;              // groups of the row
  if (n < p.N) {
    if (tid == 0) p.bound[bj] = -INFINITY;
    return;
  }
  if (tid == 0) { s_max = 0u; s_near = 0u; }
  __syncthreads();
  // rows start on 8 bytes: four groups a block
  const uint2 *row = reinterpret_cast<const uint2 *>(p.group_max + bj * p.nblk * 4);
  const int words = n / 4;
  uint2 w[kBoundRegs];
#pragma unroll
  for (int i = 0; i < kBoundRegs; ++i) {
    const int at = tid + i * kSelThreads;
    w[i] = at < words ? row[at] : make_uint2(0u, 0u);   // a key of 0 is below every score's
  }
  const auto each = [&](auto f) {
    const auto four = [&](uint2 x) { f(x.x & 0xffffu); f(x.x >> 16); f(x.y & 0xffffu); f(x.y >> 16); };
#pragma unroll
    for (int i = 0; i < kBoundRegs; ++i) {
      if (i * kSelThreads >= words) break;
      four(w[i]);
    }
    for (int at = tid + kBoundRegs * kSelThreads; at < words; at += kSelThreads) four(row[at]);
  };
  uint32_t mx = 0u;
  each([&](uint32_t k) { mx = max(mx, k); });
  mx = cta_max(mx, &s_max);
  const uint32_t near = mx >= kBins ? mx - (kBins - 1) : 1u;
  uint32_t c = 0u;
  each([&](uint32_t k) { c += k >= near; });
  c = __reduce_add_sync(0xffffffffu, c);
  if ((tid & 31) == 0 && c != 0u) atomicAdd(&s_near, c);
  __syncthreads();
  c = s_near;
  const uint32_t N = static_cast<uint32_t>(p.N);
  const uint32_t v = c >= N ? nth_largest(near, mx, N, sh, each) : nth_largest(1u, near - 1u, N - c, sh, each);
  // keys up to that of -inf, cut off, stand for it
  if (tid == 0) p.bound[bj] = v <= (order_key(-INFINITY) >> 16) ? -INFINITY : from_order_key(v << 16);
}

// ---- N-th largest of the listed scores ----------------------------------------
// One CTA per row (b, query head). The listed scores are gathered on chip (in no
// particular order; they are only counted), then their N-th largest. A sparse
// list's positions are gathered first, a thread per 32-position block, then all
// its scores at once; a dense one (more than eight a block: a short row, where N
// groups are most of it) is read a block per warp, which waits for memory at every
// few blocks where a thread would walk up to 32 entries (8 rows of 32K, N 2048: 41
// us for the refresh with positions, 69 by blocks; 8 rows of 4096 without a bound:
// 27 with positions, 22 by blocks). Lists too long for the chip (ties at the
// bound, or a large N) are read by blocks again for each histogram.
constexpr int kSelWords = kQ4SelectKeys;        // keys, or half as many keys and positions: 40 KB, four CTAs per SM

struct SelParams {
  uint32_t *lmask;
  const float *lscore, *bound;
  const int32_t *l_kv;
  float *tau;
  uint8_t *sel_mask;             // nullable
  int32_t *abort, *done;         // the call's abort word, and a counter of its rows (zero)
  int32_t *err;
  int64_t nblk, cap, max_l_kv;
  int32_t h_q, N;
  int32_t keep;                  // cut the masks down to the fresh threshold
};

__global__ void __launch_bounds__(kSelThreads, 4) q4_select_kernel(const SelParams p) {
  extern __shared__ uint32_t keys[];            // [kSelWords]
  uint32_t *const where = keys + kSelWords / 2;
  __shared__ Nth sh;
  __shared__ uint32_t s_n, s_at, s_max;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t bj = blockIdx.x;
  int L = p.l_kv[bj / p.h_q];
  const int cap = static_cast<int>(p.cap < p.max_l_kv ? p.cap : p.max_l_kv);
  L = L < 0 ? 0 : (L > cap ? cap : L);
  const int nb = (L + 31) / 32;
  uint32_t *mask = p.lmask + bj * p.nblk;
  const float *score = p.lscore + bj * p.nblk * 32;
  // f(block, mask, this lane's score) for the blocks of this warp, which all lanes call
  const auto walk = [&](auto f) {
#pragma unroll 4
    for (int i = warp; i < nb; i += kSelThreads / 32) {
      const uint32_t m = mask[i];
      f(i, m, (m >> lane) & 1u ? score[i * 32 + lane] : 0.f);
    }
  };

  // a score pass that gave up: its lists may hold anything, and there is no threshold in them
  const bool gave_up = tid == 0 && *reinterpret_cast<const volatile int32_t *>(p.abort) != 0;
  float tau = -INFINITY;
  bool sparse = false;
  uint32_t n = 0u;
  if (p.N < L) {
    const float lo = p.bound != nullptr ? p.bound[bj] : -INFINITY;
    if (tid == 0) { s_n = 0u; s_at = 0u; s_max = 0u; }
    __syncthreads();
    constexpr int U = 8;                        // masks a thread loads at once
    uint32_t m[U];
    uint32_t c = 0u;
    for (int i0 = 0; i0 < nb; i0 += kSelThreads * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kSelThreads + tid;
        m[u] = i < nb ? mask[i] : 0u;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) c += __popc(m[u]);
    }
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0 && c != 0u) atomicAdd(&s_n, c);
    __syncthreads();
    n = s_n;
    sparse = n <= kSelWords / 2 && n <= 8u * nb;
    const bool on_chip = n <= (sparse ? kSelWords / 2 : kSelWords);
    if (sparse) {
      for (int i0 = 0; i0 < nb; i0 += kSelThreads * U) {
        int mine = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * kSelThreads + tid;
          if (nb > kSelThreads * U) m[u] = i < nb ? mask[i] : 0u;   // else still at hand
          mine += __popc(m[u]);
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        uint32_t at = 0u;
        if (lane == 31 && incl != 0) at = atomicAdd(&s_at, static_cast<uint32_t>(incl));
        at = __shfl_sync(0xffffffffu, at, 31) + incl - mine;
#pragma unroll
        for (int u = 0; u < U; ++u)
          for (uint32_t x = m[u]; x != 0u && saga_in_bounds(at < kSelWords / 2, p.err); x &= x - 1u, ++at)
            where[at] = (i0 + u * kSelThreads + tid) * 32 + __ffs(x) - 1;
      }
      __syncthreads();
#pragma unroll 4
      for (uint32_t i = tid; i < n; i += kSelThreads)
        if (saga_in_bounds(where[i] < nb * 32u, p.err)) keys[i] = order_key(score[where[i]]);
    } else if (on_chip) {
      walk([&](int, uint32_t x, float a) {
        uint32_t at = 0u;
        if (lane == 0 && x != 0u) at = atomicAdd(&s_at, static_cast<uint32_t>(__popc(x)));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(x & ((1u << lane) - 1u));
        if ((x >> lane) & 1u && saga_in_bounds(at < kSelWords, p.err)) keys[at] = order_key(a);
      });
      __syncthreads();
    }
    const auto each = [&](auto f) {             // f(order key)
      if (on_chip) {
        for (uint32_t i = tid; i < n; i += kSelThreads) f(keys[i]);
      } else {
        walk([&](int, uint32_t x, float a) { if ((x >> lane) & 1u) f(order_key(a)); });
      }
    };
    uint32_t mx = 0u;
    each([&](uint32_t k) { mx = max(mx, k); });
    mx = cta_max(mx, &s_max);
    // (-0 and +0 compare equal in the scan: the bound's key is the lower one)
    tau = from_order_key(nth_largest(order_key(lo == 0.f ? -0.f : lo), mx, static_cast<uint32_t>(p.N), sh, each));
  }
  if (tid == 0) p.tau[bj] = gave_up && p.N < L ? __int_as_float(0x7fc00000) : tau;
  if (p.keep == 0) {
    // no gather follows to end the call: the last row that has read the abort word set
    // (all rows do, or none) clears it for the next call
    if (gave_up) {
      __threadfence();
      if (atomicAdd(p.done, 1) == static_cast<int32_t>(gridDim.x) - 1) *p.abort = 0;
    }
    return;
  }
  if (p.N < L) {
    const uint32_t k_tau = order_key(tau == 0.f ? -0.f : tau);
    if (sparse) {
      for (uint32_t i = tid; i < n; i += kSelThreads)
        if (keys[i] < k_tau) atomicAnd(&mask[where[i] / 32], ~(1u << (where[i] % 32)));
    } else {
      walk([&](int i, uint32_t x, float a) {
        const uint32_t kept = __ballot_sync(0xffffffffu, (x >> lane) & 1u && order_key(a) >= k_tau);
        if (lane == 0) mask[i] = kept;
      });
    }
  }
  if (p.sel_mask == nullptr) return;
  __threadfence();
  __syncthreads();
  for (int t = tid; t < L; t += kSelThreads)
    p.sel_mask[bj * p.max_l_kv + t] = static_cast<uint8_t>((*reinterpret_cast<volatile uint32_t *>(mask + t / 32) >> (t % 32)) & 1u);
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
                             QS<D, MODE, T>::kRing);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(q4_scan_kernel<D, MODE, T>, dim3(p.S), dim3(kThreads), QS<D, MODE, T>::kRing, st, p);
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

cudaError_t launch_q4_bound(const Q4Params &p, int32_t N, float *bound, cudaStream_t st) {
  const BoundParams bp{p.group_max, p.l_kv, bound, p.nblk, p.cap, p.max_l_kv, p.h_q, N};
  return launch_pdl(q4_bound_kernel, dim3(p.B * p.h_q), dim3(kSelThreads), 0, st, bp);
}

cudaError_t launch_q4_select(const Q4Params &p, int32_t N, const float *bound, float *tau, bool keep,
                             uint8_t *sel_mask, cudaStream_t st) {
  static std::atomic<bool> attr_set[kMaxDevices];
  constexpr int kSmem = kSelWords * 4;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(q4_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const SelParams sp{p.lmask, p.lscore, bound, p.l_kv, tau, sel_mask, p.abort,
                     p.tickets + p.B * p.h_q, p.err, p.nblk, p.cap, p.max_l_kv, p.h_q, N,
                     keep ? 1 : 0};
  return launch_pdl(q4_select_kernel, dim3(p.B * p.h_q), dim3(kSelThreads), kSmem, st, sp);
}

}  // namespace saga
