// The V half of the Atop-N step over a 4-bit cache (Eq. 7 over the kept entries).
//
// The scan leaves, for every 32-position block of every query head's row (b, j),
// a 32-bit mask of the kept positions and each kept score at its position. CTAs
// over (b, j, block range) turn them into softmax states, and the last CTA of a
// row to finish merges the row's states into out, in range order, so the result
// does not depend on which one it was.
//
// A warp lists the kept positions of 32 blocks at a time and takes them 32 by 32
// as the keys of a matrix product: O^T[dims x 1] += V^T p, mma.sync m16n8k16
// with the dims on M, the kept rows on K, and in column 0 the high fp16 half of
// their probabilities, in column 1 the low one. A lane loads the same dims of
// its rows straight from memory (their codes, their scale) and converts them
// into the A operand, as the dense kernel does from shared memory; the loads of
// the next 32 rows are issued before the current ones are worked on, since a
// row read at random takes a microsecond or two. Most of the product's columns
// stay empty, but one FMA per value would take twice the instructions.
//
// Bound by the reads at random, 64 bytes of DRAM each for a row's codes and for its
// scales: 256 rows (b, head) of 2048 kept positions, d 64 (19 MB of codes and
// scales): about 30 us. Four CTAs per SM with 128 registers a thread and one wave of
// them beat five and six with fewer registers (8 x 128K step: 62 us against 69 and
// 72) and two waves (66).
#include "kernels.h"
#include "plan.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch = 32;                       // kept rows per step of a warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 7.f;                   // as in the dense kernel: P is relative to its batch
constexpr float kLazy = 8.f;

// Loads of what is read once, at random: without a line in L1, which the rows of
// other lanes would push out before its other sectors are wanted (8 x 128K step: 67 ->
// 62 us). Volatile: behind the wait for the previous launch.
__device__ __forceinline__ uint32_t load_once(const uint32_t *p) {
  uint32_t x;
  asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 load_once(const uint2 *p) {
  uint2 x;
  asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t load_once(const uint8_t *p) {
  uint32_t x;
  asm volatile("ld.global.L1::no_allocate.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

// A lane's share of 32 kept rows: entries 16 j + tq + 4 i.
template <int D>
struct Rows {
  uint32_t code[2][4][D / 64];
  uint32_t scale[2][4];
  float a[2][4];                                 // scores
};

template <int D>
__global__ void __launch_bounds__(kThreads, q4_gather_ctas_per_sm(D)) q4_gather_kernel(const Q4Gather p) {
  constexpr int NM = D / 16;
  __shared__ int list[kWarps][32 * 32 + kBatch];
  __shared__ float s_acc[kWarps][D], s_m[kWarps], s_l[kWarps];
  __shared__ int s_n[kWarps], s_last;
  pdl_wait();
  pdl_trigger();

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int bj = blockIdx.x / p.SB, sb = blockIdx.x % p.SB;
  const int b = bj / p.h_q, vh = bj % p.h_q / p.hpv;
  int L = p.l_kv[b];
  const int hi = static_cast<int>(p.cap < p.max_l_kv ? p.cap : p.max_l_kv);
  L = L < 0 ? 0 : (L > hi ? hi : L);
  const int nb_row = (L + 31) / 32;
  const int blk0 = min(sb * p.blk_per_split, nb_row), blk1 = min(blk0 + p.blk_per_split, nb_row);

  const uint32_t *mask = p.lmask + static_cast<int64_t>(bj) * p.nblk;
  const float *sco = p.lscore + static_cast<int64_t>(bj) * p.nblk * 32;
  const uint8_t *codes = p.vc + b * p.vc_sb + vh * p.vc_sh + g * (D / 16);
  const uint8_t *scales = p.vs + (b * p.vc_sb + vh * p.vc_sh) / 8 + (D == 64 ? g / 2 : g);
  int *mine = list[warp];

  float m = -INFINITY, l = 0.f, acc[NM][2];
#pragma unroll
  for (int n = 0; n < NM; ++n) acc[n][0] = acc[n][1] = 0.f;
  int kept = 0;

  // n <= kBatch positions of the list, from at_list on; the others of a batch count nothing
  int at_list = 0;
  auto load = [&](int n, Rows<D> &r) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 16 * j + tq + 4 * i;
        const bool in = e < n;
        const int64_t pos = mine[at_list + (in ? e : 0)];
        const uint8_t *c = codes + pos * (D / 2);
        if constexpr (D == 64) {
          r.code[j][i][0] = load_once(reinterpret_cast<const uint32_t *>(c));
        } else {
          const uint2 w = load_once(reinterpret_cast<const uint2 *>(c));
          r.code[j][i][0] = w.x;
          r.code[j][i][1] = w.y;
        }
        r.scale[j][i] = load_once(scales + pos * (D / 16));
        r.a[j][i] = in ? __uint_as_float(load_once(reinterpret_cast<const uint32_t *>(sco + pos))) : -INFINITY;
      }
  };
  const float lo_col = g == 1 ? -1.f : 0.f;      // column 1 takes the low halves
  auto fold = [&](const Rows<D> &r) {
    float mx = r.a[0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) mx = fmaxf(mx, r.a[e / 4][e % 4]);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * kLog2e;
    if (mx > m + kLazy) {                        // the same in every lane
      const float c = m == -INFINITY ? 0.f : q4::ex2(m - mx);
      m = mx;
      l *= c;
#pragma unroll
      for (int n = 0; n < NM; ++n) { acc[n][0] *= c; acc[n][1] *= c; }
    }
    // P relative to the batch's own maximum; its sums are brought to the running one
    const float bias = mx == -INFINITY ? 0.f : kPShift - mx;
    const float f = mx == -INFINITY ? 0.f : q4::ex2(mx - m);
    float sum = 0.f;
    uint32_t pb[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {
        const float p0 = q4::ex2(fmaf(r.a[j][2 * pr], kLog2e, bias));
        const float p1 = q4::ex2(fmaf(r.a[j][2 * pr + 1], kLog2e, bias));
        sum += p0 + p1;
        const float h0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u);
        const float h1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
        pb[j][pr] = g < 2 ? q4::pack_f16_rz(fmaf(lo_col, h0, p0), fmaf(lo_col, h1, p1)) : 0u;
      }
    l = fmaf(f, sum, l);
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      uint32_t a[2][4][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int pr = 0; pr < 2; ++pr)
          q4::value_pair(r.code[j][2 * pr][u], r.code[j][2 * pr + 1][u], r.scale[j][2 * pr], r.scale[j][2 * pr + 1],
                         pr, a[j]);
      float t[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) t[n][0] = t[n][1] = t[n][2] = t[n][3] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < 4; ++n) q4::mma(t[n], a[j][n], pb[j][0], pb[j][1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        // lanes with tq == 0 hold columns 0 and 1
        acc[4 * u + n][0] = fmaf(f, t[n][0] + t[n][1], acc[4 * u + n][0]);
        acc[4 * u + n][1] = fmaf(f, t[n][2] + t[n][3], acc[4 * u + n][1]);
      }
    }
  };

  const bool gave_up = *reinterpret_cast<const volatile int32_t *>(p.abort) != 0;
  if (!gave_up) {
    const int per = (blk1 - blk0 + kWarps - 1) / kWarps;
    const int w0 = min(blk0 + per * warp, blk1), w1 = min(w0 + per, blk1);
    // The next batch onto the list: its positions, 0 when there are none left. The
    // blocks' masks are taken 32 at a time, read ahead of their use.
    int wb = w0, have = 0, used = 0;
    uint32_t next = w0 + lane < w1 ? mask[w0 + lane] : 0u;
    const auto next_batch = [&]() {
      have -= used;                              // what the last batches left moves to the front
      at_list += used;
      if (have < kBatch && at_list > 0) {
        const int v = mine[at_list + (lane < have ? lane : 0)];
        __syncwarp();
        if (lane < have) mine[lane] = v;
        at_list = 0;
      }
      while (have < kBatch && wb < w1) {
        uint32_t mk = next;
        next = wb + 32 + lane < w1 ? mask[wb + 32 + lane] : 0u;
        const int cn = __popc(mk);
        int incl = cn;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        for (int e = have + incl - cn; mk != 0u; mk &= mk - 1u, ++e) {
          const int pos = (wb + lane) * 32 + __ffs(mk) - 1;
          if (!saga_in_bounds(e < 32 * 32 + kBatch, p.err)) break;
          mine[e] = saga_in_bounds(pos < L, p.err) ? pos : 0;
        }
        const int total = __shfl_sync(0xffffffffu, incl, 31);
        have += total;
        kept += total;
        wb += 32;
      }
      __syncwarp();
      used = min(have, kBatch);
      return used;
    };
    // one batch is worked on while the next one's loads are under way
    Rows<D> r0, r1;
    int n = next_batch();
    if (n > 0) {
      load(n, r0);
      for (;;) {
        if ((n = next_batch()) == 0) { fold(r0); break; }
        load(n, r1);
        fold(r0);
        if ((n = next_batch()) == 0) { fold(r1); break; }
        load(n, r0);
        fold(r1);
      }
    }
  }

  // ---- the warps' states, then the CTA's record -------------------------------
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (tq == 0) {
#pragma unroll
    for (int n = 0; n < NM; ++n)
      *reinterpret_cast<float2 *>(&s_acc[warp][g * (D / 8) + 2 * n]) = make_float2(acc[n][0], acc[n][1]);
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; s_n[warp] = kept; }
  __syncthreads();
  constexpr int kRec = D + kRecPad;
  float *row_rec = p.partials + static_cast<int64_t>(bj) * p.SB * kRec;
  float M = s_m[0];
  int n_all = s_n[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) { M = fmaxf(M, s_m[w]); n_all += s_n[w]; }
  float lt = 0.f, at = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float c = s_m[w] == -INFINITY ? 0.f : q4::ex2(s_m[w] - M);
    lt = fmaf(c, s_l[w], lt);
    if (tid < D) at = fmaf(c, s_acc[w][tid], at);
  }
  const float gv = p.v_g != nullptr ? __ldg(p.v_g + vh) : 1.f;
  if (p.SB > 1) {
    float *rec = row_rec + sb * kRec;
    if (tid < D) __stcg(rec + kRecPad + tid, at);
    if (tid == 0) __stcg(reinterpret_cast<float4 *>(rec), make_float4(M, lt, __int_as_float(gave_up ? -1 : n_all), 0.f));
    // the record is out before the ticket is drawn; the CTA that draws the last
    // one sees every other record
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(p.tickets + bj, 1) == p.SB - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the largest maximum and the counts first, then kMergeAt records' weights at a
    // time and their sums, each thread one dim of every kPar-th record
    constexpr int kMergeAt = 64, kPar = kThreads / D;
    __shared__ float s_w[kMergeAt];
    M = -INFINITY;
    int bad = 0;
    n_all = 0;
    for (int s = tid; s < p.SB; s += kThreads) {
      const float4 h = __ldcg(reinterpret_cast<const float4 *>(row_rec + s * kRec));
      M = fmaxf(M, h.x);
      bad |= __float_as_int(h.z) < 0;
      n_all += __float_as_int(h.z);
    }
    M = warp_max(M);
    n_all = __reduce_add_sync(0xffffffffu, n_all);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) { s_m[warp] = M; s_n[warp] = bad ? INT32_MIN : n_all; }
    __syncthreads();
    M = s_m[0];
    bad = s_n[0] == INT32_MIN;
    n_all = s_n[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      M = fmaxf(M, s_m[w]);
      bad |= s_n[w] == INT32_MIN;
      n_all += s_n[w];
    }
    if (bad) n_all = -1;
    lt = at = 0.f;
    for (int s0 = 0; s0 < p.SB; s0 += kMergeAt) {
      const int n = min(kMergeAt, p.SB - s0);
      __syncthreads();
      if (tid < n) {
        const float2 h = __ldcg(reinterpret_cast<const float2 *>(row_rec + (s0 + tid) * kRec));
        const float c = h.x == -INFINITY ? 0.f : q4::ex2(h.x - M);
        s_w[tid] = c;
        lt = fmaf(c, h.y, lt);
      }
      __syncthreads();
#pragma unroll 8
      for (int s = tid / D; s < n; s += kPar)
        at = fmaf(s_w[s], __ldcg(row_rec + (s0 + s) * kRec + kRecPad + tid % D), at);
    }
    lt = warp_sum(lt);
    __syncthreads();
    if (lane == 0) s_l[warp] = lt;
    float *const half = &s_acc[0][0];            // kPar == 2: the other half's sums
    if (kPar == 2 && tid >= D) half[tid - D] = at;
    __syncthreads();
    lt = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) lt += s_l[w];
    if (kPar == 2 && tid < D) at += half[tid];
  } else if (gave_up) {
    n_all = -1;
  }
  // an empty selection is a zero row; a scan that gave up a NaN one
  if (tid < D) {
    const float o = lt > 0.f ? at / lt * kQ4Unit * gv : 0.f;
    p.out[static_cast<int64_t>(bj) * D + tid] = n_all < 0 ? __int_as_float(0x7fc00000) : o;
  }
  if (tid == 0) {
    if (p.sel_count != nullptr) p.sel_count[bj] = n_all;
    // the last row of all ends the step: its abort word is cleared for the next
    if (atomicAdd(p.tickets + p.B * p.h_q, 1) == p.B * p.h_q - 1) *p.abort = 0;
  }
}

}  // namespace

cudaError_t launch_q4_gather(const Q4Gather &p, int d, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.B * p.h_q * p.SB));
  if (d == 64) return launch_pdl(q4_gather_kernel<64>, grid, dim3(kThreads), 0, st, p);
  if (d == 128) return launch_pdl(q4_gather_kernel<128>, grid, dim3(kThreads), 0, st, p);
  return cudaErrorInvalidValue;
}

}  // namespace saga
