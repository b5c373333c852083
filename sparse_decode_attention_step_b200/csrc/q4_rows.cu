// Rows of the 4-bit cache: quantised as they are written, and read back.
//
// A block of 16 values x is stored as e4m3(max|x| / (6 g)) and 16 e2m1 codes
// of x / (scale g); see saga_q4.h. One thread quantises one block: the maximum,
// one division for the scale, 16 for the codes (true divisions, so that values
// on a rounding border go where the definition says), and the hardware's
// conversions, which round to nearest even.
#include "kernels.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t e4m3(float x) {           // x in [0, 448]
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(x));
  return d & 0xffu;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const uint32_t h = q4::scale_f16(byte);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu))) * kQ4Unit;
}

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(d)
      : "f"(hi), "f"(lo));
  return d;
}

template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
  float a[8], b[8];
  load8(p, a);
  load8(p + 8, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) { x[i] = a[i]; x[8 + i] = b[i]; }
}

template <typename T>
__device__ __forceinline__ void quantise_block(const T *src, float g, uint2 *codes, uint8_t *scale) {
  float x[16];
  load16(src, x);
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (x[i] != x[i]) x[i] = 0.f;                            // NaN counts as zero
    mx = fmaxf(mx, fabsf(x[i]));
  }
  const uint32_t s = e4m3(fminf(448.f, __fdiv_rn(mx, __fmul_rn(6.f, g))));
  const float t = __fmul_rn(e4m3_value(s), g);
  uint32_t w[2] = {0u, 0u};
  if (s != 0u) {
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      w[i / 8] |= e2m1x2(__fdiv_rn(x[i], t), __fdiv_rn(x[i + 1], t)) << (i % 8 * 4);
  }
  *codes = make_uint2(w[0], w[1]);
  *scale = static_cast<uint8_t>(s);
}

// New rows of one sequence: where they go, or n = 0 with the error recorded.
__device__ __forceinline__ int64_t append_rows(const Q4Append &p, int b, int64_t *at, bool report) {
  const int64_t l = p.l_kv[b];
  const int64_t n = p.n_new != nullptr ? p.n_new[b] : p.T;
  *at = l;
  int bad = 0;
  if (l < 0 || n < 0) bad = SAGA_DEVERR_LKV_NEGATIVE;
  else if (n > p.T || l + n > p.cap) bad = SAGA_DEVERR_LKV_TOO_LONG;
  if (bad != 0 && report) atomicOr(p.err, bad);
  return bad != 0 ? 0 : n;
}

// Block i of a head's n new rows, in position order.
template <typename T>
__device__ __forceinline__ void append_block(const Q4Append &p, int b, int hh, int64_t at, int64_t i) {
  const bool is_v = hh >= p.h_k;
  const int h = is_v ? hh - p.h_k : hh, heads = is_v ? p.h_v : p.h_k;
  const int bpr = p.d / 16;
  const int64_t r = i / bpr;
  const int w = static_cast<int>(i % bpr);
  const T *src = static_cast<const T *>(is_v ? p.v_new : p.k_new) +
                 ((static_cast<int64_t>(b) * p.T + r) * heads + h) * p.d + w * 16;
  const float *gp = is_v ? p.v_g : p.k_g;
  // codes: 8 bytes a block, scales: 1
  const int64_t blk = (is_v ? b * p.vb_sb + h * p.vb_sh : b * p.kb_sb + h * p.kb_sh) + (at + r) * bpr + w;
  quantise_block(src, gp != nullptr ? gp[h] : 1.f,
                 reinterpret_cast<uint2 *>(is_v ? p.vc : p.kc) + blk, (is_v ? p.vs : p.ks) + blk);
}

// Few rows: one CTA per sequence writes them all, then its length.
template <typename T>
__global__ void __launch_bounds__(kThreads) q4_append_small_kernel(const Q4Append p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  int64_t at;
  const int64_t n = append_rows(p, b, &at, threadIdx.x == 0);
  const int64_t per_head = n * (p.d / 16);
  for (int64_t i = threadIdx.x; i < per_head * (p.h_k + p.h_v); i += kThreads)
    append_block<T>(p, b, static_cast<int>(i / per_head), at, i % per_head);
  __syncthreads();
  if (threadIdx.x == 0 && n > 0) p.l_kv[b] = static_cast<int32_t>(at + n);
}

// Many rows: CTAs over (block ranges of a head, head, sequence); the lengths
// follow in a launch of their own, when every CTA has read them.
template <typename T>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const Q4Append p) {
  pdl_wait();
  pdl_trigger();
  const int hh = blockIdx.y % (p.h_k + p.h_v), b = blockIdx.y / (p.h_k + p.h_v);
  int64_t at;
  const int64_t n = append_rows(p, b, &at, blockIdx.x == 0 && hh == 0 && threadIdx.x == 0);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i < n * (p.d / 16)) append_block<T>(p, b, hh, at, i);
}

__global__ void q4_grow_kernel(const Q4Append p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.B) return;
  int64_t at;
  const int64_t n = append_rows(p, b, &at, false);
  if (n > 0) p.l_kv[b] = static_cast<int32_t>(at + n);
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread reads eight values of a row: four bytes of codes and their scale.
template <typename T>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const Q4Read p) {
  pdl_wait();
  pdl_trigger();
  const int hh = blockIdx.y % (p.h_k + p.h_v), b = blockIdx.y / (p.h_k + p.h_v);
  const bool is_v = hh >= p.h_k;
  const int h = is_v ? hh - p.h_k : hh, heads = is_v ? p.h_v : p.h_k;
  const int64_t l = p.l_kv[b], t0 = p.start != nullptr ? p.start[b] : 0;
  if (blockIdx.x == 0 && hh == 0 && threadIdx.x == 0 && (l < 0 || t0 < 0 || l > p.cap))
    atomicOr(p.err, l < 0 || t0 < 0 ? SAGA_DEVERR_LKV_NEGATIVE : SAGA_DEVERR_LKV_TOO_LONG);
  if (t0 < 0) return;
  const int64_t L = l < p.cap ? l : p.cap;
  const int ppr = p.d / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t r = i / ppr;
  const int w = static_cast<int>(i % ppr);
  if (r >= p.n || t0 + r >= L) return;
  const int64_t word = (is_v ? b * p.vb_sb + h * p.vb_sh : b * p.kb_sb + h * p.kb_sh) * 2 +
                       (t0 + r) * ppr + w;
  uint32_t c[4];
  q4::codes_f16(__ldg(reinterpret_cast<const uint32_t *>(is_v ? p.vc : p.kc) + word), c);
  const uint32_t s = q4::scale_f16(__ldg((is_v ? p.vs : p.ks) + word / 2));
  const float *gp = is_v ? p.v_g : p.k_g;
  const float g = (gp != nullptr ? gp[h] : 1.f);
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t v = q4::mul_f16x2(c[e], s);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
    // the stored value is exact before g: one rounding to fp32
    x[2 * e] = f.x * kQ4Unit * g;
    x[2 * e + 1] = f.y * kQ4Unit * g;
  }
  T *out = static_cast<T *>(is_v ? p.V : p.K) +
           ((static_cast<int64_t>(b) * heads + h) * p.n + r) * p.d + w * 8;
  store8(out, x);
}

}  // namespace

cudaError_t launch_q4_append(const Q4Append &p, int dtype, cudaStream_t st) {
  const int heads = p.h_k + p.h_v;
  const int64_t blocks = static_cast<int64_t>(p.T) * (p.d / 16);        // of one head
  // one CTA per sequence up to 4 blocks a thread: a launch less than the grid
  if (blocks * heads <= 4 * kThreads) {
    if (dtype == SAGA_BF16) return launch_pdl(q4_append_small_kernel<uint16_t>, dim3(p.B), dim3(kThreads), 0, st, p);
    return launch_pdl(q4_append_small_kernel<float>, dim3(p.B), dim3(kThreads), 0, st, p);
  }
  const dim3 grid(static_cast<unsigned>((blocks + kThreads - 1) / kThreads), p.B * heads);
  cudaError_t e = dtype == SAGA_BF16 ? launch_pdl(q4_append_kernel<uint16_t>, grid, dim3(kThreads), 0, st, p)
                                     : launch_pdl(q4_append_kernel<float>, grid, dim3(kThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(q4_grow_kernel, dim3((p.B + 63) / 64), dim3(64), 0, st, p);
}

cudaError_t launch_q4_read(const Q4Read &p, int dtype, cudaStream_t st) {
  const int64_t pieces = p.n * (p.d / 8);
  const dim3 grid(static_cast<unsigned>((pieces + kThreads - 1) / kThreads), p.B * (p.h_k + p.h_v));
  if (dtype == SAGA_BF16) return launch_pdl(q4_read_kernel<uint16_t>, grid, dim3(kThreads), 0, st, p);
  return launch_pdl(q4_read_kernel<float>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace saga
