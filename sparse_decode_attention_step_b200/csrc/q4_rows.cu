// Rows of the 4-bit cache: quantised as they are written, and read back.
//
// A block of 16 values x is stored as e4m3(max|x| / (6 g)) and 16 e2m1 codes
// of x / (scale g); see saga_q4.h. One thread quantises one block: the maximum,
// one division for the scale, 16 correctly rounded quotients for the codes (so
// that values on a rounding border go where the definition says), and the
// hardware's conversions, which round to nearest even. Both kernels move each
// byte once, and a thread loads several blocks before it converts the first, which
// keeps more loads in flight (8 x 32K positions of 10 heads of 64 read back in bf16:
// 430 MB in 70 us, 6.1 TB/s, against 152 us with one piece a thread). The append of a
// prompt is bound by instruction issue instead, about 10 a value (8 ragged prompts of
// up to 8192 rows of 10 heads of 64, 54 MB: 19 us, 2.8 TB/s).
#include "kernels.h"
#include "q4.cuh"
#include "q4_kernels.h"

namespace saga {

namespace {

constexpr int kThreads = 256;
template <typename T>
constexpr int kAppendBlocks = sizeof(T) == 2 ? 4 : 2;      // blocks of 16 a thread: 128 bytes in flight
constexpr int kReadPieces = 8;                             // pieces of 8 values a thread

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

// x / t, correctly rounded, by Markstein's method (IBM J. Res. Dev. 34, 1990):
// with `inv` the rounded reciprocal, one correction makes the quotient faithful
// and a second one from its exact residual rounds it correctly. For t within
// 2^+-100 and |x| <= 8 t the residuals neither overflow nor lose bits that matter
// (a quotient small enough for that rounds to code 0 all the same).
// The residual is taken as q t - x and subtracted: where q is a zero it is +0 (0 t + 0, or -0 +
// 0), so that -0 - 0 and 0 - 0 leave the quotient its sign.
__device__ __forceinline__ float quotient(float x, float t, float inv) {
  float q = x * inv;
  q = fmaf(-fmaf(q, t, -x), inv, q);
  return fmaf(-fmaf(q, t, -x), inv, q);
}

// A thread's raw block of 16 values, loaded ahead of its conversion.
struct Raw16 {
  uint4 w[4];
};
__device__ __forceinline__ void load_raw(const uint16_t *p, Raw16 &r) {
  r.w[0] = __ldg(reinterpret_cast<const uint4 *>(p));
  r.w[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
}
__device__ __forceinline__ void load_raw(const float *p, Raw16 &r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
}
template <typename T>
__device__ __forceinline__ void widen(const Raw16 &r, float (&x)[16]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) { x[8 * i + 2 * e] = bf16lo(u[e]); x[8 * i + 2 * e + 1] = bf16hi(u[e]); }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = __uint_as_float(r.w[i].x); x[4 * i + 1] = __uint_as_float(r.w[i].y);
      x[4 * i + 2] = __uint_as_float(r.w[i].z); x[4 * i + 3] = __uint_as_float(r.w[i].w);
    }
  }
}

// The largest magnitude of a block; infinite or NaN when it holds such a value.
template <typename T>
__device__ __forceinline__ float block_max(const Raw16 &r) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = 0u;                     // magnitudes order like integers, NaN above infinity
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(u[e] & 0x7fff7fffu));
    }
    return __uint_as_float(max(m << 16, m & 0xffff0000u));
  } else {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(__uint_as_float(u[e]))));
    }
    return m;
  }
}

template <typename T>
__device__ __forceinline__ void quantise_block(const Raw16 &raw, float g, uint2 *codes, uint8_t *scale) {
  float x[16];
  widen<T>(raw, x);
  float mx = block_max<T>(raw);
  const bool finite = mx < INFINITY;
  if (!finite) {                         // NaN counts as zero
    mx = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (x[i] != x[i]) x[i] = 0.f;
      mx = fmaxf(mx, fabsf(x[i]));
    }
  }
  const uint32_t s = e4m3(fminf(448.f, __fdiv_rn(mx, __fmul_rn(6.f, g))));
  const float t = __fmul_rn(e4m3_value(s), g);
  uint32_t w[2] = {0u, 0u};
  if (s != 0u) {
    // a block's maximum is about 6 t, and more only where its scale stopped at 448
    if (finite && t > 0x1p-100f && t < 0x1p100f && mx <= 8.f * t) {
      const float inv = __frcp_rn(t);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = quotient(x[i], t, inv);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], t);
    }
    // the conversion takes the sign along and everything above 6 to 6
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __byte_perm(e2m1x2(x[8 * i], x[8 * i + 1]), e2m1x2(x[8 * i + 2], x[8 * i + 3]), 0x0040);
      const uint32_t hi = __byte_perm(e2m1x2(x[8 * i + 4], x[8 * i + 5]), e2m1x2(x[8 * i + 6], x[8 * i + 7]), 0x0040);
      w[i] = __byte_perm(lo, hi, 0x5410);
    }
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
  else if (n > p.T || l + n > p.cap || l + n > INT32_MAX) bad = SAGA_DEVERR_LKV_TOO_LONG;
  if (bad != 0 && report) atomicOr(p.err, bad);
  return bad != 0 ? 0 : n;
}

// Blocks of a head's n new rows, in position order: where block i comes from
// and goes to.
template <typename T>
struct AppendHead {
  const T *src;
  uint8_t *codes, *scales;
  int64_t src_row, first;      // elements between the head's new rows; first block of row l_kv[b]
  int64_t room, given;         // blocks of the head from there on; blocks of its new rows
  int32_t *err;
  float g;
  int bpr;                     // blocks per row

  __device__ __forceinline__ AppendHead(const Q4Append &p, int b, int hh, int64_t at) {
    const bool is_v = hh >= p.h_k;
    const int h = is_v ? hh - p.h_k : hh, heads = is_v ? p.h_v : p.h_k;
    bpr = p.d / 16;
    src_row = static_cast<int64_t>(heads) * p.d;
    src = static_cast<const T *>(is_v ? p.v_new : p.k_new) + static_cast<int64_t>(b) * p.T * src_row + h * p.d;
    codes = is_v ? p.vc : p.kc;
    scales = is_v ? p.vs : p.ks;
    first = (is_v ? b * p.vb_sb + h * p.vb_sh : b * p.kb_sb + h * p.kb_sh) + at * bpr;
    room = (p.cap - at) * bpr;
    given = static_cast<int64_t>(p.T) * bpr;
    err = p.err;
    const float *gp = is_v ? p.v_g : p.k_g;
    g = gp != nullptr ? __ldg(gp + h) : 1.f;
  }
  // i / bpr by a shift: bpr is 4 or 8
  __device__ __forceinline__ const T *from(int64_t i) const {
    return src + (i >> (bpr == 4 ? 2 : 3)) * src_row + (i & (bpr - 1)) * 16;
  }
  __device__ __forceinline__ bool has(int64_t i) const { return saga_in_bounds(i >= 0 && i < given && i < room, err); }
  __device__ __forceinline__ void put(int64_t i, const Raw16 &raw) const {
    quantise_block<T>(raw, g, reinterpret_cast<uint2 *>(codes) + first + i, scales + first + i);
  }
};

// Few rows: one CTA per sequence writes them all, then its length.
template <typename T>
__global__ void __launch_bounds__(kThreads) q4_append_small_kernel(const Q4Append p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  int64_t at;
  const int64_t n = append_rows(p, b, &at, threadIdx.x == 0);
  const int per_head = static_cast<int>(n) * (p.d / 16);
  for (int i = threadIdx.x; i < per_head * (p.h_k + p.h_v); i += kThreads) {
    const AppendHead<T> h(p, b, i / per_head, at);
    Raw16 raw;
    if (!h.has(i % per_head)) continue;
    load_raw(h.from(i % per_head), raw);
    h.put(i % per_head, raw);
  }
  __syncthreads();
  if (threadIdx.x == 0 && n > 0) p.l_kv[b] = static_cast<int32_t>(at + n);
}

// Many rows: CTAs over (block ranges of a head, head, sequence); the lengths
// follow in a launch of their own, when every CTA has read them.
template <typename T>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(const Q4Append p) {
  constexpr int U = kAppendBlocks<T>;
  pdl_wait();
  pdl_trigger();
  const int hh = blockIdx.y % (p.h_k + p.h_v), b = blockIdx.y / (p.h_k + p.h_v);
  int64_t at;
  const int64_t n = append_rows(p, b, &at, blockIdx.x == 0 && hh == 0 && threadIdx.x == 0) * (p.d / 16);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * U) + threadIdx.x;
  if (i0 >= n) return;
  const AppendHead<T> h(p, b, hh, at);
  Raw16 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (i0 + u * kThreads < n && h.has(i0 + u * kThreads)) load_raw(h.from(i0 + u * kThreads), raw[u]);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (i0 + u * kThreads < n && h.has(i0 + u * kThreads)) h.put(i0 + u * kThreads, raw[u]);
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

// A thread reads kReadPieces pieces of eight values: four bytes of codes and
// their scale each.
template <typename T>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const Q4Read p) {
  constexpr int U = kReadPieces;
  pdl_wait();
  pdl_trigger();
  const int hh = blockIdx.y % (p.h_k + p.h_v), b = blockIdx.y / (p.h_k + p.h_v);
  const bool is_v = hh >= p.h_k;
  const int h = is_v ? hh - p.h_k : hh, heads = is_v ? p.h_v : p.h_k;
  const int64_t l = p.l_kv[b], t0 = p.start != nullptr ? p.start[b] : 0;
  if (blockIdx.x == 0 && hh == 0 && threadIdx.x == 0 && (l < 0 || t0 < 0 || l > p.cap))
    atomicOr(p.err, l < 0 || t0 < 0 ? SAGA_DEVERR_LKV_NEGATIVE : SAGA_DEVERR_LKV_TOO_LONG);
  if (t0 < 0) return;
  const int64_t rows = min(p.n, (l < p.cap ? l : p.cap) - t0);   // rows of the window that exist
  const int ppr = p.d / 8;
  const int64_t n = rows * ppr;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * U) + threadIdx.x;
  if (i0 >= n) return;
  const int64_t first = (is_v ? b * p.vb_sb + h * p.vb_sh : b * p.kb_sb + h * p.kb_sh) * 2 + t0 * ppr;
  const uint32_t *codes = reinterpret_cast<const uint32_t *>(is_v ? p.vc : p.kc) + first;
  const uint8_t *scales = (is_v ? p.vs : p.ks) + first / 2;      // first is even: rows are
  const float *gp = is_v ? p.v_g : p.k_g;
  const float g = gp != nullptr ? __ldg(gp + h) : 1.f;
  T *out = static_cast<T *>(is_v ? p.V : p.K) + (static_cast<int64_t>(b) * heads + h) * p.n * p.d;
  uint32_t w[U], s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * kThreads;
    // inside of the window and of the head
    if (i < n && saga_in_bounds(i < p.n * ppr && t0 * ppr + i < p.cap * ppr, p.err)) {
      w[u] = __ldg(codes + i);
      s[u] = __ldg(scales + i / 2);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * kThreads;
    if (i >= n || !saga_in_bounds(i < p.n * ppr && t0 * ppr + i < p.cap * ppr, p.err)) break;
    uint32_t c[4];
    q4::codes_f16(w[u], c);
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // code * scale (at most 2688, so exact in fp16), without the factor 2^-8 of the
      // scale; then times g, one rounding to fp32
      const uint32_t v = q4::mul_f16x2(q4::mul_f16x2(c[e], 0x5c005c00u), q4::scale_f16(s[u]));
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
      x[2 * e] = f.x * g;
      x[2 * e + 1] = f.y * g;
    }
    store8(out + i * 8, x);
  }
}

}  // namespace

cudaError_t launch_q4_append(const Q4Append &p, int dtype, cudaStream_t st) {
  const int heads = p.h_k + p.h_v;
  const int64_t blocks = static_cast<int64_t>(p.T) * (p.d / 16);        // of one head
  // one CTA per sequence up to 2 blocks a thread, which saves a launch: with 40
  // blocks a sequence 5.0 us instead of 6.0, with 320 5.8 instead of 6.1; with 1000 the
  // grid's 6.4 are less than its 7.4 (8 sequences, 10 heads of 64)
  if (blocks * heads <= 2 * kThreads) {
    if (dtype == SAGA_BF16) return launch_pdl(q4_append_small_kernel<uint16_t>, dim3(p.B), dim3(kThreads), 0, st, p);
    return launch_pdl(q4_append_small_kernel<float>, dim3(p.B), dim3(kThreads), 0, st, p);
  }
  const int64_t per_cta = kThreads * (dtype == SAGA_BF16 ? kAppendBlocks<uint16_t> : kAppendBlocks<float>);
  const dim3 grid(static_cast<unsigned>((blocks + per_cta - 1) / per_cta), p.B * heads);
  cudaError_t e = dtype == SAGA_BF16 ? launch_pdl(q4_append_kernel<uint16_t>, grid, dim3(kThreads), 0, st, p)
                                     : launch_pdl(q4_append_kernel<float>, grid, dim3(kThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(q4_grow_kernel, dim3((p.B + 63) / 64), dim3(64), 0, st, p);
}

cudaError_t launch_q4_read(const Q4Read &p, int dtype, cudaStream_t st) {
  const int64_t pieces = p.n * (p.d / 8);
  const int64_t per_cta = kThreads * kReadPieces;
  const dim3 grid(static_cast<unsigned>((pieces + per_cta - 1) / per_cta), p.B * (p.h_k + p.h_v));
  if (dtype == SAGA_BF16) return launch_pdl(q4_read_kernel<uint16_t>, grid, dim3(kThreads), 0, st, p);
  return launch_pdl(q4_read_kernel<float>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace saga
