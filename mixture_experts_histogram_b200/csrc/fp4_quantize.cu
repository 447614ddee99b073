// Microscaled 4-bit storage: quantisation, its inverse, and the gather that
// quantises activations on the way to their expert rows.
//
// MXFP4 (OCP Microscaling Formats v1.0): blocks of 32 inputs share an E8M0 scale
//   2^e, e = floor(log2(blockmax)) - 2; code = E2M1(x / 2^e), nearest, ties to
//   even, saturating at 6. Scaling by a power of two is exact, so the codes are
//   the correctly rounded ones. An all-zero block gets scale 1 (byte 127).
// NVFP4: blocks of 16 share an E4M3 scale s = E4M3(min(blockmax / (6 g), 448))
//   next to the matrix's fp32 scale g; code = E2M1(x / (s g)); s = 0 gives zero
//   codes. Both quotients are rounded once, as if computed exactly (below).
// A block with an infinity or a NaN (or a g that is not positive and finite)
// gets the scale's NaN code and zero codes: it reads back as NaN.
//
// The matrices are contiguous and K is a whole number of blocks, so codes,
// scales and inputs are flat arrays of blocks: one thread takes 8 inputs (16 or
// 32 bytes in, 4 bytes out) and 4 (MXFP4) or 2 (NVFP4) neighbouring lanes share
// a block. Bound by HBM: 2 (bf16) or 4 (fp32) bytes in and 0.53 / 0.56 out per
// input. Measured, 44 x 1536 x 4096 values: bf16 to MXFP4 118 us (700 MB, 5.9 TB/s) and
// back 104 us (6.7), fp32 to MXFP4 183 us (6.8); to NVFP4, where the arithmetic bounds it,
// bf16 235 us (3.0), fp32 207 to 218 us (6); the NVFP4 global scale 82 us bf16, 157 us fp32.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kVec = 8;       // inputs per thread and step
constexpr int kThreads = 128;
constexpr int kGatherThreads = 256;

// Steps whose loads are issued together: 128 bytes a thread, or what the registers of the
// longer arithmetic leave room for.
template <bool kMx, typename T>
constexpr int kSteps = sizeof(T) == 2 ? (kMx ? 8 : 4) : 3;
template <typename T>
constexpr int kAmaxSteps = sizeof(T) == 2 ? 8 : 4;
constexpr int kAmaxCtas = 4736;  // two rounds of 16 CTAs per SM

template <typename Tin>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_kept(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  // Largest magnitude as fp32 bits: bf16 bits order like the values.
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t a = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & a, v.y & a), __vmaxu2(v.z & a, v.w & a));
    return max(m & 0xffff0000u, m << 16);
  }
  __device__ __forceinline__ void get(float (&f)[kVec]) const {
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(b[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_kept(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ uint32_t amax() const {
    float f[kVec];
    get(f);
    return amax_bits<kVec>(f);
  }
  __device__ __forceinline__ void get(float (&f)[kVec]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

// 8 codes of an MXFP4 block part with scale byte sb.
__device__ __forceinline__ uint32_t mx_codes(const float (&f)[kVec], uint32_t sb) {
  return sb == 255u ? 0u : e2m1x8(f, e8m0_rcp(sb));
}

// NVFP4 in fp32, correctly rounded. An fp32 quotient is off by a few 2^-24; where moving
// it by 2^-20 either way does not change the rounded result it is the right one. The few
// others are redone with fp64 quotients, whose 53 bits cannot fall on the wrong side of a
// border of at most 5. bf16 values meet borders often, as their quotients have few
// distinct values; for them (kOften) the border b between two neighbouring results decides:
// x / (m g) > b just as x > (b m) g, where b m is exact and the product is taken in two
// parts. 44 x 1536 x 4096 values take 235 us with this test and 367 with fp64 quotients as
// bf16, but 225 to 234 and 207 to 218 as fp32.
template <bool kOften>
struct NvScale {
  float g, r6;  // global scale, about 1 / (6 g)
  bool ok;      // g positive and finite
  __device__ __forceinline__ explicit NvScale(float gg) : g(gg) {
    ok = gg > 0.0f && gg < INFINITY;
    r6 = __fdividef(1.0f, 6.0f * gg);
  }
  // Sign of a - c g, a within 2^-18 of c g and both far from the ends of the range: the
  // difference from the rounded product and the product's rounding error are both exact.
  static __device__ __forceinline__ float side(float a, float c, float g) {
    const float p = c * g;
    return (a - p) - fmaf(c, g, -p);
  }
  static __device__ __noinline__ uint32_t scale_slow(float bmax, float g) {
    const double q = (double)bmax / (6.0 * (double)g);
    if (q >= 448.0) return 0x7eu;
    int e = q > 0.0 ? ilogb(q) : -6;
    if (e < -6) e = -6;
    const double v = ldexp(rint(ldexp(q, 3 - e)), e - 3);
    return __nv_cvt_float_to_fp8((float)v, __NV_SATFINITE, __NV_E4M3);
  }
  // The code of a block maximum b that lies between the values of codes lo and hi.
  static __device__ __noinline__ uint32_t scale_at(float b, float g, uint32_t lo, uint32_t hi) {
    const float over = side(b, 3.0f * (e4m3_value(lo) + e4m3_value(hi)), g);
    return over > 0.0f || (over == 0.0f && (lo & 1u)) ? hi : lo;
  }
  // E4M3 code of the block scale.
  __device__ __forceinline__ uint32_t scale(uint32_t m) const {
    if (!ok || m >= 0x7f800000u) return 0x7fu;
    const float b = __uint_as_float(m);
    const float q = b * r6;
    const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(q * (1.0f - 0x1p-20f), q * (1.0f + 0x1p-20f)),
                                                  __NV_SATFINITE, __NV_E4M3);
    const bool in_range = r6 < 0x1p110f && r6 > 0x1p-110f;
    if ((two & 0xffu) == (two >> 8) && in_range) return two & 0xffu;
    if (kOften && in_range) return scale_at(b, g, two & 0xffu, two >> 8);
    return scale_slow(b, g);
  }
  // Codes lo, of that magnitude or the next where the nibbles of `open` are not zero.
  static __device__ __noinline__ uint32_t codes_at(float4 a, float4 b, float s, float g, uint32_t lo, uint32_t open) {
    const float f[kVec] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t w = lo;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (!((open >> (4 * i)) & 7u)) continue;
      const uint32_t c = (lo >> (4 * i)) & 7u;
      const float border = c < 4 ? 0.25f + 0.5f * (float)c : c == 6 ? 5.0f : (float)c - 1.5f;
      const float over = side(fabsf(f[i]), border * s, g);
      if (over > 0.0f || (over == 0.0f && (c & 1u))) w += 1u << (4 * i);
    }
    return w;
  }
  static __device__ __noinline__ uint32_t code_slow(float f, double d) {
    const double a = fabs((double)f) / d;
    const uint32_t c = (a > 0.25) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0);
    return c | (signbit(f) ? 8u : 0u);
  }
  __device__ __forceinline__ uint32_t codes(const float (&f)[kVec], uint32_t sb) const {
    const float s = e4m3_value(sb);
    if (sb == 0x7fu) return 0u;
    if (s == 0.0f) return 0u;
    const float d = s * g, r = __fdividef(1.0f, d);
    const uint32_t lo = e2m1x8(f, r * (1.0f - 0x1p-20f)), hi = e2m1x8(f, r * (1.0f + 0x1p-20f));
    if (lo == hi && d > 0x1p-110f && d < 0x1p110f) return lo;
    if (kOften && d > 0x1p-110f && d < 0x1p110f)
      return codes_at(make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7]), s, g, lo, lo ^ hi);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) w |= code_slow(f[i], (double)s * (double)g) << (4 * i);
    return w;
  }
};

// Grid: x over a matrix's vectors, y over matrices (MXFP4 ignores matrix borders: y = 1),
// both taken from the end: what a pass over x before this one (the global scale's) left
// in L2 is its end, and the inverse, from the front, finds the codes written last (24 x
// 1001 x 1536 fp32, the three passes: 84 us instead of 86). 128 threads with 128 bytes in
// flight each, rather than 256 with 64: bf16 to MXFP4 118 us instead of 140.
template <bool kMx, typename Tin>
__global__ void __launch_bounds__(kThreads) quantize_kernel(int64_t n_mat, int64_t vecs, const Tin* __restrict__ x,
                                                            const float* __restrict__ g, uint32_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  constexpr int kLanes = kMx ? 4 : 2;  // lanes of a block
  constexpr int kUnroll = kSteps<kMx, Tin>;
  for (int64_t mat = n_mat - 1 - blockIdx.y; mat >= 0; mat -= gridDim.y) {
    const int64_t base = mat * vecs;
    const NvScale<sizeof(Tin) == 2> nv(kMx ? 1.0f : g[mat]);
    const int64_t v0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
    Raw<Tin> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t v = v0 + u * kThreads;
      if (v < vecs) raw[u].load(x + (base + v) * kVec);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t v = v0 + u * kThreads;
      const bool live = v < vecs;  // whole blocks: the lanes of a block agree
      float f[kVec] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) raw[u].get(f);
      uint32_t m = live ? raw[u].amax() : 0u;
#pragma unroll
      for (int o = 1; o < kLanes; o *= 2) {
        const uint32_t t = __shfl_xor_sync(0xffffffffu, m, o);
        m = t > m ? t : m;
      }
      const uint32_t sb = kMx ? e8m0_of(m) : nv.scale(m);
      const uint32_t c = kMx ? mx_codes(f, sb) : nv.codes(f, sb);
      if (!live) continue;
      codes[base + v] = c;
      if (v % kLanes == 0) scales[(base + v) / kLanes] = (uint8_t)sb;
    }
  }
}

// Largest magnitude of each matrix, as fp32 bits in g (zeroed before).
template <typename Tin>
__global__ void __launch_bounds__(kThreads) amax_kernel(int64_t n_mat, int64_t vecs, const Tin* __restrict__ x,
                                                        uint32_t* __restrict__ g) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t part[kThreads / 32];
  constexpr int kUnroll = kAmaxSteps<Tin>;
  for (int64_t mat = blockIdx.y; mat < n_mat; mat += gridDim.y) {
    uint32_t m = 0;
    for (int64_t v0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x; v0 < vecs;
         v0 += (int64_t)gridDim.x * (kThreads * kUnroll)) {
      Raw<Tin> raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (v0 + u * kThreads < vecs) raw[u].load_kept(x + (mat * vecs + v0 + u * kThreads) * kVec);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (v0 + u * kThreads >= vecs) break;
        m = max(m, raw[u].amax());
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
      m = __reduce_max_sync(0xffffffffu, threadIdx.x < kThreads / 32 ? part[threadIdx.x] : 0u);
      if (threadIdx.x == 0) atomicMax(&g[mat], m);
    }
    __syncthreads();
  }
}

// g = amax / (6 * 448), rounded once; 1 for an all-zero matrix. A quotient that rounds to
// zero (amax below 2^-138.6) becomes the smallest fp32 number: with g = 0 a finite matrix
// would have no codes.
__global__ void __launch_bounds__(kThreads) global_scale_kernel(int64_t n_mat, float* g) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n_mat) return;
  const float q = __fdiv_rn(g[i], 2688.0f);
  g[i] = g[i] == 0.0f ? 1.0f : q == 0.0f ? 0x1p-149f : q;
}

// A thread writes 16 bytes a step, so that a warp's stores are whole lines: 8 bf16 values,
// or 4 fp32 ones (half a word of codes: 24 x 1001 x 1536 NVFP4 to fp32 27 us, 40 with a word's 8 by two stores).
template <bool kMx, typename Tout>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(int64_t n_mat, int64_t vecs,
                                                              const uint32_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              const float* __restrict__ g, Tout* __restrict__ y) {
  pdl_wait();
  pdl_trigger();
  constexpr int kOut = 16 / sizeof(Tout), kParts = kVec / kOut;  // values of a step, steps of a word
  constexpr int kLanes = (kMx ? 4 : 2) * kParts;                 // steps of a block
  constexpr int kUnroll = 4;
  const int64_t steps = vecs * kParts;
  for (int64_t mat = blockIdx.y; mat < n_mat; mat += gridDim.y) {
    const int64_t base = mat * steps;
    const float gs = kMx ? 1.0f : g[mat];
    const int64_t v0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint32_t w[kUnroll], sb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t v = v0 + u * kThreads;
      if (v < steps) {
        w[u] = __ldcs(codes + (base + v) / kParts);
        sb[u] = scales[(base + v) / kLanes];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t v = v0 + u * kThreads;
      if (v >= steps) break;
      if (kParts == 2) w[u] >>= 16 * (v & 1);  // (a matrix is whole words)
      // Value = (code x block scale) x global scale: the first product is exact.
      const float s = kMx ? e8m0_value(sb[u]) : e4m3_value(sb[u]);
      float f[kOut];
#pragma unroll
      for (int i = 0; i < kOut; ++i) {
        // E2M1 as fp32: exponent and mantissa bits in place, then rescaled by 2^126 (exact, zero and 0.5 included).
        const uint32_t c = w[u] >> (4 * i);
        const float e = __uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * 0x1p126f;
        f[i] = kMx ? e * s : __fmul_rn(__fmul_rn(e, s), gs);
      }
      if constexpr (kOut == 8) {
        uint4 o;
        __nv_bfloat162* ob = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
        for (int i = 0; i < 4; ++i) ob[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        __stcs(reinterpret_cast<uint4*>(y) + base + v, o);
      } else {
        __stcs(reinterpret_cast<float4*>(y) + base + v, make_float4(f[0], f[1], f[2], f[3]));
      }
    }
  }
}

// gather with MXFP4 quantisation: one CTA per token, 8 inputs per thread and
// step; codes and scales go to every row that the token feeds, row-major
// [rows, H/2] and [rows, H/32].
template <int kMaxSlots>
__global__ void __launch_bounds__(kGatherThreads) gather_mx_kernel(const GatherParams p) {
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  int32_t rows[kMaxSlots];
#pragma unroll
  for (int j = 0; j < kMaxSlots; ++j) rows[j] = j < p.S ? p.pos[t * p.S + j] : -1;
  const int nvec = p.H / kVec;  // a multiple of 32: whole warps
  const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(p.x) + t * p.H;
  for (int v = threadIdx.x; v < nvec; v += kGatherThreads) {
    Raw<__nv_bfloat16> raw;
    raw.load(x + v * kVec);
    float f[kVec];
    raw.get(f);
    uint32_t m = raw.amax();
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
      const uint32_t u = __shfl_xor_sync(0xffffffffu, m, o);
      m = u > m ? u : m;
    }
    const uint32_t sb = e8m0_of(m), c = mx_codes(f, sb);
#pragma unroll
    for (int j = 0; j < kMaxSlots; ++j) {
      const int64_t row = rows[j];
      if (row < 0) continue;
      static_cast<uint32_t*>(p.xp)[row * nvec + v] = c;
      if (v % 4 == 0) reinterpret_cast<uint8_t*>(p.sxp)[row * (nvec / 4) + v / 4] = (uint8_t)sb;
    }
  }
}

// CTAs for n_mat matrices of `steps` steps, `unroll` a thread.
dim3 step_grid(int64_t n_mat, int64_t steps, int unroll) {
  return dim3((unsigned)ceil_div(steps, kThreads * unroll), (unsigned)(n_mat < 65535 ? n_mat : 65535));
}
}  // namespace

cudaError_t launch_quantize_fp4(bool mx, bool f32, int64_t n_mat, int64_t elems, const void* x, const float* g,
                                uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  if (mx) {  // no per-matrix state: one flat array
    elems *= n_mat;
    n_mat = 1;
  }
  const int64_t vecs = elems / kVec;
  const int steps = mx ? (f32 ? kSteps<true, float> : kSteps<true, __nv_bfloat16>)
                       : (f32 ? kSteps<false, float> : kSteps<false, __nv_bfloat16>);
  const dim3 grid = step_grid(n_mat, vecs, steps);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(x);
  const float* xf = static_cast<const float*>(x);
  if (mx)
    return f32 ? launch_pdl(quantize_kernel<true, float>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, xf, g, c, scales)
               : launch_pdl(quantize_kernel<true, __nv_bfloat16>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, xb, g, c,
                            scales);
  return f32 ? launch_pdl(quantize_kernel<false, float>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, xf, g, c, scales)
             : launch_pdl(quantize_kernel<false, __nv_bfloat16>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, xb, g, c,
                          scales);
}

cudaError_t launch_fp4_global_scale(bool f32, int64_t n_mat, int64_t elems, const void* x, float* g, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(g, 0, (size_t)n_mat * 4, s);
  if (e != cudaSuccess) return e;
  const dim3 each((unsigned)ceil_div(n_mat, kThreads));
  if (elems == 0) return launch_pdl(global_scale_kernel, each, dim3(kThreads), 0, s, 1, n_mat, g);
  const int64_t vecs = elems / kVec;
  dim3 grid = step_grid(n_mat, vecs, f32 ? kAmaxSteps<float> : kAmaxSteps<__nv_bfloat16>);
  const unsigned most = (unsigned)ceil_div(kAmaxCtas, grid.y);
  if (grid.x > most) grid.x = most;
  uint32_t* gb = reinterpret_cast<uint32_t*>(g);
  e = f32 ? launch_pdl(amax_kernel<float>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, static_cast<const float*>(x), gb)
          : launch_pdl(amax_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs,
                       static_cast<const __nv_bfloat16*>(x), gb);
  if (e != cudaSuccess) return e;
  return launch_pdl(global_scale_kernel, each, dim3(kThreads), 0, s, 1, n_mat, g);
}

cudaError_t launch_dequantize_fp4(bool mx, bool f32, int64_t n_mat, int64_t elems, const uint8_t* codes,
                                  const uint8_t* scales, const float* g, void* y, cudaStream_t s) {
  if (mx) {
    elems *= n_mat;
    n_mat = 1;
  }
  const int64_t vecs = elems / kVec;
  const dim3 grid = step_grid(n_mat, f32 ? 2 * vecs : vecs, 4);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  __nv_bfloat16* yb = static_cast<__nv_bfloat16*>(y);
  float* yf = static_cast<float*>(y);
  if (mx)
    return f32 ? launch_pdl(dequantize_kernel<true, float>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, c, scales, g, yf)
               : launch_pdl(dequantize_kernel<true, __nv_bfloat16>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, c,
                            scales, g, yb);
  return f32 ? launch_pdl(dequantize_kernel<false, float>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, c, scales, g, yf)
             : launch_pdl(dequantize_kernel<false, __nv_bfloat16>, grid, dim3(kThreads), 0, s, 1, n_mat, vecs, c,
                          scales, g, yb);
}

cudaError_t launch_gather_mx(const GatherParams& p, cudaStream_t s) {
  if (p.T == 0) return cudaSuccess;
  const dim3 grid((unsigned)p.T), block(kGatherThreads);
  if (p.S <= 9) return launch_pdl(gather_mx_kernel<9>, grid, block, 0, s, 1, p);
  return launch_pdl(gather_mx_kernel<kMaxTopK + 1>, grid, block, 0, s, 1, p);
}

}  // namespace moe
