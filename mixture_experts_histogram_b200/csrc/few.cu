// The whole layer for a few tokens (1 to 8) in two kernels.
//
// With so few tokens the layer is a stream over the touched experts' weights
// (FP8, T = 1: 9 experts, 170 MB, 26 us at the measured HBM rate); the launches,
// the permutation and each GEMM's start and end cost more than that. Here one
// launch computes the router logits and a second, cooperative one (one CTA per
// SM) does the rest without ever letting the weight stream stop:
//
//   top-k    every CTA selects all tokens' experts from the logits and lists the
//            distinct ones (the shared expert first), so each expert's weights are
//            read once whatever number of tokens chose it.
//   gate/up  the listed experts' features are divided evenly over the CTAs. A tile
//            is 8 features: 8 rows of W1 and the same 8 rows of W3 make the 16 rows
//            of an mma.sync tile whose 8 columns are the tokens, so a thread holds
//            the gate and the up sum of the same feature.
//   grid barrier, during which the rings fill with W2.
//   down     each CTA owns H / CTAs output rows for every listed expert and adds
//            the gate-weighted products up: no partial output leaves the SM, and
//            the sum's order (experts ascending, then the shared one) does not
//            depend on the other tokens. Four warps bring each expert's h, as fp32
//            from L2, into shared memory in the storage's activation format.
//
// One thread streams weight rows by TMA (boxes of 128 bytes x 8 rows x 8 lines, in the
// down phase of up to 32 rows and fewer lines, 128B-swizzled; bulk copies row by row
// reached 4.1 TB/s, boxes the HBM rate) into a ring, another the scale bytes of 4-bit
// storage, and two of the h warps the up rows and theirs; eight warps multiply, each a
// whole stage in its turn, and two add up their partial sums in stage order and finish
// the tiles. (With every stage split over the warps the waits and the address
// arithmetic cost more than the products: 2.0 TB/s for FP8.) The shared expert's rows
// are known before the routing is: their copies start at once, while the experts are
// selected.
// Tensor-core work is mma.sync (m16n8): at 23 weight bytes per clock and SM the
// MMAs are far from a limit, and 8 columns fit 8 tokens without padding.
//
// Measured (H = 4096, I = 1536, 352 experts, top-8 and a shared one, in long runs under
// the power limit; the floor is the weights at 6.45 TB/s): BF16 T = 3 153 us (0.94 of the
// floor's rate), FP8 T = 8 224 us (0.79; 212 us in short runs at full clocks), T = 1 47 us
// (0.57: of these the logits, the cooperative launch and the selection take 8 us, the
// first tile 3 and the barrier 4). 4-bit storage is bound by the expansion of the codes,
// about 370 warp instructions for a 2 KB line of 16 rows: MXFP4 T = 8 216 us (0.44), T = 1
// 49 us; NVFP4 T = 5 144 us (0.45). Twelve multiplying warps instead of eight leave 96
// registers each: MXFP4 T = 8 242 us; the halves of a line as a rolled loop: 230 us, two
// lines unrolled: 288 us.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "few.cuh"
#include "fp4.cuh"
#include "gemm_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kAcc = 2;                      // warps that add up
constexpr int kPrep = 4;                     // warps that bring h
constexpr int kTeam = 1;                     // multiplying warps that share a stage
constexpr int kHRing = 24;                   // experts of h in shared memory at most
constexpr int kRows = 16;                    // rows of a stage
constexpr int kLine = 128;                   // bytes of a row that a step multiplies
constexpr int kMaxRing = 24;
constexpr int kMaxU = kFewMaxTokens * kMaxTopK + 1;
constexpr int kRouterThreads = 256;
constexpr int kRouterExperts = 2;            // experts of a router CTA

// Per storage: inputs per 2 bytes of a weight row, bytes of a row in a stage (a
// slab), scale bytes per row and slab (4-bit storage), padding of an activation row in
// shared memory that keeps the fragment loads free of bank conflicts, inputs per
// activation block that has a scale (0: activations stay bf16), and multiplying warps.
template <int kW>
struct Fmt;
template <>
struct Fmt<MOE_WDTYPE_BF16> {
  static constexpr int kPer2 = 1, kSlab = 1024, kScaleSlab = 0, kXPad = 64, kBlock = 0, kWarps = 8;
};
template <>
struct Fmt<MOE_WDTYPE_FP8_E4M3> {
  static constexpr int kPer2 = 2, kSlab = 1024, kScaleSlab = 0, kXPad = 16, kBlock = 128, kWarps = 8;
};
template <>
struct Fmt<MOE_WDTYPE_NVFP4> {
  static constexpr int kPer2 = 4, kSlab = 1024, kScaleSlab = kSlab / 8, kXPad = 64, kBlock = 128, kWarps = 8;
};
template <>
struct Fmt<MOE_WDTYPE_MXFP4> {
  static constexpr int kPer2 = 4, kSlab = 1024, kScaleSlab = kSlab / 16, kXPad = 64, kBlock = 128, kWarps = 8;
};

template <int kW>
struct Smem {
  using F = Fmt<kW>;
  static constexpr int kWarps = F::kWarps, kTeams = kWarps / kTeam;
  static constexpr int kProducers = F::kScaleSlab ? 2 : 1;  // weight rows, scale bytes
  static constexpr int kConsumers = (kWarps + kAcc + kPrep) * 32;
  static constexpr int kThreads = kConsumers + kProducers * 32;
  static_assert(kMaxRing <= 32 && kHRing <= 32 && kTeams <= 32 && kWarps >= kFewMaxTokens, "one thread per barrier");
  static_assert(kTeams < kHRing, "a team's stages must not skip a whole ring of experts");
  static constexpr int kStageScales = kRows * F::kScaleSlab;  // a stage's scale bytes
  static constexpr int kStage = kRows * F::kSlab + kStageScales;
  // Fixed part: barriers, tables, partial sums. Then the activations (x, later rows
  // of h), the scale bytes and the weight tiles.
  static constexpr int kBars = 0;
  static constexpr int kNumBars = 2 * kMaxRing + 2 * kTeams + 2 * kHRing + 3 + kAcc;
  static constexpr int kMisc = (kBars + kNumBars * 8 + 15) / 16 * 16;  // abort flag, list length
  static constexpr int kTopIdx = kMisc + 64;                         // int [8][16]
  static constexpr int kTopW = kTopIdx + kFewMaxTokens * kMaxTopK * 4;
  static constexpr int kBits = kTopW + kFewMaxTokens * kMaxTopK * 4; // uint [16] chosen experts, int [16] prefix
  static constexpr int kList = kBits + 2 * 16 * 4;                   // int [kMaxU] experts
  static constexpr int kUsed = kList + ((kMaxU * 4 + 15) / 16) * 16; // uint [kMaxU] token masks
  static constexpr int kFirst = kUsed + ((kMaxU * 4 + 15) / 16) * 16;  // int [kMaxU + 1] rows of h before an entry
  static constexpr int kGate = kFirst + ((kMaxU * 4 + 4 + 15) / 16) * 16;  // float [kMaxU][8]
  static constexpr int kRed = kGate + kMaxU * kFewMaxTokens * 4;     // float [kWarps][2][32][4] partial sums
  static constexpr int kDown = kRed + kWarps * 256 * 4;              // float [kFewDownTiles][32][4] output sums
  static constexpr int kX = kDown + kFewDownTiles * 128 * 4;
  static_assert(kX % 16 == 0, "alignment");
  // A row of K activations: operands, padding, block scales.
  static __host__ __device__ int scales_at(int K) { return K * 2 + F::kXPad; }
  static __host__ __device__ int pitch(int K) {
    return F::kBlock ? (scales_at(K) + K / F::kBlock * 4 + 63) / 128 * 128 + 64 + (F::kXPad == 16 ? 16 : 0) : scales_at(K);
  }
  // Bytes for T rows of x, and then for rows of h: T at least, and up to a dozen so
  // that the next experts' can be brought while one is used.
  static __host__ __device__ int act_bytes(int T, int H, int I) {
    const int x = T * pitch(H), some = 40 * 1024 / pitch(I), rows = some > 12 ? 12 : some;
    const int h = (rows > T ? rows : T) * pitch(I);
    return (x > h ? x : h);
  }
  static __host__ __device__ int scale_offset(int T, int H, int I) {
    return (kX + act_bytes(T, H, I) + 127) / 128 * 128;
  }
  static __host__ __device__ int tile_offset(int T, int H, int I, int stages) {
    return (scale_offset(T, H, I) + stages * kStageScales + 1023) / 1024 * 1024;
  }
  static __host__ __device__ int stages(int T, int H, int I) {
    const int n = (kFewSmem - 2048 - scale_offset(T, H, I)) / kStage;  // both alignments
    return n > kMaxRing ? kMaxRing : n;
  }
};

// ------------------------------------------------------------------- pieces --

__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// 3-D tiled tensor load: 128 bytes x rows from `row` x 8 lines of 128 bytes from `line`.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t row,
                                              int32_t line) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(row), "r"(line)
      : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_b16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Activations are 16-bit operands: bf16 (BF16); the f16 values of the E4M3 codes
// (FP8; exact); or, for 4-bit weights, f16 next to a power of two for each 128 inputs:
// NVFP4, whose activations are not quantised, with the largest at [2^14, 2^15); MXFP4,
// whose quantised values have exponents of their own for each 32 inputs, with the
// largest of these at 2^12. What f16 cannot hold then is below 2^-31 (NVFP4 values) or
// 2^-35 (MXFP4 blocks) of the largest, where the fp32 sums have 24 bits. Values lie in input order, but for NVFP4,
// whose groups of 8 inputs are transposed 4 x 4 within 32 x 4 inputs, as its lanes
// read them.
template <int kW>
__device__ __forceinline__ int x_group(int v) {
  return kW == MOE_WDTYPE_NVFP4 ? (v & ~15) | (v & 3) << 2 | ((v >> 2) & 3) : v;
}

// The f16 values of four E4M3 codes, in order.
__device__ __forceinline__ void f16_of_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// The f16 values of a word of eight E2M1 codes, in order.
__device__ __forceinline__ void f16_of_e2m1x8(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The four E8M0 scales of a word as fp32 (by way of bf16, which holds them all; 255: NaN).
__device__ __forceinline__ void e8m0_weights(uint32_t word, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(word));
  f[0] = __uint_as_float(lo << 16);
  f[1] = __uint_as_float(lo & 0xffff0000u);
  f[2] = __uint_as_float(hi << 16);
  f[3] = __uint_as_float(hi & 0xffff0000u);
}

// Sums of a stage, in as many independent chains of MMAs as hide their latency.
struct Sums {
  float a[4][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) a[i][j] = 0.0f;
  }
  __device__ __forceinline__ float4 total() const {
    float s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = (a[0][j] + a[1][j]) + (a[2][j] + a[3][j]);
    return make_float4(s[0], s[1], s[2], s[3]);
  }
};

// Shared-memory loads by 32-bit address: through generic pointers every one of them
// would carry 64-bit address arithmetic.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

// What a lane needs of a line of a stage, as shared-memory addresses: its two weight
// rows (g, g + 8 of an MMA tile) and their scale bytes, the token's activations (token
// g) and the block scales of the tokens of its columns (2c, 2c + 1).
struct Operands {
  uint32_t a0, a1, c0, c1, x, s0, s1;
};

// acc += rows x tokens over a line. sb0, sb1 (FP8): weight scales of rows g and g + 8
// in this line's 128 inputs.
template <int kW>
__device__ __forceinline__ void line_mma(Sums& acc, const Operands& o, float sb0, float sb1, int lane) {
  const int c = lane % 4;
  // The 128-byte swizzle: 16-byte unit i of a line lies at i ^ (line address / 128 % 8).
  const uint32_t x0 = (o.a0 >> 3) & 0x70u, x1 = (o.a1 >> 3) & 0x70u;
  if constexpr (kW == MOE_WDTYPE_MXFP4) {
    // Eight 32-input blocks, two MMAs each (lane c takes the block's word c); a block's
    // sum is weighted by the weights' scale, and four blocks' by the activations'.
    const uint32_t a0 = o.a0 + 4 * c, a1 = o.a1 + 4 * c;
    const uint2 w0 = lds64(o.c0), w1 = lds64(o.c1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[4] = {0.f, 0.f, 0.f, 0.f}, f0[4], f1[4];
      e8m0_weights(h ? w0.y : w0.x, f0);
      e8m0_weights(h ? w1.y : w1.x, f1);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t u = (uint32_t)(4 * h + b) << 4;
        uint32_t va[4], vb[4];
        f16_of_e2m1x8(lds32(a0 + (u ^ x0)), va);
        f16_of_e2m1x8(lds32(a1 + (u ^ x1)), vb);
        const uint4 x = lds128(o.x + (4 * h + b) * 64 + 16 * c);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(d, va[0], vb[0], va[1], vb[1], x.x, x.y);
        mma_f16(d, va[2], vb[2], va[3], vb[3], x.z, x.w);
        t[0] = fmaf(d[0], f0[b], t[0]);
        t[1] = fmaf(d[1], f0[b], t[1]);
        t[2] = fmaf(d[2], f1[b], t[2]);
        t[3] = fmaf(d[3], f1[b], t[3]);
      }
      const float sx0 = __uint_as_float(lds32(o.s0 + 4 * h)), sx1 = __uint_as_float(lds32(o.s1 + 4 * h));
      acc.a[h][0] = fmaf(t[0], sx0, acc.a[h][0]);
      acc.a[h][1] = fmaf(t[1], sx1, acc.a[h][1]);
      acc.a[h][2] = fmaf(t[2], sx0, acc.a[h][2]);
      acc.a[h][3] = fmaf(t[3], sx1, acc.a[h][3]);
    }
  } else {
    const uint32_t a0 = o.a0 + ((c << 4) ^ x0), a1 = o.a1 + ((c << 4) ^ x1);
    float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // halves of the line, 64 bytes
      const uint4 a = lds128(h ? a0 ^ 64u : a0), b = lds128(h ? a1 ^ 64u : a1);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
      if constexpr (kW == MOE_WDTYPE_BF16) {
        const uint4 x = lds128(o.x + h * 64 + 16 * c);
        mma_b16(acc.a[2 * h], aw[0], bw[0], aw[1], bw[1], x.x, x.y);
        mma_b16(acc.a[2 * h + 1], aw[2], bw[2], aw[3], bw[3], x.z, x.w);
      } else if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
        const uint4 xa = lds128(o.x + h * 128 + 32 * c), xb = lds128(o.x + h * 128 + 32 * c + 16);
        const uint32_t xv[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a_lo, a_hi, b_lo, b_hi;
          f16_of_e4m3x4(aw[j], a_lo, a_hi);
          f16_of_e4m3x4(bw[j], b_lo, b_hi);
          mma_f16(d[j & 1], a_lo, b_lo, a_hi, b_hi, xv[2 * j], xv[2 * j + 1]);
        }
      } else {
        // NVFP4: the codes times their 16-input scale, exact in f16 (5 significant
        // bits, 2^-10 to 2688); 128 inputs a half, with one activation scale.
        const uint32_t sa = lds16(o.c0 + h * 8 + 2 * c), sb = lds16(o.c1 + h * 8 + 2 * c);
        const uint32_t wa[2] = {f16x2_of_e4m3x2(__byte_perm(sa, 0, 0x00)), f16x2_of_e4m3x2(__byte_perm(sa, 0, 0x11))};
        const uint32_t wb[2] = {f16x2_of_e4m3x2(__byte_perm(sb, 0, 0x00)), f16x2_of_e4m3x2(__byte_perm(sb, 0, 0x11))};
        float e[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 x = lds128(o.x + h * 256 + 64 * j + 16 * c);
          uint32_t va[4], vb[4];
          f16_of_e2m1x8(aw[j], va);
          f16_of_e2m1x8(bw[j], vb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            va[i] = mul_f16x2(va[i], wa[j / 2]);
            vb[i] = mul_f16x2(vb[i], wb[j / 2]);
          }
          mma_f16(e[j & 1], va[0], vb[0], va[1], vb[1], x.x, x.y);
          mma_f16(e[j & 1], va[2], vb[2], va[3], vb[3], x.z, x.w);
        }
        const float sx0 = __uint_as_float(lds32(o.s0 + 4 * h)), sx1 = __uint_as_float(lds32(o.s1 + 4 * h));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc.a[0][2 * i] = fmaf(e[0][2 * i] + e[1][2 * i], sx0, acc.a[0][2 * i]);
          acc.a[0][2 * i + 1] = fmaf(e[0][2 * i + 1] + e[1][2 * i + 1], sx1, acc.a[0][2 * i + 1]);
        }
      }
    }
    if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
      const float sx0 = __uint_as_float(lds32(o.s0)), sx1 = __uint_as_float(lds32(o.s1));
      acc.a[0][0] = fmaf(d[0][0] + d[1][0], sx0 * sb0, acc.a[0][0]);
      acc.a[0][1] = fmaf(d[0][1] + d[1][1], sx1 * sb0, acc.a[0][1]);
      acc.a[0][2] = fmaf(d[0][2] + d[1][2], sx0 * sb1, acc.a[0][2]);
      acc.a[0][3] = fmaf(d[0][3] + d[1][3], sx1 * sb1, acc.a[0][3]);
    }
  }
}

// What FP8 h is quantised with: its block's scale s as e4m3_scale gives it, and codes
// (h up) r, with up = 2^64 where s or its reciprocal could leave the normal range, else 1.
// Quotient and reciprocal are corrected by their residuals in fused arithmetic (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990) and
// equal __fdiv_rn and __frcp_rn for every finite largest magnitude (an infinite one gives
// NaN codes). With those two functions T = 8 took 4% longer, T = 1 0.5 us.
struct HScale {
  float s, up, r;
  __device__ __forceinline__ explicit HScale(float amax) {
    constexpr float c = 1.0f / 448.0f;
    const bool small = amax < 0x1p-60f;
    up = small ? kE4m3Lift : 1.0f;
    const float a = amax * up, q = a * c;
    s = fmaf(fmaf(-q, 448.0f, a), c, q);
    if (small) s = amax > 0.0f ? fmaxf(s * (1.0f / kE4m3Lift), 0x1p-149f) : 1.0f;
    if (!(amax <= INFINITY)) s = 1.0f;  // a NaN among the values: its code is NaN
    const float b = s * up;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
    r = fmaf(r, fmaf(-b, r, 1.0f), r);
  }
};

// 8 values of a row (inputs 8 v .. 8 v + 7; all lanes of the warp take part, `live`
// ones hold values) into the operand row at `row` with scales behind it. FP8:
// kDivide quantises by quotients (x, as moe_quantize_act defines it), else by products
// with the scale's reciprocal, correctly rounded (h, as the grouped GEMMs do).
template <int kW, bool kDivide>
__device__ __forceinline__ void store_operand(uint8_t* row, int scales_at, int v, const float (&f)[8], bool live) {
  using F = Fmt<kW>;
  if constexpr (F::kBlock == 0) {
    if (live)
      *reinterpret_cast<uint4*>(row + v * 16) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                           pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
    uint32_t m = amax_bits<8>(f);
    constexpr int kLanes = F::kBlock / 8;  // 16 lanes share a block
    constexpr int kQuantLanes = kW == MOE_WDTYPE_MXFP4 ? 4 : kLanes;
#pragma unroll
    for (int o = 1; o < kQuantLanes; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    uint32_t mx_top = 0;  // MXFP4: the largest scale byte of the 128 inputs, blocks of zeros left out
    if constexpr (kW == MOE_WDTYPE_MXFP4) {
      mx_top = m ? e8m0_of(m) : 0u;
#pragma unroll
      for (int o = 4; o < kLanes; o *= 2) mx_top = max(mx_top, __shfl_xor_sync(0xffffffffu, mx_top, o));
    }
    float s;
    uint32_t h[4];
    if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
      // (A NaN fails the comparison, keeps scale 1 and becomes a NaN code.)
      const float amax = __uint_as_float(m);
      const HScale hs(amax);
      s = kDivide ? e4m3_scale(amax) : hs.s;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 q = kDivide ? make_float2(__fdiv_rn(f[2 * j], s), __fdiv_rn(f[2 * j + 1], s))
                                 : make_float2(f[2 * j] * hs.up * hs.r, f[2 * j + 1] * hs.up * hs.r);
        h[j] = f16x2_of_e4m3x2(__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3));
      }
    } else if constexpr (kW == MOE_WDTYPE_MXFP4) {
      const uint32_t sb = e8m0_of(m);
      f16_of_e2m1x8(sb == 255u ? 0u : e2m1x8(f, e8m0_rcp(sb)), h);
      // Code x 2^(sb - mx_top + 12); a non-finite block makes the scale NaN.
      const int up = (int)min(sb, mx_top) - (int)mx_top + 12;
      const __half2 r2 = __float2half2_rn(up < -30 ? 0.0f : __uint_as_float((uint32_t)(127 + up) << 23));
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = mul_f16x2(h[j], *reinterpret_cast<const uint32_t*>(&r2));
      s = e8m0_value(mx_top) * 0x1p-12f;
    } else {
      // bf16 values (h is rounded to bf16, as x is) times 2^k, k = 14 - floor(log2(m)); a
      // non-finite or zero block keeps k = 0. 2^k and 2^-k are both normal for eb in [15, 254].
      const uint32_t eb = max(m >> 23, 15u);
      const bool plain = m == 0u || eb == 255u;
      const float r = plain ? 1.0f : __uint_as_float((268u - eb) << 23);
      s = plain ? 1.0f : __uint_as_float((eb - 14u) << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b2 = pack_bf16x2(f[2 * j], f[2 * j + 1]);
        const float2 q = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&b2));
        const __half2 v2 = __floats2half2_rn(q.x * r, q.y * r);
        h[j] = *reinterpret_cast<const uint32_t*>(&v2);
      }
    }
    if (live) *reinterpret_cast<uint4*>(row + x_group<kW>(v) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
    if (live && v % kLanes == 0) reinterpret_cast<float*>(row + scales_at)[v / kLanes] = s;
  }
}

// ------------------------------------------------------------------ router --

// Two experts per CTA: logits [T, E] of all tokens, fp32 sums in a fixed order, a
// thread's loads all issued together. The CTAs after those bring x into the operand
// layout, rows of Smem::pitch(H) bytes. CTA 0 also clears the status record and the
// second kernel's barrier counter.
template <int kW>
__global__ void __launch_bounds__(kRouterThreads) few_router_kernel(const FewParams p) {
  using L = Smem<kW>;
  pdl_wait();
  const int router_ctas = (p.E + kRouterExperts - 1) / kRouterExperts;
  if ((int)blockIdx.x >= router_ctas) {
    const int per_row = p.H / 8, v = ((int)blockIdx.x - router_ctas) * kRouterThreads + threadIdx.x;  // 16 k per row
    const bool live = v < p.T * per_row;
    const uint4 raw = live ? __ldg(reinterpret_cast<const uint4*>(p.x) + v) : make_uint4(0, 0, 0, 0);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&raw);
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 w2 = __bfloat1622float2(b[j]);
      f[2 * j] = w2.x;
      f[2 * j + 1] = w2.y;
    }
    store_operand<kW, true>(p.xrows + v / per_row * L::pitch(p.H), L::scales_at(p.H), v % per_row, f, live);
    return;
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < (int)(kStatusBytes / 4); i += kRouterThreads) p.status[i] = 0;
    if (threadIdx.x == 0) *p.counter = 0;
  }
  __shared__ float part[kRouterThreads / 32][kRouterExperts][kFewMaxTokens];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, nvec = p.H / 8;
  const int e0 = blockIdx.x * kRouterExperts;
  const uint4* w[kRouterExperts];
#pragma unroll
  for (int e = 0; e < kRouterExperts; ++e)
    w[e] = reinterpret_cast<const uint4*>(p.router_w) + (int64_t)min(e0 + e, p.E - 1) * nvec;
  const uint4* x = reinterpret_cast<const uint4*>(p.x);
  float acc[kRouterExperts][kFewMaxTokens];
#pragma unroll
  for (int e = 0; e < kRouterExperts; ++e)
#pragma unroll
    for (int t = 0; t < kFewMaxTokens; ++t) acc[e][t] = 0.0f;
  for (int v0 = threadIdx.x; v0 < nvec; v0 += 2 * kRouterThreads) {
    uint4 wv[2][kRouterExperts], xv[2][kFewMaxTokens];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = v0 + i * kRouterThreads;
      if (v >= nvec) break;
#pragma unroll
      for (int e = 0; e < kRouterExperts; ++e) wv[i][e] = __ldcs(w[e] + v);
#pragma unroll
      for (int t = 0; t < kFewMaxTokens; ++t)
        if (t < p.T) xv[i][t] = __ldg(x + t * nvec + v);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (v0 + i * kRouterThreads >= nvec) break;
#pragma unroll
      for (int t = 0; t < kFewMaxTokens; ++t) {
        if (t >= p.T) break;
        const __nv_bfloat162* xb = reinterpret_cast<const __nv_bfloat162*>(&xv[i][t]);
#pragma unroll
        for (int e = 0; e < kRouterExperts; ++e) {
          const __nv_bfloat162* wb = reinterpret_cast<const __nv_bfloat162*>(&wv[i][e]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = __bfloat1622float2(wb[j]), b = __bfloat1622float2(xb[j]);
            acc[e][t] = fmaf(a.x, b.x, acc[e][t]);
            acc[e][t] = fmaf(a.y, b.y, acc[e][t]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kRouterExperts; ++e) {
#pragma unroll
    for (int t = 0; t < kFewMaxTokens; ++t) {
      if (t >= p.T) break;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) acc[e][t] += __shfl_xor_sync(0xffffffffu, acc[e][t], o);
      if (lane == 0) part[warp][e][t] = acc[e][t];
    }
  }
  __syncthreads();
  const int e = threadIdx.x / kFewMaxTokens, t = threadIdx.x % kFewMaxTokens;
  if (e < kRouterExperts && e0 + e < p.E && t < p.T) {
    float l = 0.0f;
    for (int i = 0; i < kRouterThreads / 32; ++i) l += part[i][e][t];
    if (p.bias) l += p.bias[e0 + e];
    p.logits[t * p.E + e0 + e] = l;
  }
}

// ------------------------------------------------------------- the schedule --

// Quotients by a fixed divisor d: exact for n * d < 2^32.
struct Div {
  uint32_t d, m;
  __device__ __forceinline__ explicit Div(int dd) : d((uint32_t)dd), m(dd > 1 ? 0xffffffffu / (uint32_t)dd + 1u : 0u) {}
  __device__ __forceinline__ int quot(int n) const { return m ? (int)__umulhi((uint32_t)n, m) : n; }
  __device__ __forceinline__ int rem(int n) const { return n - quot(n) * (int)d; }
};

// cp.async.bulk: `bytes` (a multiple of 16) from global to shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The work of a CTA as a sequence of tiles, each a sequence of K slabs; the
// producer and the consumers walk it alike.
struct Tile {
  int u, r0;  // index in the expert list, first feature
};

// Gate/up: the concatenated I-long feature ranges of list entries u0, u0 + 1, ...,
// 8 features to a tile, tiles [pos, end) of them.
struct GateUpWalk {
  int pos, end, u0, per;  // per: tiles of an expert
  __device__ __forceinline__ bool next(Tile& t) {
    if (pos >= end) return false;
    t = tile(pos++);
    return true;
  }
  __device__ __forceinline__ Tile tile(int at) const {
    const int q = Div(per).quot(at);
    return Tile{u0 + q, (at - q * per) * 8};
  }
};

// This CTA's even share of the shared expert, and of the routed ones after it.
__device__ __forceinline__ int share(const FewParams& p, int experts, int cta) {
  return (int)((uint32_t)(experts * (p.I / 8)) * (uint32_t)cta / gridDim.x);  // below 2^31
}
__device__ __forceinline__ GateUpWalk shared_walk(const FewParams& p) {
  return GateUpWalk{share(p, p.S, blockIdx.x), share(p, p.S, blockIdx.x + 1), 0, p.I / 8};
}
__device__ __forceinline__ GateUpWalk routed_walk(const FewParams& p, int U) {
  // The two shares together are even where a CTA has a tile of each expert or more
  // (then no CTA's routed share comes out negative).
  auto at = [&](int cta) {
    return p.I / 8 >= (int)gridDim.x ? share(p, U, cta) - share(p, p.S, cta) : share(p, U - p.S, cta);
  };
  return GateUpWalk{at(blockIdx.x), at(blockIdx.x + 1), p.S, p.I / 8};
}

// Down: this CTA's output rows [r0, r0 + rows), in groups of p.group_rows (a multiple
// of 4, at most 32: two 16-row MMA tiles); every list entry in turn (the shared expert
// last), every group of it, every slab of p.down_lines lines.
struct DownRows {
  int r0, rows, groups, per, slabs, lines;
  __device__ __forceinline__ int first(int group) const { return r0 + per * group; }
  __device__ __forceinline__ int count(int group) const { return min(per, rows - per * group); }
};

__device__ __forceinline__ DownRows down_rows(const FewParams& p, int row_lines) {
  DownRows d;
  d.r0 = (int)blockIdx.x * p.cta_rows;
  d.rows = max(0, min(p.cta_rows, p.H - d.r0));
  d.per = p.group_rows;
  d.groups = (d.rows + d.per - 1) / d.per;
  d.lines = p.down_lines;
  d.slabs = (row_lines + d.lines - 1) / d.lines;
  return d;
}

// List entry of step i of the down phase.
__device__ __forceinline__ int down_entry(int i, int U, int S) { return S == 0 ? i : i + 1 < U ? i + 1 : 0; }

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n) {
    if (++stage == n) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// A producer thread's view of the ring: kScales false: the weight rows, true: their scale bytes.
template <bool kScales>
struct Producer {
  uint8_t* dst;
  uint64_t *full, *empty;
  int n_stages;
  Ring rg;
  uint32_t issued = 0, issued_phase = 0;  // per slot: loaded at all, and the phase of the last load
};

// Loads the K slabs of a tile: a box of rows from row0 and slab_bytes of each to
// `offset` in every slot. One thread and one TMA instruction per stage (it costs the
// thread more than 100 clocks, and at the HBM rate a stage takes about 350): gate and
// up rows, and the scale bytes of each, have threads of their own.
template <int kW, bool kScales>
__device__ __forceinline__ bool load_tile(const FewParams& p, Producer<kScales>& pr, const CUtensorMap* m, int row0,
                                          int offset, int bytes, int slab_bytes, int slabs, bool both,
                                          volatile int* abort_flag) {
  using F = Fmt<kW>;
  constexpr int kSlot = kRows * (kScales ? F::kScaleSlab : F::kSlab);
  for (int k = 0; k < slabs; ++k) {
    const int st = pr.rg.stage;
    if (!mbar_wait(&pr.empty[st], pr.rg.phase ^ 1u, p.status, abort_flag, 0x2001, k, p.wait_ns)) return false;
    uint64_t* bar = &pr.full[st];
    mbar_arrive_expect_tx(bar, (uint32_t)bytes);
    if (both) mbar_arrive(bar);  // nothing comes from the other thread
    uint8_t* dst = pr.dst + st * kSlot + offset;
    if constexpr (kScales) tma_load_2d(dst, m, bar, k * slab_bytes, row0);
    else tma_load_rows(dst, m, bar, row0, k * (slab_bytes / 128));
    pr.issued |= 1u << st;
    pr.issued_phase ^= ((pr.issued_phase >> st ^ pr.rg.phase) & 1u) << st;
    pr.rg.step(pr.n_stages);
  }
  return true;
}

// Everything a producing thread does: kUp false: the gate rows and, after them, the
// down rows; true: the up rows only.
template <int kW, bool kScales, bool kUp>
__device__ __forceinline__ void produce(const FewParams& p, const FewMaps& tm, uint8_t* dst, uint64_t* full,
                                        uint64_t* empty, const int* list, volatile int* n_list, volatile int* abort_flag,
                                        int h_slabs, const DownRows& dr, int lane) {
  constexpr int kBytes = kScales ? Fmt<kW>::kScaleSlab : Fmt<kW>::kSlab;
  Producer<kScales> pr{dst, full, empty, p.n_stages};
  bool ok = p.inject != 1;
  const CUtensorMap* w = kScales ? (kUp ? &tm.s3 : &tm.s1) : (kUp ? &tm.w3 : &tm.w1);
  const CUtensorMap* sw = kScales ? (kUp ? &tm.ss3 : &tm.ss1) : (kUp ? &tm.sw3 : &tm.sw1);
  auto gate_up = [&](GateUpWalk walk) {
    Tile t;
    while (ok && walk.next(t)) {
      const bool sh = p.S && t.u == 0;
      ok = load_tile<kW, kScales>(p, pr, sh ? sw : w, (sh ? 0 : list[t.u]) * p.I + t.r0, kUp ? 8 * kBytes : 0, 8 * kBytes,
                                  kBytes, h_slabs, false, abort_flag);
    }
  };
  if (lane == 0) gate_up(shared_walk(p));  // the shared expert: needs no routing
  __syncwarp();
  named_bar_sync(1, Smem<kW>::kThreads);  // the expert list is ready
  if (lane == 0) {
    const int U = *n_list;
    gate_up(routed_walk(p, U));
    if (!kUp) {
      const CUtensorMap *d = kScales ? &tm.s2 : &tm.w2, *sd = kScales ? &tm.ss2 : &tm.sw2;
      const int slab_bytes = dr.lines * (kScales ? Fmt<kW>::kScaleSlab / (Fmt<kW>::kSlab / kLine) : kLine);
      for (int i = 0; i < U && ok; ++i) {
        const int e = down_entry(i, U, p.S);
        const bool sh = p.S && e == 0;
        const int base = (sh ? 0 : list[e]) * p.H;
        for (int q = 0; q < dr.groups && ok; ++q)
          ok = load_tile<kW, kScales>(p, pr, sh ? sd : d, base + dr.first(q), 0, dr.per * slab_bytes, slab_bytes, dr.slabs,
                                      true, abort_flag);
      }
    }
    // Let every copy land before the thread leaves (the others wait for them too, unless a
    // wait gave up; the slots of the up rows are used again by then).
    for (int s = 0; s < p.n_stages && (!kUp || !ok); ++s) {
      if (!(pr.issued & (1u << s))) continue;
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&full[s], (pr.issued_phase >> s) & 1u) && global_timer_ns() - t0 < 200000000ull) {}
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- the layer --

template <int kW>
__global__ void __launch_bounds__(Smem<kW>::kThreads, 1)
    few_experts_kernel(const FewParams p, const __grid_constant__ FewMaps tm) {
  using F = Fmt<kW>;
  using L = Smem<kW>;
  constexpr int kWarps = L::kWarps, kTeams = L::kTeams, kConsumers = L::kConsumers, kThreads = L::kThreads;
  constexpr bool kScaleBytes = F::kScaleSlab != 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + kMaxRing;
  uint64_t* pfull = empty + kMaxRing;    // a team's partial sums are in its buffers
  uint64_t* pempty = pfull + kTeams;     // ... and have been read
  uint64_t* hfull = pempty + kTeams;     // an expert's rows of h are in shared memory
  uint64_t* hempty = hfull + kHRing;     // ... and have been used by all of its stages
  uint64_t* h_ready = hempty + kHRing;   // every CTA's h is written
  uint64_t* x_ready = h_ready + 1;       // x is in shared memory
  uint64_t* x_done = x_ready + 1;        // ... and has been read for the last time; first[] is complete
  uint64_t* turns = x_done + 1;          // an adding warp's turn to take sums
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
  volatile int* n_list = abort_flag + 1;
  int* top_idx = reinterpret_cast<int*>(smem + L::kTopIdx);
  float* top_w = reinterpret_cast<float*>(smem + L::kTopW);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + L::kBits);
  int* prefix = reinterpret_cast<int*>(bits + 16);
  int* list = reinterpret_cast<int*>(smem + L::kList);
  uint32_t* used = reinterpret_cast<uint32_t*>(smem + L::kUsed);
  int* first = reinterpret_cast<int*>(smem + L::kFirst);
  float* gates = reinterpret_cast<float*>(smem + L::kGate);
  float* red = reinterpret_cast<float*>(smem + L::kRed);
  float* down = reinterpret_cast<float*>(smem + L::kDown);
  uint8_t* act = smem + L::kX;
  const int n_stages = p.n_stages;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = p.S, T = p.T, H = p.H, I = p.I;
  uint8_t* scales = smem + L::scale_offset(T, H, I);
  uint8_t* tiles = smem + L::tile_offset(T, H, I, n_stages);
  const int h_bytes = H * 2 / F::kPer2, i_bytes = I * 2 / F::kPer2;  // bytes of a W1/W3 and a W2 row
  const int h_slabs = (h_bytes + F::kSlab - 1) / F::kSlab;
  const int xpitch = L::pitch(H), hpitch = L::pitch(I);
  const int h_rows = L::act_bytes(T, H, I) / hpitch;  // rows of h that the activations' space holds, T at least
  const DownRows dr = down_rows(p, i_bytes / kLine);

  // (One barrier per thread: a single thread's hundred took 0.6 us.)
  if (warp == 0 && lane < n_stages) {
    mbar_init(&full[lane], kScaleBytes ? 4 : 2);
    mbar_init(&empty[lane], kTeam);
  } else if (warp == 1 && lane < kHRing) {
    mbar_init(&hfull[lane], kPrep);
    mbar_init(&hempty[lane], dr.rows ? dr.groups * dr.slabs * kTeam : 1);
  } else if (warp == 2 && lane < kTeams) {
    mbar_init(&pfull[lane], kTeam);
    mbar_init(&pempty[lane], 1);
  } else if (warp == 3 && lane == 0) {
    mbar_init(h_ready, 1);
    mbar_init(x_ready, 1);
    mbar_init(x_done, kWarps + 1);
    for (int i = 0; i < kAcc; ++i) mbar_init(&turns[i], 1);
    *abort_flag = 0;
  }
  fence_mbar_init();
  // The logits of the selecting warps, while the rest is set up.
  constexpr int kPer = kMaxExperts / 32;
  float logit[kPer];
  if (warp < T) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      logit[i] = i * 32 + lane < p.E ? __ldcg(p.logits + warp * p.E + i * 32 + lane) : 0.0f;
  }
  for (int i = threadIdx.x; i < 16; i += kThreads) bits[i] = 0;
  for (int i = threadIdx.x; i < kMaxU; i += kThreads) used[i] = 0;
  for (int i = threadIdx.x; i < kMaxU * kFewMaxTokens; i += kThreads) gates[i] = 0.0f;
  __syncthreads();

  if (warp == kWarps + kAcc + kPrep) {
    produce<kW, false, false>(p, tm, tiles, full, empty, list, n_list, abort_flag, h_slabs, dr, lane);
    return;
  }
  if (kScaleBytes && warp == kWarps + kAcc + kPrep + 1) {
    produce<kW, true, false>(p, tm, scales, full, empty, list, n_list, abort_flag, h_slabs, dr, lane);
    return;
  }

  // The first of the warps that bring h load the up rows and their scale bytes before.
  constexpr int kUpWarps = kScaleBytes ? 2 : 1;
  constexpr int kPrep0 = kWarps + kAcc;
  if (warp == kPrep0) {
    produce<kW, false, true>(p, tm, tiles, full, empty, list, n_list, abort_flag, h_slabs, dr, lane);
  } else if (kScaleBytes && warp == kPrep0 + 1) {
    produce<kW, true, true>(p, tm, scales, full, empty, list, n_list, abort_flag, h_slabs, dr, lane);
  }
  const int g = lane / 4, c = lane % 4;
  constexpr int kOthers = kConsumers - kUpWarps * 32;  // threads of the selection
  if (warp < kPrep0 || warp >= kPrep0 + kUpWarps) {
    if (threadIdx.x == kConsumers - 32) {  // (a warp without a token to select for)
      mbar_arrive_expect_tx(x_ready, (uint32_t)(T * xpitch));
      bulk_load(act, p.xrows, (uint32_t)(T * xpitch), x_ready);
    }
    if (warp < T) {
      // Top-k of token `warp`: order-preserving integer keys, ties to the lower
      // index, a NaN below everything; a taken expert's key is 0.
      uint32_t key[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = i * 32 + lane;
        key[i] = 0;
        if (e < p.E) {
          const uint32_t b = __float_as_uint(logit[i]);
          key[i] = (b & 0x7fffffffu) > 0x7f800000u ? 1u : ((b >> 31) ? ~b : (b | 0x80000000u));
          if (key[i] == 0x7fffffffu) key[i] = 0x80000000u;  // -0 equals +0
        }
      }
      float w = 0.0f, l0 = 0.0f;
      int mine = 0;
      for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = kPer - 1; i >= 0; --i)
          if (key[i] == best) at = i * 32 + lane;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (at == (uint32_t)(i * 32 + lane)) key[i] = 0;
        const float l = best == 1u ? __uint_as_float(0x7fffffffu)
                                   : __uint_as_float((best >> 31) ? best ^ 0x80000000u : ~best);
        if (j == 0) l0 = l;
        if (lane == j) {
          w = l;
          mine = (int)at;
        }
      }
      // Gates: the chosen logits' softmax.
      const float ex = lane < p.k ? expf(w - l0) : 0.0f;
      float z = ex;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
      if (lane < p.k) {
        const float gate = ex / z;
        top_idx[warp * p.k + lane] = mine;
        top_w[warp * p.k + lane] = gate;
        atomicOr(&bits[mine >> 5], 1u << (mine & 31));
        if (blockIdx.x == 0 && p.topk_idx) {
          p.topk_idx[warp * p.k + lane] = mine;
          p.topk_w[warp * p.k + lane] = gate;
        }
      }
    }
    named_bar_sync(2, kOthers);
    if (warp == 0) {
      // The distinct experts, ascending, after the shared one.
      const uint32_t word = lane < 16 ? bits[lane] : 0u;
      int sum = __popc(word);
      const int own = sum;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      int at = S + sum - own;
      if (lane < 16) prefix[lane] = at;
      for (uint32_t b = word; b; b &= b - 1) list[at++] = lane * 32 + __ffs(b) - 1;
      if (lane == 31) *n_list = S + sum;
      if (S && lane == 0) {
        list[0] = p.E;
        used[0] = (1u << T) - 1u;
      }
      if (S && lane < T) gates[lane] = 1.0f;
    }
    named_bar_sync(2, kOthers);
    for (int i = threadIdx.x; i < T * p.k; i += kConsumers) {
      const int e = top_idx[i], t = i / p.k;
      const int u = prefix[e >> 5] + __popc(bits[e >> 5] & ((1u << (e & 31)) - 1u));
      gates[u * kFewMaxTokens + t] = top_w[i];
      atomicOr(&used[u], 1u << t);
    }
    // The expert list is ready. The producing threads wait for it; the others do not
    // wait for them, whose ring may be full of the shared expert's rows. (The warps that
    // bring h load the up rows and their scale bytes until then.)
    named_bar_sync(2, kOthers);
    named_bar_arrive(1, kThreads);
  }
  const int U = *n_list;

  // Stages are numbered in the producers' order; stage n is in ring slot n % n_stages
  // and belongs to team n % A of kTeam warps, each of which takes every kTeam-th line.
  const int A = min(kTeams, n_stages);
  const GateUpWalk walk0 = shared_walk(p), walk1 = routed_walk(p, U);
  const int tiles0 = walk0.end - walk0.pos;
  const int gu_tiles = tiles0 + walk1.end - walk1.pos, gu_stages = gu_tiles * h_slabs;
  const int per_entry = dr.groups * dr.slabs;  // stages of a list entry in the down phase
  const Div by_h(h_slabs), by_i(dr.slabs), by_entry(per_entry), by_expert(I / 8), by_rows(h_rows);
  const int all_stages = gu_stages + U * per_entry;
  bool ok = true;

  if (warp < kWarps) {
    const int team = warp / kTeam, tw = warp % kTeam;
    // ------------------------------------------------------------ multiply --
    Ring rg, pr;  // this team's next ring slot; phase of its buffers
    auto advance = [&](int n) {
      rg.stage += n;
      while (rg.stage >= n_stages) {
        rg.stage -= n_stages;
        rg.phase ^= 1u;
      }
    };
    advance(team);
    // FP8: a stage's weight scales: lane l < 8 holds that of rows 0..7 (down: of the
    // tile's first row's block) and K block l, lane 8 + l that of rows 8..15 (of its
    // last row's block); fetched a turn ahead.
    auto fetch_scale = [&](int m) {
      if (kW != MOE_WDTYPE_FP8_E4M3 || m >= all_stages || lane >= 16) return 0.0f;
      const int l = lane % 8;
      const float* f;
      int kb;
      if (m < gu_stages) {
        const int tile = by_h.quot(m), at = tile < tiles0 ? walk0.pos + tile : walk1.pos + tile - tiles0;
        const int q = by_expert.quot(at), r0 = 8 * (at - q * (I / 8));
        const bool sh = tile < tiles0;
        kb = (m - tile * h_slabs) * 8 + l;
        if (kb >= H / 128) return 0.0f;
        f = (lane < 8 ? (sh ? p.w.ss1 : p.w.s1) : (sh ? p.w.ss3 : p.w.s3)) +
            ((int64_t)(sh ? 0 : list[S + q]) * (I / 128) + r0 / 128) * (H / 128);
      } else {
        m -= gu_stages;
        const int i = by_entry.quot(m), u = down_entry(i, U, S), q = by_i.quot(m - i * per_entry);
        const bool sh = S && u == 0;
        kb = (m - i * per_entry - q * dr.slabs) * dr.lines + l;
        if (l >= dr.lines || kb >= I / 128) return 0.0f;
        const int row = dr.first(q) + (lane < 8 ? 0 : dr.count(q) - 1);
        f = (sh ? p.w.ss2 : p.w.s2) + ((int64_t)(sh ? 0 : list[u]) * (H / 128) + row / 128) * (I / 128);
      }
      return __ldg(f + kb);
    };
    if (ok) ok = warp_wait<false>(x_ready, 0, p.status, abort_flag, 0x200d, 0, p.wait_ns);
    const uint32_t act_a = smem_u32(act), tiles_a = smem_u32(tiles), scales_a = smem_u32(scales);
    float next_scale = team < A ? fetch_scale(team) : 0.0f;
    bool x_used = true;
    for (int n = team; n < all_stages && team < A; n += A) {
      const float scale = next_scale;
      next_scale = fetch_scale(n + A);
      const bool gate_up = n < gu_stages;
      if (!gate_up && x_used) {
        x_used = false;
        __syncwarp();
        if (lane == 0) mbar_arrive(x_done);
      }
      // The stage's lines, the token rows, and where the weight rows lie: line after line
      // of eight gate rows, and the same of the up rows behind them; or of a group's rows.
      int kl0, lines, entry = 0, group = 0, per = 8;
      uint32_t xa, s0a, s1a;
      if (gate_up) {
        kl0 = by_h.rem(n) * (F::kSlab / kLine);
        lines = min(F::kSlab / kLine, h_bytes / kLine - kl0);
        // Lanes past the last token repeat it; their columns are not used.
        xa = act_a + min(g, T - 1) * xpitch;
        s0a = act_a + min(2 * c, T - 1) * xpitch + L::scales_at(H);
        s1a = act_a + min(2 * c + 1, T - 1) * xpitch + L::scales_at(H);
      } else {
        entry = by_entry.quot(n - gu_stages);
        const int m = n - gu_stages - entry * per_entry, u = down_entry(entry, U, S);
        group = by_i.quot(m);
        kl0 = (m - group * dr.slabs) * dr.lines;
        lines = min(dr.lines, i_bytes / kLine - kl0);
        per = dr.per;
        if (ok)
          ok = warp_wait<false>(&hfull[entry % kHRing], (uint32_t)(entry / kHRing) & 1u, p.status, abort_flag, 0x2005, n,
                                p.wait_ns);
        // Row of a token that uses the expert; the other columns repeat its first row and
        // are not used. (first[] is complete before any entry is.)
        const uint32_t mask = used[u];
        const int row0 = ok ? by_rows.rem(first[entry]) : 0;
        auto row_of = [&](int tok) {
          const int r = row0 + ((mask >> tok) & 1u ? __popc(mask & ((1u << tok) - 1u)) : 0);
          return act_a + (r >= h_rows ? r - h_rows : r) * hpitch;
        };
        xa = row_of(g);
        s0a = row_of(2 * c) + L::scales_at(I);
        s1a = row_of(2 * c + 1) + L::scales_at(I);
      }
      // Per line: bytes of activations, and of their scales.
      constexpr uint32_t kXLine = 128 * F::kPer2, kSLine = F::kBlock ? 64 * F::kPer2 / F::kBlock * 4 : 0;
      constexpr uint32_t kCLine = F::kScaleSlab / (F::kSlab / kLine);
      xa += (kl0 + tw) * kXLine;
      s0a += (kl0 + tw) * kSLine;
      s1a += (kl0 + tw) * kSLine;
      // Stage n's slot held stage n - n_stages before, which another team may not even
      // have seen land: its release is waited for first, or the parity of `full` could
      // be taken for the phase before. (The release before that one is certain: stage
      // n - A was loaded, so every stage up to n - A - n_stages has been released, and
      // A <= n_stages.)
      if (ok) ok = warp_wait<false>(&empty[rg.stage], rg.phase ^ 1u, p.status, abort_flag, 0x2007, n, p.wait_ns);
      if (ok) ok = warp_wait<false>(&full[rg.stage], rg.phase, p.status, abort_flag, 0x2002, n, p.wait_ns);
      // Gate/up: one tile of 8 + 8 rows; down: one or two of 16 rows of the group.
      const uint32_t tile = tiles_a + rg.stage * (kRows * F::kSlab), sc = scales_a + rg.stage * L::kStageScales;
      const int parts = gate_up ? 1 : (dr.count(group) + 15) / 16;
      if (ok) ok = warp_wait<false>(&pempty[team], pr.phase ^ 1u, p.status, abort_flag, 0x2004, n, p.wait_ns);
      // (Loops kept rolled: unrolled, the instruction fetch cost more than it hid.)
#pragma unroll 1
      for (int part = 0; part < parts; ++part) {
        int sel0 = tw, sel1 = 8 + tw;
        Operands o{0, 0, 0, 0, xa, s0a, s1a};
        if (gate_up) {
          o.a0 = tile + g * 128 + tw * (8 * 128);
          o.a1 = o.a0 + 8 * F::kSlab;
          o.c0 = sc + g * F::kScaleSlab + tw * kCLine;
          o.c1 = o.c0 + 8 * F::kScaleSlab;
        } else {
          // (Rows past the group repeat its last one; their sums are not used.)
          const int ra = min(16 * part + g, per - 1), rb = min(16 * part + g + 8, per - 1);
          o.a0 = tile + (ra + tw * per) * 128;
          o.a1 = tile + (rb + tw * per) * 128;
          o.c0 = sc + (ra * dr.lines + tw) * kCLine;
          o.c1 = sc + (rb * dr.lines + tw) * kCLine;
          if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
            const int top = dr.first(group) / 128;
            sel0 = tw + ((dr.first(group) + ra) / 128 != top ? 8 : 0);
            sel1 = tw + ((dr.first(group) + rb) / 128 != top ? 8 : 0);
          }
        }
        const uint32_t step = per * 128 * kTeam;
        Sums acc;
        acc.clear();
        if (ok) {
#pragma unroll 1
          for (int l = tw; l < lines; l += kTeam) {
            float sb0 = 1.0f, sb1 = 1.0f;
            if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
              sb0 = __shfl_sync(0xffffffffu, scale, sel0);
              sb1 = __shfl_sync(0xffffffffu, scale, sel1);
              sel0 += kTeam;
              sel1 += kTeam;
            }
            line_mma<kW>(acc, o, sb0, sb1, lane);
            o.a0 += step;
            o.a1 += step;
            o.c0 += kCLine * kTeam;
            o.c1 += kCLine * kTeam;
            o.x += kXLine * kTeam;
            o.s0 += kSLine * kTeam;
            o.s1 += kSLine * kTeam;
          }
        }
        *reinterpret_cast<float4*>(red + warp * 256 + part * 128 + lane * 4) = acc.total();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&empty[rg.stage]);
        if (!gate_up) mbar_arrive(&hempty[entry % kHRing]);
      }
      advance(A);
      if (lane == 0) mbar_arrive(&pfull[team]);
      pr.phase ^= 1u;
    }
    if (x_used) {
      __syncwarp();
      if (lane == 0) mbar_arrive(x_done);
    }
    return;
  }

  if (warp >= kWarps + kAcc) {
    // ------------------------------------------------------- h for the down phase --
    // The rows of a list entry's tokens lie one after another in the activations'
    // space, entries following entries around it (first[] counts the rows).
    const int me = warp - kWarps - kAcc;
    if (dr.rows == 0) return;  // no rows of the output here
    if (me == kPrep - 1 && lane == 0) {  // (a warp that loads nothing before)
      int rows = 0;
      for (int i = 0; i < U; ++i) {
        first[i] = rows;
        rows += __popc(used[down_entry(i, U, S)]);
      }
      mbar_arrive(x_done);
    }
    // The warps take the rows in turn; a row goes in steps of 96 groups of 8 values,
    // and a step's values are fetched while the step before is stored. A first turn of
    // the loop stores nothing: it brings the loop's instructions near while the weights
    // of the gate/up phase stream (fetched through a busy HBM they took 3 us).
    constexpr int kBatch = 3;
    const int groups = I / 8;
    struct Step {
      int i, u, r, j;  // entry, its list index, row of the entry, first group
      uint32_t mask;   // the entry's tokens from this row on
    };
    auto settle = [&](Step st) {  // from row st.r on to this warp's next row, in whatever entry
      while (true) {
        for (; st.mask; ++st.r, st.mask &= st.mask - 1)
          if ((first[st.i] + st.r) % kPrep == me) return st;
        if (++st.i >= U) return st;
        st.u = down_entry(st.i, U, S);
        st.mask = used[st.u];
        st.r = 0;
      }
    };
    auto after = [&](Step st) {
      if (st.i >= U) return st;
      st.j += 32 * kBatch;
      if (st.j < groups) return st;
      st.j = 0;
      ++st.r;
      st.mask &= st.mask - 1;
      return settle(st);
    };
    struct Values {
      float4 v[2 * kBatch];
    };
    auto fetch = [&](const Step& st) {
      Values o;
      const float4* src = nullptr;
      if (st.i < U)
        src = reinterpret_cast<const float4*>(p.h + ((int64_t)st.u * kFewMaxTokens + __ffs(st.mask) - 1) * I) +
              2 * (st.j + lane);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool live = src && st.j + 32 * k + lane < groups;
        o.v[2 * k] = live ? __ldcg(src + 64 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
        o.v[2 * k + 1] = live ? __ldcg(src + 64 * k + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      return o;
    };
    int freed = 0, told = 0;  // entries whose rows are free again, and that this warp has reported
    auto until_freed = [&](int i) {  // entry i's rows are free again
      for (; ok && freed <= i; ++freed)
        ok = warp_wait<false>(&hempty[freed % kHRing], (uint32_t)(freed / kHRing) & 1u, p.status, abort_flag, 0x200c, i,
                              p.wait_ns);
    };
    bool dry = true;
    Step st{0, 0, 0, 0, 1u};
    Values cur = fetch(st);
#pragma unroll 1
    while (true) {
      if (!dry) {
        // Every entry before this step's has this warp's rows. An entry is reported once the
        // one a ring before it has been used: hfull counts arrivals whoever they come from,
        // and an earlier one would stand for a warp that has yet to report that older entry.
        __syncwarp();
        for (; told < min(st.i, U); ++told) {
          until_freed(told - kHRing);
          if (lane == 0) mbar_arrive(&hfull[told % kHRing]);
        }
        if (st.i >= U) break;
      }
      const Step nx = dry ? st : after(st);
      const Values next = fetch(nx);
      if (!dry && st.j == 0) {
        // Room for the row: first[] counts on from entry to entry, the oldest go first.
        const int end = first[st.i] + st.r + 1;
        while (ok && first[freed] < end - h_rows) until_freed(freed);
      }
      uint8_t* row = act + (dry ? 0 : by_rows.rem(first[st.i] + st.r)) * hpitch;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int g8 = st.j + 32 * k + lane;
        const float f[8] = {cur.v[2 * k].x,     cur.v[2 * k].y,     cur.v[2 * k].z,     cur.v[2 * k].w,
                            cur.v[2 * k + 1].x, cur.v[2 * k + 1].y, cur.v[2 * k + 1].z, cur.v[2 * k + 1].w};
        store_operand<kW, false>(row, L::scales_at(I), g8, f, !dry && g8 < groups);
      }
      if (dry) {
        dry = false;
        if (ok) ok = warp_wait<false>(x_done, 0, p.status, abort_flag, 0x200a, 0, p.wait_ns);
        if (ok) ok = warp_wait<false>(h_ready, 0, p.status, abort_flag, 0x200b, 0, p.wait_ns);
        st.u = down_entry(0, U, S);
        st.mask = used[st.u];
        st = ok ? settle(st) : Step{U, 0, 0, 0, 0u};
        cur = fetch(st);
      } else {
        st = nx;
        cur = next;
      }
    }
    return;
  }

  // ------------------------------------------------------------------ add up --
  // Lane (g, c) holds rows g and g + 8 of tokens 2c, 2c + 1. The warps take the
  // sums of the tiles strictly in turn, so that a buffer's parity is never that of
  // an earlier stage, and finish them side by side.
  const int me = warp - kWarps;
  int n = 0, turn = 0;
  uint32_t turn_phase = 0;
  const Div by_a(A);
  auto take = [&](float (&s)[2][4], int parts) {  // stage n's partial sums
    const int round = by_a.quot(n), w = n - round * A;
    if (ok) ok = warp_wait<false>(&pfull[w], (uint32_t)round & 1u, p.status, abort_flag, 0x2006, n, p.wait_ns);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= parts) break;
#pragma unroll
      for (int k = 0; k < kTeam; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(red + (w * kTeam + k) * 256 + i * 128 + lane * 4);
        s[i][0] += v.x;
        s[i][1] += v.y;
        s[i][2] += v.z;
        s[i][3] += v.w;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&pempty[w]);
    ++n;
  };
  auto begin_turn = [&] {
    if (turn == 0) return;
    if (ok) ok = warp_wait<false>(&turns[me], turn_phase, p.status, abort_flag, 0x2009, n, p.wait_ns);
    turn_phase ^= 1u;
  };
  auto end_turn = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&turns[(me + 1) % kAcc]);
  };
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    GateUpWalk w = part == 0 ? walk0 : walk1;
    Tile t;
    for (; w.next(t); ++turn) {
      if (turn % kAcc != me) {
        n += h_slabs;
        continue;
      }
      begin_turn();
      float both[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      for (int k = 0; k < h_slabs; ++k) take(both, 1);
      end_turn();
      float(&s)[4] = both[0];
      if constexpr (kW == MOE_WDTYPE_NVFP4) {
        const bool sh = S && t.u == 0;
        const int e = sh ? 0 : list[t.u];
        const float f1 = (sh ? p.w.sg1 : p.w.g1)[e], f3 = (sh ? p.w.sg3 : p.w.g3)[e];
        s[0] *= f1;
        s[1] *= f1;
        s[2] *= f3;
        s[3] *= f3;
      }
      const uint32_t mask = used[t.u];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int tok = 2 * c + j;
        if ((mask >> tok) & 1u)
          __stcg(p.h + ((int64_t)t.u * kFewMaxTokens + tok) * I + t.r0 + g, silu_mul(s[j], s[2 + j]));
      }
    }
  }

  // Grid barrier: every h is written.
  named_bar_sync(3, kAcc * 32);
  if (me == 0 && lane == 0) {
    // (The release covers the other threads' stores too: they come before the barrier.)
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.counter) : "memory");
    const uint64_t start = global_timer_ns();
    uint32_t spins = 0;
    while (true) {
      int v;
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p.counter) : "memory");
      if (v >= (int)gridDim.x) break;
      if ((++spins & 63u) == 0 && (*abort_flag || global_timer_ns() - start > p.wait_ns)) {
        if (!*abort_flag) latch_timeout(p.status, 0x2003, v);
        *abort_flag = 1;
        break;
      }
    }
    mbar_arrive(h_ready);
  }

  // Down: one warp adds up, entry by entry; a token without the expert takes nothing
  // from it, whatever its weights hold.
  if (me != turn % kAcc) return;
  begin_turn();
  for (int i = lane; i < dr.groups * 256; i += 32) down[i] = 0.0f;
  __syncwarp();
  for (int i = 0; i < U; ++i) {
    const int u = down_entry(i, U, S);
    const uint32_t mask = used[u];
    float s = 1.0f;
    if constexpr (kW == MOE_WDTYPE_NVFP4) s = (S && u == 0) ? p.w.sg2[0] : p.w.g2[list[u]];
    const float g0 = s * gates[u * kFewMaxTokens + 2 * c], g1 = s * gates[u * kFewMaxTokens + 2 * c + 1];
    for (int q = 0; q < dr.groups; ++q) {
      const int parts = (dr.count(q) + 15) / 16;
      float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      for (int k = 0; k < dr.slabs; ++k) take(d, parts);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part >= parts) break;
        float4* at = reinterpret_cast<float4*>(down + (2 * q + part) * 128 + lane * 4);
        float4 acc = *at;
        if ((mask >> (2 * c)) & 1u) {
          acc.x = fmaf(d[part][0], g0, acc.x);
          acc.z = fmaf(d[part][2], g0, acc.z);
        }
        if ((mask >> (2 * c + 1)) & 1u) {
          acc.y = fmaf(d[part][1], g1, acc.y);
          acc.w = fmaf(d[part][3], g1, acc.w);
        }
        *at = acc;
      }
    }
  }
  if (!ok || *abort_flag) return;
  for (int q = 0; q < dr.groups; ++q) {
    for (int part = 0; 16 * part < dr.count(q); ++part) {
      const float4 acc = *reinterpret_cast<const float4*>(down + (2 * q + part) * 128 + lane * 4);
      const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * part + g + 8 * (j / 2), tok = 2 * c + j % 2;
        if (r < dr.count(q) && tok < T) p.out[(int64_t)tok * H + dr.first(q) + r] = __float2bfloat16_rn(v[j]);
      }
    }
  }
}

template <int kW>
cudaError_t prepare_one() {
  // The limit belongs to the function: the same for every call, or another host thread's
  // smaller one could come between this and the launch.
  const cudaError_t e =
      cudaFuncSetAttribute(few_experts_kernel<kW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  if (e != cudaSuccess) return e;
  // The router CTAs ask for the shared-memory split of the second kernel, whose CTAs
  // could otherwise not start on their SMs before they end.
  return cudaFuncSetAttribute(few_router_kernel<kW>, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

template <int kW>
cudaError_t launch_one(FewParams p, const FewMaps& tm, int sms, cudaStream_t s) {
  auto kern = few_experts_kernel<kW>;
  p.n_stages = Smem<kW>::stages(p.T, p.H, p.I);
  const int smem = Smem<kW>::tile_offset(p.T, p.H, p.I, p.n_stages) + p.n_stages * kRows * Fmt<kW>::kSlab + 1024;
  auto router = few_router_kernel<kW>;
  const unsigned ctas = (unsigned)(ceil_div(p.E, kRouterExperts) + ceil_div((int64_t)p.T * p.H / 8, kRouterThreads));
  const cudaError_t e = launch_pdl(router, dim3(ctas), dim3(kRouterThreads), 0, s, 1, p);
  if (e != cudaSuccess) return e;
  // Cooperative: the CTAs wait for one another, so all of them have to be resident.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(Smem<kW>::kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  // (Programmatic stream serialization has no effect on a cooperative launch; without
  // the latter it starts 3 us earlier, but two calls at once could wait for each other.)
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return counted_launch(cudaLaunchKernelEx(&cfg, kern, p, tm));
}

template <int kW>
bool fits(int T, int H, int I, int sms) {
  // A ring of some stages, and room for the output sums of a CTA's rows.
  const FewRows r = few_rows(kW, H, sms);
  return Smem<kW>::stages(T, H, I) >= 3 && 2 * ceil_div(r.cta, r.group) <= kFewDownTiles;
}

}  // namespace

int64_t few_x_bytes(int wdtype, int T, int H) {
  switch (wdtype) {
    case MOE_WDTYPE_BF16: return (int64_t)T * Smem<MOE_WDTYPE_BF16>::pitch(H);
    case MOE_WDTYPE_FP8_E4M3: return (int64_t)T * Smem<MOE_WDTYPE_FP8_E4M3>::pitch(H);
    case MOE_WDTYPE_NVFP4: return (int64_t)T * Smem<MOE_WDTYPE_NVFP4>::pitch(H);
    default: return (int64_t)T * Smem<MOE_WDTYPE_MXFP4>::pitch(H);
  }
}

bool few_fits(int wdtype, int T, int H, int I, int sms) {
  switch (wdtype) {
    case MOE_WDTYPE_BF16: return fits<MOE_WDTYPE_BF16>(T, H, I, sms);
    case MOE_WDTYPE_FP8_E4M3: return fits<MOE_WDTYPE_FP8_E4M3>(T, H, I, sms);
    case MOE_WDTYPE_NVFP4: return fits<MOE_WDTYPE_NVFP4>(T, H, I, sms);
    default: return fits<MOE_WDTYPE_MXFP4>(T, H, I, sms);
  }
}

cudaError_t prepare_few(int wdtype) {
  switch (wdtype) {
    case MOE_WDTYPE_BF16: return prepare_one<MOE_WDTYPE_BF16>();
    case MOE_WDTYPE_FP8_E4M3: return prepare_one<MOE_WDTYPE_FP8_E4M3>();
    case MOE_WDTYPE_NVFP4: return prepare_one<MOE_WDTYPE_NVFP4>();
    default: return prepare_one<MOE_WDTYPE_MXFP4>();
  }
}

cudaError_t launch_few(const FewParams& p, const FewMaps& tm, int wdtype, int sms, cudaStream_t s) {
  switch (wdtype) {
    case MOE_WDTYPE_BF16: return launch_one<MOE_WDTYPE_BF16>(p, tm, sms, s);
    case MOE_WDTYPE_FP8_E4M3: return launch_one<MOE_WDTYPE_FP8_E4M3>(p, tm, sms, s);
    case MOE_WDTYPE_NVFP4: return launch_one<MOE_WDTYPE_NVFP4>(p, tm, sms, s);
    default: return launch_one<MOE_WDTYPE_MXFP4>(p, tm, sms, s);
  }
}

}  // namespace moe
