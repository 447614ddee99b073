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
//   h        is stored in the form the down products read. FP8 and MXFP4 quantise
//            it: whoever completes a 128- or 32-feature block does that.
//   grid barrier, during which the rings fill with W2.
//   down     each CTA owns H / CTAs output rows for every listed expert and adds
//            the gate-weighted products in registers: no partial output leaves
//            the SM, and the sum's order (experts ascending, the shared one first)
//            does not depend on the other tokens.
//
// One thread streams weight rows by TMA (1 KB of 16 rows a stage: boxes of 128 bytes
// x 8 or 4 rows x 8 lines, 128B-swizzled; row by row bulk copies of 1 KB reached
// 4.1 TB/s, boxes the HBM rate) into a ring; eight warps multiply, each taking every
// eighth 64-byte chunk of the rows, and add up through shared memory once per tile. The shared expert's rows are
// known before the routing is: their copies start before the logits are ready.
// Tensor-core work is mma.sync (m16n8): at 23 weight bytes per clock and SM the
// MMAs are far from a limit, and 8 columns fit 8 tokens without padding.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "few.cuh"
#include "fp4.cuh"
#include "gemm_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;                    // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;    // + the producer warp
constexpr int kRows = 16;                    // rows of a stage
constexpr int kSlab = 1024;                  // bytes of a row in a stage
constexpr int kChunk = 64;                   // bytes of a row that one warp takes at a time
constexpr int kMaxRing = 16;
constexpr int kMaxU = kFewMaxTokens * kMaxTopK + 1;
constexpr int kRouterThreads = 128;

// Per storage: inputs per 2 bytes of a weight row, scale bytes per row and slab
// (4-bit storage), padding of an activation row in shared memory that keeps the
// fragment loads free of bank conflicts, and inputs per activation block (0:
// activations stay bf16).
template <int kW>
struct Fmt;
template <>
struct Fmt<MOE_WDTYPE_BF16> {
  static constexpr int kPer2 = 1, kScaleSlab = 0, kXPad = 64, kBlock = 0;
};
template <>
struct Fmt<MOE_WDTYPE_FP8_E4M3> {
  static constexpr int kPer2 = 2, kScaleSlab = 0, kXPad = 16, kBlock = 128;
};
template <>
struct Fmt<MOE_WDTYPE_NVFP4> {
  static constexpr int kPer2 = 4, kScaleSlab = kSlab / 8, kXPad = 64, kBlock = 0;
};
template <>
struct Fmt<MOE_WDTYPE_MXFP4> {
  static constexpr int kPer2 = 4, kScaleSlab = kSlab / 16, kXPad = 64, kBlock = 32;
};

template <int kW>
struct Smem {
  using F = Fmt<kW>;
  // A stage's scales: 16 rows of scale bytes, or 8 + 8 fp32 block scales.
  static constexpr int kStageScales = kW == MOE_WDTYPE_FP8_E4M3 ? 128 : kRows * F::kScaleSlab;
  static constexpr int kStage = kRows * kSlab + kStageScales;
  // Fixed part: barriers, tables, reduction buffers. Then x, the scales, the tiles.
  static constexpr int kBars = 0;
  static constexpr int kMisc = kBars + 2 * kMaxRing * 8;             // abort flag, list length
  static constexpr int kTopIdx = kMisc + 64;                         // int [8][16]
  static constexpr int kTopW = kTopIdx + kFewMaxTokens * kMaxTopK * 4;
  static constexpr int kBits = kTopW + kFewMaxTokens * kMaxTopK * 4; // uint [16] chosen experts, int [16] prefix
  static constexpr int kList = kBits + 2 * 16 * 4;                   // int [kMaxU] experts
  static constexpr int kUsed = kList + ((kMaxU * 4 + 15) / 16) * 16; // uint [kMaxU] token masks
  static constexpr int kGate = kUsed + ((kMaxU * 4 + 15) / 16) * 16; // float [kMaxU][8]
  static constexpr int kRed = kGate + kMaxU * kFewMaxTokens * 4;     // float [2][kWarps][4][32]
  static constexpr int kX = kRed + 2 * kWarps * 128 * 4;             // activations
  static_assert(kX % 16 == 0, "alignment");
  static __host__ __device__ int x_pitch(int H) { return H * 2 + F::kXPad; }
  static __host__ __device__ int x_scales(int H) { return F::kBlock ? H / F::kBlock : 0; }
  static __host__ __device__ int scale_offset(int T, int H) {
    return (kX + T * x_pitch(H) + T * x_scales(H) * 4 + 127) / 128 * 128;
  }
  static __host__ __device__ int tile_offset(int T, int H, int stages) {
    return (scale_offset(T, H) + stages * kStageScales + 1023) / 1024 * 1024;
  }
  static __host__ __device__ int stages(int T, int H) {
    const int n = (kFewSmem - 2048 - scale_offset(T, H)) / kStage;  // both alignments
    return n > kMaxRing ? kMaxRing : n;
  }
};

// ------------------------------------------------------------------ router --

// One CTA per expert: logits [T, E] of all tokens, fp32 sums in a fixed order.
// CTA 0 also clears the status record and the counters of the second kernel.
__global__ void __launch_bounds__(kRouterThreads) few_router_kernel(const FewParams p) {
  pdl_wait();
  pdl_trigger();  // after the wait: the next kernel may read everything that this one may
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < (int)(kStatusBytes / 4); i += kRouterThreads) p.status[i] = 0;
  }
  const int n_count = p.n_counters;
  for (int i = blockIdx.x * kRouterThreads + threadIdx.x; i < n_count; i += gridDim.x * kRouterThreads) p.counters[i] = 0;
  __shared__ float part[kRouterThreads / 32][kFewMaxTokens];
  const int e = blockIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint4* w = reinterpret_cast<const uint4*>(p.router_w) + (int64_t)e * (p.H / 8);
  float acc[kFewMaxTokens];
#pragma unroll
  for (int t = 0; t < kFewMaxTokens; ++t) acc[t] = 0.0f;
  for (int v = threadIdx.x; v < p.H / 8; v += kRouterThreads) {
    const uint4 wv = __ldg(w + v);
    const __nv_bfloat162* wb = reinterpret_cast<const __nv_bfloat162*>(&wv);
#pragma unroll
    for (int t = 0; t < kFewMaxTokens; ++t) {
      if (t >= p.T) break;
      const uint4 xv = __ldg(reinterpret_cast<const uint4*>(p.x) + (int64_t)t * (p.H / 8) + v);
      const __nv_bfloat162* xb = reinterpret_cast<const __nv_bfloat162*>(&xv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = __bfloat1622float2(wb[i]), b = __bfloat1622float2(xb[i]);
        acc[t] = fmaf(a.x, b.x, acc[t]);
        acc[t] = fmaf(a.y, b.y, acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kFewMaxTokens; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
    if (lane == 0) part[warp][t] = acc[t];
  }
  __syncthreads();
  if (threadIdx.x < p.T) {
    float l = 0.0f;
    for (int i = 0; i < kRouterThreads / 32; ++i) l += part[i][threadIdx.x];
    if (p.bias) l += p.bias[e];
    p.logits[threadIdx.x * p.E + e] = l;
  }
}

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

// Activations are 16-bit operands: bf16 (BF16, NVFP4), or the f16 values of the
// E4M3 and E2M1 codes (exact). Element k of a row sits in place, but for NVFP4:
// within 128 inputs, [word j][lane c][pair r] holds inputs 32 c + 8 j + r and
// + r + 4, the pairs that its expansion of a code word gives.
template <int kW>
__device__ __forceinline__ int x_place(int k) {
  if constexpr (kW == MOE_WDTYPE_NVFP4) {
    const int c = (k >> 5) & 3, j = (k >> 3) & 3, i = k & 7;
    return (k & ~127) + 32 * j + 8 * c + 2 * (i & 3) + (i >> 2);
  } else {
    return k;
  }
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

// E8M0 byte as fp32 (0: 2^-127; 255: infinity, which makes the sums non-finite).
__device__ __forceinline__ float e8m0_weight(uint32_t word, int i) {
  return __uint_as_float(max((word << (24 - 8 * i)) >> 24 << 23, 0x00400000u));
}

// A lane's activation fragment of one chunk: the token's 16 (BF16), 32 (FP8) or
// 64 (4-bit) bytes, and its block scales for tokens 2c and 2c + 1.
template <int kW>
struct XFrag {
  static constexpr int kVecs = kW == MOE_WDTYPE_BF16 ? 1 : kW == MOE_WDTYPE_FP8_E4M3 ? 2 : 4;
  static constexpr int kScales = kW == MOE_WDTYPE_MXFP4 ? 4 : 1;
  uint4 v[kVecs];
  float s0[kScales], s1[kScales];
};

// Byte offset of vector i of lane c's fragment of chunk q in a row of activations.
template <int kW>
__device__ __forceinline__ int frag_offset(int q, int c, int i) {
  if constexpr (kW == MOE_WDTYPE_BF16) return q * 64 + 16 * c;
  if constexpr (kW == MOE_WDTYPE_FP8_E4M3) return q * 128 + 32 * c + 16 * i;
  return q * 256 + 64 * i + 16 * c;
}

// Where a lane's two weight rows (g and g + 8 of the tile) lie in a stage: line l
// at base + l * step, 16-byte unit i of it at ((i ^ x) << 4) for x = (l * step +
// base) / 128 % 8 (the 128-byte swizzle).
struct Rows {
  const uint8_t* tile;     // the stage
  const uint8_t* scales;   // of the stage
  int r0, r1, step;        // offsets of line 0 of the two rows, and from line to line
  __device__ __forceinline__ const uint8_t* at(int row, int line, int unit) const {
    const int o = row + line * step;
    return tile + o + ((unit ^ ((o >> 7) & 7)) << 4);
  }
};

// acc += rows x tokens over one chunk (64 bytes of the stage's 16 rows). FP8:
// sb0, sb1 = weight scales of rows 0..7 and 8..15.
template <int kW>
__device__ __forceinline__ void chunk_mma(float (&acc)[4], const Rows& rows, int q, const XFrag<kW>& x, float sb0,
                                          float sb1, int lane) {
  using F = Fmt<kW>;
  const int g = lane / 4, c = lane % 4;
  const int line = q / 2, unit = (q & 1) * 4;
  if constexpr (kW == MOE_WDTYPE_MXFP4) {
    // Two MMAs per 32-input block (lane c takes the block's word c); the block's
    // sum is weighted by both scales.
    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(rows.scales + g * F::kScaleSlab + q * 4);
    const uint32_t w1 = *reinterpret_cast<const uint32_t*>(rows.scales + (g + 8) * F::kScaleSlab + q * 4);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t va[4], vb[4];
      f16_of_e2m1x8(reinterpret_cast<const uint32_t*>(rows.at(rows.r0, line, unit + b))[c], va);
      f16_of_e2m1x8(reinterpret_cast<const uint32_t*>(rows.at(rows.r1, line, unit + b))[c], vb);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_f16(d, va[0], vb[0], va[1], vb[1], x.v[b].x, x.v[b].y);
      mma_f16(d, va[2], vb[2], va[3], vb[3], x.v[b].z, x.v[b].w);
      const float f0 = e8m0_weight(w0, b), f1 = e8m0_weight(w1, b);
      acc[0] = fmaf(d[0] * x.s0[b], f0, acc[0]);
      acc[1] = fmaf(d[1] * x.s1[b], f0, acc[1]);
      acc[2] = fmaf(d[2] * x.s0[b], f1, acc[2]);
      acc[3] = fmaf(d[3] * x.s1[b], f1, acc[3]);
    }
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(rows.at(rows.r0, line, unit + c));
    const uint4 b = *reinterpret_cast<const uint4*>(rows.at(rows.r1, line, unit + c));
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
    if constexpr (kW == MOE_WDTYPE_BF16) {
      mma_b16(acc, a.x, b.x, a.y, b.y, x.v[0].x, x.v[0].y);
      mma_b16(acc, a.z, b.z, a.w, b.w, x.v[0].z, x.v[0].w);
    } else if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
      const uint32_t xv[8] = {x.v[0].x, x.v[0].y, x.v[0].z, x.v[0].w, x.v[1].x, x.v[1].y, x.v[1].z, x.v[1].w};
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        mma_f16(d, f16x2_of_e4m3x2(aw[j]), f16x2_of_e4m3x2(bw[j]), f16x2_of_e4m3x2(aw[j] >> 16),
                f16x2_of_e4m3x2(bw[j] >> 16), xv[2 * j], xv[2 * j + 1]);
      acc[0] = fmaf(d[0], x.s0[0] * sb0, acc[0]);
      acc[1] = fmaf(d[1], x.s1[0] * sb0, acc[1]);
      acc[2] = fmaf(d[2], x.s0[0] * sb1, acc[2]);
      acc[3] = fmaf(d[3], x.s1[0] * sb1, acc[3]);
    } else {
      // Codes times block scale as bf16, exactly: the code's bits placed in the
      // bf16 exponent and mantissa are code x 2^-126, the scale comes as s x 2^118.
      auto scales = [](const uint8_t* at, uint32_t (&s)[2]) {
        const uint32_t h2 = f16x2_of_e4m3x2(*reinterpret_cast<const uint16_t*>(at));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        s[0] = pack_bf16x2(f.x * 0x1p118f, f.x * 0x1p118f);
        s[1] = pack_bf16x2(f.y * 0x1p118f, f.y * 0x1p118f);
      };
      uint32_t s0[2], s1[2];
      scales(rows.scales + g * F::kScaleSlab + q * 8 + 2 * c, s0);
      scales(rows.scales + (g + 8) * F::kScaleSlab + q * 8 + 2 * c, s1);
      auto expand = [](uint32_t w, int r, uint32_t s) {
        const uint32_t t = w << (12 - 4 * r);
        const uint32_t v = (t & 0x80008000u) | ((t >> 6) & 0x01c001c0u);
        uint32_t o;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(v), "r"(s));
        return o;
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t sa = s0[j / 2], sb = s1[j / 2];
        mma_b16(acc, expand(aw[j], 0, sa), expand(bw[j], 0, sb), expand(aw[j], 1, sa), expand(bw[j], 1, sb), x.v[j].x,
                x.v[j].y);
        mma_b16(acc, expand(aw[j], 2, sa), expand(bw[j], 2, sb), expand(aw[j], 3, sa), expand(bw[j], 3, sb), x.v[j].z,
                x.v[j].w);
      }
    }
  }
}

// ------------------------------------------------------------- the schedule --

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
    t.u = u0 + pos / per;
    t.r0 = pos % per * 8;
    ++pos;
    return true;
  }
};

// This CTA's even share of `experts` experts from list entry u0.
__device__ __forceinline__ GateUpWalk gate_up_walk(const FewParams& p, int u0, int experts) {
  const int per = p.I / 8, total = experts * per;
  return GateUpWalk{(int)((int64_t)total * blockIdx.x / gridDim.x), (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x),
                    u0, per};
}

// Down: output rows [r, end), multiples of 4, up to 16 at a time within a 128-row
// block, every list entry each.
struct DownWalk {
  int r, end;
  __device__ __forceinline__ bool next(int& r0, int& n) {
    if (r >= end) return false;
    r0 = r;
    n = min(min(16, end - r), 128 - r % 128);
    r += n;
    return true;
  }
};

__device__ __forceinline__ DownWalk down_walk(const FewParams& p) {
  const int units = p.H / 4;
  return DownWalk{4 * (int)((int64_t)units * blockIdx.x / gridDim.x),
                  4 * (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x)};
}

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

// Copies the K slabs of a tile of `boxes` boxes of `box_rows` rows each, box b from
// row(b) of map(b); 4-bit storage: their scales from smap(b). FP8: lanes 0..15
// fetch the weight scales of the slab's K blocks from fs0 (rows 0..7) and fs1.
template <int kW, typename Map, typename SMap, typename Row>
__device__ __forceinline__ bool load_tile(const FewParams& p, uint8_t* tiles, uint8_t* scales, uint64_t* full,
                                          uint64_t* empty, Ring& rg, int boxes, int box_rows, Map map, SMap smap, Row row,
                                          const float* fs0, const float* fs1, int row_bytes, int lane,
                                          volatile int* abort_flag, uint32_t& issued, uint32_t& issued_phase) {
  using F = Fmt<kW>;
  using L = Smem<kW>;
  for (int k0 = 0; k0 < row_bytes; k0 += kSlab) {
    if (!warp_wait<false>(&empty[rg.stage], rg.phase ^ 1u, p.status, abort_flag, 0x2001, k0, p.wait_ns)) return false;
    uint8_t* st = tiles + rg.stage * (kRows * kSlab);
    uint8_t* sc = scales + rg.stage * L::kStageScales;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[rg.stage], (uint32_t)(boxes * box_rows * (kSlab + F::kScaleSlab)));
      for (int b = 0; b < boxes; ++b) {
        tma_load_rows(st + b * box_rows * kSlab, map(b), &full[rg.stage], row(b), k0 / 128);
        if (F::kScaleSlab)
          tma_load_2d(sc + b * box_rows * F::kScaleSlab, smap(b), &full[rg.stage], k0 / kSlab * F::kScaleSlab, row(b));
      }
    }
    if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
      // K block k0 / 128 + lane % 8 of rows 0..7 (lanes 0..7) or 8..15 (lanes 8..15).
      if (lane < 16 && k0 + lane % 8 * 128 < row_bytes)
        cp_async_4(sc + lane * 4, (lane < 8 ? fs0 : fs1) + k0 / 128 + lane % 8);
      cp_async_arrive(&full[rg.stage]);
    }
    issued |= 1u << rg.stage;
    issued_phase = (issued_phase & ~(1u << rg.stage)) | (rg.phase << rg.stage);
    rg.step(p.n_stages);
  }
  return true;
}

// ---------------------------------------------------------------- the layer --

template <int kW>
__global__ void __launch_bounds__(kThreads, 1) few_experts_kernel(const FewParams p, const __grid_constant__ FewMaps tm) {
  using F = Fmt<kW>;
  using L = Smem<kW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + kMaxRing;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
  volatile int* n_list = abort_flag + 1;
  int* top_idx = reinterpret_cast<int*>(smem + L::kTopIdx);
  float* top_w = reinterpret_cast<float*>(smem + L::kTopW);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + L::kBits);
  int* prefix = reinterpret_cast<int*>(bits + 16);
  int* list = reinterpret_cast<int*>(smem + L::kList);
  uint32_t* used = reinterpret_cast<uint32_t*>(smem + L::kUsed);
  float* gates = reinterpret_cast<float*>(smem + L::kGate);
  float* red = reinterpret_cast<float*>(smem + L::kRed);
  uint8_t* sx = smem + L::kX;
  float* sxs = reinterpret_cast<float*>(sx + p.T * L::x_pitch(p.H));
  const int n_stages = p.n_stages;
  uint8_t* scales = smem + L::scale_offset(p.T, p.H);
  uint8_t* tiles = smem + L::tile_offset(p.T, p.H, n_stages);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = p.S, T = p.T, H = p.H, I = p.I;
  const int h_bytes = H * 2 / F::kPer2, i_bytes = I * 2 / F::kPer2;  // bytes of a W1/W3 and a W2 row
  const int xp = L::x_pitch(H), xs = L::x_scales(H);

  if (threadIdx.x == 0) {
    for (int i = 0; i < n_stages; ++i) {
      mbar_init(&full[i], kW == MOE_WDTYPE_FP8_E4M3 ? 33 : 1);
      mbar_init(&empty[i], kWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 16; i += kThreads) bits[i] = 0;
  for (int i = threadIdx.x; i < kMaxU; i += kThreads) used[i] = 0;
  for (int i = threadIdx.x; i < kMaxU * kFewMaxTokens; i += kThreads) gates[i] = 0.0f;
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer --
    Ring rg;
    uint32_t issued = 0, issued_phase = 0;
    bool ok = p.inject != 1;
    auto gate_up = [&](GateUpWalk w) {
      Tile t;
      while (ok && w.next(t)) {
        const bool sh = S && t.u == 0;
        const int e = sh ? 0 : list[t.u];
        const int64_t blk = ((int64_t)e * (I / 128) + t.r0 / 128) * (H / 128);
        const float* f0 = kW == MOE_WDTYPE_FP8_E4M3 ? (sh ? p.w.ss1 : p.w.s1) + blk : nullptr;
        const float* f1 = kW == MOE_WDTYPE_FP8_E4M3 ? (sh ? p.w.ss3 : p.w.s3) + blk : nullptr;
        ok = load_tile<kW>(
            p, tiles, scales, full, empty, rg, 2, 8,
            [&](int b) { return b == 0 ? (sh ? &tm.sw1 : &tm.w1) : (sh ? &tm.sw3 : &tm.w3); },
            [&](int b) { return b == 0 ? (sh ? &tm.ss1 : &tm.s1) : (sh ? &tm.ss3 : &tm.s3); },
            [&](int) { return e * I + t.r0; }, f0, f1, h_bytes, lane, abort_flag, issued, issued_phase);
      }
    };
    gate_up(gate_up_walk(p, 0, S));  // the shared expert: needs no routing
    named_bar_sync(1, kThreads);     // the expert list is ready
    const int U = *n_list;
    gate_up(gate_up_walk(p, S, U - S));
    DownWalk dw = down_walk(p);
    int r0, n;
    while (ok && dw.next(r0, n)) {
      for (int u = 0; u < U && ok; ++u) {
        const bool sh = S && u == 0;
        const int e = sh ? 0 : list[u];
        const float* f = kW == MOE_WDTYPE_FP8_E4M3
                             ? (sh ? p.w.ss2 : p.w.s2) + ((int64_t)e * (H / 128) + r0 / 128) * (I / 128)
                             : nullptr;
        ok = load_tile<kW>(
            p, tiles, scales, full, empty, rg, n / 4, 4, [&](int) { return sh ? &tm.sw2 : &tm.w2; },
            [&](int) { return sh ? &tm.ss2 : &tm.s2; }, [&](int b) { return e * H + r0 + 4 * b; }, f, f, i_bytes, lane,
            abort_flag, issued, issued_phase);
      }
    }
    if (kW == MOE_WDTYPE_FP8_E4M3) asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) {
      // Let every copy land before the warp leaves (the consumers wait for them too, unless a wait gave up).
      for (int s = 0; s < n_stages; ++s) {
        if (!(issued & (1u << s))) continue;
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&full[s], (issued_phase >> s) & 1u) && global_timer_ns() - t0 < 200000000ull) {}
      }
    }
    return;
  }

  // ------------------------------------------------------------- consumers --
  const int g = lane / 4, c = lane % 4;
  // Activations into shared memory, in the operand layout. (x was complete
  // before the router kernel passed its own wait.)
  for (int t = 0; t < T; ++t) {
    const uint4* xr = reinterpret_cast<const uint4*>(p.x) + (int64_t)t * (H / 8);
    for (int v = threadIdx.x; v < H / 8; v += kConsumers) {  // H a multiple of 128: whole half-warps
      const uint4 raw = __ldg(xr + v);
      if constexpr (kW == MOE_WDTYPE_BF16) {
        *reinterpret_cast<uint4*>(sx + t * xp + v * 16) = raw;
      } else if constexpr (kW == MOE_WDTYPE_NVFP4) {
        const uint16_t* e = reinterpret_cast<const uint16_t*>(&raw);
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<uint16_t*>(sx + t * xp + 2 * x_place<kW>(v * 8 + i)) = e[i];
      } else {
        const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&raw);
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 w2 = __bfloat1622float2(b[i]);
          f[2 * i] = w2.x;
          f[2 * i + 1] = w2.y;
        }
        const uint32_t act = H / 8 - (v - lane) >= 32 ? 0xffffffffu : 0xffffu;  // H/8 is a multiple of 16
        uint32_t m = amax_bits<8>(f);
        constexpr int kLanes = F::kBlock / 8;  // 16 (FP8) or 4 (MXFP4) lanes share a block
#pragma unroll
        for (int o = 1; o < kLanes; o *= 2) m = max(m, __shfl_xor_sync(act, m, o));
        if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
          const float amax = __uint_as_float(m);
          const float s = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[2 * i], s), __fdiv_rn(f[2 * i + 1], s)),
                                            __NV_SATFINITE, __NV_E4M3);
          *reinterpret_cast<uint4*>(sx + t * xp + v * 16) = make_uint4(f16x2_of_e4m3x2(w[0]), f16x2_of_e4m3x2(w[1]),
                                                                       f16x2_of_e4m3x2(w[2]), f16x2_of_e4m3x2(w[3]));
          if (v % kLanes == 0) sxs[t * xs + v / kLanes] = s;
        } else {
          const uint32_t sb = e8m0_of(m);
          uint32_t h[4];
          f16_of_e2m1x8(sb == 255u ? 0u : e2m1x8(f, e8m0_rcp(sb)), h);
          *reinterpret_cast<uint4*>(sx + t * xp + v * 16) = make_uint4(h[0], h[1], h[2], h[3]);
          if (v % kLanes == 0) sxs[t * xs + v / kLanes] = e8m0_value(sb);
        }
      }
    }
  }

  pdl_wait();  // the logits, the cleared counters
  if (warp < T) {
    // Top-k of token `warp`: order-preserving integer keys, ties to the lower
    // index, a NaN below everything; a taken expert's key is 0.
    constexpr int kPer = kMaxExperts / 32;
    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 32 + lane;
      key[i] = 0;
      if (e < p.E) {
        const uint32_t b = __float_as_uint(__ldcg(p.logits + warp * p.E + e));
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
      const float l = __ldcg(p.logits + warp * p.E + at);
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
  named_bar_sync(2, kConsumers);
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
  named_bar_sync(2, kConsumers);
  for (int i = threadIdx.x; i < T * p.k; i += kConsumers) {
    const int e = top_idx[i], t = i / p.k;
    const int u = prefix[e >> 5] + __popc(bits[e >> 5] & ((1u << (e & 31)) - 1u));
    gates[u * kFewMaxTokens + t] = top_w[i];
    atomicOr(&used[u], 1u << t);
  }
  // The expert list is ready. The producer waits for it here; the consumers do not
  // wait for the producer, whose ring may be full of the shared expert's rows.
  named_bar_arrive(1, kThreads);
  named_bar_sync(2, kConsumers);
  const int U = *n_list;

  Ring rg;
  bool ok = true;
  uint32_t buf = 0;
  auto wait_full = [&] {
    if (ok) ok = warp_wait<false>(&full[rg.stage], rg.phase, p.status, abort_flag, 0x2002, (int)buf, p.wait_ns);
    return ok;
  };
  auto release = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[rg.stage]);
    rg.step(n_stages);
  };
  const int xt = min(g, T - 1);  // lanes past the last token repeat it; their columns are not used
  const int t0 = min(2 * c, T - 1), t1 = min(2 * c + 1, T - 1);

  // ---- gate/up ----
  auto gate_up = [&](GateUpWalk w) {
    Tile t;
    while (w.next(t)) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k0 = 0; k0 < h_bytes; k0 += kSlab) {
        const int chunks = min(kSlab, h_bytes - k0) / kChunk;
        if (wait_full()) {
          const Rows rows{tiles + rg.stage * (kRows * kSlab), scales + rg.stage * L::kStageScales, g * 128,
                          8 * kSlab + g * 128, 8 * 128};
          for (int q = warp; q < chunks; q += kWarps) {
            const int kq = k0 / kChunk + q;
            XFrag<kW> x;
#pragma unroll
            for (int i = 0; i < XFrag<kW>::kVecs; ++i)
              x.v[i] = *reinterpret_cast<const uint4*>(sx + xt * xp + frag_offset<kW>(kq, c, i));
            float sb0 = 1.0f, sb1 = 1.0f;
            if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
              x.s0[0] = sxs[t0 * xs + kq / 2];
              x.s1[0] = sxs[t1 * xs + kq / 2];
              const float* fs = reinterpret_cast<const float*>(rows.scales);
              sb0 = fs[q / 2];
              sb1 = fs[8 + q / 2];
            } else if constexpr (kW == MOE_WDTYPE_MXFP4) {
              *reinterpret_cast<float4*>(x.s0) = *reinterpret_cast<const float4*>(sxs + t0 * xs + kq * 4);
              *reinterpret_cast<float4*>(x.s1) = *reinterpret_cast<const float4*>(sxs + t1 * xs + kq * 4);
            }
            chunk_mma<kW>(acc, rows, q, x, sb0, sb1, lane);
          }
        }
        release();
      }
      float* part = red + (buf & 1u) * (kWarps * 128);
      *reinterpret_cast<float4*>(part + warp * 128 + lane * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      named_bar_sync(2, kConsumers);
      // One warp finishes the tile (each in turn): lane (g, c) sums feature g of tokens 2c, 2c + 1.
      if (warp == (int)(buf % kWarps)) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(part + i * 128 + lane * 4);
          s[0] += v.x;
          s[1] += v.y;
          s[2] += v.z;
          s[3] += v.w;
        }
        if constexpr (kW == MOE_WDTYPE_NVFP4) {
          const bool sh = S && t.u == 0;
          const int e = sh ? 0 : list[t.u];
          const float f1 = (sh ? p.w.sg1 : p.w.g1)[e] * 256.0f, f3 = (sh ? p.w.sg3 : p.w.g3)[e] * 256.0f;
          s[0] *= f1;
          s[1] *= f1;
          s[2] *= f3;
          s[3] *= f3;
        }
        const uint32_t mask = used[t.u];
        const int f = t.r0 + g;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int tok = 2 * c + j;
          if ((mask >> tok) & 1u) {
            const float h = silu_mul(s[j], s[2 + j]);
            const int64_t row = (int64_t)t.u * kFewMaxTokens + tok;
            if constexpr (F::kBlock == 0)
              p.hq[row * I + x_place<kW>(f)] = __bfloat16_as_ushort(__float2bfloat16_rn(h));
            else
              __stcg(p.h + row * I + f, h);
          }
        }
        if constexpr (F::kBlock != 0) {
          // Whoever completes a block quantises it for the tokens that use it.
          __syncwarp();
          const int b = t.r0 / F::kBlock;
          int old = 0;
          if (lane == 0) {
            __threadfence();
            old = atomicAdd(&p.counters[1 + t.u * (I / F::kBlock) + b], 8);
          }
          old = __shfl_sync(0xffffffffu, old, 0);
          if (old + 8 == F::kBlock) {
            __threadfence();
            for (uint32_t mm = mask; mm; mm &= mm - 1) {
              const int64_t row = (int64_t)t.u * kFewMaxTokens + __ffs(mm) - 1;
              if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p.h + row * I + b * 128) + lane);
                float amax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
                uint32_t nan = (isnan(v.x) || isnan(v.y) || isnan(v.z) || isnan(v.w)) ? 1u : 0u;
#pragma unroll
                for (int o = 16; o > 0; o /= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                nan = __any_sync(0xffffffffu, nan);
                const float sc = nan ? __uint_as_float(0x7fffffffu) : amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
                const float inv = amax > 0.0f ? __frcp_rn(sc) : 0.0f;
                const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v.x * inv, v.y * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t d = __nv_cvt_float2_to_fp8x2(make_float2(v.z * inv, v.w * inv), __NV_SATFINITE, __NV_E4M3);
                reinterpret_cast<uint2*>(p.hq + row * I + b * 128)[lane] =
                    make_uint2(f16x2_of_e4m3x2(a), f16x2_of_e4m3x2(d));
                if (lane == 0) p.hs[row * (I / 128) + b] = sc;
              } else {
                // Four lanes, 8 features each.
                float v[8];
                if (lane < 4) {
                  *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(p.h + row * I + b * 32) + 2 * lane);
                  *reinterpret_cast<float4*>(v + 4) =
                      __ldcg(reinterpret_cast<const float4*>(p.h + row * I + b * 32) + 2 * lane + 1);
                }
                uint32_t m = lane < 4 ? amax_bits<8>(v) : 0u;
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t sb = e8m0_of(m);
                if (lane < 4) {
                  uint32_t hv[4];
                  f16_of_e2m1x8(sb == 255u ? 0u : e2m1x8(v, e8m0_rcp(sb)), hv);
                  *reinterpret_cast<uint4*>(p.hq + row * I + b * 32 + lane * 8) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
                  if (lane == 0) p.hs[row * (I / 32) + b] = e8m0_value(sb);
                }
              }
            }
          }
        }
      }
      ++buf;
    }
  };
  gate_up(gate_up_walk(p, 0, S));
  gate_up(gate_up_walk(p, S, U - S));

  // ---- grid barrier: every h is written ----
  __threadfence();
  named_bar_sync(2, kConsumers);
  if (threadIdx.x == 0) {
    atomicAdd(&p.counters[0], 1);
    const uint64_t start = global_timer_ns();
    uint32_t spins = 0;
    while (true) {
      int v;
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p.counters) : "memory");
      if (v >= (int)gridDim.x) break;
      if ((++spins & 63u) == 0 && (*abort_flag || global_timer_ns() - start > p.wait_ns)) {
        if (!*abort_flag) latch_timeout(p.status, 0x2003, v);
        *abort_flag = 1;
        break;
      }
    }
    __threadfence();
  }
  named_bar_sync(2, kConsumers);

  // ---- down ----
  DownWalk dw = down_walk(p);
  int r0, n;
  while (dw.next(r0, n)) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int u = 0; u < U; ++u) {
      const uint32_t mask = used[u];
      const float g0 = gates[u * kFewMaxTokens + 2 * c], g1 = gates[u * kFewMaxTokens + 2 * c + 1];
      const bool on = (mask >> g) & 1u, on0 = (mask >> (2 * c)) & 1u, on1 = (mask >> (2 * c + 1)) & 1u;
      const int64_t row = (int64_t)u * kFewMaxTokens;
      const uint8_t* hrow = reinterpret_cast<const uint8_t*>(p.hq + (row + g) * I);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k0 = 0; k0 < i_bytes; k0 += kSlab) {
        const int chunks = min(kSlab, i_bytes - k0) / kChunk;
        constexpr int kPer = kSlab / kChunk / kWarps;
        // This stage's activations, before the wait for its weights.
        XFrag<kW> x[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int q = warp + j * kWarps, kq = k0 / kChunk + q;
          const bool live = q < chunks;
#pragma unroll
          for (int i = 0; i < XFrag<kW>::kVecs; ++i)
            x[j].v[i] = live && on ? __ldcg(reinterpret_cast<const uint4*>(hrow + frag_offset<kW>(kq, c, i)))
                                   : make_uint4(0, 0, 0, 0);
          if constexpr (kW == MOE_WDTYPE_FP8_E4M3) {
            x[j].s0[0] = live && on0 ? __ldcg(p.hs + (row + 2 * c) * (I / 128) + kq / 2) : 0.0f;
            x[j].s1[0] = live && on1 ? __ldcg(p.hs + (row + 2 * c + 1) * (I / 128) + kq / 2) : 0.0f;
          } else if constexpr (kW == MOE_WDTYPE_MXFP4) {
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(x[j].s0) =
                live && on0 ? __ldcg(reinterpret_cast<const float4*>(p.hs + (row + 2 * c) * (I / 32) + kq * 4)) : z;
            *reinterpret_cast<float4*>(x[j].s1) =
                live && on1 ? __ldcg(reinterpret_cast<const float4*>(p.hs + (row + 2 * c + 1) * (I / 32) + kq * 4)) : z;
          }
        }
        if (wait_full()) {
          // Boxes of four rows.
          const int r = (g / 4) * 4 * kSlab + (g % 4) * 128;
          const Rows rows{tiles + rg.stage * (kRows * kSlab), scales + rg.stage * L::kStageScales, r, r + 8 * kSlab,
                          4 * 128};
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int q = warp + j * kWarps;
            if (q >= chunks) break;
            float sb = 1.0f;
            if constexpr (kW == MOE_WDTYPE_FP8_E4M3)
              sb = reinterpret_cast<const float*>(rows.scales)[q / 2];
            chunk_mma<kW>(d, rows, q, x[j], sb, sb, lane);
          }
        }
        release();
      }
      float s = 1.0f;
      if constexpr (kW == MOE_WDTYPE_NVFP4) s = ((S && u == 0) ? p.w.sg2[0] : p.w.g2[list[u]]) * 256.0f;
      // A token without this expert takes nothing from it, whatever its weights hold.
      if (on0) {
        acc[0] = fmaf(d[0], s * g0, acc[0]);
        acc[2] = fmaf(d[2], s * g0, acc[2]);
      }
      if (on1) {
        acc[1] = fmaf(d[1], s * g1, acc[1]);
        acc[3] = fmaf(d[3], s * g1, acc[3]);
      }
    }
    float* part = red + (buf & 1u) * (kWarps * 128);
    *reinterpret_cast<float4*>(part + warp * 128 + lane * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    named_bar_sync(2, kConsumers);
    if (warp == (int)(buf % kWarps) && ok) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(part + i * 128 + lane * 4);
        s[0] += v.x;
        s[1] += v.y;
        s[2] += v.z;
        s[3] += v.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = g + 8 * (j / 2), tok = 2 * c + j % 2;
        if (r < n && tok < T) p.out[(int64_t)tok * H + r0 + r] = __float2bfloat16_rn(s[j]);
      }
    }
    ++buf;
  }
}

template <int kW>
cudaError_t launch_one(FewParams p, const FewMaps& tm, int sms, cudaStream_t s) {
  auto kern = few_experts_kernel<kW>;
  p.n_stages = Smem<kW>::stages(p.T, p.H);
  const int smem = Smem<kW>::tile_offset(p.T, p.H, p.n_stages) + p.n_stages * kRows * kSlab + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(few_router_kernel, dim3((unsigned)p.E), dim3(kRouterThreads), 0, s, 1, p);
  if (e != cudaSuccess) return e;
  // Cooperative: the CTAs wait for one another, so all of them have to be resident.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return counted_launch(cudaLaunchKernelEx(&cfg, kern, p, tm));
}

template <int kW>
bool fits(int T, int H) {
  return Smem<kW>::stages(T, H) >= 3;
}

}  // namespace

bool few_fits(int wdtype, int T, int H) {
  switch (wdtype) {
    case MOE_WDTYPE_BF16: return fits<MOE_WDTYPE_BF16>(T, H);
    case MOE_WDTYPE_FP8_E4M3: return fits<MOE_WDTYPE_FP8_E4M3>(T, H);
    case MOE_WDTYPE_NVFP4: return fits<MOE_WDTYPE_NVFP4>(T, H);
    default: return fits<MOE_WDTYPE_MXFP4>(T, H);
  }
}

int few_counters(int wdtype, int T, int k, int S, int I) {
  const int block = wdtype == MOE_WDTYPE_FP8_E4M3 ? 128 : wdtype == MOE_WDTYPE_MXFP4 ? 32 : 0;
  return 1 + (block ? (T * k + S) * (I / block) : 0);
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
