// Grouped expert GEMMs on MXFP4 storage: E2M1 weights and activations, one E8M0
// scale per 32 inputs on both sides, multiplied by the block-scaled tensor core
// (tcgen05.mma kind::mxf4: 64 inputs per instruction, the products of a 32-input
// block weighted by both blocks' scales, fp32 sums in TMEM).
//
//   GEMM1 (gate/up + SwiGLU): h[r, j] = silu(A[r] . W1_g[j]) * (A[r] . W3_g[j]),
//     quantised to MXFP4 in the epilogue (a thread owns whole 32-column blocks of
//     its row, so the block maximum needs no exchange).
//   GEMM2 (down): y[r, c] = gate[r] * (h[r] . W2_g[c]), stored bf16.
//
// Tile: 128 rows x 256 columns (GEMM1: 128 gate and the matching 128 up columns
// side by side), K stages of 256 inputs (128 bytes). Operand tiles come by TMA
// (128B swizzle) and so do the scales, as row-major 16-byte boxes that cover two
// stages. The tensor core reads scales from TMEM, four bytes (128 inputs) per
// 32-bit column, row r in lane r % 32 and column r / 32, repeated in the four
// lane quarters; four scale warps write that layout (24 columns a stage: 8 for A,
// 16 for B).
//
// TMEM: the two accumulator buffers of 256 columns overlap by 96 columns
// (0..255 and 160..415), which leaves 96 columns for the scales of the four
// stages. The epilogue reads a buffer's shared columns first and then lets the
// next tile's MMAs begin.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2..5 scale writers, 6..13 epilogue.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp4.cuh"
#include "gemm_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kStages = 4;
constexpr int kScaleWarps = 4;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * (kScaleWarps + kEpiWarps);
constexpr int kStageK = 256;                       // inputs per stage
constexpr int kABytes = kTileM * kStageBytesK;     // 16 KB
constexpr int kBBytes = 256 * kStageBytesK;        // 32 KB
constexpr int kScBuf = (kTileM + 256) * 16;        // scales of two stages: 128 A rows, 256 B rows
constexpr int kScBufs = kStages / 2;
constexpr int kMaxGroups = kMaxExperts + 1;
constexpr uint32_t kAccStep = 160;                 // column offset of the second accumulator buffer
constexpr uint32_t kSfCol = 416;                   // first scale column
constexpr uint32_t kSfCols = 24;                   // scale columns per stage

constexpr size_t kOffB = (size_t)kStages * kABytes;
constexpr size_t kOffSc = kOffB + (size_t)kStages * kBBytes;
constexpr size_t kOffBars = kOffSc + (size_t)kScBufs * kScBuf;
constexpr int kNumBars = 3 * kStages + 2 + 1 + 1;
constexpr size_t kOffMisc = kOffBars + ((kNumBars * 8 + 127) / 128) * 128;
constexpr size_t kOffMt = kOffMisc + 64;
constexpr size_t kOffOff = kOffMt + (kMaxGroups + 1) * 4;
constexpr size_t kDynamic = kOffOff + (kMaxGroups + 1) * 4 + 1024;
static_assert(kDynamic <= 227 * 1024, "shared memory budget");
static_assert(kSfCol + kStages * kSfCols <= 512, "TMEM columns");

// Instruction descriptor of kind::mxf4: E2M1 operands (K-major), E8M0 scales,
// M x N; sf = which half of a scale column's four bytes this instruction's 64
// inputs use (0 or 2).
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) |
         (sf << 29);
}

__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <bool kGemm1>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_gemm_kernel(const GemmParams p, const __grid_constant__ AMaps tm_a, const __grid_constant__ MxMaps tm) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kOffB;
  uint8_t* sSc = smem + kOffSc;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBars);  // operands (and scales) landed
  uint64_t* empty = full + kStages;                               // the stage's MMAs completed
  uint64_t* sfull = empty + kStages;                              // the stage's scales are in TMEM
  uint64_t* tfull = sfull + kStages;                              // accumulator buffer complete
  uint64_t* tempty = tfull + 2;                                   // the overlap has been read
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_mt = reinterpret_cast<int*>(smem + kOffMt);
  int* s_off = reinterpret_cast<int*>(smem + kOffOff);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], kScaleWarps);
    }
    for (int b = 0; b < 2; ++b) mbar_init(&tfull[b], 1);
    mbar_init(tempty, kEpiWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a.rows128);
    tma_prefetch_desc(&tm_a.rows64);
    tma_prefetch_desc(&tm_a.rows32);
    tma_prefetch_desc(&tm.code0);
    tma_prefetch_desc(&tm.a_scale);
    tma_prefetch_desc(&tm.scale0);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i <= p.G; i += kThreads) {
    s_mt[i] = p.mt_prefix[i];
    s_off[i] = p.offsets[i];
  }
  __syncthreads();
  const int total = s_mt[p.G] * p.n_tiles;
  const int kstages = p.K / kStageK;  // even
  const int site0 = 0x1000 | (kGemm1 ? 0x200 : 0);
  auto item_of = [&](int item) {
    return decode_item(item, p.n_tiles, p.G, kTileM, s_mt, s_off, p.n_fastest != 0);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer --
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_phase = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < total && ok && p.inject != 1; item += gridDim.x) {
        const Item it = item_of(item);
        const bool shared = it.g == p.E;
        const int yb = (shared ? 0 : it.g * p.N) + it.n * (kGemm1 ? 128 : 256);
        const CUtensorMap* c0 = shared ? &tm.scode0 : &tm.code0;
        const CUtensorMap* c1 = shared ? &tm.scode1 : &tm.code1;
        const CUtensorMap* f0 = shared ? &tm.sscale0 : &tm.scale0;
        const CUtensorMap* f1 = shared ? &tm.sscale1 : &tm.scale1;
        const int rows = it.end - it.row0;
        const int a_rows = rows <= 32 ? 32 : (rows <= 64 ? 64 : 128);
        const CUtensorMap* amap = a_rows == 32 ? &tm_a.rows32 : (a_rows == 64 ? &tm_a.rows64 : &tm_a.rows128);
        for (int ks = 0; ks < kstages; ++ks) {
          if (!mbar_wait(&empty[stage], phase ^ 1, p.status, abort_flag, site0 | 1, item, p.wait_ns)) {
            ok = false;
            break;
          }
          const bool even = (ks & 1) == 0;
          mbar_arrive_expect_tx(&full[stage], (uint32_t)(a_rows * kStageBytesK + kBBytes + (even ? kScBuf : 0)));
          if (even) {
            // Both stages' scales; the buffer's previous pair was read when its even stage was.
            uint8_t* sc = sSc + (stage / 2) * kScBuf;
            const int kx = ks * (kStageK / 32);
            tma_load_2d(sc, &tm.a_scale, &full[stage], kx, it.row0);
            tma_load_2d(sc + kTileM * 16, f0, &full[stage], kx, yb);
            if (kGemm1) tma_load_2d(sc + 2 * kTileM * 16, f1, &full[stage], kx, yb);
          }
          const int kx = ks * kStageBytesK;
          tma_load_2d(sA + stage * kABytes, amap, &full[stage], kx, it.row0);
          tma_load_2d(sB + stage * kBBytes, c0, &full[stage], kx, yb);
          if (kGemm1) tma_load_2d(sB + stage * kBBytes + kBBytes / 2, c1, &full[stage], kx, yb);
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        // Let the tensor copies already in flight land before the CTA leaves.
        for (int s = 0; s < kStages; ++s) {
          if (!(issued & (1u << s))) continue;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(&full[s], (issued_phase >> s) & 1u) && global_timer_ns() - t0 < 200000000ull) {}
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer --
    if (lane == 0) {
      constexpr uint32_t kId0 = idesc_mx(kTileM, 256, 0), kId2 = idesc_mx(kTileM, 256, 2);
      int stage = 0;
      uint32_t phase = 0, tile = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < total && ok; item += gridDim.x, ++tile) {
        const uint32_t b = tile & 1u;
        // The previous tile's overlap (and so all of the tile before it) has been read.
        if (!mbar_wait(tempty, (tile & 1u) ^ 1u, p.status, abort_flag, site0 | 3, (int)tile, p.wait_ns)) break;
        tc_fence_after_sync();
        const uint32_t d = tmem + b * kAccStep;
        for (int ks = 0; ks < kstages; ++ks) {
          if (!mbar_wait(&full[stage], phase, p.status, abort_flag, site0 | 4, (int)tile, p.wait_ns) ||
              !mbar_wait(&sfull[stage], phase, p.status, abort_flag, site0 | 5, (int)tile, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t ad = sdesc_k_sw128(sA + stage * kABytes);
          const uint64_t bd = sdesc_k_sw128(sB + stage * kBBytes);
          const uint32_t sf = tmem + kSfCol + stage * kSfCols;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_mx(d, ad + 2 * kk, bd + 2 * kk, (kk & 1) ? kId2 : kId0, sf + 4 * (kk / 2), sf + 8 + 8 * (kk / 2),
                   (ks || kk) ? 1u : 0u);
          mma_commit(&empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (ok) mma_commit(&tfull[b]);
      }
      mma_commit(drain);  // every MMA issued so far has completed once this arrives
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < 200000000ull) {}
    }
  } else if (warp < 2 + kScaleWarps) {
    // -------------------------------------------------------- scale writers --
    // Lane l holds rows l, l + 32, ... of both operands: 12 rows x 16 bytes, the
    // first 8 bytes for the even stage, the others kept for the odd one.
    const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
      for (int ks = 0; ks < kstages && ok; ks += 2) {
        if (!warp_wait<false>(&full[stage], phase, p.status, abort_flag, site0 | 6, item, p.wait_ns)) {
          ok = false;
          break;
        }
        uint4 sc[12];
        const uint4* src = reinterpret_cast<const uint4*>(sSc + (stage / 2) * kScBuf) + lane;
#pragma unroll
        for (int i = 0; i < 12; ++i) sc[i] = src[32 * i];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // The stage's scale columns are free once the MMAs of its previous use completed.
          if (!warp_wait<false>(&empty[stage], phase ^ 1, p.status, abort_flag, site0 | 7, item, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t col = tmem + lane_base + kSfCol + stage * kSfCols;
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = half ? sc[i].z : sc[i].x;
            v[4 + i] = half ? sc[i].w : sc[i].y;
          }
          tmem_st8(col, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = half ? sc[4 + i].z : sc[4 + i].x;
          tmem_st8(col + 8, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = half ? sc[4 + i].w : sc[4 + i].y;
          tmem_st8(col + 16, v);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue --
    const int q = warp % 4;                 // TMEM lane quarter
    const int hf = (warp - 6) / 4;          // half of the tile's columns
    const int rl = q * 32 + lane;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    auto release = [&] {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty);
    };
    uint32_t tile = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < total; item += gridDim.x, ++tile) {
      const Item it = item_of(item);
      const int64_t row = (int64_t)it.row0 + rl;
      const bool row_ok = row < it.end;
      const uint32_t b = tile & 1u;
      if (ok) ok = warp_wait<false>(&tfull[b], (tile >> 1) & 1u, p.status, abort_flag, site0 | 8, (int)tile, p.wait_ns);
      tc_fence_after_sync();
      const uint32_t base = tmem + lane_base + b * kAccStep;
      if (kGemm1) {
        // h columns n*128 + 64 hf + 32 ch: gate columns 64 hf + 32 ch, up columns 128 more.
        // The overlap is up columns 32.. of buffer 0 and gate columns 0..95 of buffer 1, so
        // the blocks are taken 1, 0 from buffer 0 and 0, 1 from buffer 1, and one of the two
        // halves needs its first block only.
        const int last = (b == 0) == (hf == 0) ? 0 : 1;  // step after which the overlap has been read
        const int64_t h0 = row * p.N + it.n * 128 + 64 * hf;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const int ch = b == 0 ? 1 - st : st;
          uint32_t g[32], u[32];
          tmem_ld32(base + 64 * hf + 32 * ch, g);
          tmem_ld32(base + 128 + 64 * hf + 32 * ch, u);
          tmem_ld_wait(g);
          tmem_ld_wait(u);
          if (st == last) release();
          if (p.raw_out) {
            // The fp32 gate and up sums themselves (stage entry point, tests).
            if (ok && row_ok) {
              float4* dg = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * 2 * p.N + it.n * 128 +
                                                     64 * hf + 32 * ch);
              float4* du = dg + p.N / 4;
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                dg[v] = make_float4(__uint_as_float(g[4 * v]), __uint_as_float(g[4 * v + 1]),
                                    __uint_as_float(g[4 * v + 2]), __uint_as_float(g[4 * v + 3]));
                du[v] = make_float4(__uint_as_float(u[4 * v]), __uint_as_float(u[4 * v + 1]),
                                    __uint_as_float(u[4 * v + 2]), __uint_as_float(u[4 * v + 3]));
              }
            }
            continue;
          }
          float h[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) h[i] = silu_mul(__uint_as_float(g[i]), __uint_as_float(u[i]));
          const uint32_t sb = e8m0_of(amax_bits<32>(h));
          uint4 w = make_uint4(0, 0, 0, 0);
          if (sb != 255u) {
            const float r = e8m0_rcp(sb);
            w = make_uint4(e2m1x8(h, r), e2m1x8(h + 8, r), e2m1x8(h + 16, r), e2m1x8(h + 24, r));
          }
          if (ok && row_ok) {
            const int64_t c = h0 + 32 * ch;
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + c / 2) = w;
            reinterpret_cast<uint8_t*>(p.out_scale)[c / 32] = (uint8_t)sb;
          }
        }
      } else {
        // y columns n*256 + 128 hf + 32 ch. The overlap is columns 160.. of buffer 0 (this
        // warp's blocks 1..3 if hf = 1, none if hf = 0) and 0..95 of buffer 1 (blocks 0..2 if
        // hf = 0, none if hf = 1); a warp without any releases at once.
        const bool mine = (b == 0) == (hf == 1);
        const float gw = row_ok ? (p.row_gate ? p.row_gate[row] : 1.0f) : 0.0f;
        if (!mine) release();
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          const int ch = b == 0 ? (st + 1) & 3 : st;
          uint32_t v[32];
          tmem_ld32(base + 128 * hf + 32 * ch, v);
          tmem_ld_wait(v);
          if (mine && st == 2) release();
          if (ok && row_ok) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.N + it.n * 256 + 128 * hf +
                                                  32 * ch);
#pragma unroll
            for (int w = 0; w < 4; ++w)
              dst[w] = make_uint4(
                  pack_bf16x2(__uint_as_float(v[8 * w]) * gw, __uint_as_float(v[8 * w + 1]) * gw),
                  pack_bf16x2(__uint_as_float(v[8 * w + 2]) * gw, __uint_as_float(v[8 * w + 3]) * gw),
                  pack_bf16x2(__uint_as_float(v[8 * w + 4]) * gw, __uint_as_float(v[8 * w + 5]) * gw),
                  pack_bf16x2(__uint_as_float(v[8 * w + 6]) * gw, __uint_as_float(v[8 * w + 7]) * gw));
          }
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <bool kGemm1>
cudaError_t launch_one(const GemmParams& p, int grid, const AMaps& a, const MxMaps& tm, cudaStream_t s) {
  auto kern = mxfp4_gemm_kernel<kGemm1>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDynamic);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), kDynamic, s, 1, p, a, tm);
}

}  // namespace

cudaError_t launch_mxfp4_gemm(const GemmParams& p, bool gemm1, int grid, const AMaps& tm_a, const MxMaps& tm,
                              cudaStream_t s) {
  return gemm1 ? launch_one<true>(p, grid, tm_a, tm, s) : launch_one<false>(p, grid, tm_a, tm, s);
}

}  // namespace moe
