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
// side by side), K stages of 256 inputs (128 bytes); or, as a pair of CTAs with 2-SM
// MMAs, 256 rows, each CTA holding 128 rows of A and half of the weight rows. An SM's
// shared memory moves 128 bytes a clock: single CTAs write 51 KB and read 48 KB of it
// for 512 clocks of MMA, a pair's CTA 35 KB and 32 KB.
//
// A tile loads the smallest box that covers its group's rows (8, 32, 64 or 128); the other
// rows of the MMA are zeros or an earlier tile's, and their results are not stored. Under
// the power limit, where decode batches run, boxes from 8 rows and zeroed buffers take
// 64 tokens on 352 experts from 528 to 490 us (at 32 rows and more, with what lay there).
//
// Operand tiles come by TMA (128B swizzle) and so do the scales, as row-major 16-byte
// boxes that cover two stages. The tensor core reads scales from TMEM, four bytes (128
// inputs) per 32-bit column, row r in lane r % 32 and column r / 32, repeated in the
// four lane quarters; four scale warps write that layout (24 columns a stage: 8 for
// this CTA's A rows, 16 for all B rows) into a ring of four.
//
// TMEM: the two accumulator buffers of 256 columns overlap by 96 columns
// (0..255 and 160..415), which leaves 96 columns for the scales. The epilogue reads a
// buffer's shared columns first and then lets the next tile's MMAs begin.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2..5 scale writers, 6..13 epilogue.
//
// Measured (H = 4096, I = 1536): 16 tokens on 88 experts, single CTAs: gate/up 82 us, 468
// MB at 69% of DRAM peak, the weight stream. 8192 tokens on 352 experts, pairs: gate/up 625
// us (3.0 PFLOP/s) and down 390 us (2.4); loads alone, without MMAs and epilogue, take 462
// and 358 us, so the tiles' way from L2 bounds the second and most of the first (the
// layer on single CTAs: 1.35 ms, on pairs 1.20).
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp4.cuh"
#include "gemm_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kScaleWarps = 4;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * (kScaleWarps + kEpiWarps);
constexpr int kStageK = 256;                       // inputs per stage
constexpr int kABytes = kTileM * kStageBytesK;     // 16 KB
constexpr int kScBuf = (kTileM + 256) * 16;        // scales of two stages: 128 A rows, 256 B rows
constexpr int kScBufs = 3;
constexpr int kSfSlots = 4;                        // stages of scales in TMEM
constexpr int kMaxStages = 6;
constexpr int kMaxGroups = kMaxExperts + 1;
constexpr uint32_t kAccStep = 160;                 // column offset of the second accumulator buffer
constexpr uint32_t kSfCol = 416;                   // first scale column
constexpr uint32_t kSfCols = 24;                   // scale columns per stage
constexpr int kYBox = 32 * 128;                    // bytes of one y store box: 32 rows x 64 bf16 columns
constexpr int kYWarp = 2 * kYBox;                  // an epilogue warp's 32 rows x 128 columns
static_assert(kSfCol + kSfSlots * kSfCols <= 512, "TMEM columns");

// kStoreY: y tiles leave through shared memory and TMA stores (pairs only, 64 KB).
template <bool kPair, bool kStoreY>
struct Cfg {
  static constexpr int kStages = kPair ? (kStoreY ? 4 : 6) : 4;
  static constexpr int kBBytes = (kPair ? 128 : 256) * kStageBytesK;  // this CTA's share of the B tile
  static constexpr size_t kB = (size_t)kStages * kABytes;
  static constexpr size_t kY = kB + (size_t)kStages * kBBytes;
  static constexpr size_t kSc = kY + (kStoreY ? kEpiWarps * kYWarp : 0);
  static constexpr size_t kBars = kSc + (size_t)kScBufs * kScBuf;
  static constexpr int kNumBars = 2 * kMaxStages + 2 * kScBufs + 2 * kSfSlots + 2 + 1 + 1;
  static constexpr size_t kMisc = kBars + ((kNumBars * 8 + 127) / 128) * 128;
  static constexpr size_t kMt = kMisc + 64;
  static constexpr size_t kOff = kMt + (kMaxGroups + 1) * 4;
  static constexpr size_t kDynamic = kOff + (kMaxGroups + 1) * 4 + 1024;
  static_assert(kDynamic <= 227 * 1024, "shared memory budget");
};

// Instruction descriptor of kind::mxf4: E2M1 operands (K-major), E8M0 scales,
// M x N; sf = which half of a scale column's four bytes this instruction's 64
// inputs use (0 or 2).
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) |
         (sf << 29);
}

template <bool kPair>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
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

template <bool kGemm1, bool kPair, bool kStoreY>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_gemm_kernel(const GemmParams p, const __grid_constant__ AMaps tm_a, const __grid_constant__ MxMaps tm) {
  static_assert(!kStoreY || (kPair && !kGemm1), "staged y stores belong to the down GEMM on pairs");
  using C = Cfg<kPair, kStoreY>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::kB;
  uint8_t* sSc = smem + C::kSc;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);  // operands landed (pair: both CTAs', on the leader)
  uint64_t* empty = full + kMaxStages;                            // the stage's MMAs completed
  uint64_t* scfull = empty + kMaxStages;                          // scales of two stages landed
  uint64_t* scempty = scfull + kScBufs;                           // ... and have been read
  uint64_t* sfull = scempty + kScBufs;                            // a stage's scales are in TMEM (pair: both CTAs')
  uint64_t* sempty = sfull + kSfSlots;                            // ... and its MMAs completed
  uint64_t* tfull = sempty + kSfSlots;                            // accumulator buffer complete
  uint64_t* tempty = tfull + 2;                                   // the overlap has been read
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_mt = reinterpret_cast<int*>(smem + C::kMt);
  int* s_off = reinterpret_cast<int*>(smem + C::kOff);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = kPair ? cluster_cta_rank() : 0u;  // 0 = the pair's MMA issuer
  const int unit = kPair ? (int)(blockIdx.x / 2) : (int)blockIdx.x;
  const int n_units = kPair ? (int)(gridDim.x / 2) : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kScBufs; ++s) {
      mbar_init(&scfull[s], 1);
      mbar_init(&scempty[s], kScaleWarps);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sfull[s], kPair ? 2 * kScaleWarps : kScaleWarps);
      mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(&tfull[b], 1);
    mbar_init(tempty, kPair ? 2 * kEpiWarps : kEpiWarps);
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
    if (kPair) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  // Rows that no box has filled yet multiply as zeros, which draws less power than what
  // an earlier kernel left there.
  for (int i = threadIdx.x; i < C::kStages * kABytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(sA)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncthreads();
  if (kPair) cluster_sync();  // the peer's barriers are initialised before any remote arrive
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
  const int site0 = 0x1000 | (kGemm1 ? 0x200 : 0) | (kPair ? 0x400 : 0) | (int)(rank << 11);
  const int my_off = kPair ? kTileM * (int)rank : 0;  // this CTA's rows inside a work item
  auto item_of = [&](int item) {
    return decode_item(item, p.n_tiles, p.G, kPair ? 2 * kTileM : kTileM, s_mt, s_off, p.n_fastest != 0);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer --
    if (lane == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, sc_phase = 0, issued = 0, issued_phase = 0, sc_issued = 0, sc_issued_phase = 0;
      bool ok = true;
      for (int item = unit; item < total && ok && p.inject != 1; item += n_units) {
        const Item it = item_of(item);
        const bool shared = it.g == p.E;
        const int yb = (shared ? 0 : it.g * p.N) + it.n * (kGemm1 ? 128 : 256);
        const CUtensorMap* c0 = shared ? &tm.scode0 : &tm.code0;
        const CUtensorMap* c1 = shared ? &tm.scode1 : &tm.code1;  // GEMM2: the same rows in 128-row boxes
        const CUtensorMap* f0 = shared ? &tm.sscale0 : &tm.scale0;
        const CUtensorMap* f1 = shared ? &tm.sscale1 : &tm.scale1;
        const int my_row0 = it.row0 + my_off;
        auto a_rows = [&](int row0) {
          const int v = it.end - row0;
          return v <= 8 ? 8 : v <= 32 ? 32 : v <= 64 ? 64 : 128;
        };
        const int my_a = a_rows(my_row0);
        const CUtensorMap* amap =
            my_a == 8 ? &tm.a8 : my_a == 32 ? &tm_a.rows32 : (my_a == 64 ? &tm_a.rows64 : &tm_a.rows128);
        const CUtensorMap* smap = my_a == 8 ? &tm.a_scale8 : &tm.a_scale;
        const uint32_t sc_tx = my_a == 8 ? kScBuf - (kTileM - 8) * 16 : kScBuf;
        const uint32_t tx = kPair ? (uint32_t)(a_rows(it.row0) + a_rows(it.row0 + kTileM)) * kStageBytesK + 2u * C::kBBytes
                                  : (uint32_t)my_a * kStageBytesK + C::kBBytes;
        for (int ks = 0; ks < kstages; ++ks) {
          if ((ks & 1) == 0) {
            if (!mbar_wait(&scempty[buf], sc_phase ^ 1, p.status, abort_flag, site0 | 2, item, p.wait_ns)) {
              ok = false;
              break;
            }
            uint8_t* sc = sSc + buf * kScBuf;
            const int kx = ks * (kStageK / 32);
            mbar_arrive_expect_tx(&scfull[buf], sc_tx);
            tma_load_2d(sc, smap, &scfull[buf], kx, my_row0);
            tma_load_2d(sc + kTileM * 16, f0, &scfull[buf], kx, yb);
            if (kGemm1) tma_load_2d(sc + 2 * kTileM * 16, f1, &scfull[buf], kx, yb);
            sc_issued |= 1u << buf;
            sc_issued_phase = (sc_issued_phase & ~(1u << buf)) | (sc_phase << buf);
            if (++buf == kScBufs) { buf = 0; sc_phase ^= 1; }
          }
          if (!mbar_wait(&empty[stage], phase ^ 1, p.status, abort_flag, site0 | 1, item, p.wait_ns)) {
            ok = false;
            break;
          }
          const int kx = ks * kStageBytesK;
          if (kPair) {
            // Both CTAs' tiles complete on the leader's barrier, which expects them all.
            const uint32_t bar0 = map_to_cta(&full[stage], 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], tx);
            tma_load_2d_pair(sA + stage * kABytes, amap, bar0, kx, my_row0);
            // GEMM1: the leader holds the gate rows, its peer the up rows; GEMM2: rows 0..127 and 128..255.
            tma_load_2d_pair(sB + stage * C::kBBytes, (kGemm1 && rank == 0) ? c0 : c1, bar0, kx,
                             kGemm1 ? yb : yb + 128 * (int)rank);
          } else {
            mbar_arrive_expect_tx(&full[stage], tx);
            tma_load_2d(sA + stage * kABytes, amap, &full[stage], kx, my_row0);
            tma_load_2d(sB + stage * C::kBBytes, c0, &full[stage], kx, yb);
            if (kGemm1) tma_load_2d(sB + stage * C::kBBytes + C::kBBytes / 2, c1, &full[stage], kx, yb);
          }
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        // Let the tensor copies already in flight land before the CTA leaves.
        for (int s = 0; s < C::kStages && rank == 0; ++s) {
          if (!(issued & (1u << s))) continue;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(&full[s], (issued_phase >> s) & 1u) && global_timer_ns() - t0 < 200000000ull) {}
        }
        for (int s = 0; s < kScBufs; ++s) {
          if (!(sc_issued & (1u << s))) continue;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(&scfull[s], (sc_issued_phase >> s) & 1u) && global_timer_ns() - t0 < 200000000ull) {}
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer --
    if (lane == 0 && rank == 0) {
      constexpr int kM = kPair ? 2 * kTileM : kTileM;
      constexpr uint32_t kId0 = idesc_mx(kM, 256, 0), kId2 = idesc_mx(kM, 256, 2);
      auto commit = [&](uint64_t* bar) {
        if (kPair) mma_commit_pair(bar, 0x3);
        else mma_commit(bar);
      };
      auto wait = [&](uint64_t* bar, uint32_t par, int site, uint32_t at) {
        return kPair ? mbar_wait_cluster(bar, par, p.status, abort_flag, site0 | site, (int)at, p.wait_ns)
                     : mbar_wait(bar, par, p.status, abort_flag, site0 | site, (int)at, p.wait_ns);
      };
      int stage = 0, slot = 0;
      uint32_t phase = 0, sf_phase = 0, tile = 0;
      bool ok = true;
      for (int item = unit; item < total && ok; item += n_units, ++tile) {
        const uint32_t b = tile & 1u;
        // The previous tile's overlap (and so all of the tile before it) has been read.
        if (!wait(tempty, (tile & 1u) ^ 1u, 3, tile)) break;
        tc_fence_after_sync();
        const uint32_t d = tmem + b * kAccStep;
        for (int ks = 0; ks < kstages; ++ks) {
          if (!wait(&full[stage], phase, 4, tile) || !wait(&sfull[slot], sf_phase, 5, tile)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t ad = sdesc_k_sw128(sA + stage * kABytes);
          const uint64_t bd = sdesc_k_sw128(sB + stage * C::kBBytes);
          const uint32_t sf = tmem + kSfCol + slot * kSfCols;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_mx<kPair>(d, ad + 2 * kk, bd + 2 * kk, (kk & 1) ? kId2 : kId0, sf + 4 * (kk / 2), sf + 8 + 8 * (kk / 2),
                          (ks || kk) ? 1u : 0u);
          commit(&empty[stage]);
          commit(&sempty[slot]);
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
          if (++slot == kSfSlots) { slot = 0; sf_phase ^= 1; }
        }
        if (ok) commit(&tfull[b]);
      }
      if (kPair) mma_commit_pair(drain, 0x1);
      else mma_commit(drain);  // every MMA issued so far has completed once this arrives
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < 200000000ull) {}
    }
  } else if (warp < 2 + kScaleWarps) {
    // -------------------------------------------------------- scale writers --
    // Lane l holds rows l, l + 32, ... of both operands: 12 rows x 16 bytes, the
    // first 8 bytes for the even stage, the others for the odd one.
    const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
    int buf = 0, slot = 0;
    uint32_t sc_phase = 0, sf_phase = 0;
    bool ok = true;
    for (int item = unit; item < total && ok; item += n_units) {
      for (int ks = 0; ks < kstages && ok; ks += 2) {
        if (!warp_wait<false>(&scfull[buf], sc_phase, p.status, abort_flag, site0 | 6, item, p.wait_ns)) {
          ok = false;
          break;
        }
        uint4 sc[12];
        const uint4* src = reinterpret_cast<const uint4*>(sSc + buf * kScBuf) + lane;
#pragma unroll
        for (int i = 0; i < 12; ++i) sc[i] = src[32 * i];
        // Both stages' columns, one after the other, then one wait for the stores: waiting
        // and arriving per stage took longer than a stage's MMAs.
        const int slot0 = slot;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // The slot is free once the MMAs of its previous use completed.
          if (ok) ok = warp_wait<kPair>(&sempty[slot0 + half], sf_phase ^ 1, p.status, abort_flag, site0 | 7, item, p.wait_ns);
          tc_fence_after_sync();
          const uint32_t col = tmem + lane_base + kSfCol + (slot0 + half) * kSfCols;
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
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scempty[buf]);  // (every lane's values are in registers)
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // (The leader's MMAs read these scales in both CTAs' tensor memory.)
            if (kPair) mbar_arrive_cluster(map_to_cta(&sfull[slot0 + half], 0));
            else mbar_arrive(&sfull[slot0 + half]);
          }
        }
        slot += 2;
        if (slot == kSfSlots) { slot = 0; sf_phase ^= 1; }
        if (++buf == kScBufs) { buf = 0; sc_phase ^= 1; }
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
      if (lane == 0) {
        if (kPair) mbar_arrive_cluster(map_to_cta(tempty, 0));
        else mbar_arrive(tempty);
      }
    };
    uint32_t tile = 0;
    bool ok = true;
    for (int item = unit; item < total; item += n_units, ++tile) {
      const Item it = item_of(item);
      const int64_t row = (int64_t)it.row0 + my_off + rl;
      const bool row_ok = row < it.end;
      const uint32_t b = tile & 1u;
      if (ok) ok = warp_wait<kPair>(&tfull[b], (tile >> 1) & 1u, p.status, abort_flag, site0 | 8, (int)tile, p.wait_ns);
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
        // A warp whose 32 rows all lie inside the group writes them as two 32 x 64 boxes
        // staged in shared memory (128B-swizzled) and stored by TMA, whole 128-byte
        // lines; the warp straddling the group's end stores its rows from registers.
        const int64_t wrow0 = (int64_t)it.row0 + my_off + q * 32;
        const bool staged = kStoreY && ok && wrow0 + 32 <= it.end;
        uint8_t* ys = smem + C::kY + (warp - 6) * kYWarp;
        if (staged) {
          if (lane == 0) bulk_wait_group_read0();  // the previous tile's boxes have been read
          __syncwarp();
        }
        if (!mine) release();
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          const int ch = b == 0 ? (st + 1) & 3 : st;
          uint32_t v[32];
          tmem_ld32(base + 128 * hf + 32 * ch, v);
          tmem_ld_wait(v);
          if (mine && st == 2) release();
          auto packed = [&](int w) {  // columns 32 ch + 8 w .. + 7 of this row, gated, bf16
            return make_uint4(pack_bf16x2(__uint_as_float(v[8 * w]) * gw, __uint_as_float(v[8 * w + 1]) * gw),
                              pack_bf16x2(__uint_as_float(v[8 * w + 2]) * gw, __uint_as_float(v[8 * w + 3]) * gw),
                              pack_bf16x2(__uint_as_float(v[8 * w + 4]) * gw, __uint_as_float(v[8 * w + 5]) * gw),
                              pack_bf16x2(__uint_as_float(v[8 * w + 6]) * gw, __uint_as_float(v[8 * w + 7]) * gw));
          };
          if (staged) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
              *reinterpret_cast<uint4*>(ys + (ch >> 1) * kYBox + lane * 128 +
                                        ((((ch & 1) * 4 + w) ^ (lane & 7)) << 4)) = packed(w);
          } else if (ok && row_ok) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * p.N + it.n * 256 + 128 * hf +
                                                  32 * ch);
#pragma unroll
            for (int w = 0; w < 4; ++w) dst[w] = packed(w);
          }
        }
        if (staged) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm.y, ys, it.n * 256 + 128 * hf, (int32_t)wrow0);
            tma_store_2d(&tm.y, ys + kYBox, it.n * 256 + 128 * hf + 64, (int32_t)wrow0);
            bulk_commit_group();
          }
        }
      }
    }
    if (kStoreY && lane == 0) bulk_wait_group0();  // y boxes written before the CTA leaves
  }
  tc_fence_before_sync();
  __syncthreads();
  if (kPair) cluster_sync();  // neither CTA frees the pair's TMEM while the other still uses it
  if (warp == 1) {
    tc_fence_after_sync();
    if (kPair) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

template <bool kGemm1, bool kPair, bool kStoreY>
cudaError_t launch_one(const GemmParams& p, int grid, const AMaps& a, const MxMaps& tm, cudaStream_t s) {
  auto kern = mxfp4_gemm_kernel<kGemm1, kPair, kStoreY>;
  constexpr size_t kDynamic = Cfg<kPair, kStoreY>::kDynamic;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDynamic);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((unsigned)(kPair ? grid & ~1 : grid)), dim3(kThreads), kDynamic, s, kPair ? 2 : 1, p, a, tm);
}

}  // namespace

cudaError_t launch_mxfp4_gemm(const GemmParams& p, bool gemm1, bool pair, int grid, const AMaps& tm_a, const MxMaps& tm,
                              cudaStream_t s) {
  if (pair) return gemm1 ? launch_one<true, true, false>(p, grid, tm_a, tm, s) : launch_one<false, true, true>(p, grid, tm_a, tm, s);
  return gemm1 ? launch_one<true, false, false>(p, grid, tm_a, tm, s) : launch_one<false, false, false>(p, grid, tm_a, tm, s);
}

}  // namespace moe
