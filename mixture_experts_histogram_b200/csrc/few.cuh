// Parameters and launchers of the few-token layer (few.cu).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

constexpr int kFewMaxTokens = MOE_FEW_MAX_TOKENS;
constexpr int kFewSmem = 227 * 1024;  // shared memory of a CTA
constexpr int kFewDownTiles = 16;     // 16-row tiles of the output that a CTA may own

struct FewParams {
  int32_t T, H, I, E, k, S;
  int32_t n_stages;        // weight ring (set by the launcher)
  const uint16_t* x;       // [T, H] bf16
  const uint16_t* router_w;
  const float* bias;       // [E] or null
  moe_weights w;
  __nv_bfloat16* out;      // [T, H]
  int32_t* topk_idx;       // [T, k] or null
  float* topk_w;
  float* logits;           // [T, E]
  uint8_t* xrows;          // x as the gate/up products read it
  float* h;                // [list entries, 8, I]
  int* counter;            // grid barrier
  int* status;
  uint64_t wait_ns;
  int32_t inject;
};

// Weight tensor maps: rows as [128 bytes, rows, lines], boxes of 128 bytes x 8 rows
// (w1, w3) or 4 rows (w2) x a slab's 8 (BF16, FP8) or 4 lines, 128B-swizzled; 4-bit
// storage: scale bytes [rows, K / block] in boxes of the same rows x a slab's scales.
struct FewMaps {
  CUtensorMap w1, w3, w2, sw1, sw3, sw2, s1, s3, s2, ss1, ss3, ss2;
};

// Whether T tokens leave room for the weight ring in shared memory.
bool few_fits(int wdtype, int T, int H, int I, int sms);
int64_t few_x_bytes(int wdtype, int T, int H);  // of FewParams::xrows
cudaError_t launch_few(const FewParams& p, const FewMaps& tm, int wdtype, int sms, cudaStream_t s);

}  // namespace moe
