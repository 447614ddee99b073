// Parameters and launchers of the few-token layer (few.cu).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

constexpr int kFewMaxTokens = MOE_FEW_MAX_TOKENS;
constexpr int kFewSmem = 227 * 1024;  // shared memory of a CTA
constexpr int kFewDownTiles = 16;     // 16-row tiles of the output that a CTA may own (in pairs)

struct FewParams {
  int32_t T, H, I, E, k, S;
  int32_t n_stages;        // weight ring (set by the launcher)
  int32_t cta_rows, group_rows, down_lines;  // see FewRows
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

// Output rows of a CTA (a multiple of 4), the rows of them that a stage holds (as
// even a split as fits 32), and lines of 128 bytes of each (a stage is 16 KB, or 8 KB
// for 4-bit storage; MXFP4's 8 scale bytes of a line need a second line to make 16).
struct FewRows {
  int cta, group, lines;
};
inline FewRows few_rows(int wdtype, int H, int sms) {
  FewRows r;
  r.cta = (int)ceil_div(H / 4, sms) * 4;
  const int groups = (int)ceil_div(r.cta, 32);
  r.group = (int)ceil_div(r.cta / 4, groups) * 4;
  r.lines = 16384 / (r.group * 128);
  if (r.lines > 8) r.lines = 8;
  if (wdtype == MOE_WDTYPE_MXFP4) r.lines &= ~1;
  return r;
}

// Weight tensor maps: rows as [128 bytes, rows, lines], 128B-swizzled boxes of 8 rows
// x 8 lines (w1, w3), or as FewRows says (w2); 4-bit storage: scale
// bytes [rows, K / block] in boxes of the same rows and inputs.
struct FewMaps {
  CUtensorMap w1, w3, w2, sw1, sw3, sw2, s1, s3, s2, ss1, ss3, ss2;
};

// Whether T tokens leave room for the weight ring in shared memory.
bool few_fits(int wdtype, int T, int H, int I, int sms);
int64_t few_x_bytes(int wdtype, int T, int H);  // of FewParams::xrows
cudaError_t prepare_few(int wdtype);  // the kernels' settings, before each launch_few
cudaError_t launch_few(const FewParams& p, const FewMaps& tm, int wdtype, int sms, cudaStream_t s);

}  // namespace moe
