// The few-token layer (include/moe.h: moe_few_tokens): arguments, workspace
// and launcher of ops/few.hip.
#pragma once

#include "mx.h"

namespace moe {

struct FewDims {
  int T, D, L, E, k, H, S, HS;
  int X, x0;  // experts held here: x0 .. x0 + X - 1
  bool bf16, mx;
};

// Activations between the phases.  bf16 layers: an fp32 value as two bf16
// parts (value = hi + lo to 2^-17), which the bf16 matrix instructions take
// one after the other; fp32 layers: the value (lo unused).
struct FewAct {
  void* hi;
  void* lo;
};

struct FewWs {  // byte offsets
  size_t logits, mask, active, first, count, gate, z, z_lo, hs, hs_lo, h, h_lo, part, c, c_lo, arrived, total;
  int parts, tiles, down_rt;  // the down product: shares, row tiles, 16-row groups of a tile
};
FewWs few_layout(const FewDims& d);

struct FewArgs {
  FewDims d;
  const void *x, *w_router, *w_down, *w13, *w2, *w_up, *ws13, *ws2;
  const uint8_t *w13_scales, *w2_scales;
  const float* bias;
  int bias_row_tokens;
  int32_t* topk_idx;
  float* topk_w;
  void* out;
  // workspace
  float* logits;      // [T][E]
  uint64_t* mask;     // [X] tokens of each chosen expert, in the order of `active`
  int32_t* active;    // [X] chosen experts (local index), ascending
  int32_t* first;     // [X] first pair row of each chosen expert
  int32_t* count;     // [0]: chosen experts
  float* gate;        // [T][X] routing weights of the chosen pairs
  FewAct z, hs, h, c; // [T][L], [T][S * HS], [T * k][H], [T][L]
  float* part;        // [parts][T][L], where parts > 1
  int32_t* arrived;   // [tiles] shares of a tile that are done
  int parts, tiles, down_rt;
};
hipError_t launch_few_project(const FewArgs& a, hipStream_t st);
hipError_t launch_few_select(const FewArgs& a, hipStream_t st);
hipError_t launch_few_gate_up(const FewArgs& a, hipStream_t st);
hipError_t launch_few_down(const FewArgs& a, hipStream_t st);
hipError_t launch_few_up(const FewArgs& a, hipStream_t st);

}  // namespace moe
