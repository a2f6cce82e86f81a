// moe_decode.h -- launcher interface of the MoE layer for a few tokens.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

constexpr int kMoeDecodeMaxTokens = 32;

struct MoeDecodeArgs {
  const void* x;          // [tokens, hidden]
  int dtype;
  const void* router;     // [experts, hidden], the type of x
  const float* bias;      // [experts]
  const uint8_t* w1;      // [experts, inter or 2 inter, hidden] NVFP4
  const uint8_t* w1_sf;
  const float* w1_g;
  const uint8_t* w2;      // [experts, hidden, inter] NVFP4
  const uint8_t* w2_sf;
  const float* w2_g;
  void* out;              // [tokens, hidden]
  int32_t* ids_out;
  float* w_out;
  int tokens, experts, top_k, hidden, inter, act, n_group, topk_group, norm;
  float scaling;
  int tiled;              // expert weights in the pre-tiled layout
  void* workspace;
};
size_t moe_decode_workspace_bytes(int tokens, int experts, int top_k, int hidden, int inter);
hipError_t launch_moe_decode(const MoeDecodeArgs& m, hipStream_t s);

}  // namespace nvfp4
