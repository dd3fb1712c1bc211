// What the prompt delta rule's translation units share.
#pragma once
#include "launchers.hpp"
#include "prompt.cuh"

namespace tv {

// Longest sequence (host bound) from which a call takes the block form: one
// full block.  Measured for 48 value heads of 128 x 128: 64 rows take 28.7 us in
// blocks and 28.6 row by row, 32 rows 27.7 and 16.4, 128 rows 30.8 and 51.2.
constexpr int kBlocksFrom = 64;

struct GdnPromptParams {
  PromptRows pr;
  float* S[TV_MAX_SEQ];
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  void* out;
  int Hk, Hv, dv;
  float scale;
};

bool gdn_prompt_tc_fits(const tv_gdn_layer* l, const tv_prompt* pr);
size_t gdn_prompt_tc_ws_bytes(const tv_gdn_layer* l, const tv_prompt* pr);
tv_status gdn_prompt_tc_launch(const tv_gdn_layer* l, const GdnPromptParams& a, void* ws, size_t ws_bytes, const tv_prompt* pr,
                               cudaStream_t st);

}  // namespace tv
