// What the prompt delta rule's translation units share.
#pragma once
#include "launchers.hpp"
#include "prompt.cuh"

namespace tv {

// Longest sequence (host bound) from which a call takes the block form.  In
// blocks and row by row: 48 value heads of 128 x 128 take 15.8 us and 14.7 at 32
// rows, 15.8 and 20.4 at 48, 16.0 and 26.0 at 63; 32 of them 15.7 and 11.9, 15.8 and
// 16.3, 16.0 and 20.5; 8 of 64 x 64 13.3 and 9.0, 13.4 and 12.4, 13.5 and 15.5.
constexpr int kBlocksFrom = 48;

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
