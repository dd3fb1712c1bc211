// What the prompt delta rule's translation units share.
#pragma once
#include "launchers.hpp"
#include "prompt.cuh"

namespace tv {

constexpr int kBlocksFrom = 32;  // longest sequence from which a call takes the block form

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
