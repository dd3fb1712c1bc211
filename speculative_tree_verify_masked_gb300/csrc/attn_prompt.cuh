// What the prompt attention's translation units share.
#pragma once
#include "launchers.hpp"
#include "prompt.cuh"

namespace tv {

struct AttnPromptCudaParams {
  PromptRows pr;
  void* K[TV_MAX_SEQ];
  void* V[TV_MAX_SEQ];
  const void* q;
  const void* gate;  // or null
  void* out;
  int Hq, Hkv;
  float c;  // scale * log2(e)
};

// One tv_attn_prompt call whose arguments have been checked.
struct AttnPromptCall {
  const tv_attn_layer* layer;
  const tv_prompt* prompt;
  const int32_t* len;
  int max_len;
  const void* q;
  const void* gate;
  void* out;
  float scale;
  void* ws;
  size_t ws_bytes;
};
tv_status attn_prompt_tc_launch(const AttnPromptCall& a, cudaStream_t st);
size_t attn_prompt_tc_ws_bytes(const tv_attn_layer* l, const tv_prompt* pr, int max_len);

}  // namespace tv
