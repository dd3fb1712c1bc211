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

}  // namespace tv
