// A span of prompt rows as a whole: the check ahead of its first layer, and the
// lengths behind its last.  A launch's latency each.
#include "prompt.cuh"

namespace tv {

// What every prompt call checks for itself.  The GDN calls know no lengths, so
// without this a span that an attention layer refuses would have moved the
// states of the GDN layers before it.
__global__ void __launch_bounds__(32) prompt_check_kernel(PromptRows p) {
  pdl_wait();
  const WarpSeqs w = load_seqs(p, threadIdx.x);
  if (threadIdx.x == 0 && w.code) set_status(p.status, w.code);
}

__global__ void __launch_bounds__(32) prompt_advance_kernel(PromptRows p, int32_t* len) {
  pdl_wait();
  if (status_bad(p.status)) return;
  const WarpSeqs w = load_seqs(p, threadIdx.x);
  if (w.code) {
    if (threadIdx.x == 0) set_status(p.status, w.code);
  } else if (threadIdx.x < p.n_seq) {
    len[threadIdx.x] += w.end - w.off;
  }
}

}  // namespace tv

using namespace tv;

extern "C" tv_status tv_prompt_check(const tv_prompt* pr, const int32_t* len, int32_t max_len, int32_t cap,
                                     tv_stream stream) {
  if (!prompt_ok(pr) || !len || max_len < 0 || cap < 1 || max_len > cap) return TV_ERR_ARG;
  if (!aligned16(len)) return TV_ERR_ALIGN;
  if (pr->n_total == 0) return TV_OK;
  launch_k(true, prompt_check_kernel, dim3(1), dim3(32), 0, reinterpret_cast<cudaStream_t>(stream),
           prompt_rows(pr, len, max_len, cap));
  return launch_status();
}

extern "C" tv_status tv_prompt_advance(const tv_prompt* pr, int32_t* len, tv_stream stream) {
  if (!prompt_ok(pr) || !len) return TV_ERR_ARG;
  if (!aligned16(len)) return TV_ERR_ALIGN;
  if (pr->n_total == 0) return TV_OK;
  launch_k(true, prompt_advance_kernel, dim3(1), dim3(32), 0, reinterpret_cast<cudaStream_t>(stream),
           prompt_rows(pr, nullptr, 0, 0), len);
  return launch_status();
}
