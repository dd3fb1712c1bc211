// The gated delta rule over a prompt's packed rows, states advanced in place:
// the entry point, and the row-by-row kernel (fp32 layers, state widths the
// block form does not take, and short prompts; blocks: gdn_prompt_tc.cu).
//
// A lane group holds one state row in registers and steps through
// its sequence's tokens with the step function of decode (gdn_step.cuh), the
// next token's key, query, value and gates in flight during the current step.
// The bits are those of decoding the tokens one by one.
#include <cmath>

#include "gdn_prompt.cuh"
#include "gdn_step.cuh"

namespace tv {

template <typename T, int LPR>
struct TokenIn {
  f2_t k[kPairs], q[kPairs];
  float v, alpha, beta;
  __device__ __forceinline__ void load(const GdnPromptParams& p, size_t t, int g, int h, int row, bool valid, int j) {
    constexpr int DK = 2 * kPairs * LPR;
    load_row_any<LPR>(k, static_cast<const T*>(p.k) + (t * p.Hk + g) * DK, j);
    load_row_any<LPR>(q, static_cast<const T*>(p.q) + (t * p.Hk + g) * DK, j);
    const size_t hi = t * p.Hv + h;
    v = valid ? to_f32(static_cast<const T*>(p.v)[hi * p.dv + row]) : 0.f;
    alpha = p.alpha[hi];
    beta = p.beta[hi];
  }
};

template <typename T, int LPR>
__global__ void __launch_bounds__(128) gdn_prompt_rec_kernel(const __grid_constant__ GdnPromptParams p) {
  constexpr int DK = 2 * kPairs * LPR;
  constexpr int R = 128 / LPR;
  const int s = blockIdx.y;
  const int rb_per_head = (p.dv + R - 1) / R;
  const int h = blockIdx.x / rb_per_head, rb = blockIdx.x % rb_per_head;
  if (status_bad(p.pr.status)) return;
  const WarpSeqs w = load_seqs(p.pr, threadIdx.x & 31);
  if (w.code) {
    set_status(p.pr.status, w.code);
    return;
  }
  const int off = __shfl_sync(0xffffffffu, w.off, s), n = __shfl_sync(0xffffffffu, w.end, s) - off;
  if (n <= 0) return;
  const int g = h / (p.Hv / p.Hk);
  const int j = threadIdx.x % LPR, row = rb * R + threadIdx.x / LPR;
  const bool valid = row < p.dv;
  float* Srow = p.S[s] + (static_cast<size_t>(h) * p.dv + (valid ? row : 0)) * DK;
  f2_t st[kPairs];
  if (valid) {
    load_row<LPR>(st, Srow, j);
  } else {
#pragma unroll
    for (int e = 0; e < kPairs; e++) st[e] = 0ull;
  }
  TokenIn<T, LPR> cur, nxt;
  cur.load(p, off, g, h, row, valid, j);
  for (int t = 0; t < n; t++) {
    const int tn = t + 1 < n ? t + 1 : t;
    nxt.load(p, static_cast<size_t>(off) + tn, g, h, row, valid, j);
    const float kq = kq_group<LPR>(cur.k, cur.q);
    const float o = gdn_row_step<LPR, true>(st, cur.k, cur.q, kq, cur.v, cur.alpha, cur.beta, p.scale, true);
    if (valid && j == 0)
      static_cast<T*>(p.out)[((static_cast<size_t>(off) + t) * p.Hv + h) * p.dv + row] = from_f32<T>(o);
    cur = nxt;
  }
  if (valid) store_row<LPR>(Srow, st, j);
}

template <typename T, int LPR>
static void launch_rec(const GdnPromptParams& p, cudaStream_t st) {
  constexpr int R = 128 / LPR;
  const dim3 grid(p.Hv * ((p.dv + R - 1) / R), p.pr.n_seq);
  gdn_prompt_rec_kernel<T, LPR><<<grid, 128, 0, st>>>(p);
}

}  // namespace tv

using namespace tv;

static bool prompt_shape_ok(const tv_gdn_layer* l) {
  return l->Hk >= 1 && l->Hv >= 1 && l->Hv % l->Hk == 0 && l->Hv <= 4096 && (l->dk == 64 || l->dk == 128) &&
         l->dv >= 1 && l->dv <= 256;
}

extern "C" size_t tv_gdn_prompt_workspace_bytes(const tv_gdn_layer* l, const tv_prompt* pr) {
  if (!l || !prompt_ok(pr) || !prompt_shape_ok(l) || !gdn_prompt_tc_fits(l, pr)) return 0;
  return gdn_prompt_tc_ws_bytes(l, pr);
}

extern "C" tv_status tv_gdn_prompt(const tv_gdn_layer* l, const tv_prompt* pr, const void* q, const void* k,
                                   const void* v, const float* alpha, const float* beta, void* out, float scale,
                                   void* ws, size_t ws_bytes, tv_stream stream) {
  if (!l || !l->S || !prompt_ok(pr)) return TV_ERR_ARG;
  if (l->dtype != TV_F32 && l->dtype != TV_BF16) return TV_ERR_DTYPE;
  if (!prompt_shape_ok(l)) return TV_ERR_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale)) return TV_ERR_ARG;
  GdnPromptParams p{};
  for (int s = 0; s < pr->n_seq; s++) {
    if (!l->S[s]) return TV_ERR_ARG;
    if (!aligned16(l->S[s])) return TV_ERR_ALIGN;
    p.S[s] = l->S[s];
  }
  if (pr->n_total == 0) return TV_OK;
  if (!q || !k || !v || !alpha || !beta || !out) return TV_ERR_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(alpha) || !aligned16(beta) || !aligned16(out))
    return TV_ERR_ALIGN;
  p.pr = prompt_rows(pr, nullptr, 0, 0);
  p.q = q; p.k = k; p.v = v; p.alpha = alpha; p.beta = beta; p.out = out;
  p.Hk = l->Hk; p.Hv = l->Hv; p.dv = l->dv; p.scale = scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (gdn_prompt_tc_fits(l, pr)) return gdn_prompt_tc_launch(l, p, ws, ws_bytes, pr, st);
  const bool bf = l->dtype == TV_BF16;
  if (l->dk == 128) {
    if (bf) launch_rec<__nv_bfloat16, 8>(p, st); else launch_rec<float, 8>(p, st);
  } else {
    if (bf) launch_rec<__nv_bfloat16, 4>(p, st); else launch_rec<float, 4>(p, st);
  }
  return launch_status();
}
