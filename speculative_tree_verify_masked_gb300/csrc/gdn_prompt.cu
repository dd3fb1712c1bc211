// The gated delta rule over a prompt's packed rows, states advanced in place:
// the entry point, and the row-by-row kernel (fp32 layers, state widths the
// block form does not take, and short prompts; blocks: gdn_prompt_tc.cu).
//
// A lane group holds one state row in registers and steps through its
// sequence's tokens with the step function of decode (gdn_step.cuh): the bits
// are those of decoding the tokens one by one.  Bound by the chain of steps (a
// dot product, its butterfly, the update), so everything else is kept out of
// it: tokens come into shared memory kTok at a time, the next group by cp.async
// under the steps of this one (loading a token ahead from global memory made a
// step wait for memory: 650 cycles), and a group's products k . q are formed at
// once, one lane group a token.  256 + 37 fp32 rows of two heads of 64 x 64:
// 49.5 us, 0.19 us a step.
#include <cmath>

#include "gdn_prompt.cuh"
#include "gdn_step.cuh"
#include "mma_tile.cuh"
#include "ptx.cuh"

namespace tv {

constexpr int kTok = 16;  // tokens in shared memory at a time (two such groups)

template <typename T, int LPR>
__global__ void __launch_bounds__(128) gdn_prompt_rec_kernel(const __grid_constant__ GdnPromptParams p) {
  constexpr int DK = 2 * kPairs * LPR;
  constexpr int R = 128 / LPR;
  __shared__ __align__(16) T ks[2][kTok][DK], qs[2][kTok][DK];
  __shared__ T vs[2][kTok][R];
  __shared__ float al[2][kTok], be[2][kTok], kqs[kTok];
  const int s = blockIdx.y, tid = threadIdx.x;
  const int rb_per_head = (p.dv + R - 1) / R;
  const int h = blockIdx.x / rb_per_head, rb = blockIdx.x % rb_per_head;
  pdl_wait();
  if (status_bad(p.pr.status)) return;
  const WarpSeqs w = load_seqs(p.pr, tid & 31);
  if (w.code) {
    set_status(p.pr.status, w.code);
    return;
  }
  const int off = __shfl_sync(0xffffffffu, w.off, s), n = __shfl_sync(0xffffffffu, w.end, s) - off;
  if (n <= 0) return;
  const int g = h / (p.Hv / p.Hk);
  const int j = tid % LPR, r = tid / LPR, row = rb * R + r;
  const bool valid = row < p.dv;
  float* Srow = p.S[s] + (static_cast<size_t>(h) * p.dv + (valid ? row : 0)) * DK;
  f2_t st[kPairs];
  if (valid) {
    load_row<LPR>(st, Srow, j);
  } else {
#pragma unroll
    for (int e = 0; e < kPairs; e++) st[e] = 0ull;
  }
  // tokens t0 .. of a group into buffer b: keys and queries by cp.async; values
  // and gates through registers, stored one group later
  constexpr int CH = DK * static_cast<int>(sizeof(T)) / 16;  // 16-byte pieces of a row
  constexpr int VN = kTok * R / 128;                         // values a thread brings
  T vr[VN];
  float gr = 0.f;
  auto fetch = [&](int t0, int b) {
    for (int e = tid; e < 2 * kTok * CH; e += 128) {
      const int t = e / (2 * CH), c = e % (2 * CH), cc = c % CH;
      const size_t src = (static_cast<size_t>(off) + min(t0 + t, n - 1)) * p.Hk + g;
      if (c < CH) cp_async16(smem_u32(&ks[b][t][0]) + cc * 16, static_cast<const char*>(p.k) + src * (CH * 16) + cc * 16, true);
      else cp_async16(smem_u32(&qs[b][t][0]) + cc * 16, static_cast<const char*>(p.q) + src * (CH * 16) + cc * 16, true);
    }
    cp_async_commit();
#pragma unroll
    for (int i = 0; i < VN; i++) {
      const int e = tid + 128 * i, t = e / R, x = e % R;
      const size_t hi = (static_cast<size_t>(off) + min(t0 + t, n - 1)) * p.Hv + h;
      vr[i] = static_cast<const T*>(p.v)[hi * p.dv + min(rb * R + x, p.dv - 1)];
    }
    if (tid < 2 * kTok) {
      const size_t hi = (static_cast<size_t>(off) + min(t0 + tid % kTok, n - 1)) * p.Hv + h;
      gr = tid < kTok ? p.alpha[hi] : p.beta[hi];
    }
  };
  auto settle = [&](int b) {  // the group in flight is in shared memory
#pragma unroll
    for (int i = 0; i < VN; i++) {
      const int e = tid + 128 * i;
      vs[b][e / R][e % R] = vr[i];
    }
    if (tid < kTok) al[b][tid] = gr;
    else if (tid < 2 * kTok) be[b][tid - kTok] = gr;
    cp_async_wait_group<0>();
    __syncthreads();
  };
  fetch(0, 0);
  settle(0);
  for (int t0 = 0, b = 0; t0 < n; t0 += kTok, b ^= 1) {
    if (t0 + kTok < n) fetch(t0 + kTok, b ^ 1);
    const int m = min(kTok, n - t0);
    f2_t k[kPairs], q[kPairs], kn[kPairs], qn[kPairs];
    static_assert(R >= kTok, "a lane group for each token");
    if (r < kTok) {  // (whole warps: R and kTok are multiples of a warp's lane groups)
      load_row_any<LPR>(k, &ks[b][r][0], j);
      load_row_any<LPR>(q, &qs[b][r][0], j);
      const float kq = kq_group<LPR>(k, q);
      if (j == 0) kqs[r] = kq;
    }
    __syncthreads();
    load_row_any<LPR>(k, &ks[b][0][0], j);
    load_row_any<LPR>(q, &qs[b][0][0], j);
    float kq = kqs[0], v = to_f32(vs[b][0][r]), a = al[b][0], bt = be[b][0];
    for (int t = 0; t < m; t++) {
      const int tn = t + 1 < m ? t + 1 : t;
      load_row_any<LPR>(kn, &ks[b][tn][0], j);
      load_row_any<LPR>(qn, &qs[b][tn][0], j);
      const float kqn = kqs[tn], v_n = to_f32(vs[b][tn][r]), an = al[b][tn], bn = be[b][tn];
      const float o = gdn_row_step<LPR, true>(st, k, q, kq, v, a, bt, p.scale, true);
      if (valid && j == 0) static_cast<T*>(p.out)[((static_cast<size_t>(off) + t0 + t) * p.Hv + h) * p.dv + row] = from_f32<T>(o);
#pragma unroll
      for (int e = 0; e < kPairs; e++) {
        k[e] = kn[e];
        q[e] = qn[e];
      }
      kq = kqn;
      v = v_n;
      a = an;
      bt = bn;
    }
    if (t0 + kTok < n) {
      __syncthreads();  // (vs, al, be of the other buffer were last read a group ago)
      settle(b ^ 1);
    }
  }
  if (valid) store_row<LPR>(Srow, st, j);
}

template <typename T, int LPR>
static void launch_rec(const GdnPromptParams& p, cudaStream_t st) {
  constexpr int R = 128 / LPR;
  const dim3 grid(p.Hv * ((p.dv + R - 1) / R), p.pr.n_seq);
  launch_k(true, gdn_prompt_rec_kernel<T, LPR>, grid, dim3(128), 0, st, p);
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
  const int64_t kc = static_cast<int64_t>(l->Hk) * l->dk, vc = static_cast<int64_t>(l->Hv) * l->dv;
  if (overlap(v, out, pr->n_total, vc, vc, l->dtype) || overlap(q, out, pr->n_total, kc, vc, l->dtype) ||
      overlap(k, out, pr->n_total, kc, vc, l->dtype) || overlap(alpha, out, pr->n_total, l->Hv, vc, TV_F32, l->dtype) ||
      overlap(beta, out, pr->n_total, l->Hv, vc, TV_F32, l->dtype))
    return TV_ERR_ARG;  // other heads and blocks still read them
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
