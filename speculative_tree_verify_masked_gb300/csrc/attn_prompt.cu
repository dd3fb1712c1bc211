// Causal grouped-query attention over a prompt's packed rows: the entry point,
// and the fp32 path on the CUDA cores (bf16 runs on the tensor cores,
// attn_prompt_tc.cu).  Row i of a sequence sees cache rows 0 .. len + i (the prompt's own
// keys and values are already in the cache).
//
// A CTA owns kRows consecutive (token, query head) rows of one KV head, token
// major, so the G heads that share a KV head share its tiles too.  Keys and
// values pass through shared memory in tiles of 32 positions; a warp keeps
// four rows with one running maximum and sum each: lane j scores position j
// of the tile in fp32, and the value rows are added in position order, up to
// each row's own last position and no further, so nothing behind it (later
// rows, rows the cache does not hold yet) can reach the result.
#include <cmath>

#include "attn_prompt.cuh"
#include "ptx.cuh"

namespace tv {

constexpr int kRowsCuda = 16;

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_prompt_cuda_kernel(const __grid_constant__ AttnPromptCudaParams p) {
  constexpr int CPL = D / 32, RPW = kRowsCuda / 4, LD = D + 4;
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                     // [kRowsCuda][D]
  float* kv = qs + kRowsCuda * D;     // [32][LD]: keys, then values
  __shared__ float ps[kRowsCuda][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (status_bad(p.pr.status)) return;
  const WarpSeqs w = load_seqs(p.pr, lane);
  if (w.code) {
    if (lane == 0) set_status(p.pr.status, w.code);
    return;
  }
  const int s = blockIdx.z, g = blockIdx.y, G = p.Hq / p.Hkv;
  const int off = __shfl_sync(0xffffffffu, w.off, s), n = __shfl_sync(0xffffffffu, w.end, s) - off;
  const int L = __shfl_sync(0xffffffffu, w.len, s);
  const int64_t rows = static_cast<int64_t>(n) * G;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRowsCuda;
  if (row0 >= rows) return;
  const int live = static_cast<int>(rows - row0 < kRowsCuda ? rows - row0 : kRowsCuda);
  const T* q = static_cast<const T*>(p.q);
  auto row_at = [&](int r) {  // packed (token, head) row of the buffers
    const int64_t fr = row0 + r;
    return (static_cast<size_t>(off) + static_cast<size_t>(fr / G)) * p.Hq + static_cast<size_t>(g) * G + static_cast<size_t>(fr % G);
  };
  for (int e = threadIdx.x; e < kRowsCuda * (D / 8); e += 128) {
    const int r = e / (D / 8), c = e % (D / 8) * 8;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < live) load8(q + row_at(r) * D + c, x);
    store8(qs + r * D + c, x);
  }
  int last[RPW];  // last visible position of each of this warp's rows, -1: no row
  float m[RPW], l[RPW], acc[RPW][CPL];
#pragma unroll
  for (int i = 0; i < RPW; i++) {
    const int r = warp * RPW + i;
    last[i] = r < live ? L + static_cast<int>((row0 + r) / G) : -1;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; c++) acc[i][c] = 0.f;
  }
  const int end = L + static_cast<int>((row0 + live - 1) / G) + 1;  // positions any row here sees
  const T* K = static_cast<const T*>(p.K[s]) + static_cast<size_t>(g) * p.pr.cap * D;
  const T* V = static_cast<const T*>(p.V[s]) + static_cast<size_t>(g) * p.pr.cap * D;
  for (int t0 = 0; t0 < end; t0 += 32) {
    const int nt = min(32, end - t0);
    auto fill = [&](const T* src) {
      for (int e = threadIdx.x; e < 32 * (D / 8); e += 128) {
        const int r = e / (D / 8), c = e % (D / 8) * 8;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < nt) load8(src + static_cast<size_t>(t0 + r) * D + c, x);
        store8(kv + r * LD + c, x);
      }
    };
    __syncthreads();
    fill(K);
    __syncthreads();
    float sc[RPW];
#pragma unroll
    for (int i = 0; i < RPW; i++) sc[i] = 0.f;
    for (int d = 0; d < D; d += 4) {
      const float4 k4 = *reinterpret_cast<const float4*>(kv + lane * LD + d);
#pragma unroll
      for (int i = 0; i < RPW; i++) {
        const float4 q4 = *reinterpret_cast<const float4*>(qs + (warp * RPW + i) * D + d);
        sc[i] = __fmaf_rn(q4.w, k4.w, __fmaf_rn(q4.z, k4.z, __fmaf_rn(q4.y, k4.y, __fmaf_rn(q4.x, k4.x, sc[i]))));
      }
    }
#pragma unroll
    for (int i = 0; i < RPW; i++) {
      const float v = t0 + lane <= last[i] ? __fmul_rn(sc[i], p.c) : -INFINITY;
      float mx = v;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[i], mx);
      const float alpha = mn == m[i] ? 1.f : exp2f(__fsub_rn(m[i], mn));
      const float pj = t0 + lane <= last[i] ? exp2f(__fsub_rn(v, mn)) : 0.f;
      float sum = pj;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      l[i] = __fmaf_rn(l[i], alpha, sum);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < CPL; c++) acc[i][c] = __fmul_rn(acc[i][c], alpha);
      ps[warp * RPW + i][lane] = pj;
    }
    __syncthreads();
    fill(V);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RPW; i++) {
      const int nv = min(nt, last[i] - t0 + 1);
      for (int j = 0; j < nv; j++) {
        const float pj = ps[warp * RPW + i][j];
#pragma unroll
        for (int c = 0; c < CPL; c++) acc[i][c] = __fmaf_rn(pj, kv[j * LD + lane + 32 * c], acc[i][c]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RPW; i++) {
    const int r = warp * RPW + i;
    if (r >= live) continue;
    const size_t o = row_at(r) * D;
#pragma unroll
    for (int c = 0; c < CPL; c++) {
      const size_t oi = o + lane + 32 * c;
      const float y = __fdiv_rn(acc[i][c], l[i]);
      static_cast<T*>(p.out)[oi] = from_f32<T>(p.gate ? gate_mul(y, to_f32(static_cast<const T*>(p.gate)[oi])) : y);
    }
  }
}

template <typename T, int D>
static tv_status launch_cuda(const AttnPromptCudaParams& p, cudaStream_t st) {
  constexpr int smem = (kRowsCuda * D + 32 * (D + 4)) * 4;
  const int64_t rows = static_cast<int64_t>(p.pr.n_max) * (p.Hq / p.Hkv);
  const int64_t gx = (rows + kRowsCuda - 1) / kRowsCuda;
  if (gx > 0x7fffffff || p.Hkv > 65535) return TV_ERR_SHAPE;
  if (smem > 48 * 1024) {
    static bool set = false;
    if (!set) {
      if (cudaFuncSetAttribute(attn_prompt_cuda_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return TV_ERR_CUDA;
      set = true;
    }
  }
  attn_prompt_cuda_kernel<T, D><<<dim3(static_cast<unsigned>(gx), p.Hkv, p.pr.n_seq), 128, smem, st>>>(p);
  return launch_status();
}

template <typename T>
static tv_status launch_cuda_d(const AttnPromptCudaParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_cuda<T, 64>(p, st);
    case 128: return launch_cuda<T, 128>(p, st);
    default: return launch_cuda<T, 256>(p, st);
  }
}

}  // namespace tv

using namespace tv;

static tv_status prompt_layer_check(const tv_attn_layer* l, int32_t max_len) {
  if (l->dtype != TV_F32 && l->dtype != TV_BF16) return TV_ERR_DTYPE;
  if (l->Hq < 1 || l->Hkv < 1 || l->Hq % l->Hkv || l->Hq > 4096 || l->Hq / l->Hkv > 128 ||
      (l->D != 64 && l->D != 128 && l->D != 256))
    return TV_ERR_SHAPE;
  return l->cap < 1 || max_len < 0 || max_len > l->cap ? TV_ERR_ARG : TV_OK;
}

extern "C" size_t tv_attn_prompt_workspace_bytes(const tv_attn_layer* l, const tv_prompt* pr, int32_t max_len) {
  if (!l || !prompt_ok(pr) || prompt_layer_check(l, max_len) != TV_OK || l->dtype != TV_BF16) return 0;
  return attn_prompt_tc_ws_bytes(l, pr, max_len);
}

extern "C" tv_status tv_attn_prompt(const tv_attn_layer* l, const tv_prompt* pr, const int32_t* len, int32_t max_len,
                                    const void* q, const void* gate, void* out, float scale, void* ws,
                                    size_t ws_bytes, tv_stream stream) {
  if (!l || !prompt_ok(pr) || !len || !l->K || !l->V) return TV_ERR_ARG;
  const tv_status c = prompt_layer_check(l, max_len);
  if (c != TV_OK) return c;
  if (!(scale > 0.f) || !std::isfinite(scale)) return TV_ERR_ARG;
  AttnPromptCudaParams p{};
  for (int s = 0; s < pr->n_seq; s++) {
    if (!l->K[s] || !l->V[s]) return TV_ERR_ARG;
    if (!aligned16(l->K[s]) || !aligned16(l->V[s])) return TV_ERR_ALIGN;
    p.K[s] = l->K[s];
    p.V[s] = l->V[s];
  }
  if (!aligned16(len)) return TV_ERR_ALIGN;
  if (pr->n_total == 0) return TV_OK;
  if (!q || !out) return TV_ERR_ARG;
  if (!aligned16(q) || !aligned16(gate) || !aligned16(out)) return TV_ERR_ALIGN;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (l->dtype == TV_BF16)
    return attn_prompt_tc_launch(AttnPromptCall{l, pr, len, max_len, q, gate, out, scale, ws, ws_bytes}, st);
  p.pr = prompt_rows(pr, len, max_len, l->cap);
  p.q = q;
  p.gate = gate;
  p.out = out;
  p.Hq = l->Hq;
  p.Hkv = l->Hkv;
  p.c = scale * 1.4426950408889634f;
  return launch_cuda_d<float>(p, l->D, st);
}
