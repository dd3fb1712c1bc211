// Causal grouped-query attention over a prompt's packed rows: the entry point,
// and the fp32 path on the CUDA cores (bf16 runs on the tensor cores,
// attn_prompt_tc.cu).  Row i of a sequence sees cache rows 0 .. len + i (the prompt's own
// keys and values are already in the cache).
//
// A CTA owns a few consecutive (token, query head) rows of one KV head, token
// major, so the G heads that share a KV head share its tiles too.  Keys and
// values pass through shared memory in tiles of 32 positions, the next tile by
// cp.async under this one's arithmetic; a warp keeps RPW rows with one running
// maximum and sum each: lane j scores position j of the tile in fp32, and the
// value rows are added in position order, up to each row's own last position
// and no further, so nothing behind it (later rows, rows the cache does not
// hold yet) can reach the result.  Bound by the walk over the keys of the CTA
// with the longest row: 2 + 1 heads of 64, 256 + 37 rows 14.2 us (with four rows
// a warp and tiles loaded on demand 35.6).
#include <cmath>

#include "attn_prompt.cuh"
#include "mma_tile.cuh"
#include "ptx.cuh"

namespace tv {

template <int D, int RPW>
struct Cuda {
  static constexpr int ROWS = 4 * RPW;  // rows of a CTA
  static constexpr int LD = D + 4;      // a lane reads its own key row, 16 bytes at a time: rows 4 banks apart
  static constexpr int TILE = 32 * LD;
  static constexpr int SMEM = (ROWS * D + 4 * TILE + 4 * 32 * RPW) * 4;
};

template <int D, int RPW>
__global__ void __launch_bounds__(128) attn_prompt_cuda_kernel(const __grid_constant__ AttnPromptCudaParams p) {
  using C = Cuda<D, RPW>;
  constexpr int CPL = D / 32, LD = C::LD;
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                      // [ROWS][D]
  float* kb = qs + C::ROWS * D;        // [2][32][LD] keys
  float* vb = kb + 2 * C::TILE;        // [2][32][LD] values
  float* ps = vb + 2 * C::TILE;        // [warp][32][RPW] probabilities
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
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
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * C::ROWS;
  if (row0 >= rows) return;
  const int live = static_cast<int>(rows - row0 < C::ROWS ? rows - row0 : C::ROWS);
  auto row_at = [&](int r) {  // packed (token, head) row of the buffers
    const int64_t fr = row0 + r;
    return (static_cast<size_t>(off) + static_cast<size_t>(fr / G)) * p.Hq + static_cast<size_t>(g) * G + static_cast<size_t>(fr % G);
  };
  const int end = L + static_cast<int>((row0 + live - 1) / G) + 1;  // positions any row here sees
  const float* K = static_cast<const float*>(p.K[s]) + static_cast<size_t>(g) * p.pr.cap * D;
  const float* V = static_cast<const float*>(p.V[s]) + static_cast<size_t>(g) * p.pr.cap * D;
  auto fetch = [&](int t0, int b) {  // rows behind `end` come in as zeros
    for (int e = threadIdx.x; e < 2 * 32 * (D / 4); e += 128) {
      const int r = e / (2 * (D / 4)), c = e % (2 * (D / 4)), cc = c % (D / 4) * 4;
      const bool ok = t0 + r < end;
      const size_t src = static_cast<size_t>(ok ? t0 + r : 0) * D + cc;
      if (c < D / 4) cp_async16(smem_u32(kb + b * C::TILE + r * LD + cc), K + src, ok);
      else cp_async16(smem_u32(vb + b * C::TILE + r * LD + cc), V + src, ok);
    }
    cp_async_commit();
  };
  fetch(0, 0);
  for (int e = threadIdx.x; e < C::ROWS * (D / 4); e += 128) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    reinterpret_cast<float4*>(qs + r * D + c)[0] =
        r < live ? *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + row_at(r) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
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
  float* pw = ps + warp * 32 * RPW;
  for (int t0 = 0, b = 0; t0 < end; t0 += 32, b ^= 1) {
    cp_async_wait_group<0>();
    __syncthreads();  // the tile is in; every warp is done with the other buffer
    if (t0 + 32 < end) fetch(t0 + 32, b ^ 1);
    const float* kt = kb + b * C::TILE + lane * LD;
    float sc[RPW];
#pragma unroll
    for (int i = 0; i < RPW; i++) sc[i] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      const float4 k4 = *reinterpret_cast<const float4*>(kt + d);
#pragma unroll
      for (int i = 0; i < RPW; i++) {
        const float4 q4 = *reinterpret_cast<const float4*>(qs + (warp * RPW + i) * D + d);
        sc[i] = __fmaf_rn(q4.w, k4.w, __fmaf_rn(q4.z, k4.z, __fmaf_rn(q4.y, k4.y, __fmaf_rn(q4.x, k4.x, sc[i]))));
      }
    }
    float mx[RPW], sum[RPW];
#pragma unroll
    for (int i = 0; i < RPW; i++) mx[i] = sc[i] = t0 + lane <= last[i] ? __fmul_rn(sc[i], p.c) : -INFINITY;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
      for (int i = 0; i < RPW; i++) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
#pragma unroll
    for (int i = 0; i < RPW; i++) {
      const float mn = fmaxf(m[i], mx[i]);
      const float alpha = mn == m[i] ? 1.f : exp2f(__fsub_rn(m[i], mn));
      // (every score so far -inf: weights of 0, not of -inf - -inf)
      const float pj = t0 + lane <= last[i] ? exp2f(__fsub_rn(sc[i], mn == -INFINITY ? 0.f : mn)) : 0.f;
      pw[lane * RPW + i] = sum[i] = pj;
      l[i] = __fmul_rn(l[i], alpha);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < CPL; c++) acc[i][c] = __fmul_rn(acc[i][c], alpha);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
      for (int i = 0; i < RPW; i++) sum[i] = __fadd_rn(sum[i], __shfl_xor_sync(0xffffffffu, sum[i], o));
    int most = -1;  // the warp's rows see at most this far
#pragma unroll
    for (int i = 0; i < RPW; i++) {
      l[i] = __fadd_rn(l[i], sum[i]);
      most = max(most, last[i]);
    }
    __syncwarp();
    const int nv = min(32, most - t0 + 1);
    const float* vt = vb + b * C::TILE + lane;
#pragma unroll 4
    for (int j = 0; j < nv; j++) {
      float v[CPL];
#pragma unroll
      for (int c = 0; c < CPL; c++) v[c] = vt[j * LD + 32 * c];
#pragma unroll
      for (int i = 0; i < RPW; i++) {
        if (t0 + j > last[i]) continue;  // the whole warp
        const float pj = pw[j * RPW + i];
#pragma unroll
        for (int c = 0; c < CPL; c++) acc[i][c] = __fmaf_rn(pj, v[c], acc[i][c]);
      }
    }
    __syncwarp();
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
      static_cast<float*>(p.out)[oi] = p.gate ? gate_mul(y, static_cast<const float*>(p.gate)[oi]) : y;
    }
  }
}

template <int D, int RPW>
static tv_status launch_cuda(const AttnPromptCudaParams& p, cudaStream_t st) {
  using C = Cuda<D, RPW>;
  const int64_t rows = static_cast<int64_t>(p.pr.n_max) * (p.Hq / p.Hkv);
  const int64_t gx = rows > 0 ? (rows + C::ROWS - 1) / C::ROWS : 1;  // (n_max 0: the checks alone)
  if (gx > 0x7fffffff || p.Hkv > 65535) return TV_ERR_SHAPE;
  static bool set = false;
  if (!set) {
    if (cudaFuncSetAttribute(attn_prompt_cuda_kernel<D, RPW>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
      return TV_ERR_CUDA;
    set = true;
  }
  launch_k(true, attn_prompt_cuda_kernel<D, RPW>, dim3(static_cast<unsigned>(gx), p.Hkv, p.pr.n_seq), dim3(128), C::SMEM, st, p);
  return launch_status();
}

// Four rows a warp, or one while four would leave SMs without a CTA (a call's
// time is then one CTA's walk over the keys, which is shorter with fewer rows):
// 256 + 37 rows of 2 heads of 64 take 13.8 us with one and 20.7 with four, 512
// rows of 8 heads 46 either way, 2,048 rows of 8 heads 472 and 296.
template <int D>
static tv_status launch_cuda_rows(const AttnPromptCudaParams& p, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.pr.n_total) * p.Hq;
  return rows >= 16 * 2 * num_sms() ? launch_cuda<D, 4>(p, st) : launch_cuda<D, 1>(p, st);
}

static tv_status launch_cuda_d(const AttnPromptCudaParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_cuda_rows<64>(p, st);
    case 128: return launch_cuda_rows<128>(p, st);
    default: return launch_cuda_rows<256>(p, st);
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
  const int64_t cols = static_cast<int64_t>(l->Hq) * l->D;
  if (overlap(q, out, pr->n_total, cols, cols, l->dtype)) return TV_ERR_ARG;  // a row's heads are read after others are written
  if (gate && gate != out && overlap(gate, out, pr->n_total, cols, cols, l->dtype)) return TV_ERR_ARG;
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
  return launch_cuda_d(p, l->D, st);
}
