// Decode attention over caches in pages: the entry points, and the fp32 path on
// the CUDA cores (bf16 runs on the tensor cores, attn_paged_tc.cu).
//
//   out[s,h] = sum_t softmax_t(scale q[s,h] . K[t]) V[t], t = 0 .. len[s] or the
//   rows of the listed pages among them.
//
// fp32: a CTA owns a (slot, query head); its sixteen warps take every sixteenth run
// of eight rows (four of 256 columns), a row's D values over the 32 lanes, all loads of a run
// in flight, and keep a running maximum and sum each, which are joined at the end.  A
// warp looks up the pages of 32 runs at once.  Bound by the walk over the rows of the
// longest slot (sized for the small model of the tests): 5 slots of up to 301 rows, 2 + 1 heads of 64,
// 5.8 us (four warps, one row of each in flight: 12.2); one slot of 1,024 rows, 4 + 2 heads of 128, 14.1, of 16,384 rows 176, on
// four SMs.
#include "attn_paged.cuh"

namespace tv {

struct PagedCudaParams {
  PagedView v;
  const float* K;
  const float* V;
  const float* q;
  const float* gate;  // or null
  float* out;
  int Hq, G;
  float c;  // scale * log2(e)
};

constexpr int kCudaWarps = 16;

template <int D>
__global__ void __launch_bounds__(32 * kCudaWarps, 1) attn_paged_cuda_kernel(const __grid_constant__ PagedCudaParams p) {
  constexpr int CPL = D / 32, R = D == 256 ? 4 : 8;  // values a lane, rows of a run (never across pages: R divides them)
  __shared__ float acc_s[kCudaWarps][D], m_s[kCudaWarps], l_s[kCudaWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const bool bad = status_set(p.v.b.status);
  const int h = blockIdx.x, s = blockIdx.y, g = h / p.G;
  const size_t row0 = (static_cast<size_t>(s) * p.Hq + h) * D;
  float q[CPL], acc[CPL], m = -INFINITY, l = 0.f;
  bool met = false;  // a row that the slot sees
#pragma unroll
  for (int c = 0; c < CPL; c++) {
    q[c] = p.q[row0 + c * 32 + lane];
    acc[c] = 0.f;
  }
  const int L = paged_len(p.v.b, s);
  if (__syncthreads_or(bad) || L < 0) return;  // (another CTA may set the word between two warps' looks at it)
  const int shift = p.v.b.shift, rows = 1 << shift;
  const int n = p.v.pages(s, g, L) << shift;
  int64_t row = -1;  // of a run of this warp's next 32, a lane each: its first row in the pools, -1: none
  int seen = 0;      // and the rows of it that are seen
  for (int i = warp * R, x = 0; i < n; i += kCudaWarps * R, x = (x + 1) & 31) {
    if (x == 0) {
      const int j = i + lane * kCudaWarps * R;
      row = -1;
      seen = 0;
      if (j < n) {
        const int col = p.v.column(s, g, j >> shift), r = j & (rows - 1);
        seen = col < 0 ? 0 : min(R, L + 1 - (col * rows + r));  // (col < cols: no overflow)
        const int page = seen > 0 ? page_at(p.v.b, s, col) : -1;
        if (page >= 0) row = (static_cast<int64_t>(page) * p.v.Hkv + g) * rows + r;
      }
    }
    const int64_t first = __shfl_sync(0xffffffffu, row, x);
    const int live = __shfl_sync(0xffffffffu, seen, x);
    if (first < 0) continue;
    met = true;
    const size_t base = static_cast<size_t>(first) * D + lane;
    float k[R][CPL], v[R][CPL], sc[R];
#pragma unroll
    for (int j = 0; j < R; j++) {
      const size_t at = base + static_cast<size_t>(min(j, live - 1)) * D;
#pragma unroll
      for (int c = 0; c < CPL; c++) {
        k[j][c] = p.K[at + c * 32];
        v[j][c] = p.V[at + c * 32];
      }
    }
#pragma unroll
    for (int j = 0; j < R; j++) {
      sc[j] = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; c++) sc[j] = __fmaf_rn(q[c], k[j][c], sc[j]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
      for (int j = 0; j < R; j++) sc[j] = __fadd_rn(sc[j], __shfl_xor_sync(0xffffffffu, sc[j], o));
    float mn = m;
#pragma unroll
    for (int j = 0; j < R; j++) {
      sc[j] = __fmul_rn(sc[j], p.c);
      if (j < live) mn = fmaxf(mn, sc[j]);
    }
    const float alpha = mn == m ? 1.f : exp2f(__fsub_rn(m, mn));
    l = __fmul_rn(l, alpha);
#pragma unroll
    for (int c = 0; c < CPL; c++) acc[c] = __fmul_rn(acc[c], alpha);
#pragma unroll
    for (int j = 0; j < R; j++) {
      if (j >= live) continue;
      // (every score so far -inf: weights of 0, not of -inf - -inf)
      const float w = exp2f(__fsub_rn(sc[j], mn == -INFINITY ? 0.f : mn));
      l = __fadd_rn(l, w);
#pragma unroll
      for (int c = 0; c < CPL; c++) acc[c] = __fmaf_rn(w, v[j][c], acc[c]);
    }
    m = mn;
  }
#pragma unroll
  for (int c = 0; c < CPL; c++) acc_s[warp][c * 32 + lane] = acc[c];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  const bool any = __syncthreads_or(met) != 0;
  if (threadIdx.x >= D) return;
  float mn = -INFINITY, lt = 0.f, o = 0.f;
#pragma unroll
  for (int w = 0; w < kCudaWarps; w++) mn = fmaxf(mn, m_s[w]);
#pragma unroll
  for (int w = 0; w < kCudaWarps; w++) {
    const float f = exp2f(__fsub_rn(m_s[w], mn == -INFINITY ? 0.f : mn));
    lt = __fmaf_rn(f, l_s[w], lt);
    o = __fmaf_rn(f, acc_s[w][threadIdx.x], o);
  }
  const float y = any ? __fdiv_rn(o, lt) : 0.f;  // (no row seen: zeros; none with a score above -inf: 0 / 0, as the formula has it)
  const size_t at = row0 + threadIdx.x;
  p.out[at] = p.gate && any ? gate_mul(y, p.gate[at]) : y;
}

static tv_status launch_cuda(const PagedAttnCall& a, cudaStream_t st) {
  const tv_paged_layer* l = a.layer;
  PagedCudaParams p{};
  p.v = PagedView{paged_seqs(l, a.batch), a.sel, a.count, a.n_sel, l->Hkv};
  p.K = static_cast<const float*>(l->K);
  p.V = static_cast<const float*>(l->V);
  p.q = static_cast<const float*>(a.q);
  p.gate = static_cast<const float*>(a.gate);
  p.out = static_cast<float*>(a.out);
  p.Hq = l->Hq;
  p.G = l->Hq / l->Hkv;
  p.c = a.scale * 1.4426950408889634f;
  const dim3 g(l->Hq, a.batch->n_seq);
  switch (l->D) {
    case 64: launch_k(true, attn_paged_cuda_kernel<64>, g, dim3(32 * kCudaWarps), 0, st, p); break;
    case 128: launch_k(true, attn_paged_cuda_kernel<128>, g, dim3(32 * kCudaWarps), 0, st, p); break;
    default: launch_k(true, attn_paged_cuda_kernel<256>, g, dim3(32 * kCudaWarps), 0, st, p);
  }
  return launch_status();
}

static bool groups_ok(const tv_paged* b, const tv_paged_groups* g) {
  return g->n_group >= 1 && g->n_group <= b->n_seq && g->group_off && g->shared;
}

static tv_status paged_attn(const PagedAttnCall& a, cudaStream_t st) {
  const tv_paged_layer* l = a.layer;
  if (!l->K || !l->V || !a.q || !a.out || !(a.scale > 0.f) || !std::isfinite(a.scale)) return TV_ERR_ARG;
  if (!aligned16(a.q) || !aligned16(a.gate) || !aligned16(a.out) || !aligned16(a.ws)) return TV_ERR_ALIGN;
  // (a slot's heads, lists and lengths are read after others' rows are written; out may be gate)
  const tv_paged_groups* g = a.groups;
  const size_t n = bytes_of(a.batch->n_seq, static_cast<int64_t>(l->Hq) * l->D, l->dtype), units = static_cast<size_t>(a.batch->n_seq) * l->Hkv;
  const size_t pool = bytes_of(static_cast<int64_t>(l->n_pages) * l->Hkv * l->page, l->D, l->dtype);
  const Mem reads[] = {{a.q, n}, {a.gate == a.out ? nullptr : a.gate, n}, {l->K, pool}, {l->V, pool}, {a.sel, units * a.n_sel * 4}, {a.count, units * 4},
                       {g ? g->group_off : nullptr, g ? static_cast<size_t>(g->n_group + 1) * 4 : 0}, {g ? g->shared : nullptr, g ? static_cast<size_t>(g->n_group) * 4 : 0},
                       table_of(a.batch), lens_of(a.batch)};
  if (l->dtype != TV_BF16) return apart(a.batch->status, {{a.out, n}}, reads) ? launch_cuda(a, st) : TV_ERR_ARG;
  const size_t need = paged_attn_ws_bytes(l, a.batch, g);
  if (!apart(a.batch->status, {{a.out, n}, {a.ws, a.ws_bytes < need ? 0 : need}}, reads)) return TV_ERR_ARG;
  if (!a.ws || a.ws_bytes < need) return TV_ERR_WORKSPACE;
  return paged_attn_tc_launch(a, st);
}

}  // namespace tv

using namespace tv;

extern "C" size_t tv_paged_attn_workspace_bytes(const tv_paged_layer* l, const tv_paged* b, const tv_paged_groups* g) {
  if (paged_check(l, b) != TV_OK || l->dtype != TV_BF16 || (g && !groups_ok(b, g))) return 0;
  return paged_attn_ws_bytes(l, b, g);
}

extern "C" tv_status tv_paged_attn(const tv_paged_layer* l, const tv_paged* b, const tv_paged_groups* g, const void* q,
                                   const void* gate, void* out, float scale, void* ws, size_t ws_bytes, tv_stream stream) {
  const tv_status c = paged_check(l, b);
  if (c != TV_OK) return c;
  if (g && !groups_ok(b, g)) return TV_ERR_ARG;
  if (g && (!aligned16(g->group_off) || !aligned16(g->shared))) return TV_ERR_ALIGN;
  return paged_attn(PagedAttnCall{l, b, g, nullptr, nullptr, 0, q, gate, out, scale, ws, ws_bytes},
                    reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t tv_paged_attn_selected_workspace_bytes(const tv_paged_layer* l, const tv_paged* b, int32_t n_sel) {
  if (paged_check(l, b) != TV_OK || l->dtype != TV_BF16 || n_sel < 1 || n_sel > 4096) return 0;
  return paged_attn_ws_bytes(l, b, nullptr);
}

extern "C" tv_status tv_paged_attn_selected(const tv_paged_layer* l, const tv_paged* b, const int32_t* sel,
                                            const int32_t* count, int32_t n_sel, const void* q, const void* gate, void* out,
                                            float scale, void* ws, size_t ws_bytes, tv_stream stream) {
  const tv_status c = paged_check(l, b);
  if (c != TV_OK) return c;
  if (!sel || !count || n_sel < 1 || n_sel > 4096) return TV_ERR_ARG;
  if (!aligned16(sel) || !aligned16(count)) return TV_ERR_ALIGN;
  return paged_attn(PagedAttnCall{l, b, nullptr, sel, count, n_sel, q, gate, out, scale, ws, ws_bytes},
                    reinterpret_cast<cudaStream_t>(stream));
}
