// Gated DeltaNet front end over a prompt's packed rows: the short convolution
// along each sequence (continuing from its committed tail), SiLU, the q/k head
// norms and the gates; the tails move on to the sequence's last W-1 raw inputs.  Formulas as in front_gdn.cu.
//
// A group of DH/8 lanes owns one head (eight consecutive channels a lane, one
// 16-byte access a row) and walks a strip of consecutive rows of one sequence, a
// few loaded ahead, with the W-1 rows before the current one in registers; only
// a strip's last W-1 rows are read twice (by it and the next strip).  Taps run
// in fp32 in order, oldest first, as in the tree and decode forms.
//
// Bound by HBM, every raw channel read once and written once, with the issue
// slots behind (45 % at 58 % of DRAM throughput).  16 + 48 heads of 128,
// W = 4: 8,192 rows (342 MB) 64.8 us, 5.3 TB/s, 0.79 of a copy's rate; 731 rows
// in four sequences 10.4 us, two thirds of that one strip's latency.
#include "prompt.cuh"
#include "front_gdn.cuh"
#include "launchers.hpp"
#include "ptx.cuh"

namespace tv {

struct GdnPromptFrontParams {
  PromptRows pr;
  const void* x;
  const float* a_raw;
  const float* b_raw;
  void* q;
  void* k;
  void* v;
  float* alpha;
  float* beta;
  const float* wconv;
  void* tail[TV_MAX_SEQ];
  int Hk, Hv, C, rows, strips, head_warps;
};

// Eight channels of a row, as packed fp32 pairs.
template <typename T>
struct Row8;
template <>
struct Row8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ f2_t pair(int i) const { return f2_from_bf16x2(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w); }
};
template <>
struct Row8<float> {
  ulonglong2 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const ulonglong2*>(p)[0];
    b = reinterpret_cast<const ulonglong2*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<ulonglong2*>(p)[0] = a;
    reinterpret_cast<ulonglong2*>(p)[1] = b;
  }
  __device__ __forceinline__ f2_t pair(int i) const { return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? b.x : b.y; }
};

// SiLU of a pair, x / (1 + e^-x); from -87 on 0, from -inf NaN, as the library's
// other paths have it.
__device__ __forceinline__ f2_t silu2(f2_t x) {
  float a, b;
  f2_unpack(f2_mul(x, f2_dup(-1.4426950408889634f)), a, b);
  f2_unpack(f2_add(f2_pack(ex2_approx(a), ex2_approx(b)), f2_dup(1.f)), a, b);
  return f2_mul(x, f2_pack(rcp_approx(a), rcp_approx(b)));
}

// What a width needs in registers: the window as a ring of RING rows (even for
// widths over 2, so that rows go two at a time), groups of GROUP rows loaded one
// ahead, and the CTAs of four warps that an SM then holds.
template <typename T, int W>
struct Width {
  static constexpr int RING = W <= 2 ? W : (W + 1) / 2 * 2;
  static constexpr int GROUP = RING < 4 ? 4 : RING;
  static constexpr int CTAS = sizeof(T) == 4 ? (W <= 4 ? 2 : 1) : W <= 4 ? 4 : W <= 6 ? 3 : 2;
};

template <typename T, int DH, int W>
__global__ void __launch_bounds__(128, Width<T, W>::CTAS) gdn_prompt_front_kernel(const __grid_constant__ GdnPromptFrontParams p) {
  constexpr int LPH = DH / 8, HPW = 32 / LPH;  // lanes a head, heads a warp
  constexpr int RING = Width<T, W>::RING, GROUP = Width<T, W>::GROUP;
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  pdl_wait();
  if (status_bad(p.pr.status)) return;
  const WarpSeqs w = load_seqs(p.pr, lane);
  if (w.code) {
    if (lane == 0) set_status(p.pr.status, w.code);
    return;
  }
  const int n_live = __shfl_sync(0xffffffffu, w.off, p.pr.n_seq);
  const int64_t conv_warps = static_cast<int64_t>(p.strips) * p.head_warps;
  if (warp >= conv_warps) {  // gates: a thread a (row, value head)
    const int64_t i = (warp - conv_warps) * 32 + lane;
    if (i < static_cast<int64_t>(n_live) * p.Hv) front_gates(p.a_raw[i], p.b_raw[i], p.alpha[i], p.beta[i]);
    return;
  }
  const int units = 2 * p.Hk + p.Hv;
  int strips;
  const int base = strip_base(w, p.pr, lane, p.rows, strips);
  const int strip = static_cast<int>(warp / p.head_warps);
  if (strip >= strips) return;
  const int s = strip_seq(w, p.pr, lane, base, strip);
  const int off = __shfl_sync(0xffffffffu, w.off, s), end = __shfl_sync(0xffffffffu, w.end, s);
  const int r0 = off + (strip - __shfl_sync(0xffffffffu, base, s)) * p.rows, r1 = min(r0 + p.rows, end);
  const int u = static_cast<int>(warp % p.head_warps) * HPW + lane / LPH;
  const bool act = u < units;
  const int c0 = (act ? u : 0) * DH + (lane % LPH) * 8;  // dk = dv = DH: head u's channels start at u * DH
  f2_t tap[W][4];  // tap[j] of channels c0 + 2e, c0 + 2e + 1: wconv[c][j]
  {
    float f[8 * W];  // the lane's eight channels' taps lie side by side
#pragma unroll
    for (int i = 0; i < 2 * W; i++) {
      const float4 a = reinterpret_cast<const float4*>(p.wconv + static_cast<size_t>(c0) * W)[i];
      f[4 * i] = a.x;
      f[4 * i + 1] = a.y;
      f[4 * i + 2] = a.z;
      f[4 * i + 3] = a.w;
    }
#pragma unroll
    for (int j = 0; j < W; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) tap[j][e] = f2_pack(f[2 * e * W + j], f[(2 * e + 1) * W + j]);
  }
  const T* x = static_cast<const T*>(p.x) + c0;
  const bool norm = u < 2 * p.Hk;
  const bool any_norm = __any_sync(0xffffffffu, norm);
  T* dst;
  size_t dstride;
  if (u < p.Hk) {
    dst = static_cast<T*>(p.q) + c0;
    dstride = static_cast<size_t>(p.Hk) * DH;
  } else if (u < 2 * p.Hk) {
    dst = static_cast<T*>(p.k) + (c0 - p.Hk * DH);
    dstride = static_cast<size_t>(p.Hk) * DH;
  } else {
    dst = static_cast<T*>(p.v) + (c0 - 2 * p.Hk * DH);
    dstride = static_cast<size_t>(p.Hv) * DH;
  }
  // win[(r + j) % RING]: the input j - (W-1) rows from row r of the strip, so that
  // a step overwrites the oldest and nothing moves
  f2_t win[RING][4];
  Row8<T> cur[GROUP], next[GROUP];  // rows of this group and of the one after, in flight
  auto fetch = [&](int rg, Row8<T>* to) {
#pragma unroll
    for (int u = 0; u < GROUP; u++) to[u].load(x + static_cast<size_t>(min(rg + u, r1 - 1)) * p.C);
  };
  fetch(r0, next);
  // The rows before the strip: the tail's for a sequence's first strip, which
  // has the W-1 rows that read it, so that it alone then moves the tail on.
  T* tail = static_cast<T*>(p.tail[s]) + c0;
#pragma unroll
  for (int j = 0; j < W - 1; j++) {
    Row8<T> old;
    old.load(r0 > off ? x + static_cast<size_t>(r0 + j - (W - 1)) * p.C : tail + static_cast<size_t>(j) * p.C);
#pragma unroll
    for (int e = 0; e < 4; e++) win[j][e] = old.pair(e);
  }
  if (r0 == off && act) {
    for (int j = 0; j < W - 1; j++) {  // ascending: row j comes from the prompt or from a later row of the old tail
      const int m = end - off + j - (W - 1);
      Row8<T> to;
      to.load(m >= 0 ? x + static_cast<size_t>(off + m) * p.C : tail + static_cast<size_t>(m + W - 1) * p.C);
      to.store(tail + static_cast<size_t>(j) * p.C);
    }
  }
  for (int rg = r0; rg < r1; rg += GROUP) {
#pragma unroll
    for (int u = 0; u < GROUP; u++) cur[u] = next[u];
    if (rg + GROUP < r1) fetch(rg + GROUP, next);
    // row u of the group: the window takes it in, then convolution and SiLU
    auto conv = [&](int u, f2_t (&acc)[4]) {
#pragma unroll
      for (int e = 0; e < 4; e++) {
        win[(u + W - 1) % RING][e] = cur[u].pair(e);
        acc[e] = 0ull;
      }
#pragma unroll
      for (int j = 0; j < W; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = f2_fma(tap[j][e], win[(u + j) % RING][e], acc[e]);
#pragma unroll
      for (int e = 0; e < 4; e++) acc[e] = silu2(acc[e]);
    };
    auto squares = [&](const f2_t (&acc)[4]) {
      f2_t ss = 0ull;
#pragma unroll
      for (int e = 0; e < 4; e++) ss = f2_fma(acc[e], acc[e], ss);
      return f2_hsum(ss);
    };
    auto put = [&](int r, f2_t (&acc)[4], float ss) {
      if (any_norm) {
        const f2_t sc = f2_dup(norm ? rsqrtf(__fadd_rn(ss, kNormEps)) : 1.f);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = f2_mul(acc[e], sc);
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; e++) f2_unpack(acc[e], y[2 * e], y[2 * e + 1]);
      if (act) store8(dst + static_cast<size_t>(r) * dstride, y);
    };
    if (rg + GROUP <= r1) {  // a whole group: two rows side by side
#pragma unroll
      for (int u = 0; u < GROUP; u += 2) {
        f2_t acc[2][4];
        float ss[2];
        conv(u, acc[0]);
        conv(u + 1, acc[1]);
        if (any_norm) {
          ss[0] = squares(acc[0]);
          ss[1] = squares(acc[1]);
#pragma unroll
          for (int o = LPH / 2; o >= 1; o >>= 1)
#pragma unroll
            for (int v = 0; v < 2; v++) ss[v] = __fadd_rn(ss[v], __shfl_xor_sync(0xffffffffu, ss[v], o));
        }
        put(rg + u, acc[0], ss[0]);
        put(rg + u + 1, acc[1], ss[1]);
      }
      continue;
    }
#pragma unroll
    for (int u = 0; u < GROUP; u++) {
      const int r = rg + u;
      if (r >= r1) break;
      f2_t acc[4];
      conv(u, acc);
      float ss = 0.f;
      if (any_norm) {
        ss = squares(acc);
#pragma unroll
        for (int o = LPH / 2; o >= 1; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
      }
      put(r, acc, ss);
    }
  }
}

// Rows a warp walks: at most 64, in as even a number of waves as whole groups
// allow, since a strip loads the taps and reads W-1 rows twice; never fewer than
// read a tail.  At W = 4 and 16 + 48 heads of 128, 731 rows take 13.5 us in strips
// of 12, 15.2 of 8, 16.9 of 32; 8,192 rows 68.8 us in strips of 48 (three even
// waves), 70.8 of 32, 74.9 of 64.
template <typename T, int DH, int W>
static tv_status launch_width(GdnPromptFrontParams& p, cudaStream_t st) {
  using C = Width<T, W>;
  const int64_t n = p.pr.n_total, work = n * p.head_warps, slots = static_cast<int64_t>(4) * C::CTAS * num_sms();
  const int64_t waves = (work + slots * 64 - 1) / (slots * 64), even = (work + slots * waves - 1) / (slots * waves);
  p.rows = static_cast<int>(((even > W - 1 ? even : W - 1) + C::GROUP - 1) / C::GROUP * C::GROUP);
  p.strips = static_cast<int>(n / p.rows) + p.pr.n_seq;
  const int64_t warps = static_cast<int64_t>(p.strips) * p.head_warps + (n * p.Hv + 31) / 32, grid = (warps + 3) / 4;
  if (grid > 0x7fffffff) return TV_ERR_SHAPE;
  launch_k(true, gdn_prompt_front_kernel<T, DH, W>, dim3(static_cast<unsigned>(grid)), dim3(128), 0, st, p);
  return launch_status();
}
// A kernel of its own for every width: taps, window and rows ahead stay in
// registers at fixed places (one for any width, without that, took 184.7 us
// against 66.9 at W = 4 and 8,192 rows).
template <typename T, int DH>
static tv_status launch_prompt_front(GdnPromptFrontParams& p, int W, cudaStream_t st) {
  static_assert(kMaxConvWidth == 8, "widths");
  switch (W) {
    case 1: return launch_width<T, DH, 1>(p, st);
    case 2: return launch_width<T, DH, 2>(p, st);
    case 3: return launch_width<T, DH, 3>(p, st);
    case 4: return launch_width<T, DH, 4>(p, st);
    case 5: return launch_width<T, DH, 5>(p, st);
    case 6: return launch_width<T, DH, 6>(p, st);
    case 7: return launch_width<T, DH, 7>(p, st);
    default: return launch_width<T, DH, 8>(p, st);
  }
}

}  // namespace tv

using namespace tv;

extern "C" tv_status tv_gdn_prompt_front(const tv_gdn_front_layer* f, const tv_prompt* pr, const void* x,
                                         const float* a_raw, const float* b_raw, void* q, void* k, void* v,
                                         float* alpha, float* beta, tv_stream stream) {
  if (!f || !prompt_ok(pr)) return TV_ERR_ARG;
  if (f->dtype != TV_F32 && f->dtype != TV_BF16) return TV_ERR_DTYPE;
  if (!front_layer_ok(f) || f->Hk > 4096 || f->Hv > 4096) return TV_ERR_SHAPE;
  GdnPromptFrontParams p{};
  for (int s = 0; s < pr->n_seq; s++) {
    if (f->width > 1 && !f->tail[s]) return TV_ERR_ARG;
    if (!aligned16(f->tail[s])) return TV_ERR_ALIGN;
    p.tail[s] = f->tail[s];
  }
  if (pr->n_total == 0) return TV_OK;
  if (!x || !a_raw || !b_raw || !q || !k || !v || !alpha || !beta) return TV_ERR_ARG;
  if (!aligned16(x) || !aligned16(a_raw) || !aligned16(b_raw) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(alpha) || !aligned16(beta) || !aligned16(f->wconv))
    return TV_ERR_ALIGN;
  const int64_t kc = static_cast<int64_t>(f->Hk) * f->dk, vc = static_cast<int64_t>(f->Hv) * f->dv, C = 2 * kc + vc;
  const int64_t n = pr->n_total, hv = f->Hv;
  if (overlap(x, q, n, C, kc, f->dtype) || overlap(x, k, n, C, kc, f->dtype) || overlap(x, v, n, C, vc, f->dtype))
    return TV_ERR_ARG;  // a row is read again by the rows after it
  const float* const raw[2] = {a_raw, b_raw};
  float* const gates[2] = {alpha, beta};
  for (int i = 0; i < 2; i++) {  // (gates may be formed in place: a thread reads its two raw values first)
    if (overlap(raw[i], q, n, hv, kc, TV_F32, f->dtype) || overlap(raw[i], k, n, hv, kc, TV_F32, f->dtype) ||
        overlap(raw[i], v, n, hv, vc, TV_F32, f->dtype) || overlap(gates[i], x, n, hv, C, TV_F32, f->dtype))
      return TV_ERR_ARG;
    for (int j = 0; j < 2; j++)
      if (raw[i] != gates[j] && overlap(raw[i], gates[j], n, hv, hv, TV_F32)) return TV_ERR_ARG;
  }
  p.pr = prompt_rows(pr, nullptr, 0, 0);
  p.x = x; p.a_raw = a_raw; p.b_raw = b_raw; p.q = q; p.k = k; p.v = v; p.alpha = alpha; p.beta = beta;
  p.wconv = f->wconv;
  p.Hk = f->Hk; p.Hv = f->Hv;
  p.C = 2 * f->Hk * f->dk + f->Hv * f->dv;
  const int hpw = 256 / f->dk;
  p.head_warps = (2 * f->Hk + f->Hv + hpw - 1) / hpw;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = f->dtype == TV_BF16;
  if (f->dk == 128) return bf ? launch_prompt_front<__nv_bfloat16, 128>(p, f->width, st) : launch_prompt_front<float, 128>(p, f->width, st);
  return bf ? launch_prompt_front<__nv_bfloat16, 64>(p, f->width, st) : launch_prompt_front<float, 64>(p, f->width, st);
}
