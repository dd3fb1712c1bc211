// Head norms of queries and keys with the rotation in the same pass, for a
// tree's nodes, for decode tokens and for a prompt's packed rows; a prompt's
// keys and values go straight into the cache rows they belong to.
//
//   y = x / sqrt(mean(x^2) + eps) * w     (per head, w the query or key weights)
//   planes (j, j + rot/2) of y turn by pos * theta^(-2j/rot), the rest pass
//
// in fp32, rounded once to the row type.  The angle is carried in turns: the
// rate theta^(-2j/rot) / 2pi of plane j is a 64-bit binary fraction F_j formed
// on the host in fp64, and pos * F_j modulo 2^64 is the fraction of a turn to
// 2^-47 at any 20-bit position with three integer multiplies; its top 32 bits
// give sincospi's argument to half an fp32 step.  (fp64 sine and cosine per
// row, as tv_attn_rope forms them per row and head, would take longer here
// than the memory traffic: this GPU's fp64 rate is 1/60 of its fp32 rate.)
//
// A group of D/8 lanes owns a head, eight consecutive dimensions a lane, so a
// row moves with one 16-byte access a lane (two for fp32).  A warp keeps one
// row: its lanes form the row's sines and cosines once, in shared memory, and
// its groups walk a part of the row's heads, up to eight (fp32: four) loads in
// flight before the first is used.  Values are copied by warps of their own.
// Bound by HBM: each row is read once and written once.  A row's bits depend
// only on its own values and position, and the three forms run the same code,
// so verified, decoded and prompt rows are equal.
#include <cmath>

#include "prompt.cuh"

namespace tv {

constexpr int kMaxPlanes = 128;

struct NormRopeParams {
  PromptRows pr;  // prompt form; status and len in every form
  const void* q_raw;
  const void* k_raw;
  const void* v_raw;  // prompt form: appended to the value caches
  void* q;
  void* k;  // tree and decode forms
  void* K[TV_MAX_SEQ];
  void* V[TV_MAX_SEQ];
  const float* q_norm;  // null: no norm
  const float* k_norm;
  const int32_t* node_off;
  const void* meta;
  int form;  // 0 tree, 1 decode, 2 prompt
  int n_rows, n_seq, n_total, Hq, Hkv, rot, max_len, cap;
  int heads_per_warp, qk_parts, parts;  // warps a row: qk_parts for queries and keys, the rest for values
  float eps;
  uint64_t rate[kMaxPlanes];  // turns per position of each plane, as 64-bit fractions
};

// Eight values of a row as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void widen(float (&x)[8]) const { widen8(v, x); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(256) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPH = D / 8;                  // lanes per head
  constexpr int GPW = 32 / LPH;               // heads a warp holds at once
  constexpr int HB = sizeof(T) == 2 ? 8 : 4;  // loads a lane keeps in flight
  __shared__ __align__(16) float cs_s[8][D / 2], sn_s[8][D / 2];
  __shared__ __align__(16) float row_s[8][GPW][D];
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * 8 + wib;
  const int row = static_cast<int>(warp / p.parts), part = static_cast<int>(warp % p.parts);
  if (row >= p.n_rows) return;  // whole warps leave
  const int grp = lane / LPH, gl = lane % LPH, d0 = gl * 8;
  // this warp's heads; the first loads start before the row's place is known
  const bool vals = part >= p.qk_parts;
  const int h_first = (vals ? part - p.qk_parts : part) * p.heads_per_warp;
  const int h_end = min(vals ? p.Hkv : p.Hq + p.Hkv, h_first + p.heads_per_warp);
  const T* qr = static_cast<const T*>(p.q_raw) + static_cast<size_t>(row) * p.Hq * D + d0;
  const T* kr = static_cast<const T*>(vals ? p.v_raw : p.k_raw) + static_cast<size_t>(row) * p.Hkv * D + d0;
  auto src = [&](int h) { return vals ? kr + static_cast<size_t>(h) * D : h < p.Hq ? qr + static_cast<size_t>(h) * D : kr + static_cast<size_t>(h - p.Hq) * D; };
  Raw8<T> raw[HB];
#pragma unroll
  for (int i = 0; i < HB; i++) {
    const int h = h_first + i * GPW + grp;
    if (h < h_end) raw[i].load(src(h));
  }
  if (status_bad(p.pr.status)) return;
  // the row's sequence, position and (prompt) cache row
  int s, pos;
  if (p.form == 2) {
    const WarpSeqs w = load_seqs(p.pr, lane);
    if (w.code) {
      if (lane == 0) set_status(p.pr.status, w.code);
      return;
    }
    s = seq_of(w, p.pr, lane, row);
    if (s < 0) return;  // padding behind the last sequence
    pos = __shfl_sync(0xffffffffu, w.len, s) + row - __shfl_sync(0xffffffffu, w.off, s);
  } else {
    s = row;
    int depth = 0;
    if (p.form == 0) {
      s = 0;
      while (s < p.n_seq - 1 && row >= p.node_off[s + 1]) s++;
      depth = meta_view(const_cast<void*>(p.meta), p.n_total).depth[row];
    }
    const int len = p.pr.len[s];
    if (len < 0 || len > p.max_len) {
      if (lane == 0) set_status(p.pr.status, TV_ERR_LEN);
      return;
    }
    pos = len + depth;
  }
  if (vals) {  // bit copies into the value cache
    T* dst = static_cast<T*>(p.V[s]) + static_cast<size_t>(pos) * D + d0;
    for (int h0 = h_first;;) {
#pragma unroll
      for (int i = 0; i < HB; i++) {
        const int h = h0 + i * GPW + grp;
        if (h < h_end) raw[i].store(dst + static_cast<size_t>(h) * p.cap * D);
      }
      h0 += HB * GPW;
      if (h0 >= h_end) return;
#pragma unroll
      for (int i = 0; i < HB; i++) {
        const int h = h0 + i * GPW + grp;
        if (h < h_end) raw[i].load(src(h));
      }
    }
  }
  const int half = p.rot >> 1;
  for (int j = lane; j < half; j += 32) {
    const uint64_t turn = static_cast<uint64_t>(pos) * p.rate[j];
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;  // half turns
    sincospif(x, &sn_s[wib][j], &cs_s[wib][j]);
  }
  __syncwarp();
  // this lane's rotation factors: dimension d < rot belongs to plane d mod half;
  // the first half of a plane takes -sin of its partner, the second +sin
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const int d = d0 + e;
    const int j = d < half ? d : d - half;
    cs[e] = d < p.rot ? cs_s[wib][j] : 1.f;
    sn[e] = d < p.rot ? (d < half ? -sn_s[wib][j] : sn_s[wib][j]) : 0.f;
  }
  float wq[8], wk[8];
  if (p.q_norm) {
    load8(p.q_norm + d0, wq);
    load8(p.k_norm + d0, wk);
  }
  const bool aligned = half % 8 == 0;  // a lane's eight partners sit in one other lane
  const int partner = d0 < half ? gl + half / 8 : (d0 < p.rot ? gl - half / 8 : gl);
  for (int h0 = h_first; h0 < h_end; h0 += HB * GPW) {
    if (h0 != h_first) {
#pragma unroll
      for (int i = 0; i < HB; i++) {
        const int h = h0 + i * GPW + grp;
        if (h < h_end) raw[i].load(src(h));
      }
    }
#pragma unroll
    for (int i = 0; i < HB; i++) {
      if (h0 + i * GPW >= h_end) break;  // the whole warp
      const int h = h0 + i * GPW + grp;
      const bool act = h < h_end, is_q = h < p.Hq;
      float x[8];
      raw[i].widen(x);
      if (p.q_norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e++) ss = __fmaf_rn(x[e], x[e], ss);
#pragma unroll
        for (int o = LPH / 2; o >= 1; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
        const float inv = rsqrtf(__fmaf_rn(ss, 1.f / D, p.eps));  // 2 units in the last place, far below the output's rounding
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = __fmul_rn(__fmul_rn(x[e], inv), is_q ? wq[e] : wk[e]);
      }
      float y[8];
      if (aligned) {
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = __shfl_sync(0xffffffffu, x[e], partner, LPH);
      } else {
        store8(&row_s[wib][grp][d0], x);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int d = d0 + e;
          y[e] = d < p.rot ? row_s[wib][grp][d < half ? d + half : d - half] : 0.f;
        }
        __syncwarp();
      }
      // dimensions past rot pass bit for bit (0 times a partner would not, were it infinite)
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (d0 + e < p.rot) x[e] = __fmaf_rn(x[e], cs[e], __fmul_rn(y[e], sn[e]));
      if (act) {
        T* dst;
        if (is_q) dst = static_cast<T*>(p.q) + (static_cast<size_t>(row) * p.Hq + h) * D;
        else if (p.form != 2) dst = static_cast<T*>(p.k) + (static_cast<size_t>(row) * p.Hkv + h - p.Hq) * D;
        else dst = static_cast<T*>(p.K[s]) + (static_cast<size_t>(h - p.Hq) * p.cap + pos) * D;
        store8(dst + d0, x);
      }
    }
  }
}

// What the calls share: shape checks, rates, launch.
static tv_status norm_rope_launch(const tv_attn_layer* l, NormRopeParams& p, const float* q_norm, const float* k_norm,
                                  float eps, int rot, float theta, cudaStream_t st) {
  p.q_norm = q_norm;
  p.k_norm = k_norm;
  p.eps = eps;
  p.rot = rot;
  p.Hq = l->Hq;
  p.Hkv = l->Hkv;
  p.cap = l->cap;
  for (int j = 0; j < rot / 2; j++) {
    const double turns = std::pow(static_cast<double>(theta), -2.0 * j / rot) * 0.15915494309189533577;  // / 2 pi
    p.rate[j] = static_cast<uint64_t>(std::ldexp(turns, 64));
  }
  // heads a warp walks: one round of its loads with many rows (the row's sines
  // are formed once for them), fewer while the launch would leave SMs without work
  const int gpw = 256 / l->D;
  int hpw = gpw * (l->dtype == TV_BF16 ? 8 : 4);
  auto split = [&]() {
    p.qk_parts = (l->Hq + l->Hkv + hpw - 1) / hpw;
    p.parts = p.qk_parts + (p.form == 2 ? (l->Hkv + hpw - 1) / hpw : 0);
    return static_cast<int64_t>(p.n_rows) * p.parts;
  };
  while (hpw > gpw && split() < 16 * num_sms()) hpw >>= 1;
  p.heads_per_warp = hpw;
  const int64_t warps = split();
  const int64_t grid = (warps + 7) / 8;
  if (grid > 0x7fffffff) return TV_ERR_SHAPE;
  const dim3 g(static_cast<unsigned>(grid));
  const bool bf = l->dtype == TV_BF16;
  switch (l->D) {
    case 64:
      if (bf) norm_rope_kernel<__nv_bfloat16, 64><<<g, 256, 0, st>>>(p); else norm_rope_kernel<float, 64><<<g, 256, 0, st>>>(p);
      break;
    case 128:
      if (bf) norm_rope_kernel<__nv_bfloat16, 128><<<g, 256, 0, st>>>(p); else norm_rope_kernel<float, 128><<<g, 256, 0, st>>>(p);
      break;
    default:
      if (bf) norm_rope_kernel<__nv_bfloat16, 256><<<g, 256, 0, st>>>(p); else norm_rope_kernel<float, 256><<<g, 256, 0, st>>>(p);
  }
  return launch_status();
}

static tv_status norm_rope_check(const tv_attn_layer* l, int32_t max_len, const float* q_norm, const float* k_norm,
                                 float eps, int32_t rot, float theta) {
  if (l->dtype != TV_F32 && l->dtype != TV_BF16) return TV_ERR_DTYPE;
  if (l->Hq < 1 || l->Hkv < 1 || l->Hq % l->Hkv || l->Hq > 4096 || (l->D != 64 && l->D != 128 && l->D != 256))
    return TV_ERR_SHAPE;
  if (l->cap < 1 || max_len < 0 || max_len > l->cap) return TV_ERR_ARG;
  if (rot < 0 || rot > l->D || rot % 2 || !(theta > 1.f) || !std::isfinite(theta)) return TV_ERR_ARG;
  if ((q_norm == nullptr) != (k_norm == nullptr)) return TV_ERR_ARG;
  if (q_norm && (!(eps > 0.f) || !std::isfinite(eps))) return TV_ERR_ARG;
  if (!aligned16(q_norm) || !aligned16(k_norm)) return TV_ERR_ALIGN;
  return TV_OK;
}

}  // namespace tv

using namespace tv;

extern "C" tv_status tv_attn_norm_rope(const tv_attn_layer* l, const tv_tree* t, int32_t n_seq, const int32_t* len,
                                       int32_t max_len, const float* q_norm, const float* k_norm, float eps,
                                       int32_t rot_dims, float theta, const void* q_raw, const void* k_raw, void* q,
                                       void* k, int32_t* status, tv_stream stream) {
  if (!l || !len || !q_raw || !k_raw || !q || !k) return TV_ERR_ARG;
  const tv_status c = norm_rope_check(l, max_len, q_norm, k_norm, eps, rot_dims, theta);
  if (c != TV_OK) return c;
  if (!aligned16(len) || !aligned16(q_raw) || !aligned16(k_raw) || !aligned16(q) || !aligned16(k)) return TV_ERR_ALIGN;
  NormRopeParams p{};
  if (t) {
    if (!tree_ok(t)) return TV_ERR_ARG;
    p.form = 0;
    p.n_rows = p.n_total = t->n_total;
    p.n_seq = t->n_seq;
    p.node_off = t->node_off;
    p.meta = t->meta;
    p.pr.status = t->status;
  } else {
    if (n_seq < 1 || n_seq > TV_MAX_SEQ || !status) return TV_ERR_ARG;
    if (!aligned16(status)) return TV_ERR_ALIGN;
    p.form = 1;
    p.n_rows = p.n_seq = n_seq;
    p.pr.status = status;
  }
  p.pr.len = len;
  p.max_len = max_len;
  p.q_raw = q_raw;
  p.k_raw = k_raw;
  p.q = q;
  p.k = k;
  return norm_rope_launch(l, p, q_norm, k_norm, eps, rot_dims, theta, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" tv_status tv_attn_prompt_front(const tv_attn_layer* l, const tv_prompt* pr, const int32_t* len,
                                          int32_t max_len, const float* q_norm, const float* k_norm, float eps,
                                          int32_t rot_dims, float theta, const void* q_raw, const void* k_raw,
                                          const void* v, void* q, tv_stream stream) {
  if (!l || !prompt_ok(pr) || !len || !l->K || !l->V) return TV_ERR_ARG;
  const tv_status c = norm_rope_check(l, max_len, q_norm, k_norm, eps, rot_dims, theta);
  if (c != TV_OK) return c;
  NormRopeParams p{};
  for (int s = 0; s < pr->n_seq; s++) {
    if (!l->K[s] || !l->V[s]) return TV_ERR_ARG;
    if (!aligned16(l->K[s]) || !aligned16(l->V[s])) return TV_ERR_ALIGN;
    p.K[s] = l->K[s];
    p.V[s] = l->V[s];
  }
  if (!aligned16(len)) return TV_ERR_ALIGN;
  if (pr->n_total == 0) return TV_OK;
  if (!q_raw || !k_raw || !v || !q) return TV_ERR_ARG;
  if (!aligned16(q_raw) || !aligned16(k_raw) || !aligned16(v) || !aligned16(q)) return TV_ERR_ALIGN;
  p.form = 2;
  p.pr = prompt_rows(pr, len, max_len, l->cap);
  p.n_rows = p.n_total = pr->n_total;
  p.n_seq = pr->n_seq;
  p.max_len = max_len;
  p.q_raw = q_raw;
  p.k_raw = k_raw;
  p.v_raw = v;
  p.q = q;
  return norm_rope_launch(l, p, q_norm, k_norm, eps, rot_dims, theta, reinterpret_cast<cudaStream_t>(stream));
}
