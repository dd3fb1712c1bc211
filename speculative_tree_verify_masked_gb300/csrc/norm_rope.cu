// Head norms of queries and keys with the rotation in the same pass, for a
// tree's nodes, for decode tokens and for a prompt's packed rows; a prompt's
// keys and values go straight into the cache rows they belong to, contiguous
// or in pages.
//
//   y = x / sqrt(mean(x^2) + eps) * w     (per head, w the query or key weights)
//   planes (j, j + rot/2) of y turn by pos * theta^(-2j/rot), the rest pass
//
// in fp32, rounded once to the row type.  The angle is carried in turns: the
// rate theta^(-2j/rot) / 2pi of plane j is a 64-bit binary fraction F_j formed
// on the host in fp64, and pos * F_j modulo 2^64 is the fraction of a turn, with
// three integer multiplies and nothing lost at any 20-bit position; its top 32 bits
// give sincospi's argument to half an fp32 step.  (fp64 sine and cosine per
// row, as tv_attn_rope forms them per row and head, would take longer here
// than the memory traffic: this GPU's fp64 rate is 1/60 of its fp32 rate.)
//
// A group of D/8 lanes owns a head, eight consecutive dimensions a lane, so a
// row moves with one 16-byte access a lane (two for fp32).  A warp keeps one
// row and one kind of head (query, key or value): its lanes form the row's
// sines and cosines once, and its groups walk a part of the heads, four at a
// time with the next four in flight.  Norm weights and rotation are one
// pair of factors a dimension, y_d = inv (x_d (w_d cos) + x_p (w_p sin)), formed
// once a warp, so a head costs two packed products a pair of dimensions and its
// partners travel unwidened.
// A row's bits depend only on its own values and position, and all forms
// run the same code, so verified, decoded, prompt and paged rows are equal.
// (Pages allow 2^30 positions: the fractions' fp64 then leaves up to 2^-24 of a turn.)
//
// Bound by HBM, each row read once and written once, with the issue slots close
// behind (59 % at 53 % of DRAM throughput).  8,192 prompt rows of 24 + 4 + 4
// heads of 256 (268 MB): 51.4 us, 5.2 TB/s, 0.78 of a copy's rate; four decode
// tokens: 3.5 us, a launch's latency.  Into pages of 16 rows, 4,629 rows of four
// prompts (152 MB) 31.2 us, 4.9 TB/s, 0.73 of a copy's rate: a row's slot and page are two
// more reads in a row before its first store; 192 decode rows 4.3 us.  (Up to 16, 12 or 8 heads a
// warp for more warps: 34.4, 34.0 and 37.7 us.)
#include <cmath>

#include "paged.cuh"
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
  PagedSeqs pg;  // paged form: K[0] and V[0] are the pools
  int form;  // 0 tree, 1 decode, 2 prompt, 3 paged (a row a slot), 4 paged (packed rows)
  int n_rows, n_seq, n_total, Hq, Hkv, rot, max_len, cap;
  int heads_per_warp, q_parts, k_parts, parts;  // warps a row: for queries, for keys, the rest for values
  float eps;
  uint64_t rate[kMaxPlanes];  // turns per position of each plane, as 64-bit fractions
};

// Eight values of a row as they lie in memory, and as packed fp32 pairs.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  static constexpr int W = 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ __forceinline__ f2_t pair(int i) const { return f2_from_bf16x2(w[i]); }
};
template <>
struct Raw8<float> {
  static constexpr int W = 8;
  uint32_t w[W];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ f2_t pair(int i) const { return f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])); }
};

// The slot that packed row `row` belongs to, where its rows start and the rows it holds
// already: for up to 31 slots from one round of loads, a lane a slot; else by two looks
// at 32 offsets side by side.  (Offsets that fall are found by the rows that meet them, and
// by no other: every row checks its own slot's.)
struct PagedRow {
  int s, off, len;  // s -1: padding behind the last row, or what is not allowed
};
__device__ __forceinline__ PagedRow paged_row(const PagedSeqs& b, const int32_t* row_off, int n_total, int n_max, int row, int lane) {
  PagedRow r{-1, 0, 0};
  int s, start, end, all, zero, len;
  if (b.n_seq < 32) {
    const int o = row_off[min(lane, b.n_seq)], l = b.len[min(lane, b.n_seq - 1)];
    const unsigned m = __ballot_sync(0xffffffffu, lane <= b.n_seq && o <= row);
    s = m ? 31 - __clz(static_cast<int>(m)) : 0;
    zero = __shfl_sync(0xffffffffu, o, 0);
    all = __shfl_sync(0xffffffffu, o, b.n_seq);
    start = __shfl_sync(0xffffffffu, o, s);
    end = __shfl_sync(0xffffffffu, o, min(s + 1, b.n_seq));
    len = __shfl_sync(0xffffffffu, l, min(s, b.n_seq - 1));
  } else {
    s = 0;
    for (int step = 32;; step = 1) {
      const int i = s + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, i <= b.n_seq && row_off[i] <= row);
      s += m ? (31 - __clz(static_cast<int>(m))) * step : 0;
      if (step == 1) break;
    }
    // (the last of 32 looks may be followed by a boundary: n_seq = 32 k)
    if (s < b.n_seq && row_off[s + 1] <= row) s++;
    zero = row_off[0];
    all = row_off[b.n_seq];
    start = row_off[s];
    end = row_off[min(s + 1, b.n_seq)];
    len = b.len[min(s, b.n_seq - 1)];
  }
  int code = 0;
  if (zero != 0 || all > n_total) code = TV_ERR_ROWS;
  else if (s >= b.n_seq) return r;  // padding
  else if (end - start < 0 || end - start > n_max || row < start || row >= end || len == -1) code = TV_ERR_ROWS;
  else if (len < -1 || len > b.max_len) code = TV_ERR_LEN;
  if (code) {
    if (lane == 0) set_status(b.status, code);
    return r;
  }
  r.s = s;
  r.off = start;
  r.len = len;
  return r;
}

template <typename T, int D, bool PAGED>
__global__ void __launch_bounds__(128, sizeof(T) == 2 ? 5 : 4) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPH = D / 8;                  // lanes per head
  constexpr int GPW = 32 / LPH;               // heads a warp holds at once
  constexpr int HB = 4;                       // heads a group works on at once
  __shared__ __align__(16) float cs_s[4][D / 2], sn_s[4][D / 2];
  __shared__ __align__(16) float row_s[4][GPW][D];
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * 4 + wib, part = blockIdx.y;  // a CTA's warps have one kind of head: they end together
  pdl_wait();
  if (row >= p.n_rows) return;  // whole warps leave
  const int grp = lane / LPH, gl = lane % LPH, d0 = gl * 8;
  // this warp's heads; the first loads start before the row's place is known
  const int kind = part < p.q_parts ? 0 : part < p.q_parts + p.k_parts ? 1 : 2;  // query, key, value
  const int H = kind == 0 ? p.Hq : p.Hkv;
  const int h_first = (part - (kind == 0 ? 0 : kind == 1 ? p.q_parts : p.q_parts + p.k_parts)) * p.heads_per_warp + grp;
  const int h_end = min(H, h_first - grp + p.heads_per_warp);
  const T* src = static_cast<const T*>(kind == 0 ? p.q_raw : kind == 1 ? p.k_raw : p.v_raw) + static_cast<size_t>(row) * H * D + d0;
  Raw8<T> raw[HB];
  auto fetch = [&](int h0, Raw8<T> (&to)[HB]) {
#pragma unroll
    for (int i = 0; i < HB; i++) to[i].load(src + static_cast<size_t>(min(h0 + i * GPW, h_end - 1)) * D);
  };
  fetch(h_first, raw);
  // the row's sequence, position and (prompt) cache row
  const bool bad = PAGED ? status_set(p.pr.status) : status_bad(p.pr.status);
  int s, pos;
  if constexpr (PAGED) {
    if (bad) return;
    s = row;
    if (p.form == 4) {
      const PagedRow r = paged_row(p.pg, p.pr.row_off, p.n_total, p.pr.n_max, row, lane);
      if (r.s < 0) return;
      s = r.s;
      pos = r.len + row - r.off;
    } else {
      pos = paged_len(p.pg, s);
      if (pos < 0) return;
    }
    if ((pos >> p.pg.shift) >= p.pg.cols) {
      if (lane == 0) set_status(p.pr.status, TV_ERR_CAPACITY);
      return;
    }
  } else if (p.form == 2) {
    const WarpSeqs w = load_seqs(p.pr, lane);
    if (w.code || bad) {
      if (lane == 0 && w.code) set_status(p.pr.status, w.code);
      return;
    }
    s = seq_of(w, p.pr, lane, row);
    if (s < 0) return;  // padding behind the last sequence
    pos = __shfl_sync(0xffffffffu, w.len, s) + row - __shfl_sync(0xffffffffu, w.off, s);
  } else {
    if (bad) return;
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
  // where the heads go: head h at dst + h * step
  T* dst;
  size_t step = D;
  if (kind == 0) {
    dst = static_cast<T*>(p.q) + static_cast<size_t>(row) * H * D + d0;
  } else if (PAGED) {
    const int page = page_at(p.pg, s, pos >> p.pg.shift), r = pos & ((1 << p.pg.shift) - 1);
    if (page < 0) return;
    dst = static_cast<T*>(kind == 1 ? p.K[0] : p.V[0]) + ((static_cast<size_t>(page) * H << p.pg.shift) + r) * D + d0;
    step = static_cast<size_t>(D) << p.pg.shift;
  } else if (p.form != 2) {
    dst = static_cast<T*>(p.k) + static_cast<size_t>(row) * H * D + d0;
  } else {
    dst = static_cast<T*>(kind == 1 ? p.K[s] : p.V[s]) + static_cast<size_t>(pos) * D + d0;
    step = static_cast<size_t>(p.cap) * D;
  }
  if (kind == 2) {  // values: bit copies
    for (int h0 = h_first;;) {
#pragma unroll
      for (int i = 0; i < HB; i++)
        if (h0 + i * GPW < h_end) raw[i].store(dst + (h0 + i * GPW) * step);
      h0 += HB * GPW;
      if (h0 - grp >= h_end) return;
      fetch(h0, raw);
    }
  }
  const int half = p.rot >> 1;
  for (int j = lane; j < half; j += 32) {
    const uint64_t turn = static_cast<uint64_t>(pos) * p.rate[j];
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;  // half turns
    sincospif(x, &sn_s[wib][j], &cs_s[wib][j]);
  }
  __syncwarp();
  // this lane's factors: dimension d < rot belongs to plane d mod half; the
  // first half of a plane takes -sin of its partner, the second +sin
  const float* wn = kind == 0 ? p.q_norm : p.k_norm;
  f2_t own[4], oth[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    float a[2], b[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const int d = d0 + 2 * i + e, j = d < half ? d : d - half, q = d < half ? d + half : d - half;
      const bool turns = d < p.rot;
      a[e] = (wn ? wn[d] : 1.f) * (turns ? cs_s[wib][j] : 1.f);
      b[e] = turns ? (wn ? wn[q] : 1.f) * (d < half ? -sn_s[wib][j] : sn_s[wib][j]) : 0.f;
    }
    own[i] = f2_pack(a[0], a[1]);
    oth[i] = f2_pack(b[0], b[1]);
  }
  const bool aligned = half % 8 == 0;  // a lane's eight partners sit in one other lane
  const bool turning = d0 < p.rot;     // (aligned: all eight dimensions of the lane or none)
  const int partner = d0 < half ? gl + half / 8 : turning ? gl - half / 8 : gl;
  for (int h0 = h_first; h0 - grp < h_end; h0 += HB * GPW) {
    Raw8<T> next[HB];
    const bool more = h0 - grp + HB * GPW < h_end;
    if (more) fetch(h0 + HB * GPW, next);
    float inv[HB];
    if (wn) {  // the heads' sums side by side: their shuffles overlap
#pragma unroll
      for (int i = 0; i < HB; i++) {
        f2_t q2 = 0ull;
#pragma unroll
        for (int e = 0; e < 4; e++) q2 = f2_fma(raw[i].pair(e), raw[i].pair(e), q2);
        inv[i] = f2_hsum(q2);
      }
#pragma unroll
      for (int o = LPH / 2; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < HB; i++) inv[i] = __fadd_rn(inv[i], __shfl_xor_sync(0xffffffffu, inv[i], o));
#pragma unroll
      for (int i = 0; i < HB; i++) inv[i] = rsqrtf(__fmaf_rn(inv[i], 1.f / D, p.eps));  // 2 ulp, far below the output's rounding
    } else {
#pragma unroll
      for (int i = 0; i < HB; i++) inv[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < HB; i++) {
      const int h = h0 + i * GPW;
      f2_t y[4];
      if (aligned) {
        Raw8<T> far;
#pragma unroll
        for (int e = 0; e < Raw8<T>::W; e++) far.w[e] = __shfl_sync(0xffffffffu, raw[i].w[e], partner, LPH);
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = far.pair(e);
      } else {
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; e++) f2_unpack(raw[i].pair(e), x[2 * e], x[2 * e + 1]);
        store8(&row_s[wib][grp][d0], x);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int d = d0 + e;
          x[e] = d < p.rot ? row_s[wib][grp][d < half ? d + half : d - half] : 0.f;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = f2_pack(x[2 * e], x[2 * e + 1]);
      }
      const f2_t inv2 = f2_dup(inv[i]);
      if (turning) {
        // (a dimension past rot in a turning lane has a factor of 0 for a
        // partner that the unaligned path has set to 0)
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = f2_mul(inv2, f2_fma(raw[i].pair(e), own[e], f2_mul(y[e], oth[e])));
      } else {  // no partner: 0 times one would not do, were it infinite
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = f2_mul(inv2, f2_mul(raw[i].pair(e), own[e]));
      }
      if (h < h_end) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; e++) f2_unpack(y[e], x[2 * e], x[2 * e + 1]);
        store8(dst + h * step, x);
      }
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < HB; i++) raw[i] = next[i];
    }
  }
}

// What the calls share: shape checks, rates, launch.
template <bool PAGED>
static void norm_rope_enqueue(int D, bool bf, dim3 g, cudaStream_t st, const NormRopeParams& p) {
  switch (D) {
    case 64:
      if (bf) launch_k(true, norm_rope_kernel<__nv_bfloat16, 64, PAGED>, g, dim3(128), 0, st, p); else launch_k(true, norm_rope_kernel<float, 64, PAGED>, g, dim3(128), 0, st, p);
      break;
    case 128:
      if (bf) launch_k(true, norm_rope_kernel<__nv_bfloat16, 128, PAGED>, g, dim3(128), 0, st, p); else launch_k(true, norm_rope_kernel<float, 128, PAGED>, g, dim3(128), 0, st, p);
      break;
    default:
      if (bf) launch_k(true, norm_rope_kernel<__nv_bfloat16, 256, PAGED>, g, dim3(128), 0, st, p); else launch_k(true, norm_rope_kernel<float, 256, PAGED>, g, dim3(128), 0, st, p);
  }
}

static tv_status norm_rope_launch(const tv_attn_layer* l, NormRopeParams& p, const float* q_norm, const float* k_norm,
                                  float eps, int rot, float theta, cudaStream_t st) {
  p.q_norm = q_norm;
  p.k_norm = k_norm;
  p.eps = eps;
  p.rot = rot;
  p.Hq = l->Hq;
  p.Hkv = l->Hkv;
  p.cap = l->cap;
  // theta^(-2j/rot) / 2 pi by repeated products: j 2^-53 off at most, so an angle
  // at a 20-bit position is off by 2^-28 of a turn (theta near 1; far less above).
  // (a power for every plane is a fifth of a small call's time on the host)
  const double step = rot ? std::pow(static_cast<double>(theta), -2.0 / rot) : 0.0;
  double rate = 0.15915494309189533577 * 0x1p64;
  for (int j = 0; j < rot / 2; j++, rate *= step) p.rate[j] = static_cast<uint64_t>(rate);
  // Heads a warp walks: all of a kind with many rows (the row's factors are
  // formed once for them; up to eight rounds), fewer while the launch would
  // leave SMs without work, down to one round of four.  24 + 4 + 4 heads of 256:
  // 4 rows take 3.6 us in rounds of four, 6.1 with all 24 heads a warp; 64 rows
  // 3.8 and 6.2 (4.7 with one head a warp); 8,192 rows 50 either way.
  const int gpw = 256 / l->D;
  int hpw = 32 * gpw;
  auto split = [&]() {
    p.q_parts = (l->Hq + hpw - 1) / hpw;
    p.k_parts = (l->Hkv + hpw - 1) / hpw;
    p.parts = p.q_parts + p.k_parts + (p.form >= 2 ? p.k_parts : 0);
    return static_cast<int64_t>(p.n_rows) * p.parts;
  };
  while (hpw > 4 * gpw && split() < 16 * num_sms()) hpw >>= 1;
  p.heads_per_warp = hpw;
  split();
  if (p.parts > 65535) return TV_ERR_SHAPE;
  const dim3 g(static_cast<unsigned>((p.n_rows + 3) / 4), static_cast<unsigned>(p.parts));
  const bool bf = l->dtype == TV_BF16;
  if (p.form >= 3) norm_rope_enqueue<true>(l->D, bf, g, st, p);
  else norm_rope_enqueue<false>(l->D, bf, g, st, p);
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

// Whether rows of `n` of these are formed in place or apart from the raw rows: a
// warp writes heads of its row while others still read theirs.
static bool in_place_or_apart(const tv_attn_layer* l, int64_t n, int Hout, const void* out, const void* own_raw, int Hother,
                              const void* other_raw) {
  const int64_t c = static_cast<int64_t>(Hout) * l->D, o = static_cast<int64_t>(Hother) * l->D;
  return (out == own_raw || !overlap(out, own_raw, n, c, c, l->dtype)) && !overlap(out, other_raw, n, c, o, l->dtype);
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
  if (!in_place_or_apart(l, p.n_rows, l->Hq, q, q_raw, l->Hkv, k_raw) ||
      !in_place_or_apart(l, p.n_rows, l->Hkv, k, k_raw, l->Hq, q_raw) ||
      overlap(q, k, p.n_rows, static_cast<int64_t>(l->Hq) * l->D, static_cast<int64_t>(l->Hkv) * l->D, l->dtype))
    return TV_ERR_ARG;
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
  if (!in_place_or_apart(l, pr->n_total, l->Hq, q, q_raw, l->Hkv, k_raw) ||
      !in_place_or_apart(l, pr->n_total, l->Hq, q, q_raw, l->Hkv, v))
    return TV_ERR_ARG;
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

extern "C" tv_status tv_paged_append(const tv_paged_layer* l, const tv_paged* b, const tv_paged_rows* rows,
                                     const float* q_norm, const float* k_norm, float eps, int32_t rot_dims, float theta,
                                     const void* q_raw, const void* k_raw, const void* v, void* q, tv_stream stream) {
  tv_status c = paged_check(l, b);
  if (c == TV_OK) c = paged_rows_check(rows);
  if (c != TV_OK) return c;
  if (!l->K || !l->V) return TV_ERR_ARG;
  const tv_attn_layer a{l->dtype, l->Hq, l->Hkv, l->D, b->max_len + 1, nullptr, nullptr};
  c = norm_rope_check(&a, b->max_len, q_norm, k_norm, eps, rot_dims, theta);
  if (c != TV_OK) return c;
  const int64_t n = rows ? rows->n_total : b->n_seq;
  if (n == 0) return TV_OK;
  if (!q_raw || !k_raw || !v || !q) return TV_ERR_ARG;
  if (!aligned16(q_raw) || !aligned16(k_raw) || !aligned16(v) || !aligned16(q)) return TV_ERR_ALIGN;
  // rows, offsets and weights are read while others' rows are written; q may be q_raw
  const size_t pool = bytes_of(static_cast<int64_t>(l->n_pages) * l->Hkv * l->page, l->D, l->dtype);
  const size_t nq = bytes_of(n, static_cast<int64_t>(l->Hq) * l->D, l->dtype), nk = bytes_of(n, static_cast<int64_t>(l->Hkv) * l->D, l->dtype);
  const size_t nw = static_cast<size_t>(l->D) * 4;
  if (!apart(b->status, {{l->K, pool}, {l->V, pool}, {q, nq}},
             {{q == q_raw ? nullptr : q_raw, nq}, {k_raw, nk}, {v, nk}, {q_norm, nw}, {k_norm, nw}, offsets_of(b, rows), table_of(b), lens_of(b)}))
    return TV_ERR_ARG;
  NormRopeParams p{};
  p.form = rows ? 4 : 3;
  p.pg = paged_seqs(l, b);
  p.pr.status = b->status;
  if (rows) {
    p.pr.row_off = rows->row_off;
    p.pr.n_max = rows->n_max;
  }
  p.K[0] = l->K;
  p.V[0] = l->V;
  p.n_rows = p.n_total = static_cast<int>(n);
  p.n_seq = b->n_seq;
  p.q_raw = q_raw;
  p.k_raw = k_raw;
  p.v_raw = v;
  p.q = q;
  return norm_rope_launch(&a, p, q_norm, k_norm, eps, rot_dims, theta, reinterpret_cast<cudaStream_t>(stream));
}
