// The packed rows of a prompt call, as its kernels see them: sequence s owns
// rows row_off[s] .. row_off[s+1]-1 of the packed buffers, behind len[s] rows
// its caches already hold.  The offsets and lengths live on the device, so
// every kernel checks them for itself before it touches a row; all CTAs of a
// launch read the same values and so take the same decision.
#pragma once
#include "common.cuh"
#include "host.hpp"

namespace tv {

struct PromptRows {
  const int32_t* row_off;  // [n_seq + 1]
  const int32_t* len;      // [n_seq], or null where no cache is involved
  int32_t* status;
  int n_seq, n_total, n_max, max_len, cap;
};

// One sequence per lane (lane <= n_seq holds its offset), valid in a full warp.
struct WarpSeqs {
  int off, end, len;
  int code;  // 0, or the tv_status the launch reports
};

__device__ __forceinline__ WarpSeqs load_seqs(const PromptRows& p, int lane) {
  WarpSeqs w;
  w.off = lane <= p.n_seq ? p.row_off[lane] : 0;
  w.len = (p.len && lane < p.n_seq) ? p.len[lane] : 0;
  w.end = __shfl_down_sync(0xffffffffu, w.off, 1);
  const bool mine = lane < p.n_seq;
  const bool rows = (lane == 0 && w.off != 0) || (lane == p.n_seq && w.off > p.n_total) ||
                    (mine && (w.end < w.off || w.end - w.off > p.n_max));
  w.code = 0;
  if (__any_sync(0xffffffffu, rows)) w.code = TV_ERR_ROWS;
  else if (p.len) {
    if (__any_sync(0xffffffffu, mine && (w.len < 0 || w.len > p.max_len))) w.code = TV_ERR_LEN;
    else if (__any_sync(0xffffffffu, mine && w.end - w.off > p.cap - w.len)) w.code = TV_ERR_CAPACITY;
  }
  return w;
}
// The sequence that owns packed row `row` (the last one whose rows start at or
// before it: empty sequences share their successor's offset), -1 behind the
// last sequence.
__device__ __forceinline__ int seq_of(const WarpSeqs& w, const PromptRows& p, int lane, int row) {
  const unsigned m = __ballot_sync(0xffffffffu, lane <= p.n_seq && w.off <= row);
  const int s = 31 - __clz(static_cast<int>(m));
  return s >= p.n_seq ? -1 : s;
}

// Each sequence cut into strips of `rows` rows from its first: the strips of the
// sequences before this lane's, and of all.
__device__ __forceinline__ int strip_base(const WarpSeqs& w, const PromptRows& p, int lane, int rows, int& all) {
  const int mine = lane < p.n_seq ? (w.end - w.off + rows - 1) / rows : 0;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  all = __shfl_sync(0xffffffffu, incl, 31);
  return incl - mine;
}
// The sequence that strip `i` of these belongs to.
__device__ __forceinline__ int strip_seq(const WarpSeqs& w, const PromptRows& p, int lane, int base, int i) {
  return 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, lane < p.n_seq && w.end > w.off && base <= i)));
}

// The host's half: a well-formed descriptor (rows may be zero).
inline bool prompt_ok(const tv_prompt* p) {
  return p && p->n_seq >= 1 && p->n_seq <= TV_MAX_SEQ && p->n_total >= 0 && p->n_total <= TV_MAX_PROMPT_ROWS &&
         p->n_max >= 0 && p->n_max <= p->n_total && p->row_off && p->status && aligned16(p->row_off) &&
         aligned16(p->status);
}
// Whether [n][cols] values of type dt at a and [n][cols2] of type dt2 at b share memory.
inline bool overlap(const void* a, const void* b, int64_t n, int64_t cols, int64_t cols2, int32_t dt, int32_t dt2) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(n * cols2) * (dt2 == TV_BF16 ? 2 : 4) &&
         y < x + static_cast<uintptr_t>(n * cols) * (dt == TV_BF16 ? 2 : 4);
}
inline bool overlap(const void* a, const void* b, int64_t n, int64_t cols, int64_t cols2, int32_t dt) {
  return overlap(a, b, n, cols, cols2, dt, dt);
}
inline PromptRows prompt_rows(const tv_prompt* p, const int32_t* len, int max_len, int cap) {
  return PromptRows{p->row_off, len, p->status, p->n_seq, p->n_total, p->n_max, max_len, cap};
}

// 0xffff in each half of a bf16 pair that is finite, 0 in others.
__device__ __forceinline__ uint32_t finite2(uint32_t x) { return __vcmpltu2(x & 0x7f807f80u, 0x7f807f80u); }

// Eight consecutive values of a row, widened to fp32 (16-byte aligned).
__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
}

}  // namespace tv
