// Which pages a decode step looks at: bounds of complete pages, scores of a
// slot's pages by them, and the choice of the highest; and the advance of a
// batch's lengths.
//
//   code[0], code[1] = floor(min / 2^e), ceil(max / 2^e) of every column of a page
//   u = rint(q / 2^f), one f for the G query heads of a KV head
//   score = 2^e max_g sum_d (u > 0 ? u code[1] : u code[0])
//         = 2^e max_g (u+ . code[1] + u- . code[0])
// Codes are whole numbers within 127, so a sum is exact whatever its order (under
// 2^22), and so is its product with 2^e: no rounding decides between two pages.
// (2^f is the same for all pages of a choice and is left out.)
//
// Scores run on the integer tensor tiles (16 x 8 x 32): the group's queries as
// [u-, u+] against the codes of eight pages, read once from memory in 16-byte
// pieces.  (The order of the 2 D products is free, so a lane's piece is used as it
// lies.)  Bound by the reads of the codes, a 128th of the keys and values at pages
// of 64 rows, and for few slots by latency.
//
// The choice is a radix selection of the n-th highest key in four passes of eight
// bits, then one pass that writes the pages in rising order, of equal keys the
// lower ones.
#include "paged.cuh"
#include "prompt.cuh"

namespace tv {

// ---------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------
struct BoundsParams {
  PagedSeqs b;
  const int32_t* row_off;  // or null: a row a slot
  int n_total, n_max;
  const void* K;
  int8_t* code;
  int32_t* exp;
  int Hkv;
};

// A CTA takes a page's rows of one KV head: eight columns a lane and row.
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int LPR = D / 8, STEP = 128 / LPR;  // lanes a row, rows at a time
  __shared__ float lo_s[STEP][D], hi_s[STEP][D];
  __shared__ float top_s[4];
  pdl_wait();
  if (status_bad(p.b.status)) return;
  const int s = blockIdx.y, h = blockIdx.z;
  const int L = paged_len(p.b, s);
  if (L < 0) return;
  int n = 1;
  if (p.row_off) {
    const int off = p.row_off[s], end = p.row_off[s + 1];
    n = end - off;
    if (off < 0 || n < 0 || n > p.n_max || end > p.n_total || (s == 0 && off != 0)) {
      if (threadIdx.x == 0) set_status(p.b.status, TV_ERR_ROWS);
      return;
    }
  }
  const int64_t end = static_cast<int64_t>(L) + n;
  const int64_t j = (L >> p.b.shift) + static_cast<int64_t>(blockIdx.x);
  if (j >= (end >> p.b.shift)) return;
  if (j >= p.b.cols) {
    if (threadIdx.x == 0) set_status(p.b.status, TV_ERR_CAPACITY);
    return;
  }
  const int page = page_at(p.b, s, static_cast<int>(j));
  if (page < 0) return;
  const int rows = 1 << p.b.shift, r0 = threadIdx.x / LPR, c0 = threadIdx.x % LPR * 8;
  const size_t at = static_cast<size_t>(page) * p.Hkv + h;
  const T* src = static_cast<const T*>(p.K) + (at * rows + r0) * D + c0;
  float lo[8], hi[8];
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    lo[e] = INFINITY;
    hi[e] = -INFINITY;
  }
#pragma unroll 4
  for (int r = r0; r < rows; r += STEP, src += STEP * D) {
    float x[8];
    if constexpr (sizeof(T) == 2) {
      widen8(*reinterpret_cast<const uint4*>(src), x);
    } else {
      const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
      finite = finite && isfinite(x[e]);
      lo[e] = fminf(lo[e], x[e]);
      hi[e] = fmaxf(hi[e], x[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; e++) {
    lo_s[r0][c0 + e] = lo[e];
    hi_s[r0][c0 + e] = hi[e];
  }
  finite = __syncthreads_and(finite) != 0;
  float top = 0.f;
  constexpr int CPT = D >= 128 ? D / 128 : 1;  // columns a thread
  float a[CPT], b[CPT];
#pragma unroll
  for (int i = 0; i < CPT; i++) {
    const int c = threadIdx.x + i * 128;
    a[i] = b[i] = 0.f;
    if (c >= D) continue;
    a[i] = lo_s[0][c];
    b[i] = hi_s[0][c];
#pragma unroll
    for (int r = 1; r < STEP; r++) {
      a[i] = fminf(a[i], lo_s[r][c]);
      b[i] = fmaxf(b[i], hi_s[r][c]);
    }
    top = fmaxf(top, fmaxf(fabsf(a[i]), fabsf(b[i])));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) top_s[threadIdx.x >> 5] = top;
  __syncthreads();
  top = fmaxf(fmaxf(top_s[0], top_s[1]), fmaxf(top_s[2], top_s[3]));
  int e = 128;
  if (finite) {
    const float m = frexpf(top, &e);
    e = top > 0.f ? max(e - 7 + (m > 127.f / 128.f ? 1 : 0), -100) : -100;
  }
  const float inv = finite ? ldexpf(1.f, -e) : 0.f;
#pragma unroll
  for (int i = 0; i < CPT; i++) {
    const int c = threadIdx.x + i * 128;
    if (c >= D) continue;
    // (a product that rounds to 0 still counts as a step outward)
    const float l = finite ? floorf(__fmul_rn(a[i], inv)) : 0.f, u = finite ? ceilf(__fmul_rn(b[i], inv)) : 0.f;
    p.code[at * 2 * D + c] = static_cast<int8_t>(finite && a[i] < 0.f ? fminf(l, -1.f) : l);
    p.code[at * 2 * D + D + c] = static_cast<int8_t>(finite && b[i] > 0.f ? fmaxf(u, 1.f) : u);
  }
  if (threadIdx.x == 0) p.exp[at] = e;
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------
struct SelectParams {
  PagedSeqs b;
  const void* q;
  const int8_t* code;
  const int32_t* exp;
  float* score;  // [units][pages]
  int32_t* sel;
  int32_t* count;
  int Hq, Hkv, G, first, last, n_sel, pages;  // pages a slot has at most
};

// d += a b for one 16 x 8 x 32 tile of signed bytes
__device__ __forceinline__ void mma16832_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kScorePages = 128;  // pages of a CTA: 32 a warp

template <typename T, int D>
__global__ void __launch_bounds__(128) paged_score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int LINE = 2 * D + 16;  // bytes of a query's [u-, u+] (rows 4 banks apart)
  constexpr int Q = 2 * D / 64;     // 16-byte pieces a lane of a row
  __shared__ __align__(16) int8_t code_s[16 * LINE];
  __shared__ float top_s[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (status_bad(p.b.status)) return;
  const int u = blockIdx.y, s = u / p.Hkv, h = u - s * p.Hkv;
  const int L = paged_len(p.b, s);
  const int nb = (L >> p.b.shift) + 1;
  const int j0 = p.first + static_cast<int>(blockIdx.x) * kScorePages, end = nb - p.last;
  if (L < 0 || nb <= p.n_sel || j0 >= end) return;
  // the group's queries in whole steps
  const T* q = static_cast<const T*>(p.q) + (static_cast<size_t>(s) * p.Hq + h * p.G) * D;
  float top = 0.f;
  bool finite = true;
  for (int i = threadIdx.x; i < p.G * D; i += 128) {
    const float x = to_f32(q[i]);
    finite = finite && isfinite(x);
    top = fmaxf(top, fabsf(x));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) top_s[warp] = top;
  finite = __syncthreads_and(finite) != 0;
  top = fmaxf(fmaxf(top_s[0], top_s[1]), fmaxf(top_s[2], top_s[3]));
  int f = 0;
  if (finite && top > 0.f) {
    const float m = frexpf(top, &f);
    f = f - 7 + (m > 127.f / 128.f ? 1 : 0);
  }
  constexpr int NTW = kScorePages / 4 / 8;  // tiles of eight pages a warp
  int best[NTW][2];
  int64_t at[NTW];  // this lane's page of a tile (as the second operand's column)
#pragma unroll
  for (int t = 0; t < NTW; t++) {
    best[t][0] = best[t][1] = INT_MIN;
    const int j = j0 + (warp * NTW + t) * 8 + (lane >> 2);
    const int page = j < end ? page_at(p.b, s, j) : -1;
    at[t] = page < 0 ? -1 : static_cast<int64_t>(page) * p.Hkv + h;
  }
  for (int g0 = 0; g0 < p.G; g0 += 16) {
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * D; i += 128) {
      const int g = g0 + i / D, d = i % D;
      const int v = finite && g < p.G ? static_cast<int>(rintf(ldexpf(to_f32(q[static_cast<size_t>(g) * D + d]), -f))) : 0;
      code_s[(i / D) * LINE + d] = static_cast<int8_t>(min(v, 0));
      code_s[(i / D) * LINE + D + d] = static_cast<int8_t>(max(v, 0));
    }
    __syncthreads();
    uint4 a[Q][2];
#pragma unroll
    for (int i = 0; i < Q; i++)
#pragma unroll
      for (int r = 0; r < 2; r++)
        a[i][r] = *reinterpret_cast<const uint4*>(code_s + ((lane >> 2) + 8 * r) * LINE + i * 64 + (lane & 3) * 16);
    const int live = min(16, p.G - g0);
#pragma unroll
    for (int t = 0; t < NTW; t++) {
      const uint4* src = reinterpret_cast<const uint4*>(p.code + (at[t] < 0 ? 0 : at[t]) * 2 * D) + (lane & 3);
      uint4 b[Q];
#pragma unroll
      for (int i = 0; i < Q; i++) b[i] = at[t] < 0 ? make_uint4(0u, 0u, 0u, 0u) : src[i * 4];
      int d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < Q; i++) {
        mma16832_s8(d, a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, b[i].x, b[i].y);
        mma16832_s8(d, a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, b[i].z, b[i].w);
      }
      // the highest of the heads there are
#pragma unroll
      for (int c = 0; c < 2; c++) {
        int x = (lane >> 2) < live ? d[c] : INT_MIN;
        if ((lane >> 2) + 8 < live) x = max(x, d[2 + c]);
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        best[t][c] = max(best[t][c], x);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NTW; t++) {
    const int c = lane & 7, v = __shfl_sync(0xffffffffu, best[t][0], c >> 1), w = __shfl_sync(0xffffffffu, best[t][1], c >> 1);
    const int64_t mine = __shfl_sync(0xffffffffu, at[t], c * 4);
    const int j = j0 + (warp * NTW + t) * 8 + c;
    if (lane < 8 && j < end) {
      const int e = mine < 0 ? 0 : p.exp[mine];
      p.score[static_cast<size_t>(u) * p.pages + j] = e >= 128 ? INFINITY : ldexpf(static_cast<float>(c & 1 ? w : v), e);
    }
  }
}

// ---------------------------------------------------------------------------
// choice
// ---------------------------------------------------------------------------
constexpr int kPick = 512, kPickKeys = 8192;  // threads; keys kept in shared memory

// A rising key for a score (no NaN).
__device__ __forceinline__ uint32_t rising(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kPick) paged_pick_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t keys[kPickKeys];
  __shared__ int hist[256], part[kPick / 32][2];
  __shared__ uint32_t prefix_s;
  __shared__ int need_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = blockIdx.x, s = u / p.Hkv;
  pdl_wait();
  if (status_bad(p.b.status)) return;
  const int L = paged_len(p.b, s);
  if (L < 0) return;
  int32_t* sel = p.sel + static_cast<size_t>(u) * p.n_sel;
  const int nb = (L >> p.b.shift) + 1;
  if (nb <= p.n_sel) {
    for (int i = threadIdx.x; i < p.n_sel; i += kPick) sel[i] = i < nb ? i : -1;
    if (threadIdx.x == 0) p.count[u] = nb;
    return;
  }
  const int n = nb - p.first - p.last, want = p.n_sel - p.first - p.last;
  for (int i = threadIdx.x; i < p.first; i += kPick) sel[i] = i;
  for (int i = threadIdx.x; i < p.last; i += kPick) sel[p.n_sel - p.last + i] = nb - p.last + i;
  if (threadIdx.x == 0) p.count[u] = p.n_sel;
  if (want == 0) return;
  const float* score = p.score + static_cast<size_t>(u) * p.pages + p.first;
  const bool kept = n <= kPickKeys;
  auto key = [&](int i) { return kept ? keys[i] : rising(score[i]); };
  if (kept)
    for (int i = threadIdx.x; i < n; i += kPick) keys[i] = rising(score[i]);
  uint32_t prefix = 0;
  int need = want;  // of the keys that share the bits found so far
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPick) {
      const uint32_t k = key(i);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {  // from the top: lane 0 holds bins 255 .. 248
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; i++) sum += c[i] = hist[255 - lane * 8 - i];
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += x;
      }
      above -= sum;
      if (above < need && need <= above + sum) {
        int i = 0;
        while (above + c[i] < need) above += c[i++];
        prefix_s = prefix | (static_cast<uint32_t>(255 - lane * 8 - i) << shift);
        need_s = need - above;
      }
    }
    __syncthreads();
    prefix = prefix_s;
    need = need_s;
  }
  // every higher key, and of those equal to it the first `need`
  int out = 0, equal = 0;
  for (int i0 = 0; i0 < n; i0 += kPick) {
    const int i = i0 + threadIdx.x;
    const uint32_t k = i < n ? key(i) : 0u;
    const bool more = i < n && k > prefix, same = i < n && k == prefix;
    const unsigned ms = __ballot_sync(0xffffffffu, same), low = (1u << lane) - 1u;
    if (lane == 0) part[warp][0] = __popc(ms);
    __syncthreads();
    int rank = equal + __popc(ms & low), all_same = 0;
#pragma unroll
    for (int w = 0; w < kPick / 32; w++) {
      if (w < warp) rank += part[w][0];
      all_same += part[w][0];
    }
    const bool take = more || (same && rank < need);
    const unsigned mt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) part[warp][1] = __popc(mt);
    __syncthreads();
    int place = out + __popc(mt & low), all = 0;
#pragma unroll
    for (int w = 0; w < kPick / 32; w++) {
      if (w < warp) place += part[w][1];
      all += part[w][1];
    }
    if (take) sel[p.first + place] = p.first + i;
    out += all;
    equal += all_same;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// advance
// ---------------------------------------------------------------------------
__global__ void paged_advance_kernel(int32_t* len, const int32_t* row_off, PagedSeqs b, int n_total, int n_max) {
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  pdl_wait();
  if (s >= b.n_seq || status_bad(b.status)) return;
  const int L = paged_len(b, s);
  int n = 1;
  if (row_off) {
    const int off = row_off[s], end = row_off[s + 1];
    n = end - off;
    if (off < 0 || n < 0 || n > n_max || end > n_total || (s == 0 && off != 0) || (L < 0 && n > 0)) {
      set_status(b.status, TV_ERR_ROWS);
      return;
    }
  }
  if (L >= 0) len[s] = L + n;
}

template <int D>
static void launch_bounds_d(const BoundsParams& p, bool bf, dim3 g, cudaStream_t st) {
  if (bf) launch_k(true, paged_bounds_kernel<__nv_bfloat16, D>, g, dim3(128), 0, st, p);
  else launch_k(true, paged_bounds_kernel<float, D>, g, dim3(128), 0, st, p);
}
template <int D>
static void launch_score_d(const SelectParams& p, bool bf, dim3 g, cudaStream_t st) {
  if (bf) launch_k(true, paged_score_kernel<__nv_bfloat16, D>, g, dim3(128), 0, st, p);
  else launch_k(true, paged_score_kernel<float, D>, g, dim3(128), 0, st, p);
}

}  // namespace tv

using namespace tv;

extern "C" tv_status tv_paged_bounds(const tv_paged_layer* l, const tv_paged* b, const tv_paged_rows* rows, int8_t* code,
                                     int32_t* exp, tv_stream stream) {
  tv_status c = paged_check(l, b);
  if (c == TV_OK) c = paged_rows_check(rows);
  if (c != TV_OK) return c;
  if (!l->K || !code || !exp) return TV_ERR_ARG;
  if (!aligned16(code) || !aligned16(exp)) return TV_ERR_ALIGN;
  const size_t heads = static_cast<size_t>(l->n_pages) * l->Hkv, pool = bytes_of(static_cast<int64_t>(heads) * l->page, l->D, l->dtype);
  if (share_memory(code, heads * 2 * l->D, l->K, pool) || share_memory(exp, heads * 4, l->K, pool) ||
      share_memory(code, heads * 2 * l->D, exp, heads * 4))
    return TV_ERR_ARG;
  if (l->Hkv > 65535) return TV_ERR_SHAPE;
  BoundsParams p{};
  p.b = paged_seqs(l, b);
  if (rows) {
    p.row_off = rows->row_off;
    p.n_total = rows->n_total;
    p.n_max = rows->n_max;
  }
  p.K = l->K;
  p.code = code;
  p.exp = exp;
  p.Hkv = l->Hkv;
  const int n = rows ? rows->n_max : 1;
  const dim3 g((n + l->page - 1) / l->page, b->n_seq, l->Hkv);  // n rows complete so many pages at most
  if (n == 0) return TV_OK;
  const bool bf = l->dtype == TV_BF16;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (l->D) {
    case 64: launch_bounds_d<64>(p, bf, g, st); break;
    case 128: launch_bounds_d<128>(p, bf, g, st); break;
    default: launch_bounds_d<256>(p, bf, g, st);
  }
  return launch_status();
}

static int pages_at_most(const tv_paged_layer* l, const tv_paged* b) { return b->max_len / l->page + 1; }

extern "C" size_t tv_paged_select_workspace_bytes(const tv_paged_layer* l, const tv_paged* b) {
  if (paged_check(l, b) != TV_OK) return 0;
  return static_cast<size_t>(b->n_seq) * l->Hkv * pages_at_most(l, b) * 4;
}

extern "C" tv_status tv_paged_select(const tv_paged_layer* l, const tv_paged* b, const int8_t* code, const int32_t* exp,
                                     int32_t first, int32_t last, int32_t n_sel, const void* q, int32_t* sel, int32_t* count,
                                     void* ws, size_t ws_bytes, tv_stream stream) {
  const tv_status c = paged_check(l, b);
  if (c != TV_OK) return c;
  if (!code || !exp || !q || !sel || !count || first < 0 || last < 1 || n_sel < 1 || n_sel > 4096 || first > n_sel || last > n_sel - first)
    return TV_ERR_ARG;
  if (!aligned16(code) || !aligned16(exp) || !aligned16(q) || !aligned16(sel) || !aligned16(count) || !aligned16(ws)) return TV_ERR_ALIGN;
  if (!ws || ws_bytes < tv_paged_select_workspace_bytes(l, b)) return TV_ERR_WORKSPACE;
  SelectParams p{};
  p.b = paged_seqs(l, b);
  p.q = q;
  p.code = code;
  p.exp = exp;
  p.score = static_cast<float*>(ws);
  p.sel = sel;
  p.count = count;
  p.Hq = l->Hq;
  p.Hkv = l->Hkv;
  p.G = l->Hq / l->Hkv;
  p.first = first;
  p.last = last;
  p.n_sel = n_sel;
  p.pages = pages_at_most(l, b);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int units = b->n_seq * l->Hkv, mid = p.pages - first - last;
  if (p.pages > n_sel && n_sel > first + last) {
    const dim3 g((mid + kScorePages - 1) / kScorePages, units);
    const bool bf = l->dtype == TV_BF16;
    switch (l->D) {
      case 64: launch_score_d<64>(p, bf, g, st); break;
      case 128: launch_score_d<128>(p, bf, g, st); break;
      default: launch_score_d<256>(p, bf, g, st);
    }
  }
  launch_k(true, paged_pick_kernel, dim3(units), dim3(kPick), 0, st, p);
  return launch_status();
}

extern "C" tv_status tv_paged_advance(const tv_paged* b, const tv_paged_rows* rows, int32_t* len, tv_stream stream) {
  if (!b || !b->len || !b->status || !len || b->n_seq < 1 || b->n_seq > TV_MAX_PAGED_SEQ || b->max_len < 0 || len != b->len) return TV_ERR_ARG;
  if (!aligned16(b->len) || !aligned16(b->status)) return TV_ERR_ALIGN;
  const tv_status c = paged_rows_check(rows);
  if (c != TV_OK) return c;
  const PagedSeqs v{nullptr, b->len, b->status, b->n_seq, 0, b->max_len, 0, 0};
  launch_k(true, paged_advance_kernel, dim3((b->n_seq + 127) / 128), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), len,
           rows ? rows->row_off : nullptr, v, rows ? rows->n_total : 0, rows ? rows->n_max : 0);
  return launch_status();
}
