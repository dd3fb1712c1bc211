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
// The choice is a radix selection of the n-th highest key by digits of eight bits,
// from the highest bit in which the keys differ down, until a digit leaves no
// choice; then one pass writes the pages in rising order, of equal keys the lower
// ones.  A cluster of CTAs shares a slot's KV head: each scores its part of the pages
// into the first one's shared memory, which then chooses.
#include <climits>

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
  uint32_t* far;  // [units][pages]: keys that do not fit in shared memory
  int32_t* sel;
  int32_t* count;
  int Hq, Hkv, G, first, last, n_sel, pages;  // pages a slot has at most
  int keys;                                   // keys that shared memory holds
};

// d += a b for one 16 x 8 x 32 tile of signed bytes
__device__ __forceinline__ void mma16832_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) { widen8(*reinterpret_cast<const uint4*>(p), x); }

constexpr int kSelect = 256;        // threads of a CTA: each warp scores eight pages at a time
constexpr int kSelectKeys = 16384;  // pages whose keys fit in shared memory

// A rising key for a score (no NaN).
__device__ __forceinline__ uint32_t rising(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores into the shared memory of the cluster's first CTA.
__device__ __forceinline__ void store_first(uint32_t addr, uint32_t v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u32 [a], %1;\n\t}" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t load_first(uint32_t addr) {
  uint32_t v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, 0;\n\tld.shared::cluster.u32 %0, [a];\n\t}" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Dynamic shared memory: the keys (first CTA of a cluster; in the workspace where they do not fit).
template <typename T, int D>
__global__ void __launch_bounds__(kSelect, 2) paged_select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int LINE = 2 * D + 64;  // bytes of a query's [u-, u+] (rows half a line of banks apart)
  constexpr int Q = 2 * D / 64;     // 16-byte pieces a lane of a row
  constexpr int W = kSelect / 32;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int8_t code_s[16 * LINE];
  __shared__ int hist[256], part[W][2];
  __shared__ uint32_t red_s[W], red2_s[W];
  __shared__ uint32_t prefix_s;
  __shared__ int need_s, left_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_ctas());
  // (No CTA may store into another's shared memory before that one has started, or after it
  // has left: what the CTAs of a cluster do depends on the lengths alone, which they all read alike; an error
  // that some of them meet first keeps the first CTA from writing, no more.)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const bool bad = status_bad(p.b.status);
  const int u = blockIdx.y, s = u / p.Hkv, h = u - s * p.Hkv;
  const int L = paged_len(p.b, s);
  const int nb = (L >> p.b.shift) + 1;
  int32_t* sel = p.sel + static_cast<size_t>(u) * p.n_sel;
  if (L < 0 || nb <= p.n_sel || p.n_sel == p.first + p.last) {  // (the whole cluster)
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (L < 0 || rank > 0 || bad) return;
    const int ends = nb <= p.n_sel ? nb : p.first;
    for (int i = tid; i < p.n_sel; i += kSelect) sel[i] = i < ends ? i : nb <= p.n_sel ? -1 : nb - p.n_sel + i;
    if (tid == 0) p.count[u] = min(nb, p.n_sel);
    return;
  }
  const int n = nb - p.first - p.last;  // pages to choose from
  const bool kept = n <= p.keys;
  uint32_t* far = p.far + static_cast<size_t>(u) * p.pages;
  const uint32_t keys_at = static_cast<uint32_t>(__cvta_generic_to_shared(keys));
  // Pages are dealt to the warps eight at a time, a tile; a warp looks up four tiles' pages and exponents at once.
  // The first tile's codes are on their way while the queries are looked at.
  const int tiles = (n + 7) / 8, stride = W * ctas, tile0 = rank * W + warp;
  uint4 b[Q];
  int page = -1, e = 0;  // of place (lane & 7) of tile `first of four` + (lane >> 3) * stride
  auto look = [&](int tile) {
    const int j = (tile + (lane >> 3) * stride) * 8 + (lane & 7);
    page = j < n ? page_at(p.b, s, p.first + j) : -1;
    e = page < 0 ? 0 : p.exp[static_cast<size_t>(page) * p.Hkv + h];
  };
  auto fetch = [&](int i) {  // codes of the i-th of the four: this lane's page as the second operand's column
    const int x = __shfl_sync(0xffffffffu, page, i * 8 + (lane >> 2));
    const uint4* src = reinterpret_cast<const uint4*>(p.code + (static_cast<size_t>(x < 0 ? 0 : x) * p.Hkv + h) * 2 * D) + (lane & 3);
#pragma unroll
    for (int k = 0; k < Q; k++) b[k] = src[k * 4];
  };
  if (tile0 < tiles) {
    look(tile0);
    fetch(0);
  }
  // the group's queries in whole steps
  const T* q = static_cast<const T*>(p.q) + (static_cast<size_t>(s) * p.Hq + h * p.G) * D;
  uint32_t top = 0;  // the largest size, as bits (what is not finite comes out above every finite one)
  float mine[8];     // this thread's last eight values (its only ones in a small group)
  for (int i = tid; i < p.G * D / 8; i += kSelect) {
    load8(q + i * 8, mine);
#pragma unroll
    for (int c = 0; c < 8; c++) top = max(top, __float_as_uint(mine[c]) & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) red_s[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; w++) top = max(top, red_s[w]);
  const bool finite = top < 0x7f800000u;
  int f = 0;
  if (finite && top > 0) {
    const float m = frexpf(__uint_as_float(top), &f);
    f = f - 7 + (m > 127.f / 128.f ? 1 : 0);
  }
  // times 2^-f in two steps, each a power of two that fp32 holds (a product that is rounded on the way is under 1/2 in the end)
  const int f1 = -f / 2;
  const float by1 = finite ? ldexpf(1.f, f1) : 0.f, by2 = finite ? ldexpf(1.f, -f - f1) : 0.f;
  const int pages0 = p.first;
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  for (int g0 = 0; g0 < p.G; g0 += 16) {
    if (g0 > 0) __syncthreads();
    for (int i = tid; i < 16 * D / 8; i += kSelect) {
      const int g = i / (D / 8), d = i % (D / 8) * 8;
      float x[8];
      if (finite && g0 + g < p.G) {
        if (p.G <= 16 && p.G * D <= kSelect * 8) {
#pragma unroll
          for (int c = 0; c < 8; c++) x[c] = mine[c];
        } else {
          load8(q + static_cast<size_t>(g0 + g) * D + d, x);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = 0.f;
      }
      uint32_t lo[2] = {0u, 0u}, hi[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int v = __float2int_rn(__fmul_rn(__fmul_rn(x[e], by1), by2));
        lo[e / 4] |= (static_cast<uint32_t>(min(v, 0)) & 255u) << (e % 4 * 8);
        hi[e / 4] |= (static_cast<uint32_t>(max(v, 0)) & 255u) << (e % 4 * 8);
      }
      *reinterpret_cast<uint2*>(code_s + g * LINE + d) = make_uint2(lo[0], lo[1]);
      *reinterpret_cast<uint2*>(code_s + g * LINE + D + d) = make_uint2(hi[0], hi[1]);
    }
    __syncthreads();
    const int live = min(16, p.G - g0);
    const int8_t* row = code_s + (lane >> 2) * LINE + (lane & 3) * 16;
    int i = 0;
    for (int tile = tile0; tile < tiles; tile += stride, i = (i + 1) & 3) {
      if (i == 0 && (g0 > 0 || tile > tile0)) {
        look(tile);
        fetch(0);
      }
      int d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < Q; k++) {
        const uint4 x = *reinterpret_cast<const uint4*>(row + k * 64);
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (live > 8) y = *reinterpret_cast<const uint4*>(row + 8 * LINE + k * 64);
        mma16832_s8(d, x.x, y.x, x.y, y.y, b[k].x, b[k].y);
        mma16832_s8(d, x.z, y.z, x.w, y.w, b[k].z, b[k].w);
      }
      if (i < 3 && tile + stride < tiles) fetch(i + 1);  // the next ones under what follows
      // the highest of the heads there are, of pages 2 (lane & 3) and 2 (lane & 3) + 1
      int best[2];
#pragma unroll
      for (int c = 0; c < 2; c++) {
        int x = (lane >> 2) < live ? d[c] : INT_MIN;
        if ((lane >> 2) + 8 < live) x = max(x, d[2 + c]);
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        best[c] = x;
      }
      const int v0 = __shfl_sync(0xffffffffu, best[0], (lane & 7) >> 1), v1 = __shfl_sync(0xffffffffu, best[1], (lane & 7) >> 1);
      const int ex = __shfl_sync(0xffffffffu, e, i * 8 + (lane & 7)), j = tile * 8 + lane;
      if (lane < 8 && j < n) {
        uint32_t key = rising(ex >= 128 ? INFINITY : ldexpf(static_cast<float>(lane & 1 ? v1 : v0), ex));
        if (kept) {  // (later heads' scores of a page are this lane's own again)
          if (g0 > 0) key = max(key, load_first(keys_at + j * 4));
          store_first(keys_at + j * 4, key);
        } else {
          far[j] = g0 > 0 ? max(key, far[j]) : key;
        }
      }
    }
  }
  if (ctas > 1) {
    if (!kept) __threadfence();
    cluster_sync();
    if (rank > 0) return;
  } else {
    __syncthreads();
  }
  if (bad) return;
  // ---- the choice
  auto key = [&](int i) { return kept ? keys[i] : __ldcg(far + i); };
  uint32_t low = 0xffffffffu, high = 0;
  for (int i = tid; i < n; i += kSelect) {
    const uint32_t k = key(i);
    low = min(low, k);
    high = max(high, k);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    red_s[warp] = low;
    red2_s[warp] = high;
  }
  hist[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; w++) {
    low = min(low, red_s[w]);
    high = max(high, red2_s[w]);
  }
  // Keys are low plus an offset of `bits` bits; of those whose offset starts with prefix, `need` are to be taken.
  int bits = 32 - __clz(static_cast<int>(high - low)), need = p.n_sel - p.first - p.last;
  uint32_t prefix = 0;
  bool all = false;
  while (bits > 0 && !all) {
    const int shift = max(bits - 8, 0);
    const uint32_t mask = (1u << (bits - shift)) - 1u;
    for (int i = tid; i < n; i += kSelect) {
      const uint32_t k = key(i) - low;
      if (bits == 32 || (k >> bits) == (prefix >> bits)) atomicAdd(&hist[(k >> shift) & mask], 1);
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
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if (above < need && need <= above + c[i]) {
            prefix_s = prefix | (static_cast<uint32_t>(255 - lane * 8 - i) << shift);
            need_s = need - above;
            left_s = c[i];
            break;
          }
          above += c[i];
        }
      }
    }
    __syncthreads();
    prefix = prefix_s;
    need = need_s;
    all = left_s == need;  // the whole digit is taken
    bits = shift;
    hist[tid] = 0;
    __syncthreads();
  }
  // every higher key, and of those that share all bits found the first `need`
  const uint32_t border = prefix >> bits;  // (bits 32: no key differs in any)
  int out = 0, equal = 0;
  for (int i = tid; i < p.first; i += kSelect) sel[i] = i;
  for (int i = tid; i < p.last; i += kSelect) sel[p.n_sel - p.last + i] = nb - p.last + i;
  if (tid == 0) p.count[u] = p.n_sel;
  for (int i0 = 0; i0 < n; i0 += kSelect) {
    const int i = i0 + tid;
    const uint32_t k = i < n ? (key(i) - low) >> bits : 0u;
    const bool more = i < n && k > border, same = i < n && k == border;
    const unsigned ms = __ballot_sync(0xffffffffu, same), below = (1u << lane) - 1u;
    bool take = more || same;
    int all_same = 0;
    if (!all) {  // (else every equal one is taken)
      if (lane == 0) part[warp][0] = __popc(ms);
      __syncthreads();
      int before = equal + __popc(ms & below);
#pragma unroll
      for (int w = 0; w < W; w++) {
        if (w < warp) before += part[w][0];
        all_same += part[w][0];
      }
      take = more || (same && before < need);
    }
    const unsigned mt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) part[warp][1] = __popc(mt);
    __syncthreads();
    int place = out + __popc(mt & below), sum = 0;
#pragma unroll
    for (int w = 0; w < W; w++) {
      if (w < warp) place += part[w][1];
      sum += part[w][1];
    }
    if (take) sel[pages0 + place] = pages0 + i;
    out += sum;
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
template <typename T, int D>
static bool launch_select_t(const SelectParams& p, int ctas, int units, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  const int bytes = p.keys * 4;
  if (!allow_smem(paged_select_kernel<T, D>, kSelectKeys * 4, set)) return false;
  launch_k_cluster(true, ctas, paged_select_kernel<T, D>, dim3(ctas, units), dim3(kSelect), bytes, st, p);
  return true;
}
template <int D>
static bool launch_select_d(const SelectParams& p, bool bf, int ctas, int units, cudaStream_t st) {
  return bf ? launch_select_t<__nv_bfloat16, D>(p, ctas, units, st) : launch_select_t<float, D>(p, ctas, units, st);
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
  if (paged_check(l, b) != TV_OK || pages_at_most(l, b) <= kSelectKeys) return 0;
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
  const size_t need = tv_paged_select_workspace_bytes(l, b);
  if (need > 0 && (!ws || ws_bytes < need)) return TV_ERR_WORKSPACE;
  SelectParams p{};
  p.b = paged_seqs(l, b);
  p.q = q;
  p.code = code;
  p.exp = exp;
  p.far = static_cast<uint32_t*>(ws);
  p.sel = sel;
  p.count = count;
  p.Hq = l->Hq;
  p.Hkv = l->Hkv;
  p.G = l->Hq / l->Hkv;
  p.first = first;
  p.last = last;
  p.n_sel = n_sel;
  p.pages = pages_at_most(l, b);
  const int units = b->n_seq * l->Hkv;
  const int most = p.pages > n_sel && n_sel > first + last ? p.pages - first - last : 0;  // pages to choose from, at most
  p.keys = most < kSelectKeys ? most : kSelectKeys;
  // CTAs for a slot's KV head: up to eight, while the GPU has room and each has 128 pages (the queries' codes take each as
  // long as some 100 pages)
  int ctas = 1;
  while (ctas < 8 && units * ctas < 2 * num_sms() && ctas * 2 * 128 <= most) ctas *= 2;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = l->dtype == TV_BF16;
  const bool ok = l->D == 64 ? launch_select_d<64>(p, bf, ctas, units, st) : l->D == 128 ? launch_select_d<128>(p, bf, ctas, units, st)
                                                                                        : launch_select_d<256>(p, bf, ctas, units, st);
  return ok ? launch_status() : TV_ERR_CUDA;
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
