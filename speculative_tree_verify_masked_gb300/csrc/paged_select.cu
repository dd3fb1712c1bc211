// Which pages a decode step looks at: bounds of complete pages, scores of a
// slot's pages by them, and the choice of the highest; and the advance of a
// batch's lengths.
//
//   code[0], code[1] = floor(min / 2^e), ceil(max / 2^e) of every column of a page
//   u = rint(q / 2^f), one f for the G query heads of a KV head
//   score = 2^e max_g sum_d (u > 0 ? u code[1] : u code[0])
//         = 2^e max_g (u+ . code[1] + u- . code[0])
// Codes are whole numbers within 127, so a sum is exact whatever its order (under
// 2^22), and so is its product with 2^(e - 24), which fp32 holds for every e from -100 to
// 127: no rounding decides between two pages.  (2^f and 2^24 are the same for all
// pages of a choice and are left out.)
//
// Scores run on 16 x 8 x 16 tensor-core tiles, sixteen pages by eight query heads,
// with codes and queries as fp16 and sums in fp32, which hold these whole numbers exactly
// (the integer tiles of this GPU take 190 cycles a product of half the size: 12,000
// cycles a CTA against 4,500).  Codes are read once from memory in 16-byte pieces and widened in
// registers; the order of the 2 D products is free, so a lane's piece is used as it
// lies.  Bound by latency for few slots: one of 2,048 pages (24 + 4 heads of 256) 8.8 us,
// of which half are lengths, table, exponents and codes, read one behind the other, the rest the digits' rounds; by
// the reads of the codes (a 128th of the keys and values at pages of 64 rows), in pieces of 512 bytes all over, for many:
// 24 slots of up to 65,536 rows 12.5 us for 18 MB.
//
// The bounds are bound by reads of whole pages, one CTA each: 16,421 rows of two prompts (33.6 MB of keys) 8.9 us, 3.8
// TB/s in a grid of 1,032 CTAs that runs once; a step of 192 slots 2.7 us, a launch's latency.  (Up to eight rows of a lane
// are in flight, two of small pages; four in one loop 9.3 us, and 5.3 against 4.6 for a few pages of 128 rows of 256; CTAs of
// 256 threads 11.0, and 3.4 a step.)  The grid has the pages of n_max rows for every slot, whatever rows it has: one slice of
// 4,096 rows beside 191 decode rows, 24 + 4 heads of 256, 100 us in pages of 16 and 27 in pages of 64, nearly all of it CTAs that find no page.
//
// The choice is a radix selection of the n-th highest key by digits of eight bits,
// from the highest bit in which the keys differ down, until a digit leaves no
// choice; then one pass writes the pages in rising order, of equal keys the lower
// ones.  A cluster of CTAs shares a slot's KV head: each scores its part of the pages
// into the first one's shared memory, which then chooses.
#include <climits>
#include <cuda_fp16.h>
#include <type_traits>

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

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) { widen8(*reinterpret_cast<const uint4*>(p), x); }

// A CTA takes a page's rows of one KV head: eight columns a lane and row.
template <typename T, int D>
__global__ void __launch_bounds__(128) paged_bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int LPR = D / 8, STEP = 128 / LPR;  // lanes a row, rows at a time
  __shared__ float lo_s[STEP][D], hi_s[STEP][D];
  __shared__ float top_s[4];
  pdl_wait();
  const bool bad = status_set(p.b.status);
  const int s = blockIdx.y, h = blockIdx.z;
  const int L = paged_len(p.b, s);
  if (__syncthreads_or(bad) || L < 0) return;  // (another CTA may set the word between two warps' looks at it)
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
  auto take = [&](auto n) {  // so many rows of this lane, all on their way together
    constexpr int N = decltype(n)::value;
    uint4 raw[N][sizeof(T) / 2];
#pragma unroll
    for (int k = 0; k < N; k++)
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); i++)
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(raw[k][i].x), "=r"(raw[k][i].y), "=r"(raw[k][i].z), "=r"(raw[k][i].w)
                     : "l"(reinterpret_cast<const uint4*>(src + k * STEP * D) + i));
    src += N * STEP * D;
#pragma unroll
    for (int k = 0; k < N; k++) {
      float x[8];
      if constexpr (sizeof(T) == 2) widen8(raw[k][0], x);
      else memcpy(x, raw[k], 32);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        finite = finite && isfinite(x[e]);
        lo[e] = fminf(lo[e], x[e]);
        hi[e] = fmaxf(hi[e], x[e]);
      }
    }
  };
  int left = (rows - r0 + STEP - 1) / STEP;
#pragma unroll 1
  for (; left >= 8; left -= 8) take(std::integral_constant<int, 8>());
#pragma unroll 1
  for (; left >= 2; left -= 2) take(std::integral_constant<int, 2>());
  if (left > 0) take(std::integral_constant<int, 1>());
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

// d += a b for one 16 x 8 x 16 tile of fp16 with fp32 sums
__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four codes as two fp16 pairs: behind 0x64 a byte is 1024 and itself, and the code's sign bit turned makes it 128 more.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const __half2 off = __float2half2_rn(1152.f);
  uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off), y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

constexpr int kSelectKeys = 16384;  // pages whose keys fit in shared memory

// A rising key for a score (no NaN, no -0).
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
// TH threads, of which each warp scores sixteen pages at a time.
template <typename T, int D, int TH>
__global__ void __launch_bounds__(TH, 512 / TH) paged_select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int LINE = 2 * D + 8;   // fp16 values of a query's [u-, u+] (rows 4 banks apart)
  constexpr int Q = 2 * D / 64;     // 16-byte pieces a lane of a row
  constexpr int W = TH / 32;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) __half u_s[8 * LINE];
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
  // Another CTA of this launch may set the word between two warps' looks at it, so a CTA leaves by what all its
  // threads have seen: warps that went on alone would place pages by counts that the others never wrote.
  bool bad = status_set(p.b.status);
  const int u = blockIdx.y, s = u / p.Hkv, h = u - s * p.Hkv;
  const int L = paged_len(p.b, s);
  const int nb = (L >> p.b.shift) + 1;
  int32_t* sel = p.sel + static_cast<size_t>(u) * p.n_sel;
  if (L < 0 || nb <= p.n_sel || p.n_sel == p.first + p.last) {  // (the whole cluster)
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (__syncthreads_or(bad) || L < 0 || rank > 0) return;
    const int ends = nb <= p.n_sel ? nb : p.first;
    for (int i = tid; i < p.n_sel; i += TH) sel[i] = i < ends ? i : nb <= p.n_sel ? -1 : nb - p.n_sel + i;
    if (tid == 0) p.count[u] = min(nb, p.n_sel);
    return;
  }
  const int n = nb - p.first - p.last;  // pages to choose from
  const bool kept = n <= p.keys;
  uint32_t* far = p.far + static_cast<size_t>(u) * p.pages;
  const uint32_t keys_at = static_cast<uint32_t>(__cvta_generic_to_shared(keys));
  // Pages are dealt to the warps sixteen at a time, a tile; a warp looks up two tiles' pages and exponents at once.
  // The first tile's codes are on their way while the queries are looked at, each later one's under the products before.
  const int tiles = (n + 15) / 16, stride = W * ctas, tile0 = rank * W + warp;
  uint4 c[2][Q];         // of pages (lane >> 2) and 8 + (lane >> 2): bytes 64 k + 16 (lane & 3) .. of their codes
  int page = -1, e = 0;  // of place (lane & 15) of tile `first of two` + (lane >> 4) * stride
  auto look = [&](int tile) {
    const int j = (tile + (lane >> 4) * stride) * 16 + (lane & 15);
    page = j < n ? page_at(p.b, s, p.first + j) : -1;
    e = page < 0 ? 0 : p.exp[static_cast<size_t>(page) * p.Hkv + h];
  };
  auto codes = [&](int i, int r) {  // of the i-th of the two
    const int x = __shfl_sync(0xffffffffu, page, i * 16 + r * 8 + (lane >> 2));
    return reinterpret_cast<const uint4*>(p.code + (static_cast<size_t>(x < 0 ? 0 : x) * p.Hkv + h) * 2 * D) + (lane & 3);
  };
  auto fetch = [&]() {
    const uint4 *x = codes(0, 0), *y = codes(0, 1);
#pragma unroll
    for (int k = 0; k < Q; k++) {
      c[0][k] = x[k * 4];
      c[1][k] = y[k * 4];
    }
  };
  if (tile0 < tiles) {
    look(tile0);
    fetch();
  }
  // the group's queries in whole steps
  const T* q = static_cast<const T*>(p.q) + (static_cast<size_t>(s) * p.Hq + h * p.G) * D;
  uint32_t top = 0;  // the largest size, as bits (what is not finite comes out above every finite one)
  float mine[8];     // this thread's last eight values (its only ones where the group has eight heads or fewer)
  for (int i = tid; i < p.G * D / 8; i += TH) {
    load8(q + i * 8, mine);
#pragma unroll
    for (int c = 0; c < 8; c++) top = max(top, __float_as_uint(mine[c]) & 0x7fffffffu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) red_s[warp] = top;
  bad = __syncthreads_or(bad) != 0;
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
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  for (int g0 = 0; g0 < p.G; g0 += 8) {
    if (g0 > 0) __syncthreads();
#pragma unroll
    for (int i8 = tid; i8 < D; i8 += TH) {  // (eight values each of eight heads)
      const int g = i8 / (D / 8), d = i8 % (D / 8) * 8;
      float x[8];
      if (finite && g0 + g < p.G) {
        if (TH == 256 && p.G <= 8) {
#pragma unroll
          for (int i = 0; i < 8; i++) x[i] = mine[i];
        } else {
          load8(q + static_cast<size_t>(g0 + g) * D + d, x);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = 0.f;
      }
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float v0 = rintf(__fmul_rn(__fmul_rn(x[i], by1), by2)), v1 = rintf(__fmul_rn(__fmul_rn(x[i + 1], by1), by2));
        const __half2 a = __floats2half2_rn(fminf(v0, 0.f), fminf(v1, 0.f)), b = __floats2half2_rn(fmaxf(v0, 0.f), fmaxf(v1, 0.f));
        lo[i / 2] = *reinterpret_cast<const uint32_t*>(&a);
        hi[i / 2] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(u_s + g * LINE + d) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(u_s + g * LINE + D + d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
    __syncthreads();
    const int live = min(8, p.G - g0);
    const __half* row = u_s + (lane >> 2) * LINE + (lane & 3) * 16;
    for (int two = tile0; two < tiles; two += 2 * stride) {
      if (g0 > 0 || two > tile0) {
        look(two);
        fetch();
      }
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int tile = two + i * stride;
        if (tile >= tiles) break;
        const bool next = i == 0 && tile + stride < tiles;
        const uint4 *x = codes(1, 0), *y = codes(1, 1);
        float d[2][4];  // (two sums: products that follow one another wait)
#pragma unroll
        for (int k = 0; k < 4; k++) d[0][k] = d[1][k] = 0.f;
#pragma unroll
        for (int k = 0; k < Q; k++) {
          const uint4 u0 = *reinterpret_cast<const uint4*>(row + k * 64), u1 = *reinterpret_cast<const uint4*>(row + k * 64 + 8);
          const uint32_t w0[4] = {c[0][k].x, c[0][k].y, c[0][k].z, c[0][k].w}, w1[4] = {c[1][k].x, c[1][k].y, c[1][k].z, c[1][k].w};
          const uint32_t u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
          for (int j = 0; j < 4; j++) {
            uint32_t a0, a1, a2, a3;
            widen4(w0[j], a0, a2);
            widen4(w1[j], a1, a3);
            mma16816_f16(d[j & 1], a0, a1, a2, a3, u[2 * j], u[2 * j + 1]);
          }
          if (next) {
            c[0][k] = x[k * 4];
            c[1][k] = y[k * 4];
          }
        }
        // the highest of the heads there are, of pages (lane >> 2) and 8 + (lane >> 2)
        const int h0 = (lane & 3) * 2;
        float best[2];
#pragma unroll
        for (int r = 0; r < 2; r++) {
          float v = h0 < live ? __fadd_rn(d[0][2 * r], d[1][2 * r]) : -INFINITY;
          if (h0 + 1 < live) v = fmaxf(v, __fadd_rn(d[0][2 * r + 1], d[1][2 * r + 1]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          best[r] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        }
        const int r = lane & 1, at = r * 8 + (lane >> 2), j = tile * 16 + at;
        const int ex = __shfl_sync(0xffffffffu, e, i * 16 + at);
        if ((lane & 2) == 0 && j < n) {
          uint32_t key = rising(ex >= 128 ? INFINITY : ldexpf(__fadd_rn(best[r], 0.f), ex - 24));
          if (kept) {  // (later heads' scores of a page are this lane's own again)
            if (g0 > 0) key = max(key, load_first(keys_at + j * 4));
            store_first(keys_at + j * 4, key);
          } else {
            far[j] = g0 > 0 ? max(key, far[j]) : key;
          }
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
  // ---- the choice: a run of keys a thread; three to eight in registers (shared memory then holds all of them), one or two in
  // a loop, since all of this runs once, from cold code (64 pages 4.5 us, 4.7 from registers; 2,048 pages 8.7, 10.0 in a loop)
  constexpr int RUN = 8;
  const int run = (n + TH - 1) / TH, i0 = min(tid * run, n), i1 = min(i0 + run, n);
  const bool few = run > 2 && run <= RUN;
  uint32_t own[RUN];
  if (few) {
#pragma unroll
    for (int j = 0; j < RUN; j++) own[j] = i0 + j < i1 ? keys[i0 + j] : 0u;
  }
  auto each = [&](auto f) {
    if (few) {
#pragma unroll
      for (int j = 0; j < RUN; j++)
        if (i0 + j < i1) f(i0 + j, own[j]);
    } else {
#pragma unroll 1
      for (int i = i0; i < i1; i++) f(i, kept ? keys[i] : __ldcg(far + i));
    }
  };
  uint32_t low = 0xffffffffu, high = 0;
  each([&](int, uint32_t k) {
    low = min(low, k);
    high = max(high, k);
  });
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    red_s[warp] = low;
    red2_s[warp] = high;
  }
  for (int i = tid; i < 256; i += TH) hist[i] = 0;
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
    each([&](int, uint32_t x) {
      const uint32_t k = x - low;
      if (bits == 32 || (k >> bits) == (prefix >> bits)) atomicAdd(&hist[(k >> shift) & mask], 1);
    });
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
    all = left_s == need_s;  // the whole digit is taken
    bits = shift;
    for (int i = tid; i < 256; i += TH) hist[i] = 0;
    __syncthreads();
  }
  // every higher key, and of those that share all bits found the first `need`: the threads' counts summed over the CTA
  const uint32_t border = prefix >> bits;
  int higher = 0, equal = 0;
  each([&](int, uint32_t x) {
    const uint32_t k = (x - low) >> bits;
    higher += k > border;
    equal += k == border;
  });
  int more_in = higher, same_in = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, more_in, o), y = __shfl_up_sync(0xffffffffu, same_in, o);
    if (lane >= o) {
      more_in += x;
      same_in += y;
    }
  }
  if (lane == 31) {
    part[warp][0] = more_in;
    part[warp][1] = same_in;
  }
  __syncthreads();
  int before = more_in - higher, same = same_in - equal;
#pragma unroll
  for (int w = 0; w < W; w++)
    if (w < warp) {
      before += part[w][0];
      same += part[w][1];
    }
  int place = p.first + before + min(same, need);  // (where a digit was taken whole, need is all of the equal ones)
  each([&](int i, uint32_t x) {
    const uint32_t k = (x - low) >> bits;
    if (k > border || (k == border && same++ < need)) sel[place++] = p.first + i;
  });
  for (int i = tid; i < p.first; i += TH) sel[i] = i;
  for (int i = tid; i < p.last; i += TH) sel[p.n_sel - p.last + i] = nb - p.last + i;
  if (tid == 0) p.count[u] = p.n_sel;
}

// ---------------------------------------------------------------------------
// advance
// ---------------------------------------------------------------------------
__global__ void paged_advance_kernel(int32_t* len, const int32_t* row_off, PagedSeqs b, int n_total, int n_max) {
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  pdl_wait();
  if (s >= b.n_seq || status_set(b.status)) return;
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
template <typename T, int D, int TH>
static bool launch_select_t(const SelectParams& p, int ctas, int units, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  const int bytes = p.keys * 4;
  if (!allow_smem(paged_select_kernel<T, D, TH>, kSelectKeys * 4, set)) return false;
  if (ctas > 1) launch_k_cluster(true, ctas, paged_select_kernel<T, D, TH>, dim3(ctas, units), dim3(TH), bytes, st, p);
  else launch_k(true, paged_select_kernel<T, D, TH>, dim3(1, units), dim3(TH), bytes, st, p);
  return true;
}
template <int D>
static bool launch_select_d(const SelectParams& p, bool bf, int ctas, int units, cudaStream_t st) {
  // CTAs of 256 threads while all run at once (two an SM), else of 128: 364 slots' heads of some 85 pages 8.9 us and 12.5
  // with 256, 372 of some 160 10.1 and 12.5, 1,168 that choose nothing 2.2 and 3.5.
  if (units <= 2 * num_sms()) return bf ? launch_select_t<__nv_bfloat16, D, 256>(p, ctas, units, st) : launch_select_t<float, D, 256>(p, ctas, units, st);
  return bf ? launch_select_t<__nv_bfloat16, D, 128>(p, ctas, units, st) : launch_select_t<float, D, 128>(p, ctas, units, st);
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
  if (!apart(b->status, {{code, heads * 2 * l->D}, {exp, heads * 4}}, {{l->K, pool}, offsets_of(b, rows), table_of(b), lens_of(b)})) return TV_ERR_ARG;
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
  const size_t units_b = static_cast<size_t>(b->n_seq) * l->Hkv, heads = static_cast<size_t>(l->n_pages) * l->Hkv;
  const size_t need = tv_paged_select_workspace_bytes(l, b);
  if (need > 0 && (!ws || ws_bytes < need)) return TV_ERR_WORKSPACE;
  // lists are written while others' bounds and queries are read
  if (!apart(b->status, {{sel, units_b * n_sel * 4}, {count, units_b * 4}, {ws, need}},
             {{code, heads * 2 * l->D}, {exp, heads * 4}, {q, bytes_of(b->n_seq, static_cast<int64_t>(l->Hq) * l->D, l->dtype)}, table_of(b), lens_of(b)}))
    return TV_ERR_ARG;
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
  // CTAs for a slot's KV head: up to eight, while all run at once (two an SM) and each has 128 pages (the queries' codes take each as
  // long as some 100 pages)
  int ctas = 1;
  while (ctas < 8 && units * ctas <= num_sms() && ctas * 2 * 128 <= most) ctas *= 2;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = l->dtype == TV_BF16;
  const bool ok = l->D == 64 ? launch_select_d<64>(p, bf, ctas, units, st) : l->D == 128 ? launch_select_d<128>(p, bf, ctas, units, st)
                                                                                        : launch_select_d<256>(p, bf, ctas, units, st);
  return ok ? launch_status() : TV_ERR_CUDA;
}

extern "C" tv_status tv_paged_advance(const tv_paged* b, const tv_paged_rows* rows, int32_t* len, tv_stream stream) {
  if (!b || !b->len || !b->status || !len || b->n_seq < 1 || b->n_seq > TV_MAX_PAGED_SEQ || b->max_len < 0 || b->max_len >= 1 << 30 || len != b->len) return TV_ERR_ARG;
  if (!aligned16(b->len) || !aligned16(b->status)) return TV_ERR_ALIGN;
  const tv_status c = paged_rows_check(rows);
  if (c != TV_OK) return c;
  if (!apart(b->status, {lens_of(b)}, {offsets_of(b, rows)})) return TV_ERR_ARG;
  const PagedSeqs v{nullptr, b->len, b->status, b->n_seq, 0, b->max_len, 0, 0};
  launch_k(true, paged_advance_kernel, dim3((b->n_seq + 127) / 128), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), len,
           rows ? rows->row_off : nullptr, v, rows ? rows->n_total : 0, rows ? rows->n_max : 0);
  return launch_status();
}
