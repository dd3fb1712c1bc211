// Decode attention over bf16 caches in pages, on the tensor cores.
//
// A unit is one slot and KV head: its G query heads (eight at a time, or sixteen: an
// item) against the keys and values that the slot sees, in tiles of 64 rows (128
// of 64 columns).  Each tile is used by so few query rows that the call is bound by
// the reads of keys and values; the products run on warp-level tiles (16 x 8 x 16)
// with the cache on the long side, S^T = K Q^T and O^T = V^T P^T, so that eight heads
// fill them.  An item runs flash style:
//   m = running maximum of the scaled scores, p = 2^(s c - m) rounded to bf16 for
//   the product with V, l += p (fp32, as they were), O = O a + P V.
// p is rounded because the tensor cores take P and V in one type; each weight is
// off by 2^-8 of itself at most, independently, and l adds them unrounded.
//
// Work split.  The tiles of all items, one behind another, are cut into one
// range of equal length for each CTA (one per SM), so every SM streams the same
// number of bytes whatever the lengths are.  An item that lies in one CTA's range
// is written by it; one that a cut goes through leaves a piece (O, m and l in fp32)
// with each of its CTAs, two a CTA at most, and the join adds them up.  Where the host's bounds
// leave no item more than a few tiles, ranges end with items and there is no join.  Every
// CTA finds its range from the device-side lengths by itself.
//
// Roles.  A producer warp brings keys and values by TMA; it reads the table (and
// the selection) 32 entries at a time, a batch ahead.  Two teams of four warps take
// turns at the tiles, each with its own ring of slots, O, m and l, joined at the end
// of an item.  (One ring for both would not do: a team would wait for a slot's
// next filling but one without having seen the one between, which the other
// takes, and copies do not land in order: the parity of a barrier cannot tell them
// apart.)  Within a team a warp scores 16 of the tile's 64 rows and,
// when the scores have gone through shared memory, owns a quarter of the columns
// of O; every warp forms all 16 x 64 weights for itself, in registers, where its
// products want them.
//
// Masked rows (behind len[s], in the last page of the slot): the scores are
// replaced, and the values zeroed in shared memory (a weight of zero would still
// make NaN of an infinity there).  Pages hold whole rows behind the last one, so
// nothing outside the pools is read.
//
// Bound by HBM while slots are long: 8 slots of 65,536 rows (1.07 GB, pages of 64) 161 to 169 us for
// heads of 64, 128 and 256, 0.95 to 0.99 of a copy's rate; 96 ragged slots up to 32,768 rows
// (16 + 2 heads of 128, pages of 32, 563 MB) 94.3 us, 6.0 TB/s, 0.88: some 3 us until the first tile is there, the
// pieces and the join are the rest.  Short slots are bound by latency: 4 up to 1,025 rows (24 + 4 heads of 256)
// 9.9 us, of which the lengths, the table, keys and values are reads one behind the other, some 3.4 the join.
// Heads of 64 in pages of 16 rows reach 0.66: a copy of 2 KB a page is too small.  More than sixteen query heads a KV head
// walk its keys and values once for each sixteen: 8 slots of 65,536 rows, 1 KV head of 128 (39.8 us of bytes), 49.7 us with 8 query heads,
// 51.9 with 16, 91.0 with 32, 165 with 64, 314 with 128.
// (Query heads on the long side of the tiles, as many as 16 fill: 256 slots of 100 rows 46 us against 35.)
#include <algorithm>
#include <cstring>

#include "attn_paged.cuh"
#include "attn_paged_prefix.cuh"
#include "mma_tile.cuh"
#include "ptx.cuh"
#include "tensor_map.hpp"

namespace tv {

constexpr int kItemMax = 16;  // query heads of an item, at most
constexpr int kConsumers = 256, kThreads = kConsumers + 32;

template <int D, int NB>
struct Pg {
  // Rows of a key tile: with 64 columns a tile of 64 rows is over before the next
  // barrier: 8 slots of 65,536 rows, 8 + 8 heads of 64, 171 us with 128 rows, 296 with 64.
  static constexpr int ROWS = D == 64 ? 128 : 64;
  static constexpr int EXTRA = D == 256 ? 1 : 2;         // steps of an item beside its tiles
  static constexpr int WR = ROWS / 4, SG = ROWS / 16;    // rows a warp scores, groups of 16 rows
  static constexpr int SLOT = ROWS * D * 2;              // a tile of keys or of values
  static constexpr int NS = D == 256 ? 3 : D == 128 ? 6 : 5;  // slots of a team's ring
  static constexpr int HEADS = 8 * NB;                   // query heads of an item
  static constexpr int CPW = D / 4, MT = CPW / 16;       // columns of O a warp, in tiles of 16
  static constexpr int SLD = ROWS + 8;                   // floats of a head's scores (conflict-free pairs)
  static constexpr int SBUF = HEADS * SLD * 4;
  static constexpr int OLD = D + 4;                      // floats of a head of O
  static constexpr int SOFF = 2 * NS * SLOT;             // scores [team][2]
  static constexpr int OOFF = SOFF + 4 * SBUF;           // the teams' O, eight heads at a time: [team][8]
  static constexpr int MOFF = OOFF + 2 * 8 * OLD * 4;    // and m, l: [team][HEADS]
  static constexpr int VOFF = MOFF + 2 * HEADS * 8;      // rows seen of each 16 of a slot's tile: [2 NS][SG]
  static constexpr int BOFF = VOFF + 2 * NS * SG * 4;
  static constexpr int LOFF = BOFF + 4 * NS * 8;
  static constexpr int SMEM = LOFF + 128 + 128;
  static_assert(SMEM <= 232448, "shared memory");
};

struct PagedTcParams {
  CUtensorMap tmK, tmV;  // pools as [D / 64][rows][64], boxes of R whole rows
  PagedView v;
  const int32_t* group_off;  // groups of slots with shared prefixes, or null
  const int32_t* shared;
  int n_group;
  int32_t* start;        // [n_seq] rows that the kernel for shared prefixes sees to, or null
  const __nv_bfloat16* q;
  const __nv_bfloat16* gate;
  __nv_bfloat16* out;
  int2* span;      // [items] first and last CTA of an item's tiles (with shared prefixes; 0, -1: none)
  int4* cut;       // [CTAs] the item that a CTA's range starts within, where it is the item's first cut:
                   // slot, KV head, item of it, last CTA; -1: none
  float* rec;      // [2 * CTAs][heads][D + 4]
  float* rec_item;  // [items][heads][D + 4]: items of slots with a shared prefix
  const float* rec_prefix;  // [pieces][128][D + 4]
  const int4* info;         // [n_seq], as the kernel for shared prefixes leaves it
  int Hq, G, MT, units;  // MT items a unit
  int item;              // query heads of an item
  int R;  // rows of a box: a page's, or a tile's
  int uncut;  // 1: ranges end with items, and there is nothing to join
  float c;        // scale * log2(e)
  uint32_t zero;  // 0
};

// Tiles of an item of unit u.
template <int ROWS>
__device__ __forceinline__ int unit_tiles(const PagedTcParams& p, int u, int s, int L) {
  if (L < 0) return 0;
  if (p.v.sel) return ((p.v.pages(s, u - s * p.v.Hkv, L) << p.v.b.shift) + ROWS - 1) / ROWS;
  return (L + 1 - (p.start ? p.start[s] : 0) + ROWS - 1) / ROWS;
}

constexpr int kNear = 16;

// Ranges are cut in steps: an item's tiles, and before them what it costs beside them (its start, the teams' join, its
// end: some 2,500 cycles, while a tile of 256 columns has 3,000 cycles of the memory's rate and a smaller one 1,500).
// 96 ragged slots of 16 + 2 heads of 128: 94.9 us, 97.5 by tiles alone.
__device__ __forceinline__ int steps_of(int tiles, int extra) { return tiles > 0 ? tiles + extra : 0; }

template <int ROWS>
__device__ __forceinline__ int unit_tiles(const PagedTcParams& p, int u) {
  const int s = u / p.v.Hkv;
  return unit_tiles<ROWS>(p, u, s, paged_len(p.v.b, s));
}

// The items of a range of tiles, one after another.
struct PagedPiece {
  int s, h, L, m, k0, k1, nt;  // slot, KV head, the slot's length, item, tiles [k0, k1) of nt
};
template <int ROWS, int EXTRA>
struct PagedWalk {
  int u, s, h;          // unit: slot and KV head
  int u0;               // the first unit of the range, and
  const int2* near;     // tiles and length of that one and the kNear - 1 after it
  int off;  // step within the unit, over its items (under 2^28: a slot has 2^30 rows at most, a unit 8 items)
  int64_t left;
  __device__ __forceinline__ bool next(const PagedTcParams& p, PagedPiece& x) {
    while (left > 0 && u < p.units) {
      const int2 n = u - u0 < kNear ? near[u - u0] : make_int2(unit_tiles<ROWS>(p, u), paged_len(p.v.b, s));
      const int steps = steps_of(n.x, EXTRA);
      if (off >= steps * p.MT) {
        off = 0;
        u++;
        if (++h == p.v.Hkv) {
          h = 0;
          s++;
        }
        continue;
      }
      x.s = s;
      x.h = h;
      x.L = n.y;
      x.m = off < steps ? 0 : off / steps;
      const int from = off - x.m * steps, to = static_cast<int>(min(static_cast<int64_t>(steps), from + left));
      off += to - from;
      left -= to - from;
      x.k0 = max(from - EXTRA, 0);
      x.k1 = max(to - EXTRA, 0);
      x.nt = n.x;
      if (x.k0 < x.k1) return true;
    }
    return false;
  }
};
// CTAs that share `total` tiles, and where CTA c's range starts.
// (in 32 bits where they do: 64-bit divisions took a sixth of a small call)
constexpr int64_t kFewTiles = 1 << 22;  // times 1,024 CTAs at most
__device__ __forceinline__ int64_t range_start(int64_t total, int ctas, int c) {
  if (total < kFewTiles) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(ctas);
  return total * c / ctas;
}
__device__ __forceinline__ int range_of(int64_t total, int ctas, int64_t tile) {
  if (total < kFewTiles) return static_cast<int>((static_cast<uint32_t>(tile + 1) * static_cast<uint32_t>(ctas) - 1u) / static_cast<uint32_t>(total));
  return static_cast<int>(((tile + 1) * ctas - 1) / total);
}
__device__ __forceinline__ int ctas_for(int64_t total, int grid) { return static_cast<int>(min(static_cast<int64_t>(grid), total)); }

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void sts1(uint32_t a, float x) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory"); }
__device__ __forceinline__ float2 lds2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, 1) attn_paged_tc_kernel(const __grid_constant__ PagedTcParams p) {
  using C = Pg<D, NB>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // tiles are swizzled in 1024-byte atoms
  const uint32_t sb = smem_u32(smem_raw);
  const uint32_t FULL0 = sb + C::BOFF, EMPTY0 = FULL0 + 16u * C::NS;
  int32_t* seen_s = reinterpret_cast<int32_t*>(smem_raw + C::VOFF);
  struct Local {
    int64_t left, before, total, at, end;
    int u, off, skip, ctas;
    int abort_flag;
  };
  Local& lo = *reinterpret_cast<Local*>(smem_raw + C::LOFF);
  int64_t* sums = reinterpret_cast<int64_t*>(smem_raw + C::SOFF);  // tiles of each warp's units (scores are not in use yet)
  static_assert(sizeof(Local) <= 128, "local data");
  int2* lo_near = reinterpret_cast<int2*>(smem_raw + C::LOFF + 128);
  volatile int* abort_flag = &lo.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * C::NS; i++) {
      mbar_init(FULL0 + 8u * i, 1);
      mbar_init(EMPTY0 + 8u * i, 4);
    }
    lo.abort_flag = 0;
    lo.left = 0;
    lo.u = 0;
    lo.off = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (threadIdx.x == 0) {
    lo.skip = status_set(p.v.b.status) || (sb & 1023u) ? 1 : 0;
    if (sb & 1023u) set_status(p.v.b.status, TV_ERR_CUDA);
  }
  __syncthreads();
  if (lo.skip) return;
  if (p.group_off) {  // (every CTA writes the same)
    int* at = reinterpret_cast<int*>(smem_raw);  // (the rings are not in use yet)
    constexpr int N = TV_MAX_PAGED_SEQ + 4;
    GroupCheck<kThreads> check{at, at + N, at + 2 * N, at + 3 * N, at + 4 * N, reinterpret_cast<unsigned long long*>(at + 5 * N)};
    const int code = check.run(p.v.b, p.group_off, p.shared, p.n_group, kv_row_bytes(p.v.Hkv, D), 0);
    if (code) {
      set_status(p.v.b.status, code);
      return;
    }
    for (int s = threadIdx.x; p.start && s < p.v.b.n_seq; s += kThreads) p.start[s] = check.rows[check.of(p.n_group, s)];
    fence_proxy_async_smem();
    __syncthreads();
  }
  // this CTA's range: a run of units for each thread, their tiles summed over the CTA
  int64_t left;
  {
    const int per = (p.units + kThreads - 1) / kThreads;
    const int u0 = min(static_cast<int>(threadIdx.x) * per, p.units), u1 = min(u0 + per, p.units);
    int64_t mine = 0;
    int2 last = make_int2(0, -1);  // of the thread's only unit, where it has one
    for (int u = u0; u < u1; u++) {
      const int s = u / p.v.Hkv;
      last.y = paged_len(p.v.b, s);
      last.x = unit_tiles<C::ROWS>(p, u, s, last.y);
      mine += static_cast<int64_t>(steps_of(last.x, C::EXTRA)) * p.MT;
      // an empty list: zeros (by the thread that has met it: a look at a CTA's share of the units takes a read of the
      // count behind one of the length for each, one by one; 46 slots 18.5 us with their selection and 20.1)
      if (last.x == 0 && last.y >= 0 && u % gridDim.x == blockIdx.x) {
        uint4* out = reinterpret_cast<uint4*>(p.out + (static_cast<size_t>(s) * p.Hq + (u - s * p.v.Hkv) * p.G) * D);
        for (int i = 0; i < p.G * D / 8; i++) out[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t base = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
      if (w < warp) base += sums[w];
      total += sums[w];
    }
    const int ctas = ctas_for(total, gridDim.x), me = static_cast<int>(blockIdx.x);
    if (me == 0 && p.start) {  // for the join
      int64_t at = base;
      for (int u = u0; u < u1; u++) {
        const int tiles = per == 1 ? last.x : unit_tiles<C::ROWS>(p, u), steps = steps_of(tiles, C::EXTRA);
        for (int m = 0; m < p.MT; m++, at += steps)
          p.span[u * p.MT + m] = tiles > 0 ? make_int2(range_of(total, ctas, at + C::EXTRA), range_of(total, ctas, at + steps - 1)) : make_int2(0, -1);
      }
    }
    if (threadIdx.x == 0) lo.ctas = ctas;
    if (me < ctas) {
      const int64_t a = range_start(total, ctas, me), b = range_start(total, ctas, me + 1);
#pragma unroll 1
      for (int k = 0; k <= p.uncut; k++) {
        const int64_t t = k ? b : a;
        if (t < base || t >= base + mine) continue;
        int64_t at = base;
        int u = u0, steps;
        for (;; u++) {
          steps = steps_of(per == 1 ? last.x : unit_tiles<C::ROWS>(p, u), C::EXTRA);
          if (t < at + static_cast<int64_t>(steps) * p.MT || u + 1 >= u1) break;
          at += static_cast<int64_t>(steps) * p.MT;
        }
        int off = static_cast<int>(t - at);
        if (p.uncut) off = (off + steps - 1) / steps * steps;  // where the next item starts
        if (k) {
          lo.end = at + off;
        } else {
          lo.u = u;
          lo.off = off;
          lo.left = b - a;
          lo.before = me > 0 ? a - range_start(total, ctas, me - 1) : 0;
          lo.total = total;
          lo.at = at + off;
        }
      }
      if (b == total && threadIdx.x == 0) lo.end = total;
    }
    __syncthreads();
    left = p.uncut && me < ctas ? lo.end - lo.at : lo.left;
    if (left > 0) {  // what the next units hold
      if (per == 1) {
        if (u0 < u1 && u0 >= lo.u && u0 < lo.u + kNear) lo_near[u0 - lo.u] = last;
      } else if (threadIdx.x < kNear && lo.u + static_cast<int>(threadIdx.x) < p.units) {
        const int u = lo.u + threadIdx.x, s = u / p.v.Hkv, L = paged_len(p.v.b, s);
        lo_near[threadIdx.x] = make_int2(unit_tiles<C::ROWS>(p, u, s, L), L);
      }
    }
    __syncthreads();
  }
  PagedWalk<C::ROWS, C::EXTRA> walk{lo.u, lo.u / p.v.Hkv, lo.u % p.v.Hkv, lo.u, lo_near, lo.off, left};
  PagedPiece x;
  pdl_trigger();
  if (warp == kConsumers / 32) {
    // ---------------- producer ----------------
    const int R = p.R, nsub = C::ROWS / R, rows = 1 << p.v.b.shift, per_page = rows / R;
    uint32_t tile = 0;                // tiles of the CTA
    uint32_t fills0 = 0, fills1 = 0;  // of each team's ring
    bool ok = true;
    // part i of a piece's item: box rows i * R .. of its rows: its row in the pools, -1: none; rows of it that are seen
    auto part = [&](const PagedPiece& x, int i, int& seen) -> int {
      seen = 0;
      if (i >= x.k1 * nsub) return -1;
      const int place = (p.start ? p.start[x.s] >> p.v.b.shift : 0) + i / per_page;
      if (place >= p.v.pages(x.s, x.h, x.L)) return -1;
      const int col = p.v.column(x.s, x.h, place);
      if (col < 0) return -1;
      const int r = (i % per_page) * R, n = min(R, x.L + 1 - (col * rows + r));
      if (n <= 0) return -1;
      const int page = page_at(p.v.b, x.s, col);
      if (page < 0) return -1;
      seen = n;
      return (page * p.v.Hkv + x.h) * rows + r;
    };
    PagedPiece y;
    bool more = walk.next(p, x);
    int row = -1, seen = 0, row2 = -1, seen2 = 0, next_row = -1, next_seen = 0;
    if (more) row = part(x, x.k0 * nsub + lane, seen);
    if (lane == 0) {  // where this CTA's range starts within an item, for the join
      int4 c = make_int4(-1, 0, 0, 0);
      if (more && x.k0 > 0 && x.k0 <= lo.before)
        c = make_int4(x.s, x.h, x.m, range_of(lo.total, lo.ctas, lo.at - x.k0 + x.nt - 1));
      p.cut[blockIdx.x] = c;
    }
    while (ok && more) {
      bool following = false;
      int i0 = x.k0 * nsub;
      for (int k = x.k0; k < x.k1 && ok; k++, tile++) {
        const int at = (k - x.k0) * nsub % 32;
        if (at == 0 && k != x.k0) {
          row = row2;
          seen = seen2;
          i0 += 32;
        }
        // of this tile: part y's row and count in lane at + y
        const int mine = __shfl_sync(0xffffffffu, row, min(at + lane, 31));  // this lane's box
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, lane < nsub && mine >= 0)) * R * D * 2;
        // rows seen of each 16 of the tile
        const int q16 = lane & (C::SG - 1), py = q16 * 16 / R;
        const int cnt = min(16, max(0, __shfl_sync(0xffffffffu, seen, at + py) - (q16 * 16 - py * R)));
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
          const uint32_t it = tile & 1 ? fills1 : fills0, slot = (tile & 1) * C::NS + it % C::NS, full = FULL0 + 8u * slot;
          ok = ok && wait_warp(EMPTY0 + 8u * slot, ((it / C::NS) & 1) ^ 1, abort_flag, kWaitCycles);
          if (!ok) break;
          if (tile & 1) fills1++;
          else fills0++;
          if (lane < C::SG) seen_s[slot * C::SG + lane] = cnt;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(full, bytes);
          __syncwarp();
          if (lane < nsub && mine >= 0) tma_load_3d(sb + slot * C::SLOT + lane * R * D * 2, kv ? &p.tmV : &p.tmK, full, 0, mine, 0);
          __syncwarp();
        }
        if (at == 0) row2 = part(x, i0 + 32 + lane, seen2);  // the next 32, under this tile's copies
        if (k == x.k0) {                                     // and the next piece's first
          following = walk.next(p, y);
          if (following) next_row = part(y, y.k0 * nsub + lane, next_seen);
        }
      }
      x = y;
      more = following;
      row = next_row;
      seen = next_seen;
    }
    if (!ok && lane == 0) set_status(p.v.b.status, TV_ERR_TIMEOUT);
    // every issued copy lands before shared memory is released
    for (uint32_t team = 0; team < 2; team++) {
      const uint32_t it = team ? fills1 : fills0;
      for (uint32_t i = it > C::NS ? it - C::NS : 0; i < it; i++)
        mbar_wait(FULL0 + 8u * (team * C::NS + i % C::NS), (i / C::NS) & 1, kWaitCycles);
    }
    return;
  }

  // ---------------- consumers ----------------
  const int team = warp >> 2, w = warp & 3;
  // in a 16 x 8 result this lane has rows gr, gr + 8 and columns gc, gc + 1; in a second operand column gr
  const int gr = lane >> 2, gc = (lane & 3) * 2;
  const uint32_t sc0 = sb + C::SOFF + team * 2 * C::SBUF;
  float* o_s = reinterpret_cast<float*>(smem_raw + C::OOFF);
  float2* ml_s = reinterpret_cast<float2*>(smem_raw + C::MOFF);
  uint32_t tile = 0, turn = 0;  // tiles of the CTA, tiles of this team
  bool ok = true;  // (a warp whose wait gave up goes on through the barriers, idle)
  const f2_t c2 = f2_dup(p.c);
  // a tile lies as its boxes do: [box][64 columns][R rows][128 bytes]
  const uint32_t chunk = p.R * 128, rmask = p.R - 1;
  auto row_at = [&](uint32_t r) { return (r & ~rmask) * (D * 2) + (r & rmask) * 128; };
  // query heads of an item, straight into the second operand's layout
  uint32_t qb[NB][D / 16][2];
  auto load_q = [&](const PagedPiece& x) {
    const int heads = min(C::HEADS, p.G - x.m * C::HEADS);
    const __nv_bfloat16* q = p.q + (static_cast<size_t>(x.s) * p.Hq + x.h * p.G + x.m * C::HEADS) * D + gc;
#pragma unroll
    for (int b = 0; b < NB; b++) {  // (past the last head: the first again, never written)
      const uint32_t* src = reinterpret_cast<const uint32_t*>(q + static_cast<size_t>(gr + 8 * b < heads ? gr + 8 * b : 0) * D);
#pragma unroll
      for (int kk = 0; kk < D / 16; kk++) {
        qb[b][kk][0] = src[kk * 8];
        qb[b][kk][1] = src[kk * 8 + 4];
      }
    }
  };
  bool more = walk.next(p, x);
  if (more) load_q(x);
  while (more) {
    const int heads = min(C::HEADS, p.G - x.m * C::HEADS);
    PagedPiece y;
    const bool following = walk.next(p, y);
    bool loaded = !following;  // the next piece's queries: under this one's last tile
    float o[NB][C::MT][4];     // O transposed: columns of the cache by query heads
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int n = 0; n < C::MT; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[b][n][e] = 0.f;
    float m[NB], l[NB];  // of head gr (+ 8)
#pragma unroll
    for (int b = 0; b < NB; b++) {
      m[b] = -INFINITY;
      l[b] = 0.f;
    }
    bool met = false;
    for (int k = x.k0; k < x.k1; k++, tile++) {
      if ((tile & 1) != static_cast<uint32_t>(team)) continue;
      const uint32_t r0 = team * C::NS, ki = 2 * turn, vi = ki + 1;  // fills of this team's ring
      const uint32_t ks = r0 + ki % C::NS, kph = (ki / C::NS) & 1, vs = r0 + vi % C::NS, vph = (vi / C::NS) & 1;
      const uint32_t sc = sc0 + (turn & 1) * C::SBUF;
      turn++;
      // S transposed = K Q^T, this warp's rows of keys
      ok = ok && wait_warp(FULL0 + 8u * ks, kph, abort_flag, kWaitCycles);
      int vis[C::SG / 4], most = 0;  // rows seen of this warp's groups of 16
      bool whole_tile = ok;
#pragma unroll
      for (int i = 0; i < C::SG; i++) {
        const int n = ok ? seen_s[ks * C::SG + i] : 0;
        whole_tile = whole_tile && n == 16;
        most = max(most, n);
      }
#pragma unroll
      for (int i = 0; i < C::SG / 4; i++) vis[i] = ok ? seen_s[ks * C::SG + w * (C::SG / 4) + i] : 0;
      met = met || most > 0;
#pragma unroll
      for (int i = 0; i < C::SG / 4; i++) {  // 16 rows: within one box
        float s0[NB][2][4];                  // (two sums: products that follow one another wait)
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
          for (int e = 0; e < 4; e++) s0[b][0][e] = s0[b][1][e] = 0.f;
        if (ok) {
          const int kr = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
          const uint32_t kb = sb + ks * C::SLOT + row_at(w * C::WR + i * 16) + kr * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; kk++) {
            uint32_t a[4];
            ldsm_x4(kb + (kk >> 2) * chunk + ((((kk & 3) * 2 + half) ^ (kr & 7)) << 4), a);
#pragma unroll
            for (int b = 0; b < NB; b++) mma16816(s0[b][kk & 1], a, qb[b][kk][0], qb[b][kk][1]);
          }
        }
        const bool lo_in = gr < vis[i], hi_in = gr + 8 < vis[i];
        const uint32_t at = sc + (gc * C::SLD + w * C::WR + i * 16 + gr) * 4;
#pragma unroll
        for (int b = 0; b < NB; b++) {
          float s[4];
#pragma unroll
          for (int e = 0; e < 4; e++) s[e] = (e < 2 ? lo_in : hi_in) ? __fadd_rn(s0[b][0][e], s0[b][1][e]) : -INFINITY;
          sts1(at + b * 8 * C::SLD * 4, s[0]);
          sts1(at + (b * 8 + 1) * C::SLD * 4, s[1]);
          sts1(at + b * 8 * C::SLD * 4 + 32, s[2]);
          sts1(at + (b * 8 + 1) * C::SLD * 4 + 32, s[3]);
        }
      }
      // Only now: an arrival does not wait for loads, the stores have waited for the
      // products and these for theirs.
      __syncwarp();
      if (lane == 0) mbar_arrive(EMPTY0 + 8u * ks);
      if (!loaded && k + 2 >= x.k1) {
        load_q(y);
        loaded = true;
      }
      ok = ok && wait_warp(FULL0 + 8u * vs, vph, abort_flag, kWaitCycles);
      if (!whole_tile && ok) {  // values that nothing sees, of this warp's rows
#pragma unroll
        for (int i = 0; i < C::SG / 4; i++) {
          const uint32_t vb = sb + vs * C::SLOT + row_at(w * C::WR + i * 16);
          constexpr int RW = 256 / D;  // rows at a time
          const int e = lane % (D / 8);
          for (int r = vis[i] + lane / (D / 8); r < 16; r += RW)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (e >> 3) * chunk + r * 128 + (e & 7) * 16), "r"(0) : "memory");
        }
        fence_proxy_async_smem();  // before the slot's next copy
      }
      bar_sync(1 + team, 128);
      // weights of head gr (+ 8), in the second operand's layout
      uint32_t pb[NB][C::SG][2];
#pragma unroll
      for (int b = 0; b < NB; b++) {
        float2 sv[C::SG][2];
        float mx = -INFINITY;
#pragma unroll
        for (int kk = 0; kk < C::SG; kk++) {
          const uint32_t a = sc + ((b * 8 + gr) * C::SLD + kk * 16 + gc) * 4;
          sv[kk][0] = lds2(a);
          sv[kk][1] = lds2(a + 32);
          mx = fmaxf(mx, fmaxf(fmaxf(sv[kk][0].x, sv[kk][0].y), fmaxf(sv[kk][1].x, sv[kk][1].y)));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[b], __fmul_rn(mx, p.c));
        const float alpha = mn == m[b] ? 1.f : ex2_approx(__fsub_rn(m[b], mn));
        const f2_t neg2 = f2_dup(mn == -INFINITY ? 0.f : -mn);  // nothing seen yet: every weight is 2^-inf = 0
        m[b] = mn;
        float sum = 0.f;
#pragma unroll
        for (int kk = 0; kk < C::SG; kk++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float u, v;
            f2_unpack(f2_fma(f2_pack(sv[kk][e].x, sv[kk][e].y), c2, neg2), u, v);
            u = ex2_approx(u);
            v = ex2_approx(v);
            sum = __fadd_rn(sum, __fadd_rn(u, v));
            pb[b][kk][e] = pack_bf16x2(u, v);
          }
        l[b] = __fmaf_rn(l[b], alpha, sum);
        if (__any_sync(0xffffffffu, alpha != 1.f)) {  // heads gc, gc + 1 of O
          const float a0 = __shfl_sync(0xffffffffu, alpha, gc * 4), a1 = __shfl_sync(0xffffffffu, alpha, gc * 4 + 4);
#pragma unroll
          for (int n = 0; n < C::MT; n++) {
            o[b][n][0] = __fmul_rn(o[b][n][0], a0);
            o[b][n][1] = __fmul_rn(o[b][n][1], a1);
            o[b][n][2] = __fmul_rn(o[b][n][2], a0);
            o[b][n][3] = __fmul_rn(o[b][n][3], a1);
          }
        }
      }
      // O transposed += V^T P^T, this warp's columns
      uint32_t dep = 0;  // (0, but known only when the last load is there)
      if (ok) {
        const int vr = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < C::SG; kk++) {
          const uint32_t vb = sb + vs * C::SLOT + row_at(kk * 16) + vr * 128;
#pragma unroll
          for (int n = 0; n < C::MT; n++) {
            const int ch = w * (C::CPW / 8) + n * 2 + ((lane >> 3) & 1);  // 16 bytes of the row
            uint32_t a[4];
            ldsm_x4_t(vb + (ch >> 3) * chunk + (((ch & 7) ^ (vr & 7)) << 4), a);
#pragma unroll
            for (int b = 0; b < NB; b++) mma16816(o[b][n], a, pb[b][kk][0], pb[b][kk][1]);
            if (kk == C::SG - 1 && n == C::MT - 1) dep = a[3] & p.zero;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(EMPTY0 + 8u * vs + dep);
    }
    if (!loaded) load_q(y);
    // the teams' parts, joined by all eight warps, eight heads at a time
#pragma unroll
    for (int b = 0; b < NB; b++) {
      l[b] = __fadd_rn(l[b], __shfl_xor_sync(0xffffffffu, l[b], 1));
      l[b] = __fadd_rn(l[b], __shfl_xor_sync(0xffffffffu, l[b], 2));
      if (met && m[b] == -INFINITY) m[b] = kNoScore;
      if (w == 0 && gc == 0) ml_s[team * C::HEADS + b * 8 + gr] = make_float2(m[b], l[b]);
    }
    const bool whole = x.k0 == 0 && x.k1 == x.nt, alone = !p.start || p.start[x.s] == 0;
#pragma unroll
    for (int b = 0; b < NB; b++) {
      float* mine = o_s + (team * 8 + gc) * C::OLD + w * C::CPW + gr;
#pragma unroll
      for (int n = 0; n < C::MT; n++) {
        mine[n * 16] = o[b][n][0];
        mine[C::OLD + n * 16] = o[b][n][1];
        mine[n * 16 + 8] = o[b][n][2];
        mine[C::OLD + n * 16 + 8] = o[b][n][3];
      }
      bar_sync(3, kConsumers);
      constexpr int V = D / 32;  // columns a thread, a warp a head
      const int head = b * 8 + warp, col = lane * V;
      if (head < heads && ok) {
        const float2 ma = ml_s[head], mb = ml_s[C::HEADS + head];
        const float mn = fmaxf(ma.x, mb.x);
        const float fa = mn == ma.x ? 1.f : ex2_approx(__fsub_rn(ma.x, mn)), fb = mn == mb.x ? 1.f : ex2_approx(__fsub_rn(mb.x, mn));
        const float lt = __fadd_rn(__fmul_rn(ma.y, fa), __fmul_rn(mb.y, fb));
        float v[V];
#pragma unroll
        for (int e = 0; e < V; e++)
          v[e] = __fadd_rn(__fmul_rn(o_s[warp * C::OLD + col + e], fa), __fmul_rn(o_s[(8 + warp) * C::OLD + col + e], fb));
        if (whole && alone) {
          const size_t at = (static_cast<size_t>(x.s) * p.Hq + x.h * p.G + x.m * C::HEADS + head) * D + col;
          const float inv = mn == -INFINITY ? 0.f : __fdiv_rn(1.f, lt);  // (no row seen: O is 0)
          uint32_t y2[V / 2];
#pragma unroll
          for (int e = 0; e < V; e++) v[e] = __fmul_rn(v[e], inv);
          if (p.gate && mn != -INFINITY) {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const uint32_t g = *reinterpret_cast<const uint32_t*>(p.gate + at + e);
              v[e] = gate_mul(v[e], bf16_lo(g));
              v[e + 1] = gate_mul(v[e + 1], bf16_hi(g));
            }
          }
#pragma unroll
          for (int e = 0; e < V / 2; e++) y2[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
          if constexpr (V == 8) *reinterpret_cast<uint4*>(p.out + at) = make_uint4(y2[0], y2[1], y2[2], y2[3]);
          else if constexpr (V == 4) *reinterpret_cast<uint2*>(p.out + at) = make_uint2(y2[0], y2[1]);
          else *reinterpret_cast<uint32_t*>(p.out + at) = y2[0];
        } else {
          float* rec = (whole ? p.rec_item + (static_cast<size_t>(x.s * p.v.Hkv + x.h) * p.MT + x.m) * C::HEADS * (D + 4)
                              : p.rec + (static_cast<size_t>(blockIdx.x) * 2 + (x.k0 == 0 ? 1 : 0)) * C::HEADS * (D + 4)) +
                       head * (D + 4);
#pragma unroll
          for (int e = 0; e < V; e += 2) *reinterpret_cast<float2*>(rec + col + e) = make_float2(v[e], v[e + 1]);
          if (lane == 0) *reinterpret_cast<float2*>(rec + D) = make_float2(mn, lt);
        }
      }
      bar_sync(3, kConsumers);  // before the buffer is written again
    }
    x = y;
    more = following;
  }
  if (!ok && lane == 0) set_status(p.v.b.status, TV_ERR_TIMEOUT);
}

// Joins pieces, in order: of items that were cut, or, where slots share prefixes, of every row with pieces (the prefix's,
// then the slot's own).  A CTA takes a row (blockIdx.x: the item's first cut, or the slot's query head), four columns a
// thread, the pieces dealt to groups of threads that cover a row each, kJ loads in flight.  For cut
// items it is small enough to wait beside the kernel before it; where slots share prefixes there are many rows with some
// dozen pieces, and more CTAs serve better than more loads each.
template <int D, bool SHARED>
__global__ void __launch_bounds__(256, SHARED ? 6 : 4) attn_paged_join_kernel(const __grid_constant__ PagedTcParams p) {
  constexpr int kJ = SHARED ? 3 : 6, LANES = D / 4, GROUPS = 256 / LANES;
  __shared__ float acc_s[GROUPS][D];
  __shared__ float2 ml_s[GROUPS];
  const int grp = threadIdx.x / LANES, col = threadIdx.x % LANES * 4;
  const uint32_t line = static_cast<uint32_t>(p.item) * (D + 4);  // (offsets in 32 bits: all pieces are under 2^32 values)
  pdl_wait();
  // (A warp that finds the word set leaves; another stream's call may set it between two warps' looks, so those that
  // stay write only where all have come to the barrier.  The decision at a barrier up here is 0.25 us of a call.)
  const bool bad = status_set(p.v.b.status);
  int s, h, head, c0, n, np = 0;  // head: of the KV head's; CTAs c0 .. hold pieces, n with the np of a prefix
  const float *own, *pre = nullptr;
  uint32_t step = 0;
  if constexpr (SHARED) {
    s = static_cast<int>(blockIdx.y);
    h = static_cast<int>(blockIdx.x) / p.G;
    head = static_cast<int>(blockIdx.x) - h * p.G;
    const int u = s * p.v.Hkv + h, m = p.MT > 1 ? head / p.item : 0;
    const int2 span = p.span[u * p.MT + m];
    const int4 g = p.info[s];
    if (bad || span.y < 0) return;  // (an idle slot's row is left as it was)
    c0 = span.x;
    const int c1 = span.y, row = g.w * p.G + head;
    np = g.z;
    if (np == 0 && c0 == c1) return;  // written whole
    n = np + c1 - c0 + 1;
    step = static_cast<uint32_t>(g.y) * 128 * (D + 4);
    if (np > 0) pre = p.rec_prefix + (static_cast<size_t>(g.x + h * np * g.y + row / 128) * 128 + row % 128) * (D + 4);
    own = (c0 == c1 ? p.rec_item + (static_cast<size_t>(u) * p.MT + m) * line : p.rec + (static_cast<size_t>(c0) * 2 + 1) * line) +
          static_cast<size_t>(head - m * p.item) * (D + 4);
  } else {
    const int4 c = p.cut[blockIdx.x];
    s = c.x;
    h = c.y;
    head = c.z * p.item + static_cast<int>(blockIdx.y);
    if (s < 0 || head >= p.G || bad) return;
    c0 = static_cast<int>(blockIdx.x) - 1;
    n = c.w - c0 + 1;
    own = p.rec + (static_cast<size_t>(c0) * 2 + 1) * line + static_cast<size_t>(blockIdx.y) * (D + 4);
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  for (int j0 = grp; j0 < n; j0 += kJ * GROUPS) {
    float4 o[kJ];
    float2 ml[kJ];
#pragma unroll
    for (int j = 0; j < kJ; j++) {
      // the prefix's pieces; the first CTA's second record; the others' first
      const int i = j0 + j * GROUPS, k = i - np;
      const float* x = SHARED && k < 0 ? pre + step * static_cast<uint32_t>(i) : own + (k == 0 ? 0u : (2u * static_cast<uint32_t>(k) - 1u) * line);
      o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      ml[j] = make_float2(-INFINITY, 0.f);
      if (i < n) {
        o[j] = *reinterpret_cast<const float4*>(x + col);
        ml[j] = *reinterpret_cast<const float2*>(x + D);
      }
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < kJ; j++) mn = fmaxf(mn, ml[j].x);
    const float a = m == -INFINITY ? 0.f : exp2f(__fsub_rn(m, mn));
    l = __fmul_rn(l, a);
    acc = make_float4(__fmul_rn(acc.x, a), __fmul_rn(acc.y, a), __fmul_rn(acc.z, a), __fmul_rn(acc.w, a));
#pragma unroll
    for (int j = 0; j < kJ; j++) {
      if (ml[j].x == -INFINITY) continue;  // no row seen in the piece (or no piece)
      const float f = exp2f(__fsub_rn(ml[j].x, mn));
      l = __fmaf_rn(f, ml[j].y, l);
      acc = make_float4(__fmaf_rn(f, o[j].x, acc.x), __fmaf_rn(f, o[j].y, acc.y), __fmaf_rn(f, o[j].z, acc.z), __fmaf_rn(f, o[j].w, acc.w));
    }
    m = mn;
  }
  *reinterpret_cast<float4*>(&acc_s[grp][col]) = acc;
  if (col == 0) ml_s[grp] = make_float2(m, l);
  if (__syncthreads_count(1) != static_cast<int>(blockDim.x)) return;
  const int t = threadIdx.x;
  if (t >= D / 2) return;  // two columns a thread
  float mn = -INFINITY, lt = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
  for (int g = 0; g < GROUPS; g++) mn = fmaxf(mn, ml_s[g].x);
#pragma unroll
  for (int g = 0; g < GROUPS; g++) {
    if (ml_s[g].x == -INFINITY) continue;
    const float f = exp2f(__fsub_rn(ml_s[g].x, mn));
    lt = __fmaf_rn(f, ml_s[g].y, lt);
    y0 = __fmaf_rn(f, acc_s[g][2 * t], y0);
    y1 = __fmaf_rn(f, acc_s[g][2 * t + 1], y1);
  }
  const size_t at = (static_cast<size_t>(s) * p.Hq + h * p.G + head) * D + 2 * t;
  const float inv = __fdiv_rn(1.f, lt);
  y0 = __fmul_rn(y0, inv);
  y1 = __fmul_rn(y1, inv);
  if (mn == -INFINITY) {
    y0 = y1 = 0.f;  // no row seen
  } else if (p.gate) {
    const uint32_t g = *reinterpret_cast<const uint32_t*>(p.gate + at);
    y0 = gate_mul(y0, bf16_lo(g));
    y1 = gate_mul(y1, bf16_hi(g));
  }
  *reinterpret_cast<uint32_t*>(p.out + at) = pack_bf16x2(y0, y1);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// A pool as a tensor of rows cut into blocks of 64 columns, in boxes of `rows` rows and `cols` blocks.
static bool encode_pool_map(CUtensorMap* m, void* base, int D, int64_t all, int rows, int cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t d = static_cast<cuuint64_t>(D), dims[3] = {64, static_cast<cuuint64_t>(all), d / 64}, strides[2] = {d * 2, 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(cols)}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query heads of an item: eight, a tile's columns, or sixteen, two tiles that share the
// reads of keys and values, for groups of more.
static int item_heads(const tv_paged_layer* l) { return l->Hq / l->Hkv <= 8 ? 8 : kItemMax; }

// A call's scratch, in bytes from its start.
struct PagedSpace {
  size_t cut, rec, span, rec_item, rec_prefix, info, start, all;
};
static PagedSpace space_of(const tv_paged_layer* l, const tv_paged* b, const tv_paged_groups* g) {
  const size_t line = static_cast<size_t>(l->D + 4) * 4, units = static_cast<size_t>(b->n_seq) * l->Hkv;
  const int item = item_heads(l);
  const size_t items = units * ((l->Hq / l->Hkv + item - 1) / item);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t x = at;
    at += (n + 15) / 16 * 16;
    return x;
  };
  PagedSpace s{};
  s.cut = take(static_cast<size_t>(num_sms()) * 16);
  s.rec = take(static_cast<size_t>(2) * num_sms() * item * line);
  if (g) {
    s.span = take(items * 8);
    s.rec_item = take(items * item * line);
    s.rec_prefix = take(static_cast<size_t>(paged_prefix_slots(l, b, g->n_group)) * 128 * line);
    s.info = take(static_cast<size_t>(b->n_seq) * 16);
    s.start = take(static_cast<size_t>(b->n_seq) * 4);
  }
  s.all = at;
  return s;
}
size_t paged_attn_ws_bytes(const tv_paged_layer* l, const tv_paged* b, const tv_paged_groups* g) { return space_of(l, b, g).all; }

template <int D, int NB>
static tv_status launch_tc(PagedTcParams& p, const PagedAttnCall& a, cudaStream_t st) {
  using C = Pg<D, NB>;
  const tv_paged_layer* l = a.layer;
  p.R = l->page < C::ROWS ? l->page : C::ROWS;
  const int64_t all = static_cast<int64_t>(l->n_pages) * l->Hkv * l->page;
  if (!encode_pool_map(&p.tmK, l->K, D, all, p.R, D / 64) || !encode_pool_map(&p.tmV, l->V, D, all, p.R, D / 64)) return TV_ERR_CUDA;
  static std::atomic<uint64_t> set{0};
  if (!allow_smem(attn_paged_tc_kernel<D, NB>, C::SMEM, set)) return TV_ERR_CUDA;
  const int grid = num_sms();
  const bool may_share = p.start != nullptr;
  // Where no item can have more than four tiles, each is one CTA's, and the call saves the join, which takes longer than the
  // tiles that others would have taken: 24 + 4 heads of 256 or 32 + 4 of 128, 2 slots of up to 98 rows 7.6 us and 9.3
  // with ranges cut evenly, 30 of up to 250 9.4 and 11.8, 3 of up to 216 9.4 and 10.2 (seven tiles would lose).
  const int64_t most = a.sel ? std::min<int64_t>(static_cast<int64_t>(a.n_sel) * l->page, a.batch->max_len + 1) : a.batch->max_len + 1;
  p.uncut = !may_share && most <= 4 * C::ROWS ? 1 : 0;
  launch_k(true, attn_paged_tc_kernel<D, NB>, dim3(grid), dim3(kThreads), C::SMEM, st, p);
  if (may_share) {
    PagedPrefixParams x;
    memset(&x, 0, sizeof(x));
    int k_cols, v_cols;
    paged_prefix_boxes(D, l->page, x, k_cols, v_cols);
    if (!encode_pool_map(&x.tmK, l->K, D, all, x.RK, k_cols) || !encode_pool_map(&x.tmV, l->V, D, all, x.RV, v_cols)) return TV_ERR_CUDA;
    x.b = p.v.b;
    x.group_off = a.groups->group_off;
    x.shared = a.groups->shared;
    x.q = p.q;
    x.rec = const_cast<float*>(p.rec_prefix);
    x.info = const_cast<int4*>(p.info);
    x.n_group = a.groups->n_group;
    x.slots = paged_prefix_slots(l, a.batch, x.n_group);
    x.Hq = p.Hq;
    x.Hkv = l->Hkv;
    x.G = p.G;
    x.all_rows = static_cast<int>(all);
    x.c = p.c;
    if (!paged_prefix_launch(x, D, st)) return TV_ERR_CUDA;
  }
  if (p.uncut) return launch_status();
  if (may_share) launch_k(true, attn_paged_join_kernel<D, true>, dim3(l->Hq, a.batch->n_seq), dim3(256), 0, st, p);
  else launch_k(true, attn_paged_join_kernel<D, false>, dim3(grid, p.G < p.item ? p.G : p.item), dim3(256), 0, st, p);
  return launch_status();
}

tv_status paged_attn_tc_launch(const PagedAttnCall& a, cudaStream_t st) {
  const tv_paged_layer* l = a.layer;
  PagedTcParams p;
  memset(&p, 0, sizeof(p));
  p.v = PagedView{paged_seqs(l, a.batch), a.sel, a.count, a.n_sel, l->Hkv};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.gate = static_cast<const __nv_bfloat16*>(a.gate);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  char* ws = static_cast<char*>(a.ws);
  const PagedSpace x = space_of(l, a.batch, a.groups);
  p.cut = reinterpret_cast<int4*>(ws + x.cut);
  p.rec = reinterpret_cast<float*>(ws + x.rec);
  if (a.groups) {
    p.group_off = a.groups->group_off;
    p.shared = a.groups->shared;
    p.n_group = a.groups->n_group;
  }
  // (where no lengths within the bound could save enough, the groups are only checked)
  if (a.groups && (a.batch->n_seq - 1) * static_cast<int64_t>(a.batch->max_len) * kv_row_bytes(l->Hkv, l->D) >= kSharedBytes) {
    p.span = reinterpret_cast<int2*>(ws + x.span);
    p.rec_item = reinterpret_cast<float*>(ws + x.rec_item);
    p.rec_prefix = reinterpret_cast<const float*>(ws + x.rec_prefix);
    p.info = reinterpret_cast<const int4*>(ws + x.info);
    p.start = reinterpret_cast<int32_t*>(ws + x.start);
  }
  p.Hq = l->Hq;
  p.G = l->Hq / l->Hkv;
  p.item = item_heads(l);
  p.MT = (p.G + p.item - 1) / p.item;
  p.units = a.batch->n_seq * l->Hkv;
  p.c = a.scale * 1.4426950408889634f;
  switch (l->D) {
    case 64: return p.item == 8 ? launch_tc<64, 1>(p, a, st) : launch_tc<64, 2>(p, a, st);
    case 128: return p.item == 8 ? launch_tc<128, 1>(p, a, st) : launch_tc<128, 2>(p, a, st);
    default: return p.item == 8 ? launch_tc<256, 1>(p, a, st) : launch_tc<256, 2>(p, a, st);
  }
}

}  // namespace tv
