// The prefixes that groups of slots share, for bf16 caches in pages, on the
// tcgen05 tensor cores.
//
// All members of a group see all rows of its prefix, so the group's query rows of
// a KV head (members x G query heads) meet the prefix's keys as one product: an
// item is 128 of these rows against the keys, cut into pieces of S key tiles of
// 128 rows.  A piece runs flash style
//   S = Q K^T (tensor core, fp32), m = running maximum of scaled scores,
//   p = 2^(s c - m), l += sum of p (fp32), p rounded to bf16,
//   O = O 2^(m_old - m) + P V (tensor core, fp32)
// and leaves O, m and l in fp32, which the join of the call adds to what each slot
// sees by itself.  The maximum moves only when a tile exceeds it by more than 8 in
// log2 units (p then stays below 2^8), so O is rescaled rarely.  p is rounded
// because the tensor cores take P and V in one type (by 2^-8 of itself at most; l
// adds them as they were).
//
// Roles (384 threads, one CTA per SM, persistent).  Warp 11 looks up pages, a thread of
// warp 0 streams key and value units by TMA through one ring in the order the tensor
// core takes them: K0, K1 V0, K2 V1, ...  Warp 1 issues Q K^T, warp 10 P V.  Warps 2-9 do the softmax, two threads to a row (64 scores each).
// Tensor memory holds O [D columns], S [128] and Q [D/2, the A operand of Q K^T];
// P goes through shared memory.  PV of tile t-1 sits between Q K^T of t and of t+1
// on the tensor pipe: S(t) is read out during it, and one S buffer is enough.
//
// It follows the kernel for what each slot sees by itself and starts on SMs as that one
// leaves them.
//
// Work split.  Every CTA derives the same plan from the device-side groups and
// lengths: S with the fewest tiles for the busiest CTA; pieces of the same keys lie
// next to each other in the order of all, so CTAs that run at the same time read
// them from L2.  Rows of the last tile behind the prefix are filled with zeros by
// TMA (a box behind the pools' end) and masked.
//
// Bound by the tensor cores: in the steady state a tile takes 1.1 times its products' time in pages
// of 128 rows, 1.2 in pages of 64; smaller pages are bound by the copies one thread issues (64 members on 32,768 rows,
// 24 + 4 heads of 256: 68.6, 71.6, 93.5 and 126 us in pages of 128, 64, 32 and 16).  64 + 6 slots on prefixes of 32,768
// and 8,192 rows 80 us in all (817 slot by slot): 32 of products here, some 8 until the first ones, 3.5 for what pieces leave, 9 of join,
// and 15 to 20 of the kernel before, for what each slot sees by itself.
#include "attn_paged.cuh"
#include "attn_paged_prefix.cuh"
#include "ptx.cuh"

namespace tv {

namespace {

constexpr int kKeyTile = 128;
constexpr float kMoveMax = 8.f;
constexpr int kPrefixThreads = 384;
constexpr int kIds = 128;  // parts that are looked up at once (a multiple of a tile's)

template <int D>
struct Px {
  static constexpr int UPT = D == 256 ? 2 : 1;              // ring units per key (or value) tile
  static constexpr int UNIT = kKeyTile * D * 2 / UPT;       // bytes of a unit
  static constexpr int NU = D == 64 ? 8 : D == 128 ? 4 : 5;
  static constexpr int KBOX = kKeyTile * 128;               // bytes of 128 rows, 64 columns of keys
  static constexpr int KBU = D / 64 / UPT;                  // column boxes of a key unit
  static constexpr int VROWS = kKeyTile / UPT;              // rows of a value unit
  static constexpr int VBOX = VROWS * 128;
  static constexpr int VB = D / 64;                         // column boxes of a value unit
  static constexpr int PT = 128 * kKeyTile * 2;
  static constexpr int QH = D == 64 ? 1 : 2, QR = D == 256 ? 2 : 1;  // halves that move Q, 64 columns at a time
  static constexpr int T_O = 0, T_S = D, T_Q = D + 128, COLS = 512;
  static_assert(T_Q + D / 2 <= COLS, "tensor memory");
  static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, kKeyTile, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true);
  static constexpr int POFF = NU * UNIT;
  static constexpr int XOFF = POFF + PT;                    // exchanged values [2][2][128]
  static constexpr int GOFF = XOFF + 2 * 2 * 128 * 4;       // groups: first slot, pieces before, key tiles, table row
  static constexpr int IOFF = GOFF + 4 * (TV_MAX_PAGED_SEQ + 4) * 4;  // rows of the parts [2][kIds]
  static constexpr int BOFF = IOFF + 2 * kIds * 4;
  static constexpr int NBAR = 2 * NU + 5 + 4 + 2 + 4;
  static constexpr int LOFF = (BOFF + NBAR * 8 + 15) / 16 * 16;
  static constexpr int SMEM = LOFF + 64;
  static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
__device__ __forceinline__ uint4 ldg16(const void* p) { return *static_cast<const uint4*>(p); }
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// The groups of a call, in shared memory.
struct Groups {
  int *off, *cum, *nk, *src;  // first slot [n + 1], pieces before [n + 1], key tiles, slot whose table is read
};
struct PrefixItem {
  int g, h, r, k0, k1, n;  // group, KV head, row tile, key tiles [k0, k1), member rows of the tile's group
};
__device__ __forceinline__ PrefixItem prefix_item(const PagedPrefixParams& p, const Groups& G, int S, int x) {
  int lo = 0, hi = p.n_group;  // the last group that starts at or before x and has pieces
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (G.cum[mid] <= x) lo = mid;
    else hi = mid;
  }
  PrefixItem I;
  I.g = lo;
  I.n = (G.off[lo + 1] - G.off[lo]) * p.G;
  const int R = ceil_div(I.n, 128), np = ceil_div(G.nk[lo], S), y = x - G.cum[lo];
  I.r = y % R;
  const int j = y / R % np;
  I.h = y / R / np;
  I.k0 = j * S;
  I.k1 = min(I.k0 + S, G.nk[lo]);
  return I;
}

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1) attn_paged_prefix_kernel(const __grid_constant__ PagedPrefixParams p) {
  using C = Px<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // tiles are swizzled in 1024-byte atoms
  const uint32_t sb = smem_u32(smem_raw), ring = sb, pbuf = sb + C::POFF;
  float* xmax = reinterpret_cast<float*>(smem_raw + C::XOFF);
  const uint32_t UFULL0 = sb + C::BOFF, UEMPTY0 = UFULL0 + 8u * C::NU, SFULL = UEMPTY0 + 8u * C::NU, SFREE = SFULL + 8u,
                 PFULL = SFULL + 16u, ODONE = SFULL + 24u, QREADY = SFULL + 32u, XBAR0 = SFULL + 40u, DRAIN = XBAR0 + 32u, IDFULL0 = DRAIN + 16u, IDEMPTY0 = IDFULL0 + 16u;
  volatile int* ids = reinterpret_cast<volatile int*>(smem_raw + C::IOFF);
  struct Local {
    uint32_t tmem;
    int abort_flag, most;
    unsigned long long best;
  };
  Local& lo = *reinterpret_cast<Local*>(smem_raw + C::LOFF);
  static_assert(sizeof(Local) <= 64, "local data");
  volatile int* abort_flag = &lo.abort_flag;
  Groups gr;
  gr.off = reinterpret_cast<int*>(smem_raw + C::GOFF);
  gr.cum = gr.off + TV_MAX_PAGED_SEQ + 4;
  gr.nk = gr.cum + TV_MAX_PAGED_SEQ + 4;
  gr.src = gr.nk + TV_MAX_PAGED_SEQ + 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < C::NU; i++) {
      mbar_init(UFULL0 + 8u * i, 1);
      mbar_init(UEMPTY0 + 8u * i, 1);
    }
    mbar_init(SFULL, 1);
    mbar_init(SFREE, 8);
    mbar_init(PFULL, 8);
    mbar_init(ODONE, 1);
    mbar_init(QREADY, 8);
    for (int i = 0; i < 4; i++) mbar_init(XBAR0 + 8u * i, 2);
    mbar_init(DRAIN, 1);
    mbar_init(DRAIN + 8u, 1);
    for (int i = 0; i < 4; i++) mbar_init(IDFULL0 + 8u * i, 1);
    lo.abort_flag = 0;
    lo.best = ~0ull;
    lo.most = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&lo.tmem), C::COLS);
    tmem_relinquish();
  }
  // (The kernel before on the stream is the call's own, for what each slot sees by itself; it has waited before it let
  // this one in, and writes nothing that is read here, nor the other way round.)
  pdl_trigger();
  const int NG = p.n_group;
  int* count = reinterpret_cast<int*>(smem_raw);  // (the ring is not in use yet)
  GroupCheck<kPrefixThreads> check{gr.off, count, count + TV_MAX_PAGED_SEQ, gr.src, gr.nk,
                                   reinterpret_cast<unsigned long long*>(count + 2 * TV_MAX_PAGED_SEQ)};
  int code = sb & 1023u ? TV_ERR_CUDA : 0;
  code = check.run(p.b, p.group_off, p.shared, NG, kv_row_bytes(p.Hkv, D), code);
  if (code || __syncthreads_or(status_set(p.b.status))) {
    if (code) set_status(p.b.status, code);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(lo.tmem, C::COLS);
    pdl_wait();
    return;
  }
  // (nk holds the shared rows so far)
  int most = 0;
  for (int g = tid; g < NG; g += kPrefixThreads) most = max(most, gr.nk[g] = ceil_div(gr.nk[g], kKeyTile));
  if (most > 0) atomicMax(&lo.most, most);
  __syncthreads();
  most = lo.most;  // key tiles of the longest prefix
  // S: candidates by the pieces that the longest prefix is cut into, a thread each; the cost is the tiles of
  // the CTA with most pieces, and about four for each to start, to end and to be joined
  if (most > 0) {
    const int S = max(ceil_div(most, tid + 1), 2);
    float pieces = 0.f;  // (whole numbers, exact where they count: the workspace holds fewer than 2^24)
    for (int g = 0; g < NG; g++)
      if (gr.nk[g] > 0) pieces += static_cast<float>(p.Hkv * ceil_div((gr.off[g + 1] - gr.off[g]) * p.G, 128)) * static_cast<float>(ceil_div(gr.nk[g], S));
    const float cost = ceilf(__fdividef(pieces, static_cast<float>(gridDim.x))) * static_cast<float>(min(S, most) + 4);
    if (pieces <= static_cast<float>(p.slots) || tid == 0) atomicMin(&lo.best, static_cast<unsigned long long>(__float_as_uint(cost)) << 10 | tid);
  }
  __syncthreads();
  const int S = most > 0 ? max(ceil_div(most, static_cast<int>(lo.best & 1023u) + 1), 2) : 2;
  if (warp == 0) {  // pieces before each group
    int before = 0;
    for (int g0 = 0; g0 < NG; g0 += 32) {
      const int g = g0 + lane;
      const int n = g < NG && gr.nk[g] > 0 ? p.Hkv * ceil_div((gr.off[g + 1] - gr.off[g]) * p.G, 128) * ceil_div(gr.nk[g], S) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (g < NG) gr.cum[g] = before + incl - n;
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) gr.cum[NG] = before;
  }
  fence_proxy_async_smem();  // (the ring has held the groups' counts)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (blockIdx.x == 0) {  // for the join
    for (int g = tid; g < NG; g += kPrefixThreads)
      for (int s = gr.off[g]; s < gr.off[g + 1]; s++)
        p.info[s] = make_int4(gr.cum[g], ceil_div((gr.off[g + 1] - gr.off[g]) * p.G, 128), ceil_div(gr.nk[g], S), s - gr.off[g]);
  }
  const uint32_t tbase = lo.tmem;
  const int total = gr.cum[NG];
  auto arrive = [&](uint32_t bar) {  // one arrival per warp, after every lane's fences
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  const int parts = kKeyTile / p.R;  // boxes' worth of rows in a tile
  if (warp == 11) {
    // ---------------- page lookups: where the prefix's rows lie, kIds parts at a time ----------------
    const int rows = 1 << p.b.shift, per_page = rows / p.R;
    uint32_t c = 0;  // chunks
    bool ok = true;
    for (int x = blockIdx.x; ok && x < total; x += gridDim.x) {
      const PrefixItem I = prefix_item(p, gr, S, x);
      const int s = gr.src[I.g], end = min(p.shared[I.g] / p.R, I.k1 * parts);
      for (int i0 = I.k0 * parts; ok && i0 < I.k1 * parts; i0 += kIds, c++) {
        ok = wait_warp(IDEMPTY0 + 8u * (c & 1), ((c >> 1) & 1) ^ 1, abort_flag, kWaitCycles);
        if (!ok) break;
#pragma unroll
        for (int j = lane; j < kIds; j += 32) {
          // behind the prefix, and for entries that name no page, a row behind the pools (zeros)
          const int i = i0 + j, page = i < end ? page_at(p.b, s, i / per_page) : -1;
          ids[(c & 1) * kIds + j] = page < 0 ? p.all_rows : (page * p.Hkv + I.h) * rows + (i % per_page) * p.R;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(IDFULL0 + 8u * (c & 1));
      }
    }
    if (!ok && lane == 0) set_status(p.b.status, TV_ERR_TIMEOUT);
  } else if (warp == 0 && lane == 0) {
    // ---------------- TMA producer, one thread (with a warp's votes and shuffles a unit took 760 cycles,
    // and a tile 3,800) ----------------
    const bool kwhole = p.RK == kKeyTile, vwhole = p.RV == C::VROWS;  // a unit is one box, else a box a part and 64 columns
    uint32_t it = 0, chunks = 0;  // units; chunks of the items before
    bool ok = true;
    for (int x = blockIdx.x; ok && x < total; x += gridDim.x) {
      const PrefixItem I = prefix_item(p, gr, S, x);
      const int n = I.k1 - I.k0;
      for (int e = 0; e < 2 * n && ok; e++) {
        // load order K0, K1 V0, K2 V1, ..., V(n-1)
        const bool is_k = e == 0 || ((e & 1) && e != 2 * n - 1);
        const int k = e == 0 ? 0 : is_k ? (e + 1) / 2 : (e == 2 * n - 1 ? n - 1 : (e - 2) / 2);
        const uint32_t c = chunks + static_cast<uint32_t>(k * parts / kIds);
        if (is_k && k * parts % kIds == 0) ok = wait_role(IDFULL0 + 8u * (c & 1), (c >> 1) & 1, abort_flag, kWaitCycles);
        const volatile int* id = ids + (c & 1) * kIds + k * parts % kIds;
#pragma unroll
        for (int u = 0; u < C::UPT; u++, it++) {
          const uint32_t slot = it % C::NU, full = UFULL0 + 8u * slot, dst = ring + slot * C::UNIT;
          ok = ok && wait_role(UEMPTY0 + 8u * slot, ((it / C::NU) & 1) ^ 1, abort_flag, kWaitCycles);
          if (!ok) break;
          mbar_arrive_expect_tx(full, C::UNIT);
          if (is_k) {
            if (kwhole) {
              tma_load_3d(dst, &p.tmK, full, 0, id[0], u * C::KBU);
            } else {
#pragma unroll 2
              for (int pt = 0; pt < parts; pt++) {
                const int from = id[pt];
#pragma unroll
                for (int ch = 0; ch < C::KBU; ch++)
                  tma_load_3d(dst + ch * C::KBOX + pt * p.R * 128, &p.tmK, full, 0, from, u * C::KBU + ch);
              }
            }
          } else {
            const int up = parts / C::UPT;
            if (vwhole) {
              tma_load_3d(dst, &p.tmV, full, 0, id[u * up], 0);
            } else {
#pragma unroll 2
              for (int pt = 0; pt < up; pt++) {
                const int from = id[u * up + pt];
#pragma unroll
                for (int ch = 0; ch < C::VB; ch++) tma_load_3d(dst + ch * C::VBOX + pt * p.R * 128, &p.tmV, full, 0, from, ch);
              }
            }
          }
        }
        if (!is_k && ((k + 1) * parts % kIds == 0 || k + 1 == n)) mbar_arrive(IDEMPTY0 + 8u * (c & 1));  // the chunk's last use
      }
      chunks += static_cast<uint32_t>((n * parts + kIds - 1) / kIds);
    }
    if (!ok) set_status(p.b.status, TV_ERR_TIMEOUT);
    // every issued copy lands before shared memory is released
    for (uint32_t i = it > C::NU ? it - C::NU : 0; i < it; i++) mbar_wait(UFULL0 + 8u * (i % C::NU), (i / C::NU) & 1, kWaitCycles);
  } else if (warp == 1 || warp == 10) {
    // ---------------- products: one warp each, whole-warp loops with one elected lane issuing ----------------
    const bool is_qk = warp == 1;
    uint32_t base = 0, t = 0, items = 0;  // units and tiles before the item, items
    bool ok = true;
    for (int x = blockIdx.x; ok && x < total; x += gridDim.x, items++) {
      const PrefixItem I = prefix_item(p, gr, S, x);
      const int n = I.k1 - I.k0;
      if (is_qk) ok = wait_warp(QREADY, items & 1, abort_flag, kWaitCycles);
      for (int k = 0; k < n && ok; k++, t++) {
        const uint32_t u0 = base + (is_qk ? (k == 0 ? 0 : 2 * k - 1) : (k < n - 1 ? 2 * k + 2 : 2 * n - 1)) * C::UPT;
        if (is_qk) {
          if (t > 0) ok = wait_warp(SFREE, (t - 1) & 1, abort_flag, kWaitCycles);
        } else {
          ok = wait_warp(PFULL, t & 1, abort_flag, kWaitCycles);
        }
#pragma unroll
        for (int u = 0; u < C::UPT; u++) {
          const uint32_t slot = (u0 + u) % C::NU;
          ok = ok && wait_warp(UFULL0 + 8u * slot, ((u0 + u) / C::NU) & 1, abort_flag, kWaitCycles);
          if (!ok) break;
          tc_fence_after();
          if (elect_one_sync()) {
            if (is_qk) {
              const uint64_t k0 = sdesc_sw128(ring + slot * C::UNIT, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < C::KBU * 4; kk++)
                tc_mma_ts(tbase + C::T_S, tbase + C::T_Q + (u * C::KBU * 4 + kk) * 8,
                          k0 + static_cast<uint64_t>(((kk >> 2) * C::KBOX + (kk & 3) * 32) >> 4), C::IDESC_QK,
                          (u > 0 || kk > 0) ? 1u : 0u);
            } else {
              const uint64_t v0 = sdesc_sw128(ring + slot * C::UNIT, C::VBOX, 1024), p0 = sdesc_sw128(pbuf, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < C::VROWS / 16; kk++) {
                const int pk = u * (C::VROWS / 16) + kk;  // 16-row step of the tile
                tc_mma_ss(tbase + C::T_O, p0 + static_cast<uint64_t>(((pk >> 2) * 16384 + (pk & 3) * 32) >> 4),
                          v0 + static_cast<uint64_t>((kk * 2048) >> 4), C::IDESC_PV, (k > 0 || pk > 0) ? 1u : 0u);
              }
            }
            tc_commit(UEMPTY0 + 8u * slot);
            if (u == C::UPT - 1) tc_commit(is_qk ? SFULL : ODONE);
          }
          __syncwarp();
        }
      }
      base += 2 * n * C::UPT;
    }
    if (!ok && lane == 0) set_status(p.b.status, TV_ERR_TIMEOUT);
    // every product of this warp completes before tensor and shared memory are released
    const uint32_t drain = DRAIN + (is_qk ? 0u : 8u);
    if (elect_one_sync()) tc_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, kWaitCycles);
  } else if (warp >= 2 && warp < 10) {
    // ---------------- softmax, a row's scores (and columns of O) to two threads ----------------
    const int hf = (warp - 2) >> 2, quad = warp & 3, lrow = quad * 32 + lane;
    const uint32_t tl = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t line = pbuf + hf * 16384 + (lrow >> 3) * 1024 + (lrow & 7) * 128;
    const uint32_t patch = pbuf + hf * 16384 + quad * 4096;  // 4 KB of its own between items
    uint32_t t = 0, xc = 0;  // tiles, exchanges
    bool ok = true;
    // the two threads of a row exchange a value
    auto exchange = [&](float v, float& other) {
      float* x = xmax + (xc & 1) * 256;
      x[hf * 128 + lrow] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(XBAR0 + 8u * quad);
      if (!wait_warp(XBAR0 + 8u * quad, xc & 1, abort_flag, kWaitCycles)) return false;
      other = x[(hf ^ 1) * 128 + lrow];
      xc++;
      return true;
    };
    // Q of an item into tensor memory, a warp its rows' half, 64 columns at a time turned around in its patch (free: every
    // P V of the item before has completed)
    auto load_q = [&](const PrefixItem& I) {
      if (hf < C::QH) {
        const int cl = lane & 7;  // 16 bytes of a row's 128
        uint4 v[C::QR][8];
        const __nv_bfloat16* q0 = p.q + (static_cast<size_t>(gr.off[I.g]) * p.Hq + I.h * p.G) * D + hf * (D / 2) + cl * 8;
        int row = I.r * 128 + quad * 32 + (lane >> 3), m = row / p.G, head = row - m * p.G;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const __nv_bfloat16* q = q0 + (row < I.n ? (static_cast<size_t>(m) * p.Hq + head) * D : 0);
#pragma unroll
          for (int r = 0; r < C::QR; r++) v[r][i] = ldg16(q + r * 64);
          row += 4;
          for (head += 4; head >= p.G; head -= p.G) m++;
        }
#pragma unroll
        for (int r = 0; r < C::QR; r++) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const int rr = i * 4 + (lane >> 3);
            sts16(patch + rr * 128 + (((cl ^ rr) & 7) << 4), v[r][i].x, v[r][i].y, v[r][i].z, v[r][i].w);
          }
          __syncwarp();
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const uint4 x = lds16(patch + lane * 128 + (((i ^ lane) & 7) << 4));
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
          }
          tmem_st32(tl + C::T_Q + (hf * C::QR + r) * 32, w);
        }
        tmem_st_wait();
        __syncwarp();
      }
      tc_fence_before();
      arrive(QREADY);
    };
    PrefixItem I;
    int x = blockIdx.x;
    if (x < total) {
      I = prefix_item(p, gr, S, x);
      load_q(I);
    }
    for (; ok && x < total; x += gridDim.x) {
      const int n = I.k1 - I.k0, end = p.shared[I.g];
      const bool act = I.r * 128 + lrow < I.n;
      float m = -INFINITY, l = 0.f, other = 0.f;
      for (int k = 0; k < n; k++, t++) {
        if (!wait_warp(SFULL, t & 1, abort_flag, kWaitCycles)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sv[64];
        {
          uint32_t r[32];
          tmem_ld32(tl + C::T_S + hf * 64, r);
#pragma unroll
          for (int i = 0; i < 32; i++) sv[i] = __uint_as_float(r[i]);
          tmem_ld32(tl + C::T_S + hf * 64 + 32, r);
#pragma unroll
          for (int i = 0; i < 32; i++) sv[32 + i] = __uint_as_float(r[i]);
        }
        tc_fence_before();
        arrive(SFREE);
        const int left = end - (I.k0 + k) * kKeyTile - hf * 64;  // of this half's rows, those in the prefix
        if (left < 64) {
#pragma unroll
          for (int j = 0; j < 64; j++) sv[j] = j < left ? sv[j] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 64; j += 2) mx[(j / 2) & 3] = fmaxf(mx[(j / 2) & 3], fmaxf(sv[j], sv[j + 1]));
        const float mh = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (!exchange(mh, other)) {
          ok = false;
          break;
        }
        const float mt = __fmul_rn(fmaxf(mh, other), p.c);
        float alpha = 1.f;
        if (mt > __fadd_rn(m, kMoveMax) || (m == -INFINITY && mt > -INFINITY)) {
          alpha = ex2_approx(__fsub_rn(m, mt));  // 0 from m = -inf
          m = mt;
        }
        const float neg = m == -INFINITY ? 0.f : -m;  // no score above -inf yet: every p below is 2^-inf = 0
        uint32_t P[32];
        f2_t acc[2] = {0ull, 0ull};
        const f2_t c2 = f2_dup(p.c), neg2 = f2_dup(neg);
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
          float a, b;
          f2_unpack(f2_fma(f2_pack(sv[j], sv[j + 1]), c2, neg2), a, b);
          a = ex2_approx(a);
          b = ex2_approx(b);
          acc[(j / 2) & 1] = f2_add(acc[(j / 2) & 1], f2_pack(a, b));
          P[j / 2] = pack_bf16x2(a, b);
        }
        l = __fmaf_rn(l, alpha, f2_hsum(f2_add(acc[0], acc[1])));
        // PV of the tile before is complete: P is free and O rests
        if (t > 0 && !wait_warp(ODONE, (t - 1) & 1, abort_flag, kWaitCycles)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 8; q++) sts16(line + (((q ^ lrow) & 7) << 4), P[4 * q], P[4 * q + 1], P[4 * q + 2], P[4 * q + 3]);
        if (k > 0 && __any_sync(0xffffffffu, act && alpha != 1.f)) {
#pragma unroll 1
          for (int c = hf * (D / 2); c < (hf + 1) * (D / 2); c += 32) {
            uint32_t r[32];
            tmem_ld32(tl + C::T_O + c, r);
#pragma unroll
            for (int i = 0; i < 32; i++) r[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[i]), alpha));
            tmem_st32(tl + C::T_O + c, r);
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(PFULL);
      }
      if (!ok) break;
      if (!exchange(l, other) || !wait_warp(ODONE, (t - 1) & 1, abort_flag, kWaitCycles)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // O, m and l as they are; rows leave through this warp's patch, turned around so that an instruction
      // covers whole pieces of rows
      float* rec = p.rec + (static_cast<size_t>(x) * 128 + lrow) * (D + 4);
#pragma unroll 1
      for (int c = hf * (D / 2); c < (hf + 1) * (D / 2); c += 32) {
        uint32_t r[32];
        tmem_ld32(tl + C::T_O + c, r);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; i++) sts16(patch + lane * 128 + (((i ^ lane) & 7) << 4), r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const int rr = i * 4 + (lane >> 3);
          const uint4 v = lds16(patch + rr * 128 + ((((lane & 7) ^ rr) & 7) << 4));
          if (I.r * 128 + quad * 32 + rr < I.n) *reinterpret_cast<uint4*>(rec + (rr - lane) * (D + 4) + c + (lane & 7) * 4) = v;
        }
      }
      if (act && hf == 0) {
        // (every row sees every key: where no score is above -inf, 0 / 0 is to come)
        rec[D] = m == -INFINITY ? kNoScore : m;
        rec[D + 1] = __fadd_rn(l, other);
      }
      __syncwarp();
      if (x + static_cast<int>(gridDim.x) < total) {
        I = prefix_item(p, gr, S, x + gridDim.x);
        load_q(I);
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) set_status(p.b.status, TV_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, C::COLS);
  pdl_wait();  // the join, which waits for this kernel, needs both
}

template <int D>
bool launch(const PagedPrefixParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  if (!allow_smem(attn_paged_prefix_kernel<D>, Px<D>::SMEM, set)) return false;
  launch_k(true, attn_paged_prefix_kernel<D>, dim3(num_sms()), dim3(kPrefixThreads), Px<D>::SMEM, st, p);
  return true;
}

}  // namespace

template <int D>
static void boxes(int page, PagedPrefixParams& p, int& k_cols, int& v_cols) {
  using C = Px<D>;
  p.R = page < 64 ? page : 64;
  p.RK = page < kKeyTile ? p.R : kKeyTile;
  p.RV = page < C::VROWS ? p.R : C::VROWS;
  k_cols = p.RK == kKeyTile ? C::KBU : 1;
  v_cols = p.RV == C::VROWS ? C::VB : 1;
}
void paged_prefix_boxes(int D, int page, PagedPrefixParams& p, int& k_cols, int& v_cols) {
  if (D == 64) boxes<64>(page, p, k_cols, v_cols);
  else if (D == 128) boxes<128>(page, p, k_cols, v_cols);
  else boxes<256>(page, p, k_cols, v_cols);
}

int paged_prefix_slots(const tv_paged_layer* l, const tv_paged* b, int n_group) {
  const int64_t G = l->Hq / l->Hkv, items = l->Hkv * ((b->n_seq * G + 127) / 128 + n_group);
  return static_cast<int>(items + 2 * num_sms());
}

bool paged_prefix_launch(const PagedPrefixParams& p, int D, cudaStream_t st) {
  return D == 64 ? launch<64>(p, st) : D == 128 ? launch<128>(p, st) : launch<256>(p, st);
}

}  // namespace tv
