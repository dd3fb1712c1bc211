// Causal grouped-query attention over a prompt's packed rows for bf16 caches,
// on the tcgen05 tensor cores.
//
// Row i of a sequence sees cache rows 0 .. len + i.  The rows of one KV head
// are taken token major, the G query heads that share it side by side, so a
// row tile of 128 holds T = 128 / G tokens (rows past T * G idle) and every
// key and value tile serves all of them.  An item is one row tile of one KV
// head against its keys; it runs flash style over key tiles of 128 positions:
//   S = Q K^T (tensor core, fp32), m = running maximum of scaled scores,
//   p = 2^(s c - m), l += sum of p (fp32), p rounded to bf16,
//   O = O 2^(m_old - m) + P V (tensor core, fp32), out = O / l (times the gate).
// The maximum moves only when a tile exceeds it by more than 8 in log2 units
// (p then stays below 2^8), so O is rescaled rarely.  p is rounded to bf16
// because the tensor cores take P and V in one type; each weight is off by 2^-9
// at most, independently, and l adds them as they were (adding the rounded ones
// takes a quarter of the softmax's instructions more and is no nearer: 2.3e-3
// from the result in 64 bits either way, of which 1.7e-3 is the output's rounding).
//
// Roles (384 threads, one CTA per SM, persistent).  Warp 0 streams key and
// value units by TMA through one ring in the order the tensor core takes
// them: K0, K1 V0, K2 V1, ...  Warp 11 brings each item's queries, warp 1
// issues Q K^T, warp 10 P V, each from one thread.  Warps 2-9 do the softmax.
// D = 256: two threads to a row (64 columns each).  Tensor memory holds O [D
// columns], one S [128] and Q [D/2, the A operand of Q K^T], 512 columns; P goes
// through shared memory.  Because PV of tile t-1 sits between Q K^T of t and of
// t+1 on the tensor pipe, S(t) is read out during that PV and one S buffer is
// enough, and the softmax has two products' time before PV(t) wants P(t).
// D <= 128: two groups of four warps take turns at the tiles, a thread to a row.
// A group hands the row's maximum on before it forms its weights, so that the
// other's tile can follow; each keeps its own part of l, and whichever moves the
// maximum rescales O.
//
// Masked places.  Scores of positions a row does not see are replaced, not
// added to, so a key that is not finite there cannot pass.  In PV a zero weight
// would still meet the value: in a tile that some row here does not see whole,
// values that are not finite are zeroed in shared memory before its PV (one look
// at the tile, 16 KB a warp at most), and the rows that do see them take them
// in afterwards, from the cache (add_nonfinite).
//
// Work split.  All CTAs derive the same plan from the device-side offsets and
// lengths: items in order of falling length, dealt back and forth over the
// workers; where there are too few of them (short prompts behind a long
// context) each is cut along its keys into pieces of S tiles, whose O, m and l
// go to the workspace as fp32 and are joined by a second kernel.
//
// Bound by the tensor cores: at D = 256 a tile's two products take 2,048 cycles
// and a tile takes about 2,300 (tensor pipe 77 % active over a whole call of
// 8,192 rows under a power cap).  24 + 4 heads of 256, caches cold, and the same
// operations at the measured rate of a large library product: 8,192 rows 493 us
// (432), 1,024 rows behind 130,048 1,992 us (1,722), packed 2,047 + 1 + 515 + 4,096
// rows with a gate 258 us (159; tiles that are half masked and short items), 24
// rows behind 65,536 60.6 us (40 of bytes; pieces of a few tiles, then the join).
#include <cmath>
#include <cstring>

#include "attn_prompt.cuh"
#include "ptx.cuh"
#include "tensor_map.hpp"

namespace tv {

constexpr int kKeyTile = 128;
constexpr float kMoveMax = 8.f;
constexpr int kPieceTiles = 2;     // shortest piece of a split item
constexpr int kMaxPieces = 12 * 152;  // workspace records (pieces), at most: 12 a CTA on 152 SMs

struct PromptPlan {
  int total, S;
  int seq[TV_MAX_SEQ];                                       // sequences in order of falling key tiles
  int cum[TV_MAX_SEQ + 1], slot0[TV_MAX_SEQ];                // by place in that order
  int off[TV_MAX_SEQ], n[TV_MAX_SEQ], L[TV_MAX_SEQ], rt[TV_MAX_SEQ], pm[TV_MAX_SEQ];  // by sequence
};

template <int D>
struct Pa {
  static constexpr int UPT = D == 256 ? 2 : 1;              // ring units per key (or value) tile
  static constexpr int UNIT = kKeyTile * D * 2 / UPT;       // bytes of a unit
  // Two groups of softmax warps that take turns at the tiles, a thread a row, each
  // with an S, a P and barriers of its own, where tensor memory has room: the
  // softmax of a tile takes longer than its products there (D = 256: not so, and
  // no room).  8,192 rows of 16 + 2 heads of 128 take 230 us, 270 with one group
  // (144 of operations), 8 + 8 heads of 64 109 and 135 (36).
  static constexpr bool TURNS = D <= 128;
  static constexpr int SB = TURNS ? 2 : 1;                  // S and P buffers
  static constexpr int NU = D == 64 ? 8 : D == 128 ? 4 : 5;
  static constexpr int KBOX = kKeyTile * 128;               // bytes of a K box (128 rows, 64 columns)
  static constexpr int KBU = D / 64 / UPT;                  // K boxes per unit
  static constexpr int VROWS = kKeyTile / UPT;              // positions of a V box
  static constexpr int VBOX = VROWS * 128;
  static constexpr int VB = D / 64;                         // V boxes per unit
  static constexpr int PT = 128 * kKeyTile * 2;
  static constexpr int QR = D == 256 ? 2 : 1;               // 64-column boxes of Q per half of the softmax, one at a time
  static constexpr int QH = D == 64 ? 1 : 2;                // halves that move Q
  static constexpr int QBOX = 128 * 128;
  static constexpr int T_O = 0, T_S = D, T_Q = D + SB * 128;
  static constexpr int COLS = 512;
  static_assert(T_Q + D / 2 <= COLS, "tensor memory");
  static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, kKeyTile, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true);
  static constexpr int QOFF = NU * UNIT + SB * PT;               // Q on its way into tensor memory
  static constexpr int XOFF = QOFF + QH * QBOX;             // exchanged values [2][2][128] fp32 (turns: [2][128], then maxima [2][128])
  static constexpr int BOFF = XOFF + 2 * 2 * 128 * 4;
  static constexpr int NBAR = 2 * NU + 4 * SB + 2 + 4 + 2 + 4 + 8;
  static constexpr int LOFF = (BOFF + NBAR * 8 + 15) / 16 * 16;  // TMEM base, give-up flag, skip flag, plan
  static constexpr int SMEM = LOFF + 16 + static_cast<int>(sizeof(PromptPlan));
  static_assert(KBU * KBOX == UNIT && VB * VBOX == UNIT, "unit shape");
  static_assert(SMEM <= 232448, "shared memory");
};

struct AttnPromptTcParams {
  CUtensorMap tmK[TV_MAX_SEQ];
  CUtensorMap tmV[TV_MAX_SEQ];
  CUtensorMap tmQ;  // [n_total][Hq][D] in boxes of T tokens, G heads, 64 columns
  PromptRows pr;
  const __nv_bfloat16* V[TV_MAX_SEQ];
  const __nv_bfloat16* gate;
  __nv_bfloat16* out;
  float* ws;
  int Hq, Hkv, G, T;  // T tokens per row tile
  int workers, slots;
  float c;  // scale * log2(e)
};

constexpr int64_t kNoRow = -1;

__device__ __forceinline__ void st_shared16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// Two values times the sigmoids of their gates, by the fast exponential and
// divide (a few fp32 steps, far below the bf16 rounding that follows) with one
// reciprocal for both, 1/a = b (1/ab): the special-function unit bounds the
// epilogue.  e^-g is held at 2^62 so that the product stays in range; gates that
// this would touch, under kNearGate or NaN, are seen to by far_gates.
constexpr float kNearGate = -42.75f;  // the least bf16 with e^-g <= 2^62
__device__ __forceinline__ f2_t gate2(f2_t x, uint32_t g) {
  float u, v;
  f2_unpack(f2_mul(f2_from_bf16x2(g), f2_dup(-1.4426950408889634f)), u, v);
  f2_unpack(f2_add(f2_pack(ex2_approx(fminf(u, 62.f)), ex2_approx(fminf(v, 62.f))), f2_dup(1.f)), u, v);
  return f2_mul(x, f2_mul(f2_dup(rcp_approx(__fmul_rn(u, v))), f2_pack(v, u)));
}
// The smaller of each half of two bf16 pairs, NaN where either is.
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// For gates that are not near: columns of O, before they are read out, times what
// such a gate has beyond gate2's factor of 2^-62: 2^62 sigmoid(g), or NaN.
static __device__ __noinline__ void far_gates(uint32_t o, const __nv_bfloat16* gate, int cols, bool act) {
  for (int c = 0; c < cols; c++) {
    const float x = tmem_ld1(o + c), g = act ? __bfloat162float(gate[c]) : 0.f;
    tmem_st1(o + c, g >= kNearGate ? x : __fmul_rn(gate_mul(x, g), 0x1p62f));
    __syncwarp();
  }
  tmem_st_wait();
}
__device__ __forceinline__ uint32_t bf16_of(f2_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return pack_bf16x2(a, b);
}

// 2^(s c + neg) of two scores, added to a sum, and as a bf16 pair.
__device__ __forceinline__ uint32_t weights(float s0, float s1, f2_t c, f2_t neg, f2_t& sum) {
  float a, b;
  f2_unpack(f2_fma(f2_pack(s0, s1), c, neg), a, b);
  a = ex2_approx(a);
  b = ex2_approx(b);
  sum = f2_add(sum, f2_pack(a, b));
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ uint32_t times_zero_plus(uint32_t x, uint32_t acc) {  // bf16 pairs
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  return r;
}
// Columns of O, before they are read out, plus the values of rows [from, to) that
// are not finite.  Their weights are taken as above zero and so change nothing (one
// of exactly zero, from a score of -inf, would make NaN of an infinity).
static __device__ __noinline__ void add_nonfinite(uint32_t o, const __nv_bfloat16* v, int stride, int cols, int from, int to) {
  for (int c = 0; c < cols; c++) {
    float x = tmem_ld1(o + c);
    for (int t = from; t < to; t++) {
      const float y = __bfloat162float(v[static_cast<size_t>(t) * stride + c]);
      if (!isfinite(y)) x = __fadd_rn(x, y);
    }
    __syncwarp();
    tmem_st1(o + c, x);
  }
  tmem_st_wait();
}

// Zeroes the values that are not finite in rows row, row + step, .. below `to` of a
// value tile, a 16-byte piece of a row a lane; b0, b1: its units.
template <int VROWS>
static __device__ __noinline__ void zero_nonfinite(uint32_t b0, uint32_t b1, int row, int step, int to) {
  for (; row < to; row += step) {
    const uint32_t a = (row >= VROWS ? b1 : b0) + (row % VROWS) * 128;
    const uint4 v = ld_shared16(a);
    st_shared16(a, make_uint4(v.x & finite2(v.x), v.y & finite2(v.y), v.z & finite2(v.z), v.w & finite2(v.w)));
  }
}

// The first row that is loaded for the key tile at position pos: a tile that
// would reach past the rows the sequence holds (the cache may end there, or its
// pages) is taken from further up, and the positions before pos in it are masked.
// Rows before the cache's first come in as zeros.
__device__ __forceinline__ int tile_row(int pos, int end) { return min(pos, end - kKeyTile); }

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The plan, by one warp.  Cost of a candidate, in key tiles: the waves of
// pieces at their mean length, the longest piece's overhang, about three tiles
// to start and end a piece and four more to write and join a partial one.  Both
// kernels make it for themselves, so every step rounds by itself: contracted
// differently in the two, near ties would give two plans.
__device__ inline void make_plan(const AttnPromptTcParams& p, const WarpSeqs& w, int lane, PromptPlan& pl) {
  const int n = w.end - w.off;
  const bool live = lane < p.pr.n_seq && n > 0;
  const int rt = live ? ceil_div(n, p.T) : 0;
  const int nk = live ? ceil_div(w.len + n, kKeyTile) : 0;
  const int nk0 = live ? ceil_div(w.len + min(n, p.T), kKeyTile) : 0;
  int nkmax = nk;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) nkmax = max(nkmax, __shfl_xor_sync(0xffffffffu, nkmax, o));
  const int wide = lane < 16 ? lane + 1 : 0;
  // pieces of the longest item to try: 1 .. 16, then in steps of about a fifth
  int cand = wide ? wide : static_cast<int>(16.f * exp2f((lane - 15) * 0.25f));
  int S = max(max(ceil_div(nkmax, cand), kPieceTiles), 1);
  float W = 0.f, P = 0.f, part = 0.f, longest = 0.f;
  for (int s = 0; s < p.pr.n_seq; s++) {
    const int r = __shfl_sync(0xffffffffu, rt, s), k1 = __shfl_sync(0xffffffffu, nk, s),
              k0 = __shfl_sync(0xffffffffu, nk0, s);
    if (r == 0) continue;
    const float items = __fmul_rn(static_cast<float>(p.Hkv), static_cast<float>(r));
    const int pm = ceil_div(k1, S);
    const float pieces = __fmul_rn(items, static_cast<float>(pm));
    W = __fadd_rn(W, __fmul_rn(__fmul_rn(items, 0.5f), static_cast<float>(k0 + k1)));
    P = __fadd_rn(P, pieces);
    if (pm > 1) part = __fadd_rn(part, pieces);
    longest = fmaxf(longest, static_cast<float>(min(S, k1)));
  }
  const float workers = static_cast<float>(p.workers), mean = __fdiv_rn(W, fmaxf(P, 1.f));
  float cost = __fmul_rn(ceilf(__fdiv_rn(P, workers)), __fadd_rn(mean, 3.f));
  cost = __fadd_rn(cost, __fmul_rn(0.5f, __fsub_rn(longest, mean)));
  cost = __fadd_rn(cost, __fdiv_rn(__fmul_rn(4.f, part), workers));
  if (part > static_cast<float>(p.slots)) cost = INFINITY;  // lane 0 (one piece) always fits
  int best = lane;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const float c2 = __shfl_xor_sync(0xffffffffu, cost, o);
    const int b2 = __shfl_xor_sync(0xffffffffu, best, o);
    if (c2 < cost || (c2 == cost && b2 < best)) {
      cost = c2;
      best = b2;
    }
  }
  S = __shfl_sync(0xffffffffu, S, best);
  const int pm = live ? ceil_div(nk, S) : 0;
  if (lane < TV_MAX_SEQ) {
    pl.off[lane] = w.off;
    pl.n[lane] = n;
    pl.L[lane] = w.len;
    pl.rt[lane] = rt;
    pl.pm[lane] = pm;
    // place in the order: longer sequences (ties: earlier ones) come first
  }
  int place = 0;
  for (int s = 0; s < p.pr.n_seq; s++) {
    const int k2 = __shfl_sync(0xffffffffu, nk, s);
    if (k2 > nk || (k2 == nk && s < lane)) place++;
  }
  if (lane < p.pr.n_seq) pl.seq[place] = lane;
  __syncwarp();
  if (lane == 0) {
    pl.S = S;
    int cum = 0, slot = 0;
    for (int i = 0; i < p.pr.n_seq; i++) {
      const int s = pl.seq[i];
      pl.cum[i] = cum;
      pl.slot0[i] = slot;
      const int cnt = pl.rt[s] * p.Hkv * pl.pm[s];
      cum += cnt;
      if (pl.pm[s] > 1) slot += cnt;
    }
    pl.cum[p.pr.n_seq] = cum;
    pl.total = cum;
  }
  __syncwarp();
}

struct PromptItem {
  int s, g, i, t0, t1, slot;  // key tiles [t0, t1); slot -1: the item is whole
};
// Piece x of the plan (pieces past a shorter item's end are empty: t0 >= t1).
__device__ __forceinline__ PromptItem item_of(const AttnPromptTcParams& p, const PromptPlan& pl, int x) {
  int at = 0;
  while (at < p.pr.n_seq - 1 && x >= pl.cum[at + 1]) at++;
  PromptItem I;
  I.s = pl.seq[at];
  const int r = x - pl.cum[at], per = p.Hkv * pl.rt[I.s];
  const int j = r / per, r2 = r % per;
  I.i = pl.rt[I.s] - 1 - r2 / p.Hkv;  // longest row tiles first
  I.g = r2 % p.Hkv;
  const int nk = ceil_div(pl.L[I.s] + min((I.i + 1) * p.T, pl.n[I.s]), kKeyTile);
  I.t0 = j * pl.S;
  I.t1 = min(I.t0 + pl.S, nk);
  I.slot = nk > pl.S ? pl.slot0[at] + r : -1;
  return I;
}
// The x-th piece of a worker: waves run back and forth over the workers, so
// the one that got the longest piece of a wave gets the shortest of the next.
__device__ __forceinline__ int piece_index(int wave, int worker, int workers) {
  return wave * workers + ((wave & 1) ? workers - 1 - worker : worker);
}

// The worker's next piece with tiles, from wave `wave` on; false: none left.
__device__ __forceinline__ bool next_item(const AttnPromptTcParams& p, const PromptPlan& pl, int total, int worker, int& wave,
                                          PromptItem& I) {
  while (wave * p.workers < total) {
    const int x = piece_index(wave, worker, p.workers);
    wave++;
    if (x >= total) continue;
    I = item_of(p, pl, x);
    if (I.t0 < I.t1) return true;
  }
  return false;
}

template <int D>
__global__ void __launch_bounds__(384, 1) attn_prompt_tc_kernel(const __grid_constant__ AttnPromptTcParams p) {
  using C = Pa<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // tiles are swizzled in 1024-byte atoms
  uint8_t* gb = smem_raw;
  const uint32_t sb = smem_u32(smem_raw);
  const uint32_t ring = sb, pbuf = sb + C::NU * C::UNIT;
  float* xmax = reinterpret_cast<float*>(gb + C::XOFF);
  const uint32_t bars = sb + C::BOFF;
  const uint32_t UFULL0 = bars, UEMPTY0 = bars + 8u * C::NU;
  const uint32_t SFULL0 = bars + 16u * C::NU, SFREE0 = SFULL0 + 8u * C::SB, PFULL0 = SFREE0 + 8u * C::SB,
                 ODONE0 = PFULL0 + 8u * C::SB, QREADY = ODONE0 + 8u * C::SB, OFREE = QREADY + 8u, XBAR0 = QREADY + 16u,
                 DRAIN = XBAR0 + 32u, QFULL0 = DRAIN + 16u, QEMPTY0 = QFULL0 + 16u, MBAR0 = QEMPTY0 + 16u;
  // tile t's barrier of a kind, and the parity of its phase there
  auto bar = [](uint32_t first, uint32_t t) { return first + (C::TURNS ? 8u * (t & 1) : 0u); };
  auto par = [](uint32_t t) { return C::TURNS ? (t >> 1) & 1 : t & 1; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gb + C::LOFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int& skip = *reinterpret_cast<int*>(tmem_slot + 2);
  volatile uint16_t* met = reinterpret_cast<volatile uint16_t*>(tmem_slot + 3);  // items that met values to zero
  PromptPlan& pl = *reinterpret_cast<PromptPlan*>(gb + C::LOFF + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NU; i++) {
      mbar_init(UFULL0 + 8u * i, 1);
      mbar_init(UEMPTY0 + 8u * i, 1);
    }
    for (int i = 0; i < C::SB; i++) {
      mbar_init(SFULL0 + 8u * i, 1);
      mbar_init(SFREE0 + 8u * i, C::TURNS ? 4 : 8);
      mbar_init(PFULL0 + 8u * i, C::TURNS ? 4 : 8);
      mbar_init(ODONE0 + 8u * i, 1);
    }
    mbar_init(QREADY, 8);
    mbar_init(OFREE, 8);
    for (int i = 0; i < 8; i++) mbar_init(MBAR0 + 8u * i, 1);
    for (int i = 0; i < 4; i++) mbar_init(XBAR0 + 8u * i, 2);
    mbar_init(DRAIN, 1);
    mbar_init(DRAIN + 8u, 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(QFULL0 + 8u * i, 1);
      mbar_init(QEMPTY0 + 8u * i, 4);
    }
    *abort_flag = 0;
    met[0] = met[1] = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();  // the join makes its plan on SMs that are done
  if (warp == 2) {  // the plan; a bad launch sets its code and every CTA leaves
    const bool bad = status_bad(p.pr.status);
    const WarpSeqs w = load_seqs(p.pr, lane);
    if (w.code && lane == 0) set_status(p.pr.status, w.code);
    if (lane == 0) {
      skip = bad || w.code || (sb & 1023u) ? 1 : 0;
      if (sb & 1023u) set_status(p.pr.status, TV_ERR_CUDA);
    }
    if (!w.code) make_plan(p, w, lane, pl);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  auto arrive = [&](uint32_t bar) {  // one arrival per warp, after every lane's fences
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  const int total = skip ? 0 : pl.total;

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer ----------------
    uint32_t it = 0;
    bool ok = true;
    int wave = 0;
    PromptItem I;
    while (ok && next_item(p, pl, total, worker, wave, I)) {
      const int n = I.t1 - I.t0, end = pl.L[I.s] + pl.n[I.s];
      for (int e = 0; e < 2 * n && ok; e++) {
        // load order K0, K1 V0, K2 V1, ..., V(n-1)
        const bool is_k = e == 0 || ((e & 1) && e != 2 * n - 1);
        const int k = e == 0 ? 0 : is_k ? (e + 1) / 2 : (e == 2 * n - 1 ? n - 1 : (e - 2) / 2);
        const int row = tile_row((I.t0 + k) * kKeyTile, end);
#pragma unroll
        for (int u = 0; u < C::UPT; u++, it++) {
          const uint32_t slot = it % C::NU, full = UFULL0 + 8u * slot;
          if (!wait_role(UEMPTY0 + 8u * slot, ((it / C::NU) & 1) ^ 1, abort_flag, kWaitCycles)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + slot * C::UNIT;
          mbar_arrive_expect_tx(full, C::UNIT);
          if (is_k) {
#pragma unroll
            for (int b = 0; b < C::KBU; b++) tma_load_3d(dst + b * C::KBOX, &p.tmK[I.s], full, (u * C::KBU + b) * 64, row, I.g);
          } else {
#pragma unroll
            for (int b = 0; b < C::VB; b++) tma_load_3d(dst + b * C::VBOX, &p.tmV[I.s], full, b * 64, row + u * C::VROWS, I.g);
          }
        }
      }
    }
    if (!ok) {
      set_status(p.pr.status, TV_ERR_TIMEOUT);
      // let every issued copy land before shared memory is released
      for (uint32_t i = it > C::NU ? it - C::NU : 0; i < it; i++)
        mbar_wait(UFULL0 + 8u * (i % C::NU), (i / C::NU) & 1, kWaitCycles);
    }
  } else if (warp == 11 && lane == 0) {
    // ---------------- queries (and, into L2, gates) of the items ahead ----------------
    uint32_t t = 0;
    bool ok = true;
    int wave = 0;
    PromptItem I;
    while (ok && next_item(p, pl, total, worker, wave, I)) {
      const int first = pl.off[I.s] + I.i * p.T, live = min(p.T, pl.n[I.s] - I.i * p.T);
      for (int r = 0; r < C::QR && ok; r++, t++)
#pragma unroll
        for (int h = 0; h < C::QH; h++) {
          ok = ok && wait_role(QEMPTY0 + 8u * h, (t & 1) ^ 1, abort_flag, kWaitCycles);
          if (!ok) break;
          mbar_arrive_expect_tx(QFULL0 + 8u * h, static_cast<uint32_t>(p.T * p.G) * 128u);
          tma_load_3d(sb + C::QOFF + h * C::QBOX, &p.tmQ, QFULL0 + 8u * h, (h * C::QR + r) * 64, I.g * p.G, first);
        }
      if (p.gate && I.slot < 0)  // (a token's heads of one KV head are contiguous)
        for (int x = 0; x < live; x++)
          bulk_prefetch_l2(p.gate + ((static_cast<int64_t>(first) + x) * p.Hq + I.g * p.G) * D, p.G * D * 2);
    }
    if (!ok) {
      set_status(p.pr.status, TV_ERR_TIMEOUT);
      for (int h = 0; h < C::QH; h++)
        if (t > 0) mbar_wait(QFULL0 + 8u * h, (t - 1) & 1, kWaitCycles);
    }
  } else if (warp == 1 || warp == 10) {
    // ---------------- MMA issuers, one warp each, whole-warp loops with one
    // elected lane issuing.  Issuing blocks while the tensor pipe's short queue
    // is full, and a wait between two products costs some hundred cycles in
    // which a single issuer would let the queue run dry: with one warp for both
    // products a tile took 2,750 cycles, with two it takes about the pipe's
    // time.  Unit numbers follow the load order. ----------------
    const bool is_qk = warp == 1;
    uint32_t base = 0, t = 0, items = 0;  // units and tiles before the item, items
    bool ok = true;
    int wave = 0;
    PromptItem I;
    while (ok && next_item(p, pl, total, worker, wave, I)) {
      const int n = I.t1 - I.t0;
      if (is_qk) ok = wait_warp(QREADY, items & 1, abort_flag, kWaitCycles);
      items++;
      for (int k = 0; k < n && ok; k++, t++) {
        if (is_qk) {
          if (t >= C::SB) ok = wait_warp(bar(SFREE0, t), par(t - C::SB), abort_flag, kWaitCycles);
          const uint32_t u0 = base + (k == 0 ? 0 : 2 * k - 1) * C::UPT;
#pragma unroll
          for (int u = 0; u < C::UPT; u++) {
            const uint32_t slot = (u0 + u) % C::NU;
            ok = ok && wait_warp(UFULL0 + 8u * slot, ((u0 + u) / C::NU) & 1, abort_flag, kWaitCycles);
            if (!ok) break;
            tc_fence_after();
            if (elect_one_sync()) {
              const uint64_t k0 = sdesc_sw128(ring + slot * C::UNIT, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < C::KBU * 4; kk++)
                tc_mma_ts(tbase + C::T_S + (t % C::SB) * 128, tbase + C::T_Q + (u * C::KBU * 4 + kk) * 8,
                          k0 + static_cast<uint64_t>(((kk >> 2) * C::KBOX + (kk & 3) * 32) >> 4), C::IDESC_QK,
                          (u > 0 || kk > 0) ? 1u : 0u);
              tc_commit(UEMPTY0 + 8u * slot);
              if (u == C::UPT - 1) tc_commit(bar(SFULL0, t));
            }
            __syncwarp();
          }
        } else {
          ok = wait_warp(bar(PFULL0, t), par(t), abort_flag, kWaitCycles);
          // (turns: O may still be on its way out of the item before)
          if (C::TURNS && k == 0 && items > 1) ok = ok && wait_warp(OFREE, (items - 2) & 1, abort_flag, kWaitCycles);
          const uint32_t u0 = base + (k < n - 1 ? 2 * k + 2 : 2 * n - 1) * C::UPT;
#pragma unroll
          for (int u = 0; u < C::UPT; u++) {
            const uint32_t slot = (u0 + u) % C::NU;
            ok = ok && wait_warp(UFULL0 + 8u * slot, ((u0 + u) / C::NU) & 1, abort_flag, kWaitCycles);
            if (!ok) break;
            tc_fence_after();
            if (elect_one_sync()) {
              const uint64_t v0 = sdesc_sw128(ring + slot * C::UNIT, C::VBOX, 1024);
              const uint64_t p0 = sdesc_sw128(pbuf + (t % C::SB) * C::PT, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < C::VROWS / 16; kk++) {
                const int pk = u * (C::VROWS / 16) + kk;  // 16-position step of the tile
                tc_mma_ss(tbase + C::T_O, p0 + static_cast<uint64_t>(((pk >> 2) * 16384 + (pk & 3) * 32) >> 4),
                          v0 + static_cast<uint64_t>((kk * 2048) >> 4), C::IDESC_PV, (k > 0 || pk > 0) ? 1u : 0u);
              }
              tc_commit(UEMPTY0 + 8u * slot);
              if (u == C::UPT - 1) tc_commit(bar(ODONE0, t));
            }
            __syncwarp();
          }
        }
      }
      base += 2 * n * C::UPT;
    }
    if (!ok && lane == 0) set_status(p.pr.status, TV_ERR_TIMEOUT);
    // every MMA of this warp completes before tensor and shared memory are released
    const uint32_t drain = DRAIN + (is_qk ? 0u : 8u);
    if (elect_one_sync()) tc_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, kWaitCycles);
  } else if (warp >= 2 && warp < 10) {
    // ---------------- softmax and output, a row's columns of O to two threads ----------------
    const int hf = (warp - 2) >> 2, quad = warp & 3, lrow = quad * 32 + lane;
    const uint32_t tl = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t patch = pbuf + hf * (C::TURNS ? C::PT : 16384) + quad * 4096;  // where this warp writes P: 4 KB of its own between items
    const int tok = lrow / p.G, head = lrow % p.G;
    uint32_t t = 0, it = 0, id = 0;  // tiles, units before the item, items (this one counted)
    bool ok = true;
    // the two threads of a row exchange a value
    auto exchange = [&](float v, float& other) {
      const uint32_t xc = C::TURNS ? id - 1 : t + id - 1;  // exchanges before: one an item (turns), or one a tile too
      float* x = xmax + (C::TURNS ? 0 : xc & 1) * 256;      // (turns: QREADY lies between two)
      x[hf * 128 + lrow] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(XBAR0 + 8u * quad);
      if (!wait_warp(XBAR0 + 8u * quad, xc & 1, abort_flag, kWaitCycles)) return false;
      other = x[(hf ^ 1) * 128 + lrow];
      return true;
    };
    // this thread's row of q and out of an item (elements); kNoRow: none
    auto row_of = [&](const PromptItem& I) -> int64_t {
      const int token = I.i * p.T + tok;
      return tok < p.T && token < pl.n[I.s] ? ((static_cast<int64_t>(pl.off[I.s]) + token) * p.Hq + I.g * p.G + head) * D : kNoRow;
    };
    // Q of an item into tensor memory, each thread its half of its row, once
    // every Q K^T of the item before has completed (its last S has been read)
    auto load_q = [&]() {
      if (hf < C::QH) {
#pragma unroll
        for (int r = 0; r < C::QR; r++) {
          if (!wait_warp(QFULL0 + 8u * hf, (id * C::QR + r) & 1, abort_flag, kWaitCycles)) return false;
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const uint4 x = ld_shared16(sb + C::QOFF + hf * C::QBOX + lrow * 128 + (((i ^ lrow) & 7) << 4));
            v[4 * i] = x.x;
            v[4 * i + 1] = x.y;
            v[4 * i + 2] = x.z;
            v[4 * i + 3] = x.w;
          }
          tmem_st32(tl + C::T_Q + (hf * C::QR + r) * 32, v);
          // Only now: the store has waited for the loads.  An arrival does not, and
          // products keep shared memory busy enough for the next box to overtake them.
          arrive(QEMPTY0 + 8u * hf);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      arrive(QREADY);
      return true;
    };
    int wave = 0;
    PromptItem I;
    bool more = next_item(p, pl, total, worker, wave, I);
    int64_t orow = kNoRow;
    if (more) {
      orow = row_of(I);
      ok = load_q();
    }
    // met[id & 1] = id (its low bits): item id met a value to zero.  (A warp may be
    // an item ahead of another, not two: their P arrivals hold them together.)
    while (ok && more) {
      id++;
      const int n = I.t1 - I.t0, L = pl.L[I.s], end = L + pl.n[I.s];
      const bool act = orow >= 0;
      const int last = act ? L + I.i * p.T + tok : -1;  // last position this row sees
      const int seen_all = L + I.i * p.T + 1;           // positions every row here sees
      float m = -INFINITY, l = 0.f, lo = 0.f;  // maximum, and the sum's two parts
      // values of tile k that are not finite, where some row here does not see all
      auto look = [&](int k, int pos) {
        const int first = max(seen_all - tile_row(pos, end), 0);
        const uint32_t u0 = it + (k < n - 1 ? 2 * k + 2 : 2 * n - 1) * C::UPT;  // the tile's value units
        uint32_t slot[C::UPT];
#pragma unroll
        for (int u = 0; u < C::UPT; u++) {
          slot[u] = (u0 + u) % C::NU;
          ok = ok && wait_warp(UFULL0 + 8u * slot[u], ((u0 + u) / C::NU) & 1, abort_flag, kWaitCycles);
        }
        if (!ok) return false;
        constexpr int PPR = C::VB * 8, RPW = 32 / PPR;  // 16-byte pieces of a row, rows a warp looks at
        const uint32_t piece = (lane % PPR >> 3) * C::VBOX + (lane & 7) * 16;
        auto at = [&](int row) {
          return ring + (C::UPT > 1 && row >= C::VROWS ? slot[C::UPT - 1] : slot[0]) * C::UNIT + (row % C::VROWS) * 128 + piece;
        };
        const int row0 = first + (C::TURNS ? quad : warp - 2) * RPW + lane / PPR;
        uint32_t sum[4] = {0u, 0u, 0u, 0u};  // of value x 0: zero, or NaN
#pragma unroll 4
        for (int row = row0; row < kKeyTile; row += (C::TURNS ? 4 : 8) * RPW) {
          const uint4 v = ld_shared16(at(row));
          sum[0] = times_zero_plus(v.x, sum[0]);
          sum[1] = times_zero_plus(v.y, sum[1]);
          sum[2] = times_zero_plus(v.z, sum[2]);
          sum[3] = times_zero_plus(v.w, sum[3]);
        }
        if ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) {
          for (int row = row0; row < kKeyTile; row += (C::TURNS ? 4 : 8) * RPW) {
            const uint4 v = ld_shared16(at(row));
            st_shared16(at(row), make_uint4(v.x & finite2(v.x), v.y & finite2(v.y), v.z & finite2(v.z), v.w & finite2(v.w)));
          }
          met[id & 1] = static_cast<uint16_t>(id);
        }
        // a tile taken from further up: rows before `pos` have no weight here, whoever
        // sees them (they count in the tile before)
        const int again = pos - tile_row(pos, end);
        if (again > 0)
          zero_nonfinite<C::VROWS>(at(0), at(C::VROWS % kKeyTile), row0 - first, (C::TURNS ? 4 : 8) * RPW, again);
        return true;
      };
      if constexpr (C::TURNS) {
        float mine_m = -INFINITY;  // the maximum that l counts from
        float* const mrow = xmax + 256;
        for (int k = 0; k < n; k++, t++) {
          if ((t & 1) != static_cast<uint32_t>(hf)) continue;  // the other group's
          if (!wait_warp(bar(SFULL0, t), par(t), abort_flag, kWaitCycles)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ts = tl + C::T_S + hf * 128;
          const int pos = (I.t0 + k) * kKeyTile, first_row = tile_row(pos, end);
          const bool whole = pos + kKeyTile <= seen_all;
          const int vis = last - first_row, from = pos - first_row;
          // 64 scores at a time: loops, not 128 scores in a row, since the code of two
          // groups and the issuers has to stay in the instruction cache
          uint32_t a[32], b[32];
          auto load = [&](int c) {
            tmem_ld32_nowait(ts + c, a);
            tmem_ld32_nowait(ts + c + 32, b);
            tmem_ld_wait(a, b);
            if (!whole) {
#pragma unroll
              for (int j = 0; j < 32; j++) {
                if (c + j < from || c + j > vis) a[j] = __float_as_uint(-INFINITY);
                if (c + 32 + j < from || c + 32 + j > vis) b[j] = __float_as_uint(-INFINITY);
              }
            }
          };
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            load(c);
#pragma unroll
            for (int j = 0; j < 32; j++) mx[j & 3] = fmaxf(mx[j & 3], fmaxf(__uint_as_float(a[j]), __uint_as_float(b[j])));
          }
          const float mt = __fmul_rn(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), p.c);
          float before = -INFINITY;  // the maximum after the tile before, from the other group
          if (k > 0) {
            if (!wait_warp(MBAR0 + 8u * (quad * 2 + (hf ^ 1)), par(t - 1), abort_flag, kWaitCycles)) {
              ok = false;
              break;
            }
            before = mrow[(hf ^ 1) * 128 + lrow];
          }
          m = before;
          if (mt > __fadd_rn(m, kMoveMax) || (m == -INFINITY && mt > -INFINITY)) m = mt;
          mrow[hf * 128 + lrow] = m;
          arrive(MBAR0 + 8u * (quad * 2 + hf));
          const float neg = m == -INFINITY ? 0.f : -m;  // nothing seen yet: every p below is 2^-inf = 0
          // this group's last P has been read
          if (t >= 2 && !wait_warp(bar(ODONE0, t), par(t - 2), abort_flag, kWaitCycles)) {
            ok = false;
            break;
          }
          f2_t acc[2] = {0ull, 0ull};
          const f2_t c2 = f2_dup(p.c), neg2 = f2_dup(neg);
          uint32_t line = pbuf + hf * C::PT + (lrow >> 3) * 1024 + (lrow & 7) * 128;
#pragma unroll 1
          for (int c = 0; c < 128; c += 64, line += 16384) {
            load(c);
            if (c > 0) {  // S is free for the tile after next, half the weights ahead of P
              tc_fence_before();
              arrive(bar(SFREE0, t));
            }
            auto put = [&](const uint32_t (&x)[32], int q0) {
#pragma unroll
              for (int q = 0; q < 4; q++) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                  w[e] = weights(__uint_as_float(x[8 * q + 2 * e]), __uint_as_float(x[8 * q + 2 * e + 1]), c2, neg2, acc[e & 1]);
                st_shared16(line + ((((q0 + q) ^ lrow) & 7) << 4), make_uint4(w[0], w[1], w[2], w[3]));
              }
            };
            put(a, 0);
            put(b, 4);
          }
          l = __fmaf_rn(l, mine_m == m ? 1.f : ex2_approx(__fsub_rn(mine_m, m)), f2_hsum(f2_add(acc[0], acc[1])));
          mine_m = m;
          const float alpha = before == m ? 1.f : ex2_approx(__fsub_rn(before, m));
          if (k > 0 && __any_sync(0xffffffffu, act && alpha != 1.f)) {  // once O rests
            if (!wait_warp(bar(ODONE0, t - 1), par(t - 1), abort_flag, kWaitCycles)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t r[32];
              tmem_ld32(tl + C::T_O + c, r);
#pragma unroll
              for (int i = 0; i < 32; i++) r[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[i]), alpha));
              tmem_st32(tl + C::T_O + c, r);
            }
            tmem_st_wait();
          }
          if (!whole && !look(k, pos)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();
          tc_fence_before();
          arrive(bar(PFULL0, t));
        }
        if (ok) {
          // the item's last maximum and S, whichever group's they were
          ok = wait_warp(MBAR0 + 8u * (quad * 2 + ((t - 1) & 1)), par(t - 1), abort_flag, kWaitCycles) &&
               wait_warp(bar(SFULL0, t - 1), par(t - 1), abort_flag, kWaitCycles);
          m = mrow[((t - 1) & 1) * 128 + lrow];
          if (mine_m != m) l = __fmul_rn(l, ex2_approx(__fsub_rn(mine_m, m)));
          tc_fence_after();
          // (before QREADY, so that the next item's cannot overtake it)
          ok = ok && exchange(l, lo);
        }
      } else {
        for (int k = 0; k < n; k++, t++) {
          if (!wait_warp(SFULL0, t & 1, abort_flag, kWaitCycles)) {
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
          arrive(SFREE0);
          const int pos = (I.t0 + k) * kKeyTile;
          if (pos + kKeyTile > seen_all) {  // a tile some row here does not see whole
            const int row = tile_row(pos, end), vis = last - (row + hf * 64), from = pos - (row + hf * 64);
#pragma unroll
            for (int j = 0; j < 64; j++) sv[j] = j >= from && j <= vis ? sv[j] : -INFINITY;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 64; j += 2) mx[(j / 2) & 3] = fmaxf(mx[(j / 2) & 3], fmaxf(sv[j], sv[j + 1]));
          float mo;
          const float mh = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (!exchange(mh, mo)) {
            ok = false;
            break;
          }
          const float mt = __fmul_rn(fmaxf(mh, mo), p.c);
          float alpha = 1.f;
          if (mt > __fadd_rn(m, kMoveMax) || (m == -INFINITY && mt > -INFINITY)) {
            alpha = ex2_approx(__fsub_rn(m, mt));  // 0 from m = -inf
            m = mt;
          }
          const float neg = m == -INFINITY ? 0.f : -m;  // nothing seen yet: every p below is 2^-inf = 0
          uint32_t P[32];
          f2_t acc[2] = {0ull, 0ull};
          const f2_t c2 = f2_dup(p.c), neg2 = f2_dup(neg);
#pragma unroll
          for (int j = 0; j < 64; j += 2) P[j / 2] = weights(sv[j], sv[j + 1], c2, neg2, acc[(j / 2) & 1]);
          l = __fmaf_rn(l, alpha, f2_hsum(f2_add(acc[0], acc[1])));
          // PV of the previous tile is complete: P is free and O rests
          if (t > 0 && !wait_warp(ODONE0, (t - 1) & 1, abort_flag, kWaitCycles)) {
            ok = false;
            break;
          }
          tc_fence_after();
          {
            const uint32_t line = pbuf + hf * 16384 + (lrow >> 3) * 1024 + (lrow & 7) * 128;
#pragma unroll
            for (int q = 0; q < 8; q++)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + (((q ^ lrow) & 7) << 4)), "r"(P[4 * q]),
                           "r"(P[4 * q + 1]), "r"(P[4 * q + 2]), "r"(P[4 * q + 3])
                           : "memory");
          }
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
          if (pos + kKeyTile > seen_all && !look(k, pos)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();
          tc_fence_before();
          arrive(PFULL0);
        }
      }
      it += 2 * n * C::UPT;
      if (!ok) break;
      const int slot = I.slot;
      const int64_t row = orow;
      const int mine = wave;
      more = next_item(p, pl, total, worker, wave, I);
      if (more) {  // the next item's first Q K^T runs beside this one's last P V and output
        orow = row_of(I);
        if (!load_q()) {
          ok = false;
          break;
        }
      }
      // the gates of this warp's rows, 16-byte pieces spread over its lanes, CW
      // columns at a time, each loaded while the columns before are worked on
      constexpr int CW = D >= 128 ? 64 : 32, Q = CW / 8;
      const int prow = lane / Q, pq = lane % Q;  // the row (of 32 / Q) and piece this lane moves
      uint4 gv[Q];
      auto fetch_gate = [&](int c) {
#pragma unroll
        for (int i = 0; i < Q; i++) {
          const int64_t ro = __shfl_sync(0xffffffffu, row, i * (32 / Q) + prow);  // (idle rows: any row will do)
          gv[i] = *reinterpret_cast<const uint4*>(p.gate + (ro < 0 ? 0 : ro) + c + pq * 8);
        }
      };
      if (p.gate && slot < 0) fetch_gate(hf * (D / 2));
      if ((!C::TURNS && !exchange(l, lo)) || !wait_warp(bar(ODONE0, t - 1), par(t - 1), abort_flag, kWaitCycles)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (met[id & 1] == static_cast<uint16_t>(id)) {
        const PromptItem J = item_of(p, pl, piece_index(mine - 1, worker, p.workers));  // this item again
        const int before = pl.L[J.s] + J.i * p.T + 1;  // seen by all rows
        add_nonfinite(tl + C::T_O + hf * (D / 2), p.V[J.s] + static_cast<size_t>(J.g) * p.pr.cap * D + hf * (D / 2), D, D / 2,
                      max(before, J.t0 * kKeyTile), row >= 0 ? min(before + tok, J.t1 * kKeyTile) : 0);
      }
      const float inv = __fdiv_rn(1.f, __fadd_rn(l, lo));
      // Rows leave through this warp's patch, where they are turned around so
      // that an instruction covers whole pieces of rows.
      if (slot >= 0) {  // a piece: O, m and l as they are, 32 columns at a time
        float* rec = p.ws + (static_cast<size_t>(slot) * 128 + lrow) * (D + 4);
#pragma unroll 1
        for (int c = hf * (D / 2); c < (hf + 1) * (D / 2); c += 32) {
          uint32_t r[32];
          tmem_ld32(tl + C::T_O + c, r);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; i++)
            st_shared16(patch + lane * 128 + (((i ^ lane) & 7) << 4), make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const int rr = 4 * i + (lane >> 3);
            const uint4 x = ld_shared16(patch + rr * 128 + (((lane ^ rr) & 7) << 4));
            if (__shfl_sync(0xffffffffu, row, rr) >= 0)
              *reinterpret_cast<uint4*>(rec + (rr - lane) * (D + 4) + c + (lane & 7) * 4) = x;
          }
        }
        if (act && hf == 0) {
          rec[D] = m;
          rec[D + 1] = __fadd_rn(l, lo);
        }
      } else {
#pragma unroll 1
        for (int c = hf * (D / 2); c < (hf + 1) * (D / 2); c += CW) {
          if (p.gate) {  // one look at all of the warp's gates of these columns
            uint32_t least = min_nan2(gv[0].x, gv[0].y);
#pragma unroll
            for (int i = 0; i < Q; i++)
              least = min_nan2(least, min_nan2(min_nan2(gv[i].x, gv[i].y), min_nan2(gv[i].z, gv[i].w)));
            if (__any_sync(0xffffffffu, !(bf16_lo(least) >= kNearGate && bf16_hi(least) >= kNearGate)))
              far_gates(tl + C::T_O + c, p.gate + row + c, CW, row >= 0);
          }
          f2_t y[CW / 2];
          const f2_t inv2 = f2_dup(inv);
#pragma unroll
          for (int b = 0; b < CW; b += 32) {
            uint32_t r[32];
            tmem_ld32(tl + C::T_O + c + b, r);
#pragma unroll
            for (int i = 0; i < 16; i++)
              y[b / 2 + i] = f2_mul(f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), inv2);
          }
          if (p.gate) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < Q; i++) {
              const int rr = i * (32 / Q) + prow;
              st_shared16(patch + rr * 128 + (((pq ^ rr) & 7) << 4), gv[i]);
            }
            __syncwarp();
            if (c + CW < (hf + 1) * (D / 2)) fetch_gate(c + CW);
#pragma unroll
            for (int i = 0; i < Q; i++) {
              const uint4 g = ld_shared16(patch + lane * 128 + (((i ^ lane) & 7) << 4));
              y[4 * i] = gate2(y[4 * i], g.x);
              y[4 * i + 1] = gate2(y[4 * i + 1], g.y);
              y[4 * i + 2] = gate2(y[4 * i + 2], g.z);
              y[4 * i + 3] = gate2(y[4 * i + 3], g.w);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < Q; i++)
            st_shared16(patch + lane * 128 + (((i ^ lane) & 7) << 4),
                        make_uint4(bf16_of(y[4 * i]), bf16_of(y[4 * i + 1]), bf16_of(y[4 * i + 2]), bf16_of(y[4 * i + 3])));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < Q; i++) {
            const int rr = i * (32 / Q) + prow;
            const uint4 x = ld_shared16(patch + rr * 128 + (((pq ^ rr) & 7) << 4));
            const int64_t ro = __shfl_sync(0xffffffffu, row, rr);
            if (ro >= 0) *reinterpret_cast<uint4*>(p.out + ro + c + pq * 8) = x;
          }
        }
      }
      if (C::TURNS) {
        tc_fence_before();
        arrive(OFREE);
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) set_status(p.pr.status, TV_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, C::COLS);
}

// Joins the pieces of split items, in order: a warp takes 128 columns of a row,
// four a lane, the loads of kJ pieces in flight.
template <int D, int kJ>
__global__ void __launch_bounds__(256) attn_prompt_join_kernel(const __grid_constant__ AttnPromptTcParams p) {
  constexpr int CB = D > 128 ? D / 128 : 1, LPR = D >= 128 ? 32 : D / 4, RPW = 32 / LPR;
  __shared__ PromptPlan pl;
  __shared__ int skip;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {  // (offsets and lengths were there before the launch that this one follows)
    const WarpSeqs w = load_seqs(p.pr, lane);
    if (lane == 0) skip = w.code;
    if (!w.code) make_plan(p, w, lane, pl);
  }
  __syncthreads();
  pdl_wait();
  if (skip || status_bad(p.pr.status)) return;
  for (int at = 0; at < p.pr.n_seq; at++) {
    const int s = pl.seq[at];
    if (pl.pm[s] < 2) continue;
    const int64_t units = (static_cast<int64_t>(pl.n[s]) * p.Hq + RPW - 1) / RPW * CB;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + warp; u < units; u += static_cast<int64_t>(gridDim.x) * 8) {
      const int64_t x = u / CB * RPW + lane / LPR;  // row (token, head)
      if (x >= static_cast<int64_t>(pl.n[s]) * p.Hq) continue;
      const int col = static_cast<int>(u % CB) * 128 + (lane % LPR) * 4;
      const int token = static_cast<int>(x / p.Hq), h = static_cast<int>(x % p.Hq), g = h / p.G;
      const int i = token / p.T, lrow = token % p.T * p.G + h % p.G;
      const int nk = ceil_div(pl.L[s] + min((i + 1) * p.T, pl.n[s]), kKeyTile);
      const int np = ceil_div(nk, pl.S);
      if (np < 2) continue;  // written whole
      const int per = p.Hkv * pl.rt[s], first = pl.slot0[at] + (pl.rt[s] - 1 - i) * p.Hkv + g;
      const float* rec = p.ws + (static_cast<size_t>(first) * 128 + lrow) * (D + 4);
      const size_t step = static_cast<size_t>(per) * 128 * (D + 4);
      // one pass with a running maximum, kJ pieces' loads in flight at a time
      float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int j0 = 0; j0 < np; j0 += kJ) {
        float4 o[kJ];
        float2 ml[kJ];
#pragma unroll
        for (int j = 0; j < kJ; j++) {
          const float* r = rec + step * (j0 + j);
          o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          ml[j] = make_float2(-INFINITY, 0.f);
          if (j0 + j < np) {
            o[j] = *reinterpret_cast<const float4*>(r + col);
            ml[j] = *reinterpret_cast<const float2*>(r + D);
          }
        }
        float mn = m;
#pragma unroll
        for (int j = 0; j < kJ; j++) mn = fmaxf(mn, ml[j].x);
        const float a = m == -INFINITY ? 0.f : exp2f(__fsub_rn(m, mn));
        l = __fmul_rn(l, a);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = __fmul_rn(acc[e], a);
#pragma unroll
        for (int j = 0; j < kJ; j++) {
          if (ml[j].y == 0.f) continue;  // no position of this row in the piece (or no piece)
          const float f = exp2f(__fsub_rn(ml[j].x, mn));
          l = __fmaf_rn(f, ml[j].y, l);
          acc[0] = __fmaf_rn(f, o[j].x, acc[0]);
          acc[1] = __fmaf_rn(f, o[j].y, acc[1]);
          acc[2] = __fmaf_rn(f, o[j].z, acc[2]);
          acc[3] = __fmaf_rn(f, o[j].w, acc[3]);
        }
        m = mn;
      }
      const size_t at_o = (static_cast<size_t>(pl.off[s]) * p.Hq + x) * D + col;
      const float inv = __fdiv_rn(1.f, l);
#pragma unroll
      for (int e = 0; e < 4; e++) acc[e] = __fmul_rn(acc[e], inv);
      if (p.gate) {
        const uint2 gv = *reinterpret_cast<const uint2*>(p.gate + at_o);
        acc[0] = gate_mul(acc[0], bf16_lo(gv.x));
        acc[1] = gate_mul(acc[1], bf16_hi(gv.x));
        acc[2] = gate_mul(acc[2], bf16_lo(gv.y));
        acc[3] = gate_mul(acc[3], bf16_hi(gv.y));
      }
      *reinterpret_cast<uint2*>(p.out + at_o) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// A bf16 cache [Hkv][cap][D] as a 3-D tensor in boxes of 64 columns of one head.
static bool encode_cache_map(CUtensorMap* m, void* base, int D, int cap, int Hkv, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(cap), static_cast<cuuint64_t>(Hkv)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(D) * 2 * cap};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [n_total][Hq][D] as a 3-D tensor in boxes of t tokens, g heads, 64 columns.
static bool encode_q_map(CUtensorMap* m, const void* base, int D, int Hq, int n_total, int g, int t) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(n_total)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(D) * 2 * Hq};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(g), static_cast<cuuint32_t>(t)}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace records (one per piece, 128 rows of D + 4 fp32) a call may use:
// never more than its items can be cut into.
static int64_t slots_for(const tv_attn_layer* l, const tv_prompt* pr, int max_len) {
  const int64_t t = 128 / (l->Hq / l->Hkv);
  const int64_t items = l->Hkv * ((pr->n_total + t - 1) / t + pr->n_seq);
  const int64_t nk = (static_cast<int64_t>(max_len) + pr->n_max + kKeyTile - 1) / kKeyTile;
  if (nk <= kPieceTiles) return 0;
  const int64_t all = items * ((nk + kPieceTiles - 1) / kPieceTiles), cap = kMaxPieces;
  return all < cap ? all : cap;
}

template <int D>
static tv_status launch_prompt_tc(AttnPromptTcParams& p, const AttnPromptCall& a, cudaStream_t st) {
  using C = Pa<D>;
  const tv_attn_layer* l = a.layer;
  for (int s = 0; s < a.prompt->n_seq; s++) {
    if (!encode_cache_map(&p.tmK[s], l->K[s], D, l->cap, l->Hkv, kKeyTile) ||
        !encode_cache_map(&p.tmV[s], l->V[s], D, l->cap, l->Hkv, C::VROWS))
      return TV_ERR_CUDA;
    p.V[s] = static_cast<const __nv_bfloat16*>(l->V[s]);
  }
  p.T = 128 / p.G;
  if (!encode_q_map(&p.tmQ, a.q, D, l->Hq, a.prompt->n_total, p.G, p.T)) return TV_ERR_CUDA;
  p.slots = static_cast<int>(slots_for(l, a.prompt, a.max_len));
  p.workers = num_sms();
  static bool set = false;
  if (!set) {
    if (cudaFuncSetAttribute(attn_prompt_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
      return TV_ERR_CUDA;
    set = true;
  }
  launch_k(true, attn_prompt_tc_kernel<D>, dim3(p.workers), dim3(384), C::SMEM, st, p);
  // The join has work only where the plan, made on the device, split items: with
  // few of them.  With few rows too, a warp each, its time is that of one row's
  // pieces, and 24 loads in flight serve best (24 rows behind 65,536: 59.9 us, 61.1
  // with 12; 8 behind 50,000, 16 + 2 heads: 22.8 and 26.9); with more rows warps do
  // (200 behind 20,000, 32 + 4 heads: 76.6 us with 12 loads and twice the CTAs, 102.7
  // with 24).  Whole prompts have next to nothing to join and want few CTAs that
  // take the SMs of the kernel before as they come free (packed 6,659 rows without
  // a gate: 235 us and 241).
  if (p.slots > 0) {
    const int sms = num_sms();
    const int64_t rows = static_cast<int64_t>(a.prompt->n_total) * l->Hq, units = rows * (D > 128 ? D / 128 : 1);
    if (units <= 8 * sms || rows >= 4 * sms * static_cast<int64_t>(p.T) * p.G)
      launch_k(true, attn_prompt_join_kernel<D, 24>, dim3(sms), dim3(256), 0, st, p);
    else
      launch_k(true, attn_prompt_join_kernel<D, 12>, dim3(2 * sms), dim3(256), 0, st, p);
  }
  return launch_status();
}

size_t attn_prompt_tc_ws_bytes(const tv_attn_layer* l, const tv_prompt* pr, int max_len) {
  return static_cast<size_t>(slots_for(l, pr, max_len)) * 128 * (l->D + 4) * 4;
}

tv_status attn_prompt_tc_launch(const AttnPromptCall& a, cudaStream_t st) {
  const tv_attn_layer* l = a.layer;
  const size_t need = attn_prompt_tc_ws_bytes(l, a.prompt, a.max_len);
  if (need > 0 && (!a.ws || a.ws_bytes < need)) return TV_ERR_WORKSPACE;
  if (!aligned16(a.ws)) return TV_ERR_ALIGN;
  AttnPromptTcParams p;
  memset(&p, 0, sizeof(p));
  p.pr = prompt_rows(a.prompt, a.len, a.max_len, l->cap);
  p.gate = static_cast<const __nv_bfloat16*>(a.gate);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ws = static_cast<float*>(a.ws);
  p.Hq = l->Hq;
  p.Hkv = l->Hkv;
  p.G = l->Hq / l->Hkv;
  p.c = a.scale * 1.4426950408889634f;
  switch (l->D) {
    case 64: return launch_prompt_tc<64>(p, a, st);
    case 128: return launch_prompt_tc<128>(p, a, st);
    default: return launch_prompt_tc<256>(p, a, st);
  }
}

}  // namespace tv
