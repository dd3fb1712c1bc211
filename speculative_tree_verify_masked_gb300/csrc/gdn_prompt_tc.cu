// The gated delta rule over a prompt's rows in blocks of 64, for bf16 layers.
//
// Within a block that starts from state S0 (rows i = 0 .. 63, D_ij the product
// of alpha over j+1 .. i, g_i = alpha_0 .. alpha_i):
//   A_ij = beta_i D_ij (k_i . k_j), j < i      T = (I + A)^-1 diag(beta)
//   R_i  = v_i - g_i S0 k_i                     C = T R      (the corrections)
//   o_i  = scale g_i S0 q_i + sum_j P_ij C_j,   P_ij = scale D_ij (q_i . k_j), j <= i
//   S    = g_63 S0 + sum_j D_63,j C_j k_j^T
// which is the recurrence exactly; rows that do not exist act as alpha = 1,
// beta = 0.  The products D_ij are formed as products, never as quotients or
// differences of logarithms, so decays of 0 and runs of tiny ones are exact.
//
// Two kernels.  The first forms T and P T of every block and value head, all
// independent.  The second walks a sequence's blocks, one CTA per (value head,
// 64 state columns dv), three chained products a block:
//   [K; Q] S0^T  ->  [T; P T] R  ->  K^T (C D_63)
// each 128 rows tall on the tcgen05 tensor cores with fp32 sums in tensor
// memory, the state in registers (a thread holds one key row, 32 columns).
//
// Precision.  k, q and v are bf16 as they come.  What is formed on the way (S,
// R, C, T) enters a product as two bf16 parts, x = hi + lo with hi = bf16(x),
// lo = bf16(x - hi), which leaves 2^-17 of each value: hi and lo stand side by
// side in the product's columns (T: in a second pass), so the state keeps fp32
// class accuracy over long prompts.  P T only reaches the bf16 output and is
// rounded once.
//
// Bound by the chain of products and tensor-memory round trips a block, not by
// bytes; the first kernel by its triangular solves.
#include <cstring>

#include "attn_shared.cuh"
#include "gdn_prompt.cuh"
#include "mma_tile.cuh"
#include "ptx.cuh"

namespace tv {

constexpr int kBlk = 64;                                // rows of a block
constexpr int kTile64 = kBlk * kBlk * 2;                // one 64 x 64 bf16 tile
constexpr int kBlkBytes = 3 * kTile64 + 2 * kBlk * 4;   // T hi, P T, T lo (swizzled images), g, D_63

struct GdnTcParams {
  CUtensorMap tmK, tmQ;
  PromptRows pr;
  float* S[TV_MAX_SEQ];
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const float* alpha;
  const float* beta;
  __nv_bfloat16* out;
  uint8_t* ws;
  int Hk, Hv, dv;
  float scale;
};

// hi and lo bf16 parts of two values, packed.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(__fsub_rn(a, bf16_lo(hi)), __fsub_rn(b, bf16_hi(hi)));
}

// Blocks of the sequences before this lane's, and of all.
__device__ __forceinline__ int block_base(const WarpSeqs& w, const PromptRows& p, int lane, int& all) {
  const int mine = lane < p.n_seq ? (w.end - w.off + kBlk - 1) / kBlk : 0;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  all = __shfl_sync(0xffffffffu, incl, 31);
  return incl - mine;
}

// ---------------------------------------------------------------------------
// first kernel: T and P T of one block, for the value heads of one key head
// ---------------------------------------------------------------------------
constexpr int kLdA = kBlk + 4;

template <int DK>
struct Prep {
  static constexpr int ROWB = DK * 2;
  static constexpr int KQ = 2 * kBlk * ROWB;               // K and Q rows, dead once G and P are formed
  static constexpr int DM = 0, AM = kBlk * kLdA * 4;       // decay table, A / T (same place)
  static constexpr int SMEM = KQ > 2 * AM ? KQ : 2 * AM;
};

template <int DK>
__global__ void __launch_bounds__(128) gdn_block_prep_kernel(const __grid_constant__ GdnTcParams p) {
  using C = Prep<DK>;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ float al_s[kBlk], be_s[kBlk];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (status_bad(p.pr.status)) return;
  const WarpSeqs w = load_seqs(p.pr, lane);
  if (w.code) {
    if (tid == 0) set_status(p.pr.status, w.code);
    return;
  }
  int all;
  const int base = block_base(w, p.pr, lane, all);
  const int blk = blockIdx.x;
  if (blk >= all) return;
  const unsigned m = __ballot_sync(0xffffffffu, lane < p.pr.n_seq && w.end > w.off && base <= blk);
  const int s = 31 - __clz(static_cast<int>(m));
  const int row0 = __shfl_sync(0xffffffffu, w.off, s) + (blk - __shfl_sync(0xffffffffu, base, s)) * kBlk;
  const int nv = min(kBlk, __shfl_sync(0xffffffffu, w.end, s) - row0);
  const int g = blockIdx.y;
  const uint32_t ks = smem_u32(sm), qs = ks + kBlk * C::ROWB;
  for (int e = tid; e < kBlk * (DK / 8); e += 128) {
    const int r = e / (DK / 8), c = e % (DK / 8);
    const bool ok = r < nv;
    const size_t src = (static_cast<size_t>(row0 + (ok ? r : 0)) * p.Hk + g) * DK + c * 8;
    cp_async16(ks + swz(r, c, C::ROWB), p.k + src, ok);
    cp_async16(qs + swz(r, c, C::ROWB), p.q + src, ok);
  }
  cp_async_commit();
  cp_async_wait_group<0>();
  __syncthreads();
  // G = K K^T and Q K^T: warp w forms rows 16w .. 16w+15, columns up to its own rows
  float G[8][4], Pq[8][4];
#pragma unroll
  for (int t = 0; t < 8; t++)
#pragma unroll
    for (int e = 0; e < 4; e++) G[t][e] = Pq[t][e] = 0.f;
  const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
  for (int kt = 0; kt < DK / 16; kt++) {
    uint32_t ak[4], aq[4];
    const int ar = 16 * warp + (mi & 1) * 8 + mr, ac = kt * 2 + (mi >> 1);
    ldsm_x4(ks + swz(ar, ac, C::ROWB), ak);
    ldsm_x4(qs + swz(ar, ac, C::ROWB), aq);
#pragma unroll
    for (int n2 = 0; n2 < 4; n2++) {
      if (n2 <= warp) {
        uint32_t b[4];
        ldsm_x4(ks + swz(16 * n2 + (mi >> 1) * 8 + mr, kt * 2 + (mi & 1), C::ROWB), b);
        mma16816(G[2 * n2], ak, b[0], b[1]);
        mma16816(G[2 * n2 + 1], ak, b[2], b[3]);
        mma16816(Pq[2 * n2], aq, b[0], b[1]);
        mma16816(Pq[2 * n2 + 1], aq, b[2], b[3]);
      }
    }
  }
  __syncthreads();  // the rows are dead: the tables take their place
  float* Dm = reinterpret_cast<float*>(sm + C::DM);
  float* Am = reinterpret_cast<float*>(sm + C::AM);
  const int fr = 16 * warp + (lane >> 2), fc = 2 * (lane & 3);  // fragment row (and +8), column in a tile
  const int r = p.Hv / p.Hk;
  for (int hh = 0; hh < r; hh++) {
    const int h = g * r + hh;
    uint8_t* dst = p.ws + (static_cast<size_t>(blk) * p.Hv + h) * kBlkBytes;
    if (tid < kBlk) {
      const size_t gi = static_cast<size_t>(row0 + tid) * p.Hv + h;
      al_s[tid] = tid < nv ? p.alpha[gi] : 1.f;
      be_s[tid] = tid < nv ? p.beta[gi] : 0.f;
    }
    __syncthreads();
    if (tid < kBlk) {
      // column tid of the decay table, and g
      float d = 1.f, gp = 1.f;
      for (int i = 0; i < kBlk; i++) {
        const float a = al_s[i];
        if (i > tid) d = __fmul_rn(d, a);
        if (i <= tid) gp = __fmul_rn(gp, a);
        Dm[i * kLdA + tid] = i >= tid ? d : 0.f;
      }
      reinterpret_cast<float*>(dst + 3 * kTile64)[tid] = gp;
      reinterpret_cast<float*>(dst + 3 * kTile64)[kBlk + tid] = d;
    }
    __syncthreads();
    // A (zeros on and above the diagonal), and this warp's rows of P
    float Pd[8][4];
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int i = fr + (e >> 1) * 8, j = 8 * t + fc + (e & 1);
        const float d = Dm[i * kLdA + j];
        Am[i * kLdA + j] = j < i ? __fmul_rn(be_s[i], __fmul_rn(d, G[t][e])) : 0.f;
        Pd[t][e] = j <= i ? __fmul_rn(p.scale, __fmul_rn(d, Pq[t][e])) : 0.f;
      }
    __syncthreads();
    // column c of (I + A)^-1 by substitution, two threads a column: thread
    // `par` sums over the groups of four rows j with (j / 4) % 2 == par
    const int c = tid >> 1, par = tid & 1;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; i++) x[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kBlk; i++) {
      float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
      for (int gp = 0; gp < (i + 7) / 8; gp++) {
        const float4 a = *reinterpret_cast<const float4*>(Am + i * kLdA + 8 * gp + 4 * par);
        a0 = __fmaf_rn(a.x, x[4 * gp], a0);
        a1 = __fmaf_rn(a.y, x[4 * gp + 1], a1);
        a2 = __fmaf_rn(a.z, x[4 * gp + 2], a2);
        a3 = __fmaf_rn(a.w, x[4 * gp + 3], a3);
      }
      float sum = __fadd_rn(__fadd_rn(a0, a1), __fadd_rn(a2, a3));
      sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 1));
      const float xi = i == c ? 1.f : -sum;
      if (((i >> 2) & 1) == par) x[(i >> 3) * 4 + (i & 3)] = xi;
    }
    __syncthreads();
    {
      const float b = be_s[c];
#pragma unroll
      for (int e = 0; e < 32; e++) Am[((e >> 2) * 8 + par * 4 + (e & 3)) * kLdA + c] = __fmul_rn(x[e], b);
    }
    __syncthreads();
    // T as two bf16 parts, in the swizzled image the second kernel copies
    {
      const int row = tid >> 1, c0 = (tid & 1) * 32;
#pragma unroll
      for (int q4 = 0; q4 < 4; q4++) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float2 t2 = *reinterpret_cast<const float2*>(Am + row * kLdA + c0 + q4 * 8 + 2 * e);
          split2(t2.x, t2.y, hi[e], lo[e]);
        }
        const int at = row * 128 + (((c0 / 8 + q4) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(dst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + 2 * kTile64 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    // P T by warp tiles, both split in two: P hi T hi + P hi T lo + P lo T hi
    float O[8][4];
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int e = 0; e < 4; e++) O[t][e] = 0.f;
#pragma unroll
    for (int kt = 0; kt < 4; kt++) {
      if (kt > warp) continue;  // P is zero right of its rows
      uint32_t ph[4], pl[4];
      split2(Pd[2 * kt][0], Pd[2 * kt][1], ph[0], pl[0]);
      split2(Pd[2 * kt][2], Pd[2 * kt][3], ph[1], pl[1]);
      split2(Pd[2 * kt + 1][0], Pd[2 * kt + 1][1], ph[2], pl[2]);
      split2(Pd[2 * kt + 1][2], Pd[2 * kt + 1][3], ph[3], pl[3]);
#pragma unroll
      for (int t = 0; t < 8; t++) {
        if (t > 2 * kt + 1) continue;  // T is zero right of its rows
        const float* tb = Am + (16 * kt + fc) * kLdA + 8 * t + (lane >> 2);
        uint32_t h0, l0, h1, l1;
        split2(tb[0], tb[kLdA], h0, l0);
        split2(tb[8 * kLdA], tb[9 * kLdA], h1, l1);
        mma16816(O[t], ph, h0, h1);
        mma16816(O[t], ph, l0, l1);
        mma16816(O[t], pl, h0, h1);
      }
    }
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int row = fr + e * 8;
        *reinterpret_cast<uint32_t*>(dst + kTile64 + row * 128 + ((t ^ (row & 7)) << 4) + fc * 2) =
            pack_bf16x2(O[t][2 * e], O[t][2 * e + 1]);
      }
    __syncthreads();  // the tables are reused for the next head
  }
}

// ---------------------------------------------------------------------------
// second kernel: the blocks of a sequence in order
// ---------------------------------------------------------------------------
constexpr int kDvs = 64;  // state columns (dv) a CTA holds

template <int DK>
struct Walk {
  static constexpr int KQ = 2 * kBlk * DK * 2;          // [box of 64 columns][K rows, Q rows]
  static constexpr int KQBOX = 2 * kBlk * 128;          // K and Q rows of one 64-column box
  static constexpr int TIMG = 3 * kTile64;
  static constexpr int STAGE = KQ + TIMG + kTile64;     // T lo is followed by zeros
  static constexpr int B1 = 2 * DK * 128, B2 = 2 * kBlk * 128, B3 = B2;  // [hi | lo] rows of 64 columns each
  static constexpr int BOFF = 2 * STAGE + B1 + B2 + B3;
  static constexpr int NBAR = 2 + 2 + 6 + 1;
  static constexpr int SMEM = BOFF + NBAR * 8 + 16;
  static constexpr int COLS = 512;
  static constexpr int T_D1 = 0, T_D2 = 128, T_D3 = 256;
  static constexpr uint32_t IDESC = idesc_bf16_f32(128, 2 * kDvs, false, true);
  static constexpr uint32_t IDESC_KT = idesc_bf16_f32(128, 2 * kDvs, true, true);
  static_assert(SMEM <= 232448, "shared memory");
};

// 32 values as hi and lo parts into row r of a [rows][128 bytes] hi tile and
// the lo tile `lo_off` behind it (16-byte chunks swizzled), column half wg.
__device__ __forceinline__ void store_split(uint32_t tile, uint32_t lo_off, int r, int wg, const float (&x)[32]) {
#pragma unroll
  for (int q = 0; q < 4; q++) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; e++) split2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1], hi[e], lo[e]);
    const uint32_t a = tile + r * 128 + (((wg * 4 + q) ^ (r & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a + lo_off), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                 : "memory");
  }
}
// The hi and lo halves of a product's 32 columns of this thread's row, added.
__device__ __forceinline__ void load_sum(uint32_t taddr, float (&x)[32]) {
  uint32_t a[32], b[32];
  tmem_ld32(taddr, a);
  tmem_ld32(taddr + kDvs, b);
#pragma unroll
  for (int i = 0; i < 32; i++) x[i] = __fadd_rn(__uint_as_float(a[i]), __uint_as_float(b[i]));
}

template <int DK>
__global__ void __launch_bounds__(320, 1) gdn_block_walk_kernel(const __grid_constant__ GdnTcParams p) {
  using C = Walk<DK>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const uint32_t b1 = sb + 2 * C::STAGE, b2 = b1 + C::B1, b3 = b2 + C::B2;
  const uint32_t bars = sb + C::BOFF;
  const uint32_t FULL0 = bars, EMPTY0 = bars + 16u, B1R = bars + 32u, D1F = bars + 40u, B2R = bars + 48u,
                 D2F = bars + 56u, B3R = bars + 64u, D3F = bars + 72u, DRAIN = bars + 80u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::BOFF + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* skip = reinterpret_cast<int*>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WarpSeqs w = load_seqs(p.pr, lane);
  int all;
  const int base = block_base(w, p.pr, lane, all);
  // sequences in order of falling length along the grid: the long ones start first
  const int per = p.Hv * (p.dv / kDvs);
  const int place = blockIdx.x / per, rem = blockIdx.x % per;
  const int n_l = lane < p.pr.n_seq ? w.end - w.off : -1;
  int pos = 0;
  for (int i = 0; i < p.pr.n_seq; i++) {
    const int o = __shfl_sync(0xffffffffu, n_l, i);
    if (o > n_l || (o == n_l && i < lane)) pos++;
  }
  const int s = __ffs(__ballot_sync(0xffffffffu, lane < p.pr.n_seq && pos == place)) - 1;
  const int h = rem / (p.dv / kDvs), dv0 = rem % (p.dv / kDvs) * kDvs, g = h / (p.Hv / p.Hk);
  if (threadIdx.x == 0) {
    *skip = status_bad(p.pr.status) || w.code || (sb & 1023u) ? 1 : 0;
    if (sb & 1023u) set_status(p.pr.status, TV_ERR_CUDA);
    for (int i = 0; i < 2; i++) {
      mbar_init(FULL0 + 8u * i, 1);
      mbar_init(EMPTY0 + 8u * i, 1);
    }
    mbar_init(B1R, 8);
    mbar_init(D1F, 1);
    mbar_init(B2R, 4);
    mbar_init(D2F, 1);
    mbar_init(B3R, 4);
    mbar_init(D3F, 1);
    mbar_init(DRAIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const int off = __shfl_sync(0xffffffffu, w.off, s), n = __shfl_sync(0xffffffffu, w.end, s) - off;
  const int blk0 = __shfl_sync(0xffffffffu, base, s);
  if (*skip || n <= 0) return;
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const int nb = (n + kBlk - 1) / kBlk;
  const size_t ws_step = static_cast<size_t>(p.Hv) * kBlkBytes;
  const uint8_t* ws0 = p.ws + (static_cast<size_t>(blk0) * p.Hv + h) * kBlkBytes;

  if (warp == 9) {
    // ---------------- producer ----------------
    if (lane == 0) {
      int c = 0;
      for (; c < nb; c++) {
        const int st = c & 1;
        if (!wait_role(EMPTY0 + 8u * st, ((c >> 1) & 1) ^ 1, abort_flag, kWaitCycles)) break;
        const uint32_t full = FULL0 + 8u * st, dst = sb + st * C::STAGE;
        mbar_arrive_expect_tx(full, C::KQ + C::TIMG);
#pragma unroll
        for (int kb = 0; kb < DK / 64; kb++) {
          tma_load_2d(dst + kb * C::KQBOX, &p.tmK, full, g * DK + kb * 64, off + c * kBlk);
          tma_load_2d(dst + kb * C::KQBOX + kBlk * 128, &p.tmQ, full, g * DK + kb * 64, off + c * kBlk);
        }
        bulk_g2s(dst + C::KQ, ws0 + c * ws_step, C::TIMG, full);
      }
      if (c < nb) {
        set_status(p.pr.status, TV_ERR_TIMEOUT);
        for (int i = c > 2 ? c - 2 : 0; i < c; i++) mbar_wait(FULL0 + 8u * (i & 1), (i >> 1) & 1, kWaitCycles);
      }
    }
  } else if (warp == 8) {
    // ---------------- MMA issuer ----------------
    bool ok = true;
    for (int c = 0; c < nb && ok; c++) {
      const int st = c & 1;
      const uint32_t kq = sb + st * C::STAGE, ti = kq + C::KQ;
      ok = wait_warp(FULL0 + 8u * st, (c >> 1) & 1, abort_flag, kWaitCycles) &&
           wait_warp(B1R, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      if (elect_one_sync()) {
        const uint64_t a0 = sdesc_sw128(kq, 16, 1024), d0 = sdesc_sw128(b1, DK * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < DK / 16; kk++)
          tc_mma_ss(tbase + C::T_D1, a0 + static_cast<uint64_t>(((kk >> 2) * C::KQBOX + (kk & 3) * 32) >> 4),
                    d0 + static_cast<uint64_t>((kk * 2048) >> 4), C::IDESC, kk > 0 ? 1u : 0u);
        tc_commit(D1F);
      }
      __syncwarp();
      ok = wait_warp(B2R, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      if (elect_one_sync()) {
        const uint64_t a0 = sdesc_sw128(ti, 16, 1024), d0 = sdesc_sw128(b2, kBlk * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; kk++)  // [T hi; P T], then [T lo; 0]
          tc_mma_ss(tbase + C::T_D2, a0 + static_cast<uint64_t>(((kk >> 2) * 2 * kTile64 + (kk & 3) * 32) >> 4),
                    d0 + static_cast<uint64_t>(((kk & 3) * 2048) >> 4), C::IDESC, kk > 0 ? 1u : 0u);
        tc_commit(D2F);
      }
      __syncwarp();
      ok = wait_warp(B3R, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      if (elect_one_sync()) {
        // K^T: 64-wide boxes of key columns; for DK = 64 the second box (rows
        // 64 .. 127 of the product, never read) is the Q rows behind
        const uint64_t a0 = sdesc_sw128(kq, DK == 128 ? C::KQBOX : kBlk * 128, 1024),
                       d0 = sdesc_sw128(b3, kBlk * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; kk++)
          tc_mma_ss(tbase + C::T_D3, a0 + static_cast<uint64_t>((kk * 2048) >> 4),
                    d0 + static_cast<uint64_t>((kk * 2048) >> 4), C::IDESC_KT, kk > 0 ? 1u : 0u);
        tc_commit(D3F);
        tc_commit(EMPTY0 + 8u * st);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) set_status(p.pr.status, TV_ERR_TIMEOUT);
    if (elect_one_sync()) tc_commit(DRAIN);
    __syncwarp();
    mbar_wait(DRAIN, 0, kWaitCycles);
  } else {
    // ---------------- state, splits and outputs: 8 warps ----------------
    // warps 0-3 hold columns dv0 .. +31, warps 4-7 the next 32; a thread's
    // tensor-memory lane i is key row i of the state, row i of [K; Q] and of [T; P T]
    const int wg = warp >> 2, i = (warp & 3) * 32 + lane;
    const bool krow = (warp & 3) < 2;  // lanes 0 .. 63: corrections; 64 .. 127: outputs
    const int ri = krow ? i : i - kBlk;
    const uint32_t tl = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * 32;
    float* Sg = p.S[s] + (static_cast<size_t>(h) * p.dv + dv0 + wg * 32) * DK + i;
    float S[32];
#pragma unroll
    for (int e = 0; e < 32; e++) S[e] = (DK == 128 || krow) ? Sg[static_cast<size_t>(e) * DK] : 0.f;
    auto arrive = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // what block c needs from memory besides the copies: this row's value, g and D_63
    uint4 vq[4];
    float gi, dl, gl;
    auto fetch = [&](int c) {
      const float* gd = reinterpret_cast<const float*>(ws0 + c * ws_step + 3 * kTile64);
      gi = gd[ri];
      dl = gd[kBlk + ri];
      gl = gd[kBlk - 1];
      const bool live = krow && c * kBlk + ri < n;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.v + ((static_cast<size_t>(off) + c * kBlk + (live ? ri : 0)) * p.Hv + h) * p.dv + dv0 + wg * 32);
#pragma unroll
      for (int e = 0; e < 4; e++) vq[e] = live ? src[e] : make_uint4(0u, 0u, 0u, 0u);
    };
    bool ok = true;
    // the state's two parts for the first product of block c, whose rows
    // behind the sequence's end (another sequence's, or anything) are zeroed:
    // a zero correction would still meet them in the last product
    auto offer = [&](int c) {
      if (DK == 128 || krow) store_split(b1, DK * 128, i, wg, S);
      const int live = n - c * kBlk;
      if (live < kBlk) {
        ok = wait_warp(FULL0 + 8u * (c & 1), (c >> 1) & 1, abort_flag, kWaitCycles);
        if (!ok) return;
        const uint32_t kq = sb + (c & 1) * C::STAGE;
        for (int e = threadIdx.x; e < (kBlk - live) * (DK / 8); e += 256) {
          const int r = live + e / (DK / 8), ch = e % (DK / 8);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(kq + (ch >> 3) * C::KQBOX + r * 128 + (ch & 7) * 16), "r"(0)
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(B1R);
    };
    for (int e = threadIdx.x; e < 2 * (kTile64 / 16); e += 256)  // the zeros under T lo
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(sb + (e / (kTile64 / 16)) * C::STAGE + C::KQ + C::TIMG +
                                                                      (e % (kTile64 / 16)) * 16), "r"(0)
                   : "memory");
    offer(0);
    fetch(0);
    for (int c = 0; c < nb && ok; c++) {
      float x[32];
      ok = wait_warp(D1F, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      load_sum(tl + C::T_D1, x);
      const float gc = gl, gr = gi, dr = dl;
      if (krow) {
        float v[8], r[32];
#pragma unroll
        for (int q = 0; q < 4; q++) {
          widen8(vq[q], v);
#pragma unroll
          for (int e = 0; e < 8; e++) r[8 * q + e] = c * kBlk + ri < n ? __fmaf_rn(-gr, x[8 * q + e], v[e]) : 0.f;
        }
        store_split(b2, kBlk * 128, ri, wg, r);
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(B2R);
      }
      if (c + 1 < nb) fetch(c + 1);
      ok = wait_warp(D2F, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      float z[32];
      load_sum(tl + C::T_D2, z);
      if (krow) {
#pragma unroll
        for (int e = 0; e < 32; e++) z[e] = __fmul_rn(z[e], dr);
        store_split(b3, kBlk * 128, ri, wg, z);
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(B3R);
      } else if (c * kBlk + ri < n) {
        const float f = __fmul_rn(p.scale, gr);
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; e++)
          o[e] = pack_bf16x2(__fmaf_rn(f, x[2 * e], z[2 * e]), __fmaf_rn(f, x[2 * e + 1], z[2 * e + 1]));
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((static_cast<size_t>(off) + c * kBlk + ri) * p.Hv + h) * p.dv + dv0 + wg * 32);
#pragma unroll
        for (int e = 0; e < 4; e++) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
      ok = wait_warp(D3F, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      load_sum(tl + C::T_D3, x);
#pragma unroll
      for (int e = 0; e < 32; e++) S[e] = __fmaf_rn(gc, S[e], x[e]);
      if (c + 1 < nb) offer(c + 1);
    }
    if (ok && (DK == 128 || krow)) {
#pragma unroll
      for (int e = 0; e < 32; e++) Sg[static_cast<size_t>(e) * DK] = S[e];
    }
    if (!ok && lane == 0) set_status(p.pr.status, TV_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tbase, C::COLS);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static int64_t blocks_bound(const tv_prompt* pr) { return pr->n_total / kBlk + pr->n_seq; }

// Blocks pay from about one block of rows on: below that the row-by-row
// kernel ends sooner.
bool gdn_prompt_tc_fits(const tv_gdn_layer* l, const tv_prompt* pr) {
  return l->dtype == TV_BF16 && l->dv % kDvs == 0 && pr->n_max >= kBlocksFrom;
}

size_t gdn_prompt_tc_ws_bytes(const tv_gdn_layer* l, const tv_prompt* pr) {
  return static_cast<size_t>(blocks_bound(pr)) * l->Hv * kBlkBytes;
}

template <int DK>
static tv_status launch_tc(const GdnTcParams& p, int64_t blocks, cudaStream_t st) {
  static bool set = false;
  if (!set) {
    if (cudaFuncSetAttribute(gdn_block_walk_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, Walk<DK>::SMEM) != cudaSuccess)
      return TV_ERR_CUDA;
    set = true;
  }
  gdn_block_prep_kernel<DK><<<dim3(static_cast<unsigned>(blocks), p.Hk), 128, Prep<DK>::SMEM, st>>>(p);
  gdn_block_walk_kernel<DK><<<dim3(p.pr.n_seq * p.Hv * (p.dv / kDvs)), 320, Walk<DK>::SMEM, st>>>(p);
  return launch_status();
}

tv_status gdn_prompt_tc_launch(const tv_gdn_layer* l, const GdnPromptParams& a, void* ws, size_t ws_bytes, const tv_prompt* pr,
                               cudaStream_t st) {
  if (!ws || ws_bytes < gdn_prompt_tc_ws_bytes(l, pr)) return TV_ERR_WORKSPACE;
  if (!aligned16(ws)) return TV_ERR_ALIGN;
  GdnTcParams p;
  memset(&p, 0, sizeof(p));
  auto fn = encode_fn();
  if (!fn) return TV_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(l->Hk) * l->dk, static_cast<cuuint64_t>(pr->n_total)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(l->Hk) * l->dk * 2};
  const cuuint32_t box[2] = {64, kBlk}, estr[2] = {1, 1};
  for (int i = 0; i < 2; i++)
    if (fn(i ? &p.tmQ : &p.tmK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(i ? a.q : a.k), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return TV_ERR_CUDA;
  p.pr = a.pr;
  for (int s = 0; s < pr->n_seq; s++) p.S[s] = a.S[s];
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.alpha = a.alpha;
  p.beta = a.beta;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ws = static_cast<uint8_t*>(ws);
  p.Hk = a.Hk;
  p.Hv = a.Hv;
  p.dv = a.dv;
  p.scale = a.scale;
  return l->dk == 128 ? launch_tc<128>(p, blocks_bound(pr), st) : launch_tc<64>(p, blocks_bound(pr), st);
}

}  // namespace tv
