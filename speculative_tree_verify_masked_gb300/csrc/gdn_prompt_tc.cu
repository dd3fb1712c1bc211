// The gated delta rule over a prompt's rows in blocks of 64, for bf16 layers.
//
// Within a block that starts from state S0 (rows i = 0 .. 63, D_ij the product
// of alpha over j+1 .. i, g_i = alpha_0 .. alpha_i):
//   A_ij = beta_i D_ij (k_i . k_j), j < i      T = (I + A)^-1 diag(beta)
//   R_i  = v_i - g_i S0 k_i                    (T R are the block's corrections)
//   o_i  = scale g_i S0 q_i + (P T R)_i,       P_ij = scale D_ij (q_i . k_j), j <= i
//   S    = g_63 S0 + (W R)^T,                  W = K^T diag(D_63) T   [dk x 64]
// which is the recurrence exactly; rows that do not exist act as alpha = 1,
// beta = 0.  The products D_ij are formed as products, never as quotients or
// differences of logarithms, so decays of 0 and runs of tiny ones are exact.
//
// Two kernels.  The first forms W and P T of every block and value head, all
// independent (with T applied ahead of time, the walk has two products in its
// chain instead of three: 359 us against 544 at 8,192 rows).  The second walks a
// sequence's blocks, one CTA per (value head, 64 state columns dv), as two
// halves of 32 columns that run for themselves, so that one's products run
// under the other's splits:
//   [K; Q] S0^T  ->  R  ->  W R  ->  S,   and beside the chain  P T R -> o,
// each 128 rows tall on the tcgen05 tensor cores with fp32 sums in tensor
// memory, the state in registers (a thread holds one key row, 32 columns).
//
// Precision.  k, q and v are bf16 as they come.  What is formed on the way (S,
// R, W, and T where it enters W and P T) enters a product as two bf16 parts, x =
// hi + lo with hi = bf16(x), lo = bf16(x - hi), which leaves 2^-17 of each value
// at most: in the walk hi and lo of S and R stand side by side in a product's
// columns and W's take a pass each; in the first kernel lo lo is left out.  One
// part alone would leave 2^-9, far above what a state that lives over a long
// prompt can take.  The inverse itself is formed in fp32 (diagonal blocks) and
// two tf32 parts: where keys resemble each other A is far from zero and the
// inverse's entries are what its sums leave.  From the recurrence in 64 bits the
// state is (rel-L2) 4.3e-6 after 8,192 rows with independent keys and drawn gates;
// over gates beta 0.9 .. 1, alpha 0.99 .. 1 and up to 2,000 rows 6.0e-6 with
// independent keys, 7.0e-6 at a mean cosine of 0.8, 2.1e-5 with equal keys, 2.7e-5
// with two keys in turn (heads of 64: 3.9e-5), where W's two parts add up.  P T
// only reaches the bf16 output and is rounded once.
//
// Bound by the chain of products, tensor-memory round trips and splits a block,
// not by bytes: 16 + 48 heads of 128 x 128, 8,192 rows 335 us (127 + 207; 41.5
// of bytes), about 3,000 cycles a block and CTA, the tensor pipe busy for 62 % of
// them; 2,047 + 1 + 515 + 4,096 rows 234 us (104 + 127).  The first kernel waits
// for its own steps (35 % of issue slots; registers hold it to three CTAs an SM).
#include <cstring>

#include "gdn_prompt.cuh"
#include "mma_tile.cuh"
#include "ptx.cuh"
#include "tensor_map.hpp"

namespace tv {

constexpr int kBlk = 64;                  // rows of a block
constexpr int kTile64 = kBlk * kBlk * 2;  // one 64 x 64 bf16 tile

// What the first kernel leaves of a block and value head: P T [64][64], then W
// as hi and lo [DK rows][64], swizzled as the second kernel's operands; then g (fp32).
template <int DK>
struct Image {
  static constexpr int WB = DK * 128;       // bytes of W hi (or lo)
  static constexpr int W = kTile64;         // offset of W hi
  static constexpr int G = W + 2 * WB;
  static constexpr int BYTES = G + kBlk * 4;
};

struct GdnTcParams {
  CUtensorMap tmK, tmQ, tmV;
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
  int heads;  // value heads a CTA of the first kernel takes, one after the other
  float scale;
};

// hi and lo bf16 parts of two values, packed.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(__fsub_rn(a, bf16_lo(hi)), __fsub_rn(b, bf16_hi(hi)));
}

// ---------------------------------------------------------------------------
// first kernel: W and P T of one block, for value heads of one key head
// ---------------------------------------------------------------------------
// 16 x 16 blocks by warp-level tiles.  A matrix lives as accumulators (C
// layout: row lane / 4 and +8, columns 2 (lane % 4) and +1 of two 8-wide
// tiles), which are its A operand once packed; as B operand it is read back
// from [64][64] bf16 hi and lo tiles in shared memory.
struct Op16 {
  uint32_t h[4], l[4];
};
__device__ __forceinline__ Op16 split_op(const float (&c0)[4], const float (&c1)[4]) {
  Op16 o;
  split2(c0[0], c0[1], o.h[0], o.l[0]);
  split2(c0[2], c0[3], o.h[1], o.l[1]);
  split2(c1[0], c1[1], o.h[2], o.l[2]);
  split2(c1[2], c1[3], o.h[3], o.l[3]);
  return o;
}
// B operand: block (rows r0 .., columns c0 ..) of a hi tile and the lo tile behind it
__device__ __forceinline__ Op16 load_op(uint32_t tile, int r0, int c0, int lane) {
  Op16 o;
  const int mi = lane >> 3, r = r0 + (mi & 1) * 8 + (lane & 7);
  const uint32_t a = tile + swz(r, c0 / 8 + (mi >> 1), 128);
  ldsm_x4_t(a, o.h);
  ldsm_x4_t(a + kTile64, o.l);
  return o;
}
// acc += a b, hi hi + hi lo + lo hi
__device__ __forceinline__ void mma_split(float (&c0)[4], float (&c1)[4], const Op16& a, const Op16& b) {
  mma16816(c0, a.h, b.h[0], b.h[1]);
  mma16816(c1, a.h, b.h[2], b.h[3]);
  mma16816(c0, a.h, b.l[0], b.l[1]);
  mma16816(c1, a.h, b.l[2], b.l[3]);
  mma16816(c0, a.l, b.h[0], b.h[1]);
  mma16816(c1, a.l, b.h[2], b.h[3]);
}
// Forming the inverse takes more: what is left of its sums cancels where keys
// resemble each other.  A and the inverse's diagonal blocks lie in shared memory
// as fp32 [64][64], column c of row r at c ^ 8 (r / 2 mod 4) so that a warp's
// reads below fall on distinct banks, and a product takes both operands as two
// tf32 parts (11 bits each, lo lo left out: 2^-22).
__device__ __forceinline__ uint32_t f32_at(uint32_t tile, int r, int c) {
  return tile + static_cast<uint32_t>((r * kBlk + (c ^ ((r >> 1 & 3) << 3))) * 4);
}
__device__ __forceinline__ float ld_f32(uint32_t a) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ void st_f32x2(uint32_t a, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
struct Tf32 {
  uint32_t h, l;
};
__device__ __forceinline__ Tf32 split_tf32(float x) {
  Tf32 t;
  t.h = __float_as_uint(x) & 0xffffe000u;
  t.l = __float_as_uint(__fsub_rn(x, __uint_as_float(t.h))) & 0xffffe000u;
  return t;
}
// d += a b for one 16 x 8 x 8 tile
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// acc += x B of 16 x 16 blocks: x as accumulators, B the fp32 tile's block at (r0,
// c0).  The sum runs over columns 2t, 2t+1 of x where a tile has k = t, t+4, so
// that accumulators are operands as they lie; B's rows are taken likewise.
__device__ __forceinline__ void mma_block(float (&acc)[2][4], const float (&x)[2][4], uint32_t tile, int r0, int c0, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int s = 0; s < 2; s++) {
    Tf32 a[4];
#pragma unroll
    for (int e = 0; e < 4; e++) a[e] = split_tf32(x[s][e]);
#pragma unroll
    for (int n = 0; n < 2; n++) {
      const Tf32 b0 = split_tf32(ld_f32(f32_at(tile, r0 + 8 * s + 2 * t, c0 + 8 * n + g)));
      const Tf32 b1 = split_tf32(ld_f32(f32_at(tile, r0 + 8 * s + 2 * t + 1, c0 + 8 * n + g)));
      mma1688(acc[n], a[0].h, a[2].h, a[1].h, a[3].h, b0.h, b1.h);
      mma1688(acc[n], a[0].h, a[2].h, a[1].h, a[3].h, b0.l, b1.l);
      mma1688(acc[n], a[0].l, a[2].l, a[1].l, a[3].l, b0.h, b1.h);
    }
  }
}
__device__ __forceinline__ void stsm_x4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
// hi and lo parts of a block (the lo tile `lo_off` behind)
__device__ __forceinline__ void store_op(uint32_t tile, uint32_t lo_off, int r0, int c0, int lane, const Op16& o) {
  const int mi = lane >> 3, r = r0 + (mi & 1) * 8 + (lane & 7);
  const uint32_t a = tile + swz(r, c0 / 8 + (mi >> 1), 128);
  stsm_x4(a, o.h);
  stsm_x4(a + lo_off, o.l);
}

template <int DK>
struct Prep {
  static constexpr int ROWB = DK * 2;
  static constexpr int KS = kBlk * ROWB;              // the key rows stay
  static constexpr int DX = KS, AT = DX + 2 * kTile64, XT = AT + 2 * kTile64;  // hi and lo tiles
  static constexpr int IMG = AT - kTile64;            // the image takes the place of DX lo, A and X
  static constexpr int SMEM = XT + 2 * kTile64;       // 64 KB (DK = 128): three CTAs an SM
  static_assert(IMG + Image<DK>::G <= SMEM, "image");
};

template <int DK>
__global__ void __launch_bounds__(128, 3) gdn_block_prep_kernel(const __grid_constant__ GdnTcParams p) {
  using C = Prep<DK>;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ float al_s[kBlk], be_s[kBlk], dl_s[kBlk];
  __shared__ int cut_s[2];  // first row with a gate that is not finite, in rows 0 .. 31 and 32 .. 63
  __shared__ float win[4][16][17];  // win[b][i][j]: product of alpha over rows j+1 .. i of 16-row group b
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  if (status_bad(p.pr.status)) return;
  const WarpSeqs w = load_seqs(p.pr, lane);
  if (w.code) {
    if (tid == 0) set_status(p.pr.status, w.code);
    return;
  }
  int all;
  const int base = strip_base(w, p.pr, lane, kBlk, all);
  const int blk = blockIdx.x;
  if (blk >= all) return;
  const int s = strip_seq(w, p.pr, lane, base, blk);
  const int row0 = __shfl_sync(0xffffffffu, w.off, s) + (blk - __shfl_sync(0xffffffffu, base, s)) * kBlk;
  const int nv = min(kBlk, __shfl_sync(0xffffffffu, w.end, s) - row0);
  const int h0 = blockIdx.y * p.heads, g = h0 / (p.Hv / p.Hk);  // this CTA's first value head, their key head
  const uint32_t ks = smem_u32(sm), qs = ks + C::DX;  // the query rows are dead before DX is written
  const uint32_t dx = ks + C::DX, at = ks + C::AT, xt = ks + C::XT, img = ks + C::IMG;
  for (int e = tid; e < kBlk * (DK / 8); e += 128) {
    const int r = e / (DK / 8), c = e % (DK / 8);
    const bool ok = r < nv;
    const size_t src = (static_cast<size_t>(row0 + (ok ? r : 0)) * p.Hk + g) * DK + c * 8;
    cp_async16(ks + swz(r, c, C::ROWB), p.k + src, ok);
    cp_async16(qs + swz(r, c, C::ROWB), p.q + src, ok);
  }
  cp_async_commit();
  cp_async_wait_group<0>();
  // a key that is not finite must not meet the zeros of rows before it (this
  // thread's own pieces; the walk reads the key as it is)
#pragma unroll 2
  for (int e = tid; e < kBlk * (DK / 8); e += 128) {
    const uint32_t a = ks + swz(e / (DK / 8), e % (DK / 8), C::ROWB);
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    const uint32_t x = finite2(v.x), y = finite2(v.y), z = finite2(v.z), u = finite2(v.w);
    if (~(x & y & z & u))
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x & x), "r"(v.y & y), "r"(v.z & z), "r"(v.w & u) : "memory");
  }
  __syncthreads();
  // K K^T and Q K^T: warp w forms rows 16w .. 16w+15, columns up to its own rows
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
  const int fr = lane >> 2, fc = 2 * (lane & 3);  // fragment row (and +8) and column in a 16-row group
  // a row's gates, one head ahead of their use
  const bool gate_row = tid < nv;  // (nv <= 64)
  const size_t gate0 = static_cast<size_t>(row0 + (gate_row ? tid : 0)) * p.Hv + h0;
  float al_n = gate_row ? p.alpha[gate0] : 1.f, be_n = gate_row ? p.beta[gate0] : 0.f;
  for (int hh = 0; hh < p.heads; hh++) {
    const int h = h0 + hh;
    uint8_t* dst = p.ws + (static_cast<size_t>(blk) * p.Hv + h) * Image<DK>::BYTES;
    if (tid < kBlk) {
      const bool fin = isfinite(al_n) && isfinite(be_n);
      al_s[tid] = fin ? al_n : 1.f;
      be_s[tid] = fin ? be_n : 0.f;
      const unsigned m = __ballot_sync(0xffffffffu, !fin);
      if (lane == 0) cut_s[warp] = m ? 32 * warp + __ffs(m) - 1 : kBlk;
    }
    __syncthreads();
    if (gate_row && hh + 1 < p.heads) {
      al_n = p.alpha[gate0 + hh + 1];
      be_n = p.beta[gate0 + hh + 1];
    }
    if (tid == 0 && hh > 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last image has left
    if (tid < kBlk) {
      const int b = tid >> 4, j = tid & 15;
      float d = 1.f;
#pragma unroll
      for (int i = 0; i < 16; i++) {
        if (i > j) d = __fmul_rn(d, al_s[16 * b + i]);
        win[b][i][j] = i >= j ? d : 0.f;
      }
    }
    __syncthreads();
    float grp[4];  // product of alpha over each 16-row group
#pragma unroll
    for (int b = 0; b < 4; b++) grp[b] = __fmul_rn(al_s[16 * b], win[b][15][0]);
    if (tid < kBlk) {
      const int b = tid >> 4, j = tid & 15;
      float gi = __fmul_rn(al_s[16 * b], win[b][j][0]), dl = win[b][15][j];
#pragma unroll
      for (int x = 0; x < 4; x++) {
        if (x < b) gi = __fmul_rn(gi, grp[x]);
        if (x > b) dl = __fmul_rn(dl, grp[x]);
      }
      dl_s[tid] = dl;
      // from a gate that is not finite on, nothing of the head is: the walk takes that from g
      reinterpret_cast<float*>(dst + Image<DK>::G)[tid] = tid < min(cut_s[0], cut_s[1]) ? gi : __int_as_float(0x7fc00000);
    }
    // the decays of this warp's rows against block column b, in C layout (zero
    // above the diagonal; on it 1)
    const float pre0 = __fmul_rn(al_s[16 * warp], win[warp][fr][0]), pre1 = __fmul_rn(al_s[16 * warp], win[warp][fr + 8][0]);
    auto decays = [&](int b, float (&d)[2][4]) {
      if (b < warp) {
        float mid = 1.f;  // the groups between
#pragma unroll
        for (int x = 1; x < 3; x++)
          if (x > b && x < warp) mid = __fmul_rn(mid, grp[x]);
        const float m0 = __fmul_rn(mid, pre0), m1 = __fmul_rn(mid, pre1);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const float sfx = win[b][15][8 * t + fc + e];
            d[t][e] = __fmul_rn(sfx, m0);
            d[t][e + 2] = __fmul_rn(sfx, m1);
          }
      } else {
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 4; e++) d[t][e] = win[b][fr + (e >> 1) * 8][8 * t + fc + (e & 1)];
      }
    };
    // this warp's rows of A
    const float be0 = be_s[16 * warp + fr], be1 = be_s[16 * warp + fr + 8];
#pragma unroll
    for (int b = 0; b < 4; b++) {
      if (b > warp) continue;
      float A[2][4];
      decays(b, A);
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int r = 16 * warp + fr + 8 * e, c = 16 * b + 8 * t + fc;
          const float x0 = __fmul_rn(e ? be1 : be0, __fmul_rn(A[t][2 * e], G[2 * b + t][2 * e]));
          const float x1 = __fmul_rn(e ? be1 : be0, __fmul_rn(A[t][2 * e + 1], G[2 * b + t][2 * e + 1]));
          st_f32x2(f32_at(at, r, c), x0, x1);  // (on and above the diagonal: not read)
        }
    }
    // The inverse of this warp's diagonal block by forward substitution, a column
    // a lane, into a block of A's tile above the diagonal.  (As a product of
    // powers, (I - A)(I + A^2)(I + A^4)(I + A^8), it loses what A^8 grows by: for
    // equal keys and gates of 1 its entries reach 3,432, the inverse's 1.)
    __syncwarp();
    const int ir = warp < 3 ? 0 : 16, ic = warp < 3 ? 16 * (warp + 1) : 32;  // where that block lies
    float X[4][2][4];  // this warp's row of blocks of (I + A)^-1; X[b] is block column b
    float D[2][4];
    {
      const int c = lane & 15;  // (the upper lanes do the same once more)
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; i++) {
        float r = i == c ? 1.f : 0.f;
#pragma unroll
        for (int k = 0; k < i; k += 4) {
          float a[4];
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3])
                       : "r"(f32_at(at, 16 * warp + i, 16 * warp + k))
                       : "memory");
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (k + e < i) r = __fmaf_rn(-a[e], x[k + e], r);
        }
        x[i] = r;
      }
#pragma unroll
      for (int i = 0; i < 16; i++)
        if (lane < 16) asm volatile("st.shared.f32 [%0], %1;" ::"r"(f32_at(at, ir + i, ic + c)), "f"(x[i]) : "memory");
      __syncwarp();
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) D[t][e] = ld_f32(f32_at(at, ir + fr + 8 * (e >> 1), ic + 8 * t + fc + (e & 1)));
    }
    __syncthreads();
    // the rest of the row: X_wj = -(sum over j < k <= w of X_wk A_kj) X_jj
#pragma unroll
    for (int b = 3; b >= 0; b--) {
      if (b == warp) {
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 4; e++) X[b][t][e] = D[t][e];
      } else if (b < warp) {
        float acc[2][4];
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 4; e++) acc[t][e] = X[b][t][e] = 0.f;
#pragma unroll
        for (int k = 3; k >= 1; k--)
          if (k > b && k <= warp) mma_block(acc, X[k], at, 16 * k, 16 * b, lane);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 4; e++) acc[t][e] = -acc[t][e];
        mma_block(X[b], acc, at, 0, 16 * (b + 1), lane);  // X_jj
      }
    }
    {
      const float d0 = dl_s[16 * warp + fr], d1 = dl_s[16 * warp + fr + 8];
#pragma unroll
      for (int b = 0; b < 4; b++) {
        if (b > warp) continue;
        store_op(xt, kTile64, 16 * warp, 16 * b, lane, split_op(X[b][0], X[b][1]));
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 4; e++) X[b][t][e] = __fmul_rn(X[b][t][e], (e >> 1) ? d1 : d0);
        store_op(dx, kTile64, 16 * warp, 16 * b, lane, split_op(X[b][0], X[b][1]));
      }
    }
    __syncthreads();
    // P T: this warp's rows; columns scaled by beta
    uint32_t pt[16];
    {
      float O[8][4];
#pragma unroll
      for (int t = 0; t < 8; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) O[t][e] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; k++) {
        if (k > warp) continue;
        float P[2][4];
        decays(k, P);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 4; e++) P[t][e] = __fmul_rn(p.scale, __fmul_rn(P[t][e], Pq[2 * k + t][e]));
        const Op16 po = split_op(P[0], P[1]);
#pragma unroll
        for (int b = 0; b <= k; b++) mma_split(O[2 * b], O[2 * b + 1], po, load_op(xt, 16 * k, 16 * b, lane));
      }
#pragma unroll
      for (int t = 0; t < 8; t++) {
        const float b0 = be_s[8 * t + fc], b1 = be_s[8 * t + fc + 1];
        pt[2 * t] = pack_bf16x2(__fmul_rn(O[t][0], b0), __fmul_rn(O[t][1], b1));
        pt[2 * t + 1] = pack_bf16x2(__fmul_rn(O[t][2], b0), __fmul_rn(O[t][3], b1));
      }
    }
    __syncthreads();  // A and X are dead: W takes their place
    // W = K^T (D_63 X) diag(beta), k exact in bf16: this warp's key columns,
    // 16 columns of W at a time
    constexpr int MT = DK / 64;  // groups of 16 key columns a warp
#pragma unroll
    for (int b = 0; b < 4; b++) {
      float O[MT][2][4];
#pragma unroll
      for (int t = 0; t < MT; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) O[t][0][e] = O[t][1][e] = 0.f;
#pragma unroll
      for (int k = b; k < 4; k++) {
        const Op16 x = load_op(dx, 16 * k, 16 * b, lane);
#pragma unroll
        for (int t = 0; t < MT; t++) {
          uint32_t a[4];
          ldsm_x4_t(ks + swz(16 * k + (mi >> 1) * 8 + mr, 2 * (warp * MT + t) + (mi & 1), C::ROWB), a);
          mma16816(O[t][0], a, x.h[0], x.h[1]);
          mma16816(O[t][1], a, x.h[2], x.h[3]);
          mma16816(O[t][0], a, x.l[0], x.l[1]);
          mma16816(O[t][1], a, x.l[2], x.l[3]);
        }
      }
      const float b0 = be_s[16 * b + fc], b1 = be_s[16 * b + fc + 1], b2 = be_s[16 * b + 8 + fc], b3 = be_s[16 * b + 9 + fc];
#pragma unroll
      for (int t = 0; t < MT; t++) {
#pragma unroll
        for (int e = 0; e < 4; e++) {
          O[t][0][e] = __fmul_rn(O[t][0][e], (e & 1) ? b1 : b0);
          O[t][1][e] = __fmul_rn(O[t][1][e], (e & 1) ? b3 : b2);
        }
        store_op(img + Image<DK>::W, Image<DK>::WB, 16 * (warp * MT + t), 16 * b, lane, split_op(O[t][0], O[t][1]));
      }
    }
    __syncthreads();  // DX is dead: P T takes the place of its second half
#pragma unroll
    for (int b = 0; b < 4; b++) {
      const uint32_t v[4] = {pt[4 * b], pt[4 * b + 1], pt[4 * b + 2], pt[4 * b + 3]};
      stsm_x4(img + swz(16 * warp + (mi & 1) * 8 + mr, 2 * b + (mi >> 1), 128), v);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (tid == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(img), "r"(Image<DK>::G) : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------
// second kernel: the blocks of a sequence in order
// ---------------------------------------------------------------------------
constexpr int kDvs = 64;  // state columns (dv) a CTA holds

template <int DK>
struct Walk {
  static constexpr int KQ = 2 * kBlk * DK * 2;          // [box of 64 columns][K rows, Q rows]
  static constexpr int KQBOX = 2 * kBlk * 128;          // K and Q rows of one 64-column box
  static constexpr int VOFF = KQ + Image<DK>::G;        // 64 value rows
  static constexpr int GOFF = VOFF + kBlk * kDvs * 2;   // g
  static constexpr int STAGE = GOFF + 1024;
  static constexpr int B1 = DK * 128, B2 = kBlk * 128;  // of one half: rows of [32 hi | 32 lo] columns
  static constexpr int OBUF = 2 * STAGE + 2 * (B1 + B2);  // output rows, turned around by their warps
  static constexpr int BOFF = OBUF + 4 * 2048;
  static constexpr int NBAR = 4 + 2 * 6;
  static constexpr int SMEM = BOFF + NBAR * 8 + 16 + (128 + 4) * 4;
  static constexpr int COLS = 512;
  // of one half, 256 columns: D1 twice, by block parity (its output rows are read late)
  static constexpr int T_D1 = 0, T_D2 = 128, T_D3 = 192;
  static constexpr uint32_t IDESC = idesc_bf16_f32(128, kDvs, false, true);
  static_assert(SMEM <= 232448, "shared memory");
};

// Packed pairs as bf16 pairs: the rounded pair, and hi and lo parts.
__device__ __forceinline__ uint32_t pack_f2(f2_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ void split_f2(f2_t x, uint32_t& hi, uint32_t& lo) {
  hi = pack_f2(x);
  lo = pack_f2(f2_fma(f2_dup(-1.f), f2_from_bf16x2(hi), x));  // x - hi, exact
}
// 32 values into row r (128 bytes) of a half's tile: hi parts, then lo parts
// (16-byte chunks swizzled).
__device__ __forceinline__ void store_split(uint32_t tile, int r, const f2_t (&x)[16]) {
#pragma unroll
  for (int q = 0; q < 4; q++) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; e++) split_f2(x[4 * q + e], hi[e], lo[e]);
    const uint32_t a = tile + r * 128 + ((q ^ (r & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a ^ 64u), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
  }
}
// The hi and lo parts of a product's 32 columns of this thread's row, added.
__device__ __forceinline__ void load_sum(uint32_t taddr, f2_t (&x)[16]) {
  uint32_t a[32], b[32];
  tmem_ld32_nowait(taddr, a);
  tmem_ld32_nowait(taddr + 32, b);
  tmem_ld_wait(a, b);
#pragma unroll
  for (int i = 0; i < 16; i++)
    x[i] = f2_add(f2_pack(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])),
                  f2_pack(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1])));
}

template <int DK>
__global__ void __launch_bounds__(352, 1) gdn_block_walk_kernel(const __grid_constant__ GdnTcParams p) {
  using C = Walk<DK>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const uint32_t bars = sb + C::BOFF;
  const uint32_t FULL0 = bars, EMPTY0 = bars + 16u, half0 = bars + 32u;  // then six barriers a half
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::BOFF + C::NBAR * 8);
  int* first_bad = reinterpret_cast<int*>(tmem_slot + 4);  // [block parity][64 columns], then [parity][half]: see mark()
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* skip = reinterpret_cast<int*>(tmem_slot + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // warps 0-3 and 8 serve columns 0 .. 31 of the slice, warps 4-7 and 9 the rest
  const int hf = warp < 8 ? warp >> 2 : warp & 1;
  const uint32_t hb = half0 + 48u * hf;
  const uint32_t B1R = hb, D1F = hb + 8u, B2R = hb + 16u, D2F = hb + 24u, D3F = hb + 32u, DRAIN = hb + 40u;
  const uint32_t b1 = sb + 2 * C::STAGE + hf * C::B1, b2 = sb + 2 * C::STAGE + 2 * C::B1 + hf * C::B2;
  const WarpSeqs w = load_seqs(p.pr, lane);
  int all;
  const int base = strip_base(w, p.pr, lane, kBlk, all);
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
  if (threadIdx.x < 128 + 4) first_bad[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    *skip = status_bad(p.pr.status) || w.code || (sb & 1023u) ? 1 : 0;
    if (sb & 1023u) set_status(p.pr.status, TV_ERR_CUDA);
    for (int i = 0; i < 2; i++) {
      mbar_init(FULL0 + 8u * i, 1);
      mbar_init(EMPTY0 + 8u * i, 2);
      const uint32_t x = half0 + 48u * i;
      mbar_init(x, 4);        // B1R
      mbar_init(x + 8u, 1);   // D1F
      mbar_init(x + 16u, 4);  // B2R
      mbar_init(x + 24u, 1);  // D2F
      mbar_init(x + 32u, 1);  // D3F
      mbar_init(x + 40u, 1);  // DRAIN
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const int off = __shfl_sync(0xffffffffu, w.off, s), n = __shfl_sync(0xffffffffu, w.end, s) - off;
  const int blk0 = __shfl_sync(0xffffffffu, base, s);
  // the images come from the launch before; all else was there before that began
  if (*skip || n <= 0) {
    pdl_wait();
    return;
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot + hf * 256;
  const int nb = (n + kBlk - 1) / kBlk;
  const size_t ws_step = static_cast<size_t>(p.Hv) * Image<DK>::BYTES;
  const uint8_t* ws0 = p.ws + (static_cast<size_t>(blk0) * p.Hv + h) * Image<DK>::BYTES;

  if (warp == 10) {
    // ---------------- producer ----------------
    pdl_wait();
    if (lane == 0) {
      int c = 0;
      for (; c < nb; c++) {
        const int st = c & 1;
        if (!wait_role(EMPTY0 + 8u * st, ((c >> 1) & 1) ^ 1, abort_flag, kWaitCycles)) break;
        const uint32_t full = FULL0 + 8u * st, dst = sb + st * C::STAGE;
        mbar_arrive_expect_tx(full, C::KQ + Image<DK>::BYTES + kBlk * kDvs * 2);
#pragma unroll
        for (int kb = 0; kb < DK / 64; kb++) {
          tma_load_2d(dst + kb * C::KQBOX, &p.tmK, full, g * DK + kb * 64, off + c * kBlk);
          tma_load_2d(dst + kb * C::KQBOX + kBlk * 128, &p.tmQ, full, g * DK + kb * 64, off + c * kBlk);
        }
        tma_load_2d(dst + C::VOFF, &p.tmV, full, h * p.dv + dv0, off + c * kBlk);
        bulk_g2s(dst + C::GOFF, ws0 + c * ws_step + Image<DK>::G, kBlk * 4, full);
        bulk_g2s(dst + C::KQ, ws0 + c * ws_step, Image<DK>::G, full);
      }
      if (c < nb) {
        set_status(p.pr.status, TV_ERR_TIMEOUT);
        for (int i = c > 2 ? c - 2 : 0; i < c; i++) mbar_wait(FULL0 + 8u * (i & 1), (i >> 1) & 1, kWaitCycles);
      }
    }
  } else if (warp >= 8) {
    // ---------------- MMA issuers, one a half ----------------
    bool ok = true;
    for (int c = 0; c < nb && ok; c++) {
      const int st = c & 1;
      const uint32_t kq = sb + st * C::STAGE, ti = kq + C::KQ;
      ok = wait_warp(FULL0 + 8u * st, (c >> 1) & 1, abort_flag, kWaitCycles) &&
           wait_warp(B1R, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      if (elect_one_sync()) {
        const uint64_t a0 = sdesc_sw128(kq, 16, 1024), d0 = sdesc_sw128(b1, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < DK / 16; kk++)
          tc_mma_ss(tbase + C::T_D1 + (c & 1) * 64, a0 + static_cast<uint64_t>(((kk >> 2) * C::KQBOX + (kk & 3) * 32) >> 4),
                    d0 + static_cast<uint64_t>((kk * 2048) >> 4), C::IDESC, kk > 0 ? 1u : 0u);
        tc_commit(D1F);
      }
      __syncwarp();
      ok = wait_warp(B2R, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      if (elect_one_sync()) {
        const uint64_t a0 = sdesc_sw128(ti + Image<DK>::W, 16, 1024), d0 = sdesc_sw128(b2, 16, 1024);
        // W hi, then W lo (its lo lo part is far below the rest; DK = 64: rows
        // 64 .. 127 of the product come from what lies behind and are never read)
#pragma unroll
        for (int kk = 0; kk < 8; kk++)
          tc_mma_ss(tbase + C::T_D3, a0 + static_cast<uint64_t>(((kk >> 2) * Image<DK>::WB + (kk & 3) * 32) >> 4),
                    d0 + static_cast<uint64_t>(((kk & 3) * 2048) >> 4), C::IDESC, kk > 0 ? 1u : 0u);
        tc_commit(D3F);
        // P T in rows 64 .. 127, the output rows' lanes (the rows before are never read)
        const uint64_t p0 = sdesc_sw128(ti - kTile64, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; kk++)
          tc_mma_ss(tbase + C::T_D2, p0 + static_cast<uint64_t>((kk * 32) >> 4), d0 + static_cast<uint64_t>((kk * 2048) >> 4),
                    C::IDESC, kk > 0 ? 1u : 0u);
        tc_commit(D2F);
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
    // a thread's
    // tensor-memory lane i is key row i of the state, row i of [K; Q] and of [T; P T]
    const int i = (warp & 3) * 32 + lane;
    const bool krow = (warp & 3) < 2;  // lanes 0 .. 63: corrections; 64 .. 127: outputs
    const int ri = krow ? i : i - kBlk;
    const uint32_t tl = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* Sg = p.S[s] + (static_cast<size_t>(h) * p.dv + dv0 + hf * 32) * DK + i;
    f2_t S[16];
#pragma unroll
    for (int e = 0; e < 16; e++)
      S[e] = (DK == 128 || krow) ? f2_pack(Sg[static_cast<size_t>(2 * e) * DK], Sg[static_cast<size_t>(2 * e + 1) * DK]) : 0ull;
    auto arrive = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    // Corrections that are not finite.  A zero of W or P T would carry them to
    // rows before their own, so they enter the products as zeros, and what they
    // reach is set afterwards: of their column, the outputs from their row on
    // and the state.  A column's entry holds (block + 1) * 64 + 63 - row, raised
    // by its block's rows: the first such row, if it is of this block.  By block
    // parity, since the output rows' warps may be a block behind.
    int* const col_bad = first_bad + hf * 32;
    auto bad_row = [&](int c, int col) {  // (64 and more: none)
      const int e = *reinterpret_cast<volatile int*>(col_bad + (c & 1) * 64 + col);
      return e >> 6 == c + 1 ? 63 - (e & 63) : kBlk;
    };
    auto any_bad = [&](int c) { return *reinterpret_cast<volatile int*>(first_bad + 128 + (c & 1) * 2 + hf) == c + 1; };
    auto mark = [&](int c, f2_t (&z)[16]) {
#pragma unroll
      for (int e = 0; e < 16; e++) {
        float a, b;
        f2_unpack(z[e], a, b);
        if (!isfinite(a)) atomicMax(col_bad + (c & 1) * 64 + 2 * e, (c + 1) * 64 + 63 - ri);
        if (!isfinite(b)) atomicMax(col_bad + (c & 1) * 64 + 2 * e + 1, (c + 1) * 64 + 63 - ri);
        z[e] = f2_pack(isfinite(a) ? a : 0.f, isfinite(b) ? b : 0.f);
      }
      *reinterpret_cast<volatile int*>(first_bad + 128 + (c & 1) * 2 + hf) = c + 1;
    };
    auto poison = [&](f2_t (&x)[16], int c, int row) {  // NaN in the columns whose first such row is `row` or before
#pragma unroll
      for (int e = 0; e < 16; e++) {
        float a, b;
        f2_unpack(x[e], a, b);
        x[e] = f2_pack(bad_row(c, 2 * e) <= row ? __int_as_float(0x7fc00000) : a,
                       bad_row(c, 2 * e + 1) <= row ? __int_as_float(0x7fc00000) : b);
      }
    };
    // the state's two parts for the first product of the next block
    auto offer = [&]() {
      if (DK == 128 || krow) store_split(b1, i, S);
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(B1R);
    };
    offer();
    for (int c = 0; c < nb && ok; c++) {
      const uint32_t stg = sb + (c & 1) * C::STAGE;
      const int live = n - c * kBlk;  // rows of the block that exist (64 and more: all)
      f2_t x[16], z[16];
      ok = wait_warp(FULL0 + 8u * (c & 1), (c >> 1) & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      const float* gd = reinterpret_cast<const float*>(sm + (c & 1) * C::STAGE + C::GOFF);
      const float gr = gd[ri];
      // The state decays here, so that both loads have been served before the
      // arrival below gives the stage back: an arrival does not wait for them, and
      // the products can keep them waiting.  (g, NaN from some row on if at all, is
      // so in the last row: gr's share of 0 changes nothing.)
      const f2_t g2 = f2_dup(__fmaf_rn(gr, 0.f, gd[kBlk - 1]));
#pragma unroll
      for (int e = 0; e < 16; e++) S[e] = f2_mul(g2, S[e]);
      if (krow) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(stg + C::VOFF + ri * 128 + (((hf * 4 + q) ^ (ri & 7)) << 4)));
          z[4 * q] = f2_from_bf16x2(v.x);
          z[4 * q + 1] = f2_from_bf16x2(v.y);
          z[4 * q + 2] = f2_from_bf16x2(v.z);
          z[4 * q + 3] = f2_from_bf16x2(v.w);
        }
      }
      ok = wait_warp(D1F, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      if (krow) {
        load_sum(tl + C::T_D1 + (c & 1) * 64, x);
        const f2_t ng = f2_dup(-gr);
#pragma unroll
        for (int e = 0; e < 16; e++) z[e] = f2_fma(ng, x[e], z[e]);
        if (live < kBlk && ri >= live) {  // no such row
#pragma unroll
          for (int e = 0; e < 16; e++) z[e] = 0ull;
        }
        f2_t nil[4] = {0ull, 0ull, 0ull, 0ull};  // sums of z x 0: zero, or NaN
#pragma unroll
        for (int e = 0; e < 16; e++) nil[e & 3] = f2_fma(z[e], 0ull, nil[e & 3]);
        store_split(b2, ri, z);
        if (!(f2_hsum(f2_add(f2_add(nil[0], nil[1]), f2_add(nil[2], nil[3]))) == 0.f)) {
          mark(c, z);
          store_split(b2, ri, z);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      arrive(B2R);  // (the output rows' warps: done with the stage and with the last P T R)
      ok = wait_warp(D3F, c & 1, abort_flag, kWaitCycles);
      if (!ok) break;
      tc_fence_after();
      const bool bad = any_bad(c);
      load_sum(tl + C::T_D3, z);
#pragma unroll
      for (int e = 0; e < 16; e++) S[e] = f2_add(S[e], z[e]);
      if (bad) poison(S, c, kBlk - 1);
      if (c + 1 < nb) offer();
      if (!krow) {
        ok = wait_warp(D2F, c & 1, abort_flag, kWaitCycles);
        if (!ok) break;
        tc_fence_after();
        load_sum(tl + C::T_D2, z);
        load_sum(tl + C::T_D1 + (c & 1) * 64, x);
        const f2_t f = f2_dup(__fmul_rn(p.scale, gr));
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; e++) x[e] = f2_fma(f, x[e], z[e]);
        if (bad) poison(x, c, ri);
#pragma unroll
        for (int e = 0; e < 16; e++) o[e] = pack_f2(x[e]);
        // a thread holds 64 bytes of one row: turned around so that a store
        // covers whole rows' pieces, not 16 bytes of each of 32 rows
        const uint32_t ob = sb + C::OBUF + (hf * 2 + (warp & 1)) * 2048;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; q++)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(ob + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)),
                       "r"(o[4 * q]), "r"(o[4 * q + 1]), "r"(o[4 * q + 2]), "r"(o[4 * q + 3])
                       : "memory");
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const int rr = 8 * k + (lane >> 2), q = lane & 3, orow = (ri - lane) + rr;
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(ob + rr * 64 + ((q ^ ((rr >> 1) & 3)) << 4)));
          if (orow < live)
            reinterpret_cast<uint4*>(p.out + ((static_cast<size_t>(off) + c * kBlk + orow) * p.Hv + h) * p.dv + dv0 + hf * 32)[q] = v;
        }
      }
    }
    if (ok && (DK == 128 || krow)) {
#pragma unroll
      for (int e = 0; e < 16; e++)
        f2_unpack(S[e], Sg[static_cast<size_t>(2 * e) * DK], Sg[static_cast<size_t>(2 * e + 1) * DK]);
    }
    if (!ok && lane == 0) set_status(p.pr.status, TV_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(*tmem_slot, C::COLS);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static int64_t blocks_bound(const tv_prompt* pr) { return pr->n_total / kBlk + pr->n_seq; }

bool gdn_prompt_tc_fits(const tv_gdn_layer* l, const tv_prompt* pr) {
  return l->dtype == TV_BF16 && l->dv % kDvs == 0 && pr->n_max >= kBlocksFrom;
}

size_t gdn_prompt_tc_ws_bytes(const tv_gdn_layer* l, const tv_prompt* pr) {
  return static_cast<size_t>(blocks_bound(pr)) * l->Hv * (l->dk == 128 ? Image<128>::BYTES : Image<64>::BYTES);
}

template <int DK>
static tv_status launch_tc(const GdnTcParams& p, int64_t blocks, cudaStream_t st) {
  static bool set = false;
  if (!set) {
    if (cudaFuncSetAttribute(gdn_block_walk_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, Walk<DK>::SMEM) != cudaSuccess ||
        cudaFuncSetAttribute(gdn_block_prep_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, Prep<DK>::SMEM) != cudaSuccess)
      return TV_ERR_CUDA;
    set = true;
  }
  launch_k(true, gdn_block_prep_kernel<DK>, dim3(static_cast<unsigned>(blocks), p.Hv / p.heads), dim3(128), Prep<DK>::SMEM, st, p);
  launch_k(true, gdn_block_walk_kernel<DK>, dim3(p.pr.n_seq * p.Hv * (p.dv / kDvs)), dim3(352), Walk<DK>::SMEM, st, p);
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
  auto encode = [&](CUtensorMap* m, const void* base, int64_t cols) {  // [n_total][cols] in 64 x 64 boxes
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(pr->n_total)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
    const cuuint32_t box[2] = {64, kBlk}, estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const int64_t kcols = static_cast<int64_t>(l->Hk) * l->dk, vcols = static_cast<int64_t>(l->Hv) * l->dv;
  if (!encode(&p.tmK, a.k, kcols) || !encode(&p.tmQ, a.q, kcols) || !encode(&p.tmV, a.v, vcols)) return TV_ERR_CUDA;
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
  // The value heads of a key head share its K K^T and Q K^T, but one after the
  // other they are a call's latency where a CTA for each still makes one wave:
  // 48 heads of 128, 64 rows 16.0 us (25.9), 300 rows 25.5 (33.0), 512 rows 32.8
  // (38.9); 1,024 rows, two waves, 58.4 (57.9), 1,536 rows 84.1 (76.9).
  p.heads = blocks_bound(pr) * a.Hv <= 3 * num_sms() ? 1 : a.Hv / a.Hk;
  return l->dk == 128 ? launch_tc<128>(p, blocks_bound(pr), st) : launch_tc<64>(p, blocks_bound(pr), st);
}

}  // namespace tv
