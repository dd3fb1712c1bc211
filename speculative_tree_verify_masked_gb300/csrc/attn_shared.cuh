// Pieces the tensor-core attention kernels share: a query row's way into
// tensor memory, and the driver's tensor-map encoder.
#pragma once
#include <cudaTypedefs.h>

#include "common.cuh"
#include "ptx.cuh"

namespace tv {

// Queries of one row into TMEM (bf16 pairs, columns T_Q ..).  For D >= 128
// each half-tile thread moves its half of the row (D/4 columns from hf*D/4);
// for D = 64 the half-0 thread moves the whole row (32 columns).
template <int D>
struct QShare {
  static constexpr int N = D >= 128 ? D / 16 : D / 8;  // 16-byte pieces per thread
  static constexpr int COL0 = D >= 128 ? D / 4 : 0;    // first column of half 1
};
template <int D>
__device__ __forceinline__ void q_fetch(const __nv_bfloat16* qrow, int hf, uint4 (&qv)[QShare<D>::N]) {
  const bool act = qrow != nullptr && (D >= 128 || hf == 0);
  const uint4* q4 = act ? reinterpret_cast<const uint4*>(qrow) + hf * QShare<D>::N : nullptr;
#pragma unroll
  for (int i = 0; i < QShare<D>::N; i++) qv[i] = act ? q4[i] : make_uint4(0u, 0u, 0u, 0u);
}
template <int D>
__device__ __forceinline__ void q_store(uint32_t tq, int hf, const uint4 (&qv)[QShare<D>::N]) {
  if (D < 128 && hf != 0) return;
#pragma unroll
  for (int j = 0; j < QShare<D>::N / 8; j++) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      r[4 * i] = qv[8 * j + i].x;
      r[4 * i + 1] = qv[8 * j + i].y;
      r[4 * i + 2] = qv[8 * j + i].z;
      r[4 * i + 3] = qv[8 * j + i].w;
    }
    tmem_st32(tq + hf * QShare<D>::COL0 + 32 * j, r);
  }
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

}  // namespace tv
