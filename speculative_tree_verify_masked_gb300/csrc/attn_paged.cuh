// What the translation units of paged decode attention share.
#pragma once
#include "paged.cuh"

namespace tv {

// One call whose arguments have been checked.
struct PagedAttnCall {
  const tv_paged_layer* layer;
  const tv_paged* batch;
  const tv_paged_groups* groups;  // or null
  const int32_t* sel;             // [n_seq][Hkv][n_sel] and
  const int32_t* count;           // [n_seq][Hkv], or null
  int n_sel;
  const void* q;
  const void* gate;
  void* out;
  float scale;
  void* ws;
  size_t ws_bytes;
};
size_t paged_attn_ws_bytes(const tv_paged_layer* l, const tv_paged* b, const tv_paged_groups* g);
tv_status paged_attn_tc_launch(const PagedAttnCall& a, cudaStream_t st);

constexpr float kNoScore = -3.402823466e38f;  // the maximum of a row that sees keys, none with a score above -inf

// The pages that a slot's queries look at, in order: all up to the row's own,
// or the listed ones.
struct PagedView {
  PagedSeqs b;
  const int32_t* sel;    // [n_seq][Hkv][n_sel], or null
  const int32_t* count;  // [n_seq][Hkv]
  int n_sel, Hkv;

  __device__ __forceinline__ int pages(int s, int h, int L) const {
    if (L < 0) return 0;
    if (!sel) return (L >> b.shift) + 1;
    const int c = count[s * Hkv + h];
    if (c < 0 || c > n_sel) {
      set_status(b.status, TV_ERR_ROWS);
      return 0;
    }
    return c;
  }
  // Column of the table that place i of the order names, -1 where it names none.
  __device__ __forceinline__ int column(int s, int h, int i) const {
    if (!sel) return i;
    const int j = sel[(static_cast<size_t>(s) * Hkv + h) * n_sel + i];
    if (j >= 0 && j < b.cols) return j;
    set_status(b.status, TV_ERR_PAGE);
    return -1;
  }
};

}  // namespace tv
