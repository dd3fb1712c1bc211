// The kernel for shared prefixes, as the call that launches it sees it.
#pragma once
#include <climits>
#include <cuda.h>

#include "paged.cuh"

namespace tv {

struct PagedPrefixParams {
  CUtensorMap tmK, tmV;  // pools as [rows][D], boxes of R rows, 64 columns
  PagedSeqs b;
  const int32_t* group_off;  // [n_group + 1]
  const int32_t* shared;     // [n_group]
  const __nv_bfloat16* q;
  float* rec;       // [slots][128][D + 4]: O, m and l of a piece's rows
  int4* info;       // [n_group]: first piece, row tiles, pieces along the keys, first slot
  int32_t* group_of;  // [n_seq]
  int32_t* start;     // [n_seq]: rows that the pieces cover, 0: none
  int n_group, slots, Hq, Hkv, G, R;
  int all_rows;  // of a pool
  float c;       // scale * log2(e)
};
int paged_prefix_slots(const tv_paged_layer* l, const tv_paged* b, int n_group);
bool paged_prefix_launch(const PagedPrefixParams& p, int D, cudaStream_t st);

}  // namespace tv
