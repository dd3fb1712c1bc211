// The kernel for shared prefixes, as the call that launches it sees it.
#pragma once
#include <climits>
#include <cuda.h>

#include "paged.cuh"

namespace tv {

struct PagedPrefixParams {
  CUtensorMap tmK, tmV;  // pools as [D / 64][rows][64], boxes of RK and RV rows, of a unit's columns where they are a whole unit's rows, else of 64
  PagedSeqs b;
  const int32_t* group_off;  // [n_group + 1]
  const int32_t* shared;     // [n_group]
  const __nv_bfloat16* q;
  float* rec;       // [slots][128][D + 4]: O, m and l of a piece's rows
  int4* info;       // [n_seq], for the join: the group's first piece, row tiles, pieces along the keys (0: nothing shared), place in it
  int n_group, slots, Hq, Hkv, G;
  int R, RK, RV;  // rows of a part: a page's, up to 64; of a box of keys and of values
  int all_rows;  // of a pool
  float c;       // scale * log2(e)
};
// What sharing has to save to pay for its launch, its start and the longer join: so many bytes of keys
// and values that members would read again (from L2, mostly).  24 + 4 heads of 256, us a call shared
// and slot by slot: 8 members of 16,384 rows (470 MB saved) 32.5 and 42.8, 4 (201 MB) 30.3 and 28.4; of 4,096 rows
// 16 members (252 MB) 26.0 and 28.6, 8 (117 MB) 24.8 and 21.0; 2 of 65,536 (268 MB) 67.2 and 67.2.  16 + 2
// heads of 128: 8 of 65,536 (470 MB) 32.8 and 67.7, 4 (201 MB) 39.9 and 38.8.  All of that in pages of 64 rows.  In
// pages of 16, whose copies bind the kernel for prefixes, the bound is low: 8 members of 16,384 39.6 and 50.1, 5 (268 MB) 37.0 and
// 35.2, 56 of 1,024 (231 MB) 32.2 and 30.1; of 32, 34.2 and 43.9, 31.2 and 31.7, 29.3 and 28.1.
constexpr int64_t kSharedBytes = 200 << 20;  // 210 MB
// Bytes of a row's keys and values in bf16.
__host__ __device__ inline int64_t kv_row_bytes(int Hkv, int D) { return static_cast<int64_t>(Hkv) * D * 4; }

// The groups of a call, checked by a whole CTA of THREADS: first slots [n + 1] into off; active members,
// their least length and first one into count, least and src [n]; into rows [n] how many
// rows a group shares (0 where that would not pay).  All in shared memory.
template <int THREADS>
struct GroupCheck {
  int *off, *count, *least, *src, *rows;
  unsigned long long* again;  // rows that members would read again

  // The group that slot s belongs to: the last that starts at or before it.
  __device__ __forceinline__ int of(int n, int s) const {
    int a = 0, z = n;
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (off[mid] <= s) a = mid;
      else z = mid;
    }
    return a;
  }
  // 0, or what is wrong (every thread gets it).
  __device__ int run(const PagedSeqs& b, const int32_t* group_off, const int32_t* shared, int n, int64_t row_bytes, int code) {
    const int tid = threadIdx.x;
    if (tid == 0) *again = 0;
    const int L0 = tid < b.n_seq ? paged_len(b, tid) : -1;  // (these loads are on their way together)
    for (int g = tid; g <= n; g += THREADS) {
      const int o = group_off[g];
      off[g] = o;
      if ((g == 0 && o != 0) || (g == n && o != b.n_seq) || (g < n && group_off[g + 1] < o)) code = TV_ERR_ROWS;
      if (g < n) {
        rows[g] = shared[g];
        count[g] = 0;
        least[g] = src[g] = INT_MAX;
      }
    }
    if (__syncthreads_or(code)) return code ? code : TV_ERR_ROWS;
    for (int s = tid; s < b.n_seq; s += THREADS) {
      const int L = s == tid ? L0 : paged_len(b, s);
      if (L < 0) continue;
      const int g = of(n, s);
      atomicAdd(&count[g], 1);
      atomicMin(&least[g], L);
      atomicMin(&src[g], s);
    }
    __syncthreads();
    for (int g = tid; g < n; g += THREADS) {
      const int x = rows[g];
      if (x < 0 || (x & ((1 << b.shift) - 1)) || (count[g] > 0 && x > least[g])) code = TV_ERR_ROWS;
      if (count[g] < 2) rows[g] = 0;
      else if (!code) atomicAdd(again, static_cast<unsigned long long>(count[g] - 1) * rows[g]);
    }
    if (__syncthreads_or(code)) return TV_ERR_ROWS;
    if (static_cast<int64_t>(*again) * row_bytes < kSharedBytes) {
      for (int g = tid; g < n; g += THREADS) rows[g] = 0;
      __syncthreads();
    }
    return 0;
  }
};

// Rows and 64-column blocks of the boxes for pages of `page` rows.
void paged_prefix_boxes(int D, int page, PagedPrefixParams& p, int& k_cols, int& v_cols);
int paged_prefix_slots(const tv_paged_layer* l, const tv_paged* b, int n_group);
bool paged_prefix_launch(const PagedPrefixParams& p, int D, cudaStream_t st);

}  // namespace tv
