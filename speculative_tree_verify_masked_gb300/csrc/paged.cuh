// Caches in pages, as the kernels and the entry points see them: row
// j * page + r of sequence s is row r of page table[s][j] of the pools
// [n_pages][Hkv][page][D].  Tables and lengths live on the device, so every
// kernel checks what it uses of them before it touches a row.
#pragma once
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "host.hpp"

namespace tv {

struct PagedSeqs {
  const int32_t* table;  // [n_seq][cols]
  const int32_t* len;    // [n_seq], -1: an idle slot
  int32_t* status;
  int n_seq, cols, max_len, n_pages;
  int shift;  // log2 of a page's rows
};

// Whether a call before has set the word.  A plain load, which L1 serves after an SM's first: what
// earlier kernels wrote is visible behind the wait for them, and read past L1 by every warp of a
// large grid the one line costs a microsecond or more (the join of cut items 4.3 us and 3.4).
__device__ __forceinline__ bool status_set(const int32_t* st) { return *st != 0; }
// Rows a slot holds before this step, -1 where it is idle or its length is not allowed.
__device__ __forceinline__ int paged_len(const PagedSeqs& b, int s) {
  const int L = b.len[s];
  if (L < -1 || L > b.max_len) {
    set_status(b.status, TV_ERR_LEN);
    return -1;
  }
  return L;
}
// The page that column j of a table row names, -1 (and the status word set) where it names none.
__device__ __forceinline__ int page_at(const PagedSeqs& b, int s, int j) {
  const int id = b.table[static_cast<size_t>(s) * b.cols + j];
  if (id >= 0 && id < b.n_pages) return id;
  set_status(b.status, TV_ERR_PAGE);
  return -1;
}

// ---------------------------------------------------------------------------
// the host's half
// ---------------------------------------------------------------------------
constexpr int kMaxPagedUnits = (1 << 16) - 1;  // (slot, KV head) pairs of one call

inline int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : 0; }

// What every paged call asks of its layer and batch.
inline tv_status paged_check(const tv_paged_layer* l, const tv_paged* b) {
  if (!l || !b || !b->table || !b->len || !b->status) return TV_ERR_ARG;
  if (l->dtype != TV_F32 && l->dtype != TV_BF16) return TV_ERR_DTYPE;
  if (l->Hq < 1 || l->Hkv < 1 || l->Hq % l->Hkv || l->Hq > 4096 || l->Hq / l->Hkv > 128 ||
      (l->D != 64 && l->D != 128 && l->D != 256) || !page_shift(l->page))
    return TV_ERR_SHAPE;
  if (b->n_seq < 1 || b->n_seq > TV_MAX_PAGED_SEQ || b->cols < 1 || b->max_len < 0 || l->n_pages < 1 ||
      static_cast<int64_t>(b->cols) * l->page <= b->max_len || static_cast<int64_t>(b->cols) * l->page > (1ll << 30) ||
      static_cast<int64_t>(l->n_pages) * l->Hkv * l->page >= (1ll << 31))
    return TV_ERR_ARG;
  if (static_cast<int64_t>(b->n_seq) * l->Hkv > kMaxPagedUnits) return TV_ERR_SHAPE;
  if (!aligned16(b->table) || !aligned16(b->len) || !aligned16(b->status) || !aligned16(l->K) || !aligned16(l->V))
    return TV_ERR_ALIGN;
  return TV_OK;
}
inline PagedSeqs paged_seqs(const tv_paged_layer* l, const tv_paged* b) {
  return PagedSeqs{b->table, b->len, b->status, b->n_seq, b->cols, b->max_len, l->n_pages, page_shift(l->page)};
}
inline tv_status paged_rows_check(const tv_paged_rows* r) {
  if (!r) return TV_OK;
  if (!r->row_off || r->n_total < 0 || r->n_total > TV_MAX_PROMPT_ROWS || r->n_max < 0 || r->n_max > r->n_total)
    return TV_ERR_ARG;
  return aligned16(r->row_off) ? TV_OK : TV_ERR_ALIGN;
}

// Lets a kernel have more than 48 KB of shared memory, once a device.
template <typename K>
inline bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// Bytes of [rows][cols] values of type dt.
inline size_t bytes_of(int64_t rows, int64_t cols, tv_dtype dt) { return static_cast<size_t>(rows * cols) * (dt == TV_BF16 ? 2 : 4); }
// Memory that a call reads or writes; null: not there.
struct Mem {
  const void* at;
  size_t bytes;
};
inline bool share_memory(const Mem& a, const Mem& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// Whether what a call writes, the status word among it, shares memory with nothing else that it writes or reads.
template <size_t W, size_t R>
inline bool apart(const int32_t* status, const Mem (&writes)[W], const Mem (&reads)[R]) {
  const Mem word{status, 4};
  for (size_t i = 0; i < W; i++) {
    if (share_memory(writes[i], word)) return false;
    for (size_t j = i + 1; j < W; j++)
      if (share_memory(writes[i], writes[j])) return false;
    for (const Mem& r : reads)
      if (share_memory(writes[i], r)) return false;
  }
  for (const Mem& r : reads)
    if (share_memory(word, r)) return false;
  return true;
}
inline Mem table_of(const tv_paged* b) { return {b->table, static_cast<size_t>(b->n_seq) * b->cols * 4}; }
inline Mem lens_of(const tv_paged* b) { return {b->len, static_cast<size_t>(b->n_seq) * 4}; }
inline Mem offsets_of(const tv_paged* b, const tv_paged_rows* r) {
  return {r ? r->row_off : nullptr, static_cast<size_t>(b->n_seq + 1) * 4};
}

}  // namespace tv
