// batch.cuh — what the kernels over many sequences share (pf_batch in pf.h): a sequence's rows and
// start, the slot of a position, a node's parent. Every number comes from device memory and is checked
// here; none that is out of range is followed.
#pragma once
#include "ptx.cuh"

namespace pf {

__device__ __forceinline__ void batch_record(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

struct SeqRows {
  int at;     // first row in the row arrays
  int n;      // rows (0: none, or the sequence is left out)
  int start;  // positions in the cache before them
  int err;    // pf_status to record, PF_OK
};

// Rows of sequence b (its start is read where `cached`).
__device__ __forceinline__ SeqRows batch_seq(const BatchDev& B, int b, bool cached) {
  SeqRows s;
  s.at = B.row_begin[b];
  const int end = B.row_begin[b + 1];
  s.start = cached ? B.start[b] : 0;
  s.err = PF_OK;
  if (s.at < 0 || end < s.at || end > B.n_rows || end - s.at > B.max_rows) {
    s.n = 0;
    s.err = PF_ERR_SHAPE;
    return s;
  }
  s.n = end - s.at;
  if (cached && (s.start < 0 || s.start > B.max_seq - s.n)) {
    s.n = 0;
    s.err = PF_ERR_KV_CAPACITY;
  }
  return s;
}

// Slot of sequence b's position p (0 <= p < max_seq), or -1 when its table entry names no block.
__device__ __forceinline__ int batch_slot(const BatchDev& B, int b, int p) {
  if (B.table == nullptr) return p;
  const int k = B.table[static_cast<size_t>(b) * B.pages + p / PF_KV_BLOCK];
  return k < 0 || k >= B.pool ? -1 : k * PF_KV_BLOCK + p % PF_KV_BLOCK;
}

// The node before row i of a sequence, -1 for the cached positions; `bad` where the entry is out of range.
__device__ __forceinline__ int tree_parent(const int* parent, int i, bool& bad) {
  const int p = parent[i];
  bad = p < -1 || p >= i;
  return bad ? -1 : p;
}

}  // namespace pf
