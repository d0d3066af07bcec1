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

// ------------------------------------------------------------------ work of a batch cut into even ranges
// The attention kernels lay the work of all sequences in one line: sequence b has `tasks` tasks (a kv head, or a kv
// head and a block of rows) of `units` key units each, one after the other. CTA c of C takes units [W c / C, W (c + 1) / C),
// however the lengths lie; a task that a border cuts has one part per CTA.
struct SeqWork {
  int tasks, units;
};

// First unit of sequence b0 that unit `at` lies in, and W, from a scan over all sequences (all threads of the CTA;
// `work` gives a sequence's SeqWork). `prefix` (may be NULL): receives the first unit of every sequence.
struct WorkStart {
  long long total, first;  // W; first unit of sequence b
  int b;
};
template <int THREADS, typename Work, typename At>
__device__ __forceinline__ WorkStart batch_scan(const BatchDev& B, Work work, At at, long long* prefix, int* status) {
  constexpr int NW = THREADS / 32, PER = (PF_MAX_SEQS + THREADS - 1) / THREADS;
  __shared__ long long warp_sum[NW];
  __shared__ long long first_s;
  __shared__ int b_s;
  const int per = (B.n_seq + THREADS - 1) / THREADS, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b0 = threadIdx.x * per;
  long long mine[PER], sum = 0;
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    mine[x] = 0;
    if (x < per && b0 + x < B.n_seq) {
      const SeqRows s = batch_seq(B, b0 + x, true);
      if (s.err != PF_OK && blockIdx.x == 0) batch_record(status, s.err);
      const SeqWork w = work(s);
      mine[x] = static_cast<long long>(w.tasks) * w.units;
    }
    sum += mine[x];
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  long long before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const long long unit = at(total);
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    if (x < per && b0 + x < B.n_seq) {
      if (prefix != nullptr) prefix[b0 + x] = before;
      if (unit >= before && unit < before + mine[x]) {
        first_s = before;
        b_s = b0 + x;
      }
      before += mine[x];
    }
  }
  __syncthreads();
  return {total, first_s, b_s};
}

// A place in that line, walked forward.
template <typename Work>
struct WorkCursor {
  int b, task, u;
  SeqRows s;
  SeqWork w;
  __device__ __forceinline__ void seek(const BatchDev& B, Work work, int b_, long long off) {
    b = b_;
    s = batch_seq(B, b, true);
    w = work(s);
    task = static_cast<int>(off / w.units);
    u = static_cast<int>(off - static_cast<long long>(task) * w.units);
  }
  // d units on; the caller knows that the line reaches that far
  __device__ __forceinline__ void advance(const BatchDev& B, Work work, int d) {
    u += d;
    while (u >= w.units) {
      u -= w.units;
      if (++task == w.tasks) {
        task = 0;
        do {
          if (++b >= B.n_seq) {  // past the end: only after the last unit
            b = B.n_seq - 1;
            w = {1, 0x7fffffff};
            return;
          }
          s = batch_seq(B, b, true);
          w = work(s);
        } while (w.units == 0);
      }
    }
  }
};

__device__ __forceinline__ long long range_begin(long long total, int c, int ctas) { return total * c / ctas; }
// The CTA whose range holds `unit`.
__device__ __forceinline__ int range_owner(long long total, long long unit, int ctas) {
  return static_cast<int>(((unit + 1) * ctas - 1) / total);
}
// Parts of a cut task lie in scratch by CTA: a task that began before the CTA's range in its place 0, one that begins in it in place 1.
__device__ __forceinline__ int part_place(long long total, int c, int ctas, long long task_first) {
  return 2 * c + (task_first > range_begin(total, c, ctas) ? 1 : 0);
}

}  // namespace pf
