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
// The attention kernels lay the work of all sequences in one line of fewer than 2^31 units: sequence b has `tasks` tasks
// (a kv head, or a kv head and a block of rows) of `units` units each, one after the other: task_lead(..) units that stand for
// what a task costs beside its keys, then its key units. CTA c takes units [begin(c), begin(c + 1)), however the lengths
// lie; a task whose keys a border cuts has one part per CTA.
struct SeqWork {
  int tasks, units;
};

// Units that a task counts beside its keys (`most` where lengths differ: alone, a sequence's tasks all cost the same).
__device__ __forceinline__ int task_lead(const BatchDev& B, int most) { return B.n_seq == 1 ? 0 : most; }

struct Line {
  int total, ctas;  // units; CTAs that have any
  int q, rem;       // the first `rem` of a run of CTAs take q + 1 units, the others q
  int parts, task;  // one sequence, no more tasks than CTAs: each task is a run of `parts` CTAs and of `task` units; else 0
  // `fill`: units that keep a CTA busy at once
  __device__ __forceinline__ void cut(int total_, int n_seq, const SeqWork& w, int grid, int fill) {
    total = total_;
    parts = 0;
    if (n_seq == 1 && w.tasks > 0 && w.tasks <= grid && total > 0) {
      task = w.units;
      parts = min(grid / w.tasks, (w.units + fill - 1) / fill);
      ctas = parts * w.tasks;
      q = task / parts;
      rem = task - q * parts;
    } else {
      ctas = min(grid, (total + fill - 1) / fill);
      q = ctas > 0 ? total / ctas : 0;
      rem = total - q * ctas;
    }
  }
  __device__ __forceinline__ int begin(int c) const {
    if (parts == 0) return c * q + min(c, rem);
    const int t = c / parts, p = c - t * parts;
    return t * task + p * q + min(p, rem);
  }
  // the CTA whose range holds `unit`
  __device__ __forceinline__ int owner(int unit) const {
    int run = 0;
    if (parts != 0) {
      const int t = unit / task;
      run = t * parts;
      unit -= t * task;
    }
    const int wide = rem * (q + 1);
    return run + (unit < wide ? unit / (q + 1) : rem + (unit - wide) / q);
  }
  // Parts of a cut task lie in scratch by CTA: a task that began before the CTA's range (or with it) in its place 0, one
  // that begins inside it in place 1 (only the task's first part may).
  __device__ __forceinline__ int place(int c, int task_first) const { return 2 * c + (task_first > begin(c) ? 1 : 0); }
};

// The line of a batch, and the first unit of the sequence b that this CTA's range begins in (all threads of the CTA;
// work(s): a sequence's SeqWork). `prefix` (may be NULL) receives the first unit of every sequence.
struct WorkStart {
  Line line;
  int first, b;
};
template <int THREADS, typename Work>
__device__ __forceinline__ WorkStart batch_scan(const BatchDev& B, Work work, int fill, int* prefix, int* status) {
  constexpr int NW = THREADS / 32, PER = (PF_MAX_SEQS + THREADS - 1) / THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x;
  WorkStart r;
  if (B.n_seq <= 32) {  // every warp by itself, a sequence a lane
    SeqWork w{0, 0};
    if (lane < B.n_seq) {
      const SeqRows s = batch_seq(B, lane, true);
      if (s.err != PF_OK && cta == 0 && warp == 0) batch_record(status, s.err);
      w = work(s);
    }
    const int mine = w.tasks * w.units;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const int total = __shfl_sync(0xffffffffu, inc, 31);
    w.tasks = __shfl_sync(0xffffffffu, w.tasks, 0);
    w.units = __shfl_sync(0xffffffffu, w.units, 0);
    r.line.cut(total, B.n_seq, w, gridDim.x, fill);
    const int before = inc - mine, unit = cta < r.line.ctas ? r.line.begin(cta) : 0;
    if (prefix != nullptr && warp == 0 && lane < B.n_seq) prefix[lane] = before;
    const unsigned here = __ballot_sync(0xffffffffu, unit >= before && unit < inc);
    r.b = here != 0 ? __ffs(here) - 1 : 0;
    r.first = __shfl_sync(0xffffffffu, before, r.b);
    return r;
  }
  __shared__ int warp_sum[NW];
  __shared__ int first_s, b_s;
  const int per = (B.n_seq + THREADS - 1) / THREADS;
  const int b0 = threadIdx.x * per;
  int mine[PER], sum = 0;
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    mine[x] = 0;
    if (x < per && b0 + x < B.n_seq) {
      const SeqRows s = batch_seq(B, b0 + x, true);
      if (s.err != PF_OK && cta == 0) batch_record(status, s.err);
      const SeqWork w = work(s);
      mine[x] = w.tasks * w.units;
    }
    sum += mine[x];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  r.line.cut(total, B.n_seq, SeqWork{0, 0}, gridDim.x, fill);
  const int unit = cta < r.line.ctas ? r.line.begin(cta) : 0;
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
  r.first = first_s;
  r.b = b_s;
  return r;
}

// A place in the line, walked forward.
template <typename Work>
struct WorkCursor {
  int b, task, u;
  SeqRows s;
  SeqWork w;
  __device__ __forceinline__ void seek(const BatchDev& B, Work work, int b_, int off) {
    b = b_;
    s = batch_seq(B, b, true);
    w = work(s);
    task = off / w.units;
    u = off - task * w.units;
  }
  // d units on; the caller knows that the line reaches that far
  __device__ __forceinline__ void advance(const BatchDev& B, Work work, int d) {
    u += d;
    while (u >= w.units) {
      u -= w.units;
      if (++task == w.tasks) {
        task = 0;
        do {
          if (++b >= B.n_seq) {  // never, as long as the caller is right
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

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ void prefetch_tmap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

}  // namespace pf
