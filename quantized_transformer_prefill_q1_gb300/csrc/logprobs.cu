// logprobs.cu — log probabilities of given tokens, the entropy and the top alternatives of each row
// of logits. With m = max_i x_i, S = sum_i e^(x_i - m), T = sum_i (x_i - m) e^(x_i - m):
//   logprob(t) = x_t - m - ln S,   entropy = -sum_i p_i ln p_i = ln S - T / S
// (both terms of the entropy are >= 0: nothing cancels). A logit of -inf has probability 0 and adds
// nothing to S and T; a NaN, a +inf or a row of -inf alone makes the row's results NaN.
//
// One pass over the logits: every thread keeps a running (m, S, T) of its own, rescaled when its
// maximum rises (T' = a (T + (m - m') S) with a = e^(m - m')). A row belongs to a cluster of 1, 2, 4
// or 8 CTAs (as many as fill the GPU), whose results meet in the first CTA through distributed
// shared memory: no scratch, one launch.
//
// Alternatives: the maxima of 32 groups of threads are 32 different values of the row, so the k-th
// largest of them bounds the k-th largest value from below. Only the threads whose own maximum
// reaches the bound have anything that counts (some tens as a rule). Each remembers the batch of
// 16 that held its maximum and the largest value of its other batches: as long as that one is below
// the bound, only the batch is read once more, otherwise all of the thread's values. (Reading all of
// them took 15 us of the 72 for 512 rows of 151,936: they have left L2 by then.) Those at or above the
// bound gather, by a unique key (value, then lowest index), in the warps' buffers. A warp that finds 32 keeps only what is larger than the 32nd largest
// it has, so ties and constant rows end in as few sorts as any other. What the warps kept is ranked by
// counting.
//
// Bound: HBM (4 bytes a logit) for many rows: 512 x 151,936 with 20 alternatives 60.8 us = 5.1 TB/s, 0.77
// of the measured copy rate (55.3 with the ones summed like the others, which loses an entropy near 0
// by 1e-6 of itself and more; 72 with __expf in place of the bare instruction, 79 with expf). Latency for
// few: one row 11.2 us.
#include "ptx.cuh"

namespace pf {
namespace {

constexpr int THREADS = 256;      // four CTAs an SM: 512 rows run side by side and end together
constexpr int WARPS = THREADS / 32;
constexpr int Q = 4;             // 16-byte loads a thread and batch
constexpr int MAX_CLUSTER = 8;
typedef unsigned long long Key;

// Order of the alternatives: larger logit first, lower index first among equals (-0 = +0); 0 for a
// NaN, below every number's key. Unique within a row.
__device__ __forceinline__ Key order_key(float x, int i) {
  if (x != x) return 0ull;
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<Key>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int key_index(Key k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ Key kmax(Key a, Key b) { return a > b ? a : b; }
__device__ __forceinline__ Key kmin(Key a, Key b) { return a > b ? b : a; }

// A warp's 32 keys, one a lane: sorted largest first (bitonic).
__device__ __forceinline__ Key warp_sort(Key k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const Key o = __shfl_xor_sync(0xffffffffu, k, d);
      const bool down = (lane & size) == 0 || size == 32;  // this block largest first
      k = ((lane & d) == 0) == down ? kmax(k, o) : kmin(k, o);
    }
  return k;
}
// The 32 largest of two sorted lists, sorted: element-wise maxima of one and the other reversed form a
// bitonic sequence.
__device__ __forceinline__ Key warp_merge(Key a, Key b, int lane) {
  a = kmax(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const Key o = __shfl_xor_sync(0xffffffffu, a, d);
    a = (lane & d) == 0 ? kmax(a, o) : kmin(a, o);
  }
  return a;
}
// The 32 largest of `count` <= THREADS keys (0: none) in sorted[0 .. 31], by the whole CTA: a key's rank is
// the number of larger ones (the order in which they lie does not matter).
__device__ __forceinline__ void rank_keys(const Key* keys, int count, Key* sorted) {
  Key k = 0;
  int rank = 32;
  if (threadIdx.x < count && (k = keys[threadIdx.x]) != 0) {
    rank = 0;
#pragma unroll 8
    for (int i = 0; i < count; ++i) rank += keys[i] > k;
  }
  __syncthreads();
  if (threadIdx.x < 32) sorted[threadIdx.x] = 0;
  __syncthreads();
  if (rank < 32) sorted[rank] = k;
  __syncthreads();
}

constexpr float LOG2E = 1.4426950408889634f;
// 2^x (relative error 2^-22; subnormal results flush to zero, which next to a weight of 1 is nothing).
// With the product x log2(e) before it, a weight e^d is off by about (2^-22 + |d| 2^-24) of itself.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// m the maximum, n how many values equal it, s and t the sums over the others: S = n + s. Apart from
// the ones, since a row of one likely token has S = 1 + (little), and ln S and the entropy are that little.
struct Sums {
  float m, n, s, t;
};
// Brings a to the maximum m_new >= m.
__device__ __forceinline__ void raise(Sums& a, float m_new) {
  if (a.m == m_new) return;
  const float d = a.m - m_new, w = expf(d), all = a.n + a.s;
  a.t = all > 0.f && d > -1e30f ? w * fmaf(d, all, a.t) : w * a.t;  // (0 before the first number: d = -inf)
  a.s = w * all;
  a.n = 0.f;
  a.m = m_new;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m);
  raise(b, m);
  return {m, a.n + b.n, a.s + b.s, a.t + b.t};
}
__device__ __forceinline__ Sums shfl_xor(Sums a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.n, o), __shfl_xor_sync(0xffffffffu, a.s, o),
          __shfl_xor_sync(0xffffffffu, a.t, o)};
}

__device__ __forceinline__ uint32_t map_cta(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

__global__ void __launch_bounds__(THREADS, 4)
    logprobs_kernel(const float* logits, int n, long long ld, int cs, const int* tokens, float* lp, float* ent, int top,
                    int* top_ids, float* top_lp, int* status) {
  PF_TIMELINE(TL_LOGPROBS);
  __shared__ Key lists[WARPS * 32];   // what the warps kept
  __shared__ Key sorted[32];
  __shared__ Key found[WARPS][64];
  __shared__ float maxima[THREADS];
  __shared__ float bound_s;
  __shared__ int chosen[THREADS];     // first quads to read again: one batch (from the front), all of a thread's (from the back)
  __shared__ int n_batch, n_all, n_kept;
  __shared__ Sums part[WARPS];
  __shared__ __align__(16) Sums mine;
  griddep_launch_dependents();
  griddep_wait();
  const int row = static_cast<int>(blockIdx.x) / cs, rank = static_cast<int>(blockIdx.x) % cs;
  const float* x = logits + row * ld;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The row in quads of 4 values at 16-byte boundaries: quad q holds values 4 q - lead + (0 .. 3),
  // the first and last of them maybe only in part. This CTA's quads are [q0, q1), its thread t's
  // q0 + t, q0 + t + 256, ...
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
  const int quads = static_cast<int>((static_cast<long long>(n) + lead + 3) / 4);
  const int q0 = static_cast<int>(static_cast<long long>(quads) * rank / cs), q1 = static_cast<int>(static_cast<long long>(quads) * (rank + 1) / cs);
  // (no invariant loads: the logits come from the kernel before, and such a load may move ahead of the
  // wait for it)
  auto load = [&](int q) {
    const long long i = 4ll * q - lead;
    float4 v;
    if (i >= 0 && i + 4 <= n) {
      asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(x + i));
      return v;
    }
    v.x = i >= 0 && i < n ? x[i] : -INFINITY;
    v.y = i + 1 >= 0 && i + 1 < n ? x[i + 1] : -INFINITY;
    v.z = i + 2 >= 0 && i + 2 < n ? x[i + 2] : -INFINITY;
    v.w = i + 3 >= 0 && i + 3 < n ? x[i + 3] : -INFINITY;
    return v;
  };
  auto load_batch = [&](int q, float4 (&f)[Q]) {
#pragma unroll
    for (int u = 0; u < Q; ++u)
      f[u] = q + u * THREADS < q1 ? load(q + u * THREADS) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  };
  Sums a{-INFINITY, 0.f, 0.f, 0.f};
  float other = -INFINITY;  // largest value outside the batch at best_q, which holds the maximum
  int best_q = q0 + threadIdx.x;
  float4 next[Q];
  load_batch(q0 + threadIdx.x, next);
  for (int q = q0 + threadIdx.x; q < q1; q += Q * THREADS) {
    float v[4 * Q];
#pragma unroll
    for (int u = 0; u < Q; ++u) {
      v[4 * u] = next[u].x;
      v[4 * u + 1] = next[u].y;
      v[4 * u + 2] = next[u].z;
      v[4 * u + 3] = next[u].w;
    }
    load_batch(q + Q * THREADS, next);  // in flight while this one is summed
    float bm = v[0];
#pragma unroll
    for (int e = 1; e < 4 * Q; ++e) bm = fmaxf(bm, v[e]);
    other = fmaxf(other, fminf(bm, a.m));
    if (bm > a.m) {
      best_q = q;
      raise(a, bm);
    }
    const float mm = a.m == -INFINITY ? 0.f : a.m;
    float s[2] = {0.f, 0.f}, t[2] = {0.f, 0.f};
    float all[2] = {0.f, 0.f};  // the ones too: their number is what s lacks (cheaper than counting them)
#pragma unroll
    for (int e = 0; e < 4 * Q; ++e) {
      const float d = v[e] - mm, w = ex2(d * LOG2E);
      s[e & 1] += d == 0.f ? 0.f : w;
      all[e & 1] += w;
      t[e & 1] = fmaf(fmaxf(d, -1e30f), w, t[e & 1]);  // -inf has weight 0, and 0 * -inf would be NaN
    }
    a.n += rintf((all[0] + all[1]) - (s[0] + s[1]));
    a.s += s[0] + s[1];
    a.t += t[0] + t[1];
  }
  const float best = a.m;  // the thread's maximum (-inf without a number)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = join(a, shfl_xor(a, o));
  if (lane == 0) part[warp] = a;
  if (top > 0) {
    maxima[threadIdx.x] = best;
    if (threadIdx.x == 0) n_batch = n_all = n_kept = 0;
  }
  __syncthreads();

  if (top > 0) {
    if (warp == 0) {
      float g = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) g = fmaxf(g, maxima[32 * w + lane]);
      // sorted largest first (bitonic)
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
          const float o = __shfl_xor_sync(0xffffffffu, g, d);
          const bool down = (lane & size) == 0 || size == 32;
          g = ((lane & d) == 0) == down ? fmaxf(g, o) : fminf(g, o);
        }
      if (lane == top - 1) bound_s = g;
    }
    __syncthreads();
    const float bound = bound_s;
    if (best >= bound) {
      if (other >= bound)
        chosen[THREADS - 1 - atomicAdd(&n_all, 1)] = q0 + threadIdx.x;
      else
        chosen[atomicAdd(&n_batch, 1)] = best_q;
    }
    __syncthreads();
    Key list = 0, least = 0;  // the warp's 32 largest once it has found 32, and the least of them
    int held = 0;
    bool full = false;
    auto flush = [&](int count) {  // the buffer's first `count` keys into the list
      list = warp_merge(list, warp_sort(lane < count ? found[warp][lane] : 0ull, lane), lane);
      least = __shfl_sync(0xffffffffu, list, 31);
    };
    // (the quads dealt out to all threads alike)
    const int nq = (q1 - q0 + THREADS - 1) / THREADS, in_batches = n_batch * Q, items = in_batches + n_all * nq;
    for (int base = 0; base < items; base += Q * THREADS) {
      float4 f[Q];
      int at[Q];  // quads, or -1
#pragma unroll
      for (int u = 0; u < Q; ++u) {
        const int item = base + u * THREADS + static_cast<int>(threadIdx.x);
        int q = q1;
        if (item < in_batches) {
          q = chosen[item / Q] + item % Q * THREADS;
        } else if (item < items) {
          const int j = (item - in_batches) / nq;
          q = chosen[THREADS - 1 - j] + (item - in_batches - j * nq) * THREADS;
        }
        at[u] = q < q1 ? q : -1;
        f[u] = q < q1 ? load(q) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      }
#pragma unroll 1
      for (int u = 0; u < Q; ++u) {
        const float4 w = u == 0 ? f[0] : u == 1 ? f[1] : u == 2 ? f[2] : f[3];
        const int q = u == 0 ? at[0] : u == 1 ? at[1] : u == 2 ? at[2] : at[3];
        if (!__any_sync(0xffffffffu, q >= 0 && fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)) >= bound)) continue;
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          const float v = e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w;
          const long long i = 4ll * q - lead + e;
          const Key c = q >= 0 && i >= 0 && i < n && v >= bound ? order_key(v, static_cast<int>(i)) : 0ull;
          const unsigned hit = __ballot_sync(0xffffffffu, c > least);
          if (hit == 0) continue;
          if (hit >> lane & 1) found[warp][held + __popc(hit & ((1u << lane) - 1))] = c;
          held += __popc(hit);
          __syncwarp();
          if (held >= 32) {
            flush(32);
            full = true;
            __syncwarp();
            held -= 32;
            const Key rest = lane < held ? found[warp][32 + lane] : 0ull;
            __syncwarp();
            found[warp][lane] = rest;
            __syncwarp();
          }
        }
      }
    }
    if (full && held > 0) flush(held);
    const Key mine_k = full ? list : (lane < held ? found[warp][lane] : 0ull);
    const unsigned has = __ballot_sync(0xffffffffu, mine_k != 0);
    int at = 0;
    if (lane == 0) at = atomicAdd(&n_kept, __popc(has));
    at = __shfl_sync(0xffffffffu, at, 0);
    if (mine_k != 0) lists[at + __popc(has & ((1u << lane) - 1))] = mine_k;
    __syncthreads();
    rank_keys(lists, n_kept, sorted);
  }
  if (warp == 0) {
    a = lane < WARPS ? part[lane] : Sums{-INFINITY, 0.f, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      a = join(a, shfl_xor(a, o));
    if (lane == 0) mine = a;
    __syncwarp();
  }
  if (cs > 1) cluster_sync_all();
  if (rank == 0) {
    if (cs > 1) {  // the other CTAs' results, all fetched at once
      if (threadIdx.x < cs) {
        const uint32_t at = map_cta(smem_u32(&mine), threadIdx.x);
        Sums b;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(b.m), "=f"(b.n), "=f"(b.s), "=f"(b.t) : "r"(at) : "memory");
        part[threadIdx.x] = b;
      }
      if (threadIdx.x < cs * top) {
        Key o;
        const uint32_t at = map_cta(smem_u32(sorted + threadIdx.x % top), threadIdx.x / top);
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(o) : "r"(at) : "memory");
        lists[threadIdx.x] = o;
      }
      __syncthreads();
      if (warp == 0) {
        a = part[0];
        for (int r = 1; r < cs; ++r) a = join(a, part[r]);
      }
      if (top > 0) rank_keys(lists, cs * top, sorted);
    }
    if (warp == 0) {
      const Key list = top > 0 ? sorted[lane] : 0ull;
      const float ls = logf(a.n) + log1pf(a.s / a.n);  // ln S
      if (lane == 0) {
        if (lp) {
          const int t = tokens[row];
          if (t < 0 || t >= n) {
            lp[row] = NAN;
            if (status) atomicCAS(status, 0, PF_ERR_TOKEN_OUT_OF_VOCAB);
          } else {
            lp[row] = x[t] - a.m - ls;
          }
        }
        if (ent) ent[row] = ls - a.t / (a.n + a.s);
      }
      if (lane < top) {
        const size_t at = static_cast<size_t>(row) * top + lane;
        top_ids[at] = list ? key_index(list) : -1;
        if (top_lp) top_lp[at] = list ? key_value(list) - a.m - ls : NAN;
      }
    }
  }
  __syncwarp();  // the cluster's barrier takes converged warps
  if (cs > 1) cluster_sync_all();  // the first CTA has read the others' shared memory
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, cudaStream_t stream) {
  // One CTA an SM while the rows leave SMs free (37 rows of 100,003 took 19.4 us in clusters of 8, which do
  // not all fit at once, and 12.5 in clusters of 4), each with at least two batches' worth of values.
  const int sms = device_sm_count();
  int cs = 1;
  while (cs < MAX_CLUSTER && static_cast<long long>(a.rows) * cs * 2 <= sms && a.n / (2 * cs) >= 2 * 4 * Q * THREADS) cs *= 2;
  return launch_pdl_cluster(logprobs_kernel, dim3(static_cast<unsigned>(a.rows) * cs), dim3(THREADS), 0, stream, cs, a.logits, a.n,
                            static_cast<long long>(a.ld), cs, a.tokens, a.logprobs, a.entropy, a.top, a.top_ids,
                            a.top_logprobs, a.status);
}

}  // namespace pf

PF_TIMELINE_SETTER(logprobs)
