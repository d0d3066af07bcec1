// batch.cu — the cache's part of a step over many sequences: QK-norm + RoPE + KV store of their rows, and
// the acceptance of a drafted tree's path with its K and V moved up.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "batch.cuh"

namespace pf {
namespace {

// ------------------------------------------------------------------ append
// x = a head of the f32 projection. Q and K heads: x / sqrt(mean x^2 + eps) * w (optional), then pairs
// (x_i, x_{i + hd/2}) turned by the angle of position start + depth; K and V rounded to the cache's type at the
// slot of position start + i. As qk_norm_rope_kv_kernel, HD / 8 lanes hold a head, four elements of each half.
//
// A CTA takes PAIRS (row, head) pairs of one sequence. What a row needs (slot, depth in its tree) is a chain of
// dependent loads (rows -> parents -> table): one thread per row runs it while the heads' values are on their way. That chain
// bounds few rows (one token 2.1 us, a tree of 40 nodes of each of 16 sequences 6.9 us for 27 MB), memory many: four
// chunks of 300 .. 512 rows (60 MB, part of them in L2 in a replay) 9.15 us, 6.6 TB/s.
constexpr int AP_THREADS = 256;
constexpr int AP_ROWS = 20;  // most rows that a CTA's pairs lie in: 64 / 4 + 2 at hd 64 (4 heads or more), 32 / 3 + 2 at 128

template <typename T>
__device__ __forceinline__ void put4(T* dst, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void put4<__half>(__half* dst, float a, float b, float c, float d) {
  const __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}
template <>
__device__ __forceinline__ void put4<__nv_bfloat16>(__nv_bfloat16* dst, float a, float b, float c, float d) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

template <int HD, typename T, int SLOTS>
__global__ void __launch_bounds__(AP_THREADS) batch_append_kernel(const BatchDev B, const float* qkv,
                                                                  const float* __restrict__ qn, const float* __restrict__ kn,
                                                                  const float* __restrict__ rope, int nq, int nkv, int layer,
                                                                  float eps, int qk_norm, T* __restrict__ q_out,
                                                                  T* __restrict__ kc, T* __restrict__ vc, int* status) {
  PF_TIMELINE(TL_BATCH_APPEND);
  constexpr int HALF = HD / 2, LPH = HD / 8, PER = AP_THREADS / LPH, PAIRS = PER * SLOTS;
  __shared__ int row_slot[AP_ROWS], row_pos[AP_ROWS];
  griddep_launch_dependents();
  const int heads = nq + 2 * nkv;
  const int group = threadIdx.x / LPH, l = threadIdx.x % LPH;
  const int b = blockIdx.y;
  const int p0 = blockIdx.x * PAIRS;
  griddep_wait();
  const SeqRows s = batch_seq(B, b, true);
  if (s.err != PF_OK && blockIdx.x == 0 && threadIdx.x == 0) batch_record(status, s.err);
  const int pairs = s.n * heads;
  if (p0 >= pairs) return;
  float4 A[SLOTS], C[SLOTS];
#pragma unroll
  for (int x = 0; x < SLOTS; ++x) {
    const int p = p0 + x * PER + group;
    A[x] = C[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p < pairs) {
      const float4* src = reinterpret_cast<const float4*>(qkv + (static_cast<size_t>(s.at) * heads + p) * HD);
      A[x] = src[l];
      C[x] = src[LPH + l];
    }
  }
  const int r0 = p0 / heads, r1 = min(p0 + PAIRS - 1, pairs - 1) / heads;
  if (static_cast<int>(threadIdx.x) <= r1 - r0) {
    const int i = r0 + threadIdx.x;
    const int slot = batch_slot(B, b, s.start + i);
    int depth = i;
    if (B.parent != nullptr) {
      depth = 0;
      bool bad;
      for (int j = tree_parent(B.parent + s.at, i, bad); j >= 0; ++depth) {
        bool skip;  // a bad ancestor is recorded by its own row
        j = tree_parent(B.parent + s.at, j, skip);
      }
      if (bad) batch_record(status, PF_ERR_INVALID_ARG);
    }
    row_slot[threadIdx.x] = slot;
    row_pos[threadIdx.x] = s.start + depth;
    if (slot < 0) batch_record(status, PF_ERR_KV_CAPACITY);
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < SLOTS; ++x) {
    const int p = p0 + x * PER + group;
    const int r = p / heads, j = p - r * heads;
    float4 a = A[x], c = C[x];
    float ss = a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w + c.x * c.x + c.y * c.y + c.z * c.z + c.w * c.w;
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (p >= pairs) continue;
    const int slot = row_slot[r - r0];
    const bool is_q = j < nq, is_v = j >= nq + nkv;
    if (!is_v) {
      const float4* cs = reinterpret_cast<const float4*>(rope + (static_cast<size_t>(row_pos[r - r0]) * HALF + 4 * l) * 2);
      const float4 c01 = __ldg(cs), c23 = __ldg(cs + 1);
      if (qk_norm) {
        const float f = rsqrtf(ss / static_cast<float>(HD) + eps);
        const float4* w4 = reinterpret_cast<const float4*>(is_q ? qn : kn);
        const float4 wa = __ldg(w4 + l), wb = __ldg(w4 + LPH + l);
        a = make_float4(a.x * f * wa.x, a.y * f * wa.y, a.z * f * wa.z, a.w * f * wa.w);
        c = make_float4(c.x * f * wb.x, c.y * f * wb.y, c.z * f * wb.z, c.w * f * wb.w);
      }
      const float4 u = a, v = c;
      a = make_float4(u.x * c01.x - v.x * c01.y, u.y * c01.z - v.y * c01.w, u.z * c23.x - v.z * c23.y, u.w * c23.z - v.w * c23.w);
      c = make_float4(v.x * c01.x + u.x * c01.y, v.y * c01.z + u.y * c01.w, v.z * c23.x + u.z * c23.y, v.w * c23.z + u.w * c23.w);
    }
    T* dst;
    if (is_q) {
      dst = q_out + (static_cast<size_t>(s.at + r) * nq + j) * HD;
    } else {
      if (slot < 0) continue;
      const int kvh = j - nq - (is_v ? nkv : 0);
      dst = (is_v ? vc : kc) + ((static_cast<size_t>(layer) * nkv + kvh) * B.slots + slot) * HD;
    }
    put4<T>(dst + 4 * l, a.x, a.y, a.z, a.w);
    put4<T>(dst + HALF + 4 * l, c.x, c.y, c.z, c.w);
  }
}

template <int HD, typename T>
cudaError_t append(const pf_config& c, const pf_batch& b, const float* qkv, const float* qn, const float* kn, const float* rope,
                   int layer, void* q, void* kc, void* vc, int* status, cudaStream_t stream) {
  constexpr int PER = AP_THREADS / (HD / 8);
  const int pairs = std::min(b.max_rows, b.n_rows) * (c.n_q_heads + 2 * c.n_kv_heads);
  auto go = [&](auto kernel, int per) {
    return launch_pdl(kernel, dim3((pairs + per - 1) / per, b.n_seq), dim3(AP_THREADS), 0, stream, batch_dev(c, b), qkv, qn, kn, rope,
                      c.n_q_heads, c.n_kv_heads, layer, c.eps, c.qk_norm, static_cast<T*>(q), static_cast<T*>(kc),
                      static_cast<T*>(vc), status);
  };
  // One pair a thread group while the CTAs fit on the chip at once, two in flight beyond. Measured, one against two: one row 2.1 and
  // 2.5 us, 48 sequences of one 2.5 and 2.8, eight of 8 2.8 and 2.9, eight of 60 5.7 and 4.4, the chunks above 11.5 and 9.2 (four: 9.7).
  const int64_t ctas = static_cast<int64_t>((pairs + PER - 1) / PER) * b.n_seq;
  return ctas <= 2 * device_sm_count() ? go(batch_append_kernel<HD, T, 1>, PER) : go(batch_append_kernel<HD, T, 2>, 2 * PER);
}

// ------------------------------------------------------------------ accept
// The walk: node = -1, want = root id; the lowest child of node with token == want is accepted, want = its id;
// until there is none. One warp holds a sequence's parents and tokens, eight nodes a lane, and finds the child with
// one reduction a step. Every CTA of a sequence walks for itself and then moves its share of the (layer, head,
// K or V) lines; path[j] >= j and both rise, so moving rows in order of j, eight read before eight are written,
// reads none that was written. What bounds it is latency: rows, tokens, walk, table and the rows that move depend on
// one another (a tree of 26 nodes 3.2 us, 16 of 31 .. 61 nodes 3.7 us, two layers' K and V moved).
constexpr int AC_THREADS = 256;

__global__ void __launch_bounds__(AC_THREADS) tree_accept_kernel(const BatchDev B, const int* tokens, const int* ids, const int* root,
                                                                 int* path_out, int* n_out, int* next_out, uint4* kc, uint4* vc, int heads,
                                                                 int vec, int* status) {
  PF_TIMELINE(TL_TREE_ACCEPT);
  __shared__ int path[PF_MAX_TREE], id_s[PF_MAX_TREE], from[PF_MAX_TREE], to[PF_MAX_TREE];
  __shared__ int count_s, next_s, moves_s;
  griddep_launch_dependents();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  griddep_wait();
  const SeqRows s = batch_seq(B, b, true);
  const bool first = blockIdx.y == 0;
  if (s.err != PF_OK && first && threadIdx.x == 0) batch_record(status, s.err);
  if (threadIdx.x < 32) {
    constexpr int PER = PF_MAX_TREE / 32;
    int par[PER], tok[PER], want = root[b];
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int i = lane + 32 * x;
      par[x] = -2;
      tok[x] = 0;
      if (i < s.n) {
        bool bad = false;
        par[x] = B.parent != nullptr ? tree_parent(B.parent + s.at, i, bad) : i - 1;
        if (bad && first) batch_record(status, PF_ERR_INVALID_ARG);
        tok[x] = tokens[s.at + i];
        id_s[i] = ids[s.at + i];
      }
    }
    __syncwarp();
    int node = -1, count = 0;
    while (count < s.n) {
      unsigned m = 0xffffffffu;
#pragma unroll
      for (int x = PER - 1; x >= 0; --x)
        if (par[x] == node && tok[x] == want) m = lane + 32 * x;
      m = __reduce_min_sync(0xffffffffu, m);
      if (m == 0xffffffffu) break;
      if (lane == 0) path[count] = m;
      ++count;
      node = m;
      want = id_s[m];
    }
    if (lane == 0) {
      count_s = count;
      next_s = want;
    }
    __syncwarp();
    // the rows that move, as slots
    int moves = 0;
    for (int j0 = 0; j0 < count && kc != nullptr; j0 += 32) {
      const int j = j0 + lane;
      int f = -1, t = -1;
      if (j < count && path[j] != j) {
        f = batch_slot(B, b, s.start + path[j]);
        t = batch_slot(B, b, s.start + j);
        if ((f < 0 || t < 0) && first) batch_record(status, PF_ERR_KV_CAPACITY);
      }
      const unsigned some = __ballot_sync(0xffffffffu, f >= 0 && t >= 0);
      if (f >= 0 && t >= 0) {
        const int k = moves + __popc(some & ((1u << lane) - 1u));
        from[k] = f;
        to[k] = t;
      }
      moves += __popc(some);
    }
    if (lane == 0) moves_s = moves;
  }
  __syncthreads();
  if (first) {
    for (int j = threadIdx.x; j < s.n; j += AC_THREADS) path_out[s.at + j] = j < count_s ? path[j] : -1;
    if (threadIdx.x == 0) {
      n_out[b] = count_s;
      next_out[b] = next_s;
    }
  }
  const int moves = moves_s;
  if (moves == 0) return;
  // `vec` lanes hold a row (16 B each); lines = (layer, kv head) of K, then of V
  const int line = (blockIdx.y * AC_THREADS + threadIdx.x) / vec, v = threadIdx.x % vec;
  if (line >= 2 * heads) return;
  uint4* c = (line < heads ? kc : vc) + static_cast<size_t>(line < heads ? line : line - heads) * B.slots * vec + v;
  for (int j = 0; j < moves; j += 8) {
    uint4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + u < moves) x[u] = c[static_cast<size_t>(from[j + u]) * vec];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + u < moves) c[static_cast<size_t>(to[j + u]) * vec] = x[u];
  }
}

}  // namespace

cudaError_t launch_batch_append(const pf_config& c, const pf_batch& b, const float* qkv, const float* qn, const float* kn,
                                const float* rope, int layer, void* q, void* kc, void* vc, int* status, cudaStream_t stream) {
  const bool bf = c.kv_dtype == PF_KV_BF16;
  if (c.head_dim == 128)
    return bf ? append<128, __nv_bfloat16>(c, b, qkv, qn, kn, rope, layer, q, kc, vc, status, stream)
              : append<128, __half>(c, b, qkv, qn, kn, rope, layer, q, kc, vc, status, stream);
  return bf ? append<64, __nv_bfloat16>(c, b, qkv, qn, kn, rope, layer, q, kc, vc, status, stream)
            : append<64, __half>(c, b, qkv, qn, kn, rope, layer, q, kc, vc, status, stream);
}

cudaError_t launch_tree_accept(const pf_config& c, const pf_batch& b, const int* tokens, const int* ids, const int* root, int* path,
                               int* n_accepted, int* next, void* kc, void* vc, int* status, cudaStream_t stream) {
  const int vec = c.head_dim / 8, heads = c.n_layers * c.n_kv_heads;
  const int lines = AC_THREADS / vec;
  const dim3 grid(b.n_seq, kc != nullptr ? (2 * heads + lines - 1) / lines : 1);
  return launch_pdl(tree_accept_kernel, grid, dim3(AC_THREADS), 0, stream, batch_dev(c, b), tokens, ids, root, path, n_accepted,
                    next, static_cast<uint4*>(kc), static_cast<uint4*>(vc), heads, vec, status);
}

}  // namespace pf

PF_TIMELINE_SETTER(batch)
