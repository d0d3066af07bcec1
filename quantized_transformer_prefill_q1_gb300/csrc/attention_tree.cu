// attention_tree.cu — attention of many sequences' rows (trees of drafted tokens, single tokens) over the cache.
//
// For row i of a sequence and its head h (kv head h / G) over the keys j that it sees (the cached positions, its
// ancestors, itself): s_j = q . k_j / sqrt(hd), p = softmax_j(s), o = sum_j p_j v_j.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "batch.cuh"

namespace pf {
namespace {

constexpr int THREADS = 128;

__device__ __forceinline__ float2 pair(__half2 x) { return __half22float2(x); }
__device__ __forceinline__ float2 pair(__nv_bfloat162 x) { return __bfloat1622float2(x); }

// One CTA per (row, sequence, kv head), a warp per query head, keys one after the other.
template <int HD, typename T2>
__global__ void __launch_bounds__(THREADS) tree_rows_kernel(const BatchDev B, const T2* __restrict__ q, const T2* __restrict__ kc,
                                                            const T2* __restrict__ vc, int nq, int nkv, int layer, float scale,
                                                            __half* __restrict__ out, int* status) {
  PF_TIMELINE(TL_ATTENTION_TREE);
  constexpr int PER = HD / 64;  // pairs of elements a lane
  __shared__ uint32_t see[PF_MAX_TREE / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int i = blockIdx.x, b = blockIdx.y, kvh = blockIdx.z;
  const int G = nq / nkv, lane = threadIdx.x & 31;
  const SeqRows s = batch_seq(B, b, true);
  if (s.err != PF_OK && threadIdx.x == 0) batch_record(status, s.err);
  if (i >= s.n) return;
  if (threadIdx.x < PF_MAX_TREE / 32) see[threadIdx.x] = 0;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int j = i; j >= 0;) {
      see[j >> 5] |= 1u << (j & 31);
      bool bad = false;
      const int p = B.parent != nullptr ? tree_parent(B.parent + s.at, j, bad) : j - 1;
      if (bad) batch_record(status, PF_ERR_INVALID_ARG);
      j = p;
    }
  }
  __syncthreads();
  const size_t head = (static_cast<size_t>(layer) * nkv + kvh) * B.slots;
  for (int h = kvh * G + (threadIdx.x >> 5); h < (kvh + 1) * G; h += THREADS / 32) {
    float2 x[PER], o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      x[e] = pair(q[(static_cast<size_t>(s.at + i) * nq + h) * (HD / 2) + lane + 32 * e]);
      o[e] = make_float2(0.f, 0.f);
    }
    float m = -INFINITY, l = 0.f;
    for (int p = 0; p <= s.start + i; ++p) {
      const int j = p - s.start;
      if (j >= 0 && !(see[j >> 5] >> (j & 31) & 1u)) continue;
      int slot = batch_slot(B, b, p);
      if (slot < 0) {
        if (lane == 0) batch_record(status, PF_ERR_KV_CAPACITY);
        slot = 0;
      }
      const size_t at = (head + slot) * (HD / 2) + lane;
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const float2 k = pair(kc[at + 32 * e]);
        d = fmaf(x[e].x, k.x, fmaf(x[e].y, k.y, d));
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
      d *= scale;
      const float mn = fmaxf(m, d), a = expf(m - mn), e2 = expf(d - mn);
      m = mn;
      l = l * a + e2;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const float2 v = pair(vc[at + 32 * e]);
        o[e].x = o[e].x * a + e2 * v.x;
        o[e].y = o[e].y * a + e2 * v.y;
      }
    }
    __half2* dst = reinterpret_cast<__half2*>(out) + (static_cast<size_t>(s.at + i) * nq + h) * (HD / 2) + lane;
#pragma unroll
    for (int e = 0; e < PER; ++e) dst[32 * e] = __floats2half2_rn(o[e].x / l, o[e].y / l);
  }
}

template <int HD, typename T2>
cudaError_t launch_rows(const TreeAttnArgs& a, cudaStream_t stream) {
  const pf_config& c = *a.c;
  return launch_pdl(tree_rows_kernel<HD, T2>, dim3(a.b->max_rows, a.b->n_seq, c.n_kv_heads), dim3(THREADS), 0, stream,
                    batch_dev(c, *a.b), static_cast<const T2*>(a.q), static_cast<const T2*>(a.k_cache),
                    static_cast<const T2*>(a.v_cache), c.n_q_heads, c.n_kv_heads, a.layer, 1.f / sqrtf(static_cast<float>(HD)),
                    static_cast<__half*>(a.out), a.status);
}

}  // namespace

size_t attention_tree_scratch_bytes(const pf_config& c, int n_seq, int max_rows) { return 256; }

cudaError_t launch_attention_tree(const TreeAttnArgs& a, cudaStream_t stream) {
  const bool bf = a.c->kv_dtype == PF_KV_BF16;
  if (a.c->head_dim == 128) return bf ? launch_rows<128, __nv_bfloat162>(a, stream) : launch_rows<128, __half2>(a, stream);
  return bf ? launch_rows<64, __nv_bfloat162>(a, stream) : launch_rows<64, __half2>(a, stream);
}

}  // namespace pf

PF_TIMELINE_SETTER(attention_tree)
