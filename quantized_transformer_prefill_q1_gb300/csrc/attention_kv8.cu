// attention_kv8.cu — causal GQA attention over the 8-bit KV cache.
//
// For the query at position i of head h (kv head h / G) over keys j <= i:
//   s_j = (q . c^K_j) sK[block(j)] / sqrt(hd),  p = softmax_j(s),  o = sum_j p_j c^V_j sV[block(j)].
#include "kv8.cuh"

namespace pf {
namespace {

constexpr int SQ = 16;  // query rows per CTA

// 128 threads, 16 rows of one kv head (row = token * G + head in the group), 32 keys (one scale
// block) at a time in shared memory as f32. Thread (r, u) = (tid / 8, tid % 8) scores keys
// 4u .. 4u + 3 of row r and then owns columns u + 8 i of its output.
template <int HD, int T>
__global__ void __launch_bounds__(128) attn_kv8_kernel(const __half* __restrict__ q, Kv8Layer c, int nq, int nkv, int M,
                                                       const int* __restrict__ start_dev, int start_host, float scale_log2,
                                                       __half* __restrict__ out, int* status) {
  PF_TIMELINE(TL_ATTENTION_KV8);
  __shared__ float qs[SQ][HD + 1], ks[32][HD + 1], vs[32][HD], ps[SQ][33];
  griddep_launch_dependents();
  griddep_wait();
  const int start = start_dev ? *start_dev : start_host;
  const int G = nq / nkv, kvh = blockIdx.y;
  const int rows = M * G;
  const int r = threadIdx.x >> 3, u = threadIdx.x & 7;
  const int row = blockIdx.x * SQ + r;
  const int t = row / G, h = kvh * G + row % G;
  const int pos = row < rows ? start + t : -1;
  const int last = start + min(rows - 1, static_cast<int>(blockIdx.x) * SQ + SQ - 1) / G;
  for (int i = u; i < HD; i += 8) qs[r][i] = row < rows ? __half2float(q[(static_cast<size_t>(t) * nq + h) * HD + i]) : 0.f;
  float m = -INFINITY, l = 0.f, o[HD / 8];
#pragma unroll
  for (int i = 0; i < HD / 8; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 <= last; j0 += 32) {
    __syncthreads();
    int slot = kv8_slot(c, j0);
    if (slot < 0) {
      if (threadIdx.x == 0 && status) atomicCAS(status, 0, PF_ERR_KV_CAPACITY);
      slot = 0;
    }
    const float sk = c.ks[static_cast<size_t>(kvh) * c.nblk + slot / 32], sv = c.vs[static_cast<size_t>(kvh) * c.nblk + slot / 32];
    for (int i = threadIdx.x; i < 32 * HD / 4; i += 128) {
      const int key = i / (HD / 4), d = (i % (HD / 4)) * 4;
      uint32_t a = 0, b = 0;
      if (j0 + key <= last) {
        const size_t at = (static_cast<size_t>(kvh) * c.slots + slot + key) * HD + d;
        a = *reinterpret_cast<const uint32_t*>(c.k + at);
        b = *reinterpret_cast<const uint32_t*>(c.v + at);
      }
      for (int e = 0; e < 4; ++e) {
        ks[key][d + e] = Kv8<T>::decode((a >> (8 * e)) & 255u) * sk;
        vs[key][d + e] = j0 + key <= last ? Kv8<T>::decode((b >> (8 * e)) & 255u) * sv : 0.f;
      }
    }
    __syncthreads();
    float s[4], mx = -INFINITY;
    for (int e = 0; e < 4; ++e) {
      const int key = 4 * u + e;
      float x = 0.f;
      for (int i = 0; i < HD; ++i) x = fmaf(qs[r][i], ks[key][i], x);
      s[e] = j0 + key <= pos ? x * scale_log2 : -INFINITY;
      mx = fmaxf(mx, s[e]);
    }
    for (int w = 4; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const float mn = fmaxf(m, mx), alpha = mn == -INFINITY ? 1.f : exp2f(m - mn);
    float sum = 0.f;
    for (int e = 0; e < 4; ++e) {
      const float p = mn == -INFINITY ? 0.f : exp2f(s[e] - mn);
      sum += p;
      ps[r][4 * u + e] = p;
    }
    for (int w = 4; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * alpha + sum;
    m = mn;
    __syncwarp();
    for (int i = 0; i < HD / 8; ++i) o[i] *= alpha;
    for (int key = 0; key < 32; ++key) {
      const float p = ps[r][key];
      if (p == 0.f) continue;  // a hidden key's row may hold anything
      for (int i = 0; i < HD / 8; ++i) o[i] = fmaf(p, vs[key][u + 8 * i], o[i]);
    }
  }
  if (row < rows)
    for (int i = 0; i < HD / 8; ++i) out[(static_cast<size_t>(t) * nq + h) * HD + u + 8 * i] = __float2half_rn(o[i] / l);
}

}  // namespace

size_t attention_kv8_scratch_bytes(const pf_config&, int) { return KV8_COUNTER_BYTES; }

cudaError_t launch_attention_kv8(const Kv8AttnArgs& a, cudaStream_t stream) {
  const pf_config& c = *a.c;
  const Kv8Layer L = kv8_layer(c, a.k_cache, a.v_cache, a.layer, a.blocks);
  const int G = c.n_q_heads / c.n_kv_heads;
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.M) * G + SQ - 1) / SQ), c.n_kv_heads);
  const float sl2 = 1.4426950408889634f / sqrtf(static_cast<float>(c.head_dim));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(128), 0, stream, static_cast<const __half*>(a.q), L, static_cast<int>(c.n_q_heads),
                      static_cast<int>(c.n_kv_heads), a.M, a.start_dev, a.start_host, sl2, static_cast<__half*>(a.out), a.status);
  };
  if (c.head_dim == 128)
    return c.kv_dtype == PF_KV_E4M3 ? go(attn_kv8_kernel<128, PF_KV_E4M3>) : go(attn_kv8_kernel<128, PF_KV_INT8>);
  return c.kv_dtype == PF_KV_E4M3 ? go(attn_kv8_kernel<64, PF_KV_E4M3>) : go(attn_kv8_kernel<64, PF_KV_INT8>);
}

}  // namespace pf

PF_TIMELINE_SETTER(attention_kv8)
