// logprobs.cu — log probabilities of given tokens, the entropy and the top alternatives of each row
// of logits. With m = max_i x_i, S = sum_i e^(x_i - m), T = sum_i (x_i - m) e^(x_i - m):
//   logprob(t) = x_t - m - ln S,   entropy = -sum_i p_i ln p_i = ln S - T / S
// (both terms of the entropy are >= 0: nothing cancels). A logit of -inf has probability 0 and adds
// nothing to S and T; a NaN, a +inf or a row of -inf alone makes the row's results NaN.
#include "ptx.cuh"

namespace pf {
namespace {

// Order of the alternatives: larger logit first, lower index first among equals (-0 = +0); NaN last.
// The key of a value and its index is unique within a row.
__device__ __forceinline__ unsigned long long order_key(float x, int i) {
  if (x != x) return 0ull;
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<unsigned long long>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}

__global__ void __launch_bounds__(1024) logprobs_kernel(const float* __restrict__ logits, int n, long long ld,
                                                        const int* __restrict__ tokens, float* __restrict__ lp,
                                                        float* __restrict__ ent, int top, int* __restrict__ top_ids,
                                                        float* __restrict__ top_lp, int* status) {
  PF_TIMELINE(TL_LOGPROBS);
  __shared__ float rs[32], rt[32];
  __shared__ unsigned long long rk[32];
  griddep_launch_dependents();
  griddep_wait();
  const float* x = logits + blockIdx.x * ld;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float m = -INFINITY;
  bool nan = false;
  for (int i = threadIdx.x; i < n; i += 1024) {
    nan |= x[i] != x[i];
    m = fmaxf(m, x[i]);
  }
  nan = __syncthreads_or(nan);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) rs[warp] = m;
  __syncthreads();
  for (int w = 0; w < 32; ++w) m = fmaxf(m, rs[w]);
  __syncthreads();
  if (nan) m = NAN;
  float S = 0.f, T = 0.f;
  for (int i = threadIdx.x; i < n; i += 1024) {
    const float d = x[i] - m, e = __expf(d);
    S += e;
    if (d != -INFINITY) T += d * e;
  }
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, o);
    T += __shfl_xor_sync(0xffffffffu, T, o);
  }
  if (lane == 0) {
    rs[warp] = S;
    rt[warp] = T;
  }
  __syncthreads();
  S = T = 0.f;
  for (int w = 0; w < 32; ++w) {
    S += rs[w];
    T += rt[w];
  }
  const float ls = logf(S);
  if (threadIdx.x == 0) {
    if (lp) {
      const int t = tokens[blockIdx.x];
      if (t < 0 || t >= n) {
        lp[blockIdx.x] = NAN;
        if (status) atomicCAS(status, 0, PF_ERR_TOKEN_OUT_OF_VOCAB);
      } else {
        lp[blockIdx.x] = x[t] - m - ls;
      }
    }
    if (ent) ent[blockIdx.x] = ls - T / S;
  }
  unsigned long long before = ~0ull;
  for (int k = 0; k < top; ++k) {
    unsigned long long best = 0;
    for (int i = threadIdx.x; i < n; i += 1024) {
      const unsigned long long key = order_key(x[i], i);
      if (key < before && key > best) best = key;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long b = __shfl_xor_sync(0xffffffffu, best, o);
      best = b > best ? b : best;
    }
    __syncthreads();
    if (lane == 0) rk[warp] = best;
    __syncthreads();
    for (int w = 0; w < 32; ++w) best = rk[w] > best ? rk[w] : best;
    if (threadIdx.x == 0) {
      const int id = best ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
      top_ids[static_cast<size_t>(blockIdx.x) * top + k] = id;
      if (top_lp) top_lp[static_cast<size_t>(blockIdx.x) * top + k] = id < 0 ? NAN : x[id] - m - ls;
    }
    before = best;
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, cudaStream_t stream) {
  return launch_pdl(logprobs_kernel, dim3(a.rows), dim3(1024), 0, stream, a.logits, a.n, static_cast<long long>(a.ld), a.tokens,
                    a.logprobs, a.entropy, a.top, a.top_ids, a.top_logprobs, a.status);
}

}  // namespace pf

PF_TIMELINE_SETTER(logprobs)
