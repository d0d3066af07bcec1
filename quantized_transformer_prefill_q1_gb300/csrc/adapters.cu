// adapters.cu — low-rank adapters of many sequences beside a shared projection:
// out[m] = base[m] + scale[a] (x[m] A_a^T) B_a^T with a the adapter of row m's sequence.
#include <cuda_fp16.h>

#include "batch.cuh"

namespace pf {
namespace {

// The sequence's adapter, -1 for none.
__device__ __forceinline__ int adapter_of(const int* adapter, int b, int count, int* status, bool tell) {
  const int a = adapter[b];
  if (a >= -1 && a < count) return a;
  if (tell) batch_record(status, PF_ERR_INVALID_ARG);
  return -1;
}

// h[m][r] = scale x[m] . A[r], a warp each
__global__ void __launch_bounds__(256) adapter_down_kernel(const BatchDev B, const __half* __restrict__ x, int64_t ldx, int K, int rank,
                                                           int count, const int* __restrict__ adapter,
                                                           const __half* __restrict__ wa, const float* __restrict__ scale,
                                                           float* __restrict__ h, int* status) {
  PF_TIMELINE(TL_ADAPTER_DOWN);
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const SeqRows s = batch_seq(B, b, false);
  if (s.err != PF_OK && blockIdx.x == 0 && threadIdx.x == 0) batch_record(status, s.err);
  const int a = adapter_of(adapter, b, count, status, blockIdx.x == 0 && threadIdx.x == 0);
  const int i = blockIdx.x;
  if (i >= s.n || a < 0) return;
  const __half2* xr = reinterpret_cast<const __half2*>(x + (s.at + i) * ldx);
  for (int r = threadIdx.x >> 5; r < rank; r += 8) {
    const __half2* w = reinterpret_cast<const __half2*>(wa + (static_cast<size_t>(a) * rank + r) * K);
    float d = 0.f;
    for (int k = lane; k < K / 2; k += 32) {
      const float2 u = __half22float2(xr[k]), v = __half22float2(w[k]);
      d = fmaf(u.x, v.x, fmaf(u.y, v.y, d));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) h[static_cast<size_t>(s.at + i) * rank + r] = d * scale[a];
  }
}

// out[m][n] = base[m][n] + h[m] . B[n]
__global__ void __launch_bounds__(256) adapter_up_kernel(const BatchDev B, const float* base, int64_t ldb, float* out, int64_t ldo,
                                                         int N, int rank, int count, const int* __restrict__ adapter,
                                                         const __half* __restrict__ wb, const float* __restrict__ h) {
  PF_TIMELINE(TL_ADAPTER_UP);
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.z, i = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  const SeqRows s = batch_seq(B, b, false);
  const int a = adapter_of(adapter, b, count, nullptr, false);
  if (i >= s.n || n >= N || (a < 0 && base == out)) return;
  float d = base[(s.at + i) * ldb + n];
  if (a >= 0) {
    const __half* w = wb + (static_cast<size_t>(a) * N + n) * rank;
    float e = 0.f;
    for (int r = 0; r < rank; ++r) e = fmaf(h[static_cast<size_t>(s.at + i) * rank + r], __half2float(w[r]), e);
    d += e;
  }
  out[(s.at + i) * ldo + n] = d;
}

}  // namespace

size_t adapters_scratch_bytes(int n_rows, int rank) { return (static_cast<size_t>(n_rows) * rank * 4 + 15) / 16 * 16; }

cudaError_t launch_adapters(const AdapterArgs& a, cudaStream_t stream) {
  BatchDev B{};
  B.n_seq = a.b->n_seq;
  B.n_rows = a.b->n_rows;
  B.max_rows = a.b->max_rows;
  B.row_begin = a.b->row_begin_dev;
  float* h = static_cast<float*>(a.scratch);
  cudaError_t e = launch_pdl(adapter_down_kernel, dim3(a.b->max_rows, a.b->n_seq), dim3(256), 0, stream, B,
                             static_cast<const __half*>(a.x), a.ldx, a.K, a.rank, a.n_adapters, a.adapter,
                             static_cast<const __half*>(a.wa), a.scale, h, a.status);
  if (e != cudaSuccess) return e;
  return launch_pdl(adapter_up_kernel, dim3((a.N + 255) / 256, a.b->max_rows, a.b->n_seq), dim3(256), 0, stream, B, a.base, a.ld_base,
                    a.out, a.ld_out, a.N, a.rank, a.n_adapters, a.adapter, static_cast<const __half*>(a.wb),
                    static_cast<const float*>(h));
}

}  // namespace pf

PF_TIMELINE_SETTER(adapters)
