// kv8.cu — the 8-bit KV cache: quantising store and read-back.
//
// Store: positions start .. start + M - 1 of K and V, f16 rows, into codes with one scale for each
// 32 slots of a kv head. For one (kv head, block of 32 positions) with new rows x:
//   amax = max |x| over the finite new values; e = the least integer with amax <= CMAX 2^e,
//   e >= -32; s = 2^e, or max(s_old, 2^e) when the block holds positions before `start`;
//   old codes of a block whose scale grows: c <- RNE(c s_old / s);  new codes: c = RNE(x / s).
// s is a power of two, so x / s and c s_old / s are exact and each code has one rounding; e4m3 keeps
// its full relative precision under such a scale, int8 at worst half of its steps.
#include "kv8.cuh"

namespace pf {
namespace {

constexpr int ST_THREADS = 128;
constexpr int E_MIN = -32;  // exponent of an all-zero block: the smallest f16 (2^-24) over 448 needs -32

// Least e with amax <= CMAX 2^e. amax = m 2^x, 1 <= m < 2: CMAX 2^e = (CMAX / 2^top) 2^(e + top).
template <int T>
__device__ __forceinline__ int scale_exponent(float amax) {
  constexpr int TOP = T == PF_KV_E4M3 ? 8 : 6;                      // 448 = 1.75 2^8, 127 = 1.984375 2^6
  constexpr uint32_t MANT = T == PF_KV_E4M3 ? 0x600000u : 0x7E0000u;  // their fractions
  if (!(amax > 0.f)) return E_MIN;
  const uint32_t u = __float_as_uint(amax);
  const int x = static_cast<int>(u >> 23) - 127;  // an f16's magnitude is a normal f32
  return max(E_MIN, x - TOP + ((u & 0x7FFFFFu) > MANT ? 1 : 0));
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Eight f16 values times inv (a power of two from 2^-15 to 2^15) to codes. The product is exact in f16
// unless it is below 2^-14, where both types' codes are 0 (their smallest nonzero values' halves are
// 2^-10 and 1/2) whatever it was rounded to, so the code has one rounding.
template <int T>
__device__ __forceinline__ uint2 encode8(uint4 raw, __half2 inv) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t n[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&w[2 * j]), inv), b = __hmul2(*reinterpret_cast<const __half2*>(&w[2 * j + 1]), inv);
    if (T == PF_KV_E4M3) {
      asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\tmov.b32 %0, {x, y};\n\t}"
          : "=r"(n[j])
          : "r"(*reinterpret_cast<const uint32_t*>(&a)), "r"(*reinterpret_cast<const uint32_t*>(&b)));
    } else {
      // 1536 + x, |x| <= 127, has steps of 1 in f16: the sum rounds x to an integer, ties to even, and its
      // low byte is that integer's
      const __half2 m = __floats2half2_rn(1536.f, 1536.f);
      const __half2 c = __hadd2(a, m), d = __hadd2(b, m);
      n[j] = __byte_perm(*reinterpret_cast<const uint32_t*>(&c), *reinterpret_cast<const uint32_t*>(&d), 0x6420);
    }
  }
  return make_uint2(n[0], n[1]);
}

// One CTA = one block of 32 positions of one kv head, K (blockIdx.z 0) or V (1). Eight values a
// thread and pass, the block's new rows held in registers between the maximum and the rounding, so
// each row is read once; both in packed f16 arithmetic (in f32, one value at a time, the ALU was 68 %
// busy and 8,192 tokens of 8 heads of 128 took 15.5 us under the profiler, now 11.5 with the ALU 37 % busy).
// Bound: latency at one token (one CTA per head; 1.9 us), memory at long chunks (8,192 tokens 6.4 us in a
// replayed graph, part of it in L2).
template <int HD, int T>
__global__ void __launch_bounds__(ST_THREADS) kv8_store_kernel(const __half* kx, const __half* vx, long long tok_stride,
                                                               long long head_stride, const int* start_dev,
                                                               int start_host, int M, Kv8Layer c, int* status) {
  PF_TIMELINE(TL_KV8_STORE);
  constexpr int LPR = HD / 8;                // threads per row
  constexpr int RPP = ST_THREADS / LPR;      // rows per pass
  constexpr int NP = PF_KV8_BLOCK / RPP;     // passes
  __shared__ float red[ST_THREADS / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int start = start_dev ? *start_dev : start_host;
  const int base = (start / PF_KV8_BLOCK + static_cast<int>(blockIdx.x)) * PF_KV8_BLOCK;  // first position
  const int end = start + M;
  if (base >= end) return;
  const int kvh = blockIdx.y;
  const __half* x = blockIdx.z ? vx : kx;
  const int slot0 = kv8_slot(c, base);
  if (slot0 < 0) {
    if (threadIdx.x == 0 && status) atomicCAS(status, 0, PF_ERR_KV_CAPACITY);
    return;
  }
  uint8_t* codes = (blockIdx.z ? c.v : c.k) + (static_cast<size_t>(kvh) * c.slots + slot0) * HD;
  float* scale = (blockIdx.z ? c.vs : c.ks) + static_cast<size_t>(kvh) * c.nblk + slot0 / PF_KV8_BLOCK;
  const int row0 = threadIdx.x / LPR, col = (threadIdx.x % LPR) * 8;
  const int lo = start - base;  // rows below it were there before (none when <= 0)
  const float s_old = lo > 0 ? *scale : 0.f;
  uint4 raw[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = row0 + i * RPP;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r >= lo && base + r < end)
      raw[i] = *reinterpret_cast<const uint4*>(x + (base + r - start) * tok_stride + kvh * head_stride + col);
  }
  __half2 top = __floats2half2_rn(0.f, 0.f);  // NaN if there is one
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __half2*>(&w[j])));
  }
  const float2 tops = __half22float2(top);
  const bool odd = !(tops.x <= 65504.f && tops.y <= 65504.f);  // a NaN or an infinity
  float amax = fmaxf(tops.x, tops.y);
  if (odd) {  // the finite values' maximum, one by one
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        if (fabsf(f.x) <= 65504.f) amax = fmaxf(amax, fabsf(f.x));
        if (fabsf(f.y) <= 65504.f) amax = fmaxf(amax, fabsf(f.y));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  const int bad = __syncthreads_or(odd);
#pragma unroll
  for (int i = 0; i < ST_THREADS / 32; ++i) amax = fmaxf(amax, red[i]);
  const float s_new = pow2i(scale_exponent<T>(amax));
  const float s = fmaxf(s_old, s_new);
  const float inv = 1.f / s;  // exact: s is a power of two
  const bool packed = !bad && inv <= 0x1p15f && inv >= 0x1p-15f;
  const __half2 inv2 = __floats2half2_rn(inv, inv);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = row0 + i * RPP;
    uint2* dst = reinterpret_cast<uint2*>(codes + r * HD + col);
    if (r < lo) {
      if (s > s_old) {  // the block's scale grows: its old codes follow
        const float ratio = s_old * inv;
        const uint2 old = *dst;
        uint32_t o[2] = {old.x, old.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t n = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) n |= Kv8<T>::encode(Kv8<T>::decode((o[j] >> (8 * b)) & 255u) * ratio) << (8 * b);
          o[j] = n;
        }
        *dst = make_uint2(o[0], o[1]);
      }
    } else if (base + r < end && packed) {
      *dst = encode8<T>(raw[i], inv2);
    } else if (base + r < end) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t n[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        const uint32_t a = f.x == f.x ? Kv8<T>::encode(f.x * inv) : 0u;  // a NaN is held as zero
        const uint32_t b = f.y == f.y ? Kv8<T>::encode(f.y * inv) : 0u;
        n[j >> 1] |= (a | b << 8) << (16 * (j & 1));
      }
      *dst = make_uint2(n[0], n[1]);
    }
  }
  if (threadIdx.x == 0) {
    *scale = s;
    if (bad && status) atomicCAS(status, 0, PF_ERR_NONFINITE);
  }
}

// Read-back: out[t][kvh][i] = code * scale of position start + t. A warp takes four tokens of one kv head
// (hd 64: eight), four codes a lane, so that every access is contiguous and four are in flight. HBM bound.
constexpr int LD_TOKENS = 32;  // tokens per CTA at hd 128
template <int HD, int T>
__global__ void __launch_bounds__(256) kv8_load_kernel(const uint8_t* codes, const float* scales, Kv8Layer c, int nkv, int start,
                                                       int M, float* out, int* status) {
  PF_TIMELINE(TL_KV8_LOAD);
  constexpr int LPR = HD / 4, RPW = 32 / LPR;  // lanes per row, rows per warp and pass
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, kvh = blockIdx.y;
  const int t0 = (static_cast<int>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5)) * 4 * RPW + lane / LPR, d = (lane % LPR) * 4;
  codes += static_cast<size_t>(kvh) * c.slots * HD + d;
  scales += static_cast<size_t>(kvh) * c.nblk;
  uint32_t w[4];
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i * RPW;
    w[i] = 0;
    s[i] = 0.f;
    if (t >= M) continue;
    const int slot = kv8_slot(c, start + t);
    if (slot < 0) {
      if (status) atomicCAS(status, 0, PF_ERR_KV_CAPACITY);
      continue;
    }
    w[i] = *reinterpret_cast<const uint32_t*>(codes + static_cast<size_t>(slot) * HD);
    s[i] = scales[slot / PF_KV8_BLOCK];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i * RPW;
    if (t >= M) break;
    *reinterpret_cast<float4*>(out + (static_cast<size_t>(t) * nkv + kvh) * HD + d) =
        make_float4(Kv8<T>::decode(w[i] & 255u) * s[i], Kv8<T>::decode((w[i] >> 8) & 255u) * s[i],
                    Kv8<T>::decode((w[i] >> 16) & 255u) * s[i], Kv8<T>::decode(w[i] >> 24) * s[i]);
  }
}

}  // namespace

Kv8Layer kv8_layer(const pf_config& c, const void* k, const void* v, int layer, const int* table) {
  Kv8Layer L{};
  const size_t slots = cache_slots(c), rows = static_cast<size_t>(c.n_kv_heads) * slots;
  L.slots = static_cast<int>(slots);
  L.nblk = (L.slots + PF_KV8_BLOCK - 1) / PF_KV8_BLOCK;
  const size_t at = kv8_scales_offset(c) + static_cast<size_t>(layer) * c.n_kv_heads * L.nblk * sizeof(float);
  auto* kb = static_cast<uint8_t*>(const_cast<void*>(k));
  auto* vb = static_cast<uint8_t*>(const_cast<void*>(v));
  if (kb) {
    L.k = kb + layer * rows * c.head_dim;
    L.ks = reinterpret_cast<float*>(kb + at);
  }
  if (vb) {
    L.v = vb + layer * rows * c.head_dim;
    L.vs = reinterpret_cast<float*>(vb + at);
  }
  L.table = c.kv_block_pool > 0 ? table : nullptr;
  L.pool = c.kv_block_pool;
  return L;
}

cudaError_t launch_kv8_store(const Kv8StoreArgs& a, cudaStream_t stream) {
  const pf_config& c = *a.c;
  const Kv8Layer L = kv8_layer(c, a.k_cache, a.v_cache, a.layer, a.blocks);
  // M positions touch at most ceil(M / 32) + 1 blocks wherever they start
  const dim3 grid((a.M + PF_KV8_BLOCK - 1) / PF_KV8_BLOCK + 1, c.n_kv_heads, 2);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(ST_THREADS), 0, stream, static_cast<const __half*>(a.k), static_cast<const __half*>(a.v),
                      static_cast<long long>(a.tok_stride), static_cast<long long>(a.head_stride), a.start_dev, a.start_host,
                      a.M, L, a.status);
  };
  if (c.head_dim == 128)
    return c.kv_dtype == PF_KV_E4M3 ? go(kv8_store_kernel<128, PF_KV_E4M3>) : go(kv8_store_kernel<128, PF_KV_INT8>);
  return c.kv_dtype == PF_KV_E4M3 ? go(kv8_store_kernel<64, PF_KV_E4M3>) : go(kv8_store_kernel<64, PF_KV_INT8>);
}

cudaError_t launch_kv8_load(const pf_config& c, const void* cache, int layer, int start, int M, const int* blocks,
                            float* out, int* status, cudaStream_t stream) {
  const Kv8Layer L = kv8_layer(c, cache, nullptr, layer, blocks);
  const int tokens = c.head_dim == 128 ? LD_TOKENS : 2 * LD_TOKENS;
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3((M + tokens - 1) / tokens, c.n_kv_heads), dim3(256), 0, stream, static_cast<const uint8_t*>(L.k),
                      static_cast<const float*>(L.ks), L, static_cast<int>(c.n_kv_heads), start, M, out, status);
  };
  if (c.head_dim == 128) return c.kv_dtype == PF_KV_E4M3 ? go(kv8_load_kernel<128, PF_KV_E4M3>) : go(kv8_load_kernel<128, PF_KV_INT8>);
  return c.kv_dtype == PF_KV_E4M3 ? go(kv8_load_kernel<64, PF_KV_E4M3>) : go(kv8_load_kernel<64, PF_KV_INT8>);
}

}  // namespace pf

PF_TIMELINE_SETTER(kv8)
