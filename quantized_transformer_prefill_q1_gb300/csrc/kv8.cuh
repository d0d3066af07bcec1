// kv8.cuh — what the kernels of the 8-bit KV cache share: the slot of a position, and the two
// code types' conversions.
//
// A cache buffer (K or V) holds one-byte codes [n_layers][nkv][slots][hd] and, from
// pf_kv8_scales_offset() on, f32 scales [n_layers][nkv][ceil(slots / 32)]: the value of a code in
// slot s is code * scale[s / 32]. The scales that the store writes are powers of two, so scaling a
// value for the code and a code back to its value never rounds.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"

namespace pf {

// Slot of position p, or -1 when its block table entry names no block of the pool.
__device__ __forceinline__ int kv8_slot(const Kv8Layer& c, int p) {
  if (c.table == nullptr) return p;
  const int b = c.table[p / PF_KV_BLOCK];
  return b < 0 || b >= c.pool ? -1 : b * PF_KV_BLOCK + p % PF_KV_BLOCK;
}

template <int T>
struct Kv8 {
  static constexpr float CMAX = T == PF_KV_E4M3 ? 448.f : 127.f;
  // Nearest code, ties to even, saturating; |x| beyond CMAX only for infinities.
  static __device__ __forceinline__ uint32_t encode(float x) {
    if (T == PF_KV_E4M3)
      return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
    else
      return static_cast<uint32_t>(static_cast<int>(rintf(fminf(fmaxf(x, -127.f), 127.f)))) & 255u;
  }
  // The values of a word's four codes as f16 pairs (codes 0, 1 and 2, 3): every code is exact in f16.
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (T == PF_KV_E4M3) {
      asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
          : "=r"(lo), "=r"(hi)
          : "r"(w));
    } else {
      // 0x6400 | u is the f16 1024 + u for u in 0 .. 255; u = code + 128
      const uint32_t u = w ^ 0x80808080u;
      const __half2 off = __floats2half2_rn(1152.f, 1152.f);
      uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
      const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off), y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
      lo = *reinterpret_cast<const uint32_t*>(&x);
      hi = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  static __device__ __forceinline__ float decode(uint32_t c) {
    if (T == PF_KV_E4M3) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E4M3);
      return __half2float(__half(h));
    } else {
      return static_cast<float>(static_cast<int>(static_cast<int8_t>(c)));
    }
  }
};

}  // namespace pf
