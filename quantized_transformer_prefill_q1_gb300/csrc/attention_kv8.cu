// attention_kv8.cu — causal GQA attention over the 8-bit KV cache, few query rows per kv head
// (decoded tokens, short drafts): the cache is read once and nothing else weighs, so the kernel is
// built around streaming it.
//
// For the query at position i of head h (kv head h / G) over keys j <= i:
//   s_j = (q . c^K_j) sK[block(j)] / sqrt(hd),  p = softmax_j(s),  o = sum_j p_j c^V_j sV[block(j)].
// The scales never touch the codes: with u_j = log2(e) s_j + log2 sV[block(j)], one exponential gives
// the weight w_j = 2^(u_j - m) = p_j sV 2^..., ready for the product with the value codes, and the
// softmax's sum takes w_j / sV, one multiplication per block of 32 keys. The running maximum m is
// that of u, so weights stay in f16's range whatever the blocks' scales are; it is raised only when
// exceeded by more than 2^8.
//
// The rows of one kv head (row = token * G + head in the group, at most 8 NB) are the n side of
// warp-level MMAs m16n8k16 (f16, f32 accumulation; every code is exact in f16):
//   S^T [keys x rows] = K [16 keys x 16 d] Q^T, O^T [d x rows] += V^T [16 d x 16 keys] P^T,
// with K and V as the A operand straight from their codes in registers. The order of d inside a
// row and of keys inside a block is free as long as both operands agree: a lane takes the 16-byte
// pieces that make its shared-memory reads conflict-free in the 128-byte swizzle. P^T comes from
// S^T by a register transpose (movmatrix).
//
// Each of the CTA's 8 warps walks its own blocks of 32 keys (one scale each) through its own ring
// of TMA stages, K 4 KB + V 4 KB at hd 128, with its own m, l and O; no warp waits for another
// until the end. The keys are split over CTAs; parts meet in scratch and the part that completes
// the kv head's arrival count merges them. Waits are bounded (PF_ERR_DEVICE_TIMEOUT).
//
// Rounding: P to f16 (the value codes' type in the product), the output to f16; all else f32.
//
// Bound: HBM for long caches (one token of 32/8 heads of 128 over 131,072 e4m3 keys 45.4 us = 5.9 TB/s,
// 0.88 of the measured copy rate; converting e4m3 takes 85 codes a cycle and SM, of which 23 arrive),
// launch, load and merge latency for short ones (6.4 us over 512 keys, int8 9.2 over 8,192). With 16 rows the
// merge of wide parts and the second MMA column block show: four tokens over 8,192 int8 keys 13.1 us.
#include <algorithm>

#include "kv8.cuh"

namespace pf {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int UK = PF_KV8_BLOCK;      // keys per unit: one scale block
constexpr int MAX_SPLIT = 64;         // parts per kv head (one kv head, 16 rows, 131,072 keys: 22.5 us; 128 parts 24.2,
                                      // since one CTA merges them)
// Most rows per kv head of this kernel. 16 rows (four tokens of 32/8 heads of 128, int8) here and in the form
// for chunks: 13.1 and 15.6 us over 8,192 keys, 20.4 and 34.7 over 32,768, 9.1 and 8.2 over 512 (the rule does not
// look at the length).
constexpr int FEW_ROWS = 16;
constexpr float RESCALE_LOG2 = 8.f;

template <int HD, int NB>
struct DSmem {
  static constexpr int NS = 2;              // stages per warp: 128 KB in flight an SM at hd 128 (three gained nothing)
  static constexpr int TILE = UK * HD;      // bytes of a K or V unit
  static constexpr int RING = WARPS * NS * 2 * TILE;
  static constexpr int ROWS = 8 * NB;
  static constexpr int OW = HD + 4;         // floats between rows of the warps' O
  static constexpr int MERGE = WARPS * ROWS * (OW + 2) * 4 + ROWS * MAX_SPLIT * 4;
  static constexpr int BYTES = 1024 + (RING > MERGE ? RING : MERGE) + WARPS * NS * 8;
  static_assert(BYTES <= 232448, "shared memory");
};

struct DecParams {
  Kv8Layer c;
  const __half* q;
  int M, nq, nkv;
  const int* start_dev;
  int start_host;
  float scale_log2;
  int n_split;
  __half* out;
  int* counters;
  float* part;  // [nkv][n_split][rows][HD], then (m, l) per row
  int* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// 16-byte chunk `chunk` of row `row` in a tile that TMA wrote with its row-wide swizzle (128-byte
// rows: chunk ^ row % 8; 64-byte rows: chunk ^ row / 2 % 4).
template <int HD>
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int row, int chunk) {
  return HD == 128 ? tile + row * 128 + ((chunk ^ (row & 7)) << 4) : tile + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

template <int HD, int T, int NB>
__global__ void __launch_bounds__(THREADS, 1)
    attn_kv8_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecParams P) {
  PF_TIMELINE(TL_ATTENTION_KV8);
  using L = DSmem<HD, NB>;
  constexpr int KS = HD / 16;       // k-steps of a score
  constexpr int DT = HD / 16;       // 16-wide tiles of d
  constexpr int ROWS = L::ROWS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_s, last_s;
  volatile int* abort_flag = &abort_s;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = base + warp * (L::NS * 2 * L::TILE);
  const uint32_t bars = base + (L::BYTES - 1024 - WARPS * L::NS * 8) + warp * L::NS * 8;
  griddep_launch_dependents();
  if (threadIdx.x == 0) abort_s = 0;
  if (lane == 0) {
    for (int s = 0; s < L::NS; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  griddep_wait();
  const int start = P.start_dev ? *P.start_dev : P.start_host;
  const int G = P.nq / P.nkv, R = P.M * G;
  const int kvh = blockIdx.y, split = blockIdx.x;
  const int len = start + P.M;                      // keys of the last row
  const int units = (len + UK - 1) / UK;
  // every part has a unit for each warp, as far as the keys go
  const int parts = min(P.n_split, (units + WARPS - 1) / WARPS);
  if (split >= parts) return;
  const int ub = static_cast<int>(static_cast<long long>(units) * split / parts);
  const int ue = static_cast<int>(static_cast<long long>(units) * (split + 1) / parts);
  const int nu = max(0, (ue - ub - warp + WARPS - 1) / WARPS);  // units ub + warp, + 8, ... of this warp
  const float* ks = P.c.ks + static_cast<size_t>(kvh) * P.c.nblk;
  const float* vs = P.c.vs + static_cast<size_t>(kvh) * P.c.nblk;

  // slot of the warp's unit i (clamped to its last), 0 for an entry outside the pool
  auto slot_of = [&](int i) {
    const int s = kv8_slot(P.c, (ub + warp + WARPS * min(i, nu - 1)) * UK);
    if (s < 0 && lane == 0 && P.status) atomicCAS(P.status, 0, PF_ERR_KV_CAPACITY);
    return max(s, 0);
  };
  auto issue = [&](int i, int slot) {
    if (lane == 0) {
      const int s = i % L::NS, row = kvh * P.c.slots + slot;
      const uint32_t dst = ring + s * (2 * L::TILE);
      mbar_arrive_expect_tx(bars + 8 * s, 2 * L::TILE);
      tma_load_2d(dst, &tm_k, 0, row, bars + 8 * s);
      tma_load_2d(dst + L::TILE, &tm_v, 0, row, bars + 8 * s);
    }
  };

  float o[NB][DT][4], m[NB][2], l[NB][2];
  int lim[NB][2];  // last position that the lane's rows (columns 2t, 2t + 1 of each block of 8) may see
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[b][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[b][e] = -INFINITY;
      l[b][e] = 0.f;
      lim[b][e] = start + min(8 * b + 2 * t + e, R - 1) / G;
    }
  }
  int issued = 0, done = 0;
  if (nu > 0) {
    int sl[L::NS + 1];  // slots of units i .. i + NS
#pragma unroll
    for (int s = 0; s <= L::NS; ++s) sl[s] = slot_of(s);
#pragma unroll
    for (int s = 0; s < L::NS; ++s)
      if (s < nu) {
        issue(s, sl[s]);
        ++issued;
      }
    float sk = ks[sl[0] / UK], sv = vs[sl[0] / UK];
    // Q^T as the B operand: row 8 b + g, for each k-step the four d's of the lane's code word
    uint32_t qf[NB][KS][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = 8 * b + g;
      const __half* src = P.q + (static_cast<size_t>(r / G) * P.nq + kvh * G + r % G) * HD;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int d = 16 * (t + 4 * (k >> 2)) + 4 * (k & 3);
        const uint2 x = r < R ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
        qf[b][k][0] = x.x;
        qf[b][k][1] = x.y;
      }
    }
    // key row of the lane's fragment row g within each 8 keys: chosen so that the eight lanes of a
    // shared-memory phase touch eight different 16-byte columns, reading K (rows pi(g), chunks t) and
    // V (rows pi(2t), chunks g)
    auto pi = [](int r) { return (r >> 1) | ((((r >> 1) ^ r) & 1) << 2); };
    const int kg = pi(g), k0 = pi(2 * t), k1 = pi(2 * t + 1);
    for (int i = 0; i < nu; ++i) {
      const int s = i % L::NS;
      const uint32_t kt = ring + s * (2 * L::TILE), vt = kt + L::TILE;
      const float c_k = sk * P.scale_log2;
      const float svc = fminf(fmaxf(sv, 0x1p-60f), 0x1p60f);  // scales lie in 0 .. 2^16: moves values by less than 2^-51
      const float lsv = __log2f(svc), isv = 1.f / svc;
      if (i + 1 < nu) {
        sk = ks[sl[1] / UK];
        sv = vs[sl[1] / UK];
      }
      const int key0 = (ub + warp + WARPS * i) * UK;
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * s, (i / L::NS) & 1, abort_flag))) break;
      ++done;
      if (key0 + UK > len) {  // the last unit: codes past the sequence may be NaN
        for (int x = lane; x < UK * (HD / 16); x += 32) {
          const int row = x / (HD / 16);
          if (key0 + row >= len)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(chunk_at<HD>(vt, row, x % (HD / 16))), "r"(0) : "memory");
        }
        __syncwarp();
      }
      // scores of 32 keys: two tiles of 16
      float sc[NB][2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[b][mt][e] = 0.f;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h) {
          const uint4 ra = lds128(chunk_at<HD>(kt, 16 * mt + kg, t + 4 * h));
          const uint4 rb = lds128(chunk_at<HD>(kt, 16 * mt + 8 + kg, t + 4 * h));
          const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            Kv8<T>::pairs(wa[j], a0, a2);
            Kv8<T>::pairs(wb[j], a1, a3);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816(sc[b][mt], a0, a1, a2, a3, qf[b][4 * h + j][0], qf[b][4 * h + j][1]);
          }
        }
      }
      // u = log2(e) s + log2 sV; hidden keys -inf
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[b][mt][e] = fmaf(sc[b][mt][e], c_k, lsv);
      if (key0 + UK - 1 > start) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + 16 * mt + 8 * (e >> 1) + kg > lim[b][e & 1]) sc[b][mt][e] = -INFINITY;
      }
      float mx[NB][2];
      bool raise = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[b][e] = fmaxf(fmaxf(sc[b][0][e], sc[b][0][e + 2]), fmaxf(sc[b][1][e], sc[b][1][e + 2]));
          raise |= mx[b][e] > m[b][e] + RESCALE_LOG2;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = mx[b][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
            const float mn = fmaxf(m[b][e], x);
            const float alpha = mn == -INFINITY ? 1.f : ex2(m[b][e] - mn);
            m[b][e] = mn;
            l[b][e] *= alpha;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              o[b][d][e] *= alpha;
              o[b][d][e + 2] *= alpha;
            }
          }
      }
      uint32_t pf[NB][2][2];  // P^T as the B operand: [16-key tile][register]
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float n0 = m[b][0] == -INFINITY ? 0.f : m[b][0], n1 = m[b][1] == -INFINITY ? 0.f : m[b][1];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float p0 = ex2(sc[b][mt][2 * hh] - n0), p1 = ex2(sc[b][mt][2 * hh + 1] - n1);
            s0 += p0;
            s1 += p1;
            pf[b][mt][hh] = transpose8x8(f16x2(p0, p1));
          }
        l[b][0] = fmaf(s0, isv, l[b][0]);
        l[b][1] = fmaf(s1, isv, l[b][1]);
      }
      // O^T += V^T P^T: the lane's HD / 8 d's of four keys per 16-key tile
#pragma unroll
      for (int kt2 = 0; kt2 < 2; ++kt2) {
        uint32_t w[4][HD / 32];
        const int rows[4] = {16 * kt2 + k0, 16 * kt2 + k1, 16 * kt2 + 8 + k0, 16 * kt2 + 8 + k1};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (HD == 128) {
            const uint4 v = lds128(chunk_at<HD>(vt, rows[x], g));
            w[x][0] = v.x;
            w[x][1] = v.y;
            w[x][HD / 32 - 2] = v.z;
            w[x][HD / 32 - 1] = v.w;
          } else {
            const uint2 v = lds64(chunk_at<HD>(vt, rows[x], g >> 1) + 8 * (g & 1));
            w[x][0] = v.x;
            w[x][1] = v.y;
          }
        }
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) {
          // bytes of two keys side by side: (k0, k1) and (k0 + 8, k1 + 8)
          uint32_t a[2][4];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            Kv8<T>::pairs(__byte_perm(w[2 * x][j], w[2 * x + 1][j], 0x5140), a[x][0], a[x][1]);
            Kv8<T>::pairs(__byte_perm(w[2 * x][j], w[2 * x + 1][j], 0x7362), a[x][2], a[x][3]);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            mma16816(o[b][2 * j], a[0][0], a[0][1], a[1][0], a[1][1], pf[b][kt2][0], pf[b][kt2][1]);
            mma16816(o[b][2 * j + 1], a[0][2], a[0][3], a[1][2], a[1][3], pf[b][kt2][0], pf[b][kt2][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (i + L::NS < nu) {
        issue(i + L::NS, sl[L::NS]);
        ++issued;
      }
#pragma unroll
      for (int x = 0; x < L::NS; ++x) sl[x] = sl[x + 1];
      sl[L::NS] = slot_of(i + L::NS + 1);
    }
    // after a timeout: let the copies in flight land before shared memory is released
    for (; done < issued; ++done) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bars + 8 * (done % L::NS), (done / L::NS) & 1) && global_timer_ns() - t0 < PF_WAIT_LIMIT_NS) {}
    }
  }
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0 && P.status) atomicCAS(P.status, 0, PF_ERR_DEVICE_TIMEOUT);
    return;
  }

  // the warps' parts meet in shared memory (the rings are idle): O [warp][row][OW], (m, l) [warp][row]
  float* os = reinterpret_cast<float*>(gbase);
  float2* mls = reinterpret_cast<float2*>(os + WARPS * ROWS * L::OW);
  float* wts = reinterpret_cast<float*>(mls + WARPS * ROWS);  // [row][part] merge weights
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * b + 2 * t + e;
      float x = l[b][e];
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      if (g == 0) mls[warp * ROWS + r] = make_float2(m[b][e], x);
      float* dst = os + (warp * ROWS + r) * L::OW + g * (HD / 8);
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<float2*>(dst + 2 * d) = make_float2(o[b][d][e], o[b][d][e + 2]);
    }
  __syncthreads();
  constexpr int LPR = HD / 4;  // threads per row, four columns each
  const int col = (threadIdx.x % LPR) * 4;
  auto store_out = [&](int r, float4 x, float inv) {
    const int tok = r / G;
    uint2 h = make_uint2(f16x2(x.x * inv, x.y * inv), f16x2(x.z * inv, x.w * inv));
    *reinterpret_cast<uint2*>(P.out + (static_cast<size_t>(tok) * P.nq + kvh * G + r % G) * HD + col) = h;
  };
  float* po = P.part + (static_cast<size_t>(kvh) * P.n_split) * ROWS * HD;
  float2* pm = reinterpret_cast<float2*>(P.part + static_cast<size_t>(P.nkv) * P.n_split * ROWS * HD) +
               static_cast<size_t>(kvh) * P.n_split * ROWS;
  for (int r = threadIdx.x / LPR; r < R; r += THREADS / LPR) {
    float mw[WARPS], mr = -INFINITY, lr = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      mw[w] = mls[w * ROWS + r].x;
      mr = fmaxf(mr, mw[w]);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float a = mw[w] == -INFINITY ? 0.f : ex2(mw[w] - mr);
      const float4 x = *reinterpret_cast<const float4*>(os + (w * ROWS + r) * L::OW + col);
      lr = fmaf(a, mls[w * ROWS + r].y, lr);
      acc = make_float4(fmaf(a, x.x, acc.x), fmaf(a, x.y, acc.y), fmaf(a, x.z, acc.z), fmaf(a, x.w, acc.w));
    }
    if (parts == 1) {
      store_out(r, acc, 1.f / lr);
    } else {
      *reinterpret_cast<float4*>(po + (static_cast<size_t>(split) * ROWS + r) * HD + col) = acc;
      if (col == 0) pm[split * ROWS + r] = make_float2(mr, lr);
    }
  }
  if (parts == 1) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last_s = atomicAdd(P.counters + kvh, 1) == parts - 1;
  __syncthreads();
  if (!last_s) return;
  __threadfence();
  // merge: O = sum_s 2^(m_s - m*) O_s / sum_s 2^(m_s - m*) l_s, one warp per row for the weights
  for (int r = warp; r < R; r += WARPS) {
    float2 a[MAX_SPLIT / 32];
    float mr = -INFINITY, lr = 0.f;
#pragma unroll
    for (int x = 0; x < MAX_SPLIT / 32; ++x) {
      const int sp = lane + 32 * x;
      a[x] = sp < parts ? __ldcg(pm + sp * ROWS + r) : make_float2(-INFINITY, 0.f);
      mr = fmaxf(mr, a[x].x);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, w));
#pragma unroll
    for (int x = 0; x < MAX_SPLIT / 32; ++x) {
      a[x].x = a[x].x == -INFINITY ? 0.f : ex2(a[x].x - mr);
      lr = fmaf(a[x].x, a[x].y, lr);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) lr += __shfl_xor_sync(0xffffffffu, lr, w);
#pragma unroll
    for (int x = 0; x < MAX_SPLIT / 32; ++x) wts[r * MAX_SPLIT + lane + 32 * x] = a[x].x / lr;
  }
  __syncthreads();
  for (int r = threadIdx.x / LPR; r < R; r += THREADS / LPR) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = po + static_cast<size_t>(r) * HD + col;
    for (int s0 = 0; s0 < parts; s0 += 8) {
      float4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        x[u] = s0 + u < parts ? __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(s0 + u) * ROWS * HD))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float a = s0 + u < parts ? wts[r * MAX_SPLIT + s0 + u] : 0.f;
        acc = make_float4(fmaf(a, x[u].x, acc.x), fmaf(a, x[u].y, acc.y), fmaf(a, x[u].z, acc.z), fmaf(a, x[u].w, acc.w));
      }
    }
    store_out(r, acc, 1.f);
  }
  if (threadIdx.x == 0) P.counters[kvh] = 0;  // every part is in: ready for the next launch
}

// Parts per kv head of the few-row kernel on `sms` SMs.
int few_splits(const pf_config& c, int sms) { return std::max(1, std::min(MAX_SPLIT, sms / c.n_kv_heads)); }

template <int HD, int T, int NB>
cudaError_t launch_few(const Kv8AttnArgs& a, const Kv8Layer& L, cudaStream_t stream) {
  const pf_config& c = *a.c;
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(c.n_kv_heads) * L.slots;
  if (!encode_tmap_8(&tk, L.k, HD, rows, HD, UK, HD) || !encode_tmap_8(&tv, L.v, HD, rows, HD, UK, HD)) return cudaErrorInvalidValue;
  DecParams p{};
  p.c = L;
  p.q = static_cast<const __half*>(a.q);
  p.M = a.M;
  p.nq = c.n_q_heads;
  p.nkv = c.n_kv_heads;
  p.start_dev = a.start_dev;
  p.start_host = a.start_host;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HD));
  p.n_split = few_splits(c, std::min(device_sm_count(), GEMM_MAX_CTAS));
  p.out = static_cast<__half*>(a.out);
  p.counters = static_cast<int*>(a.scratch);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.scratch) + KV8_COUNTER_BYTES);
  p.status = a.status;
  return launch_pdl(attn_kv8_few_kernel<HD, T, NB>, dim3(p.n_split, c.n_kv_heads), dim3(THREADS), DSmem<HD, NB>::BYTES, stream,
                    tk, tv, p);
}

template <int HD, int T>
cudaError_t launch_rows(const Kv8AttnArgs& a, cudaStream_t stream) {
  const pf_config& c = *a.c;
  const Kv8Layer L = kv8_layer(c, a.k_cache, a.v_cache, a.layer, a.blocks);
  const long long R = static_cast<long long>(a.M) * (c.n_q_heads / c.n_kv_heads);
  if (R <= 8) return launch_few<HD, T, 1>(a, L, stream);
  if (R <= FEW_ROWS) return launch_few<HD, T, 2>(a, L, stream);
  return launch_attention_kv8_tc(a, L, stream);
}

template <int HD, int T>
cudaError_t set_attr_few() {
  cudaError_t e = cudaFuncSetAttribute(attn_kv8_few_kernel<HD, T, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, DSmem<HD, 1>::BYTES);
  cudaError_t f = cudaFuncSetAttribute(attn_kv8_few_kernel<HD, T, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, DSmem<HD, 2>::BYTES);
  return e != cudaSuccess ? e : f;
}

}  // namespace

size_t attention_kv8_scratch_bytes(const pf_config& c, int M) {
  // the counters, then O sums and (max, sum) of each part's rows
  const size_t rows = static_cast<size_t>(std::min<long long>(FEW_ROWS, (static_cast<long long>(M) * (c.n_q_heads / c.n_kv_heads) + 7) / 8 * 8));
  return KV8_COUNTER_BYTES + static_cast<size_t>(c.n_kv_heads) * few_splits(c, GEMM_MAX_CTAS) * rows * (c.head_dim + 2) * sizeof(float);
}

cudaError_t prepare_attention_kv8_kernels() {
  cudaError_t e = cudaSuccess, r;
  if ((r = set_attr_few<128, PF_KV_E4M3>()) != cudaSuccess) e = r;
  if ((r = set_attr_few<128, PF_KV_INT8>()) != cudaSuccess) e = r;
  if ((r = set_attr_few<64, PF_KV_E4M3>()) != cudaSuccess) e = r;
  if ((r = set_attr_few<64, PF_KV_INT8>()) != cudaSuccess) e = r;
  return e;
}

cudaError_t launch_attention_kv8(const Kv8AttnArgs& a, cudaStream_t stream) {
  const pf_config& c = *a.c;
  if (c.head_dim == 128)
    return c.kv_dtype == PF_KV_E4M3 ? launch_rows<128, PF_KV_E4M3>(a, stream) : launch_rows<128, PF_KV_INT8>(a, stream);
  return c.kv_dtype == PF_KV_E4M3 ? launch_rows<64, PF_KV_E4M3>(a, stream) : launch_rows<64, PF_KV_INT8>(a, stream);
}

}  // namespace pf

PF_TIMELINE_SETTER(attention_kv8)
