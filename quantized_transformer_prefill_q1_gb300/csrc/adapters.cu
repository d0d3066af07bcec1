// adapters.cu — low-rank adapters of many sequences beside a shared projection:
// out[m] = base[m] + scale[a] (x[m] A_a^T) B_a^T with a the adapter of row m's sequence.
//
// One kernel: a cluster of 8 CTAs takes RT rows of one sequence. The CTAs split K for h = x A^T (m16n8k16 on tiles of x
// and A that TMA brings through rings), add their shares through distributed shared memory, and split N for h B^T, whose
// accumulators go straight onto base: x, base and out pass once, h never leaves the chip. A CTA's 8 warps are KW = 8 / MG
// groups over K (MG = RT / 16 warps with 16 rows each), every group with a ring of its own.
//
// What bounds it: few rows the chain of launch, first copies, the cluster's barrier and the second product (one token, rank 16,
// 4,096 -> 4,096: 4.1 us; 24 of them with 16 adapters, 4,096 -> 6,144: 5.4 us). Many rows the copies, since every tile of rows
// reads its A and B again, and a CTA's phases follow one another: four chunks of 300 .. 700 rows, rank 64, 12,288 -> 4,096, take
// 33.5 us, 13 the first product (x and A, 100 MB), 6 the sum over the cluster, 12 the second (B, base and out, 81 MB). The
// products are 4 GFLOP: warp MMAs do. Tried and not kept: tiles of 128 rows (49 .. 57 us), base by TMA or two tiles ahead in registers (33.5 .. 34.5).
//
// Rounding: x A^T is summed in f32 and enters the second product as two f16 terms, hi + lo (22 bits), after a power of
// two that brings the row's largest to 2^13 .. 2^14, so that neither its overflow nor its underflow counts; all else f32.
#include <cuda_fp16.h>

#include <algorithm>

#include "batch.cuh"

namespace pf {
namespace {

constexpr int CL = 8;  // CTAs of a cluster
constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int KB = 64;  // K of a stage: 128 bytes of a row
constexpr uint32_t NO_SHARE = 0x7fc0dead;  // a NaN that no addition gives: in the place of a CTA's sums after a wait that gave up

// RT rows a cluster, rank up to 16 KS
template <int RT, int KS>
struct ASmem {
  static constexpr int R = 16 * KS;
  static constexpr int MG = RT / 16, KW = WARPS / MG;
  static constexpr int STAGE = (RT + R) * 128;
  // stages of a group's ring: up to 96 KB a CTA, two CTAs an SM up to rank 64
  static constexpr int WS = RT == 16 ? (KS == 1 ? 3 : (KS == 2 ? 2 : 1)) : (KS <= 2 ? 4 : 2);
  static constexpr int NS = KW * WS;
  static constexpr int RED = KW * RT * R * 4;   // the groups' sums, over the rings
  static constexpr int PART = RT * R * 4;       // the CTA's
  static constexpr int RING = NS * STAGE > RED + PART ? NS * STAGE : RED + PART;
  static constexpr int PITCH = (4 * R + 127) / 128 * 128 + 32;  // bytes between rows of h: conflict-free 8-byte reads of 4 rows
  static constexpr int BYTES = 1024 + RING + RT * PITCH + RT * 4 + NS * 8;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct AdapterParams {
  BatchDev B;
  const float* base;
  int64_t ldb;
  float* out;
  int64_t ldo;
  int K, N, rank, count;
  const int* adapter;
  const __half* wb;
  const float* scale;
  int* status;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// 16-byte chunk of a row in a tile of 128-byte rows (128-byte swizzle)
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int row, int chunk) { return tile + row * 128 + ((chunk ^ (row & 7)) << 4); }
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
// Two f32 values as f16 pairs hi + lo.
__device__ __forceinline__ void split(float2 v, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  const float2 b = __half22float2(h);
  const float rx = v.x - b.x, ry = v.y - b.y;  // 0 beside an infinity or a NaN
  const __half2 l = __floats2half2_rn(fabsf(rx) <= 65504.f ? rx : 0.f, fabsf(ry) <= 65504.f ? ry : 0.f);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ bool bar_and(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

template <int RT, int KS>
__global__ void __launch_bounds__(THREADS, KS == 8 ? 1 : 2)
    adapters_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_a, const AdapterParams P) {
  PF_TIMELINE(TL_ADAPTERS);
  using L = ASmem<RT, KS>;
  constexpr int MG = L::MG, KW = L::KW, R = L::R;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  const uint32_t raw = smem_u32(smem_raw), ring = (raw + 1023u) & ~1023u;
  uint8_t* gring = smem_raw + (ring - raw);
  float* red = reinterpret_cast<float*>(gring);
  float* part = reinterpret_cast<float*>(gring + L::RED);
  uint8_t* h_s = gring + L::RING;  // [row][PITCH]: hi of the R columns, then lo
  float* rs_s = reinterpret_cast<float*>(h_s + RT * L::PITCH);
  const uint32_t bars = ring + L::RING + RT * L::PITCH + RT * 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int c = blockIdx.x, b = blockIdx.z, t0 = blockIdx.y * RT;
  griddep_launch_dependents();
  if (threadIdx.x < L::NS) mbar_init(bars + 8 * threadIdx.x, 1);
  if (threadIdx.x == 0) abort_s = 0;
  fence_barrier_init();
  fence_proxy_async_smem();
  __syncthreads();
  griddep_wait();
  const SeqRows s = batch_seq(P.B, b, false);
  int a = P.adapter[b];
  if (c == 0 && t0 == 0 && threadIdx.x == 0) {
    if (s.err != PF_OK) batch_record(P.status, s.err);
    if (a < -1 || a >= P.count) batch_record(P.status, PF_ERR_INVALID_ARG);
  }
  if (a < -1 || a >= P.count) a = -1;
  const int rows = min(RT, s.n - t0);  // the same in every CTA of the cluster, and so is what follows from it
  if (rows <= 0) return;
  const float* base = P.base + (s.at + t0) * P.ldb;
  float* out = P.out + (s.at + t0) * P.ldo;
  if (a < 0) {
    if (P.base == P.out) return;
    const int n4 = P.N / 4;
    for (int i = c * THREADS + threadIdx.x; i < rows * n4; i += CL * THREADS) {
      const int r = i / n4, q = i - r * n4;
      reinterpret_cast<float4*>(out + r * P.ldo)[q] = reinterpret_cast<const float4*>(base + r * P.ldb)[q];
    }
    return;
  }

  // Columns of the second product, 32 at a time (see below): groups gb .. ge - 1 of this CTA.
  const int groups = (P.N + 31) / 32;
  const int gb = groups * c / CL, ge = groups * (c + 1) / CL;

  // ------------------------------------------------------------------ h = x A^T over this CTA's share of K
  const int mg = warp % MG, kw = warp / MG;
  const int chunks = (P.K + KB - 1) / KB;
  const int kb = chunks * c / CL + kw, ke = chunks * (c + 1) / CL;  // chunks kb, kb + KW, .. of this group
  const bool leader = mg == 0 && lane == 0;
  int issued = 0;
  auto issue = [&](int k) {
    const int st = kw * L::WS + issued % L::WS;
    const uint32_t dst = ring + st * L::STAGE, bar = bars + 8 * st;
    mbar_arrive_expect_tx(bar, (RT + P.rank) * 128);
    tma_load_2d(dst, &tm_x, k * KB, s.at + t0, bar);
    tma_load_2d(dst + RT * 128, &tm_a, k * KB, a * P.rank, bar);
    ++issued;
  };
  if (leader)
    for (int i = 0; i < L::WS && kb + KW * i < ke; ++i) issue(kb + KW * i);
  float acc[2 * KS][4];
#pragma unroll
  for (int j = 0; j < 2 * KS; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  const int xrow = 16 * mg + (lane & 7) + ((lane >> 3) & 1) * 8, xch = lane >> 4;
  const int arow = (lane & 7) + (lane >> 4) * 8, ach = (lane >> 3) & 1;
  bool ok = true;
  for (int k = kb, i = 0; k < ke; k += KW, ++i) {
    const int st = kw * L::WS + i % L::WS;
    ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * st, (i / L::WS) & 1, abort_flag));
    if (ok) {
      const uint32_t xt = ring + st * L::STAGE, at = xt + RT * 128;
#pragma unroll
      for (int ks = 0; ks < KB / 16; ++ks) {
        uint32_t x[4];
        ldsm4(x, chunk_at(xt, xrow, 2 * ks + xch));
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          uint32_t w[4];
          ldsm4(w, chunk_at(at, 16 * j + arow, 2 * ks + ach));
          mma16816(acc[2 * j], x, w[0], w[1]);
          mma16816(acc[2 * j + 1], x, w[2], w[3]);
        }
      }
    }
    // the whole group has read the stage
    if (MG == 1) {
      __syncwarp();
    } else {
      ok = bar_and(1 + kw, 32 * MG, ok);
    }
    if (!ok) break;
    if (leader && k + KW * L::WS < ke) issue(k + KW * L::WS);
  }
  if (!ok && leader) {  // let the copies in flight land before their place is used again
    for (int i = max(0, issued - L::WS); i < issued; ++i) {
      const uint64_t w0 = global_timer_ns();
      while (!mbar_try_wait(bars + 8 * (kw * L::WS + i % L::WS), (i / L::WS) & 1) && global_timer_ns() - w0 < PF_WAIT_LIMIT_NS) {}
    }
  }
  __syncthreads();  // the rings are idle
#pragma unroll
  for (int j = 0; j < 2 * KS; ++j) {
    float* dst = red + ((kw * RT) + 16 * mg + g) * R + 8 * j + 2 * t;
    *reinterpret_cast<float2*>(dst) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(dst + 8 * R) = make_float2(acc[j][2], acc[j][3]);
  }
  __syncthreads();
  const bool complete = !*abort_flag;
  for (int i = threadIdx.x; i < RT * R / 4; i += THREADS) {
    float4 v = reinterpret_cast<const float4*>(red)[i];
#pragma unroll
    for (int w = 1; w < KW; ++w) {
      const float4 y = reinterpret_cast<const float4*>(red)[w * (RT * R / 4) + i];
      v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
    }
    if (!complete) v.x = v.y = v.z = v.w = __uint_as_float(NO_SHARE);
    reinterpret_cast<float4*>(part)[i] = v;
  }

  // ------------------------------------------------------------------ B and base of the warp's first columns, while the shares meet
  // Pair p (16 columns) of MMA tiles; n = g of tile u is column 16 p + 4 (g / 2) + g % 2 + 2 u, so that a lane's four
  // accumulators of a row are four columns in a line. k runs as 4 t .. 4 t + 3 in both operands.
  const __half* wb = P.wb + static_cast<size_t>(a) * P.N * P.rank;
  uint2 wf[4][KS];
  auto load_b = [&](int gi) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int col = 32 * gi + 16 * (u >> 1) + 4 * (g >> 1) + (g & 1) + 2 * (u & 1);
#pragma unroll
      for (int k = 0; k < KS; ++k)
        wf[u][k] = col < P.N && 16 * k + 4 * t < P.rank
                       ? *reinterpret_cast<const uint2*>(wb + static_cast<size_t>(col) * P.rank + 16 * k + 4 * t)
                       : make_uint2(0u, 0u);
    }
  };
  auto load_base = [&](int gi, int m, float4 (&y)[2][2]) {  // [row half][pair]
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int r = 16 * m + 8 * hh + g, col = 32 * gi + 16 * p + 4 * t;
        y[hh][p] = r < rows && col < P.N ? *reinterpret_cast<const float4*>(base + r * P.ldb + col) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
  };
  float4 y[2][2];
  if (gb + warp < ge) {
    load_b(gb + warp);
    load_base(gb + warp, 0, y);
  }

  // ------------------------------------------------------------------ the cluster's sum, a warp a row, a lane two columns
  // RT 16: every CTA adds all rows for itself (one barrier of latency); RT 64: CTA c adds rows 8 c .. 8 c + 7 for all.
  __syncwarp();
  cluster_arrive_release();
  cluster_wait();
  const float scale = P.scale[a];
  constexpr int OWN = RT == 16 ? RT : RT / CL;
  for (int i = warp; i < OWN; i += WARPS) {
    const int r = RT == 16 ? i : c * OWN + i;
    if (r >= rows) break;
    constexpr int PER = (R + 63) / 64;
    float2 v[PER];
    float big = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int col = 2 * lane + 64 * e;
      v[e] = make_float2(0.f, 0.f);
      if (col < P.rank) {
        const uint32_t at = smem_u32(part + r * R + col);
        float2 y2[CL];
#pragma unroll
        for (int w = 0; w < CL; ++w) y2[w] = ld_cluster(remote(at, w));
        bool lacking = false;
#pragma unroll
        for (int w = 0; w < CL; ++w) {
          lacking |= __float_as_uint(y2[w].x) == NO_SHARE;
          v[e] = make_float2(v[e].x + y2[w].x, v[e].y + y2[w].y);
        }
        if (lacking) {  // row 0 says so to every CTA, whether it adds rows or not
          for (int w = 0; w < CL; ++w) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(smem_u32(&abort_s), w)), "r"(1) : "memory");
        }
      }
      big = fmaxf(big, fmaxf(fabsf(v[e].x), fabsf(v[e].y)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    // 2^up brings the largest into 2^13 .. 2^14; the power is kept within f32's own range
    int up = 0;
    if (big > 0.f && big <= 3.4028235e38f) up = min(max(13 - ilogbf(big), -100), 100);
    const float f = __int_as_float((up + 127) << 23), back = __int_as_float((127 - up) << 23) * scale;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int col = 2 * lane + 64 * e;
      if (col >= R) continue;
      uint32_t hi, lo;
      split(make_float2(v[e].x * f, v[e].y * f), hi, lo);
      uint8_t* at = h_s + r * L::PITCH + 2 * col;
      if (RT == 16) {
        *reinterpret_cast<uint32_t*>(at) = hi;
        *reinterpret_cast<uint32_t*>(at + 2 * R) = lo;
      } else {
#pragma unroll
        for (int w = 0; w < CL; ++w) {
          const uint32_t dst = remote(smem_u32(at), w);
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst), "r"(hi) : "memory");
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + 2 * R), "r"(lo) : "memory");
        }
      }
    }
    if (RT == 16) {
      if (lane == 0) rs_s[r] = back;
    } else if (lane < CL) {
      const uint32_t dst = remote(smem_u32(rs_s + r), lane);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(back) : "memory");
    }
  }
  __syncwarp();
  cluster_arrive_release();  // this CTA has read the others' shares (RT 64: and written theirs)
  if (RT == 16)
    __syncthreads();
  else
    cluster_wait();

  // ------------------------------------------------------------------ out = base + scale h B^T
  const bool whole = !*abort_flag;  // else the sum lacks a share, and out stays as it is
  for (int gi = gb + warp; whole && gi < ge; gi += WARPS) {
#pragma unroll 1
    for (int m = 0; m < MG; ++m) {
      if (16 * m >= rows) break;
      float d[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[u][e] = 0.f;
      const uint8_t* hr = h_s + (16 * m + g) * L::PITCH;
#pragma unroll
      for (int half = 1; half >= 0; --half)  // lo first: the small terms add up before the large
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint2 v0 = *reinterpret_cast<const uint2*>(hr + 2 * R * half + 32 * k + 8 * t);
          const uint2 v1 = *reinterpret_cast<const uint2*>(hr + 8 * L::PITCH + 2 * R * half + 32 * k + 8 * t);
          const uint32_t x[4] = {v0.x, v1.x, v0.y, v1.y};
#pragma unroll
          for (int u = 0; u < 4; ++u) mma16816(d[u], x, wf[u][k].x, wf[u][k].y);
        }
      // the next rows' base, or the next columns' B and base, are requested before this tile's results are stored
      float4 z[2][2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int p = 0; p < 2; ++p) z[hh][p] = y[hh][p];
      if (m + 1 < MG && 16 * (m + 1) < rows) {
        load_base(gi, m + 1, y);
      } else if (gi + WARPS < ge) {
        load_b(gi + WARPS);
        load_base(gi + WARPS, 0, y);
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = 16 * m + 8 * hh + g;
        if (r >= rows) continue;
        const float f = rs_s[r];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int col = 32 * gi + 16 * p + 4 * t;
          if (col >= P.N) continue;
          const float4 q = z[hh][p];
          *reinterpret_cast<float4*>(out + r * P.ldo + col) =
              make_float4(fmaf(f, d[2 * p][2 * hh], q.x), fmaf(f, d[2 * p][2 * hh + 1], q.y), fmaf(f, d[2 * p + 1][2 * hh], q.z),
                          fmaf(f, d[2 * p + 1][2 * hh + 1], q.w));
        }
      }
    }
  }
  if (RT == 16) cluster_wait();  // the others have read this CTA's share
  if (threadIdx.x == 0 && *abort_flag) batch_record(P.status, PF_ERR_DEVICE_TIMEOUT);
}

template <int RT, int KS>
cudaError_t launch(const AdapterArgs& a, cudaStream_t stream) {
  using L = ASmem<RT, KS>;
  CUtensorMap tx, ta;
  const uint64_t xd[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.b->n_rows)}, xs[1] = {static_cast<uint64_t>(a.ldx) * 2};
  const uint64_t ad[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.n_adapters) * a.rank}, as[1] = {static_cast<uint64_t>(a.K) * 2};
  const uint32_t xb[2] = {KB, RT}, ab[2] = {KB, static_cast<uint32_t>(a.rank)};
  if (!encode_tmap_16(&tx, 0, 2, a.x, xd, xs, xb) || !encode_tmap_16(&ta, 0, 2, a.wa, ad, as, ab)) return cudaErrorInvalidValue;
  AdapterParams p{};
  p.B.n_seq = a.b->n_seq;
  p.B.n_rows = a.b->n_rows;
  p.B.max_rows = a.b->max_rows;
  p.B.row_begin = a.b->row_begin_dev;
  p.base = a.base;
  p.ldb = a.ld_base;
  p.out = a.out;
  p.ldo = a.ld_out;
  p.K = a.K;
  p.N = a.N;
  p.rank = a.rank;
  p.count = a.n_adapters;
  p.adapter = a.adapter;
  p.wb = static_cast<const __half*>(a.wb);
  p.scale = a.scale;
  p.status = a.status;
  const int tiles = (std::min(a.b->max_rows, a.b->n_rows) + RT - 1) / RT;
  return launch_pdl_cluster(adapters_kernel<RT, KS>, dim3(CL, tiles, a.b->n_seq), dim3(THREADS), L::BYTES, stream, CL, tx, ta, p);
}

template <int RT>
cudaError_t launch_rank(const AdapterArgs& a, cudaStream_t stream) {
  if (a.rank <= 16) return launch<RT, 1>(a, stream);
  if (a.rank <= 32) return launch<RT, 2>(a, stream);
  if (a.rank <= 64) return launch<RT, 4>(a, stream);
  return launch<RT, 8>(a, stream);
}

template <int RT, int KS>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(adapters_kernel<RT, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, ASmem<RT, KS>::BYTES);
}

}  // namespace

cudaError_t prepare_adapters_kernels() {
  cudaError_t e = cudaSuccess, r;
  if ((r = set_attr<16, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr<16, 2>()) != cudaSuccess) e = r;
  if ((r = set_attr<16, 4>()) != cudaSuccess) e = r;
  if ((r = set_attr<16, 8>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, 2>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, 4>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, 8>()) != cudaSuccess) e = r;
  return e;
}

cudaError_t launch_adapters(const AdapterArgs& a, cudaStream_t stream) {
  // 16 rows a cluster spread few rows over more SMs and need one barrier less; A and B are then read for every 16 rows, so
  // they pay while all clusters are resident at once (two CTAs an SM up to rank 64), or where a sequence has no more.
  // Both sides measured, 16 against 64 rows, rank 64, 4,096 -> 6,144: eight sequences of 64 rows (256 CTAs of 304) 13.9 and 20.3 us,
  // one of 300 13.7 and 17.2, 24 of 32 (384 CTAs) 24.4 and 20.1, one of 1,200 (600) 37.5 and 28.2; 32 sequences of 16 13.9 and 16.3.
  const int rows = std::min(a.b->max_rows, a.b->n_rows);
  const int tiles = std::min(a.b->n_seq * ((rows + 15) / 16), a.b->n_rows / 16 + a.b->n_seq);  // of 16 rows, at most
  const int resident = (a.rank <= 64 ? 2 : 1) * device_sm_count();
  return rows <= 16 || tiles * CL <= resident ? launch_rank<16>(a, stream) : launch_rank<64>(a, stream);
}

}  // namespace pf

PF_TIMELINE_SETTER(adapters)
