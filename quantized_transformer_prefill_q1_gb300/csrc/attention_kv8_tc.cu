// attention_kv8_tc.cu — causal GQA attention of a chunk over the 8-bit KV cache on the 5th-generation
// tensor cores (tcgen05 / TMEM): the form for more rows than attention_kv8.cu takes. Mathematics as
// there: with u_j = log2(e) s_j + log2 sV, weights w_j = 2^(u_j - m) = p_j sV up to the row's factor go
// into the product with the value codes, and the softmax's sum takes w_j / sV per scale block; neither
// scale touches a code, and every code is exact in f16.
//
// One CTA = one kv head and up to 256 of its query rows (row = token * G + head in the group) in two
// MMA tiles A and B of 128, so one conversion of the codes serves both and the tensor cores work on
// one tile while the other is in its softmax. Where only 128 rows remain, both tiles hold the same
// rows and take the key tiles in turn (A even, B odd). A cluster of up to 8 CTAs shares one set of
// rows and cuts the keys between them; at the end every CTA leaves its rows' sums, maxima and O in
// its shared memory, and each merges its share of the rows over the cluster.
//
// Warps (16, registers moved between the warpgroups):
//   0        Q tiles by TMA;
//   1        TMEM (S_A, S_B, O_A, O_B of 128 columns each) and the MMAs: per step (tile X, key
//            tile j) O_X += P_X V_j (P over S's columns), then S_X = Q_X K^T of X's next key tile;
//   4..7     codes: loaded a key tile ahead into registers, converted to f16 and written to shared
//            memory in the MMA's 128-byte swizzle, K and V two stages each; the tile's scales;
//   8..15    softmax, one thread per row (8..11 tile A, 12..15 tile B): S from TMEM, running maximum
//            raised only when exceeded by more than 2^8 (then O is rescaled in TMEM), P as f16 back.
// Every wait is bounded; a timeout aborts the CTA and records PF_ERR_DEVICE_TIMEOUT.
#include <algorithm>

#include "kv8.cuh"

namespace pf {
namespace {

constexpr int TQ = 128;  // rows per MMA tile
constexpr int TK = 128;  // keys per tile: one page, four scale blocks
constexpr int ST = 2;    // K and V stages
constexpr int THREADS = 512;
constexpr int SM_THREADS = 256;   // softmax threads
constexpr int DQ_THREADS = 128;   // converting threads
constexpr int NG = TK / PF_KV8_BLOCK;
constexpr int SCR = 4;   // tiles in the ring of scales
constexpr int MAX_CLUSTER = 8;
constexpr float RESCALE_LOG2 = 8.f;
constexpr uint32_t COL_O = 2 * TK;  // TMEM: S_X at X TK, O_X at COL_O + X TK

template <int HD>
struct TSmem {
  static constexpr int Q = TQ * HD * 2;
  static constexpr int KV = TK * HD * 2;
  static constexpr int ROW = HD * 4;  // a row of O at the end, over the idle Q and K tiles
  static constexpr int TILES = 2 * Q + 2 * ST * KV;
  static constexpr int SCALES = SCR * NG * 3 * 4;
  static constexpr int ML = 2 * TQ * 8;
  static constexpr int BARS = 256;
  static constexpr int BYTES = 1024 + TILES + SCALES + ML + BARS;
  static_assert(BYTES <= 232448 && 2 * TQ * ROW <= TILES, "shared memory");
};

struct TcParams {
  Kv8Layer c;
  int M, nq, nkv;
  const int* start_dev;
  int start_host;
  float scale_log2;
  int cs;  // CTAs per cluster
  __half* out;
  int* status;
};

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > PF_WAIT_LIMIT_NS) return;
  }
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
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float ex2t(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2t(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Shared address `a` of CTA `rank` of the cluster, and loads from there.
__device__ __forceinline__ uint32_t map_cta(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ldc64(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ldc128(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int HD, int T>
__global__ void __launch_bounds__(THREADS, 1)
    attn_kv8_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const TcParams P) {
  PF_TIMELINE(TL_ATTENTION_KV8_TC);
  using L = TSmem<HD>;
  constexpr int NH = HD / 64;  // 64-wide swizzle regions along head_dim
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t q_s = base, k_s = q_s + 2 * L::Q, v_s = k_s + ST * L::KV;
  float* scales = reinterpret_cast<float*>(gbase + L::TILES);  // [SCR][NG][c, log2 sV, 1 / sV]
  const uint32_t ml_s = base + L::TILES + L::SCALES;           // [2][TQ] (m, l)
  const uint32_t bar0 = ml_s + L::ML;
  auto k_full = [&](int s) { return bar0 + 8u * s; };
  auto k_empty = [&](int s) { return bar0 + 8u * (2 + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (6 + s); };
  auto s_full = [&](int x) { return bar0 + 8u * (8 + x); };
  auto p_full = [&](int x) { return bar0 + 8u * (10 + x); };
  auto pv_done = [&](int x) { return bar0 + 8u * (12 + x); };
  auto sc_full = [&](int s) { return bar0 + 8u * (14 + s); };
  const uint32_t q_full = bar0 + 8u * 18, drain_bar = bar0 + 8u * 19;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (bar0 + 8u * 20 - base));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bar0 + 8u * 21 - base));
  static_assert(8 * 22 <= L::BARS, "barrier area");

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), DQ_THREADS);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), DQ_THREADS);
      mbar_init(v_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), TQ);
      mbar_init(pv_done(s), 1);
    }
    for (int s = 0; s < SCR; ++s) mbar_init(sc_full(s), 1);
    mbar_init(q_full, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  const int start = P.start_dev ? *P.start_dev : P.start_host;
  const int G = P.nq / P.nkv, BT = TQ / G;
  const int n_set = (P.M + 2 * BT - 1) / (2 * BT);
  const int cs = P.cs, rank = static_cast<int>(blockIdx.x) % cs;
  const int set = n_set - 1 - static_cast<int>(blockIdx.x) / cs;  // longest rows first
  const int kvh = blockIdx.y;
  const int t0 = set * 2 * BT, t1 = min(t0 + 2 * BT, P.M);
  const bool dual = t1 - t0 > BT;  // two row tiles; otherwise both tiles take the one's keys in turn
  const int len = start + t1;      // keys that the last row sees
  const int n_tiles = (len + TK - 1) / TK;
  const int jb = n_tiles * rank / cs;
  const int nt = n_tiles * (rank + 1) / cs - jb;  // this CTA's key tiles jb .. jb + nt - 1
  const int steps = dual ? 2 * nt : nt;           // (tile X = s & 1, key tile dual ? s / 2 : s)
  bool all_ok = true;
  float m = -INFINITY, l = 0.f;

  if (warp < 4) {
    regs_dec<56>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- Q tiles
      mbar_arrive_expect_tx(q_full, (dual ? 2 : 1) * L::Q);
      for (int x = 0; x < (dual ? 2 : 1); ++x)
        for (int h = 0; h < NH; ++h)
          tma_load_3d(q_s + x * L::Q + h * (TQ * 128), &tm_q, h * 64, kvh * G, t0 + x * BT, q_full);
      wait_drain(q_full, 0);  // landed before shared memory is used otherwise, whatever the others do
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = idesc_f16(TQ, TK, 0, 0);
      constexpr uint32_t idesc_o = idesc_f16(TQ, HD, 0, 1);
      auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)) != 0; };
      // S of step s: the tile's previous P has been consumed (waited for by the caller)
      auto issue_s = [&](int s) -> bool {
        const int x = s & 1, j = dual ? s >> 1 : s, st = j & 1;
        if (!wait(k_full(st), (j >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t qx = q_s + (dual ? x * L::Q : 0);
#pragma unroll
        for (int kc = 0; kc < HD / 16; ++kc) {
          const uint32_t off = (kc >> 2) * (TQ * 128) + (kc & 3) * 32;
          umma_f16_ss_warp(tmem + x * TK, sdesc_kmajor_sw128(qx + off), sdesc_kmajor_sw128(k_s + st * L::KV + off), idesc_s, kc > 0);
        }
        umma_commit_warp(s_full(x));
        if (!dual || x == 1) umma_commit_warp(k_empty(st));
        return true;
      };
      bool ok = steps == 0 || wait(q_full, 0);
      if (ok && steps > 0) ok = issue_s(0);
      if (ok && steps > 1) ok = issue_s(1);
      for (int s = 0; s < steps && ok; ++s) {
        const int x = s & 1, i = s >> 1, j = dual ? s >> 1 : s, st = j & 1;
        ok = wait(p_full(x), i & 1) && wait(v_full(st), (j >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kc = 0; kc < TK / 16; ++kc)
          umma_f16_ts_warp(tmem + COL_O + x * TK, tmem + x * TK + 8 * kc, sdesc_mnmajor_sw128(v_s + st * L::KV + kc * 2048, TK * 128),
                           idesc_o, i > 0 || kc > 0);
        umma_commit_warp(pv_done(x));
        if (!dual || x == 1) umma_commit_warp(v_empty(st));
        if (s + 2 < steps) ok = wait(pv_done(x), i & 1) && issue_s(s + 2);  // S overwrites the P that PV read
      }
      if (!ok) {
        umma_commit_warp(drain_bar);
        wait_drain(drain_bar, 0);
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- codes to f16
    regs_dec<120>();
    constexpr int LPR = HD / 16;               // threads per row, 16 codes each
    constexpr int RPP = DQ_THREADS / LPR;      // rows per pass
    constexpr int NP = TK / RPP;
    const int tid = threadIdx.x - 128;
    const int row0 = tid / LPR, c16 = tid % LPR;
    const uint8_t* kb = P.c.k + static_cast<size_t>(kvh) * P.c.slots * HD + c16 * 16;
    const uint8_t* vb = P.c.v + static_cast<size_t>(kvh) * P.c.slots * HD + c16 * 16;
    auto slot_of = [&](int j) {  // of the CTA's tile j
      if (j >= nt) return 0;
      const int s = kv8_slot(P.c, (jb + j) * TK);
      if (s < 0 && tid == 0 && P.status) atomicCAS(P.status, 0, PF_ERR_KV_CAPACITY);
      return max(s, 0);
    };
    // keys past the last row's are zeros: their codes may be NaN
    auto load = [&](const uint8_t* b, int j, int slot, uint4 (&x)[NP]) {
      const int valid = j < nt ? len - (jb + j) * TK : 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int r = row0 + i * RPP;
        x[i] = r < valid ? *reinterpret_cast<const uint4*>(b + static_cast<size_t>(slot + r) * HD) : make_uint4(0, 0, 0, 0);
      }
    };
    const int swap = HD == 128 ? c16 >> 2 : 0;  // the upper region's threads write their odd 16-byte piece first: no bank twice
    auto put = [&](uint32_t tile, const uint4 (&x)[NP]) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int r = row0 + i * RPP;
        uint32_t h[8];
        Kv8<T>::pairs(x[i].x, h[0], h[1]);
        Kv8<T>::pairs(x[i].y, h[2], h[3]);
        Kv8<T>::pairs(x[i].z, h[4], h[5]);
        Kv8<T>::pairs(x[i].w, h[6], h[7]);
        const uint32_t row = tile + (c16 >> 2) * (TK * 128) + r * 128;
        const int ch = (c16 & 3) * 2;
        if (swap) {
          sts128(row + (((ch + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
          sts128(row + ((ch ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
        } else {
          sts128(row + ((ch ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
          sts128(row + (((ch + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
        }
      }
      fence_proxy_async_smem();
    };
    // the scales of tile j's block `lane` (threads 0 .. 3); 1 for a block past the sequence
    auto load_scales = [&](int j, int slot, float& a, float& b) {
      a = b = 1.f;
      if (tid < NG && j < nt && (jb + j) * TK + tid * PF_KV8_BLOCK < len) {
        const size_t at = static_cast<size_t>(kvh) * P.c.nblk + slot / PF_KV8_BLOCK + tid;
        a = P.c.ks[at];
        b = P.c.vs[at];
      }
    };
    uint4 kx[NP], vx[NP];
    float sk, sv;
    int slot = slot_of(0);
    load(kb, 0, slot, kx);
    load(vb, 0, slot, vx);
    load_scales(0, slot, sk, sv);
    for (int j = 0; j < nt; ++j) {
      const int st = j & 1;
      const int next = slot_of(j + 1);
      if (!mbar_wait(k_empty(st), ((j >> 1) & 1) ^ 1, abort_flag)) break;
      if (tid < 32) {
        if (tid < NG) {
          float* dst = scales + ((j & (SCR - 1)) * NG + tid) * 3;
          const float svc = fminf(fmaxf(sv, 0x1p-60f), 0x1p60f);
          dst[0] = fmaxf(sk * P.scale_log2, 1e-37f);  // > 0: a hidden key's -inf stays -inf
          dst[1] = __log2f(svc);
          dst[2] = 1.f / svc;
        }
        __syncwarp();
        if (tid == 0) mbar_arrive(sc_full(j & (SCR - 1)));
      }
      put(k_s + st * L::KV, kx);
      mbar_arrive(k_full(st));
      load(kb, j + 1, next, kx);
      load_scales(j + 1, next, sk, sv);
      if (!mbar_wait(v_empty(st), ((j >> 1) & 1) ^ 1, abort_flag)) break;
      put(v_s + st * L::KV, vx);
      mbar_arrive(v_full(st));
      load(vb, j + 1, next, vx);
    }
  } else {
    // ---------------------------------------------------------------- softmax rows
    regs_inc<168>();
    const int x = (warp - 8) >> 2;
    const int r = 32 * (warp & 3) + lane;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t sbuf = tmem + lane_off + x * TK, obuf = tmem + lane_off + COL_O + x * TK;
    const int tx = t0 + (dual ? x * BT : 0);
    const int pos = start + tx + r / G;
    const int first_pos = start + tx;
    const int n_x = dual ? nt : (nt - x + 1) / 2;
    bool ok = true;
    for (int i = 0; i < n_x; ++i) {
      const int j = dual ? i : 2 * i + x;
      // tcgen05.ld / st are warp-collective: waits are voted on
      ok = __all_sync(0xffffffffu, mbar_wait(sc_full(j & (SCR - 1)), (j / SCR) & 1, abort_flag) && mbar_wait(s_full(x), i & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t v[TK];
#pragma unroll
      for (int g = 0; g < NG; ++g) tmem_ld_32x32b_x32(sbuf + 32 * g, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * g));
      const float* sc = scales + (j & (SCR - 1)) * NG * 3;
      float cg[NG], lg[NG], ig[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        cg[g] = sc[3 * g];
        lg[g] = sc[3 * g + 1];
        ig[g] = sc[3 * g + 2];
      }
      tmem_ld_wait();
      const int key0 = (jb + j) * TK;
      if (key0 + TK - 1 > first_pos) {
        const int lim = pos - key0;  // last visible column
#pragma unroll
        for (int e = 0; e < TK; ++e)
          if (e > lim) v[e] = 0xff800000u;  // -inf
      }
      float um = -INFINITY;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(v[32 * g + e]);
#pragma unroll
        for (int e = 4; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(v[32 * g + e]));
        um = fmaxf(um, fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), cg[g], lg[g]));
      }
      const bool need = um > m + RESCALE_LOG2;  // the first tile's too
      if (__any_sync(0xffffffffu, need)) {
        const float alpha = need ? ex2t(m - um) : 1.f;
        l *= alpha;
        if (need) m = um;
        if (i > 0) {
          // PV of the previous step completed before this S was issued; the wait only orders it
          if (!__all_sync(0xffffffffu, mbar_wait(pv_done(x), (i - 1) & 1, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(obuf + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_32x32b_x32(obuf + 32 * c, o);
          }
        }
      }
      const float mm = m == -INFINITY ? 0.f : m;  // a row that has seen no key: every weight 2^-inf = 0
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float off = lg[g] - mm;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float p0 = ex2t(fmaf(__uint_as_float(v[32 * g + e]), cg[g], off));
          const float p1 = ex2t(fmaf(__uint_as_float(v[32 * g + e + 1]), cg[g], off));
          sum[e & 2] += p0;
          sum[(e & 2) + 1] += p1;
          v[16 * g + e / 2] = f16x2t(p0, p1);
        }
        l = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), ig[g], l);
      }
      tmem_st_32x32b_x32(sbuf, *reinterpret_cast<uint32_t(*)[32]>(v));
      tmem_st_32x32b_x32(sbuf + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_full(x));
    }
    // ---------------------------------------------------------------- O, m, l to shared memory
    if (ok && n_x > 0) ok = mbar_wait(pv_done(x), (n_x - 1) & 1, abort_flag);
    all_ok = bar_and(1, SM_THREADS, ok);  // every MMA that reads the tiles is done
    if (all_ok) {
      tc_fence_after();
      // 16-byte piece q of a row at piece q ^ (row % (HD / 4)): a warp's rows hit different banks
      const uint32_t dst = base + (x * TQ + r) * L::ROW;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        if (n_x > 0) {
          tmem_ld_32x32b_x32(obuf + 32 * c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          sts128(dst + (((8 * c + q) ^ (r & (HD / 4 - 1))) << 4), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      }
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml_s + (x * TQ + r) * 8), "f"(m), "f"(l) : "memory");
    }
  }

  // every CTA of the cluster has its rows in shared memory; each merges its share of them
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  if (warp >= 8 && all_ok) {
    const int rows = dual ? 2 * TQ : TQ, nsrc = dual ? cs : 2 * cs;  // sources of a row: ranks, and both tiles when they shared the keys
    const int rb = rows * rank / cs, re = rows * (rank + 1) / cs;
    for (int row = rb + warp - 8; row < re; row += 8) {
      const int t = t0 + row / G;
      if (t >= t1) break;
      auto src_row = [&](int s) { return dual ? row : (s & 1) * TQ + row; };
      auto src_cta = [&](int s) { return static_cast<uint32_t>(dual ? s : s >> 1); };
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < nsrc) ml = ldc64(map_cta(ml_s + src_row(lane) * 8, src_cta(lane)));
      float mr = ml.x;
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, w));
      mr = __shfl_sync(0xffffffffu, mr, 0);
      const float a = ml.x == -INFINITY ? 0.f : ex2t(ml.x - mr);
      float lr = a * ml.y;
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) lr += __shfl_xor_sync(0xffffffffu, lr, w);
      const float wgt = a / __shfl_sync(0xffffffffu, lr, 0);
      __half* dst = P.out + (static_cast<size_t>(t) * P.nq + kvh * G + row % G) * HD;
      const uint32_t piece = static_cast<uint32_t>(lane & (HD / 4 - 1));  // four columns a lane (hd 64: lanes 16.. repeat)
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < nsrc; ++s) {
        const float w = __shfl_sync(0xffffffffu, wgt, s);
        const int sr = src_row(s);
        const float4 o = ldc128(map_cta(base + sr * L::ROW + ((piece ^ (sr & (HD / 4 - 1))) << 4), src_cta(s)));
        if (w != 0.f) acc = make_float4(fmaf(w, o.x, acc.x), fmaf(w, o.y, acc.y), fmaf(w, o.z, acc.z), fmaf(w, o.w, acc.w));
      }
      if (HD == 128 || lane < 16) *reinterpret_cast<uint2*>(dst + 4 * piece) = make_uint2(f16x2t(acc.x, acc.y), f16x2t(acc.z, acc.w));
    }
  }
  __syncwarp();
  cluster_sync_all();  // nobody leaves while others read its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag && P.status) atomicCAS(P.status, 0, PF_ERR_DEVICE_TIMEOUT);
}

template <int HD, int T>
cudaError_t launch(const Kv8AttnArgs& a, const Kv8Layer& L, cudaStream_t stream) {
  const pf_config& c = *a.c;
  const int G = c.n_q_heads / c.n_kv_heads, BT = TQ / G;
  CUtensorMap tq;
  const uint64_t qd[3] = {static_cast<uint64_t>(HD), static_cast<uint64_t>(c.n_q_heads), static_cast<uint64_t>(a.M)};
  const uint64_t qs[2] = {static_cast<uint64_t>(HD) * 2, static_cast<uint64_t>(c.n_q_heads) * HD * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(BT)};
  if (!encode_tmap_16(&tq, 0, 3, a.q, qd, qs, qb)) return cudaErrorInvalidValue;
  TcParams p{};
  p.c = L;
  p.M = a.M;
  p.nq = c.n_q_heads;
  p.nkv = c.n_kv_heads;
  p.start_dev = a.start_dev;
  p.start_host = a.start_host;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HD));
  p.out = static_cast<__half*>(a.out);
  p.status = a.status;
  const int sets = (a.M + 2 * BT - 1) / (2 * BT);
  // as many CTAs on a set of rows as fill the GPU once
  const int cs = std::max(1, std::min<int>(MAX_CLUSTER, device_sm_count() / (sets * c.n_kv_heads)));
  p.cs = cs;
  return launch_pdl_cluster(attn_kv8_tc_kernel<HD, T>, dim3(cs * sets, c.n_kv_heads), dim3(THREADS), TSmem<HD>::BYTES, stream, cs,
                            tq, p);
}

template <int HD, int T>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(attn_kv8_tc_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, TSmem<HD>::BYTES);
}

}  // namespace

cudaError_t prepare_attention_kv8_tc_kernels() {
  cudaError_t e = cudaSuccess, r;
  if ((r = set_attr<128, PF_KV_E4M3>()) != cudaSuccess) e = r;
  if ((r = set_attr<128, PF_KV_INT8>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, PF_KV_E4M3>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, PF_KV_INT8>()) != cudaSuccess) e = r;
  return e;
}

cudaError_t launch_attention_kv8_tc(const Kv8AttnArgs& a, const Kv8Layer& L, cudaStream_t stream) {
  const pf_config& c = *a.c;
  if (c.head_dim == 128) return c.kv_dtype == PF_KV_E4M3 ? launch<128, PF_KV_E4M3>(a, L, stream) : launch<128, PF_KV_INT8>(a, L, stream);
  return c.kv_dtype == PF_KV_E4M3 ? launch<64, PF_KV_E4M3>(a, L, stream) : launch<64, PF_KV_INT8>(a, L, stream);
}

}  // namespace pf

PF_TIMELINE_SETTER(attention_kv8_tc)
