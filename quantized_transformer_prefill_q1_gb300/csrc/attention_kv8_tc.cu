// attention_kv8_tc.cu — causal GQA attention of a chunk over the 8-bit KV cache on the 5th-generation
// tensor cores (tcgen05 / TMEM): the form for more rows than attention_kv8.cu takes. Mathematics as
// there: with u_j = log2(e) s_j + log2 sV, weights w_j = 2^(u_j - m) = p_j sV up to the row's factor go
// into the product with the value codes, and the softmax's sum takes w_j / sV per scale block; neither
// scale touches a code, and every code is exact in f16.
//
// One CTA = one kv head and 128 of its query rows (row = token * G + head in the group) against its
// share of the key tiles: a cluster of CTAs shares the rows and cuts the keys between them; at the end
// every CTA leaves its rows' sums, maxima and O in its shared memory, and each merges its share of the
// rows over the cluster. No scratch and no second kernel.
//
// Warps (20):
//   0, 2     copies: the Q tile and the K codes (0), the V codes (2), 16 KB a tile at hd 128 into two
//            stages each;
//   1        TMEM (three S buffers of 128 columns and O) and the MMAs: S_0, S_1, then per key tile
//            S_{j+2} = Q K_{j+2}^T and O += P_j V_j (P over S's columns);
//   4..7     K, 8..11 V: codes converted to f16 into shared memory in the MMA's 128-byte swizzle, two
//            stages each; the scales;
//   12..15   softmax of the even key tiles, 16..19 of the odd ones, one thread per row, so that one
//            tile's exponentials run while the next one's maximum is taken. The two share each row's
//            running maximum: a tile's decision to raise it (only when exceeded by more than 2^8; O is
//            then rescaled in TMEM) follows the previous tile's, warp by warp through a barrier; the
//            rest runs side by side. A row's 128 scores stay in registers, which the other
//            warpgroups give up (setmaxnreg).
// Every wait is bounded; a timeout aborts the CTA and records PF_ERR_DEVICE_TIMEOUT.
#include <algorithm>

#include "kv8.cuh"

namespace pf {
namespace {

constexpr int TQ = 128;  // rows per CTA
constexpr int TK = 128;  // keys per tile: one page, four scale blocks
constexpr int ST = 2;    // K and V stages
constexpr int NSB = 3;   // S / P buffers
constexpr int THREADS = 640;
constexpr int SM_THREADS = 256;   // softmax threads: two groups of one per row
constexpr int DQ_THREADS = 128;   // converting threads, K and V each
constexpr int NG = TK / PF_KV8_BLOCK;
constexpr int SCR = 8;   // tiles in the ring of scales (K's conversion may run 4 tiles ahead of a softmax)
constexpr int MAX_CLUSTER = 8;
constexpr float RESCALE_LOG2 = 8.f;
constexpr uint32_t COL_O = NSB * TK;  // TMEM: S buffer b at b TK, O at COL_O

template <int HD>
struct TSmem {
  static constexpr int Q = TQ * HD * 2;
  static constexpr int KV = TK * HD * 2;
  static constexpr int ROW = HD * 4;  // a row of O at the end, over the idle Q and K tiles
  static constexpr int CODES = TK * HD;  // codes of a K or V tile
  static constexpr int TILES = Q + 2 * ST * KV;
  static constexpr int RINGS = 2 * ST * CODES;
  static constexpr int SCALES = SCR * NG * 4 * 4;
  static constexpr int MAXIMA = TQ * 4;
  static constexpr int BARS = 384;
  static constexpr int BYTES = 1024 + TILES + RINGS + SCALES + MAXIMA + BARS;
  // at the end, over the idle tiles: O; over the idle rings: (m, l) of each row, the groups' sums, the
  // weights of the parts
  static_assert(BYTES <= 232448 && TQ * ROW <= TILES && TQ * (8 + 2 * 4 + MAX_CLUSTER * 4) <= RINGS, "shared memory");
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
// mbar_wait with the hardware suspending the thread for up to 20 us a try: 20 warps that poll would take
// issue slots from those that work.
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > PF_WAIT_LIMIT_NS) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
// Registers a thread from here on (all warps of a warpgroup alike): 128 x (32 + 56 + 56 + 168 + 168)
// is the 640 x 96 that the CTA is launched with.
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// x * c + o on two values at once, and x + y.
__device__ __forceinline__ void fma2(float& a, float& b, float c, float o) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(o));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
// 16 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <int HD, int T>
__global__ void __launch_bounds__(THREADS, 1)
    attn_kv8_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const TcParams P) {
  PF_TIMELINE(TL_ATTENTION_KV8_TC);
  using L = TSmem<HD>;
  constexpr int NH = HD / 64;  // 64-wide swizzle regions along head_dim
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t q_s = base, k_s = q_s + L::Q, v_s = k_s + ST * L::KV;
  const uint32_t kc_s = base + L::TILES, vc_s = kc_s + ST * L::CODES;
  float4* scales = reinterpret_cast<float4*>(gbase + L::TILES + L::RINGS);  // [SCR][NG] (log2(e) sK / sqrt(hd), log2 sV, 1 / sV, -)
  const uint32_t sc_s = base + L::TILES + L::RINGS;
  volatile float* run_m = reinterpret_cast<volatile float*>(gbase + L::TILES + L::RINGS + L::SCALES);  // [TQ] running maxima
  const uint32_t ml_s = kc_s;  // [TQ] (m, l)
  volatile float* sums = reinterpret_cast<volatile float*>(gbase + L::TILES + TQ * 8);  // [2][TQ]
  const uint32_t bar0 = base + L::TILES + L::RINGS + L::SCALES + L::MAXIMA;
  auto k_full = [&](int s) { return bar0 + 8u * s; };
  auto k_empty = [&](int s) { return bar0 + 8u * (2 + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (6 + s); };
  auto s_full = [&](int b) { return bar0 + 8u * (8 + b); };
  auto s_empty = [&](int b) { return bar0 + 8u * (11 + b); };
  auto p_full = [&](int b) { return bar0 + 8u * (14 + b); };
  auto turn = [&](int quarter, int x) { return bar0 + 8u * (17 + 2 * quarter + x); };  // group x's decision on its tile
  auto sc_full = [&](int s) { return bar0 + 8u * (25 + s); };
  auto c_full = [&](int v, int s) { return bar0 + 8u * (33 + 2 * v + s); };   // codes of K (v 0), V (1)
  auto c_empty = [&](int v, int s) { return bar0 + 8u * (37 + 2 * v + s); };
  const uint32_t q_full = bar0 + 8u * 41, o_final = bar0 + 8u * 42, drain_bar = bar0 + 8u * 43;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (bar0 + 8u * 44 - base));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bar0 + 8u * 45 - base));
  static_assert(SCR == 8 && ST == 2 && 8 * 46 <= L::BARS, "barrier area");

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(k_full(s), DQ_THREADS);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), DQ_THREADS);
      mbar_init(v_empty(s), 1);
      for (int v = 0; v < 2; ++v) {
        mbar_init(c_full(v, s), 1);
        mbar_init(c_empty(v, s), DQ_THREADS);
      }
    }
    for (int b = 0; b < NSB; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(s_empty(b), 1);
      mbar_init(p_full(b), TQ);
    }
    for (int i = 0; i < 4; ++i)
      for (int x = 0; x < 2; ++x) mbar_init(turn(i, x), 1);
    for (int s = 0; s < SCR; ++s) mbar_init(sc_full(s), NG);
    mbar_init(q_full, 1);
    mbar_init(o_final, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x < TQ) run_m[threadIdx.x] = -INFINITY;
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
  const int G = P.nq / P.nkv, BT = TQ / G;  // tokens per CTA
  const int n_set = (P.M + BT - 1) / BT;
  const int cs = P.cs, rank = static_cast<int>(blockIdx.x) % cs;
  const int set = n_set - 1 - static_cast<int>(blockIdx.x) / cs;  // longest rows first
  const int kvh = blockIdx.y;
  const int t0 = set * BT, t1 = min(t0 + BT, P.M);
  const int len = start + t1;  // keys that the last row sees
  const int n_tiles = (len + TK - 1) / TK;
  const int jb = static_cast<int>(static_cast<long long>(n_tiles) * rank / cs);
  const int nt = static_cast<int>(static_cast<long long>(n_tiles) * (rank + 1) / cs) - jb;  // this CTA's tiles jb ..
  bool all_ok = true;

  auto slot_of = [&](int j) {  // of the CTA's tile j; 0 for an entry outside the pool
    const int s = kv8_slot(P.c, (jb + min(j, nt - 1)) * TK);
    if (s < 0 && lane == 0 && P.status) atomicCAS(P.status, 0, PF_ERR_KV_CAPACITY);
    return max(s, 0);
  };
  auto valid_of = [&](int j) { return min(TK, len - (jb + j) * TK); };  // keys of tile j that some row sees

  if (warp < 4) {
    regs_dec<32>();
    if ((warp == 0 || warp == 2) && lane == 0) {
      // -------------------------------------------------------------- copies
      const int v = warp >> 1;
      const uint8_t* codes = (v ? P.c.v : P.c.k) + static_cast<size_t>(kvh) * P.c.slots * HD;
      if (v == 0) {
        mbar_arrive_expect_tx(q_full, L::Q);
        for (int h = 0; h < NH; ++h) tma_load_3d(q_s + h * (TQ * 128), &tm_q, h * 64, kvh * G, t0, q_full);
      }
      int issued = 0, slot = nt > 0 ? slot_of(0) : 0;
      for (int j = 0; j < nt; ++j) {
        const int st = j % ST, next = slot_of(j + 1);
        if (!mbar_wait_long(c_empty(v, st), ((j / ST) & 1) ^ 1, abort_flag)) break;
        const uint32_t bytes = static_cast<uint32_t>(valid_of(j)) * HD;
        mbar_arrive_expect_tx(c_full(v, st), bytes);
        bulk_load((v ? vc_s : kc_s) + st * L::CODES, codes + static_cast<size_t>(slot) * HD, bytes, c_full(v, st));
        ++issued;
        slot = next;
      }
      // landed before shared memory is used otherwise, whatever the others do
      if (v == 0) wait_drain(q_full, 0);
      for (int j = max(0, issued - ST); j < issued; ++j) wait_drain(c_full(v, j % ST), (j / ST) & 1);
    }
    __syncwarp();
  }
  if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_s = idesc_f16(TQ, TK, 0, 0);
    constexpr uint32_t idesc_o = idesc_f16(TQ, HD, 0, 1);
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_long(bar, parity, abort_flag)) != 0; };
    auto issue_s = [&](int j) -> bool {
      const int b = j % NSB, st = j % ST;
      if (!wait(k_full(st), (j / ST) & 1) || !wait(s_empty(b), ((j / NSB) & 1) ^ 1)) return false;
      tc_fence_after();
#pragma unroll
      for (int kc = 0; kc < HD / 16; ++kc) {
        const uint32_t off = (kc >> 2) * (TQ * 128) + (kc & 3) * 32;
        umma_f16_ss_warp(tmem + b * TK, sdesc_kmajor_sw128(q_s + off), sdesc_kmajor_sw128(k_s + st * L::KV + off), idesc_s, kc > 0);
      }
      umma_commit_warp(s_full(b));
      umma_commit_warp(k_empty(st));
      return true;
    };
    bool ok = nt == 0 || wait(q_full, 0);
    if (ok && nt > 0) ok = issue_s(0);
    if (ok && nt > 1) ok = issue_s(1);
    for (int j = 0; j < nt && ok; ++j) {
      const int b = j % NSB, st = j % ST;
      // S_{j+2} as soon as PV_{j-1} has left its buffer, not behind P_j: the softmax group that
      // finishes tile j finds its next scores ready
      if (j + 2 < nt && !(ok = issue_s(j + 2))) break;
      ok = wait(p_full(b), (j / NSB) & 1) && wait(v_full(st), (j / ST) & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int kc = 0; kc < TK / 16; ++kc)
        umma_f16_ts_warp(tmem + COL_O, tmem + b * TK + 8 * kc, sdesc_mnmajor_sw128(v_s + st * L::KV + kc * 2048, TK * 128), idesc_o,
                         j > 0 || kc > 0);
      umma_commit_warp(s_empty(b));
      umma_commit_warp(v_empty(st));
    }
    if (ok) {
      umma_commit_warp(o_final);
    } else {
      umma_commit_warp(drain_bar);
      wait_drain(drain_bar, 0);
    }
  } else if (warp >= 4 && warp < 12) {
    // ---------------------------------------------------------------- codes to f16
    regs_dec<56>();
    const int v = warp >= 8 ? 1 : 0;
    constexpr int LPR = HD / 8;                // threads per row, 8 codes each: 16 B of f16
    constexpr int RPP = DQ_THREADS / LPR;      // rows per pass, a multiple of 8: the swizzle is the same in every pass
    constexpr int NP = TK / RPP;
    const int tid = threadIdx.x - (v ? 256 : 128);
    const int row0 = tid / LPR, c8 = tid % LPR;
    const uint32_t put = (c8 >> 3) * (TK * 128) + row0 * 128 + (((c8 & 7) ^ (row0 & 7)) << 4);
    // the scales of tile j's block tid (K threads 0 .. 3); 1 for a block past the sequence
    float sk = 1.f, sv = 1.f;
    auto load_scales = [&](int j) {
      sk = sv = 1.f;
      if (v == 0 && tid < NG && j < nt && tid * PF_KV8_BLOCK < valid_of(j)) {
        const int slot = max(kv8_slot(P.c, (jb + j) * TK), 0);
        const size_t at = static_cast<size_t>(kvh) * P.c.nblk + slot / PF_KV8_BLOCK + tid;
        sk = P.c.ks[at];
        sv = P.c.vs[at];
      }
    };
    load_scales(0);
    for (int j = 0; j < nt; ++j) {
      const int st = j % ST;
      const uint32_t codes = (v ? vc_s : kc_s) + st * L::CODES;
      if (!mbar_wait_long(c_full(v, st), (j / ST) & 1, abort_flag)) break;
      // the codes into registers at once: their stage takes the next copy while these wait for room
      const int valid = valid_of(j);
      uint2 w[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        w[i] = make_uint2(0, 0);  // keys past the last row's are zeros
        if (row0 + i * RPP < valid)
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[i].x), "=r"(w[i].y) : "r"(codes + tid * 8 + i * RPP * HD));
      }
      mbar_arrive(c_empty(v, st));
      if (!mbar_wait_long(v ? v_empty(st) : k_empty(st), ((j / ST) & 1) ^ 1, abort_flag)) break;
      const uint32_t tile = (v ? v_s : k_s) + st * L::KV;
      // K_{j-2}'s product is done, so PV_{j-5} is: softmaxes of tiles j - 4 on may still read their scales
      if (v == 0 && tid < NG) {
        const float svc = fminf(fmaxf(sv, 0x1p-60f), 0x1p60f);
        // the factor of the scores stays > 0: a hidden key's -inf stays -inf
        scales[(j % SCR) * NG + tid] = make_float4(fmaxf(sk * P.scale_log2, 1e-37f), __log2f(svc), 1.f / svc, 0.f);
        mbar_arrive(sc_full(j % SCR));
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t h0, h1, h2, h3;
        Kv8<T>::pairs(w[i].x, h0, h1);
        Kv8<T>::pairs(w[i].y, h2, h3);
        sts128(tile + put + i * RPP * 128, h0, h1, h2, h3);
      }
      fence_proxy_async_smem();
      mbar_arrive(v ? v_full(st) : k_full(st));
      load_scales(j + 1);
    }
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- softmax rows
    regs_inc<168>();
    const int x = (warp - 12) >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane;
    const uint32_t lane_off = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t obuf = tmem + lane_off + COL_O;
    const int first_pos = start + t0, pos = first_pos + r / G;
    float m = -INFINITY, l = 0.f;  // of this group's tiles; m follows the row's running maximum
    bool ok = true;
    for (int j = x; j < nt; j += 2) {
      const int b = j % NSB;
      const uint32_t sbuf = tmem + lane_off + b * TK;
      // tcgen05.ld / st are warp-collective: waits are voted on
      ok = __all_sync(0xffffffffu, mbar_wait_long(sc_full(j % SCR), (j / SCR) & 1, abort_flag) && mbar_wait_long(s_full(b), (j / NSB) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const int lim = pos - (jb + j) * TK;  // last visible column
      const bool masked = (jb + j) * TK + TK - 1 > first_pos;
      // a block's factors, read where they are used: registers are scarce
      const uint32_t sc_at = sc_s + (j % SCR) * NG * 16;
      auto factors = [&](int g) {
        float4 f;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(sc_at + 16 * g));
        return f;
      };
      uint32_t v[TK];
#pragma unroll
      for (int g = 0; g < NG; ++g) tmem_ld_32x32b_x32(sbuf + 32 * g, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * g));
      tmem_ld_wait();
      if (masked) {
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
        for (int e = 4; e < 28; e += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], __uint_as_float(v[32 * g + e + q]), __uint_as_float(v[32 * g + e + 4 + q]));
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], __uint_as_float(v[32 * g + 28 + q]));
        const float4 sc = factors(g);
        um = fmaxf(um, fmaf(max3(mx[0], mx[1], fmaxf(mx[2], mx[3])), sc.x, sc.y));
      }
      // the row's running maximum, after the other group's decision on tile j - 1
      if (j > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait_long(turn(quarter, 1 - x), ((j - 1) >> 1) & 1, abort_flag));
        if (!ok) break;
      }
      const float m_run = run_m[r];
      const bool need = um > m_run + RESCALE_LOG2;  // on the first tile too
      const float m_new = need ? um : m_run;
      const bool any = __any_sync(0xffffffffu, need);
      if (any) {
        run_m[r] = m_new;
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(turn(quarter, x));
      if (any && j > 0) {
        // O holds P_0 .. P_{j-1} V (the other group's P_{j-1} uses the maximum before this one):
        // wait for PV_{j-1}, then scale it in place; PV_j waits for this thread's P_j. (The barrier of
        // j - 1's buffer: its phase before, j - 4's, ended before S_{j-1} was issued, and its phase
        // after waits for P_j, so the parity names one phase.)
        ok = __all_sync(0xffffffffu, mbar_wait_long(s_empty((j - 1) % NSB), ((j - 1) / NSB) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const float alpha = need ? ex2t(m_run - m_new) : 1.f;
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
      if (m != m_new) {  // raised here or by the other group since this group's last tile
        l *= m == -INFINITY ? 0.f : ex2t(m - m_new);
        m = m_new;
      }
      const float mm = m == -INFINITY ? 0.f : m;  // a row that has seen no key: every weight 2^-inf = 0
      // P over the first half of S's columns
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float4 sc = factors(g);
        const float off = sc.y - mm;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float a = __uint_as_float(v[32 * g + e]), c = __uint_as_float(v[32 * g + e + 1]);
          float d = __uint_as_float(v[32 * g + e + 2]), f = __uint_as_float(v[32 * g + e + 3]);
          fma2(a, c, sc.x, off);
          fma2(d, f, sc.x, off);
          a = ex2t(a);
          c = ex2t(c);
          d = ex2t(d);
          f = ex2t(f);
          add2(s0, s1, a, c);
          add2(s2, s3, d, f);
          pk[e / 2] = f16x2t(a, c);
          pk[e / 2 + 1] = f16x2t(d, f);
        }
        l = fmaf((s0 + s1) + (s2 + s3), sc.z, l);
        tmem_st_32x32b_x16(sbuf + 16 * g, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_full(b));
    }
    // ---------------------------------------------------------------- O, m, l to shared memory
    if (ok) ok = mbar_wait_long(o_final, 0, abort_flag);
    all_ok = bar_and(1, SM_THREADS, ok);  // every MMA that reads the tiles is done, every maximum decided
    if (all_ok) {
      tc_fence_after();
      const float m_fin = run_m[r];
      sums[x * TQ + r] = m == -INFINITY ? 0.f : l * ex2t(m - m_fin);
      bar_and(1, SM_THREADS, true);
      // 16-byte piece q of a row at piece q ^ (row % (HD / 4)): a warp's rows hit different banks
      const uint32_t dst = base + r * L::ROW;
#pragma unroll 1
      for (int c = x * (HD / 64); c < (x + 1) * (HD / 64); ++c) {
        uint32_t o[32];
        if (nt > 0) {
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
      if (x == 0)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml_s + r * 8), "f"(m_fin), "f"(sums[r] + sums[TQ + r]) : "memory");
    }
  }

  // every CTA of the cluster has its rows in shared memory; each merges its share of them
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  if (warp >= 12 && all_ok) {
    // this CTA's rows: the weights of their parts, a row a thread, then four columns a lane and two
    // (hd 64: four) rows a pass and warp
    const int rb = TQ * rank / cs, re = min(TQ * (rank + 1) / cs, (t1 - t0) * G);
    float* wts = const_cast<float*>(sums) + 2 * TQ;  // [row][cs]
    const int my = rb + (static_cast<int>(threadIdx.x) - 384);
    if (my < re) {
      float mr = -INFINITY, lr = 0.f;
      float2 ml[MAX_CLUSTER];
#pragma unroll
      for (int s = 0; s < MAX_CLUSTER; ++s) {
        ml[s] = s < cs ? ldc64(map_cta(ml_s + my * 8, s)) : make_float2(-INFINITY, 0.f);
        mr = fmaxf(mr, ml[s].x);
      }
#pragma unroll
      for (int s = 0; s < MAX_CLUSTER; ++s) {
        ml[s].x = ml[s].x == -INFINITY ? 0.f : ex2t(ml[s].x - mr);
        lr = fmaf(ml[s].x, ml[s].y, lr);
      }
#pragma unroll
      for (int s = 0; s < MAX_CLUSTER; ++s)
        if (s < cs) wts[my * cs + s] = ml[s].x / lr;
    }
    bar_and(1, SM_THREADS, true);
    constexpr int RPW = 128 / HD;  // rows a warp's 32 lanes cover
    constexpr int U = 2;
    const int sub = lane / (HD / 4);
    const uint32_t piece = static_cast<uint32_t>(lane % (HD / 4));
    for (int row0 = rb + ((warp - 12) * RPW + sub); row0 < re; row0 += U * 8 * RPW) {
      float4 acc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < cs; ++s) {
        float4 o[U];
        float w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int row = min(row0 + u * 8 * RPW, re - 1);
          o[u] = ldc128(map_cta(base + row * L::ROW + ((piece ^ (row & (HD / 4 - 1))) << 4), s));
          w[u] = wts[row * cs + s];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)  // a part without a key of the row has weight 0 and O 0
          acc[u] = make_float4(fmaf(w[u], o[u].x, acc[u].x), fmaf(w[u], o[u].y, acc[u].y), fmaf(w[u], o[u].z, acc[u].z), fmaf(w[u], o[u].w, acc[u].w));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = row0 + u * 8 * RPW;
        if (row < re)
          *reinterpret_cast<uint2*>(P.out + (static_cast<size_t>(t0 + row / G) * P.nq + kvh * G + row % G) * HD + 4 * piece) =
              make_uint2(f16x2t(acc[u].x, acc[u].y), f16x2t(acc[u].z, acc[u].w));
      }
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
  const int sets = (a.M + BT - 1) / BT;
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
