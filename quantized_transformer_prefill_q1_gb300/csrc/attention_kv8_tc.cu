// attention_kv8_tc.cu — causal GQA attention of a chunk over the 8-bit KV cache on the 5th-generation
// tensor cores (tcgen05 / TMEM): the form for more rows than attention_kv8.cu takes. Mathematics as
// there: with u_j = log2(e) s_j + log2 sV, weights w_j = 2^(u_j - m) = p_j sV up to the row's factor go
// into the product with the value codes, and the softmax's sum takes w_j / sV per scale block; neither
// scale touches a code, and every code is exact in f16.
//
// One CTA = one kv head and 128 of its query rows (row = token * G + head in the group) against its
// share of the key tiles: a cluster shares the rows and cuts the keys between its CTAs; at the end
// every CTA leaves its rows' sums, maxima and O in its shared memory, and each merges its share of the
// rows over the cluster. No scratch and no second kernel. Where a cluster has more CTAs than its rows have
// key tiles (its size is that of the longest rows, or of the longest sequence when the start is on the
// device), the ones left over copy nothing, hold no part and only help to merge; rows with one part go
// straight to the output.
//
// At hd 128 and more than one row tile, two CTAs work as a pair (cta_group::2, M = 256): two row tiles
// of the same kv head, the same key tiles, and each CTA converts only half of them (K: 64 of the 128
// keys, V: 64 of the 128 columns), which is also all that its tensor core reads of them from its own
// shared memory. One CTA alone moves 224 KB a key tile through shared memory (codes in and out, f16
// written, read by both products, Q), 1,750 cycles at 128 B a cycle against 1,400 of tensor work; a
// CTA of a pair 128 KB.
//
// Warps (16):
//   0, 2     copies: Q and the K codes (0), the V codes (2), ST stages ahead;
//   1        TMEM (three S buffers of 128 columns and O) and the MMAs, S_j = Q K_j^T and
//            O += P_j V_j (P over S's columns), whichever is ready (in a pair, the even CTA's);
//   3        the scales;
//   4..7     K and V codes to f16, into shared memory in the MMA's 128-byte swizzle;
//   8..15    softmax, two threads per row (64 keys each; the maxima meet in shared memory, warp pair by
//            warp pair): S from TMEM, running maximum raised only when exceeded by more than 2^8 (then O
//            is rescaled in TMEM), P as f16 back. (Two groups of four warps on alternate key tiles, a
//            whole row a thread, held each S buffer twice as long: 300 us where this took 292 for 512
//            tokens of 32/8 heads at 32,256.)
// Every wait is bounded; a timeout aborts the CTA and records PF_ERR_DEVICE_TIMEOUT.
//
// Rounding: P to f16 (the value codes' type in the product), the output to f16; all else f32.
//
// Bound (512 tokens of 32/8 heads of 128 over 32,768 int8 keys: 293 us = 0.93 PFLOP/s, 0.49 of the
// measured burst peak on 128 of 152 SMs): a key tile takes 2,200 cycles (clock stamps in a copy), 1.15 us,
// where attention_tc.cu takes 0.85 for the same tile of a 16-bit cache. Without the conversions the case took
// 265 us (1.03 a tile) instead of 292, without the exponentials and maxima 246, without the products 250. So the conversions are
// about a third of the difference; what the rest consists of (the hand-over between the CTAs of a pair,
// the polling, the scales) was not measured apart. Tried and slower: both row tiles in one CTA (340), one CTA a
// row tile (341), P through shared memory (357). A chunk of 64 tokens at position 0, one tile and no cluster, takes 7.0 us (in
// a cluster, stamped, 10: 1 to set up, 1.5 to load, 1 to convert, 3 from the scores to O, 2 to merge). The MMA warp polls
// without sleeping: with 20 ns between its looks the long case took 293 us where it took 291.8.
#include <algorithm>
#include <type_traits>

#include "kv8.cuh"

namespace pf {
namespace {

constexpr int TQ = 128;  // rows per CTA
constexpr int TK = 128;  // keys per tile: one page, four scale blocks
constexpr int NSB = 3;   // S / P buffers
constexpr int LA = 1;    // tiles that the K codes run ahead of the V codes
constexpr int THREADS = 512;
constexpr int SM_WARP = 8;        // first softmax warp
constexpr int SM_THREADS = 256;   // softmax threads: two per row
constexpr int DQ_THREADS = 128;   // converting threads
constexpr int NG = TK / PF_KV8_BLOCK;
constexpr int SCR = 8;   // tiles in the ring of scales
constexpr int PORTABLE_CLUSTER = 8, MAX_CLUSTER = 16;  // above 8 by the attribute that set_attr sets
constexpr float RESCALE_LOG2 = 8.f;
constexpr uint32_t COL_O = NSB * TK;  // TMEM: S buffer b at b TK, O at COL_O

template <int HD, int PAIR>
struct TSmem {
  static constexpr int ST = PAIR ? 3 : 2;          // stages of f16 tiles, K and V each
  static constexpr int CK = ST, CV = !PAIR && HD == 128 ? 1 : ST;  // stages of codes (what shared memory leaves)
  static constexpr int KR = PAIR ? TK / 2 : TK;    // keys of a K tile that this CTA holds
  static constexpr int VC = PAIR ? HD / 2 : HD;    // columns of a V tile that this CTA holds
  static constexpr int Q = TQ * HD * 2;
  static constexpr int KT = KR * HD * 2;           // f16 tiles
  static constexpr int VT = TK * VC * 2;
  static constexpr int KCODES = KR * HD;
  static constexpr int VCODES = TK * VC;
  static constexpr int ROW = HD * 4;  // a row of O at the end, over the idle Q and K tiles
  static constexpr int TILES = Q + ST * (KT + VT);
  static constexpr int RINGS = CK * KCODES + CV * VCODES;
  static constexpr int SCALES = SCR * NG * 4 * 4;
  static constexpr int MAXIMA = 4 * TQ * 4;  // of each row, half and (tile parity)
  static constexpr int BARS = 512;
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
  int cs;  // parts of the keys: CTAs (pairs) per cluster
  __half* out;
  int* status;
};

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > PF_WAIT_LIMIT_NS) return;
  }
}
// (bar.red wants its warps converged: __syncwarp() before it where they come from waits or branches of single threads)
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
// mbar_wait with the hardware suspending the thread for up to 20 us a try: 16 warps that poll would take
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
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Pair MMA with A (256 rows: 128 in each CTA's tensor memory at a_tmem) from tensor memory.
__device__ __forceinline__ void umma_pair_f16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                      uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
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

__device__ __forceinline__ float4 lds128f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// CL: most CTAs of its clusters. (The merge holds a row's parts in registers; one instance for 16 took up to 5 %
// more time where 8 do.)
template <int HD, int T, int PAIR, int CL>
__global__ void __launch_bounds__(THREADS, 1)
    attn_kv8_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const TcParams P) {
  PF_TIMELINE(TL_ATTENTION_KV8_TC);
  using L = TSmem<HD, PAIR>;
  constexpr int ST = L::ST;
  constexpr int NH = HD / 64;  // 64-wide swizzle regions along head_dim
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t q_s = base, k_s = q_s + L::Q, v_s = k_s + ST * L::KT;
  const uint32_t kc_s = base + L::TILES, vc_s = kc_s + L::CK * L::KCODES;
  float4* scales = reinterpret_cast<float4*>(gbase + L::TILES + L::RINGS);  // [SCR][NG] (log2(e) sK / sqrt(hd), log2 sV, 1 / sV, -)
  const uint32_t sc_s = base + L::TILES + L::RINGS;
  volatile float* maxima = reinterpret_cast<volatile float*>(gbase + L::TILES + L::RINGS + L::SCALES);  // [2][2][TQ]
  const uint32_t ml_s = kc_s;  // [TQ] (m, l)
  volatile float* sums = reinterpret_cast<volatile float*>(gbase + L::TILES + TQ * 8);  // [2][TQ]
  const uint32_t bar0 = base + L::TILES + L::RINGS + L::SCALES + L::MAXIMA;
  auto full = [&](int v, int s) { return bar0 + 8u * (3 * v + s); };           // f16 tiles of K (v 0), V (1)
  auto empty = [&](int v, int s) { return bar0 + 8u * (6 + 3 * v + s); };
  auto c_full = [&](int v, int s) { return bar0 + 8u * (12 + 3 * v + s); };    // codes
  auto c_empty = [&](int v, int s) { return bar0 + 8u * (18 + 3 * v + s); };
  auto s_full = [&](int b) { return bar0 + 8u * (24 + b); };
  auto s_empty = [&](int b) { return bar0 + 8u * (27 + b); };
  auto p_full = [&](int b) { return bar0 + 8u * (30 + b); };
  auto sc_full = [&](int s) { return bar0 + 8u * (41 + s); };
  auto sc_free = [&](int s) { return bar0 + 8u * (55 + s); };
  const uint32_t q_full = bar0 + 8u * 49, q_ready = bar0 + 8u * 50, o_final = bar0 + 8u * 51, drain_bar = bar0 + 8u * 52;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + (bar0 + 8u * 53 - base));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bar0 + 8u * 54 - base));
  static_assert(SCR == 8 && ST <= 3 && 8 * 63 <= L::BARS, "barrier area");

  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    // arrivals are one a warp; a pair's tiles, probabilities and Q are awaited in the even CTA
    constexpr int BOTH = PAIR ? 2 : 1;
    for (int s = 0; s < ST; ++s)
      for (int v = 0; v < 2; ++v) {
        mbar_init(full(v, s), 4 * BOTH);
        mbar_init(empty(v, s), 1);
        mbar_init(c_full(v, s), 1);
        mbar_init(c_empty(v, s), 4);
      }
    for (int b = 0; b < NSB; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(s_empty(b), 1);
      mbar_init(p_full(b), 8 * BOTH);
    }
    for (int s = 0; s < SCR; ++s) {
      mbar_init(sc_full(s), 1);
      mbar_init(sc_free(s), 8);
    }
    mbar_init(q_full, 1);
    mbar_init(q_ready, BOTH);
    mbar_init(o_final, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // the other CTA's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  const int start = P.start_dev ? *P.start_dev : P.start_host;
  const int G = P.nq / P.nkv, BT = TQ / G;  // tokens per CTA
  const int cs = P.cs;
  constexpr int W = PAIR ? 2 : 1;            // row tiles that share their key tiles
  const int n_set = (P.M + W * BT - 1) / (W * BT);
  const int rank = static_cast<int>(blockIdx.x) % (W * cs);   // in the cluster
  const int half = PAIR ? rank & 1 : 0, part = rank / W;
  const int set = n_set - 1 - static_cast<int>(blockIdx.x) / (W * cs);  // longest rows first
  const int kvh = blockIdx.y;
  const int t0 = (set * W + half) * BT, t1 = min(t0 + BT, P.M);  // a pair's second tile may lie past the last token
  const int len = start + min((set + 1) * W * BT, P.M);  // keys that the last row sees
  const int n_tiles = (len + TK - 1) / TK;
  const int parts = min(cs, n_tiles);  // each has a tile; a CTA past them has none, and nothing reads its shared memory
  // its tiles jb .. (at most 2^30 positions: the products stay below 2^28)
  const int jb = n_tiles * min(part, parts) / parts, nt = n_tiles * min(part + 1, parts) / parts - jb;
  bool all_ok = true;
  auto slot_of = [&](int j) {  // of the CTA's tile j; 0 for an entry outside the pool
    const int s = kv8_slot(P.c, (jb + min(j, nt - 1)) * TK);
    if (s < 0 && lane == 0 && P.status) atomicCAS(P.status, 0, PF_ERR_KV_CAPACITY);
    return max(s, 0);
  };
  auto valid_of = [&](int j) { return min(TK, len - (jb + j) * TK); };  // keys of tile j that some row sees
  // one arrival of a converged warp, on the even CTA's barrier in a pair
  auto arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) {
      if (PAIR && half)
        mbar_arrive_cta(bar, rank - 1);
      else
        mbar_arrive(bar);
    }
  };

  if (warp < 4 && nt > 0) {
    if ((warp == 0 || warp == 2) && lane == 0) {
      // -------------------------------------------------------------- copies
      const int v = warp >> 1;
      if (v == 0) {
        mbar_arrive_expect_tx(q_full, L::Q);
        for (int h = 0; h < NH; ++h) tma_load_3d(q_s + h * (TQ * 128), &tm_q, h * 64, kvh * G, t0, q_full);
      }
      // K: this CTA's keys, all columns; V: all keys, this CTA's columns (rows past the cache are zeros)
      const CUtensorMap* map = v ? &tm_v : &tm_k;
      const uint32_t ring = v ? vc_s : kc_s, bytes = v ? L::VCODES : L::KCODES;
      const int x0 = v ? half * L::VC : 0, y0 = kvh * P.c.slots + (v ? 0 : half * L::KR);
      int issued = 0, slot = slot_of(0);
      for (int j = 0; j < nt; ++j) {
        const int sc = v ? L::CV : L::CK, st = j % sc, next = slot_of(j + 1);
        if (!mbar_wait_long(c_empty(v, st), ((j / sc) & 1) ^ 1, abort_flag)) break;
        mbar_arrive_expect_tx(c_full(v, st), bytes);
        tma_load_2d(ring + st * bytes, map, x0, y0 + slot, c_full(v, st));
        ++issued;
        slot = next;
        if (j == 0 && v == 0 && mbar_wait_long(q_full, 0, abort_flag)) {
          if (PAIR && half)
            mbar_arrive_cta(q_ready, rank - 1);
          else
            mbar_arrive(q_ready);
        }
      }
      // landed before shared memory is used otherwise, whatever the others do
      if (v == 0) wait_drain(q_full, 0);
      const int sc = v ? L::CV : L::CK;
      for (int j = max(0, issued - sc); j < issued; ++j) wait_drain(c_full(v, j % sc), (j / sc) & 1);
    }
    __syncwarp();
    if (warp == 3) {
      // -------------------------------------------------------------- scales, a lane a block of 32 keys
      auto load = [&](int j, float& sk, float& sv) {  // 1 for a block past the sequence
        sk = sv = 1.f;
        if (lane < NG && j < nt && lane * PF_KV8_BLOCK < valid_of(j)) {
          const size_t at = static_cast<size_t>(kvh) * P.c.nblk + max(kv8_slot(P.c, (jb + j) * TK), 0) / PF_KV8_BLOCK + lane;
          sk = P.c.ks[at];
          sv = P.c.vs[at];
        }
      };
      float sk, sv, nk, nv;
      load(0, sk, sv);
      load(1, nk, nv);
      for (int j = 0; j < nt; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait_long(sc_free(j % SCR), ((j / SCR) & 1) ^ 1, abort_flag))) break;
        if (lane < NG) {
          // (scales lie in 0 .. 2^16: the lower limit keeps the logarithm finite and moves values by less than 2^-51,
          // the upper one is for what is no scale)
          const float svc = fminf(fmaxf(sv, 0x1p-60f), 0x1p60f);
          // the factor of the scores stays > 0: a hidden key's -inf stays -inf
          scales[(j % SCR) * NG + lane] = make_float4(fmaxf(sk * P.scale_log2, 1e-37f), __log2f(svc), 1.f / svc, 0.f);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_full(j % SCR));
        sk = nk;
        sv = nv;
        load(j + 2, nk, nv);
      }
    }
  }
  if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (half == 0 && nt > 0) {
      constexpr uint32_t idesc_s = idesc_f16(PAIR ? 2 * TQ : TQ, TK, 0, 0);
      constexpr uint32_t idesc_o = idesc_f16(PAIR ? 2 * TQ : TQ, HD, 0, 1);
      const uint16_t mask = static_cast<uint16_t>(3u << rank);
      auto commit = [&](uint32_t bar) {
        if (PAIR)
          umma_pair_commit_warp(bar, mask);
        else
          umma_commit_warp(bar);
      };
      bool ok = __all_sync(0xffffffffu, mbar_wait_long(q_ready, 0, abort_flag));
      // S_js and PV_jp are next. The next tile's scores go before a tile's PV (its softmax waits for
      // them), those after it behind: a PV that is ready then leaves no gap while S waits for a buffer.
      int js = 0, jp = 0;
      uint64_t t_idle = 0;
      while (ok && jp < nt) {
        auto s_ready = [&] {
          return js < nt && __all_sync(0xffffffffu, mbar_test(full(0, js % ST), (js / ST) & 1) &&
                                                        mbar_test(s_empty(js % NSB), ((js / NSB) & 1) ^ 1));
        };
        auto p_ready = [&] {
          return jp < js && __all_sync(0xffffffffu, mbar_test(p_full(jp % NSB), (jp / NSB) & 1) &&
                                                        mbar_test(full(1, jp % ST), (jp / ST) & 1));
        };
        const bool s_first = js <= jp + 1;
        bool do_s = s_first && s_ready(), do_p = !do_s && p_ready();
        if (!do_s && !do_p && !s_first) do_s = s_ready();
        if (do_s) {
          const int b = js % NSB, st = js % ST;
          tc_fence_after();
#pragma unroll
          for (int kc = 0; kc < HD / 16; ++kc) {
            const uint64_t qd = sdesc_kmajor_sw128(q_s + (kc >> 2) * (TQ * 128) + (kc & 3) * 32);
            const uint64_t kd = sdesc_kmajor_sw128(k_s + st * L::KT + (kc >> 2) * (L::KR * 128) + (kc & 3) * 32);
            if (PAIR)
              umma_pair_f16_ss_warp(tmem + b * TK, qd, kd, idesc_s, kc > 0);
            else
              umma_f16_ss_warp(tmem + b * TK, qd, kd, idesc_s, kc > 0);
          }
          commit(s_full(b));
          commit(empty(0, st));
          ++js;
        } else if (do_p) {
          const int b = jp % NSB, st = jp % ST;
          tc_fence_after();
#pragma unroll
          for (int kc = 0; kc < TK / 16; ++kc) {
            const uint64_t vd = sdesc_mnmajor_sw128(v_s + st * L::VT + kc * 2048, TK * 128);
            if (PAIR)
              umma_pair_f16_ts_warp(tmem + COL_O, tmem + b * TK + 8 * kc, vd, idesc_o, jp > 0 || kc > 0);
            else
              umma_f16_ts_warp(tmem + COL_O, tmem + b * TK + 8 * kc, vd, idesc_o, jp > 0 || kc > 0);
          }
          commit(s_empty(b));
          commit(empty(1, st));
          ++jp;
        } else {
          const uint64_t now = global_timer_ns();
          if (t_idle == 0) t_idle = now;
          const bool give_up = *abort_flag || now - t_idle > PF_WAIT_LIMIT_NS;
          if (__any_sync(0xffffffffu, give_up)) {
            *abort_flag = 1;
            ok = false;
          }
          continue;
        }
        t_idle = 0;
      }
      if (ok) {
        commit(o_final);
      } else {
        commit(drain_bar);
        wait_drain(drain_bar, 0);
      }
    }
  } else if (warp >= 4 && warp < SM_WARP) {
    // ---------------------------------------------------------------- codes to f16
    const int tid = threadIdx.x - 128;
    // A tile of ROWS x C codes (K or V of tile j): 8 codes a thread and pass, one 16-byte piece of f16 in
    // regions of 64 columns (rows of 128 B, swizzled). Rows a pass are a multiple of 8: one swizzle.
    auto convert = [&](auto rows_c, auto cols_c, int v, int j, uint32_t ring, uint32_t tiles, int valid) -> bool {
      constexpr int ROWS = decltype(rows_c)::value, C = decltype(cols_c)::value;
      constexpr int LPR = C / 8, RPP = DQ_THREADS / LPR, NP = ROWS / RPP;
      const int cs = v ? L::CV : L::CK, cst = j % cs, st = j % ST, row0 = tid / LPR, c8 = tid % LPR;
      const uint32_t codes = ring + cst * (ROWS * C) + tid * 8;
      const uint32_t put = tiles + st * (ROWS * C * 2) + (c8 >> 3) * (ROWS * 128) + row0 * 128 + (((c8 & 7) ^ (row0 & 7)) << 4);
      if (!__all_sync(0xffffffffu, mbar_wait_long(c_full(v, cst), (j / cs) & 1, abort_flag))) return false;
      // the codes into registers at once: their stage takes the next copy while these wait for room
      uint2 w[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        w[i] = make_uint2(0, 0);  // keys past the last row's are zeros: their codes may be NaN
        if (row0 + i * RPP < valid)
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[i].x), "=r"(w[i].y) : "r"(codes + i * RPP * C));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(c_empty(v, cst));
      if (!__all_sync(0xffffffffu, mbar_wait_long(empty(v, st), ((j / ST) & 1) ^ 1, abort_flag))) return false;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t h0, h1, h2, h3;
        Kv8<T>::pairs(w[i].x, h0, h1);
        Kv8<T>::pairs(w[i].y, h2, h3);
        sts128(put + i * RPP * 128, h0, h1, h2, h3);
      }
      fence_proxy_async_smem();
      arrive(full(v, st));
      return true;
    };
    // K runs LA tiles ahead of V, as the scores do ahead of P V
    for (int j = 0; j < nt + LA; ++j) {
      if (j < nt && !convert(std::integral_constant<int, L::KR>{}, std::integral_constant<int, HD>{}, 0, j, kc_s, k_s, valid_of(j) - half * L::KR))
        break;
      if (j >= LA && !convert(std::integral_constant<int, TK>{}, std::integral_constant<int, L::VC>{}, 1, j - LA, vc_s, v_s, valid_of(j - LA)))
        break;
    }
  } else if (warp >= SM_WARP && nt > 0) {
    // ---------------------------------------------------------------- softmax rows
    const int x = (warp - SM_WARP) >> 2, quarter = warp & 3;  // keys [64 x, 64 x + 64) of each tile
    const int r = 32 * quarter + lane;
    const uint32_t lane_off = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t obuf = tmem + lane_off + COL_O;
    const int first_pos = start + t0, pos = first_pos + r / G;
    float m = -INFINITY, l = 0.f;  // l of this thread's keys
    bool ok = true, failed = false;
    for (int j = 0; j < nt; ++j) {
      const int b = j % NSB;
      const uint32_t sbuf = tmem + lane_off + b * TK;
      // tcgen05.ld / st are warp-collective and the two warps of a quarter meet in every tile: a failed
      // wait is carried to that meeting, where both stop
      const bool got = mbar_wait_long(sc_full(j % SCR), (j / SCR) & 1, abort_flag) && mbar_wait_long(s_full(b), (j / NSB) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, got) && !failed;
      tc_fence_after();
      const int lim = pos - (jb + j) * TK - 64 * x;  // last visible one of this thread's columns
      const bool masked = (jb + j) * TK + TK - 1 > first_pos;
      const uint32_t sc_at = sc_s + ((j % SCR) * NG + 2 * x) * 16;
      auto factors = [&](int g) {
        float4 f;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(sc_at + 16 * g));
        return f;
      };
      float4 sc[2] = {factors(0), factors(1)};
      uint32_t v[64];
      float um = -INFINITY;
      if (ok) {
        tmem_ld_32x32b_x32(sbuf + 64 * x, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld_32x32b_x32(sbuf + 64 * x + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tmem_ld_wait();
        if (masked) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e > lim) v[e] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float mx[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(v[32 * g + e]);
#pragma unroll
          for (int e = 4; e < 28; e += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], __uint_as_float(v[32 * g + e + q]), __uint_as_float(v[32 * g + e + 4 + q]));
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], __uint_as_float(v[32 * g + 28 + q]));
          um = fmaxf(um, fmaf(max3(mx[0], mx[1], fmaxf(mx[2], mx[3])), sc[g].x, sc[g].y));
        }
        maxima[(2 * (j & 1) + x) * TQ + r] = um;
      }
      // both halves of the rows have been read (P goes over them) and their maxima are in
      tc_fence_before();
      ok = bar_and(2 + quarter, 64, ok);
      if (!ok) break;
      tc_fence_after();
      um = fmaxf(um, maxima[(2 * (j & 1) + 1 - x) * TQ + r]);
      const bool need = um > m + RESCALE_LOG2;  // the first tile's too; the row's two threads decide alike
      // The weights' exponent s sK + (log2 sV - m) is rounded apart from m, by up to an ulp of m, and from |m| = 2^27
      // on that alone would take a weight out of f16's range. Scores that large are rounded before the difference,
      // as their maximum was (elsewhere the branch costs 0.6 % for long lists of keys, 2.4 for 512 tokens at 1,536).
      const bool far = fabsf(um) > 0x1p20f && um != -INFINITY;
      if (__any_sync(0xffffffffu, need || far)) {
        const float alpha = need ? ex2t(m - um) : 1.f;
        l *= alpha;
        if (j > 0) {
          // O holds P_0 .. P_{j-1} V: wait for PV_{j-1}, then scale this thread's half of the row's columns;
          // PV_j waits for this thread's P_j. (j - 1's buffer: its phase before ended before S_{j-1} was
          // issued, its phase after waits for P_j: the parity names one phase.)
          if (__all_sync(0xffffffffu, mbar_wait_long(s_empty((j - 1) % NSB), ((j - 1) / NSB) & 1, abort_flag))) {
            tc_fence_after();
#pragma unroll 1
            for (int c = x * (HD / 64); c < (x + 1) * (HD / 64); ++c) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(obuf + 32 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st_32x32b_x32(obuf + 32 * c, o);
            }
          } else {
            failed = true;
          }
        }
        if (need) m = um;
        if (far) {  // v becomes the exponent itself, with factor 1 and offset m - m
          const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float a = __uint_as_float(v[e]), c = __uint_as_float(v[e + 1]);
            fma2(a, c, sc[e >> 5].x, sc[e >> 5].y);
            add2(a, c, -mm, -mm);
            v[e] = __float_as_uint(a);
            v[e + 1] = __float_as_uint(c);
          }
          sc[0].x = sc[1].x = 1.f;
          sc[0].y = sc[1].y = mm;
        }
        __syncwarp();  // the warp-wide store of P follows
      }
      const float mm = m == -INFINITY ? 0.f : m;  // a row that has seen no key: every weight 2^-inf = 0
      // P over the first half of S's columns, this thread's 32 of them
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float off = sc[g].y - mm;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float a = __uint_as_float(v[32 * g + e]), c = __uint_as_float(v[32 * g + e + 1]);
          float d = __uint_as_float(v[32 * g + e + 2]), f = __uint_as_float(v[32 * g + e + 3]);
          fma2(a, c, sc[g].x, off);
          fma2(d, f, sc[g].x, off);
          a = ex2t(a);
          c = ex2t(c);
          d = ex2t(d);
          f = ex2t(f);
          add2(s0, s1, a, c);
          add2(s2, s3, d, f);
          pk[e / 2] = f16x2t(a, c);
          pk[e / 2 + 1] = f16x2t(d, f);
        }
        l = fmaf((s0 + s1) + (s2 + s3), sc[g].z, l);
        tmem_st_32x32b_x16(sbuf + 32 * x + 16 * g, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      arrive(p_full(b));
      if (lane == 0) mbar_arrive(sc_free(j % SCR));
    }
    // ---------------------------------------------------------------- O, m, l to shared memory
    if (ok) ok = !failed && mbar_wait_long(o_final, 0, abort_flag);
    __syncwarp();
    all_ok = bar_and(1, SM_THREADS, ok);  // every MMA that reads the tiles is done
    if (all_ok) {
      tc_fence_after();
      sums[x * TQ + r] = l;
      bar_and(1, SM_THREADS, true);
      const int t = t0 + r / G;
      const float inv = parts == 1 ? __fdividef(1.f, sums[r] + sums[TQ + r]) : 1.f;
      __half* out = P.out + (static_cast<size_t>(t) * P.nq + kvh * G + r % G) * HD;
      // 16-byte piece q of a row at piece q ^ (row % (HD / 4)): a warp's rows hit different banks
      const uint32_t dst = base + r * L::ROW;
#pragma unroll 1
      for (int c = x * (HD / 64); c < (x + 1) * (HD / 64); ++c) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(obuf + 32 * c, o);
        tmem_ld_wait();
        if (parts == 1) {  // the whole row is here: straight to the output
          if (t < t1) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = f16x2t(__uint_as_float(o[8 * q + 2 * e]) * inv, __uint_as_float(o[8 * q + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4*>(out + 32 * c + 8 * q) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          __syncwarp();  // the warp-wide load of the next columns follows
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            sts128(dst + (((8 * c + q) ^ (r & (HD / 4 - 1))) << 4), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (x == 0)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml_s + r * 8), "f"(m), "f"(sums[r] + sums[TQ + r]) : "memory");
    }
  }

  // every part of the cluster has its rows in shared memory; each CTA merges its share of them
  tc_fence_before();
  __syncwarp();
  if (cs > 1) cluster_sync_all();
  if (warp >= SM_WARP && all_ok && parts > 1) {
    // this CTA's rows: the weights of their parts, a row a thread, then four columns a lane and two
    // (hd 64: four) rows a pass and warp
    // (a pair's two row tiles are merged apart, each over the CTAs that hold it)
    const int rb = TQ * part / cs, re = min(TQ * (part + 1) / cs, (t1 - t0) * G);
    float* wts = const_cast<float*>(sums) + 2 * TQ;  // [row][parts]
    const int my = rb + (static_cast<int>(threadIdx.x) - 32 * SM_WARP);
    // (a row's parts are all requested before the first is used, and the CTA's own is read as its own:
    // loads from other CTAs move about 16 B a cycle)
    constexpr int NP = CL / W;
    if (my < re) {
      float mr = -INFINITY, lr = 0.f;
      float2 ml[NP];
#pragma unroll
      for (int s = 0; s < NP; ++s) ml[s] = s < parts ? ldc64(map_cta(ml_s + my * 8, W * s + half)) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int s = 0; s < NP; ++s) mr = fmaxf(mr, ml[s].x);
#pragma unroll
      for (int s = 0; s < NP; ++s) {
        ml[s].x = ml[s].x == -INFINITY ? 0.f : ex2t(ml[s].x - mr);
        lr = fmaf(ml[s].x, ml[s].y, lr);
      }
#pragma unroll
      for (int s = 0; s < NP; ++s)
        if (s < parts) wts[my * parts + s] = __fdividef(ml[s].x, lr);
    }
    __syncwarp();
    bar_and(1, SM_THREADS, true);
    constexpr int RPW = 128 / HD;  // rows a warp's 32 lanes cover
    constexpr int U = PAIR ? 2 : 1;
    const int sub = lane / (HD / 4);
    const uint32_t piece = static_cast<uint32_t>(lane % (HD / 4));
    for (int row0 = rb + ((warp - SM_WARP) * RPW + sub); row0 < re; row0 += U * 8 * RPW) {
      float4 o[U][NP];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = min(row0 + u * 8 * RPW, re - 1);
        const uint32_t at = base + row * L::ROW + ((piece ^ (row & (HD / 4 - 1))) << 4);
#pragma unroll
        for (int s = 0; s < NP; ++s)
          if (s < parts) o[u][s] = s == part ? lds128f(at) : ldc128(map_cta(at, W * s + half));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = row0 + u * 8 * RPW;
        if (row >= re) break;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < NP; ++s)
          if (s < parts) {  // a part without a visible key of the row has weight 0 and an O of zeros times values
            const float w = wts[row * parts + s];
            acc = make_float4(fmaf(w, o[u][s].x, acc.x), fmaf(w, o[u][s].y, acc.y), fmaf(w, o[u][s].z, acc.z), fmaf(w, o[u][s].w, acc.w));
          }
        *reinterpret_cast<uint2*>(P.out + (static_cast<size_t>(t0 + row / G) * P.nq + kvh * G + row % G) * HD + 4 * piece) =
            make_uint2(f16x2t(acc.x, acc.y), f16x2t(acc.z, acc.w));
      }
    }
  }
  __syncwarp();
  cluster_sync_all();  // nobody leaves while others read its shared memory
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag && P.status) atomicCAS(P.status, 0, PF_ERR_DEVICE_TIMEOUT);
}

// Clusters of `size` CTAs that the GPU runs at once (they must each lie in one GPC, so large ones leave
// SMs unused); filled by prepare_attention_kv8_tc_kernels.
int g_active[2][MAX_CLUSTER + 1];  // [pair][size]

template <int HD, int T, int PAIR>
cudaError_t launch(const Kv8AttnArgs& a, const Kv8Layer& l, cudaStream_t stream) {
  using L = TSmem<HD, PAIR>;
  const pf_config& c = *a.c;
  const int G = c.n_q_heads / c.n_kv_heads, BT = TQ / G, W = PAIR ? 2 : 1;
  CUtensorMap tq, tk, tv;
  const uint64_t qd[3] = {static_cast<uint64_t>(HD), static_cast<uint64_t>(c.n_q_heads), static_cast<uint64_t>(a.M)};
  const uint64_t qs[2] = {static_cast<uint64_t>(HD) * 2, static_cast<uint64_t>(c.n_q_heads) * HD * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(BT)};
  const uint64_t rows = static_cast<uint64_t>(c.n_kv_heads) * l.slots;
  if (!encode_tmap_16(&tq, 0, 3, a.q, qd, qs, qb) || !encode_tmap_8(&tk, l.k, HD, rows, HD, L::KR, 0) ||
      !encode_tmap_8(&tv, l.v, HD, rows, L::VC, TK, 0))
    return cudaErrorInvalidValue;
  TcParams p{};
  p.c = l;
  p.M = a.M;
  p.nq = c.n_q_heads;
  p.nkv = c.n_kv_heads;
  p.start_dev = a.start_dev;
  p.start_host = a.start_host;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HD));
  p.out = static_cast<__half*>(a.out);
  p.status = a.status;
  const int sets = (a.M + W * BT - 1) / (W * BT);
  // As many CTAs on a set of rows as run at once: a second wave would cost more than the parts save
  // (128 tokens of 32/8 heads over 8,192 keys took 56 us in 16 clusters of 8, of which 15 run at once, when clusters of 6
  // took 42; they take 37 now).
  // And not more CTAs than the longest rows have key tiles. A start on the device is not known here: such
  // calls go by the longest sequence, and the kernel leaves out the CTAs that have no tile (a 12-layer session's
  // chunks of 8, 64 and 200 tokens at 0: 572, 985 and 1,358 us with room for 33,000 positions, 585, 984 and 1,365
  // with room for 512). (8 tokens of 32/8 heads, int8, before both: in clusters of 8
  // 8.7 us over 8 keys, 19.0 over 8,200 and 47.6 over 32,008; now 5.7, 16.0 and 34.1. Parts up to the number of
  // tiles are the rule's end, not always its best: 32 tokens of 32/4 heads over 1,032 keys took 11.4 in 9, 11.1 in 8.)
  const long long groups = static_cast<long long>(sets) * c.n_kv_heads;
  const int tiles = ((a.start_dev ? c.max_seq : a.start_host + a.M) + TK - 1) / TK;
  p.cs = 1;
  for (int cs = 2; cs <= std::min(MAX_CLUSTER / W, tiles); ++cs)
    if (groups <= g_active[PAIR][W * cs]) p.cs = cs;
  const auto kernel = W * p.cs > PORTABLE_CLUSTER ? attn_kv8_tc_kernel<HD, T, PAIR, MAX_CLUSTER>
                                                  : attn_kv8_tc_kernel<HD, T, PAIR, PORTABLE_CLUSTER>;
  return launch_pdl_cluster(kernel, dim3(W * p.cs * sets, c.n_kv_heads), dim3(THREADS), L::BYTES, stream, W * p.cs, tq, tk, tv, p);
}

// Pairs at hd 128 as soon as there are two row tiles.
template <int HD, int T>
cudaError_t launch_form(const Kv8AttnArgs& a, const Kv8Layer& l, cudaStream_t stream) {
  const pf_config& c = *a.c;
  if (HD == 128 && a.M > TQ / (c.n_q_heads / c.n_kv_heads)) return launch<128, T, 1>(a, l, stream);
  return launch<HD, T, 0>(a, l, stream);
}

template <int HD, int T, int PAIR, int CL>
cudaError_t set_attr_cl() {
  using L = TSmem<HD, PAIR>;
  const auto kernel = attn_kv8_tc_kernel<HD, T, PAIR, CL>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e == cudaSuccess && CL > PORTABLE_CLUSTER) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int size = CL > PORTABLE_CLUSTER ? PORTABLE_CLUSTER + 1 : 2; size <= CL && e == cudaSuccess; ++size) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = L::BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;  // one CTA an SM whatever the instance: HD and T make no difference
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) g_active[PAIR][size] = n;
  }
  return e;
}

template <int HD, int T, int PAIR>
cudaError_t set_attr() {
  const cudaError_t e = set_attr_cl<HD, T, PAIR, PORTABLE_CLUSTER>(), f = set_attr_cl<HD, T, PAIR, MAX_CLUSTER>();
  return e != cudaSuccess ? e : f;
}

}  // namespace

cudaError_t prepare_attention_kv8_tc_kernels() {
  cudaError_t e = cudaSuccess, r;
  if ((r = set_attr<128, PF_KV_E4M3, 0>()) != cudaSuccess) e = r;
  if ((r = set_attr<128, PF_KV_INT8, 0>()) != cudaSuccess) e = r;
  if ((r = set_attr<128, PF_KV_E4M3, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr<128, PF_KV_INT8, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, PF_KV_E4M3, 0>()) != cudaSuccess) e = r;
  if ((r = set_attr<64, PF_KV_INT8, 0>()) != cudaSuccess) e = r;
  return e;
}

cudaError_t launch_attention_kv8_tc(const Kv8AttnArgs& a, const Kv8Layer& l, cudaStream_t stream) {
  const pf_config& c = *a.c;
  if (c.head_dim == 128)
    return c.kv_dtype == PF_KV_E4M3 ? launch_form<128, PF_KV_E4M3>(a, l, stream) : launch_form<128, PF_KV_INT8>(a, l, stream);
  return c.kv_dtype == PF_KV_E4M3 ? launch_form<64, PF_KV_E4M3>(a, l, stream) : launch_form<64, PF_KV_INT8>(a, l, stream);
}

}  // namespace pf

PF_TIMELINE_SETTER(attention_kv8_tc)
