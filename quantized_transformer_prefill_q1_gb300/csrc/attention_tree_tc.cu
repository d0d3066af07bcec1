// attention_tree_tc.cu — attention of many sequences' rows (trees of drafted tokens) over the cache on the
// 5th-generation tensor cores, for more rows per kv head than attention_tree.cu takes.
//
// The rows of one sequence and kv head (row = node * G + head in the group) in blocks of 256 are a task; its key
// units are tiles of 128 positions (a page). All tasks lie in one line, cut evenly over persistent CTAs whatever the
// lengths are (batch.cuh). A CTA holds two slots, each with 128 rows in the MMA's M side, its own S / P and O in tensor
// memory and 128 softmax threads, one a row: while one slot's softmax runs, the other's products do.
//   more than 128 rows: slot s takes rows 128 s .. +127 of every tile: K and V are read once for 256 rows;
//   128 rows or fewer:  both slots hold the same rows and take the tiles in turn; at the end their (m, l, O) are added.
//
// Warp roles:
//   warp 0      TMA: Q (3-D map over q[rows][nq][hd]), K and V tiles into one ring in the order the products need them,
//               across task borders (the next task's first tiles come before its Q);
//   warp 1      the MMAs, one elected lane issuing: S = Q K^T, O += P V with P from tensor memory over S's columns, V
//               MN-major as it lies in the cache. Products run in the order of issue, so the next S of a slot follows the
//               product that reads its P without a wait;
//   warps 2..5  softmax of slot 0 (tensor memory lane quarter = warp % 4), warps 6..9 of slot 1: a thread reads its row's
//               128 scores, hides the keys that the row does not see, exponentials in the exp2 domain, P back; the
//               running maximum is raised only when exceeded by more than 2^8 (then O is scaled in tensor memory).
// A task that lies in one CTA is written by it; parts of a cut one go to scratch as f32 and a second kernel merges
// them, a thread per row and eight columns.
//
// Measured (GB300, replayed graphs, bf16, 32/8 heads of 128): trees of 40 .. 64 nodes of eight sequences of 20,000 ..
// 32,700 positions (870 MB) 161 us, 0.81 of the copy rate with the tensor cores 61 % busy; under a load of seconds 186 us, the
// power cap's clocks. What bounds it is the softmax:
// a tile of 256 x 128 scores takes 1.8 us with its exponentials and the hand-over, the products alone 1.1 us. Short tasks
// cost about 5 us each beside their tiles, mostly waits of one role for the other (LEAD; with 0, 24 rows of each of 48
// sequences of 100 .. 900 positions took 61 us, with 1 / 2 / 4 45 / 42 / 40 us): 37 us.
//
// Rounding: P to the cache's type (the product's operand; for an f16 cache see M_DOWN; of a bf16 cache that is the largest error
// of the f16 output, 1.2e-3 in relative L2, as in the attention over one sequence: two bf16 terms, 2e-4, take 216 us instead of
// 162 on the case above and 15 to 20 % more on short tasks, since both the softmax and the products with V grow by a half), the
// output to f16; all else f32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "batch.cuh"

namespace pf {
namespace {

constexpr int TM = 128;      // rows of a slot
constexpr int BLOCK = 256;   // rows of a task
constexpr int TK = 128;      // keys per tile
constexpr int LEAD = 4;      // what a task costs beside its keys, in tiles (task_lead)
constexpr int HK = TK / 2;   // keys of one product with V
constexpr int THREADS = 320;
constexpr int SM_THREADS = 256;
constexpr float RESCALE_LOG2 = 8.f;
static_assert(TK == PF_KV_BLOCK, "a key tile is a page");
// The running maximum m of an f16 cache is kept 7 below the scores', so that the weights, their sum and O are 2^7 larger: up to
// 2^15 before m is raised, and with steps of 2^-31 of the largest at the small end instead of 2^-24, below which a long cache's
// many small weights would vanish together.
template <int BF16>
constexpr float M_DOWN = BF16 ? 0.f : 7.f;

template <int HD>
struct TSmem {
  static constexpr int QT = TM * HD * 2;   // a slot's Q
  static constexpr int KV = TK * HD * 2;   // a K or V tile
  static constexpr int NS = HD == 128 ? 5 : 10;
  static constexpr int BYTES = 1024 + 2 * QT + NS * KV + 512;
  static_assert(BYTES <= 232448 - TM * 8 - 256, "shared memory");  // beside the static arrays
};

struct TcParams {
  BatchDev B;
  int nq, nkv, layer;
  float scale_log2;
  __half* out;
  Line* line;       // the launch's line, for the merge
  int* prefix;      // the first unit of every sequence
  float* part;      // two places a CTA: [HD / 4][rows] float4, then (m, l) per row
  int part_rows;
  int* status;
};

__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < PF_WAIT_LIMIT_NS) {}
}
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ bool bar_and(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two f32 values in one register pair, for the packed multiply-add and addition.
__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 each(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Bits [0, n) set (n clamped to [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// A CTA's part of a task, as every role sees it.
struct Part {
  int kvh, rb, at, n, start;  // kv head, row block, the sequence's rows and start
  int rows;                   // rows of the task (of this block)
  int slots;                  // 2: the slots share the rows; 1: they share the tiles
  int u0, cnt;                // key tiles
  int all;                    // tiles of the task
  int units;                  // of the CTA's range: the tiles and the task's lead
};

template <int HD, int BF16>
__global__ void __launch_bounds__(THREADS, 1)
    attn_tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const TcParams P) {
  PF_TIMELINE(TL_ATTENTION_TREE_TC);
  using L = TSmem<HD>;
  constexpr int NH = HD / 64, NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_s;
  __shared__ float2 ml_s[TM];  // slot 1's (m, l), then both slots' factors
  volatile int* abort_flag = &abort_s;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t q_s = base, kv_s = q_s + 2 * L::QT, bar0 = kv_s + NS * L::KV;
  auto kv_full = [&](int s) { return bar0 + 8u * s; };
  auto kv_empty = [&](int s) { return bar0 + 8u * (NS + s); };
  auto s_full = [&](int s) { return bar0 + 8u * (2 * NS + s); };
  auto p_full = [&](int s, int h) { return bar0 + 8u * (2 * NS + 2 + 2 * s + h); };
  auto o_done = [&](int s) { return bar0 + 8u * (2 * NS + 6 + s); };
  auto o_empty = [&](int s) { return bar0 + 8u * (2 * NS + 8 + s); };
  const uint32_t q_full = bar0 + 8u * (2 * NS + 10), q_empty = q_full + 8, drain_bar = q_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + (q_full + 24 - raw));
  static_assert(8 * (2 * NS + 16) <= 512, "barrier area");
  const BatchDev& B = P.B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = P.nq / P.nkv;

  if (threadIdx.x == 64) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s, 0), TM);
      mbar_init(p_full(s, 1), TM);
      mbar_init(o_done(s), 1);
      mbar_init(o_empty(s), TM);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain_bar, 1);
    abort_s = 0;
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
  const int lead = task_lead(B, LEAD);
  auto work = [&](const SeqRows& s) -> SeqWork {
    return {P.nkv * ((s.n * G + BLOCK - 1) / BLOCK), s.n > 0 ? lead + (s.start + s.n + TK - 1) / TK : 0};
  };
  // a tile for each slot, as far as the work goes
  const int cta = blockIdx.x;
  const WorkStart ws = batch_scan<THREADS>(B, work, 2, cta == 0 ? P.prefix : nullptr, P.status);
  const Line& line = ws.line;
  if (cta == 0 && threadIdx.x == 0) *P.line = line;
  const int ub = cta < line.ctas ? line.begin(cta) : 0;
  const int count = cta < line.ctas ? line.begin(cta + 1) - ub : 0;
  WorkCursor<decltype(work)> cur;
  if (count > 0) cur.seek(B, work, ws.b, ub - ws.first);
  // the part of the task at the cursor that lies in this CTA's range, x units of which are done
  auto part = [&](int x) -> Part {
    Part p;
    const int blocks = cur.w.tasks / P.nkv;
    p.kvh = cur.task / blocks;
    p.rb = cur.task - p.kvh * blocks;
    p.at = cur.s.at;
    p.n = cur.s.n;
    p.start = cur.s.start;
    p.rows = min(BLOCK, p.n * G - p.rb * BLOCK);
    p.slots = p.rows > TM ? 2 : 1;
    p.units = min(cur.w.units - cur.u, count - x);
    p.u0 = max(cur.u - lead, 0);
    p.cnt = cur.u + p.units - lead - p.u0;  // below 1: the range ends before the task's keys
    p.all = cur.w.units - lead;
    return p;
  };
  // Order of a part's tiles in the ring: slots == 2: K0 V0 K1 V1 ..; slots == 1: K0 K1 V0 K2 V1 .. (the other
  // slot's scores come before the first slot's product).
  auto place_k = [](const Part& p, int j) { return p.slots == 2 ? 2 * j : max(0, 2 * j - 1); };
  auto place_v = [](const Part& p, int j) { return p.slots == 2 ? 2 * j + 1 : min(2 * j + 2, 2 * p.cnt - 1); };

  int issued = 0, q_issued = 0;  // copies of tiles and of Q (thread 0)
  if (warp == 0) {
    // ------------------------------------------------------------------ copies (lane 0; a lane each looks up the tiles' pages)
    int seg = 0;
    bool ok = true;
    for (int x = 0; x < count && ok; ++seg) {
      const Part p = part(x);
      if (p.cnt < 1) break;
      const int row0 = (P.layer * P.nkv + p.kvh) * B.slots;
      auto tile_row = [&](int j) {  // of tile j + lane
        int slot = 0;
        if (j + lane < p.cnt) {
          slot = batch_slot(B, cur.b, (p.u0 + j + lane) * TK);
          if (slot < 0) {
            batch_record(P.status, PF_ERR_KV_CAPACITY);
            slot = 0;
          }
        }
        return row0 + slot;
      };
      auto load = [&](const CUtensorMap* map, int row) {
        const int s = issued % NS;
        if (ok && lane == 0) {
          ok = mbar_wait(kv_empty(s), ((issued / NS) & 1) ^ 1, abort_flag);
          if (ok) {
            mbar_arrive_expect_tx(kv_full(s), L::KV);
            for (int h = 0; h < NH; ++h) tma_load_2d(kv_s + s * L::KV + h * (TK * 128), map, h * 64, row, kv_full(s));
            ++issued;
          }
        }
      };
      auto load_q = [&]() {
        if (ok && lane == 0) {
          if (seg > 0) ok = mbar_wait(q_empty, (seg - 1) & 1, abort_flag);
          if (ok) {
            mbar_arrive_expect_tx(q_full, p.slots * L::QT);
            for (int s = 0; s < p.slots; ++s)
              for (int h = 0; h < NH; ++h)
                tma_load_3d(q_s + s * L::QT + h * (TM * 128), &tm_q, h * 64, p.kvh * G, p.at + (p.rb * BLOCK + s * TM) / G, q_full);
            ++q_issued;
          }
        }
      };
      int rows = tile_row(0), rows_next = tile_row(32);  // 32 tiles, and the 32 after them
      // the tree towards L1, for the rows that look for their ancestors there
      if (B.parent != nullptr && 32 * lane < p.n && (p.u0 + p.cnt) * TK > p.start) prefetch_l1(B.parent + p.at + 32 * lane);
      if (seg == 0) load_q();
      const int lag = p.slots == 2 ? 0 : 1;  // V follows K by so many tiles
      int rv = 0;
      for (int j = 0; j < p.cnt + lag && ok; ++j) {
        if (j > 0 && (j & 31) == 0) {
          rows = rows_next;
          rows_next = tile_row(j + 32);
        }
        const int rk = __shfl_sync(0xffffffffu, rows, j & 31);
        if (j < p.cnt) load(&tm_k, rk);
        if (j >= lag) load(&tm_v, lag ? rv : rk);
        rv = rk;
        // at most four tiles before a later part's Q: the ring takes them without this part's products
        if (seg > 0 && j == min(1, p.cnt + lag - 1)) load_q();
        ok = __shfl_sync(0xffffffffu, ok, 0) != 0;
      }
      x += p.units;
      if (x < count) cur.advance(B, work, p.units);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    constexpr uint32_t idesc_s = idesc_f16(TM, TK, BF16, 0), idesc_o = idesc_f16(TM, HD, BF16, 1);
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)); };
    auto wait_kv = [&](int c) { return wait(kv_full(c % NS), (c / NS) & 1); };
    auto scores = [&](int slot, int q_slot, int c) {
      tc_fence_after();
      const uint32_t k = kv_s + (c % NS) * L::KV, q = q_s + q_slot * L::QT;
#pragma unroll
      for (int kc = 0; kc < HD / 16; ++kc)
        umma_f16_ss_warp(tmem + slot * TK, sdesc_kmajor_sw128(q + (kc >> 2) * (TM * 128) + (kc & 3) * 32),
                         sdesc_kmajor_sw128(k + (kc >> 2) * (TK * 128) + (kc & 3) * 32), idesc_s, kc > 0);
      umma_commit_warp(s_full(slot));
    };
    // the product with the V rows of a half of the tile's keys
    auto values = [&](int slot, int h, int c, bool add) {
      tc_fence_after();
      const uint32_t v = kv_s + (c % NS) * L::KV + h * (HK * 128);
#pragma unroll
      for (int kc = 0; kc < HK / 16; ++kc)
        umma_f16_ts_warp(tmem + 256 + slot * TK, tmem + slot * TK + h * HK + kc * 8, sdesc_mnmajor_sw128(v + kc * 2048, TK * 128), idesc_o,
                         add || kc > 0);
    };
    // The V of keys behind the sequence (from key nv of the tile on) may be anything, and a zero weight must not meet a NaN:
    // cleared here, while the softmax forms the weights.
    auto wait_v = [&](const Part& p, int j, int c) {
      if (!wait_kv(c)) return false;
      const int nv = p.start + p.n - (p.u0 + j) * TK;
      if (nv < TK) {
        const uint32_t vt = kv_s + (c % NS) * L::KV;
        for (int i = lane; i < NH * TK * 8; i += 32) {  // eight lanes a row of 64 columns
          const int key = (i >> 3) % TK;
          if (key >= nv)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + i * 16), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      return true;
    };
    int c0 = 0, seg = 0;
    int pc[2] = {0, 0};  // P tiles taken of each slot
    bool ok = true;
    for (int x = 0; x < count && ok; ++seg) {
      const Part p = part(x);
      if (p.cnt < 1) break;
      auto free_kv = [&](int c) { umma_commit_warp(kv_empty(c % NS)); };
      if (!(ok = wait(q_full, seg & 1))) break;
      if (p.slots == 2) {
        if (!(ok = wait_kv(c0))) break;
        scores(0, 0, c0);
        scores(1, 1, c0);
        free_kv(c0);
        if (p.cnt == 1) umma_commit_warp(q_empty);
        if (seg > 0 && !(ok = wait(o_empty(0), (seg - 1) & 1) && wait(o_empty(1), (seg - 1) & 1))) break;
        for (int j = 0; j < p.cnt && ok; ++j) {
          const int v = c0 + place_v(p, j), k = c0 + place_k(p, j + 1);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!(ok = ok && (s == 1 || wait_v(p, j, v)) && wait(p_full(s, 1), pc[s] & 1))) break;
            values(s, 1, v, j > 0);
            if (!(ok = wait(p_full(s, 0), pc[s] & 1))) break;
            values(s, 0, v, true);
            umma_commit_warp(o_done(s));
            ++pc[s];
            if (s == 1) free_kv(v);
            if (j + 1 < p.cnt) {
              if (!(ok = wait_kv(k))) break;
              scores(s, s, k);
              if (s == 1) {
                free_kv(k);
                if (j + 2 == p.cnt) umma_commit_warp(q_empty);
              }
            }
          }
        }
      } else {
        for (int j = 0; j < min(2, p.cnt) && ok; ++j) {
          const int k = c0 + place_k(p, j);
          if (!(ok = wait_kv(k))) break;
          scores(j, 0, k);
          free_kv(k);
        }
        if (!ok) break;
        if (p.cnt <= 2) umma_commit_warp(q_empty);
        if (seg > 0 && !(ok = wait(o_empty(0), (seg - 1) & 1) && wait(o_empty(1), (seg - 1) & 1))) break;
        for (int j = 0; j < p.cnt && ok; ++j) {
          const int s = j & 1, v = c0 + place_v(p, j), k = c0 + place_k(p, j + 2);
          if (!(ok = wait_v(p, j, v) && wait(p_full(s, 1), pc[s] & 1))) break;
          values(s, 1, v, j >= 2);
          if (!(ok = wait(p_full(s, 0), pc[s] & 1))) break;
          values(s, 0, v, true);
          umma_commit_warp(o_done(s));
          ++pc[s];
          free_kv(v);
          if (j + 2 < p.cnt) {
            if (!(ok = wait_kv(k))) break;
            scores(s, 0, k);
            free_kv(k);
            if (j + 3 == p.cnt) umma_commit_warp(q_empty);
          }
        }
      }
      c0 += 2 * p.cnt;
      x += p.units;
      if (x < count) cur.advance(B, work, p.units);
    }
    if (!ok) {
      umma_commit_warp(drain_bar);
      drain(drain_bar, 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax rows
    const int slot = (warp - 2) >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t sbuf = tmem + lane_off + slot * TK, obuf = tmem + lane_off + 256 + slot * TK;
    const float sl2 = P.scale_log2;
    int done = 0;  // tiles of this slot
    bool ok = true;
    // tcgen05.ld / st are warp-collective: every branch around them is warp-uniform
    for (int x = 0; x < count; ) {
      const Part p = part(x);
      if (p.cnt < 1) break;
      const int row = p.rb * BLOCK + (p.slots == 2 ? slot * TM : 0) + r;  // row of the sequence and kv head
      const int node = row / G;
      const bool mine = r < p.rows - (p.slots == 2 ? slot * TM : 0);
      float m = -INFINITY, l = 0.f;
      const int step = p.slots == 2 ? 1 : 2, j0 = p.slots == 2 ? 0 : slot;
      // Keys of a tile that the row sees: n0 = node of the tile's first key (negative: cached).
      auto sight = [&](int n0, uint32_t (&vis)[4]) {
#pragma unroll
        for (int w = 0; w < 4; ++w) vis[w] = low_bits((mine && B.parent == nullptr ? node + 1 : 0) - (n0 + 32 * w));
        if (mine && B.parent != nullptr) {
          for (int a = node; a >= 0 && a >= n0;) {  // ancestors come before their children
            const int e = a - n0;
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if ((e >> 5) == w) vis[w] |= 1u << (e & 31);
            bool bad;
            a = tree_parent(B.parent + p.at, a, bad);
            if (bad) batch_record(P.status, PF_ERR_INVALID_ARG);
          }
        }
        __syncwarp();
      };
      for (int j = j0; j < p.cnt; j += step) {
        const int key0 = (p.u0 + j) * TK;
        const bool tail = key0 + TK > p.start;  // the tile holds rows of the sequence itself, or what lies behind them
        uint32_t vis[4];
        if (tail) sight(key0 - p.start, vis);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(s_full(slot), done & 1, abort_flag)))) break;
        tc_fence_after();
        // The tile in halves of 64 keys, in loops: unrolled over a tile the code outgrows the instruction cache that two SMs
        // share. First the row's maximum, then the weights, the second half first; P takes the first 32 columns of its half's scores.
        uint32_t v[HK];
        auto load = [&](int h) {
          tmem_ld_32x32b_x32(sbuf + HK * h, *reinterpret_cast<uint32_t(*)[32]>(v));
          tmem_ld_32x32b_x32(sbuf + HK * h + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
          tmem_ld_wait();
        };
        float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (tail) {
          // Keys that the row does not see get the score -inf: it adds nothing to the maximum and has weight 0.
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t see = c == 0 ? vis[0] : (c == 1 ? vis[1] : (c == 2 ? vis[2] : vis[3]));
            uint32_t u[32];
            tmem_ld_32x32b_x32(sbuf + 32 * c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) u[e] = 0xff800000u;
            tmem_st_32x32b_x32(sbuf + 32 * c, u);
#pragma unroll
            for (int e = 0; e < 32; e += 2) mp[(e >> 1) & 3] = max3(mp[(e >> 1) & 3], __uint_as_float(u[e]), __uint_as_float(u[e + 1]));
          }
          tmem_st_wait();
        } else {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            load(h);
#pragma unroll
            for (int e = 0; e < HK; e += 2) mp[(e >> 1) & 3] = max3(mp[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
          }
        }
        const float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * sl2 - M_DOWN<BF16>;
        const bool need = mx > m + RESCALE_LOG2;
        if (j == j0) {
          m = mx;
        } else if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2(m - mx) : 1.f;
          l *= alpha;
          // O holds the tiles so far, whose products completed before this tile's scores
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
          if (need) m = mx;
        }
        const float neg_m = m == -INFINITY ? 0.f : -m;
        const uint64_t neg_two = two(neg_m, neg_m), sl2_two = two(sl2, sl2);
        uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll 1
        for (int h = 1; h >= 0; --h) {
          load(h);
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 u = each(fma_two(two(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sl2_two, neg_two));
            const float p0 = ex2(u.x), p1 = ex2(u.y);
            ls[e & 3] = add_two(ls[e & 3], two(p0, p1));
            pk[e] = pack2<BF16>(p0, p1);
          }
          tmem_st_32x32b_x32(sbuf + HK * h, pk);
          // a half's product starts while the other half's weights are formed
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(p_full(slot, h));
        }
        const float2 sum = each(add_two(add_two(ls[0], ls[1]), add_two(ls[2], ls[3])));
        l += sum.x + sum.y;
        ++done;
      }
      // ------------------------------------------------------------------ the part's end
      WorkCursor<decltype(work)> nxt = cur;  // looked up while the last product runs
      if (x + p.units < count) nxt.advance(B, work, p.units);
      const int tiles = p.slots == 2 ? p.cnt : (p.cnt - slot + 1) / 2;
      if (ok && tiles > 0) ok = __all_sync(0xffffffffu, mbar_wait(o_done(slot), (done - 1) & 1, abort_flag));
      if (p.slots == 1 && slot == 1) ml_s[r] = make_float2(m, l);
      if (!bar_and(1, SM_THREADS, ok)) break;
      tc_fence_after();
      const bool whole = p.cnt == p.all;
      const int task_first = ub + x - cur.u;
      float* place = P.part + line.place(cta, task_first) * (static_cast<size_t>(P.part_rows) * (HD + 2));
      __half* dst = P.out + (static_cast<size_t>(p.at + node) * P.nq + p.kvh * G + (row - node * G)) * HD;
      const int pr = row - p.rb * BLOCK;  // row of the place
      // 32 columns of the row's O: to the output, or as they are to the part's place
      auto put = [&](int c, const float* o, float inv) {
        if (!mine) return;
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t h[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const __half2 a = __floats2half2_rn(o[e + 2 * y] * inv, o[e + 2 * y + 1] * inv);
              h[y] = *reinterpret_cast<const uint32_t*>(&a);
            }
            *reinterpret_cast<uint4*>(dst + 32 * c + e) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            reinterpret_cast<float4*>(place)[static_cast<size_t>(8 * c + e / 4) * P.part_rows + pr] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      };
      auto put_ml = [&](float mm, float ll) {
        if (mine && !whole) reinterpret_cast<float2*>(place + static_cast<size_t>(P.part_rows) * HD)[pr] = make_float2(mm, ll);
      };
      if (p.slots == 2) {
        put_ml(m, l);
        const float inv = 1.f / l;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(obuf + 32 * c, o);
          tmem_ld_wait();
          put(c, reinterpret_cast<const float*>(o), inv);
        }
      } else {
        // The slots' sums meet where they are: a thread reads its row of both O's, slot 0 for the first half of the columns, slot 1
        // for the second. Slot 0 forms the factors from slot 1's (m, l) and hands them over.
        float2 f;
        if (slot == 0) {
          const float2 y = ml_s[r];
          const float mm = fmaxf(m, y.x);
          f = make_float2(m == -INFINITY ? 0.f : ex2(m - mm), y.x == -INFINITY ? 0.f : ex2(y.x - mm));
          const float ll = f.x * l + f.y * y.y;
          put_ml(mm, ll);
          if (whole) f = make_float2(f.x / ll, f.y / ll);
          ml_s[r] = f;
        }
        bar_sync(1, SM_THREADS);
        if (slot == 1) f = ml_s[r];
#pragma unroll 1
        for (int c = slot * (HD / 64); c < (slot + 1) * (HD / 64); ++c) {
          uint32_t o[2][32];
          tmem_ld_32x32b_x32(tmem + lane_off + 256 + 32 * c, o[0]);
          tmem_ld_32x32b_x32(tmem + lane_off + 256 + TK + 32 * c, o[1]);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {  // without a tile slot 1 holds anything; a factor of 0 keeps a NaN of V
            const float u = f.x * __uint_as_float(o[0][e]);
            v[e] = p.cnt > 1 ? fmaf(f.y, __uint_as_float(o[1][e]), u) : u;
          }
          put(c, v, 1.f);
        }
      }
      tc_fence_before();
      mbar_arrive(o_empty(slot));
      x += p.units;
      cur = nxt;
    }
  }

  tc_fence_before();
  __syncthreads();
  griddep_launch_dependents();  // not earlier: a merge that starts while few SMs are free gathers on those
  if (warp == 1) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) {
    // let copies in flight land before shared memory is released, whichever role gave up and when
    if (q_issued > 0) drain(q_full, (q_issued - 1) & 1);
    for (int k = max(0, issued - NS); k < issued; ++k) drain(kv_full(k % NS), (k / NS) & 1);
    batch_record(P.status, PF_ERR_DEVICE_TIMEOUT);
  }
}

// Merges the parts of cut tasks: with m* the largest of the parts' maxima, O = sum_c 2^(m_c - m*) O_c / sum_c 2^(m_c - m*) l_c.
// CTA = MR rows of a (sequence, kv head); a thread takes a row, eight columns and every GROUPS-th part, PF of them in
// flight. A part in which a row saw no key (m = -inf) has the factor 0 and is added like the others: l is NaN where all scores
// that the row saw were (the maximum ignores a NaN), and O where V of a hidden key was; both reach the row wherever the line is cut.
template <int HD, int MR, int GROUPS, int PF, int CTAS>
__global__ void __launch_bounds__(MR* HD / 8 * GROUPS, CTAS) tree_merge_kernel(const BatchDev B, int nq, int nkv, const Line* line_p,
                                                                               const int* prefix, const float* part, int part_rows,
                                                                               __half* out) {
  PF_TIMELINE(TL_TREE_MERGE);
  constexpr int COLS = HD / 8;
  __shared__ float join[GROUPS > 1 ? (GROUPS - 1) * MR * COLS * 10 : 1];
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.z, kvh = blockIdx.y, G = nq / nkv;
  const SeqRows s = batch_seq(B, b, true);
  const Line line = *line_p;
  const int seq_first = prefix[b];
  const int rows = s.n * G;
  if (static_cast<int>(blockIdx.x) * MR >= rows) return;
  const int row = blockIdx.x * MR + threadIdx.x % MR, oct = threadIdx.x / MR % COLS, group = threadIdx.x / (MR * COLS);
  const int rb = blockIdx.x * MR / BLOCK, blocks = (rows + BLOCK - 1) / BLOCK, lead = task_lead(B, LEAD);
  const int units = lead + (s.start + s.n + TK - 1) / TK;
  const int first = seq_first + (kvh * blocks + rb) * units;
  const int c0 = line.owner(first + lead), c1 = line.owner(first + units - 1);
  if (c0 == c1) return;  // the same for the whole CTA: its rows lie in one block
  const int pr = min(row, rows - 1) - rb * BLOCK, place0 = line.place(c0, first);
  float mr = -INFINITY, lr = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto add = [&](float m, float l, const float* w) {
    const float mn = fmaxf(mr, m);
    const float a = mr == -INFINITY ? 0.f : ex2(mr - mn), f = m == -INFINITY ? 0.f : ex2(m - mn);
    mr = mn;
    lr = lr * a + f * l;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = acc[e] * a + f * w[e];
  };
  for (int c = c0 + group; c <= c1; c += PF * GROUPS) {
    float4 v[PF][2];
    float2 ml[PF];
#pragma unroll
    for (int y = 0; y < PF; ++y) {
      const int p = c + y * GROUPS;
      if (p > c1) break;
      const float* src = part + (p == c0 ? place0 : 2 * p) * (static_cast<size_t>(part_rows) * (HD + 2));
      ml[y] = __ldcg(reinterpret_cast<const float2*>(src + static_cast<size_t>(part_rows) * HD) + pr);
#pragma unroll
      for (int u = 0; u < 2; ++u) v[y][u] = __ldcg(reinterpret_cast<const float4*>(src) + static_cast<size_t>(2 * oct + u) * part_rows + pr);
    }
#pragma unroll
    for (int y = 0; y < PF; ++y) {
      if (c + y * GROUPS > c1) break;
      add(ml[y].x, ml[y].y, reinterpret_cast<const float*>(v[y]));
    }
  }
  if (GROUPS > 1) {
    float* mine = join + (threadIdx.x - MR * COLS);  // [value][thread of the groups behind the first]
    constexpr int STRIDE = (GROUPS - 1) * MR * COLS;
    if (group > 0) {
      mine[0] = mr;
      mine[STRIDE] = lr;
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[(2 + e) * STRIDE] = acc[e];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g + 1 < GROUPS; ++g) {
      const float* other = join + g * MR * COLS + threadIdx.x;
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = other[(2 + e) * STRIDE];
      add(other[0], other[STRIDE], w);
    }
  }
  if (row >= rows) return;
  const float inv = 1.f / lr;
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 x = __floats2half2_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    h[e] = *reinterpret_cast<const uint32_t*>(&x);
  }
  const int node = row / G;
  *reinterpret_cast<uint4*>(out + (static_cast<size_t>(s.at + node) * nq + kvh * G + row - node * G) * HD + 8 * oct) = make_uint4(h[0], h[1], h[2], h[3]);
}

constexpr size_t LINE_BYTES = 64;
static_assert(sizeof(Line) <= LINE_BYTES, "the line's place in the scratch");
size_t plan_bytes(int n_seq) { return LINE_BYTES + (static_cast<size_t>(n_seq) + 63) / 64 * 64 * sizeof(int); }
int place_rows(const pf_config& c, int max_rows) { return std::min(BLOCK, (max_rows * (c.n_q_heads / c.n_kv_heads) + 31) / 32 * 32); }

template <int HD, int BF16>
cudaError_t launch_tc(const TreeAttnArgs& a, cudaStream_t stream) {
  const pf_config& c = *a.c;
  const int G = c.n_q_heads / c.n_kv_heads;
  const uint64_t dims[2] = {HD, static_cast<uint64_t>(c.n_layers) * c.n_kv_heads * cache_slots(c)}, strides[1] = {HD * 2};
  const uint32_t box[2] = {64, TK};
  const uint64_t qd[3] = {HD, static_cast<uint64_t>(c.n_q_heads), static_cast<uint64_t>(a.b->n_rows)};
  const uint64_t qs[2] = {HD * 2, static_cast<uint64_t>(c.n_q_heads) * HD * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(TM / G)};
  CUtensorMap tq, tk, tv;
  if (!encode_tmap_16(&tq, BF16, 3, a.q, qd, qs, qb) || !encode_tmap_16(&tk, BF16, 2, a.k_cache, dims, strides, box) ||
      !encode_tmap_16(&tv, BF16, 2, a.v_cache, dims, strides, box))
    return cudaErrorInvalidValue;
  const int max_rows = std::min(a.b->max_rows, a.b->n_rows);
  TcParams p{};
  p.B = batch_dev(c, *a.b);
  p.nq = c.n_q_heads;
  p.nkv = c.n_kv_heads;
  p.layer = a.layer;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HD));
  p.out = static_cast<__half*>(a.out);
  uint8_t* at = static_cast<uint8_t*>(a.scratch) + TREE_COUNTER_BYTES;
  p.line = reinterpret_cast<Line*>(at);
  p.prefix = reinterpret_cast<int*>(at + LINE_BYTES);
  p.part = reinterpret_cast<float*>(at + plan_bytes(a.b->n_seq));
  p.part_rows = place_rows(c, max_rows);
  p.status = a.status;
  const int ctas = std::min(device_sm_count(), GEMM_MAX_CTAS);
  const cudaError_t e = launch_pdl(attn_tree_tc_kernel<HD, BF16>, dim3(ctas), dim3(THREADS), TSmem<HD>::BYTES, stream, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  // Few rows may have many parts: eight rows a CTA and the parts in four groups spread them over the SMs; many rows have few
  // parts each. Both sides measured, with eight rows a CTA against sixteen, attention included: one tree of 26 nodes 15.2
  // and 17.6 us; four trees of 40 nodes 40.4 and 36.7, eight of up to 64 191 and 172.
  const int rows = max_rows * G;
  auto merge = [&](auto kernel, int per, int threads) {
    return launch_pdl(kernel, dim3((rows + per - 1) / per, c.n_kv_heads, a.b->n_seq), dim3(threads), 0, stream, p.B, p.nq, p.nkv,
                      static_cast<const Line*>(p.line), static_cast<const int*>(p.prefix), static_cast<const float*>(p.part),
                      p.part_rows, p.out);
  };
  const int64_t small = static_cast<int64_t>((rows + 7) / 8) * c.n_kv_heads * a.b->n_seq;
  return small <= 2 * ctas ? merge(tree_merge_kernel<HD, 8, 4, 5, 1>, 8, 4 * HD)
                           : merge(tree_merge_kernel<HD, 16, 1, 4, 4>, 16, 2 * HD);
}

template <int HD, int BF16>
cudaError_t set_attr_tc() {
  return cudaFuncSetAttribute(attn_tree_tc_kernel<HD, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, TSmem<HD>::BYTES);
}

}  // namespace

size_t attention_tree_tc_scratch_bytes(const pf_config& c, int n_seq, int max_rows) {
  return TREE_COUNTER_BYTES + plan_bytes(n_seq) + static_cast<size_t>(GEMM_MAX_CTAS) * 2 * place_rows(c, max_rows) * (c.head_dim + 2) * sizeof(float);
}

cudaError_t prepare_attention_tree_tc_kernels() {
  cudaError_t e = cudaSuccess, r;
  if ((r = set_attr_tc<128, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr_tc<128, 0>()) != cudaSuccess) e = r;
  if ((r = set_attr_tc<64, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr_tc<64, 0>()) != cudaSuccess) e = r;
  return e;
}

cudaError_t launch_attention_tree_tc(const TreeAttnArgs& a, cudaStream_t stream) {
  const bool bf = a.c->kv_dtype == PF_KV_BF16;
  if (a.c->head_dim == 128) return bf ? launch_tc<128, 1>(a, stream) : launch_tc<128, 0>(a, stream);
  return bf ? launch_tc<64, 1>(a, stream) : launch_tc<64, 0>(a, stream);
}

}  // namespace pf

PF_TIMELINE_SETTER(attention_tree_tc)
