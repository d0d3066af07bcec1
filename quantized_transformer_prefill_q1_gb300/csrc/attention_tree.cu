// attention_tree.cu — attention of many sequences' rows (trees of drafted tokens, single tokens) over the cache,
// few rows per kv head; more rows go to attention_tree_tc.cu.
//
// For row i of a sequence and its head h (kv head h / G) over the keys j that it sees (the cached positions, its
// ancestors, itself): s_j = q . k_j / sqrt(hd), p = softmax_j(s), o = sum_j p_j v_j.
//
// The cache is read once and nothing else weighs, so the kernel streams it: all (sequence, kv head) tasks in one
// line of units of 32 keys, cut evenly over the CTAs whatever the lengths are (batch.cuh), and a CTA's units in runs over
// its 4 warps. A warp has its own ring of TMA stages, which it refills itself across task borders, and its own running
// maximum m, sum l and O: the copies never wait for a task's end, and a warp writes the tasks that lie in its run by itself.
// Parts of tasks that a border cuts stay in shared memory to the end; there they are added, and of a task with keys in
// other CTAs the sum goes to scratch, where the CTA that completes the task's count adds all. LEAD: a task costs a warp
// about 2 us beside its keys.
//
// The rows of one kv head (row = node * G + head in the group, at most FEW_ROWS) are the n side of warp-level MMAs
// m16n8k16: S^T [keys x rows] = K [16 keys x 16 d] Q^T and O^T [d x rows] += V^T [16 d x 16 keys] P^T, K and V as A
// operands by ldmatrix (V transposed on the way); P^T comes from S^T by a register transpose (movmatrix). The tensor
// cores are 12 % busy with it; 128 rows in tensor memory would be 16 times too many.
// The running maximum is raised only when exceeded by more than 2^8.
//
// Measured (GB300, replayed graphs, 32/8 heads of 128, bf16): one token of each of 48 sequences of 300 .. 8,100 positions
// (827 MB) 131 us, 6.3 TB/s: HBM. 48 of 100 .. 900 positions 21 us, 200 of 1 .. 300 33 us: the 2 us a task. One
// token at 513 / 8,190 / 32,001 positions 8.0 / 10.4 / 27.5 us: launch, first copies, the merge of 5 / 19 / 19 parts.
// The units in turns over the warps, which met at every task's end: 131, 26, 49, 7.6 us. LEAD 0: 135, 27, 56 us; 2 to 6
// within 5 % of one another.
//
// Rounding: P to f16 (see M_DOWN), or for a bf16 cache to two bf16 terms (the product with V takes operands of one type; one
// term would be the largest error of the f16 output, 1.2e-3 against 2e-4 in relative L2, and the second costs nothing beside the
// copies), the output to f16; all else f32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "batch.cuh"

namespace pf {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int UK = 32;   // keys per unit
constexpr int LEAD = 4;  // what a task costs beside its keys, in units (task_lead)
constexpr float RESCALE_LOG2 = 8.f;
// The running maximum m of an f16 cache is kept 7 below the scores', so that the weights, their sum and O are 2^7 larger: up to
// 2^15 before m is raised, and with steps of 2^-31 of the largest at the small end instead of 2^-24, below which a long cache's
// many small weights would vanish together.
template <int BF16>
constexpr float M_DOWN = BF16 ? 0.f : 7.f;
// Most rows per kv head of this form: the n side of an MMA. Both sides measured with 8 rows of 32/8 heads of 128, this form
// against attention_tree_tc.cu: one sequence at 512 / 8,190 positions 9.4 against 10.4 and 12.3 against 13.8 us, 48
// sequences of 100 .. 900 24.7 against 30.4, of 300 .. 8,100 133 against 132. With 16 rows (two such sides) one
// sequence took 32.9 us here and 14.6 there, 16 sequences 91 and 63.
constexpr int FEW_ROWS = 8;

template <int HD>
struct FSmem {
  static constexpr int WS = HD == 64 ? 6 : 3;  // stages of a warp's ring: 192 KB in flight an SM
  static constexpr int NS = WARPS * WS;
  static constexpr int TILE = UK * HD * 2;                       // bytes of a K or V unit
  static constexpr int RING = NS * 2 * TILE;
  static constexpr int ROWS = FEW_ROWS;
  static constexpr int OW = HD + 4;  // floats between rows of the warps' O
  static constexpr int PARTS = 2 * WARPS * ROWS * (OW + 2) * 4;  // two places a warp: O, then (m, l)
  static constexpr int BYTES = 1024 + RING + PARTS + NS * 8;
  static_assert(BYTES <= 232448 - 384, "shared memory");  // beside the static arrays
};

// A warp's part of a cut task in shared memory.
struct WarpPart {
  int rows;   // 0: none
  int first;  // the task's first unit in the line
  int c0, c1; // CTAs that hold its first and its last key units
  int at, kvh;
};

struct FewParams {
  BatchDev B;
  const uint16_t* q;
  int nq, nkv, layer;
  float scale_log2;
  __half* out;
  int* counters;  // one per CTA: arrivals of the cut task whose first key units it holds (its last task, so there is one)
  float* part;    // two places a CTA: [rows][HD], then (m, l) per row
  int* status;
};

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
template <int BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// 16-byte chunk `chunk` of key `row` in a unit: boxes of 64 elements (128-byte rows, chunk ^ row % 8)
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int row, int chunk) {
  return tile + (chunk >> 3) * (UK * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int HD, int BF16>
__global__ void __launch_bounds__(THREADS, 1)
    attn_tree_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const FewParams P) {
  PF_TIMELINE(TL_ATTENTION_TREE);
  using L = FSmem<HD>;
  constexpr int KS = HD / 16, DT = HD / 16, NH = HD / 64, ROWS = L::ROWS, NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_s, last_s[2];
  __shared__ WarpPart part_s[2 * WARPS];
  __shared__ int issued_s[NS];  // copies that each stage has taken (its own warp's lane 0 counts)
  volatile int* abort_flag = &abort_s;
  const uint32_t raw = smem_u32(smem_raw), ring = (raw + 1023u) & ~1023u;
  const uint32_t bars = ring + L::RING + L::PARTS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const BatchDev& B = P.B;
  const int G = P.nq / P.nkv;
  griddep_launch_dependents();
  if (threadIdx.x == 32) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (threadIdx.x < NS) {
    mbar_init(bars + 8 * threadIdx.x, 1);
    issued_s[threadIdx.x] = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) abort_s = 0;
  if (threadIdx.x < 2 * WARPS) part_s[threadIdx.x].rows = 0;
  __syncthreads();
  griddep_wait();
  const int lead = task_lead(B, LEAD);
  auto work = [&](const SeqRows& s) -> SeqWork { return {P.nkv, s.n > 0 ? lead + (s.start + s.n + UK - 1) / UK : 0}; };
  // every CTA has a unit for each warp, as far as the work goes
  const WorkStart ws = batch_scan<THREADS>(B, work, WARPS, nullptr, P.status);
  const Line& line = ws.line;
  const int cta = blockIdx.x;
  if (cta >= line.ctas) return;
  // the warp's units: a run of the CTA's
  const int ub = line.begin(cta), count = line.begin(cta + 1) - ub;
  const int wb = warp * (count / WARPS) + min(warp, count % WARPS), we = wb + count / WARPS + (warp < count % WARPS ? 1 : 0);

  WorkCursor<decltype(work)> cur, iss;
  cur.seek(B, work, ws.b, ub - ws.first);
  if (wb < we) cur.advance(B, work, wb);
  // the warp's next copy: its place in the line, as a row of the cache
  iss = cur;
  int iu = wb;
  int irow = 0;
  auto locate = [&]() {  // the next unit with keys from iss on
    const int d = max(0, lead - iss.u);
    iu += d;
    if (iu >= we) return;
    iss.u += d;
    int slot = batch_slot(B, iss.b, (iss.u - lead) * UK);
    if (slot < 0) {
      if (lane == 0) batch_record(P.status, PF_ERR_KV_CAPACITY);
      slot = 0;
    }
    irow = (P.layer * P.nkv + iss.task) * B.slots + slot;
  };
  auto issue = [&](int st) {
    if (lane == 0) {
      const uint32_t dst = ring + st * (2 * L::TILE), bar = bars + 8 * st;
      ++issued_s[st];
      mbar_arrive_expect_tx(bar, 2 * L::TILE);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        tma_load_2d(dst + h * (UK * 128), &tm_k, 64 * h, irow, bar);
        tma_load_2d(dst + L::TILE + h * (UK * 128), &tm_v, 64 * h, irow, bar);
      }
    }
    if (++iu < we) {
      iss.advance(B, work, 1);
      locate();
    }
  };
  if (iu < we) locate();
#pragma unroll 1
  for (int y = 0; y < L::WS; ++y)
    if (iu < we) issue(warp * L::WS + y);

  float* os = reinterpret_cast<float*>(smem_raw + (ring - raw) + L::RING);  // O [place][row][OW]
  float2* mls = reinterpret_cast<float2*>(os + 2 * WARPS * ROWS * L::OW);   // (m, l) [place][row]
  constexpr int LPR = HD / 4;  // lanes per row, four columns each
  constexpr int RPW = 32 / LPR;  // rows side by side in a warp
  const int col = (lane % LPR) * 4, rl = lane / LPR;
  auto store_out = [&](int at, int kvh, int r, float4 v, float f) {
    const __half2 a = __floats2half2_rn(v.x * f, v.y * f), c = __floats2half2_rn(v.z * f, v.w * f);
    *reinterpret_cast<uint2*>(P.out + (static_cast<size_t>(at + r / G) * P.nq + kvh * G + r % G) * HD + col) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
  };

  const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kch = lane >> 4;   // ldmatrix address of K: keys x chunks
  const int vrow = (lane & 7) + (lane >> 4) * 8, vch = (lane >> 3) & 1;  // of V (transposed)
  int st = 0, ph = 0;   // stage of the warp's ring, and phase
  bool failed = false;  // after a timeout
  for (int x = wb; x < we;) {
    const int u0 = cur.u - lead, cnt = min(cur.w.units - cur.u, we - x);  // key units from u0 (below 0: the lead) on
    if (u0 + cnt <= 0) break;  // the range ends before the task's keys
    const int kvh = cur.task, at = cur.s.at, n = cur.s.n, start = cur.s.start, len = start + n, R = n * G;
    float o[DT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    uint32_t qf[KS][2];  // Q^T as the B operand: row g
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(P.q + (static_cast<size_t>(at + g / G) * P.nq + kvh * G + g % G) * HD) + t;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) qf[k][e] = g < R ? src[8 * k + 4 * e] : 0u;
    // the next task's rows and tree towards L1
    WorkCursor<decltype(work)> nxt = cur;
    if (x + cnt < we) {
      nxt.advance(B, work, cnt);
      const int r = lane / NH;
      if (r < nxt.s.n * G)
        prefetch_l1(P.q + (static_cast<size_t>(nxt.s.at + r / G) * P.nq + nxt.task * G + r % G) * HD + 64 * (lane % NH));
      if (B.parent != nullptr && lane == 0) prefetch_l1(B.parent + nxt.s.at);
    }
    // nodes that the lane's rows (2t, 2t + 1) see, while the first unit is on its way
    uint32_t see[2];
    const bool own_keys = (u0 + cnt) * UK > start;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * t + e, node = r / G;
      see[e] = 0;
      if (r >= R || !own_keys) continue;
      if (B.parent == nullptr) {
        see[e] = (2u << node) - 1u;
      } else {
        for (int j = node; j >= 0;) {
          bool bad;
          see[e] |= 1u << j;
          j = tree_parent(B.parent + at, j, bad);
          if (bad) batch_record(P.status, PF_ERR_INVALID_ARG);
        }
      }
    }
    for (int unit = max(u0, 0); unit < u0 + cnt; ++unit) {
      const int key0 = unit * UK;
      const int stage = warp * L::WS + st;
      const uint32_t kt = ring + stage * (2 * L::TILE), vt = kt + L::TILE;
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, ph, abort_flag))) {
        failed = true;
        break;
      }
      const bool tail = key0 + UK > start;
      if (key0 + UK > len) {  // values behind the sequence may be anything: a zero weight must not meet a NaN
        for (int y = lane; y < UK * (HD / 8); y += 32) {
          const int row = y / (HD / 8);
          if (key0 + row >= len)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(chunk_at(vt, row, y % (HD / 8))), "r"(0) : "memory");
        }
        fence_proxy_async_smem();  // before the copy that refills the stage
        __syncwarp();
      }
      // scores of 32 keys: two tiles of 16
      float sc[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mt][e] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t a[4];
          ldsm4(a, chunk_at(kt, 16 * mt + krow, 2 * k + kch));
          mma16816<BF16>(sc[mt], a, qf[k][0], qf[k][1]);
        }
      if (tail) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = key0 + 16 * mt + 8 * (e >> 1) + g - start;  // node of the key
            if (j >= 0 && (j >= n || !(see[e & 1] >> j & 1u))) sc[mt][e] = -INFINITY;
          }
      }
      float mx[2];
      bool raise = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(fmaxf(sc[0][e], sc[0][e + 2]), fmaxf(sc[1][e], sc[1][e + 2])) * P.scale_log2;
        raise |= mx[e] > m[e] + (RESCALE_LOG2 + M_DOWN<BF16>);
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = mx[e];
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
          const float mn = fmaxf(m[e], y - M_DOWN<BF16>);
          const float alpha = mn == -INFINITY ? 1.f : ex2(m[e] - mn);
          m[e] = mn;
          l[e] *= alpha;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            o[d][e] *= alpha;
            o[d][e + 2] *= alpha;
          }
        }
      }
      // P^T as the B operand: [16-key tile][register]; of a bf16 cache as two terms, hi + lo
      uint32_t pf[2][2], pl[2][2];
      const float n0 = m[0] == -INFINITY ? 0.f : -m[0], n1 = m[1] == -INFINITY ? 0.f : -m[1];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float p0 = ex2(fmaf(sc[mt][2 * hh], P.scale_log2, n0)), p1 = ex2(fmaf(sc[mt][2 * hh + 1], P.scale_log2, n1));
          l[0] += p0;
          l[1] += p1;
          const uint32_t hi = pack2<BF16>(p0, p1);
          pf[mt][hh] = transpose8x8(hi);
          if (BF16) pl[mt][hh] = transpose8x8(pack2<BF16>(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u)));
        }
#pragma unroll
      for (int kt2 = 0; kt2 < 2; ++kt2)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          uint32_t a[4];
          ldsm4_t(a, chunk_at(vt, 16 * kt2 + vrow, 2 * d + vch));
          if (BF16) mma16816<BF16>(o[d], a, pl[kt2][0], pl[kt2][1]);
          mma16816<BF16>(o[d], a, pf[kt2][0], pf[kt2][1]);
        }
      __syncwarp();  // every lane has read the stage
      if (iu < we) issue(stage);
      if (++st == L::WS) {
        st = 0;
        ph ^= 1;
      }
    }
    if (failed) break;
    // O and (m, l) to one of the warp's places: of a task that began before the warp's range (or with it) the first, else the
    // second, which only the warp's last task may need for a part; the whole ones before it pass through it to the output.
    const int first = ub + x - cur.u;
    const bool whole = u0 <= 0 && u0 + cnt == cur.w.units - lead;
    const int place = 2 * warp + (whole || first > ub + wb ? 1 : 0);
    if (!whole) {
      const WarpPart T{R, first, line.owner(first + lead), line.owner(first + cur.w.units - 1), at, kvh};
      if (lane == 0) part_s[place] = T;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * t + e;
      float y = l[e];
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
      if (g == 0) mls[place * ROWS + r] = make_float2(m[e], y);
      float* dst = os + (place * ROWS + r) * L::OW + g;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        dst[16 * d] = o[d][e];
        dst[16 * d + 8] = o[d][e + 2];
      }
    }
    if (whole) {
      __syncwarp();
      constexpr int RB = 4;  // rows at once: their loads overlap
      for (int r0 = rl; r0 < R; r0 += RB * RPW) {
        float4 v[RB];
        float inv[RB];
#pragma unroll
        for (int y = 0; y < RB; ++y) {
          const int r = place * ROWS + min(r0 + y * RPW, R - 1);
          v[y] = *reinterpret_cast<const float4*>(os + r * L::OW + col);
          inv[y] = 1.f / mls[r].y;
        }
#pragma unroll
        for (int y = 0; y < RB; ++y)
          if (r0 + y * RPW < R) store_out(at, kvh, r0 + y * RPW, v[y], inv[y]);
      }
    }
    x += cnt;
    cur = nxt;
  }

  // ------------------------------------------------------------------ parts of cut tasks
  // At most eight parts of five tasks lie in shared memory. Those of a task with keys in other CTAs too are added and go
  // to scratch, where the CTA that completes the task's count adds them; of the others the sum is the result.
  failed = __syncthreads_or(failed) != 0;
  // row r of place p and of the first places of the warps behind it, up to warp w1: maximum, sum and the lane's four columns
  auto add_row = [&](int p, int w1, int r, float& mr, float& lr) {
    float mw[WARPS];
    mr = -INFINITY;
    lr = 0.f;
    const int w0 = p >> 1;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      mw[w] = w >= w0 && w <= w1 ? mls[(w == w0 ? p : 2 * w) * ROWS + r].x : -INFINITY;
      mr = fmaxf(mr, mw[w]);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < w0 || w > w1) continue;
      const int i = (w == w0 ? p : 2 * w) * ROWS + r;
      const float a = mw[w] == -INFINITY ? 0.f : ex2(mw[w] - mr);
      const float4 v = *reinterpret_cast<const float4*>(os + i * L::OW + col);
      lr = fmaf(a, mls[i].y, lr);
      acc = make_float4(fmaf(a, v.x, acc.x), fmaf(a, v.y, acc.y), fmaf(a, v.z, acc.z), fmaf(a, v.w, acc.w));
    }
    return acc;
  };
  constexpr size_t PLACE = static_cast<size_t>(ROWS) * (HD + 2);
  // lane p looks at place p: first parts of a task; parts of one that began in an earlier warp; of one with others elsewhere
  const WarpPart& own = part_s[lane & (2 * WARPS - 1)];
  const bool some = lane < 2 * WARPS && own.rows > 0;
  const int first0 = own.first, first1 = __shfl_up_sync(0xffffffffu, some ? first0 : -1, 1), first2 = __shfl_up_sync(0xffffffffu, some ? first0 : -1, 2);
  const bool goes_on = some && lane >= 2 && !(lane & 1) && (first0 == first1 || first0 == first2);
  const unsigned all = __ballot_sync(0xffffffffu, some), later = __ballot_sync(0xffffffffu, goes_on), starts = all & ~later;
  const unsigned apart = __ballot_sync(0xffffffffu, some && own.c0 != own.c1);
  // f(task, its first place, the warp of its last)
  auto each_task = [&](unsigned places, auto f) {
    for (; places != 0; places &= places - 1) {
      const int p = __ffs(places) - 1;
      int w1 = p >> 1;
      // a warp's second place, where it has one, is what goes on in the next warp
      while ((later >> (2 * w1 + 2) & 1u) && (p == 2 * w1 + 1 || !(all >> (2 * w1 + 1) & 1u))) ++w1;
      f(part_s[p], p, w1);
    }
  };
  int cut[2] = {0, 0}, cuts = 0;  // first places of the tasks with parts in other CTAs
  if (!failed)
    each_task(starts & apart, [&](const WarpPart& T, int p, int w1) {
      float* mine = P.part + (2 * cta + (T.first > ub ? 1 : 0)) * PLACE;  // line.place(cta, ..)
      for (int r = warp * RPW + rl; r < T.rows; r += WARPS * RPW) {
        float mr, lr;
        const float4 acc = add_row(p, w1, r, mr, lr);
        *reinterpret_cast<float4*>(mine + r * HD + col) = acc;
        if (col == 0) reinterpret_cast<float2*>(mine + ROWS * HD)[r] = make_float2(mr, lr);
      }
      (cuts == 0 ? cut[0] : cut[1]) = p;
      ++cuts;
    });
  int before = 0;
  const bool counts = static_cast<int>(threadIdx.x) < cuts;
  const WarpPart& mine = part_s[threadIdx.x == 0 ? cut[0] : cut[1]];
  if (cuts > 0) __syncthreads();
  if (counts) {
    __threadfence();  // the CTA's part, before the count
    before = atomicAdd(P.counters + mine.c0, 1);
  }
  if (!failed)
    each_task(starts & ~apart, [&](const WarpPart& T, int p, int w1) {
      for (int r = warp * RPW + rl; r < T.rows; r += WARPS * RPW) {
        float mr, lr;
        const float4 acc = add_row(p, w1, r, mr, lr);
        store_out(T.at, T.kvh, r, acc, 1.f / lr);
      }
    });
  if (counts) {
    last_s[threadIdx.x] = before == mine.c1 - mine.c0;
    __threadfence();  // the count, before the other parts
  }
  if (cuts > 0) __syncthreads();
  for (int k = 0; k < cuts; ++k) {
    if (!last_s[k]) continue;
    const WarpPart T = part_s[k == 0 ? cut[0] : cut[1]];
    const int c0 = T.c0, c1 = T.c1;
    // O = sum_c 2^(m_c - m*) O_c / sum_c 2^(m_c - m*) l_c: warp w adds parts c0 + w, c0 + w + 4, .., as many of them in
    // flight as registers hold, and the warps' sums meet as before
    constexpr int RB = 4, PB = 5;  // rows below one another, parts
    const int place0 = line.place(c0, T.first);
    for (int r0 = rl; r0 < T.rows; r0 += RB * RPW) {
      float4 acc[RB];
      float mr[RB], lr[RB];
#pragma unroll
      for (int y = 0; y < RB; ++y) {
        acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        mr[y] = -INFINITY;
        lr[y] = 0.f;
      }
      for (int c = c0 + warp; c <= c1; c += WARPS * PB) {
        float4 v[PB][RB];
        float2 ml[PB][RB];
#pragma unroll
        for (int p = 0; p < PB; ++p) {
          const int from = c + WARPS * p;
          const float* src = P.part + static_cast<size_t>(from == c0 ? place0 : 2 * from) * PLACE;
#pragma unroll
          for (int y = 0; y < RB; ++y) {
            const int r = r0 + RPW * y;
            v[p][y] = make_float4(0.f, 0.f, 0.f, 0.f);
            ml[p][y] = make_float2(-INFINITY, 0.f);
            if (from <= c1 && r < T.rows) {
              v[p][y] = __ldcg(reinterpret_cast<const float4*>(src + r * HD + col));
              ml[p][y] = __ldcg(reinterpret_cast<const float2*>(src + ROWS * HD) + r);
            }
          }
        }
#pragma unroll
        for (int y = 0; y < RB; ++y) {
          float mn = mr[y];
#pragma unroll
          for (int p = 0; p < PB; ++p) mn = fmaxf(mn, ml[p][y].x);
          const float a = mr[y] == -INFINITY ? 0.f : ex2(mr[y] - mn);
          mr[y] = mn;
          lr[y] *= a;
          acc[y] = make_float4(acc[y].x * a, acc[y].y * a, acc[y].z * a, acc[y].w * a);
#pragma unroll
          for (int p = 0; p < PB; ++p) {
            const float w = ml[p][y].x == -INFINITY ? 0.f : ex2(ml[p][y].x - mn);
            lr[y] = fmaf(w, ml[p][y].y, lr[y]);
            acc[y] = make_float4(fmaf(w, v[p][y].x, acc[y].x), fmaf(w, v[p][y].y, acc[y].y), fmaf(w, v[p][y].z, acc[y].z),
                                 fmaf(w, v[p][y].w, acc[y].w));
          }
        }
      }
#pragma unroll
      for (int y = 0; y < RB; ++y) {
        const int r = r0 + RPW * y;
        if (r >= T.rows) break;
        *reinterpret_cast<float4*>(os + (2 * warp * ROWS + r) * L::OW + col) = acc[y];
        if (col == 0) mls[2 * warp * ROWS + r] = make_float2(mr[y], lr[y]);
      }
    }
    __syncthreads();
    for (int r = warp * RPW + rl; r < T.rows; r += WARPS * RPW) {
      float mr, lr;
      const float4 acc = add_row(0, WARPS - 1, r, mr, lr);
      store_out(T.at, T.kvh, r, acc, 1.f / lr);
    }
    if (threadIdx.x == 0) P.counters[c0] = 0;  // every part is in: ready for the next call
    __syncthreads();
  }
  if (__syncthreads_or(failed)) {
    // let the copies in flight land before shared memory is released
    if (threadIdx.x < NS && issued_s[threadIdx.x] > 0) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bars + 8 * threadIdx.x, (issued_s[threadIdx.x] - 1) & 1) && global_timer_ns() - t0 < PF_WAIT_LIMIT_NS) {}
    }
    if (threadIdx.x == 0) batch_record(P.status, PF_ERR_DEVICE_TIMEOUT);
  }
}


template <int HD, int BF16>
cudaError_t launch_few(const TreeAttnArgs& a, cudaStream_t stream) {
  using L = FSmem<HD>;
  const pf_config& c = *a.c;
  const int slots = cache_slots(c);
  const uint64_t dims[2] = {HD, static_cast<uint64_t>(c.n_layers) * c.n_kv_heads * slots}, strides[1] = {HD * 2};
  const uint32_t box[2] = {64, UK};
  CUtensorMap tk, tv;
  if (!encode_tmap_16(&tk, BF16, 2, a.k_cache, dims, strides, box) || !encode_tmap_16(&tv, BF16, 2, a.v_cache, dims, strides, box))
    return cudaErrorInvalidValue;
  FewParams p{};
  p.B = batch_dev(c, *a.b);
  p.q = static_cast<const uint16_t*>(a.q);
  p.nq = c.n_q_heads;
  p.nkv = c.n_kv_heads;
  p.layer = a.layer;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HD));
  p.out = static_cast<__half*>(a.out);
  p.counters = static_cast<int*>(a.scratch);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.scratch) + TREE_COUNTER_BYTES);
  p.status = a.status;
  const int ctas = std::min(device_sm_count(), GEMM_MAX_CTAS);
  return launch_pdl(attn_tree_few_kernel<HD, BF16>, dim3(ctas), dim3(THREADS), L::BYTES, stream, tk, tv, p);
}

template <int HD, int BF16>
cudaError_t launch_rows(const TreeAttnArgs& a, cudaStream_t stream) {
  const int R = std::min(a.b->max_rows, a.b->n_rows) * (a.c->n_q_heads / a.c->n_kv_heads);
  return R <= FEW_ROWS ? launch_few<HD, BF16>(a, stream) : launch_attention_tree_tc(a, stream);
}

template <int HD, int BF16>
cudaError_t set_attr_few() {
  return cudaFuncSetAttribute(attn_tree_few_kernel<HD, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, FSmem<HD>::BYTES);
}

}  // namespace

size_t attention_tree_scratch_bytes(const pf_config& c, int n_seq, int max_rows) {
  // either form: a call with fewer rows than max_rows may take the other
  const size_t few = TREE_COUNTER_BYTES + static_cast<size_t>(GEMM_MAX_CTAS) * 2 * FEW_ROWS * (c.head_dim + 2) * sizeof(float);
  return std::max(few, attention_tree_tc_scratch_bytes(c, n_seq, max_rows));
}

cudaError_t prepare_attention_tree_kernels() {
  cudaError_t e = cudaSuccess, r;
  if ((r = set_attr_few<128, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr_few<128, 0>()) != cudaSuccess) e = r;
  if ((r = set_attr_few<64, 1>()) != cudaSuccess) e = r;
  if ((r = set_attr_few<64, 0>()) != cudaSuccess) e = r;
  return e;
}

cudaError_t launch_attention_tree(const TreeAttnArgs& a, cudaStream_t stream) {
  const bool bf = a.c->kv_dtype == PF_KV_BF16;
  if (a.c->head_dim == 128) return bf ? launch_rows<128, 1>(a, stream) : launch_rows<128, 0>(a, stream);
  return bf ? launch_rows<64, 1>(a, stream) : launch_rows<64, 0>(a, stream);
}

}  // namespace pf

PF_TIMELINE_SETTER(attention_tree)
