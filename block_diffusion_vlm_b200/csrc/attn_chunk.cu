// Attention of ragged chunks of new rows over paged K/V caches, bf16, tcgen05.
//
// Mathematics: row t of request b (n new rows behind kv - n cached slots) sees
// slots hidden .. kv - n + t, or hidden .. kv - 1 for the request's last
// `noisy` rows; o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m) over the
// visible slots j, s = scale q.k, with the running maximum and sum of an
// online softmax; a row that sees nothing gives 0.  Partial results over
// disjoint slots combine by their (m, l): o = sum_i e^(m_i - m) o_i / sum_i
// e^(m_i - m) l_i.
//
// Tile: the G = Hq / Hkv query heads of a KV head times 128 / G rows fill the
// 128 lanes of an MMA, so a single-token row of 8 heads costs the cache read
// once, not 8 times.  A CTA works on two tiles at a time, each with its own
// softmax warpgroup (a thread owns a row):
//   pair: two neighbouring row tiles of one request and KV head over the same
//         pages (each K and V page is loaded once for 256 rows);
//   solo: one row tile; the two warpgroups take alternate pages and combine
//         their (m, l, O) through TMEM at the end, so that few rows keep both
//         halves of the SM busy.
// A step is one 64-slot page.  TMEM holds two score buffers of 64 columns per
// tile (P in bf16 takes the place of its scores) and O of both tiles (2 x 2 x
// 64 + 2 x D columns): Q K^T of the page after next is issued right behind
// P V of this one, so that scores wait for the softmax warps and not the other
// way round.  One thread issues all products, alternating between the tiles.
//
// Bound and measure: a page of a pair item takes about 2100 cycles, of which
// the exponentials of its 256 x 64 scores hold their unit for 1024 and the
// products the tensor pipe for 1050 (both 50% by the profiler's counters; 2 x
// 256 x 64 x 128 multiply-adds at the pipe's 4096 a cycle are 1024); chunks of
// rows run into the 1000 W power cap (1.74 of 1.965 GHz).  4096 rows over 12288
// slots, 16/2 heads of 128: 332 us (1.04 PFLOP/s) in short runs, 347 us back to
// back and 355 us after a second of nothing else (0.97 PFLOP/s).  Steps of two pages with one score buffer: 340 to 366 us
// (the scores' latency stands between two steps); four warpgroups with the
// keys of a page halved between two: 352 us, and with a second issuing thread
// 350 us at lower clocks; a quarter or half of the exponentials as a
// polynomial on the multiply-add pipe: 343 and 355 us.  64 single tokens over
// 900 to 16000 slots read 5.9 TB/s (86 us; 91 us after a second of nothing
// else, at the power cap and 1.65 GHz).
//
// Work split: all (request, KV head, pair or solo item) are laid end to end by
// their cost in slots, and the line is cut into equal parts, one per CTA (one
// CTA per SM).  A cut inside an item leaves partial (O, m, l) in the workspace
// (at most two per CTA) for the merge kernel; every other row is written
// directly.  The cost of a request's items is a closed form (page ends grow
// linearly), so each CTA finds its part from the lengths on the device alone:
// no host knowledge of them, no plan kernel.
#include "ptx.cuh"
#include "step.h"

namespace dvlm {

namespace {
constexpr int kAcThreads = 320;  // warp 0 loads and schedules, 1 issues MMAs, 2..5 and 6..9 softmax
constexpr int kAcKeys = 64;      // slots per step: one page
constexpr int kAcRing = 4;       // work descriptors in flight
// Fixed cost of an item, in slots of a tile (prologue and epilogue take 4300
// cycles, a slot 14.5; 256 to 512 measure alike).
constexpr int kAcItemCost = 320;
// Least cost worth a CTA of its own.  16 rows over 1360 slots 12.9 us, one
// token over 500 slots 11.7, over 4000 14.1; with 128: 12.3, 10.5 and 15.1;
// with 512: 15.8, 13.7 and 15.3; with 1024: 20.6, 19.4 and 19.4.
constexpr int kAcMinPart = 256;
constexpr float kAcLazy = 8.0f;  // log2 headroom before the running maximum moves

template <int D>
struct AcCfg {
  static constexpr int kStage = kAcKeys * D * 2;  // one K or V^T page
  static constexpr int kStages = D == 128 ? 8 : 12;
  static constexpr int kQ = 128 * D * 2;          // one Q tile
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * kQ;
  static constexpr int oBar = oKV + kStages * kStage;
  static constexpr int kBars = 2 * kAcRing + 2 + 2 * kStages + 4 + 4 + 2 + 2 + 1 + 1;
  static constexpr int oDesc = oBar + 512;
  static constexpr int oML = oDesc + kAcRing * 64;
  static constexpr int kSmem = oML + 2 * 128 * 8 + 1024;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kAcKeys);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(128, D);
  static constexpr uint32_t kIdescS64 = idesc_bf16_f32(64, kAcKeys);  // products of thin items
  static constexpr uint32_t kIdescO64 = idesc_bf16_f32(64, D);
};
constexpr uint32_t kAcColO = 256;

// One request's lengths and the closed form of its items' costs.
struct Req {
  int row0, n, kv, nclean, hid, base;
  int pairs, solo, pc;  // pair items, solo items (0 or 1), leading pairs that are whole and causal
};

__device__ __forceinline__ Req load_req(const ChunkAttnArgs& a, int b, int tpt, int* err) {
  Req r;
  int lo = a.cu_rows[b], hi = a.cu_rows[b + 1], kv = a.kv_len[b];
  const int noisy = a.n_noisy ? a.n_noisy[b] : 0, hid = a.n_hidden ? a.n_hidden[b] : 0;
  if (lo < 0 || hi < lo || hi > a.n_rows || kv < 0 || kv > a.max_pages * 64LL || hi - lo > kv) {
    *err = 1;  // takes no part
    lo = hi = kv = 0;
  }
  r.row0 = lo;
  r.n = hi - lo;
  r.kv = kv;
  r.base = kv - r.n;
  r.nclean = r.n - max(0, min(noisy, r.n));
  r.hid = max(0, min(hid, kv));
  const int tiles = (r.n + tpt - 1) / tpt;
  r.pairs = tiles >> 1;
  r.solo = tiles & 1;
  r.pc = min(r.pairs, r.nclean / (2 * tpt));
  return r;
}
// Cost of the first i pair items of a request: sum of 2 * (visible slots) +
// kAcItemCost, the slots counted from the hidden prefix's page on.
__device__ __forceinline__ long long pair_prefix(const Req& r, int tpt, int i) {
  const int p2 = 2 * tpt, off = r.base - (r.hid & ~(kAcKeys - 1));
  const long long k = min(i, r.pc);
  const long long k0 = off < 0 ? min(min(i, r.pc), -off / p2) : 0;  // leading items that end at or before the first visible page
  long long c = (k - k0) * off + p2 * ((k * (k + 1) - k0 * (k0 + 1)) / 2);
  c += (i - k) * max(0LL, static_cast<long long>(r.kv) - (r.hid & ~(kAcKeys - 1)));
  return 2 * c + static_cast<long long>(i) * kAcItemCost;
}
__device__ __forceinline__ long long solo_cost(const Req& r) {
  return max(0, r.kv - (r.hid & ~(kAcKeys - 1))) + kAcItemCost;
}
__device__ __forceinline__ long long req_cost(const Req& r, int tpt) {
  return pair_prefix(r, tpt, r.pairs) + (r.solo ? solo_cost(r) : 0);
}

// Work descriptor (16 ints in shared memory).
struct Work {
  int kind;             // 0 end, 1 pair, 2 solo
  int c0, nc;           // first page, pages
  int row0, ntok;       // first row (of all rows) and rows of the item
  int t0;               // the item's first row within the request
  int nclean, base, kv, hid;
  int g;                // KV head
  int slot;             // -1: whole item; 0 / 1: partial, this CTA's slot
  int pad[4];
};
static_assert(sizeof(Work) == 64, "descriptor size");

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Wait for this thread's TMEM loads; the registers pass through so that no
// use of them moves above the wait.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_st32_nowait(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// The rest of a wait that did not end at once, by a whole warp (out of line:
// the loops stay short).
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, int* status, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, abort_flag)) != 0;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 lanes in one 64-bit register (packed multiply-add and add).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// p_j = 2^(sl2 s_j + neg) of a 32-column block of scores, packed to bf16 (P's
// rounding: half a step of 2^-8 relative, of a weight in a sum whose divisor l
// is the fp32 sum of the unrounded weights; the tensor pipe takes P and V in
// one 16-bit type, and V comes out of its page as bf16 -- an fp16 P, as the
// block attention keeps it, wants V converted in shared memory first, a pass
// over every page for each tile pair).  Returns the fp32 sum.  A masked score (-inf) gives 0.
__device__ __forceinline__ float exp_block(const uint32_t (&s)[32], uint64_t sl2, uint64_t neg, uint32_t* pk) {
  uint64_t sum = pack2(0.f, 0.f), sum1 = sum;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint64_t x = fma2(pack2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), sl2, neg);
    float x0, x1;
    unpack2(x, x0, x1);
    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
    if (j & 1) sum1 = add2(sum1, pack2(p0, p1));
    else sum = add2(sum, pack2(p0, p1));
    pk[j] = pack_bf16(p0, p1);
  }
  float u, v;
  unpack2(add2(sum, sum1), u, v);
  return u + v;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Largest of m and 32 values, in two chains.
__device__ __forceinline__ float max32(const uint32_t (&s)[32], float m) {
  float m1 = __uint_as_float(s[0]);
#pragma unroll
  for (int j = 1; j < 29; j += 4) {
    m = max3(m, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
    m1 = max3(m1, __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
  }
  return max3(max3(m, __uint_as_float(s[29]), __uint_as_float(s[30])), m1, __uint_as_float(s[31]));
}

// Scores of a 32-slot block outside slots lo .. hi - 1 to -inf.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int hi, int lo) {
  const uint32_t below = hi >= 32 ? 0xFFFFFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t keep = below & (lo <= 0 ? 0xFFFFFFFFu : lo >= 32 ? 0u : ~((1u << lo) - 1u));
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (!(keep >> j & 1u)) s[j] = 0xFF800000u;
}
// One feature's row of a V^T page (64 slots, 128-byte swizzle): 0 outside
// slots lo .. hi - 1.
__device__ __noinline__ void clear_outside(uint8_t* v, int sw, int hi, int lo) {
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    const int s = q * 8;
    if (s + 8 <= hi && s >= lo) continue;
    uint4* pv = reinterpret_cast<uint4*>(v + ((q ^ sw) << 4));
    uint4 x = make_uint4(0, 0, 0, 0);
    if (s < hi && s + 8 > lo) {
      x = *pv;
      uint32_t* xe = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int sa = s + 2 * e;
        xe[e] &= ((sa < hi && sa >= lo) ? 0x0000FFFFu : 0u) | ((sa + 1 < hi && sa + 1 >= lo) ? 0xFFFF0000u : 0u);
      }
    }
    *pv = x;
  }
}

// floor(a / b) for a >= 0, b > 0 with a quotient below 2^20: a float estimate
// put right (64-bit integer division costs hundreds of cycles on the one warp
// that everything waits for).
__device__ __forceinline__ int div_small(long long a, long long b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  while (q > 0 && q * b > a) --q;
  while ((q + 1) * b <= a) ++q;
  return q;
}
}  // namespace

// Partial results in the workspace: per CTA two slots of two tiles, O [D / 4]
// [128][4] fp32 (a warp stores four features of 32 rows as 512 bytes) and (m, l)
// [128]; then one merge record per CTA.
struct AcPart {
  float* o;       // [P][2][2][D / 4][128][4]
  float2* ml;     // [P][2][2][128]
  int* rec;       // [P][16]
};
static __host__ __device__ AcPart ac_carve(void* ws, int P, int D) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  AcPart a;
  a.o = reinterpret_cast<float*>(p);
  p += static_cast<size_t>(P) * 4 * D * 128 * 4;
  a.ml = reinterpret_cast<float2*>(p);
  p += static_cast<size_t>(P) * 4 * 128 * 8;
  a.rec = reinterpret_cast<int*>(p);
  return a;
}
size_t attn_chunk_scratch_bytes(int P, int D) {
  return static_cast<size_t>(P) * 4 * D * 128 * 4 + static_cast<size_t>(P) * 4 * 128 * 8 + static_cast<size_t>(P) * 64;
}

template <int D>
__global__ void __launch_bounds__(kAcThreads, 1)
    attn_chunk_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapV, const ChunkAttnArgs a) {
  using C = AcCfg<D>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem + C::oQ;
  uint8_t* sKV = smem + C::oKV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::oBar);
  uint64_t* d_full = bars;                 // [kAcRing] descriptor written
  uint64_t* d_empty = d_full + kAcRing;    // [kAcRing] MMA and softmax warps done with it
  uint64_t* q_full = d_empty + kAcRing;
  uint64_t* q_empty = q_full + 1;          // every S of the item done
  uint64_t* kv_full = q_empty + 1;         // [NS]
  uint64_t* kv_empty = kv_full + NS;       // [NS]
  uint64_t* s_full = kv_empty + NS;        // [2 tiles][2 buffers] scores of a page done
  uint64_t* p_full = s_full + 4;           // [2][2] P written, O rescaled
  uint64_t* pv_done = p_full + 4;          // [2] P V of a page done (one phase per page)
  uint64_t* o_done = pv_done + 2;          // [2] last P V of the item done (pv_done may be two phases behind there)
  uint64_t* x_bar = o_done + 2;            // the softmax warps of both tiles meet (a bounded wait, unlike bar.sync)
  uint64_t* mma_idle = x_bar + 1;          // every product of this CTA done
  static_assert(C::kBars * 8 + 16 <= 512, "barrier space");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* sabort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Work* desc = reinterpret_cast<Work*>(smem + C::oDesc);
  float2* sML = reinterpret_cast<float2*>(smem + C::oML);  // [2][128] solo: both warpgroups' (m, l)
  __shared__ long long s_scan[kAcThreads / 32];
  __shared__ long long s_start;  // cost position, number and lengths of the request with this CTA's first unit
  __shared__ int s_b;
  __shared__ Req s_req;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = gridDim.x, cta = blockIdx.x;
  const int G = a.Hq / a.Hkv, tpt = 128 / G;
  const AcPart ws = ac_carve(a.workspace, P, D);

  if (warp == kAcThreads / 32 - 1) {  // (a warp that has no length to wait for in small batches)
    for (int i = lane; i < C::kBars; i += 32) {
      uint64_t* b = &bars[i];
      mbar_init(b, (b >= d_empty && b < q_full) ? 9 : (b >= p_full && b < pv_done) ? 4 : b == x_bar ? 8 : 1);
    }
    fence_mbar_init();
    if (lane == 0) {
      *sabort = 0;
      tma_prefetch_map(&mapQ);
      tma_prefetch_map(&mapK);
      tma_prefetch_map(&mapV);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  // ------------------------------------------------ this CTA's part of the line
  // (a float estimate of the share: every CTA computes the same one, and the
  // shares need only cover the line)
  const int per = (a.n_batch + kAcThreads - 1) / kAcThreads;
  const int b0 = min(a.n_batch, tid * per), b1 = min(a.n_batch, b0 + per);
  int bad = 0;
  long long mine = 0, c0 = 0;
  Req r0{};
  for (int b = b0; b < b1; ++b) {
    const Req r = load_req(a, b, tpt, &bad);
    const long long c = a.Hkv * req_cost(r, tpt);
    if (b == b0) {
      r0 = r;
      c0 = c;
    }
    mine += c;
  }
  if (bad && cta == 0) record_error(a.status, DVLM_ERR_BOUNDS);
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) s_scan[warp] = inc;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kAcThreads / 32; ++w) {
    if (w == warp) before = total;
    total += s_scan[w];
  }
  const int parts = max(1, min(P, static_cast<int>(min(1.0e6f, static_cast<float>(total) * (1.f / kAcMinPart)))));
  const long long share =
      static_cast<long long>(__fdividef(static_cast<float>(total) * 1.00001f, static_cast<float>(parts))) + 1;
  const long long lo = min(total, cta * share), hi = min(total, lo + share);
  long long at = before + inc - mine;
  if (lo < hi && at <= lo && lo < at + mine) {  // one thread's requests hold the first unit
    int b = b0;
    while (lo >= at + c0) {
      at += c0;
      r0 = load_req(a, ++b, tpt, &bad);
      c0 = a.Hkv * req_cost(r0, tpt);
    }
    s_b = b;
    s_start = at;
    s_req = r0;
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;

  // whole warps wait as one: either every lane goes on or none does
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_longer(bar, parity, a.status, sabort);
  };
  // the same where nothing hangs on the outcome and another wait has perhaps given up
  auto warp_wait_only = [&](uint64_t* bar, uint32_t parity) {
    if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) wait_longer(bar, parity, a.status, nullptr);
  };

  if (warp == 0) {
    // ------------------------------------------------ schedule and load
    // few rows read a cache once, pair items many times
    const uint64_t pol_once = l2_policy_evict_first(), pol_kept = l2_policy_evict_last();
    int it = 0;        // descriptors issued
    int pos = 0;       // K/V ring position
    int nq = 0;        // Q loads issued
    bool ok = true;
    int rec_kind = 0;  // this CTA's item that goes on in the next CTAs
    Work rw{};
    int rec_last = 0;
    if (lo < hi) {
      int b = s_b;
      long long start = s_start;  // cost position of the current item
      Req r = s_req;
      const long long per_head = req_cost(r, tpt);
      int g = div_small(lo - start, per_head);
      start += g * per_head;
      // last item whose prefix is at or below lo, 32 candidates at a time
      int i = 0;
      const int n_items = r.pairs + r.solo;
      for (int span = n_items; span > 1;) {
        const int step = (span + 31) >> 5, cand = i + lane * step;
        const bool below = lane * step < span && cand < n_items && start + pair_prefix(r, tpt, cand) <= lo;
        i += (31 - __clz(__ballot_sync(0xffffffffu, below))) * step;
        span = step;
      }
      start += pair_prefix(r, tpt, i);
      long long x = lo;
      while (x < hi && ok) {
        const bool solo = i == r.pairs;
        const long long w = solo ? solo_cost(r) : pair_prefix(r, tpt, i + 1) - pair_prefix(r, tpt, i);
        const long long xa = x - start, xb = min(w, hi - start);
        const uint64_t pol = solo ? pol_once : pol_kept;
        Work k{};
        k.kind = solo ? 2 : 1;
        k.t0 = i * 2 * tpt;
        k.ntok = min(2 * tpt, r.n - k.t0);
        if (solo) k.ntok = r.n - k.t0;
        k.row0 = r.row0 + k.t0;
        k.nclean = r.nclean;
        k.base = r.base;
        k.kv = r.kv;
        k.hid = r.hid;
        k.g = g;
        const int te = k.t0 + k.ntok, end = te > r.nclean ? r.kv : r.base + te;
        const int cb = r.hid / kAcKeys, nch = end > r.hid ? (end + kAcKeys - 1) / kAcKeys - cb : 0;
        // the part's pages (the CTA that ends here and the one that goes on
        // compute the same cut): the item's fixed cost comes first, so that a
        // CTA that begins an item has paid for it, then 128 units a page, or
        // pair of pages of a solo item (the fixed cost spread over the pages
        // left CTAs with many short items a fifth behind the others: 24 mixed
        // requests 31 us, against 29; 2 blocks of 16 rows 15.4, against 13.3)
        auto pages_before = [&](long long y) -> int {
          if (y >= w) return nch;
          const int u = static_cast<int>(max(0LL, y - kAcItemCost + kAcKeys) >> 7);
          return min(nch, solo ? 2 * u : u);
        };
        const int ca = pages_before(xa), ce = pages_before(xb);
        // an item belongs to the CTAs that hold pages of it (without any: to the one that holds its first unit)
        const bool begins = ca == 0, ends = ce == nch;
        const bool take = nch == 0 ? xa == 0 : !(begins && ce == 0) && ca < nch;
        k.c0 = cb + ca;
        k.nc = ce - ca;
        k.slot = begins && ends ? -1 : begins ? 1 : 0;
        if (take && k.slot == 1) {  // the item goes on: the CTA that holds its last pages
          rec_kind = k.kind;
          rw = k;
          rec_last = div_small(start + w - 1, share);
          while (pages_before(rec_last * share - start) >= nch) --rec_last;
        }
        // hand the descriptor over
        if (take) {
          const int slot = it % kAcRing;
          if (it >= kAcRing) ok = warp_wait(&d_empty[slot], ((it / kAcRing) - 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            desc[slot] = k;
            mbar_arrive(&d_full[slot]);
          }
          ++it;
        }
        if (take && k.nc > 0) {
          // Q: rows [row0, +tpt) (and the next tpt for a pair) of the KV head's query heads
          if (nq > 0) ok = warp_wait(q_empty, (nq - 1) & 1);
          if (!ok) break;
          const int n_q = k.kind == 1 ? 2 : 1;
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full, n_q * tpt * G * D * 2);
            for (int w2 = 0; w2 < n_q; ++w2)
              for (int d = 0; d < D / 64; ++d)
                tma_load_3d(sQ + w2 * C::kQ + d * 16384, &mapQ, q_full, d * 64, g * G, k.row0 + w2 * tpt, pol);
          }
          ++nq;
          // K and V in the order the products take them: K of the first pages
          // (two of each tile's buffers), then V(c), K(c + lag)
          const int lag = k.kind == 1 ? 2 : 4;
          const int n_held = (r.kv + 63) >> 6;
          // page numbers: a window of 64 table entries, two per lane, that
          // moves up by 32 (V lags K by less than that)
          const int32_t* table = a.block_table + static_cast<size_t>(b) * a.max_pages;
          int win = k.c0 & ~31;
          auto entry_at = [&](int p) { return p < n_held ? table[p] : -1; };
          int w0 = entry_at(win + lane), w1 = entry_at(win + 32 + lane);
          auto page_of = [&](int p) -> int {
            if (p >= win + 64) {
              win += 32;
              w0 = w1;
              w1 = entry_at(win + 32 + lane);
            }
            const int page = __shfl_sync(0xffffffffu, p < win + 32 ? w0 : w1, p & 31);
            if (page >= 0 && page < a.n_pages) return page;
            record_error(a.status, DVLM_ERR_BOUNDS);  // (only a page that some row sees)
            return 0;
          };
          auto load = [&](int c, bool is_v) {
            const int st = pos % NS;
            if (pos >= NS) ok = warp_wait(&kv_empty[st], ((pos / NS) - 1) & 1);
            if (!ok) return;
            const int entry = page_of(k.c0 + c) * a.Hkv + g;
            if (lane == 0) {
              mbar_arrive_expect_tx(&kv_full[st], C::kStage);
              uint8_t* dst = sKV + st * C::kStage;
              if (is_v) {
                tma_load_2d(dst, &mapV, &kv_full[st], 0, entry * D, pol);
              } else {
                for (int d = 0; d < D / 64; ++d)
                  tma_load_2d(dst + d * 8192, &mapK, &kv_full[st], d * 64, entry * 64, pol);
              }
            }
            ++pos;
          };
          for (int c = 0; c < min(lag, k.nc) && ok; ++c) load(c, false);
          for (int c = 0; c < k.nc && ok; ++c) {
            load(c, true);
            if (ok && c + lag < k.nc) load(c + lag, false);
          }
        }
        // next item
        x = start + xb;
        if (x < hi) {
          start += w;
          if (++i >= r.pairs + r.solo) {
            i = 0;
            if (++g >= a.Hkv) {
              g = 0;
              r.n = 0;
              while (r.n == 0 && ++b < a.n_batch) r = load_req(a, b, tpt, &bad);
              if (r.n == 0) break;  // (the line ends with the last request: only lengths changed under way come here)
            }
          }
        }
      }
    }
    if (ok) {
      const int slot = it % kAcRing;
      if (it >= kAcRing) ok = warp_wait(&d_empty[slot], ((it / kAcRing) - 1) & 1);
      if (ok && lane == 0) {
        desc[slot].kind = 0;
        mbar_arrive(&d_full[slot]);
      }
    }
    // no copy is on its way into this CTA's memory when it ends, after a wait that gave up either
    for (int p = max(0, pos - NS); p < pos; ++p) warp_wait_only(&kv_full[p % NS], (p / NS) & 1);
    if (nq > 0) warp_wait_only(q_full, (nq - 1) & 1);
    // merge record: the item this CTA began and did not finish
    if (lane == 0) {
      int* rec = ws.rec + cta * 16;
      rec[0] = rec_kind;
      rec[1] = rec_last;
      rec[2] = rw.row0;
      rec[3] = rw.ntok;
      rec[4] = rw.g;
    }
  } else if (warp == 1) {
    // ------------------------------------------------ products
    // (elect.sync rather than lane == 0: the compiler then keeps descriptors
    // in uniform registers and issues a product in half the instructions)
    if (elect_one()) {
      int pos = 0, nq = 0;
      int ni[2] = {0, 0}, np[2] = {0, 0};  // per tile: scores issued, P pages consumed (buffer = parity)
      bool ok = true;
      const uint64_t qd0 = sdesc_kmajor_sw128(smem_u32(sQ)), kd0 = sdesc_kmajor_sw128(smem_u32(sKV));
      auto kv_wait = [&](int ps) { return mbar_wait(&kv_full[ps % NS], (ps / NS) & 1, a.status, sabort); };
      for (int it = 0; ok; ++it) {
        const int slot = it % kAcRing;
        if (!mbar_wait(&d_full[slot], (it / kAcRing) & 1, a.status, sabort)) break;
        const int kind = desc[slot].kind, nc = desc[slot].nc;
        if (kind == 0) break;
        if (nc == 0) {
          mbar_arrive(&d_empty[slot]);
          continue;
        }
        // Up to 16 lanes of rows (single tokens): products of 64 rows instead of
        // 128, whose first 16 lie in the same lanes.  The same time at full
        // clocks, but half the tensor pipe's work at the power cap: 64 tokens
        // over 900 to 16000 slots again and again, 99 us against 91
        const bool solo = kind == 2, thin = solo && desc[slot].ntok * G <= 16;
        const uint32_t id_s = thin ? C::kIdescS64 : C::kIdescS, id_o = thin ? C::kIdescO64 : C::kIdescO;
        ok = mbar_wait(q_full, nq & 1, a.status, sabort);
        if (!ok) break;
        ++nq;
        auto issue_s = [&](int w, int st) {
          tc_fence_after();
          const int buf = ni[w]++ & 1;
          const uint64_t qd = qd0 + ((solo ? 0 : w * C::kQ) >> 4), kd = kd0 + ((st * C::kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_ss(tmem + w * 128 + buf * 64, qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                         kd + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), id_s, kk > 0 ? 1u : 0u);
          umma_commit(&s_full[w * 2 + buf]);
        };
        auto issue_pv = [&](int w, int st, bool first, bool last) -> bool {
          const int buf = np[w] & 1;
          if (!mbar_wait(&p_full[w * 2 + buf], (np[w] >> 1) & 1, a.status, sabort)) return false;
          ++np[w];
          tc_fence_after();
          const uint64_t vd = kd0 + ((st * C::kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16_ts(tmem + kAcColO + w * D, tmem + w * 128 + buf * 64 + kk * 8, vd + ((kk * 32) >> 4), id_o,
                        (!first || kk > 0) ? 1u : 0u);
          umma_commit(&pv_done[w]);
          if (last) umma_commit(&o_done[w]);
          return true;
        };
        const int lag = solo ? 4 : 2;
        for (int c = 0; c < min(lag, nc) && ok; ++c) {
          ok = kv_wait(pos);
          if (!ok) break;
          if (solo) {
            issue_s(c & 1, pos % NS);
          } else {
            issue_s(0, pos % NS);
            issue_s(1, pos % NS);
          }
          umma_commit(&kv_empty[pos % NS]);
          ++pos;
        }
        // Q is free behind the last scores: the next item's loads while this one's last pages run
        if (ok && nc <= lag) umma_commit(q_empty);
        for (int c = 0; c < nc && ok; ++c) {
          const int vs = pos % NS, ks = (pos + 1) % NS;
          const bool more = c + lag < nc;
          ok = kv_wait(pos) && (!more || kv_wait(pos + 1));
          if (!ok) break;
          if (solo) {
            ok = issue_pv(c & 1, vs, c < 2, c + 2 >= nc);
            if (!ok) break;
            umma_commit(&kv_empty[vs]);
            if (more) issue_s(c & 1, ks);
          } else {
            ok = issue_pv(0, vs, c == 0, c + 1 == nc);
            if (!ok) break;
            if (more) issue_s(0, ks);
            ok = issue_pv(1, vs, c == 0, c + 1 == nc);
            if (!ok) break;
            umma_commit(&kv_empty[vs]);
            if (more) issue_s(1, ks);
          }
          if (more) umma_commit(&kv_empty[ks]);
          if (c + lag + 1 == nc) umma_commit(q_empty);
          pos += more ? 2 : 1;
        }
        if (ok) mbar_arrive(&d_empty[slot]);
      }
      // nor a product under way when its TMEM is given back
      umma_commit(mma_idle);
      mbar_wait(mma_idle, 0, a.status, nullptr);
    }
  } else {
    // ------------------------------------------------ softmax and output
    const int w = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t tS = tl + w * 128, tO = tl + kAcColO + w * D;
    const int rt = row / G, rh = row - rt * G;  // row within the tile, head within the group
    const float sl2 = a.scale_log2, lazy = kAcLazy / sl2;
    int ns = 0, pos = 0;  // pages of this tile, K/V ring position
    int no = 0;           // items with pages for this tile
    int nx = 0;           // meetings of the two warpgroups
    bool ok = true;
    auto meet = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x_bar);
      const bool met = warp_wait(x_bar, nx++ & 1);
      tc_fence_after();
      return met;
    };
    // 16 features of this thread's row: to the output, or to this CTA's partial slot
    auto store_cols = [&](const Work& k, int tok, bool valid, int tile, int col, const float (&x)[16]) {
      if (!valid) return;
      if (k.slot < 0) {
        uint4* dst = reinterpret_cast<uint4*>(a.out + (static_cast<size_t>(k.row0 + tok) * a.Hq + k.g * G + rh) * D + col);
        dst[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        dst[1] = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]),
                            pack_bf16(x[14], x[15]));
      } else {
        float* dst = ws.o + ((static_cast<size_t>(cta * 2 + k.slot) * 2 + tile) * D + col) * 128 + row * 4;
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(dst + j * 128) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      }
    };
    if (tid == 64) griddep_launch_dependents();
    for (int it = 0; ok; ++it) {
      const int dslot = it % kAcRing;
      if (!warp_wait(&d_full[dslot], (it / kAcRing) & 1)) break;
      const Work k = desc[dslot];
      if (k.kind == 0) break;
      const bool solo = k.kind == 2;
      const int tok = (solo ? 0 : w * tpt) + rt;  // within the item
      const bool valid = rt < tpt && tok < k.ntok;
      const bool live = __any_sync(0xffffffffu, valid);
      const int t = k.t0 + tok;
      // visible slots hid .. lim - 1 (rows past the item: never written, left unmasked)
      const int lim = !valid ? 0x7fffffff : t >= k.nclean ? k.kv : k.base + t + 1;
      const int lo_slot = valid ? k.hid : 0;
      const int step = solo ? 2 : 1, first = solo ? w : 0;
      const int lag = solo ? 4 : 2;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int c = first; c < k.nc; c += step) {
        const int key0 = (k.c0 + c) * kAcKeys, buf = ns & 1;
        if (!warp_wait(&s_full[w * 2 + buf], (ns >> 1) & 1)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        const uint32_t tP = tS + buf * 64;
        uint32_t s0[32], s1[32];
        tmem_ld32_nowait(tP, s0);
        tmem_ld32_nowait(tP + 32, s1);
        // V of slots outside hidden .. kv - 1 may hold anything (stale pages):
        // 0 there, for 0 * NaN is not 0.  A pair's page is cleared by the first
        // tile's warps alone: both tiles' P V are issued, by one thread, behind
        // the first tile's P, so none reads the page while it is written.
        if ((solo || w == 0) && (key0 + kAcKeys > k.kv || key0 < k.hid)) {
          const int vp = pos + min(lag, k.nc) + c + min(c, max(0, k.nc - lag));
          if (!warp_wait(&kv_full[vp % NS], (vp / NS) & 1)) {
            ok = false;
            break;
          }
          if (row < D) clear_outside(sKV + (vp % NS) * C::kStage + row * 128, row & 7, k.kv - key0, k.hid - key0);
          fence_proxy_async_smem();
        }
        tmem_wait_ld32(s0);
        tmem_wait_ld32(s1);
        if (live) {
          if (__any_sync(0xffffffffu, key0 + kAcKeys > lim || key0 < lo_slot)) {
            mask32(s0, lim - key0, lo_slot - key0);
            mask32(s1, lim - key0 - 32, lo_slot - key0 - 32);
          }
          const float mx = max32(s1, max32(s0, -INFINITY));
          // the reference maximum moves only past the headroom (or from -inf):
          // P then stays below 2^8, and O is seldom rescaled
          const bool move = mx > m + lazy || (m == -INFINITY && mx > -INFINITY);
          if (__any_sync(0xffffffffu, move)) {
            const float f = move ? ex2_approx((m - mx) * sl2) : 1.f;
            if (move) m = mx;
            l *= f;
            if (c >= step) {  // once every product of the earlier pages is in O
              if (!warp_wait(&pv_done[w], (ns - 2) & 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < D; cc += 16) {
                float o[16];
                tmem_ld16(tO + cc, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_st16_nowait(tO + cc, o);
              }
            }
          }
          const float neg = m == -INFINITY ? 0.f : -m * sl2;
          const uint64_t neg2 = pack2(neg, neg), sl22 = pack2(sl2, sl2);
          uint32_t pk[32];
          const float sum = exp_block(s0, sl22, neg2, pk);
          l += sum + exp_block(s1, sl22, neg2, pk + 16);
          tmem_st32_nowait(tP, pk);
          tmem_wait_st();
        }  // else no row of this warp is one of the item's: its P and O are never used
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w * 2 + buf]);
      }
      pos += 2 * k.nc;
      if (!ok) break;
      if (k.nc > first && !warp_wait(&o_done[w], no++ & 1)) break;
      tc_fence_after();
      if (solo) {
        // both warpgroups hold the same rows over alternate pages: each
        // finishes half of the features from both accumulators
        sML[w * 128 + row] = make_float2(m, l);
        if (!meet()) break;
        const float2 o2 = sML[(w ^ 1) * 128 + row];
        const float mm = fmaxf(m, o2.x);
        const float a_own = m == -INFINITY ? 0.f : ex2_approx((m - mm) * sl2);
        const float a_oth = o2.x == -INFINITY ? 0.f : ex2_approx((o2.x - mm) * sl2);
        const float a0 = w == 0 ? a_own : a_oth, a1 = w == 0 ? a_oth : a_own;
        const float lt = l * a_own + o2.y * a_oth;
        const bool h0 = k.nc > 0, h1 = k.nc > 1;
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        const float nan = lt == lt ? 0.f : lt;  // scores that are no numbers, which the maxima pass over
        const float f0 = k.slot < 0 ? a0 * inv : a0, f1 = k.slot < 0 ? a1 * inv : a1;
        constexpr int HD = D / 2;
#pragma unroll 1
        for (int cc = 0; live && cc < HD; cc += 16) {
          const int col = w * HD + cc;
          float x[16], y[16];
          tmem_ld16(tl + kAcColO + col, x);
          tmem_ld16(tl + kAcColO + D + col, y);
#pragma unroll
          for (int j = 0; j < 16; ++j)  // an accumulator that no page reached holds anything
            x[j] = (h0 && a0 > 0.f ? x[j] * f0 : nan) + (h1 && a1 > 0.f ? y[j] * f1 : nan);
          store_cols(k, tok, valid, 0, col, x);
        }
        if (w == 0 && valid) {
          if (k.slot >= 0) ws.ml[(cta * 2 + k.slot) * 256 + row] = make_float2(mm, lt);
          else if (a.lse)
            a.lse[static_cast<size_t>(k.row0 + tok) * a.Hq + k.g * G + rh] =
                lt == 0.f ? -INFINITY : (mm * sl2 + log2f(lt)) * 0.69314718055994531f;
        }
        if (!meet()) break;  // both accumulators and sML read
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // (NaN stays NaN)
        const float f = k.slot < 0 ? inv : 1.f;
#pragma unroll 1
        for (int cc = 0; live && cc < D; cc += 64) {
          uint32_t u[2][32];
          tmem_ld32_nowait(tO + cc, u[0]);
          tmem_ld32_nowait(tO + cc + 32, u[1]);
          tmem_wait_ld32(u[0]);
          tmem_wait_ld32(u[1]);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = k.nc > 0 && l != 0.f ? __uint_as_float(u[h >> 1][(h & 1) * 16 + j]) * f : 0.f;
            store_cols(k, tok, valid, w, cc + h * 16, x);
          }
        }
        if (valid) {
          if (k.slot >= 0) ws.ml[(cta * 2 + k.slot) * 256 + w * 128 + row] = make_float2(m, l);
          else if (a.lse)
            a.lse[static_cast<size_t>(k.row0 + tok) * a.Hq + k.g * G + rh] =
                l == 0.f ? -INFINITY : (m * sl2 + log2f(l)) * 0.69314718055994531f;
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[dslot]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Rows of items that were cut: CTA p's record names the item that it began and
// others finished; its partials are combined in CTA order.  Every block lists
// the records for itself, and the warps of the grid share the items' tasks (32
// rows, a lane a row, by D / 8 features; kAmBatch partials' loads together
// with their (m, l)), so that one cut item already spreads over the GPU: 16
// rows over 1360 slots, two items of seven parts, spent 6 us in two blocks and
// spend 3 us so.
constexpr int kAmThreads = 512;
constexpr int kAmBatch = 4;
constexpr int kAmParts = 8;
template <int D>
__global__ void __launch_bounds__(kAmThreads, 1) attn_chunk_merge_kernel(const ChunkAttnArgs a, int P) {
  __shared__ int4 s_item[kAmThreads];  // first CTA, last CTA, first row, rows
  __shared__ int2 s_kind[kAmThreads];  // kind, KV head
  __shared__ int s_base[kAmThreads / 32];
  const int G = a.Hq / a.Hkv, tpt = 128 / G;
  const AcPart ws = ac_carve(a.workspace, P, D);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  int4 r4 = make_int4(0, 0, 0, 0);  // kind, last CTA, first row, rows
  int g0 = 0;
  if (tid < P) {
    r4 = *reinterpret_cast<const int4*>(ws.rec + tid * 16);
    g0 = ws.rec[tid * 16 + 4];
  }
  const unsigned cut = __ballot_sync(0xffffffffu, r4.x != 0);
  if (lane == 0) s_base[warp] = __popc(cut);
  __syncthreads();
  int at = __popc(cut & ((1u << lane) - 1u)), n_items = 0;
#pragma unroll
  for (int w = 0; w < kAmThreads / 32; ++w) {
    if (w < warp) at += s_base[w];
    n_items += s_base[w];
  }
  if (r4.x != 0) {
    s_item[at] = make_int4(tid, r4.y, r4.z, r4.w);
    s_kind[at] = make_int2(r4.x, g0);
  }
  __syncthreads();
  constexpr int F = D / kAmParts;
  constexpr int kTasks = 2 * 4 * kAmParts;  // tiles, row quarters, feature parts
  const int n_warps = gridDim.x * (kAmThreads / 32);
  // (a warp's tasks lie grid-wide apart: the first blocks do not take them all)
  for (int id = warp * gridDim.x + blockIdx.x; id < n_items * kTasks; id += n_warps) {
    const int item = id / kTasks, sub = id % kTasks, tile = sub / (4 * kAmParts), part = sub / 4 % kAmParts;
    const int row = (sub & 3) * 32 + lane;
    const int4 it = s_item[item];
    const int kind = s_kind[item].x, g = s_kind[item].y, p0 = it.x, last = it.y, row0 = it.z, ntok = it.w;
    const int rt = row / G, rh = row - rt * G, tok = tile * tpt + rt;
    if ((kind == 2 && tile > 0) || rt >= tpt || tok >= ntok) continue;
    float acc[F];
#pragma unroll
    for (int j = 0; j < F; ++j) acc[j] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int p = p0; p <= last; p += kAmBatch) {
      float2 ml[kAmBatch];
      float o[kAmBatch][F];
#pragma unroll
      for (int i = 0; i < kAmBatch; ++i) {
        const int slot = ((p + i) * 2 + (p + i == p0 ? 1 : 0)) * 2 + tile;
        ml[i] = p + i <= last ? ws.ml[slot * 128 + row] : make_float2(-INFINITY, 0.f);
        const float* src = ws.o + (static_cast<size_t>(slot) * D + part * F) * 128 + row * 4;
#pragma unroll
        for (int j = 0; j < F; j += 4) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p + i <= last) v = *reinterpret_cast<const float4*>(src + j * 128);
          o[i][j] = v.x;
          o[i][j + 1] = v.y;
          o[i][j + 2] = v.z;
          o[i][j + 3] = v.w;
        }
      }
      float mn = m;
#pragma unroll
      for (int i = 0; i < kAmBatch; ++i) mn = fmaxf(mn, ml[i].x);
      const float keep = m == -INFINITY ? 0.f : ex2_approx((m - mn) * a.scale_log2);
      l *= keep;
#pragma unroll
      for (int j = 0; j < F; ++j) acc[j] *= keep;
#pragma unroll
      for (int i = 0; i < kAmBatch; ++i) {
        // (a part that saw nothing of the row holds zeros)
        const float e = ml[i].x == -INFINITY ? 0.f : ex2_approx((ml[i].x - mn) * a.scale_log2);
        l += e * ml[i].y;
#pragma unroll
        for (int j = 0; j < F; ++j) acc[j] += e * o[i][j];
      }
      m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t o_at = static_cast<size_t>(row0 + tok) * a.Hq + g * G + rh;
    uint32_t pk[F / 2];
#pragma unroll
    for (int j = 0; j < F / 2; ++j) pk[j] = pack_bf16(acc[2 * j] * inv, acc[2 * j + 1] * inv);
    uint2* dst = reinterpret_cast<uint2*>(a.out + o_at * D + part * F);
#pragma unroll
    for (int q = 0; q < F / 4; ++q) dst[q] = make_uint2(pk[2 * q], pk[2 * q + 1]);
    if (a.lse && part == 0) a.lse[o_at] = l == 0.f ? -INFINITY : (m * a.scale_log2 + log2f(l)) * 0.69314718055994531f;
  }
}

namespace {
template <int D>
cudaError_t run_chunk(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const ChunkAttnArgs& a, int P,
                      cudaStream_t s) {
  if (P > kAmThreads) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attn_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       AcCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  attn_chunk_kernel<D><<<P, kAcThreads, AcCfg<D>::kSmem, s>>>(q, k, v, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(P);
  cfg.blockDim = dim3(kAmThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_chunk_merge_kernel<D>, a, P);
}
}  // namespace

cudaError_t launch_attn_chunk(const CUtensorMap& mapQ, const CUtensorMap& mapK, const CUtensorMap& mapV,
                              const ChunkAttnArgs& a, int D, int P, cudaStream_t s) {
  return D == 128 ? run_chunk<128>(mapQ, mapK, mapV, a, P, s) : run_chunk<64>(mapQ, mapK, mapV, a, P, s);
}

}  // namespace dvlm
