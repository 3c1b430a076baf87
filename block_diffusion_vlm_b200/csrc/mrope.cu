// Rotary positions with several axes (time, height, width of image and video
// rows), alone and fused with the write of new keys and values into a paged
// cache.
//
// Mathematics: frequency j of rot/2 turns the pair (x_j, x_{j + rot/2}) by
// theta = pos[axis(j)][row] * base^(-2j/rot); elements from rot on pass
// unchanged.  The angle is formed in turns, t = pos * (base^(-2j/rot) / 2 pi),
// and reduced to t - rint(t) in fp64: positions of 10^5 keep an absolute error
// near 1e-11 turns, where fp32 would lose the angle altogether.  The reduced
// angle is rounded to fp32 (half a step is at most 2^-26 turns, which moves its
// cosine and sine by less than 1e-7, as much as the products' own roundings),
// and the sine, the cosine, the products and the sum are fp32; one rounding at
// the store.
//
// Bound: HBM (each element read once, written once).  A warp owns a row: it
// sends out the loads of its first kMrBatch pieces per lane (16 bytes of each
// half), forms the row's (cos, sin) while they are on their way, and then
// turns and stores.  No block-wide step after the first, so that the warps of
// an SM are in different phases and the loads never pause (a block building a
// table for 32 rows first reached half the bandwidth).  V is stored
// feature-major in its page: separate blocks turn 64-row tiles of a value
// head through shared memory, all of a thread's loads out at once; eight rows
// on eight aligned slots of a page leave as 16-byte pieces.
//
// Measured: 16384 rows of 16/2 heads of 128, 35.9 us (168 MB: 4.7 TB/s; a plain
// copy of 80 MB to another 80 MB takes 27 us); 1357 rows of 14/2 heads of 64,
// 5.4 us; one block of 16 rows, 3.1 us; 4999 rows of 16 heads of 80 in fp32,
// 11.8 us, in bf16 8.0 us; 1357 rows of 16/2 heads of 128, 7.9 us, in a buffer
// of 16384 rows with the rest padding 12.6 us.  Blocks of 256 threads: 38.0, 4.7, 3.5 and 12.0 us.  Value
// tiles of 32 rows: 39.8 and 4.8 us for the first two.  Values turned by the
// block that turns their rows, instead of by blocks of their own: 50 us.  Rows
// brought in by bulk copies, a ring of rows per warp: 37 us.
#include "ptx.cuh"
#include "step.h"

namespace dvlm {

namespace {
constexpr int kMrThreads = 128;
constexpr int kMrWarps = kMrThreads / 32;
constexpr int kMrBlocks = 8;                // resident blocks per SM (64 registers a thread)
constexpr int kMrBatch = 3;                 // pieces in flight per lane
constexpr int kMrVRows = 64;                // rows of a value tile
constexpr double kInv2Pi = 0.15915494309189533577;

// Axis of frequency j: sections in order (axis 0's frequencies first), or
// interleaved (j mod n_axes, for j below n_axes * that axis's section; axis 0
// takes the rest).
__device__ __forceinline__ int mrope_axis(const MropeAxes& ax, int j) {
  if (ax.interleaved) {
    const int a = j % ax.n;
    return j < ax.n * ax.section[a] ? a : 0;
  }
  int a = 0;
  while (a + 1 < ax.n && j >= ax.section[a]) j -= ax.section[a++];
  return a;
}

// Shared memory of a block: freq [half] (turns per position, fp64), the axis
// of each frequency, then a table of cosines and sines per warp, laid out for
// pieces of N elements: element e of piece p at pair slot (e / 2) * np + p as
// (cos, cos', sin, sin') of elements e and e + 1, so that the lanes of a head
// read consecutive 16 bytes (N = 1: (cos, sin) of element p).
struct MrSmem {
  double* freq;
  float* cs;  // this warp's
  int* axis;
};
__device__ __forceinline__ MrSmem mr_carve(uint8_t* smem, int half, int warp) {
  MrSmem s;
  s.cs = reinterpret_cast<float*>(smem) + warp * ((2 * half + 3) & ~3);
  s.freq = reinterpret_cast<double*>(reinterpret_cast<float*>(smem) + kMrWarps * ((2 * half + 3) & ~3));
  s.axis = reinterpret_cast<int*>(s.freq + half);
  return s;
}
inline size_t mr_smem(int half) { return static_cast<size_t>(kMrWarps) * ((2 * half + 3) & ~3) * 4 + half * 12; }

__device__ __forceinline__ void mr_freqs(const MropeAxes& ax, const MrSmem& s) {
  for (int j = threadIdx.x; j < ax.rot / 2; j += kMrThreads) {
    s.freq[j] = exp2(-2.0 * j / ax.rot * ax.log2_base) * kInv2Pi;
    s.axis[j] = mrope_axis(ax, j);
  }
  __syncthreads();
}
// The table of a row.
template <int N>
__device__ __forceinline__ void mr_angles(const MropeAxes& ax, const MrSmem& s, int row, int n_rows, int np, int lane) {
  for (int j = lane; j < ax.rot / 2; j += 32) {
    const double t = ax.pos[static_cast<size_t>(s.axis[j]) * n_rows + row] * s.freq[j];
    float sn, c;
    sincospif(2.0f * static_cast<float>(t - rint(t)), &sn, &c);
    if constexpr (N == 1) {
      s.cs[2 * j] = c;
      s.cs[2 * j + 1] = sn;
    } else {
      float* d = s.cs + ((j % N) / 2 * np + j / N) * 4 + (j & 1);
      d[0] = c;
      d[2] = sn;
    }
  }
  __syncwarp();
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};
// Two neighbouring elements as packed fp32, and back.
__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t widen2(const float* v) { return pack_f2(v[0], v[1]); }
__device__ __forceinline__ uint64_t widen2(const bf16* v) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(v);
  return pack_f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void narrow2(uint64_t x, float* v) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(x));
}
__device__ __forceinline__ void narrow2(uint64_t x, bf16* v) {
  float a, b;
  uint32_t w;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  *reinterpret_cast<uint32_t*>(v) = w;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, bf16& y) { y = __float2bfloat16_rn(x); }

// (explicit multiply-adds: every piece width rounds alike)
template <typename T, int N>
__device__ __forceinline__ void turn(Vec<T, N>& a, Vec<T, N>& b, const float* cs, int p, int np) {
  if constexpr (N == 1) {
    const float c = cs[2 * p], s = cs[2 * p + 1], x = to_f(a.v[0]), y = to_f(b.v[0]);
    from_f(__fmaf_rn(x, c, -__fmul_rn(y, s)), a.v[0]);
    from_f(__fmaf_rn(y, c, __fmul_rn(x, s)), b.v[0]);
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float4 w = *reinterpret_cast<const float4*>(cs + ((e / 2) * np + p) * 4);
      const uint64_t c = pack_f2(w.x, w.y), s = pack_f2(w.z, w.w), ns = pack_f2(-w.z, -w.w);
      const uint64_t x = widen2(a.v + e), y = widen2(b.v + e);
      uint64_t u, v;
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(u) : "l"(y), "l"(ns));
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(s));
      asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(u) : "l"(x), "l"(c), "l"(u));
      asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(y), "l"(c), "l"(v));
      narrow2(u, a.v + e);
      narrow2(v, b.v + e);
    }
  }
}

// Pieces of a row of `heads` heads of D: piece i is (head i / np, pair piece
// i % np), np = half / N; walked by a lane in steps of 32 without dividing.
struct Walk {
  int h, p, np, dh, dp;
  __device__ __forceinline__ Walk(int lane, int np_) : np(np_) {
    h = lane / np;
    p = lane - h * np;
    dh = 32 / np;
    dp = 32 - dh * np;
  }
  __device__ __forceinline__ void next() {
    h += dh;
    p += dp;
    if (p >= np) {
      p -= np;
      ++h;
    }
  }
};

// Row of unit i (more than one group of heads only where rows are few).
__device__ __forceinline__ int unit_row(long long i, int groups) {
  return groups == 1 ? static_cast<int>(i) : static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(groups));
}

// One row: heads h of src at h * D turned into dst(h).
template <typename T, int N, typename Dst>
__device__ __forceinline__ void turn_row(const T* src, const Dst& dst, int heads, int D, const MropeAxes& ax,
                                         const MrSmem& s, int row, int n_rows, int lane, const Walk& first) {
  using V = Vec<T, N>;
  const int half = ax.rot / 2;
  Walk rd = first, wr = first;
  bool have_angles = false;
  while (__any_sync(0xffffffffu, rd.h < heads)) {
    V a[kMrBatch], b[kMrBatch];
#pragma unroll
    for (int u = 0; u < kMrBatch; ++u) {
      if (rd.h < heads) {
        const T* x = src + rd.h * D + rd.p * N;
        a[u] = *reinterpret_cast<const V*>(x);
        b[u] = *reinterpret_cast<const V*>(x + half);
      }
      rd.next();
    }
    if (!have_angles) mr_angles<N>(ax, s, row, n_rows, first.np, lane);
    have_angles = true;
#pragma unroll
    for (int u = 0; u < kMrBatch; ++u) {
      if (wr.h < heads) {
        turn(a[u], b[u], s.cs, wr.p, first.np);
        T* y = dst(wr.h) + wr.p * N;
        *reinterpret_cast<V*>(y) = a[u];
        *reinterpret_cast<V*>(y + half) = b[u];
      }
      wr.next();
    }
  }
  __syncwarp();  // the table is read before the next row's
}
// The elements from rot on of a row's heads, copied.
template <typename T, int N, typename Dst>
__device__ __forceinline__ void copy_tails(const T* src, const Dst& dst, int heads, int D, int rot, int lane) {
  using V = Vec<T, N>;
  const int nt = (D - rot) / N;
  for (int i = lane; i < heads * nt; i += 32) {
    const int h = i / nt, at = rot + (i - h * nt) * N;
    *reinterpret_cast<V*>(dst(h) + at) = *reinterpret_cast<const V*>(src + h * D + at);
  }
}
}  // namespace

// out[r, h, :] = x[r, h, :] turned.  Units: (row, group of heads).
template <typename T, int N>
__global__ void __launch_bounds__(kMrThreads, kMrBlocks) mrope_rows_kernel(const T* x, T* out, long long x_ld, long long out_ld,
                                                                int n_rows, int n_heads, int D, int groups,
                                                                const MropeAxes ax) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MrSmem s = mr_carve(smem, ax.rot / 2, warp);
  mr_freqs(ax, s);
  const Walk first(lane, ax.rot / 2 / N);
  const int hpg = (n_heads + groups - 1) / groups;
  for (long long i = static_cast<long long>(blockIdx.x) * kMrWarps + warp; i < static_cast<long long>(n_rows) * groups;
       i += static_cast<long long>(gridDim.x) * kMrWarps) {
    const int row = unit_row(i, groups), h0 = static_cast<int>(i - static_cast<long long>(row) * groups) * hpg;
    const int heads = min(hpg, n_heads - h0);
    if (heads <= 0) continue;
    const T* src = x + row * x_ld + static_cast<long long>(h0) * D;
    T* dst = out + row * out_ld + static_cast<long long>(h0) * D;
    auto at = [&](int h) { return dst + static_cast<long long>(h) * D; };
    turn_row<T, N>(src, at, heads, D, ax, s, row, n_rows, lane, first);
    if (ax.rot < D && x != out) copy_tails<T, N>(src, at, heads, D, ax.rot, lane);
  }
}

// One row of qkv = [Hq query heads | Hkv key heads | Hkv value heads]: queries
// turned into q_out, keys turned into their page slot, values into their
// feature-major page.  A row with slot -1 is padding: nothing is written.
// Blocks 0 .. v_blocks - 1 take the value tiles (64 rows of one head), the
// others (row, head group) units of the queries and keys.
template <int D, int N>
__global__ void __launch_bounds__(kMrThreads, kMrBlocks) mrope_append_kernel(const MropeAppendArgs a, int v_blocks, int groups) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_slots = a.n_pages * 64;
  auto slot_of = [&](int row) {
    const int sl = a.slot_map[row];
    if (sl >= -1 && sl < n_slots) return sl;
    record_error(a.status, DVLM_ERR_BOUNDS);
    return -1;
  };
  const bool units = static_cast<int>(blockIdx.x) >= v_blocks;
  const int idx = static_cast<int>(blockIdx.x) - (units ? v_blocks : 0);
  if (units) {
    const MrSmem s = mr_carve(smem, a.ax.rot / 2, warp);
    mr_freqs(a.ax, s);
    const Walk first(lane, a.ax.rot / 2 / N);
    const int heads = a.Hq + a.Hkv, hpg = (heads + groups - 1) / groups;
    const long long n_units = static_cast<long long>(a.n_rows) * groups;
    const long long n_warps = static_cast<long long>(gridDim.x - v_blocks) * kMrWarps;
    for (long long i = static_cast<long long>(idx) * kMrWarps + warp; i < n_units; i += n_warps) {
      const int row = unit_row(i, groups);
      const int h0 = static_cast<int>(i - static_cast<long long>(row) * groups) * hpg, hn = min(hpg, heads - h0);
      const int sl = slot_of(row);
      if (sl < 0 || hn <= 0) continue;
      const bf16* src = a.qkv + row * a.qkv_ld + h0 * D;
      bf16* q = a.q_out + (static_cast<size_t>(row) * a.Hq + h0) * D;
      bf16* k = a.k_pages + ((static_cast<size_t>(sl >> 6) * a.Hkv + h0) * 64 + (sl & 63)) * D -
                static_cast<size_t>(a.Hq) * 64 * D;
      auto at = [&](int h) { return h0 + h < a.Hq ? q + h * D : k + static_cast<size_t>(h) * 64 * D; };
      turn_row<bf16, N>(src, at, hn, D, a.ax, s, row, a.n_rows, lane, first);
      if (a.ax.rot < D) copy_tails<bf16, N>(src, at, hn, D, a.ax.rot, lane);
    }
    return;
  }
  // value tile: rows row0 .. of head g, [row][D + 2] in shared memory
  constexpr int kLd = D + 2;
  bf16* vt = reinterpret_cast<bf16*>(smem);
  int* slot = reinterpret_cast<int*>(vt + kMrVRows * kLd);
  const int row0 = idx / a.Hkv * kMrVRows, g = idx % a.Hkv;
  const int n = min(kMrVRows, a.n_rows - row0);
  const bf16* src = a.qkv + row0 * a.qkv_ld + (a.Hq + a.Hkv + g) * D;
  constexpr int kLoads = kMrVRows * (D / 8) / kMrThreads;  // 16-byte loads per thread, all on their way at once
  uint4 v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = i * kMrThreads + threadIdx.x, r = at / (D / 8);
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < n) v[i] = *reinterpret_cast<const uint4*>(src + r * a.qkv_ld + at % (D / 8) * 8);
  }
  if (threadIdx.x < kMrVRows) slot[threadIdx.x] = static_cast<int>(threadIdx.x) < n ? slot_of(row0 + threadIdx.x) : -1;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = i * kMrThreads + threadIdx.x, r = at / (D / 8);
    uint32_t* d = reinterpret_cast<uint32_t*>(vt + r * kLd + at % (D / 8) * 8);
    d[0] = v[i].x;
    d[1] = v[i].y;
    d[2] = v[i].z;
    d[3] = v[i].w;
  }
  __syncthreads();
  auto put = [&](int r, int d) {
    const int sl = slot[r];
    if (sl >= 0) a.v_pages[((static_cast<size_t>(sl >> 6) * a.Hkv + g) * D + d) * 64 + (sl & 63)] = vt[r * kLd + d];
  };
  // rows r0, r0 + 8, ... lead pieces of eight, r0 where the first row's slots
  // come to a multiple of eight; pieces whose slots do not follow one another,
  // and the rows before r0, go one by one
  const int r0 = slot[0] >= 0 ? min(n, (8 - (slot[0] & 7)) & 7) : 0;
  for (int i = threadIdx.x; i < r0 * D; i += kMrThreads) put(i / D, i % D);
  // lanes: eight pieces next to one another (a 128-byte line of a page's
  // feature row) of four feature pairs; a thread keeps its piece
  constexpr int kPieces = kMrVRows / 8;
  const int lo = r0 + static_cast<int>(threadIdx.x) % kPieces * 8, hi = min(n, lo + 8);
  if (lo >= hi) return;
  const int s0 = slot[lo];
  bool run = hi - lo == 8 && s0 >= 0 && (s0 & 7) == 0;
  if (run) {
#pragma unroll
    for (int e = 1; e < 8; ++e) run &= slot[lo + e] == s0 + e;
  }
  if (run) {
    bf16* page = a.v_pages + (static_cast<size_t>(s0 >> 6) * a.Hkv + g) * D * 64 + (s0 & 63);
#pragma unroll 4
    for (int d2 = threadIdx.x / kPieces; d2 < D / 2; d2 += kMrThreads / kPieces) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const uint32_t*>(vt + (lo + e) * kLd + 2 * d2);
      uint4 even, odd;
      even.x = __byte_perm(w[0], w[1], 0x5410);
      even.y = __byte_perm(w[2], w[3], 0x5410);
      even.z = __byte_perm(w[4], w[5], 0x5410);
      even.w = __byte_perm(w[6], w[7], 0x5410);
      odd.x = __byte_perm(w[0], w[1], 0x7632);
      odd.y = __byte_perm(w[2], w[3], 0x7632);
      odd.z = __byte_perm(w[4], w[5], 0x7632);
      odd.w = __byte_perm(w[6], w[7], 0x7632);
      *reinterpret_cast<uint4*>(page + 2 * d2 * 64) = even;
      *reinterpret_cast<uint4*>(page + (2 * d2 + 1) * 64) = odd;
    }
  } else {
    for (int d = threadIdx.x / kPieces; d < D; d += kMrThreads / kPieces)
      for (int r = lo; r < hi; ++r) put(r, d);
  }
}

namespace {
// Head groups per row: one where the rows alone fill the GPU's warps, else as
// many as give each SM a few warps of work, down to one head.
int head_groups(int n_rows, int heads) {
  const int want = device_sm_count() * 16 / n_rows;
  return want < 1 ? 1 : (want > heads ? heads : want);
}
// Blocks for n_units warps of work, at most twice what the SMs hold at once
// (a warp then takes two or three rows on one table of frequencies; once the
// residents: 37.7 us, twice: 35.9 us for 16384 rows of 16/2 heads of 128).
int unit_blocks(long long n_units) {
  const long long b = (n_units + kMrWarps - 1) / kMrWarps, most = static_cast<long long>(device_sm_count()) * 2 * kMrBlocks;
  return static_cast<int>(b < most ? b : most);
}
template <typename T, int N>
cudaError_t run_rows(const T* x, T* out, long long x_ld, long long out_ld, int n_rows, int n_heads, int D,
                     const MropeAxes& ax, cudaStream_t s) {
  const int groups = head_groups(n_rows, n_heads);
  mrope_rows_kernel<T, N><<<unit_blocks(static_cast<long long>(n_rows) * groups), kMrThreads, mr_smem(ax.rot / 2), s>>>(
      x, out, x_ld, out_ld, n_rows, n_heads, D, groups, ax);
  return cudaGetLastError();
}
template <typename T>
cudaError_t rows_by_width(const T* x, T* out, long long x_ld, long long out_ld, int n_rows, int n_heads, int D,
                          const MropeAxes& ax, cudaStream_t s) {
  // widest piece that divides both halves, the head and the strides and keeps every access aligned
  auto fits = [&](int n) {
    const long long b = n * static_cast<long long>(sizeof(T));
    return (ax.rot / 2) % n == 0 && D % n == 0 && x_ld % n == 0 && out_ld % n == 0 &&
           reinterpret_cast<uintptr_t>(x) % b == 0 && reinterpret_cast<uintptr_t>(out) % b == 0;
  };
  constexpr int kMax = 16 / sizeof(T);
  if (fits(kMax)) return run_rows<T, kMax>(x, out, x_ld, out_ld, n_rows, n_heads, D, ax, s);
  if (fits(kMax / 2)) return run_rows<T, kMax / 2>(x, out, x_ld, out_ld, n_rows, n_heads, D, ax, s);
  return run_rows<T, 1>(x, out, x_ld, out_ld, n_rows, n_heads, D, ax, s);
}
template <int D>
cudaError_t run_append(const MropeAppendArgs& a, cudaStream_t s) {
  const int groups = head_groups(a.n_rows, a.Hq + a.Hkv);
  const int v_blocks = (a.n_rows + kMrVRows - 1) / kMrVRows * a.Hkv;
  const size_t sv = kMrVRows * (D + 2) * 2 + kMrVRows * 4, sr = mr_smem(a.ax.rot / 2);
  const int blocks = v_blocks + unit_blocks(static_cast<long long>(a.n_rows) * groups);
  const size_t sm = sv > sr ? sv : sr;
  // 16-byte pieces wherever the halves allow them
  if (a.ax.rot % 16 == 0) mrope_append_kernel<D, 8><<<blocks, kMrThreads, sm, s>>>(a, v_blocks, groups);
  else mrope_append_kernel<D, 1><<<blocks, kMrThreads, sm, s>>>(a, v_blocks, groups);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_mrope_rows(const void* x, void* out, long long x_ld, long long out_ld, int n_rows, int n_heads,
                              int D, bool is_bf16, const MropeAxes& ax, cudaStream_t s) {
  if (is_bf16)
    return rows_by_width(static_cast<const bf16*>(x), static_cast<bf16*>(out), x_ld, out_ld, n_rows, n_heads, D, ax, s);
  return rows_by_width(static_cast<const float*>(x), static_cast<float*>(out), x_ld, out_ld, n_rows, n_heads, D, ax, s);
}

cudaError_t launch_mrope_append(const MropeAppendArgs& a, int D, cudaStream_t s) {
  return D == 128 ? run_append<128>(a, s) : run_append<64>(a, s);
}

}  // namespace dvlm
