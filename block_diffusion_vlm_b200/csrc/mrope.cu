// Rotary positions with several axes (time, height, width of image and video
// rows), alone and fused with the write of new keys and values into a paged
// cache.
//
// Mathematics: frequency j of rot/2 turns the pair (x_j, x_{j + rot/2}) by
// theta = pos[axis(j)][row] * base^(-2j/rot); elements from rot on pass
// unchanged.  The angle is formed in turns, t = pos * (base^(-2j/rot) / 2 pi),
// and reduced to t - rint(t) in fp64: positions of 10^5 keep an absolute error
// near 1e-11 turns, where fp32 would lose the angle altogether.  The cosine
// and sine of the reduced angle, the products and the sum are fp32; one
// rounding at the store.
//
// Bound: HBM (each element read once, written once).  A row's (cos, sin)
// table is shared by all its heads, so a block takes a tile of rows, builds
// their table once in shared memory and streams the heads past it in 16-byte
// pieces.  V is stored feature-major in its page: the block turns a 32-row
// tile through shared memory, so that one warp writes 32 consecutive slots of
// a feature.
#include "kernels.h"
#include "ptx.cuh"

namespace dvlm {

namespace {
constexpr int kMrThreads = 256;
constexpr int kMrRows = 32;                 // rows per block
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

// (cos, sin) of rows row0 .. row0 + n - 1 into cs[row][half]; freq[half] (in
// turns per position) is scratch.
__device__ __forceinline__ void mrope_table(const MropeAxes& ax, int row0, int n, int n_rows, double* freq,
                                            uint8_t* axis, float2* cs) {
  const int half = ax.rot / 2;
  for (int j = threadIdx.x; j < half; j += kMrThreads) {
    freq[j] = exp2(-2.0 * j / ax.rot * ax.log2_base) * kInv2Pi;
    axis[j] = static_cast<uint8_t>(mrope_axis(ax, j));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * half; i += kMrThreads) {
    const int r = i / half, j = i - r * half;
    const double t = ax.pos[static_cast<size_t>(axis[j]) * n_rows + row0 + r] * freq[j];
    float s, c;
    sincospif(2.0f * static_cast<float>(t - rint(t)), &s, &c);
    cs[i] = make_float2(c, s);
  }
}

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, bf16& y) { y = __float2bfloat16_rn(x); }

// (explicit multiply-adds: every piece width rounds alike)
template <typename T, int N>
__device__ __forceinline__ void turn(const Vec<T, N>& a, const Vec<T, N>& b, const float2* cs, Vec<T, N>& ya,
                                     Vec<T, N>& yb) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float x = to_f(a.v[e]), y = to_f(b.v[e]);
    from_f(__fmaf_rn(x, cs[e].x, -__fmul_rn(y, cs[e].y)), ya.v[e]);
    from_f(__fmaf_rn(y, cs[e].x, __fmul_rn(x, cs[e].y)), yb.v[e]);
  }
}
}  // namespace

// out[r, h, :] = x[r, h, :] turned (N elements of a half per piece).  grid:
// (row tiles, head groups).
template <typename T, int N>
__global__ void __launch_bounds__(kMrThreads) mrope_rows_kernel(const T* x, T* out, long long x_ld, long long out_ld,
                                                                int n_rows, int n_heads, int D, const MropeAxes ax) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int half = ax.rot / 2, row0 = blockIdx.x * kMrRows, n = min(kMrRows, n_rows - row0);
  double* freq = reinterpret_cast<double*>(smem);
  float2* cs = reinterpret_cast<float2*>(freq + half);
  uint8_t* axis = reinterpret_cast<uint8_t*>(cs + kMrRows * half);
  const int hpg = (n_heads + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * hpg, hn = min(hpg, n_heads - h0);
  mrope_table(ax, row0, n, n_rows, freq, axis, cs);
  __syncthreads();
  if (hn <= 0) return;
  const int np = half / N, tail = x == out ? 0 : (D - ax.rot) / N;  // pieces: turned pairs, then copies
  const int per_head = np + tail, per_row = hn * per_head;
#pragma unroll 2
  for (int i = threadIdx.x; i < n * per_row; i += kMrThreads) {
    const int r = i / per_row, k = i - r * per_row, h = k / per_head, p = k - h * per_head;
    const T* src = x + (row0 + r) * x_ld + static_cast<long long>(h0 + h) * D;
    T* dst = out + (row0 + r) * out_ld + static_cast<long long>(h0 + h) * D;
    using V = Vec<T, N>;
    if (p < np) {
      const V a = *reinterpret_cast<const V*>(src + p * N), b = *reinterpret_cast<const V*>(src + half + p * N);
      V ya, yb;
      turn(a, b, cs + r * half + p * N, ya, yb);
      *reinterpret_cast<V*>(dst + p * N) = ya;
      *reinterpret_cast<V*>(dst + half + p * N) = yb;
    } else {
      const int at = ax.rot + (p - np) * N;
      *reinterpret_cast<V*>(dst + at) = *reinterpret_cast<const V*>(src + at);
    }
  }
}

// One row of qkv = [Hq query heads | Hkv key heads | Hkv value heads]: queries
// turned into q_out, keys turned into their page slot, values into their
// feature-major page.  A row with slot -1 is padding: nothing is written.
// grid: (row tiles, groups of the Hq + 2 Hkv heads).
template <int D, int N>
__global__ void __launch_bounds__(kMrThreads) mrope_append_kernel(const MropeAppendArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int half = a.ax.rot / 2, row0 = blockIdx.x * kMrRows, n = min(kMrRows, a.n_rows - row0);
  bf16* vt = reinterpret_cast<bf16*>(smem);                       // [kMrRows][D + 2] one value head
  constexpr int kVtLd = D + 2;
  double* freq = reinterpret_cast<double*>(smem + kMrRows * kVtLd * 2);
  float2* cs = reinterpret_cast<float2*>(freq + half);
  int* slot = reinterpret_cast<int*>(cs + kMrRows * half);
  uint8_t* axis = reinterpret_cast<uint8_t*>(slot + kMrRows);
  const int heads = a.Hq + 2 * a.Hkv;
  const int hpg = (heads + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * hpg, h1 = min(heads, h0 + hpg);
  const int n_slots = a.n_pages * 64;
  if (threadIdx.x < kMrRows) {
    int sl = threadIdx.x < n ? a.slot_map[row0 + threadIdx.x] : -1;
    if (sl < -1 || sl >= n_slots) {
      record_error(a.status, DVLM_ERR_BOUNDS);
      sl = -1;
    }
    slot[threadIdx.x] = sl;
  }
  const int hr = min(h1, a.Hq + a.Hkv);  // heads h0 .. hr - 1 are turned, hr .. h1 - 1 are values
  if (h0 < hr) mrope_table(a.ax, row0, n, a.n_rows, freq, axis, cs);
  __syncthreads();

  using V = Vec<bf16, N>;
  const int np = half / N, per_head = np + (D - a.ax.rot) / N, per_row = max(hr - h0, 0) * per_head;
#pragma unroll 2
  for (int i = threadIdx.x; i < n * per_row; i += kMrThreads) {
    const int r = i / per_row, k = i - r * per_row, hh = k / per_head, p = k - hh * per_head, h = h0 + hh;
    const int sl = slot[r];
    if (sl < 0) continue;
    const bf16* src = a.qkv + (row0 + r) * a.qkv_ld + h * D;
    bf16* dst = h < a.Hq ? a.q_out + (static_cast<size_t>(row0 + r) * a.Hq + h) * D
                         : a.k_pages + ((static_cast<size_t>(sl >> 6) * a.Hkv + (h - a.Hq)) * 64 + (sl & 63)) * D;
    if (p < np) {
      const V x = *reinterpret_cast<const V*>(src + p * N), y = *reinterpret_cast<const V*>(src + half + p * N);
      V ya, yb;
      turn(x, y, cs + r * half + p * N, ya, yb);
      *reinterpret_cast<V*>(dst + p * N) = ya;
      *reinterpret_cast<V*>(dst + half + p * N) = yb;
    } else {
      const int at = a.ax.rot + (p - np) * N;
      *reinterpret_cast<V*>(dst + at) = *reinterpret_cast<const V*>(src + at);
    }
  }
  for (int h = max(h0, a.Hq + a.Hkv); h < h1; ++h) {
    const int g = h - a.Hq - a.Hkv;
    __syncthreads();
    for (int i = threadIdx.x; i < n * (D / 2); i += kMrThreads) {
      const int r = i / (D / 2), c = i - r * (D / 2);
      *reinterpret_cast<uint32_t*>(vt + r * kVtLd + 2 * c) =
          *reinterpret_cast<const uint32_t*>(a.qkv + (row0 + r) * a.qkv_ld + h * D + 2 * c);
    }
    __syncthreads();
    const int r = threadIdx.x & 31, sl = slot[r];
    if (sl >= 0) {
      bf16* page = a.v_pages + (static_cast<size_t>(sl >> 6) * a.Hkv + g) * D * 64 + (sl & 63);
      for (int d = threadIdx.x >> 5; d < D; d += kMrThreads / 32) page[d * 64] = vt[r * kVtLd + d];
    }
  }
}

namespace {
// Head groups (grid y): one group where the row tiles alone fill the GPU
// (the angle table is then built once a row), else as many as give every SM a
// few blocks, down to one head a block.
int head_groups(int row_tiles, int heads) {
  const int want = 4 * 148 / row_tiles;
  return want < 1 ? 1 : (want > heads ? heads : want);
}
template <typename T, int N>
cudaError_t run_rows(const T* x, T* out, long long x_ld, long long out_ld, int n_rows, int n_heads, int D,
                     const MropeAxes& ax, cudaStream_t s) {
  const int half = ax.rot / 2, tiles = (n_rows + kMrRows - 1) / kMrRows;
  const size_t sm = static_cast<size_t>(half) * (8 + 1) + static_cast<size_t>(kMrRows) * half * 8;
  mrope_rows_kernel<T, N><<<dim3(tiles, head_groups(tiles, n_heads)), kMrThreads, sm, s>>>(x, out, x_ld, out_ld, n_rows,
                                                                                        n_heads, D, ax);
  return cudaGetLastError();
}
template <typename T>
cudaError_t rows_by_width(const T* x, T* out, long long x_ld, long long out_ld, int n_rows, int n_heads, int D,
                          const MropeAxes& ax, cudaStream_t s) {
  // widest piece that divides both halves, the head and the strides and keeps every access aligned
  auto fits = [&](int n) {
    const long long b = n * static_cast<long long>(sizeof(T));
    return (ax.rot / 2) % n == 0 && D % n == 0 && ax.rot % n == 0 && x_ld % n == 0 && out_ld % n == 0 &&
           reinterpret_cast<uintptr_t>(x) % b == 0 && reinterpret_cast<uintptr_t>(out) % b == 0;
  };
  constexpr int kMax = 16 / sizeof(T);
  if (fits(kMax)) return run_rows<T, kMax>(x, out, x_ld, out_ld, n_rows, n_heads, D, ax, s);
  if (fits(kMax / 2)) return run_rows<T, kMax / 2>(x, out, x_ld, out_ld, n_rows, n_heads, D, ax, s);
  return run_rows<T, 1>(x, out, x_ld, out_ld, n_rows, n_heads, D, ax, s);
}
template <int D>
cudaError_t run_append(const MropeAppendArgs& a, cudaStream_t s) {
  const int half = a.ax.rot / 2, tiles = (a.n_rows + kMrRows - 1) / kMrRows;
  const size_t sm = kMrRows * (D + 2) * 2 + static_cast<size_t>(half) * (8 + 1) +
                    static_cast<size_t>(kMrRows) * half * 8 + kMrRows * 4;
  const dim3 grid(tiles, head_groups(tiles, a.Hq + 2 * a.Hkv));
  // 16-byte pieces wherever the halves allow them
  if (half % 8 == 0) mrope_append_kernel<D, 8><<<grid, kMrThreads, sm, s>>>(a);
  else mrope_append_kernel<D, 1><<<grid, kMrThreads, sm, s>>>(a);
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
