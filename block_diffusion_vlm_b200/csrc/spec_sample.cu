// Verification of drafted tokens by rejection sampling, from given uniform
// random numbers.
//
// Mathematics: draft x_j is accepted while u_j q_j(x_j) < p_j(x_j) (u in
// [0, 1)); at the first rejection k the next token is drawn from the residual
// r = max(p_k - q_k, 0), after K acceptances from r = p_K.  The draw inverts
// the cumulative sum: the lowest v with C(v) > u C(V - 1).  Accepted and drawn
// tokens together are distributed as the target's own samples.  The products
// u q are exact in fp64 (24 x 24 bits), and so is the decision; C is summed
// in fp64, so that it is the same token whatever the order of the sum unless
// u C lies within about 1e-13 of a step.
//
// Bound: HBM in batches (one target row, and the draft's row where it has
// probabilities, per sequence: the K + 1 rows are never read whole), latency
// alone.  One cluster per sequence: each of its warps owns a contiguous
// stretch of the vocabulary and sums it, the CTA totals meet in distributed
// shared memory, and the CTA whose stretch holds the step divides that
// stretch among its warps and walks what is left out of L2.  No scratch, no
// atomics: sums in a fixed order.  The sum takes a widening, a maximum with 0,
// a conversion and an addition per probability (comparing and selecting each
// one first took four times the instructions); rows that turn out to hold
// infinities are summed again with care.
#include "ptx.cuh"
#include "step.h"

namespace dvlm {

namespace {
constexpr int kSvThreads = 512;
constexpr int kSvWarps = kSvThreads / 32;
constexpr int kSvMaxCta = 8;
constexpr int kSvBatch = 4;  // pieces of a row in flight per lane

__device__ __forceinline__ void st_dsmem_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void widen(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
};
template <>
struct Piece<bf16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void widen(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
__device__ __forceinline__ float as_f(float x) { return x; }
__device__ __forceinline__ float as_f(bf16 x) { return __bfloat162float(x); }

// max(p - q, 0); a NaN or infinite probability counts as nothing.  One fp32
// difference tells (a bit pattern between 0's and infinity's: positive and
// finite); the value is the fp64 difference.
__device__ __forceinline__ double residual(float p, float q) {
  const uint32_t d = __float_as_uint(p - q);
  return d - 1u < 0x7f7fffffu ? static_cast<double>(p) - static_cast<double>(q) : 0.0;
}

// N consecutive probabilities at v as loaded, 0 from hi on (kVec: hi is a
// whole number of pieces).  No branch: the loads of a batch go out together.
template <typename T, bool kVec>
struct Raw {
  uint4 w;
  __device__ __forceinline__ void load(const T* row, int v, int hi) {
    w = make_uint4(0, 0, 0, 0);
    if (v < hi) w = *reinterpret_cast<const uint4*>(row + v);
  }
  __device__ __forceinline__ void widen(float (&f)[Piece<T>::n]) const { Piece<T>::widen(w, f); }
};
template <typename T>
struct Raw<T, false> {
  float x;
  __device__ __forceinline__ void load(const T* row, int v, int hi) { x = v < hi ? as_f(row[v]) : 0.f; }
  __device__ __forceinline__ void widen(float (&f)[1]) const { f[0] = x; }
};
}  // namespace

// kVec: rows and bases 16-byte aligned, 16-byte pieces; else one element a
// lane (coalesced all the same).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kSvThreads, 2) spec_sample_kernel(const SpecSampleArgs a) {
  constexpr int N = kVec ? Piece<T>::n : 1;
  constexpr int kStep = 32 * N;
  __shared__ double w_tot[kSvWarps];
  __shared__ double w_sub[kSvWarps];
  __shared__ double c_tot[kSvMaxCta];
  __shared__ int s_k;
  const int n_cta = gridDim.x, rank = blockIdx.x, seq = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = a.K, V = a.V;
  const T* tp = static_cast<const T*>(a.target_p) + static_cast<size_t>(seq) * (K + 1) * V;
  const T* dp = a.draft_p ? static_cast<const T*>(a.draft_p) + static_cast<size_t>(seq) * K * V : nullptr;
  const int32_t* ids = a.draft_ids + static_cast<size_t>(seq) * K;
  // A sequence without rows in the step (waiting for pages, idle, finished,
  // refused by the plan) has nothing to verify: its cache holds no drafts to
  // cut off, and its probabilities are those of no row.
  int most = K;
  if (a.cu_rows) {
    const long long rows = static_cast<long long>(a.cu_rows[seq + 1]) - a.cu_rows[seq];
    if (rows <= 0) {
      if (rank == 0) {
        for (int j = threadIdx.x; j <= K; j += kSvThreads) a.out_ids[static_cast<size_t>(seq) * (K + 1) + j] = -1;
        if (threadIdx.x == 0) {
          a.accept_len[seq] = 0;
          if (a.cache_len_out) a.cache_len_out[seq] = a.cache_len[seq];
        }
      }
      return;  // (the whole cluster, before its first barrier)
    }
    most = static_cast<int>(min(rows, static_cast<long long>(K)));
  }
  cluster_arrive();  // every CTA of the cluster runs before any sends into it (the wait sits before the sends)

  int nd = a.n_draft ? a.n_draft[seq] : K;
  if (nd < 0 || nd > most) {
    if (threadIdx.x == 0) record_error(a.status, DVLM_ERR_BOUNDS);
    nd = nd < 0 ? 0 : most;
  }
  // every CTA of the cluster takes the K decisions for itself
  if (warp == 0) {
    int k = nd;
    for (int j0 = 0; j0 < nd; j0 += 32) {
      const int j = j0 + lane;
      bool ok = true, known = true;
      if (j < nd) {
        const int x = ids[j];
        ok = known = x >= 0 && x < V;
        if (ok) {
          const size_t at = static_cast<size_t>(j) * V + x;
          const float p = as_f(tp[at]), q = dp ? as_f(dp[at]) : 1.f;
          const double u = a.u_accept[static_cast<size_t>(seq) * K + j];
          ok = u * q < p && fmaxf(fabsf(p), fabsf(q)) < INFINITY;
        }
      }
      const unsigned rej = __ballot_sync(0xffffffffu, !ok);
      if (rej) {
        k = j0 + __ffs(rej) - 1;
        // (drafts behind the first refused one are not looked at)
        if (j == k && !known && rank == 0) record_error(a.status, DVLM_ERR_BOUNDS);
        break;
      }
    }
    if (lane == 0) s_k = k;
  }
  __syncthreads();
  const int k = s_k;
  const T* p = tp + static_cast<size_t>(k) * V;
  const T* q = (dp && k < nd) ? dp + static_cast<size_t>(k) * V : nullptr;
  int hot = (!dp && k < nd) ? ids[k] : -1;  // a draft without probabilities: q is 1 at its token

  // warp stretches: whole steps, dealt in order over the cluster's warps
  const int n_warp = n_cta * kSvWarps;
  const int steps = (V + kStep - 1) / kStep, per = (steps + n_warp - 1) / n_warp;
  const long long lo_l = static_cast<long long>(rank * kSvWarps + warp) * per * kStep;
  const int lo = static_cast<int>(lo_l < V ? lo_l : V);
  const int hi = static_cast<int>(min(lo_l + static_cast<long long>(per) * kStep, static_cast<long long>(V)));

  // Residuals of the piece at v from its probabilities.  With q, or careful:
  // NaN and infinities count as 0; else an infinity shows in the sum, NaN and
  // negative values count as 0.
  auto values = [&](int v, bool careful, const Raw<T, kVec>& wp, const Raw<T, kVec>& wq, double (&r)[N]) {
    float fp[N];
    wp.widen(fp);
    if (q) {
      float fq[N];
      wq.widen(fq);
#pragma unroll
      for (int e = 0; e < N; ++e) r[e] = residual(fp[e], fq[e]);
    } else if (careful) {
#pragma unroll
      for (int e = 0; e < N; ++e) r[e] = residual(fp[e], v + e == hot ? 1.f : 0.f);
    } else {
      if (hot >= v && hot < v + N) {  // (one piece of the row)
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (v + e == hot) fp[e] -= 1.f;  // exact where positive: p and 1 within a factor of two
      }
#pragma unroll
      for (int e = 0; e < N; ++e) r[e] = static_cast<double>(fmaxf(fp[e], 0.f));
    }
  };
  // Sum of the steps from at to end, in every lane; kSvBatch pieces of a row
  // are on their way at once.
  auto stretch_sum = [&](int at, int end, bool careful) {
    double sum = 0.0;
    for (int v0 = at + lane * N; v0 < end; v0 += kSvBatch * kStep) {
      Raw<T, kVec> wp[kSvBatch], wq[kSvBatch];
#pragma unroll
      for (int i = 0; i < kSvBatch; ++i) wp[i].load(p, v0 + i * kStep, end);
      if (q) {
#pragma unroll
        for (int i = 0; i < kSvBatch; ++i) wq[i].load(q, v0 + i * kStep, end);
      }
#pragma unroll
      for (int i = 0; i < kSvBatch; ++i) {
        double r[N];
        values(v0 + i * kStep, careful, wp[i], wq[i], r);
#pragma unroll
        for (int e = 0; e < N; ++e) sum += r[e];
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
  };

  // u in [0, 1): anything else counts as the nearest value inside, so that a step is always found
  float uf = a.u_sample[seq];
  uf = uf >= 0.f ? fminf(uf, 0x1.fffffep-1f) : 0.f;
  const double u = static_cast<double>(uf);
  bool careful = false;
  for (int pass = 0;; ++pass) {
    const double sum = stretch_sum(lo, hi, careful);
    if (lane == 0) w_tot[warp] = sum;
    __syncthreads();
    double mine = 0.0;  // this CTA's total, in warp order
#pragma unroll
    for (int w = 0; w < kSvWarps; ++w) mine += w_tot[w];
    if (pass == 0) cluster_wait();
    if (threadIdx.x < n_cta) st_dsmem_f64(map_to_cta(smem_u32(&c_tot[rank]), threadIdx.x), mine);
    cluster_sync();
    double total = 0.0, base = 0.0;
    for (int c = 0; c < n_cta; ++c) {
      if (c == rank) base = total;
      total += c_tot[c];
    }
    if (!(total < INFINITY) && !careful) {
      careful = true;
    } else if (total > 0.0) {
      const double target = u * total;
      if (base <= target && base + mine > target) {  // the step lies in this CTA's stretches
        // the warp whose stretch holds it: the first whose end passes the target
        double from = base, run = 0.0;
        int ow = 0;
#pragma unroll
        for (int w = 0; w < kSvWarps; ++w) {
          const bool open = !(base + (run + w_tot[w]) > target);
          run += w_tot[w];
          if (open) {
            ow = w + 1;
            from = base + run;
          } else {
            break;
          }
        }
        // its steps again, a share per warp
        const int s_lo = min(V, (rank * kSvWarps + ow) * per * kStep), share = (per + kSvWarps - 1) / kSvWarps;
        const int s_hi = min(V, s_lo + per * kStep);
        const int m_lo = min(s_hi, s_lo + warp * share * kStep), m_hi = min(s_hi, m_lo + share * kStep);
        const double part = stretch_sum(m_lo, m_hi, careful);
        if (lane == 0) w_sub[warp] = part;
        __syncthreads();
        int sw = -1, last_sw = 0;
        double at = from, sw_from = from;
#pragma unroll
        for (int w = 0; w < kSvWarps; ++w) {
          const double x = w_sub[w];
          if (x > 0.0) last_sw = w;
          if (sw < 0 && at + x > target) {
            sw = w;
            sw_from = at;
          }
          at += x;
        }
        // (rounding may leave the step just past the end: then the last token
        // that has any probability)
        const bool past = sw < 0;
        if (warp == (past ? last_sw : sw)) {
          double walk = sw_from;
          int found = -1, last = -1;
          for (int v0 = m_lo; v0 < m_hi && found < 0; v0 += kStep) {
            double r[N], c[N];
            const int v = v0 + lane * N;
            Raw<T, kVec> wp, wq;
            wp.load(p, v, m_hi);
            if (q) wq.load(q, v, m_hi);
            values(v, careful, wp, wq, r);
            c[0] = r[0];
#pragma unroll
            for (int e = 1; e < N; ++e) c[e] = c[e - 1] + r[e];
            double inc = c[N - 1];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const double o = __shfl_up_sync(0xffffffffu, inc, d);
              if (lane >= d) inc += o;
            }
            const double ex = inc - c[N - 1];
            int hit = 0x7fffffff, pos = -1;
#pragma unroll
            for (int e = N - 1; e >= 0; --e) {
              if (r[e] > 0.0 && !past && walk + (ex + c[e]) > target) hit = v + e;
              if (r[e] > 0.0 && pos < 0) pos = v + e;
            }
            hit = __reduce_min_sync(0xffffffffu, hit);
            pos = __reduce_max_sync(0xffffffffu, pos);
            if (pos >= 0) last = pos;
            if (hit != 0x7fffffff) found = hit;
            walk += __shfl_sync(0xffffffffu, inc, 31);
          }
          if (lane == 0) a.out_ids[static_cast<size_t>(seq) * (K + 1) + k] = found >= 0 ? found : last;
        }
      }
      break;
    } else if (q || hot >= 0) {  // nothing left of the residual: the target's own row
      q = nullptr;
      hot = -1;
    } else {  // nothing there either
      if (rank == 0 && threadIdx.x == 0) {
        record_error(a.status, DVLM_ERR_BOUNDS);
        a.out_ids[static_cast<size_t>(seq) * (K + 1) + k] = 0;
      }
      break;
    }
    cluster_sync();  // c_tot and w_tot have been read
  }
  if (rank == 0) {
    for (int j = threadIdx.x; j <= K; j += kSvThreads)
      if (j != k) a.out_ids[static_cast<size_t>(seq) * (K + 1) + j] = j < k ? ids[j] : -1;
    if (threadIdx.x == 0) {
      a.accept_len[seq] = k;
      if (a.cache_len_out) a.cache_len_out[seq] = a.cache_len[seq] - (nd - k);
    }
  }
}

cudaError_t launch_spec_sample(const SpecSampleArgs& a, bool is_bf16, cudaStream_t s) {
  const int es = is_bf16 ? 2 : 4;
  const bool vec = (static_cast<long long>(a.V) * es) % 16 == 0 &&
                   (reinterpret_cast<uintptr_t>(a.target_p) & 15u) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.draft_p) & 15u) == 0;
  // CTAs per sequence: as many as keep the batch within what the SMs hold at
  // once (two CTAs each), up to the portable cluster size; fewer for
  // vocabularies that leave warps without a step of four pieces.  Rows of
  // 151936 with 1, 2, 4 and 8 CTAs each: one sequence of fp32 18.7, 12.4, 8.8
  // and 7.4 us; 32 of bf16 17.0, 11.8, 9.4 and 9.8; 128 of bf16 20.3, 16.7, 23.4
  // and 35.6; 64 of bf16 with the draft's rows 25.0, 16.6, 16.8 and 22.5
  const int steps = (a.V + 1023) / 1024, room = 2 * device_sm_count();
  int n_cta = 1;
  while (n_cta < kSvMaxCta && 2 * n_cta * a.b <= room && n_cta * kSvWarps / 4 < steps) n_cta *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(n_cta, a.b);
  cfg.blockDim = dim3(kSvThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = n_cta;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (is_bf16)
    return vec ? cudaLaunchKernelEx(&cfg, spec_sample_kernel<bf16, true>, a)
               : cudaLaunchKernelEx(&cfg, spec_sample_kernel<bf16, false>, a);
  return vec ? cudaLaunchKernelEx(&cfg, spec_sample_kernel<float, true>, a)
             : cudaLaunchKernelEx(&cfg, spec_sample_kernel<float, false>, a);
}

}  // namespace dvlm
