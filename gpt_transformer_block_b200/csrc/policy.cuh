// Clipped policy loss with a KL term on the logits, and its gradient.
//
// Row i holds the logits z of one sampled token a with weight w, advantage A
// and the log-probabilities lp_old, lp_ref that the sampling and the reference
// policy gave it:
//   lp   = z_a - log sum_j exp z_j
//   r    = exp(lp - lp_old),  s = min(r A, clip(r, 1 - lo, 1 + hi) A)
//   d    = lp_ref - lp,       k = exp d - d - 1      (>= 0, zero at d = 0)
//   loss = sum_i w (-s + beta k)
//   g    = d loss / d lp = w ( -[r A <= clip(r) A] r A + beta (1 - exp d) )
//   dz_j = g ([j = a] - exp(z_j) / sum exp z)
// A row of weight 0 carries nothing: its logits are not read, its gradient is 0.
//
// Bound by HBM: one read of the rows that count and one write of the gradient.
// A CTA takes one row at a time and keeps its first 64 KB on the SM between the
// three steps that need it (maximum, sum of exponentials, gradient); what is
// longer comes back from L2 for the gradient.  The next row's loads go out as
// the gradient leaves, so that HBM stays busy through the reductions.  The
// row's few scalars, loaded a row ahead, are worked out in double by one warp
// (the ratio is held against the clip borders, and the exponentials of
// differences lose digits in fp32).
// Rows that start on 16-byte boundaries stay in shared memory, filled by
// asynchronous copies: three CTAs per SM.  Other rows stay in registers, two
// CTAs per SM: vectors of 16 bytes are cut at the gradient's alignment, and
// where the logits row starts elsewhere each is put together from two
// neighbouring 16-byte loads (the second is the next lane's first: an L1 hit),
// so an odd vocabulary streams like an even one.
#pragma once
#include <cfloat>

#include "common.cuh"

namespace gptb {

constexpr int POL_THREADS = 384;
constexpr int POL_WARPS = POL_THREADS / 32;
constexpr int POL_KEEP = 11;  // 16-byte vectors of a row that a thread keeps: 66 KB per CTA
constexpr int POL_AHEAD = 2; // ... of a long row's rest that it loads at once
constexpr int POL_SMEM = POL_KEEP * POL_THREADS * 16;

struct PolicyArgs {
  const int32_t* actions;
  const float *weights, *adv, *lp_old, *lp_ref;  // weights NULL: log-probabilities only; lp_ref NULL: d = 0
  float clip_lo, clip_hi, beta;
  float* logp;     // [rows]
  double* part;    // [gridDim.x][3] this CTA's sums of w(-s + beta k), w k, w [clipped]
  long long ld, ldd;
  int rows, V;
};

// 16 bytes as elements
template <class T>
struct PolVec;
template <>
struct PolVec<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const uint4& u, int k) {  // k is a constant after unrolling
    const uint32_t w = k < 2 ? u.x : k < 4 ? u.y : k < 6 ? u.z : u.w;
    return __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};
template <>
struct PolVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const uint4& u, int k) {
    return __uint_as_float(k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w);
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    return fmaxf(fmaxf(get(u, 0), get(u, 1)), fmaxf(get(u, 2), get(u, 3)));
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

// A row of V elements as vectors of 16 bytes: vector i holds the elements
// i N - p .. i N - p + N - 1 (p: how far the gradient's row lies past a 16-byte
// boundary), the first and the last possibly in part.  ALIGNED: every row of
// both arrays starts on a boundary (p = 0, and the logits are cut likewise).
template <class T, bool ALIGNED>
struct PolicyRowView {
  static constexpr int N = PolVec<T>::N;
  const T* z;
  T* dz;
  int V, p, count;
  int last;   // the first vector that reaches past the end
  int shift;  // bytes from the 16-byte boundary below a vector's logits to them
  __device__ __forceinline__ PolicyRowView(const T* z_, T* dz_, int V_) : z(z_), dz(dz_), V(V_), p(0), shift(0) {
    if constexpr (!ALIGNED) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(dz ? (const T*)dz : z) & 15u;
      p = (int)(at / sizeof(T));
      shift = (int)((reinterpret_cast<uintptr_t>(z) - at) & 15u);
    }
    count = (V + p + N - 1) / N;
    last = (V + p) / N;
  }
  __device__ __forceinline__ bool whole(int i) const { return (ALIGNED || i * N >= p) && i < last; }
  // vector i; elements outside the row are -inf
  __device__ __forceinline__ uint4 load(int i) const {
    const int e = i * N - p;
    if (whole(i)) {
      if (ALIGNED || shift == 0) return *reinterpret_cast<const uint4*>(z + e);
      // (16 bytes from z + e on: both aligned words hold some of them)
      if (e + N + N <= V && e >= N) {
        const uint8_t* a = reinterpret_cast<const uint8_t*>(z + e) - shift;
        const uint4 x = *reinterpret_cast<const uint4*>(a), y = *reinterpret_cast<const uint4*>(a + 16);
        const bool two = shift & 8, one = shift & 4;
        const uint32_t a0 = two ? x.z : x.x, a1 = two ? x.w : x.y, a2 = two ? y.x : x.z, a3 = two ? y.y : x.w,
                       a4 = two ? y.z : y.x, a5 = two ? y.w : y.y;
        const uint32_t b0 = one ? a1 : a0, b1 = one ? a2 : a1, b2 = one ? a3 : a2, b3 = one ? a4 : a3, b4 = one ? a5 : a4;
        if constexpr (sizeof(T) == 4) return make_uint4(b0, b1, b2, b3);
        const int h = (shift & 2) * 8;
        return make_uint4(__funnelshift_r(b0, b1, h), __funnelshift_r(b1, b2, h), __funnelshift_r(b2, b3, h),
                          __funnelshift_r(b3, b4, h));
      }
    }
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = e + k >= 0 && e + k < V ? to_f(z[e + k]) : -INFINITY;
    return PolVec<T>::pack(v);
  }
  __device__ __forceinline__ void store(int i, const uint4& u) const {
    const int e = i * N - p;
    if (whole(i)) {
      *reinterpret_cast<uint4*>(dz + e) = u;
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (e + k >= 0 && e + k < V) dz[e + k] = from_f<T>(PolVec<T>::get(u, k));
    }
  }
};

// A row's scalars, copied to shared memory a row ahead (by one thread, which
// waits for them before a barrier that the others wait at too).
struct PolicyIn {
  int y;
  float w, adv, lp_old, lp_ref;
};
__device__ __forceinline__ void policy_copy(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void policy_in(const PolicyArgs& a, int i, PolicyIn* in) {
  policy_copy(&in->y, a.actions + i);
  if (a.weights) {
    policy_copy(&in->w, a.weights + i);
    policy_copy(&in->adv, a.adv + i);
    policy_copy(&in->lp_old, a.lp_old + i);
    if (a.lp_ref) policy_copy(&in->lp_ref, a.lp_ref + i);
  } else {
    in->w = 1.f;
  }
}
__device__ __forceinline__ void policy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The vectors tid, tid + POL_THREADS, ... of a row that a thread keeps: slots of
// its own, in shared memory or in registers.
template <class T, bool ALIGNED>
struct PolicyKeep;
template <class T>
struct PolicyKeep<T, true> {
  uint32_t at;  // shared-memory address of slot 0
  __device__ __forceinline__ PolicyKeep(uint8_t* smem) : at(smem_u32(smem) + threadIdx.x * 16) {}
  __device__ __forceinline__ void fill(int j, const PolicyRowView<T, true>& row, int c) {
    if (row.whole(c)) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + j * POL_THREADS * 16),
                   "l"(row.z + (long long)c * PolVec<T>::N) : "memory");
    } else {
      const uint4 u = row.load(c);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + j * POL_THREADS * 16), "r"(u.x), "r"(u.y),
                   "r"(u.z), "r"(u.w) : "memory");
    }
  }
  __device__ __forceinline__ void wait() { policy_wait(); }  // all fills so far have landed
  __device__ __forceinline__ uint4 get(int j) const {
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(at + j * POL_THREADS * 16) : "memory");
    return u;
  }
};
template <class T>
struct PolicyKeep<T, false> {
  uint4 u[POL_KEEP];
  __device__ __forceinline__ PolicyKeep(uint8_t*) {}
  __device__ __forceinline__ void fill(int j, const PolicyRowView<T, false>& row, int c) { u[j] = row.load(c); }
  __device__ __forceinline__ void wait() {}
  __device__ __forceinline__ const uint4& get(int j) const { return u[j]; }
};

// what one warp works out for a row from its maximum m, sum s = sum exp(z - m)
// and logit za: the log-probability, the gradient's coefficient g and the three sums
struct PolicyRow {
  double lp, g, loss, kl, clipped;
};
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, const PolicyIn& in, float m, float s, float za) {
  PolicyRow r;
  r.lp = ((double)za - (double)m) - log((double)s);
  r.g = r.loss = r.kl = r.clipped = 0.0;
  if (a.weights) {
    const double w = in.w, A = in.adv;
    const double d = a.lp_ref ? (double)in.lp_ref - r.lp : 0.0;
    // both exponentials at once: exp(lp - lp_old) in lane 0, exp(d) in lane 1
    const double x = exp((threadIdx.x & 31) == 1 ? d : r.lp - (double)in.lp_old);
    const double ratio = __shfl_sync(0xffffffffu, x, 0), e = __shfl_sync(0xffffffffu, x, 1);
    const double plain = ratio * A;
    const double capped = fmin(fmax(ratio, 1.0 - (double)a.clip_lo), 1.0 + (double)a.clip_hi) * A;
    const bool kept = plain <= capped;
    const double k = e - d - 1.0;
    r.g = w * ((double)a.beta * (1.0 - e) - (kept ? plain : 0.0));
    r.loss = w * ((double)a.beta * k - (kept ? plain : capped));
    r.kl = w * k;
    r.clipped = kept ? 0.0 : w;
  }
  return r;
}

// Rows first .. end-1 of a CTA: contiguous shares of equal cost, a row that is
// read and written counting 2, one that is only zeroed 1.  (With the same
// number of rows for each CTA, 28 on average of which a third do not count,
// the slowest CTA had a quarter more to do than the mean.)
__device__ __forceinline__ int2 policy_share(const PolicyArgs& a, int* s_scan, int* s_range) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.rows + POL_THREADS - 1) / POL_THREADS;
  const int lo = min(a.rows, tid * per), hi = min(a.rows, lo + per);
  int mine = 0;
  for (int i = lo; i < hi; ++i) mine += a.weights[i] != 0.f ? 2 : 1;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_scan[warp] = inc;
  if (tid < 2) s_range[tid] = a.rows;
  __syncthreads();
  int before = inc - mine, total = 0;
  for (int w = 0; w < POL_WARPS; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {  // the row in which the cost reaches the CTA's bound
    const int want = (int)((long long)(blockIdx.x + q) * total / gridDim.x);
    if (before <= want && want < before + mine) {
      int at = before;
      for (int i = lo; i < hi; ++i) {
        at += a.weights[i] != 0.f ? 2 : 1;
        if (want < at) {
          s_range[q] = i;
          break;
        }
      }
    }
  }
  __syncthreads();
  return make_int2(s_range[0], s_range[1]);
}

template <class T, bool ALIGNED>
__global__ void __launch_bounds__(POL_THREADS, ALIGNED ? 3 : 2)
    policy_rows_kernel(const T* logits, T* dlogits, PolicyArgs a) {
  constexpr int N = PolVec<T>::N;
  __shared__ float sm[POL_WARPS], ss[POL_WARPS];
  __shared__ float s_g, s_inv;
  __shared__ int s_scan[POL_WARPS], s_range[2];
  __shared__ PolicyIn s_in[2];  // of rows i and i + 1, by parity
  __shared__ double s_sum[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int first, end;
  if (a.weights) {
    const int2 r = policy_share(a, s_scan, s_range);
    first = r.x;
    end = r.y;
  } else {
    first = (int)((long long)blockIdx.x * a.rows / gridDim.x);
    end = (int)((long long)(blockIdx.x + 1) * a.rows / gridDim.x);
  }
  // f(j, c) for each kept vector: slot j of this thread, vector c of a row of `count`
  const auto each = [&](int count, auto&& f) {
    if constexpr (ALIGNED) {
      const int n = min(POL_KEEP, (count - tid + POL_THREADS - 1) / POL_THREADS);  // (the same for every row)
#pragma unroll 2
      for (int j = 0; j < n; ++j) f(j, tid + j * POL_THREADS);
    } else {
#pragma unroll
      for (int j = 0; j < POL_KEEP; ++j)  // (registers have to be named)
        if (tid + j * POL_THREADS < count) f(j, tid + j * POL_THREADS);
    }
  };
  const auto view = [&](int i) {
    return PolicyRowView<T, ALIGNED>(logits + (long long)i * a.ld, dlogits ? dlogits + (long long)i * a.ldd : nullptr, a.V);
  };
  extern __shared__ __align__(16) uint8_t pol_smem[];  // (ALIGNED)
  PolicyKeep<T, ALIGNED> keep(pol_smem);
  if (tid == 0) {
    s_sum[0] = s_sum[1] = s_sum[2] = 0.0;
    if (first < end) policy_in(a, first, &s_in[first & 1]);
    policy_wait();
  }
  __syncthreads();
  bool have = false;  // the row is being loaded already
  for (int i = first; i < end; ++i) {
    const PolicyRowView<T, ALIGNED> row = view(i);
    const int y = s_in[i & 1].y;
    const float w = s_in[i & 1].w;
    if (tid == 0 && i + 1 < end) policy_in(a, i + 1, &s_in[(i + 1) & 1]);
    // (an action outside the vocabulary is reported, never read)
    if (w == 0.f || y < 0 || y >= a.V) {
      if (dlogits)
        for (int c = tid; c < row.count; c += POL_THREADS) row.store(c, make_uint4(0, 0, 0, 0));
      if (tid == 0) {
        if (w != 0.f) record_error(ERRW_BAD_TARGET);
        a.logp[i] = 0.f;
        policy_wait();
      }
      __syncthreads();
      continue;
    }
    if (!have) each(row.count, [&](int j, int c) { keep.fill(j, row, c); });
    have = false;
    const float za = to_f(row.z[y]);
    // this thread's maximum and sum of exponentials, then the row's
    float m = -FLT_MAX;  // (so that a strip of -inf adds 0)
    keep.wait();
    each(row.count, [&](int j, int) { m = fmaxf(m, PolVec<T>::max(keep.get(j))); });
    // exp2((z - m) log2 e) of elements k, k + 1 (z - m first: z log2 e alone
    // would lose the digits of large logits, and overflow at the type's lowest)
    unsigned long long m2 = f2_pack(-m, -m);
    const unsigned long long l2 = f2_pack(LOG2E, LOG2E);
    const auto exp_pair = [&](const uint4& w, int k) {
      float lo, hi;
      f2_unpack(f2_mul(f2_add(f2_pack(PolVec<T>::get(w, k), PolVec<T>::get(w, k + 1)), m2), l2), lo, hi);
      return f2_pack(fast_exp2(lo), fast_exp2(hi));
    };
    unsigned long long s2 = 0;  // (0, 0)
    const auto add = [&](const uint4& w) {
#pragma unroll
      for (int k = 0; k < N; k += 2) s2 = f2_add(s2, exp_pair(w, k));
    };
    each(row.count, [&](int j, int) { add(keep.get(j)); });
    // the rest of a long row in one pass, the sum rescaled when the maximum grows
    for (int c0 = tid + POL_KEEP * POL_THREADS; c0 < row.count; c0 += POL_AHEAD * POL_THREADS) {
      uint4 w[POL_AHEAD];
#pragma unroll
      for (int q = 0; q < POL_AHEAD; ++q)
        if (c0 + q * POL_THREADS < row.count) w[q] = row.load(c0 + q * POL_THREADS);
#pragma unroll
      for (int q = 0; q < POL_AHEAD; ++q) {
        if (c0 + q * POL_THREADS < row.count) {
          const float mx = PolVec<T>::max(w[q]);
          if (mx > m) {
            const float r = fast_exp2((m - mx) * LOG2E);
            s2 = f2_mul(s2, f2_pack(r, r));
            m = mx;
            m2 = f2_pack(-m, -m);
          }
          add(w[q]);
        }
      }
    }
    float s, s_hi;
    f2_unpack(s2, s, s_hi);
    s += s_hi;
    const float mw = warp_max(m);
    s = warp_sum(s * fast_exp2((m - mw) * LOG2E));
    if (lane == 0) {
      sm[warp] = mw;
      ss[warp] = s;
    }
    __syncthreads();
    const float m_lane = sm[lane % POL_WARPS];
    m = warp_max(m_lane);
    m2 = f2_pack(-m, -m);
    if (warp == 0) {
      const float S = warp_sum(lane < POL_WARPS ? ss[lane] * fast_exp2((m_lane - m) * LOG2E) : 0.f);
      const PolicyRow r = policy_row(a, s_in[i & 1], m, S, za);
      if (lane == 0) {
        s_sum[0] += r.loss;
        s_sum[1] += r.kl;
        s_sum[2] += r.clipped;
        a.logp[i] = (float)r.lp;
        s_g = (float)r.g;
        s_inv = (float)(-r.g / (double)S);
        policy_wait();  // the next row's scalars
      }
    }
    __syncthreads();
    if (!dlogits) continue;
    const float g = s_g, inv = s_inv;
    const unsigned long long i2 = f2_pack(inv, inv);
    const auto grad = [&](int c, const uint4& w) {
      float v[N];
#pragma unroll
      for (int k = 0; k < N; k += 2) f2_unpack(f2_mul(exp_pair(w, k), i2), v[k], v[k + 1]);
      row.store(c, PolVec<T>::pack(v));
    };
    // the rest of a long row first, while its logits are still in L2; then what
    // was kept, each slot refilled from the next row as its gradient leaves
    for (int c0 = tid + POL_KEEP * POL_THREADS; c0 < row.count; c0 += POL_AHEAD * POL_THREADS) {
      uint4 w[POL_AHEAD];
#pragma unroll
      for (int q = 0; q < POL_AHEAD; ++q)
        if (c0 + q * POL_THREADS < row.count) w[q] = row.load(c0 + q * POL_THREADS);
#pragma unroll
      for (int q = 0; q < POL_AHEAD; ++q)
        if (c0 + q * POL_THREADS < row.count) grad(c0 + q * POL_THREADS, w[q]);
    }
    const PolicyIn& in = s_in[(i + 1) & 1];
    have = i + 1 < end && in.w != 0.f && in.y >= 0 && in.y < a.V;
    const PolicyRowView<T, ALIGNED> next = view(have ? i + 1 : i);
    if constexpr (ALIGNED) {
      each(row.count, [&](int j, int c) {
        grad(c, keep.get(j));
        if (have) keep.fill(j, next, c);
      });
    } else {
#pragma unroll
      for (int j = 0; j < POL_KEEP; ++j) {
        const int c = tid + j * POL_THREADS;
        if (c < row.count) grad(c, keep.get(j));
        if (have && c < next.count) keep.fill(j, next, c);
      }
    }
    // the action's own element, by the thread that wrote its vector
    if (tid == (y + row.p) / N % POL_THREADS)
      row.dz[y] = from_f<T>(fmaf(fast_exp2((za - m) * LOG2E), inv, g));
  }
  if (tid < 3 && a.part) a.part[blockIdx.x * 3 + tid] = s_sum[tid];
}

// the CTAs' sums, added in a fixed order: one warp per statistic
__global__ void __launch_bounds__(96) policy_stats_kernel(const double* __restrict__ part, int n, float* __restrict__ stats) {
  const int q = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double v = 0.0;
  for (int i = lane; i < n; i += 32) v += part[i * 3 + q];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) stats[q] = (float)v;
}

}  // namespace gptb
