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
// A row is held in shared memory between the three steps that need it (maximum,
// sum of exponentials, gradient), 66 KB of it by a CTA; what is longer comes
// back from L2 for the gradient.  A few rows, or long ones, are shared out over
// the CTAs of a cluster.  The next row's asynchronous copies go out as the
// gradient leaves, so that HBM stays busy through the reductions (three CTAs
// per SM, 8192 bf16 rows of 32768 of which a third do not count: 180 us, 5.0
// TB/s; the exponentials, two per element, take about 0.55 of the time on their
// unit, which the loads have to overlap with).  The row's few scalars, loaded a
// row ahead, are worked out in double by one warp (the ratio is held against
// the clip borders, and the exponentials of differences lose digits in fp32).
// Vectors of 16 bytes are cut at the logits' alignment, row by row; where the
// gradient's row lies otherwise, each 16-byte store is put together from a
// lane's vector and the next lane's, so an odd vocabulary streams like an even
// one (2000 fp32 rows of 50257, gradient rows without padding: 206 us, 3.7 TB/s;
// with loads put together from two neighbours instead, through registers, 236).
#pragma once
#include <cfloat>

#include "common.cuh"

namespace gptb {

constexpr int POL_THREADS = 384;
constexpr int POL_WARPS = POL_THREADS / 32;
constexpr int POL_CTAS = 3;    // per SM
constexpr int POL_KEEP = 11;   // 16-byte vectors of a row that a thread keeps
constexpr int POL_SMEM = POL_KEEP * POL_THREADS * 16;  // 66 KB
constexpr int POL_CLUSTER = 8; // most CTAs that share a row

struct PolicyArgs {
  const int32_t* actions;
  const float *weights, *adv, *lp_old, *lp_ref;  // weights NULL: log-probabilities only; lp_ref NULL: d = 0
  float clip_lo, clip_hi, beta;
  float* logp;     // [rows]
  double* part;    // [clusters][3] this cluster's sums of w(-s + beta k), w k, w [clipped]
  long long ld, ldd;
  int rows, V;
  int cs;  // CTAs per row (cluster size)
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
// i N - p .. i N - p + N - 1 (p: how far the logits' row lies past a 16-byte
// boundary), the first and the last possibly in part.  ALIGNED: every row of
// both arrays starts on a boundary.
template <class T, bool ALIGNED>
struct PolicyRowView {
  static constexpr int N = PolVec<T>::N;
  const T* z;
  T* dz;
  int V, p, count;
  int last;  // the first vector that reaches past the end
  int r;     // the gradient's next 16-byte boundary after a vector's first element, in elements (0: they lie alike)
  __device__ __forceinline__ PolicyRowView(const T* z_, T* dz_, int V_) : z(z_), dz(dz_), V(V_) {
    p = ALIGNED ? 0 : (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
    count = (V + p + N - 1) / N;
    last = (V + p) / N;
    r = !ALIGNED && dz ? (p - (int)((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T)) + N) % N : 0;
  }
  __device__ __forceinline__ bool whole(int i) const { return (ALIGNED || i * N >= p) && i < last; }
  // vector i; elements outside the row are -inf
  __device__ __forceinline__ uint4 load(int i) const {
    const int e = i * N - p;
    if (whole(i)) return *reinterpret_cast<const uint4*>(z + e);
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = e + k >= 0 && e + k < V ? to_f(z[e + k]) : -INFINITY;
    return PolVec<T>::pack(v);
  }
  // The warp's vectors i (lane by lane, one after the other; those of lanes
  // that are `in`) of the gradient.  A lane whose vector and the next lane's
  // are whole stores the 16 bytes from its boundary on, the elements that no
  // such store covers go out one by one.
  __device__ __forceinline__ void store(int i, bool in, const uint4& u) const {
    const int e = i * N - p, lane = threadIdx.x & 31;
    const bool all = in && whole(i);
    bool to = all, from = all;  // elements r .. N-1, and 0 .. r-1, are in a 16-byte store
    if (ALIGNED || r == 0) {
      if (all) *reinterpret_cast<uint4*>(dz + e) = u;
    } else {
      uint4 y;
      y.x = __shfl_down_sync(0xffffffffu, u.x, 1);
      y.y = __shfl_down_sync(0xffffffffu, u.y, 1);
      y.z = __shfl_down_sync(0xffffffffu, u.z, 1);
      y.w = __shfl_down_sync(0xffffffffu, u.w, 1);
      const unsigned wholes = __ballot_sync(0xffffffffu, all);
      to = all && lane < 31 && (wholes >> ((lane + 1) & 31) & 1u);
      from = all && lane > 0 && (wholes >> ((lane - 1) & 31) & 1u);
      if (to) {
        const int sh = r * (int)sizeof(T);
        const bool two = sh & 8, one = sh & 4;
        const uint32_t a0 = two ? u.z : u.x, a1 = two ? u.w : u.y, a2 = two ? y.x : u.z, a3 = two ? y.y : u.w,
                       a4 = two ? y.z : y.x, a5 = two ? y.w : y.y;
        const uint32_t b0 = one ? a1 : a0, b1 = one ? a2 : a1, b2 = one ? a3 : a2, b3 = one ? a4 : a3, b4 = one ? a5 : a4;
        const int h = (sh & 2) * 8;
        *reinterpret_cast<uint4*>(dz + e + r) =
            sizeof(T) == 4 ? make_uint4(b0, b1, b2, b3)
                           : make_uint4(__funnelshift_r(b0, b1, h), __funnelshift_r(b1, b2, h),
                                        __funnelshift_r(b2, b3, h), __funnelshift_r(b3, b4, h));
      }
    }
    if (in && !(to && from)) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (!(ALIGNED || k >= r ? to : from) && e + k >= 0 && e + k < V) dz[e + k] = from_f<T>(PolVec<T>::get(u, k));
    }
  }
};

// part `rank` of n of a row of V zeros, by the CTA
template <class T>
__device__ __forceinline__ void policy_zero(T* dz, int V, int rank, int n) {
  constexpr int N = PolVec<T>::N;
  const int p = (int)((reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T)), count = (V + p + N - 1) / N;
  const int end = (int)((long long)count * (rank + 1) / n);
  for (int i = (int)((long long)count * rank / n) + threadIdx.x; i < end; i += blockDim.x) {
    const int e = i * N - p;
    if (e >= 0 && e + N <= V) {
      *reinterpret_cast<uint4*>(dz + e) = make_uint4(0, 0, 0, 0);
    } else {
      for (int k = max(0, e); k < min(V, e + N); ++k) dz[k] = from_f<T>(0.f);
    }
  }
}

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

// exp(z - m) as exp2(z L - M), one fused operation and the exponential: M is
// m L rounded to fp32, and the sum of such exponentials times correction() is
// the sum of exp(z - m).  The product is exact inside the fused operation and
// the difference is small where it counts, so no digits are lost -- as long as
// M's rounding error, by which every exponent is off, is small itself: for |m|
// up to POL_FAR it is at most 2^-4.  (Past 3e9 it can be 128, where exp2 of it
// is infinite and that of its opposite 0.)  So a thread's maximum starts at
// -POL_FAR, which a strip masked with a large value never leaves, and a row
// whose maximum lies outside is done over with policy_far().
constexpr float POL_FAR = 0x1p20f;
struct PolicyExp {
  float ml, m;
  __device__ __forceinline__ explicit PolicyExp(float m_) : ml(m_ * LOG2E), m(m_) {}
  __device__ __forceinline__ float operator()(float z) const { return fast_exp2(fmaf(z, LOG2E, -ml)); }
  __device__ __forceinline__ float correction() const { return fast_exp2(-fmaf(m, LOG2E, -ml)); }
};
// The same from the difference: z - m is exact for z near m, and where it is
// not the exponential is 0.  (One operation more per element: 2000 fp32 rows of
// 50257 in 234 us where every vector chooses between the two forms, 214 so.)
__device__ __forceinline__ float policy_far(float z, float m) { return fast_exp2((z - m) * LOG2E); }

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
    const double k = isinf(e) ? e : e - d - 1.0;  // (an action of probability 0: inf, not inf - inf)
    const double beta = a.beta;
    const bool term = beta != 0.0;  // (without the term e and k may be infinite)
    r.g = w * ((term ? beta * (1.0 - e) : 0.0) - (kept ? plain : 0.0));
    r.loss = w * ((term ? beta * k : 0.0) - (kept ? plain : capped));
    r.kl = w * k;
    r.clipped = kept ? 0.0 : w;
  }
  return r;
}

// Rows first .. end-1 of cluster `at` of n: contiguous shares of equal cost, a row that is
// read and written counting 2, one that is only zeroed 1.  (With the same
// number of rows for each, 28 on average of which a third do not count, the
// slowest has a quarter more to do than the mean.)
__device__ __forceinline__ int2 policy_share(const PolicyArgs& a, int at, int n, int* s_scan, int* s_range) {
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
  for (int q = 0; q < 2; ++q) {  // the row in which the cost reaches the share's bound
    const int want = (int)((long long)(at + q) * total / n);
    if (before <= want && want < before + mine) {
      int sum = before;
      for (int i = lo; i < hi; ++i) {
        sum += a.weights[i] != 0.f ? 2 : 1;
        if (want < sum) {
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
__global__ void __launch_bounds__(POL_THREADS, POL_CTAS)
    policy_rows_kernel(const T* logits, T* dlogits, const PolicyArgs a) {
  constexpr int N = PolVec<T>::N;
  using Row = PolicyRowView<T, ALIGNED>;
  extern __shared__ __align__(16) uint4 pol_slots[];  // [POL_KEEP][POL_THREADS]
  __shared__ float sm[POL_WARPS], ss[POL_WARPS];
  // This CTA's maximum and sum of the row, in turn: a CTA may be an exchange
  // ahead of those that still read its part of the last one, not two.
  __shared__ float2 s_part[2];
  __shared__ float s_g, s_inv;
  __shared__ int s_scan[POL_WARPS], s_range[2];
  __shared__ PolicyIn s_in[2];  // of rows i and i + 1, by parity
  __shared__ double s_sum[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % a.cs, at = blockIdx.x / a.cs, n = gridDim.x / a.cs;
  pdl_launch();  // (policy_stats_kernel may be set up; it waits for this grid to end)
  uint4* slot = pol_slots + tid;  // slot j of this thread: slot[j * POL_THREADS]
  int first, end;
  if (a.weights) {
    const int2 r = policy_share(a, at, n, s_scan, s_range);
    first = r.x;
    end = r.y;
  } else {
    first = (int)((long long)at * a.rows / n);
    end = (int)((long long)(at + 1) * a.rows / n);
  }
  const auto view = [&](int i) {
    return Row(logits + (long long)i * a.ld, dlogits ? dlogits + (long long)i * a.ldd : nullptr, a.V);
  };
  // this CTA's vectors of a row are lo(row) .. hi(row) - 1; thread t has lo + t, lo + t + POL_THREADS, ...
  const auto lo = [&](const Row& r) { return (int)((long long)r.count * rank / a.cs); };
  const auto hi = [&](const Row& r) { return (int)((long long)r.count * (rank + 1) / a.cs); };
  // one vector of a row into slot j
  const auto copy = [&](int j, const Row& r, int c) {
    if (r.whole(c))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot + j * POL_THREADS)),
                   "l"(r.z + (c * N - r.p)) : "memory");
    else
      slot[j * POL_THREADS] = r.load(c);
  };
  if (tid == 0) {
    s_sum[0] = s_sum[1] = s_sum[2] = 0.0;
    if (first < end) policy_in(a, first, &s_in[first & 1]);
    policy_wait();
  }
  __syncthreads();
  bool have = false;  // the row is being loaded already
  int turn = 0;       // of the cluster's exchanges
  for (int i = first; i < end; ++i) {
    const Row row = view(i);
    const int c_lo = lo(row) + tid, c_hi = hi(row);
    const int y = s_in[i & 1].y;
    const float w = s_in[i & 1].w;
    if (tid == 0 && i + 1 < end) policy_in(a, i + 1, &s_in[(i + 1) & 1]);
    // (an action outside the vocabulary is reported, never read)
    if (w == 0.f || y < 0 || y >= a.V) {
      if (dlogits) policy_zero(row.dz, a.V, rank, a.cs);
      if (tid == 0) {
        if (rank == 0) {
          if (w != 0.f) record_error(ERRW_BAD_TARGET);
          a.logp[i] = 0.f;
        }
        policy_wait();
      }
      __syncthreads();
      continue;
    }
    const int kept = max(0, min(POL_KEEP, (c_hi - c_lo + POL_THREADS - 1) / POL_THREADS));
    const int c_rest = c_lo + POL_KEEP * POL_THREADS;  // the first vector that is not kept
    if (!have) {
      for (int j = 0; j < kept; ++j) copy(j, row, c_lo + j * POL_THREADS);
    }
    const float za = to_f(row.z[y]);
    // this thread's maximum and sum of exponentials, then the row's
    float m = -POL_FAR;
    policy_wait();       // (this thread's copies)
#pragma unroll 2
    for (int j = 0; j < kept; ++j) m = fmaxf(m, PolVec<T>::max(slot[j * POL_THREADS]));
    PolicyExp e(m);
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
    const auto add = [&](const uint4& u) {
#pragma unroll
      for (int k = 0; k < N; ++k) s4[k & 3] += e(PolVec<T>::get(u, k));
    };
#pragma unroll 2
    for (int j = 0; j < kept; ++j) add(slot[j * POL_THREADS]);
    // what is not kept, in one pass: the sums are rescaled when the maximum grows
    for (int c = c_rest; c < c_hi; c += POL_THREADS) {
      const uint4 u = row.load(c);
      const float mx = PolVec<T>::max(u);
      if (mx > m) {
        const float r = fast_exp2((m - mx) * LOG2E) * e.correction();
        m = mx;
        e = PolicyExp(m);
#pragma unroll
        for (int k = 0; k < 4; ++k) s4[k] *= r / e.correction();
      }
      add(u);
    }
    // the row's, from every thread's maximum and sum; S in warp 0, with a cluster in all
    float S = 0.f;
    const auto join = [&](float s) {
      const float mw = warp_max(m);
      s = warp_sum(s * fast_exp2((m - mw) * LOG2E));
      if (lane == 0) {
        sm[warp] = mw;
        ss[warp] = s;
      }
      __syncthreads();
      const float m_lane = lane < POL_WARPS ? sm[lane] : -FLT_MAX;
      m = warp_max(m_lane);
      if (warp == 0) S = warp_sum(lane < POL_WARPS ? ss[lane] * fast_exp2((m_lane - m) * LOG2E) : 0.f);
      if (a.cs > 1) {  // the cluster's: each CTA reads the others' parts
        turn ^= 1;
        if (tid == 0) s_part[turn] = make_float2(m, S);
        cluster_sync_all();
        float2 part = make_float2(-FLT_MAX, 0.f);
        if (lane < a.cs)
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(part.x), "=f"(part.y)
                       : "r"(map_shared_rank(&s_part[turn], lane)) : "memory");
        m = warp_max(part.x);
        S = warp_sum(part.y * fast_exp2((part.x - m) * LOG2E));
      }
    };
    join(((s4[0] + s4[1]) + (s4[2] + s4[3])) * e.correction());
    const bool far = !(fabsf(m) < POL_FAR);  // (the same in the whole cluster)
    if (far) {
      m = -FLT_MAX;  // (so that a strip of -inf adds 0)
      for (int c = c_lo; c < c_hi; c += POL_THREADS) m = fmaxf(m, PolVec<T>::max(row.load(c)));
      s4[0] = s4[1] = s4[2] = s4[3] = 0.f;
      for (int c = c_lo; c < c_hi; c += POL_THREADS) {
        const uint4 u = row.load(c);
#pragma unroll
        for (int k = 0; k < N; ++k) s4[k & 3] += policy_far(PolVec<T>::get(u, k), m);
      }
      __syncthreads();  // (sm and ss have been read)
      join((s4[0] + s4[1]) + (s4[2] + s4[3]));
    }
    e = PolicyExp(m);
    if (warp == 0) {
      const PolicyRow r = policy_row(a, s_in[i & 1], m, S, za);
      if (lane == 0) {
        s_sum[0] += r.loss;
        s_sum[1] += r.kl;
        s_sum[2] += r.clipped;
        if (rank == 0) a.logp[i] = (float)r.lp;
        s_g = (float)r.g;
        s_inv = (float)(-r.g / (double)S);
        policy_wait();  // the next row's scalars
      }
    }
    __syncthreads();
    if (!dlogits) continue;
    const float inv = far ? s_inv : s_inv * e.correction();
    if (far) {  // (no copies of the next row yet)
      have = false;
      for (int c = c_lo; c - lane < c_hi; c += POL_THREADS) {
        const uint4 u = c < c_hi ? row.load(c) : make_uint4(0, 0, 0, 0);
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = policy_far(PolVec<T>::get(u, k), m) * inv;
        row.store(c, c < c_hi, PolVec<T>::pack(v));
      }
    } else {
      // (the whole warp, its lanes' vectors one after the other; c of lane 0 decides)
      const auto grad = [&](int c, bool in, const uint4& u) {
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = e(PolVec<T>::get(u, k)) * inv;
        row.store(c, in, PolVec<T>::pack(v));
      };
      // what was not kept first, while it is still in L2; then the slots, each
      // refilled from the next row as its gradient leaves.  (Lane 0 has the most
      // slots; the stores of ALIGNED need no other lane.)
      for (int c = c_rest; ALIGNED ? c < c_hi : c - lane < c_hi; c += POL_THREADS)
        grad(c, c < c_hi, c < c_hi ? row.load(c) : make_uint4(0, 0, 0, 0));
      const PolicyIn& in = s_in[(i + 1) & 1];
      have = i + 1 < end && in.w != 0.f && in.y >= 0 && in.y < a.V;
      if constexpr (ALIGNED) {
        const Row next(logits + (long long)(i + 1) * a.ld, nullptr, a.V);  // (its vectors lie alike)
#pragma unroll 2
        for (int j = 0; j < kept; ++j) {
          grad(c_lo + j * POL_THREADS, true, slot[j * POL_THREADS]);
          if (have) copy(j, next, c_lo + j * POL_THREADS);
        }
      } else {
        const Row next = view(have ? i + 1 : i);
        const int n_lo = lo(next) + tid, n_hi = have ? hi(next) : n_lo;
        const int slots = __shfl_sync(0xffffffffu, kept, 0);
        int j = 0;
#pragma unroll 2
        for (; j < slots; ++j) {
          grad(c_lo + j * POL_THREADS, j < kept, slot[j * POL_THREADS]);
          if (n_lo + j * POL_THREADS < n_hi) copy(j, next, n_lo + j * POL_THREADS);
        }
        for (; j < POL_KEEP && n_lo + j * POL_THREADS < n_hi; ++j) copy(j, next, n_lo + j * POL_THREADS);
      }
    }
    __syncwarp();  // (the vectors' stores come before the next one)
    // the action's own element, by the lane whose vector it is in
    const int c_y = (y + row.p) / N;
    if (c_y >= c_lo && c_y < c_hi && (c_y - c_lo) % POL_THREADS == 0)
      row.dz[y] = from_f<T>(fmaf(far ? policy_far(za, m) : e(za), inv, s_g));
  }
  if (rank == 0 && tid < 3 && a.part) a.part[at * 3 + tid] = s_sum[tid];
  if (a.cs > 1) cluster_sync_all();  // no CTA leaves while another may read its part
}

// the clusters' sums, added in a fixed order: one warp per statistic
__global__ void __launch_bounds__(96) policy_stats_kernel(const double* part, int n, float* __restrict__ stats) {
  pdl_wait();  // (the sums)
  const int q = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double v = 0.0;
  for (int i = lane; i < n; i += 32) v += part[i * 3 + q];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) stats[q] = (float)v;
}

}  // namespace gptb
