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
// One CTA per row at a time (persistent over the rows): a pass with the
// running maximum and sum of exponentials, the row's few scalars in double by
// one thread (the ratio is held against the clip borders, and the exponentials
// of differences lose digits in fp32), then the gradient pass, which reads the
// row again from L2.
#pragma once
#include "common.cuh"
#include "elementwise.cuh"

namespace gptb {

constexpr int POL_THREADS = 512;
constexpr int POL_WARPS = POL_THREADS / 32;

struct PolicyArgs {
  const int32_t* actions;
  const float *weights, *adv, *lp_old, *lp_ref;  // weights NULL: log-probabilities only; lp_ref NULL: d = 0
  float clip_lo, clip_hi, beta;
  float* logp;     // [rows]
  double* part;    // [gridDim.x][3] this CTA's sums of w(-s + beta k), w k, w [clipped]
  long long ld, ldd;
  int rows, V;
};

// VEC elements per access: 16 bytes where every row of both arrays starts on a
// 16-byte boundary, else 1
template <class T, int VEC>
struct PolVec {
  static __device__ __forceinline__ void load(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
      load8(p, v);
    } else if constexpr (VEC == 4) {
      const float4 u = *reinterpret_cast<const float4*>(p);
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
      v[0] = to_f(p[0]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
      store8(p, v);
    } else if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      p[0] = from_f<T>(v[0]);
    }
  }
};

// what one thread works out for a row from its maximum m, sum s = sum exp(z - m)
// and logit za: the log-probability, the gradient's coefficient g and the three sums
struct PolicyRow {
  double lp, g, loss, kl, clipped;
};
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, int i, float m, float s, float za) {
  PolicyRow r;
  r.lp = ((double)za - (double)m) - log((double)s);
  r.g = r.loss = r.kl = r.clipped = 0.0;
  if (a.weights) {
    const double w = a.weights[i], A = a.adv[i], ratio = exp(r.lp - (double)a.lp_old[i]);
    const double plain = ratio * A;
    const double capped = fmin(fmax(ratio, 1.0 - (double)a.clip_lo), 1.0 + (double)a.clip_hi) * A;
    const bool kept = plain <= capped;
    const double d = a.lp_ref ? (double)a.lp_ref[i] - r.lp : 0.0, e = exp(d);
    const double k = e - d - 1.0;
    r.g = w * ((double)a.beta * (1.0 - e) - (kept ? plain : 0.0));
    r.loss = w * ((double)a.beta * k - (kept ? plain : capped));
    r.kl = w * k;
    r.clipped = kept ? 0.0 : w;
  }
  return r;
}

template <class T, int VEC>
__global__ void __launch_bounds__(POL_THREADS)
    policy_rows_kernel(const T* logits, T* dlogits, PolicyArgs a) {
  __shared__ float sm[POL_WARPS], ss[POL_WARPS];
  __shared__ float s_g, s_inv, s_m;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  double loss = 0.0, kl = 0.0, clipped = 0.0;  // thread 0
  for (int i = blockIdx.x; i < a.rows; i += gridDim.x) {
    const T* z = logits + (long long)i * a.ld;
    T* dz = dlogits ? dlogits + (long long)i * a.ldd : nullptr;
    const int nv = a.V / VEC * VEC;
    const int y = a.actions[i];
    const bool y_ok = y >= 0 && y < a.V;  // an out-of-range action is reported, never read
    const bool live = !a.weights || a.weights[i] != 0.f;
    if (!live || !y_ok) {
      if (tid == 0) {
        if (live) record_error(ERRW_BAD_TARGET);
        a.logp[i] = 0.f;
      }
      if (dz) {
        const float zero[VEC] = {};
        for (int c = tid * VEC; c < nv; c += POL_THREADS * VEC) PolVec<T, VEC>::store(dz + c, zero);
        for (int c = nv + tid; c < a.V; c += POL_THREADS) dz[c] = from_f<T>(0.f);
      }
      continue;
    }
    const float za = to_f(z[y]);
    float m = -INFINITY, s = 0.f;
    for (int c = tid * VEC; c < nv; c += POL_THREADS * VEC) {
      float v[VEC];
      PolVec<T, VEC>::load(z + c, v);
      float mx = v[0];
#pragma unroll
      for (int k = 1; k < VEC; ++k) mx = fmaxf(mx, v[k]);
      const float mn = fmaxf(m, mx);
      float acc = (m == -INFINITY) ? 0.f : s * fast_exp2((m - mn) * LOG2E);
      const float mu = (mn == -INFINITY) ? 0.f : mn;
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc += fast_exp2((v[k] - mu) * LOG2E);
      m = mn;
      s = acc;
    }
    for (int c = nv + tid; c < a.V; c += POL_THREADS) {
      const float v = to_f(z[c]);
      lse_combine(m, s, v, v == -INFINITY ? 0.f : 1.f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      lse_combine(m, s, m2, s2);
    }
    __syncthreads();  // the previous row's s_* and sm/ss are read
    if (lane == 0) {
      sm[warp] = m;
      ss[warp] = s;
    }
    __syncthreads();
    if (tid == 0) {
      float M = sm[0], S = ss[0];
      for (int w = 1; w < POL_WARPS; ++w) lse_combine(M, S, sm[w], ss[w]);
      const PolicyRow r = policy_row(a, i, M, S, za);
      a.logp[i] = (float)r.lp;
      loss += r.loss;
      kl += r.kl;
      clipped += r.clipped;
      s_g = (float)r.g;
      s_inv = (float)(-r.g / (double)S);
      s_m = M;
    }
    if (!dz) continue;
    __syncthreads();
    const float g = s_g, inv = s_inv, mm = s_m;
    for (int c = tid * VEC; c < nv; c += POL_THREADS * VEC) {
      float v[VEC];
      PolVec<T, VEC>::load(z + c, v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        v[k] = fast_exp2((v[k] - mm) * LOG2E) * inv;
        if (c + k == y) v[k] += g;
      }
      PolVec<T, VEC>::store(dz + c, v);
    }
    for (int c = nv + tid; c < a.V; c += POL_THREADS) {
      const float v = fast_exp2((to_f(z[c]) - mm) * LOG2E) * inv;
      dz[c] = from_f<T>(c == y ? v + g : v);
    }
  }
  if (tid == 0 && a.part) {
    a.part[blockIdx.x * 3 + 0] = loss;
    a.part[blockIdx.x * 3 + 1] = kl;
    a.part[blockIdx.x * 3 + 2] = clipped;
  }
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
