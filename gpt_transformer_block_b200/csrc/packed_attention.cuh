// Causal grouped-query attention over packed sequences of different lengths
// (bf16, hd = 128), forward and backward, on the 5th-generation tensor cores.
//
// The rows of all sequences lie one after the other; cu[s] .. cu[s+1]-1 are
// those of sequence s.  Row t of sequence s sees the rows
//   vis(t) = { j : cu[s] <= j <= t and (W < 0 or t - j <= W) }
//   S = q k^T / sqrt(hd), lse = log sum_vis exp S, P = exp(S - lse), o = P v
//   D = rowsum(dO o), dS = P (dO v^T - D) / sqrt(hd)
//   dq = dS k, dk = sum over the group's heads of dS^T q, dv = ... of P^T dO
//
// Tiles are cut out of the packed rows, not out of the sequences: a tile may
// hold the end of one sequence and several short ones, each row carries its
// own visible range, and only the tiles that some row sees are visited.  So
// the grid needs neither the lengths nor a plan made from them (they stay on
// the device), and short sequences share tiles instead of padding one each.
// Products with P = 0 are part of the matrix products, and 0 * NaN is NaN.  Rows
// behind the last sequence are zeroed before them; so are, in the backward, rows
// that are not finite, with P or dS made NaN for the pairs that are visible.  V
// does not show itself in time, so in the forward a row whose result is not
// finite is worked out again from the rows that it sees.
//
// Forward: 128 queries of one head per CTA over 64-key tiles, two CTAs per SM.
// Backward: the schedule of attention_tc.cuh, 128 keys of one kv head per CTA
// over 64-query tiles; D, and the zeroing of the fp32 dQ sums, in a pass of its
// own before, the rounding of dQ to bf16 in one after.
#pragma once
#include "attention_tc.cuh"
#include "common.cuh"

namespace gptb {

// rows that belong to sequences, inside the arrays whatever cu holds
__device__ __forceinline__ int packed_rows(const int32_t* __restrict__ cu, int n_seq, int total) {
  return max(0, min(cu[n_seq], total));
}

// first row and end of the sequence that holds row t < n_rows (found by
// bisection; t itself lies inside the result whatever cu holds)
__device__ __forceinline__ int2 packed_seq(const int32_t* __restrict__ cu, int n_seq, int t, int n_rows) {
  int lo = 0, hi = n_seq;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return make_int2(max(0, min(cu[lo], t)), min(max(cu[hi], t + 1), n_rows));
}

// offsets that are not 0 = cu[0] <= cu[1] <= ... <= total are reported (one CTA calls this)
__device__ __forceinline__ void packed_check(const int32_t* __restrict__ cu, int n_seq, int total) {
  for (int s = threadIdx.x; s <= n_seq; s += blockDim.x) {
    const int c = cu[s];
    if ((s == 0 && c != 0) || (s > 0 && cu[s - 1] > c) || c > total) record_error(ERRW_BAD_OFFSETS);
  }
}

// one row (two 128-byte halves `half` bytes apart) of a swizzled tile
__device__ __forceinline__ void zero_tile_row(uint8_t* tile, int half, int r) {
#pragma unroll
  for (int c = 0; c < 16; ++c)
    *reinterpret_cast<uint4*>(tile + (c >> 3) * half + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
}

// q, k and v as rows, for what the tensor cores cannot be asked
struct PackedRows {
  const bf16 *q, *k, *v;
  long long ldq, ldk, ldv;
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The rows of `again` (a bit per lane; the lane has row row0 + lane's first
// visible key, maximum and inverse sum) once more, by the warp from the rows
// that they see: o = sum of exp2(s - m) inv v, s in base 2, 4 columns per lane.
// In the columns that are not finite at `at` (row 0, `pitch` bytes from row to
// row; or, pitch 0, the swizzled tile), and for a row that sees many keys only in
// those in which a V row is not finite that its tiles hold (v_first .. v_last)
// and it does not see: else one NaN early in a long sequence would send all the
// rows that do see it through here (8192 rows of 12 heads: 49 ms).  From the
// newest key back, until none of those columns is finite any more: nothing makes
// them so again.
constexpr int PF_ALONE = 1024;  // keys
__device__ __noinline__ void packed_rows_alone(unsigned again, int row0, int kv_lo, float m_used, float inv_l, int v_first,
                                               int v_last, const bf16* q, long long ldq, const bf16* k, long long ldk,
                                               const bf16* v, long long ldv, uint8_t* at0, long long pitch) {
  const int lane = threadIdx.x & 31, c = lane * 4;
  const auto four = [](const uint2& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xffff0000u);
  };
  const auto load4 = [&](const bf16* p, float (&x)[4]) { four(*reinterpret_cast<const uint2*>(p + c), x); };
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int x = __ffs(again) - 1, t = row0 + x;
    const int lo = __shfl_sync(0xffffffffu, kv_lo, x);
    const float m = __shfl_sync(0xffffffffu, m_used, x), inv = __shfl_sync(0xffffffffu, inv_l, x);
    uint2* at = reinterpret_cast<uint2*>(
        pitch ? at0 + x * pitch + lane * 8
              : at0 + (lane >> 4) * 16384 + x * 128 + ((((lane & 15) >> 1) ^ (x & 7)) << 4) + (lane & 1) * 8);
    float old[4], a[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, foreign[4] = {0.f, 0.f, 0.f, 0.f};
    four(*at, old);
    const int before = max(0, lo - v_first), unseen = before + v_last - t;
    if (t - lo < max(unseen, PF_ALONE)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) foreign[i] = INFINITY;
    } else {  // (0 * x is NaN where x is not finite)
#pragma unroll 4
      for (int i = 0; i < unseen; ++i) {
        float y[4];
        load4(v + (long long)(i < before ? v_first + i : t + 1 + i - before) * ldv, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) foreign[e] = fmaf(0.f, y[e], foreign[e]);
      }
    }
    bool want[4], open = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) open |= want[i] = !finite(old[i]) && foreign[i] != 0.f;
    load4(q + t * ldq, a);
#pragma unroll 1
    for (int j0 = t; j0 >= lo && __any_sync(0xffffffffu, open); j0 -= 4) {
      float s[4], y[4][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const long long j = max(j0 - e, lo);
        float b[4];
        load4(k + j * ldk, b);
        load4(v + j * ldv, y[e]);
        s[e] = fmaf(a[0], b[0], fmaf(a[1], b[1], fmaf(a[2], b[2], a[3] * b[3])));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] = warp_sum(s[e]);
        if (j0 - e < lo) continue;
        const float p = fast_exp2(fmaf(s[e], LOG2E / sqrtf(128.f), -m)) * inv;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(p, y[e][i], acc[i]);
      }
      open = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) open |= want[i] && finite(acc[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) old[i] = want[i] ? acc[i] : old[i];
    *at = make_uint2(pack_bf16(old[0], old[1]), pack_bf16(old[2], old[3]));
  }
}

// Forward.  CTA = 128 consecutive packed rows of one head, two CTAs per SM, 6
// warps: 0 TMA producer (Q once; K and V tiles of 64 keys, two stages each), 1
// TMEM owner and MMA issuer, 2-5 softmax (thread = query row, its TMEM lane).
// S = Q K^T of tile i in TMEM columns 64 (i % 2) .., P (bf16 pairs) over the
// first half of it, O in columns 128-255.  S of tile i+1 is issued before PV of
// tile i, so the softmax warps find the next scores ready and the tensor core
// works while they do.  O is rescaled only when a
// row's running maximum grows by more than 8 in base 2 (P stays below 256 in
// bf16, and the normalisation uses the same maximum, so the result is exact).
// What bounds it: the softmax (its exponentials alone take half of the time on
// their unit), and the start and end of a CTA, which the other CTA of the SM
// fills.  One sequence of 8192 rows, 12 heads: 205 us, 24 ragged ones (30 to 2000
// rows, 10 heads, window 1024): 65 us.  With 128-key tiles, and so no room for a
// second S, 204 and 73: the long sequence gains nothing by it, the ragged ones
// do.  As one CTA of two query tiles per SM (attention_tc.cuh) 220 and 84.  (All
// on one GPU; the long sequence takes up to 235 us on others, or where the power
// cap holds the clock lower.)
constexpr int PF_THREADS = 192;
constexpr int PF_BN = 64;
constexpr int PF_LONG = 32;                                // key tiles, 2048 keys
constexpr int PF_KV = PF_BN * 128 * 2;                     // one K or V tile: two 64-column swizzled halves of 8 KB
constexpr int PF_SMEM = 1024 + FA_TILE /*Q*/ + 4 * PF_KV;  // K, V x2

__global__ void __launch_bounds__(PF_THREADS, 2)
    packed_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                           const PackedRows in, bf16* __restrict__ o, long long ldo, float* __restrict__ lse,
                           const int32_t* __restrict__ cu, int n_seq, int total, int H, int Hkv, int window) {
  extern __shared__ uint8_t fa_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(fa_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + FA_TILE;    // 2 stages
  uint8_t* sV = sK + 2 * PF_KV;  // 2 stages
  __shared__ __align__(8) uint64_t bars[16];
  uint64_t* q_full = bars + 0;
  uint64_t* k_full = bars + 1;   // [2 stages]
  uint64_t* k_empty = bars + 3;  // [2 stages]
  uint64_t* v_full = bars + 5;   // [2 stages]
  uint64_t* v_empty = bars + 7;  // [2 stages]
  uint64_t* s_full = bars + 9;   // [2 score tiles]
  uint64_t* p_full = bars + 11;  // [2 score tiles] one arrival per softmax warp
  uint64_t* o_done = bars + 13;  // [2 score tiles] O += P V done (one barrier for all would be a phase behind or
                                 // two: PV of the tile before may still run when a softmax ends)
  uint64_t* drain = bars + 15;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  __shared__ int s_lo;  // first visible row of the tile's first query
  volatile int* abort_flag = &s_abort;

  // the last rows first: the end of a long sequence is its heaviest part
  const int nqb = (total + FA_BM - 1) / FA_BM;
  const int qb = nqb - 1 - (int)blockIdx.x / H;
  const int h = (int)blockIdx.x % H;
  const int kvh = h / (H / Hkv);
  const int q0 = qb * FA_BM;
  const int n_rows = packed_rows(cu, n_seq, total);
  if (blockIdx.x == 0) packed_check(cu, n_seq, total);
  if (q0 >= n_rows) return;  // (the whole CTA: rows behind the last sequence)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(drain, 1);
    s_abort = 0;
    fence_mbar_init();
    // (Q needs no lookup)
    mbar_arrive_expect_tx(q_full, FA_TILE);
    tma_load_2d(sQ, &tm_q, q_full, h * 128, q0);
    tma_load_2d(sQ + 16384, &tm_q, q_full, h * 128 + 64, q0);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, 256);
  // a softmax thread's query row sees the packed rows kv_lo .. kv_hi
  int tq = 0, kv_lo = 0, kv_hi = -1;
  if (warp >= 2) {
    tq = q0 + (warp & 3) * 32 + lane;
    if (tq < n_rows) {
      kv_lo = packed_seq(cu, n_seq, tq, n_rows).x;
      if (window >= 0) kv_lo = max(kv_lo, tq - window);
      kv_hi = tq;
    }
    if (tq == q0) s_lo = kv_lo;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int jlo = s_lo / PF_BN, jhi = min(q0 + FA_BM - 1, n_rows - 1) / PF_BN;
  const int n = jhi - jlo + 1;  // key tiles

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < n; ++i) {
        const int st = i & 1, kr = (jlo + i) * PF_BN;
        const uint32_t par = ((i >> 1) & 1) ^ 1u;
        uint8_t *k = sK + st * PF_KV, *v = sV + st * PF_KV;
        if (!mbar_wait(&k_empty[st], par, abort_flag, ERRW_TIMEOUT_PRODUCER)) break;
        mbar_arrive_expect_tx(&k_full[st], PF_KV);
        tma_load_2d(k, &tm_k, &k_full[st], kvh * 128, kr);
        tma_load_2d(k + 8192, &tm_k, &k_full[st], kvh * 128 + 64, kr);
        if (!mbar_wait(&v_empty[st], par, abort_flag, ERRW_TIMEOUT_PRODUCER)) break;
        mbar_arrive_expect_tx(&v_full[st], PF_KV);
        tma_load_2d(v, &tm_v, &v_full[st], kvh * 128, kr);
        tma_load_2d(v + 8192, &tm_v, &v_full[st], kvh * 128 + 64, kr);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t IDESC_S = make_idesc(128, PF_BN, false, false, false);
      constexpr uint32_t IDESC_O = make_idesc(128, 128, false, true, false);
      const uint32_t aQ = smem_u32(sQ);
      bool ok = mbar_wait(q_full, 0, abort_flag, ERRW_TIMEOUT_MMA);
      for (int i = 0; ok && i <= n; ++i) {
        if (i < n) {  // S of tile i
          const int st = i & 1;
          const uint32_t aK = smem_u32(sK + st * PF_KV);
          if (!mbar_wait(&k_full[st], (i >> 1) & 1, abort_flag, ERRW_TIMEOUT_MMA)) break;
          // it overwrites P of tile i - 2: products of different shapes may
          // overlap, so the one that reads it has to be done
          if (i >= 2 && !mbar_wait(&o_done[st], ((i >> 1) - 1) & 1, abort_flag, ERRW_TIMEOUT_MMA)) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss(tmem + st * PF_BN, fa_desc_k(aQ, k),
                        smem_desc_sw128(aK + (uint32_t)((k >> 2) * 8192 + (k & 3) * 32), 16, 1024), IDESC_S, k > 0 ? 1u : 0u);
          mma_commit(&s_full[st]);
          mma_commit(&k_empty[st]);
        }
        if (i > 0) {  // O += P V of tile i - 1, P read from TMEM
          const int st = (i - 1) & 1;
          const uint32_t par = ((i - 1) >> 1) & 1, aV = smem_u32(sV + st * PF_KV);
          if (!mbar_wait(&v_full[st], par, abort_flag, ERRW_TIMEOUT_MMA) ||
              !mbar_wait(&p_full[st], par, abort_flag, ERRW_TIMEOUT_MMA))
            break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ts(tmem + 128, tmem + st * PF_BN + k * 8, smem_desc_sw128(aV + (uint32_t)(k * 2048), 8192, 1024),
                        IDESC_O, (i > 1 || k > 0) ? 1u : 0u);
          mma_commit(&v_empty[st]);
          mma_commit(&o_done[st]);
        }
      }
      if (*abort_flag) {
        mma_commit(drain);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0))
          if (globaltimer_ns() - t0 > 100000000ull) { record_error(ERRW_TIMEOUT_DRAIN); break; }
      }
    }
  } else {
    const int qw = warp & 3;       // TMEM lane quarter
    const int r = qw * 32 + lane;  // row within the query tile
    const uint32_t lane_addr = tmem + ((uint32_t)(qw * 32) << 16);
    const float sl2 = LOG2E / sqrtf(128.f);
    const int lo = s_lo;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      const int k0 = (jlo + c) * PF_BN, st = c & 1;
      const uint32_t s_addr = lane_addr + st * PF_BN;
      ok = mbar_wait_warp(&s_full[st], (c >> 1) & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE);
      if (!ok) break;
      tc_fence_after();
      uint32_t v[64];
#pragma unroll
      for (int k = 0; k < 2; ++k) tmem_ld_32x32b_x32(s_addr + k * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[k * 32]));
      tmem_ld_wait();
      // rows are masked in a tile that reaches past the first query, or
      // before what the last one sees (kv_lo grows with the row)
      if (__any_sync(0xffffffffu, k0 < kv_lo || k0 + PF_BN - 1 > kv_hi)) {
#pragma unroll
        for (int i = 0; i < PF_BN; ++i) {
          const int jk = k0 + i;
          v[i] = (jk >= kv_lo && jk <= kv_hi) ? v[i] : __float_as_uint(-INFINITY);
        }
      }
      float mp[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) mp[i] = __uint_as_float(v[i]);
#pragma unroll
      for (int i = 8; i < 56; i += 16) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mp[k] = fmax3(mp[k], __uint_as_float(v[i + k]), __uint_as_float(v[i + 8 + k]));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) mp[k] = fmaxf(mp[k], __uint_as_float(v[56 + k]));
      const float mx = fmax3(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7])) * sl2;
      // the running max moves only when it grows by more than 8 (base 2)
      const bool grow = mx > m_used + 8.f;
      const float corr = grow ? fast_exp2(m_used - mx) : 1.f;  // 0 when m_used is -inf
      if (grow) {
        l *= corr;
        m_used = mx;
      }
      const float mu = (m_used == -INFINITY) ? 0.f : m_used;
      // P = exp2(s*scale - m) as bf16 pairs (key 2c in the low half)
      const f32x2 sl2_2 = f2_pack(sl2, sl2), mu_2 = f2_pack(-mu, -mu);
      f32x2 lp[2] = {0, 0};
#pragma unroll
      for (int hq = 0; hq < 2; ++hq) {  // 32 keys (16 columns of P) at a time
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int i = hq * 32 + 2 * e;
          float p0, p1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sl2_2, mu_2), p0, p1);
          p0 = fast_exp2(p0);  // exp2(-inf) = 0 for masked keys
          p1 = fast_exp2(p1);
          lp[e & 1] = f2_add(lp[e & 1], f2_pack(p0, p1));
          pk[e] = pack_bf16(p0, p1);
        }
        tmem_st_32x32b_x16(s_addr + hq * 16, pk);
      }
      float l0, l1;
      f2_unpack(f2_add(lp[0], lp[1]), l0, l1);
      l += l0 + l1;
      // V rows that no query of this CTA sees may hold anything (0 * NaN is NaN).
      // Those behind the last sequence are zeroed before the product that reads
      // them, those before the first query's range where a CTA has many key
      // tiles: else a NaN before a long sequence would send all of it through
      // packed_rows_alone().  (For few tiles that is cheap, and the zeroing
      // is not: 512 sequences of 24 rows, 12 heads, 50 us with it, 47 without.)
      if ((n_rows < total && k0 + PF_BN > n_rows) || (n > PF_LONG && k0 < lo)) {
        ok = mbar_wait_warp(&v_full[st], (c >> 1) & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE);
        if (!ok) break;
        if (r < PF_BN && (k0 + r >= n_rows || k0 + r < lo)) zero_tile_row(sV + st * PF_KV, 8192, r);
        fence_proxy_async_smem();
      }
      // O to the new max, once it holds every PV product up to tile c-1 (the
      // TMEM accesses are warp-collective: the whole warp enters, rows that keep
      // their max use 1)
      if (c > 0 && __any_sync(0xffffffffu, grow)) {
        ok = mbar_wait_warp(&o_done[st ^ 1], ((c - 1) >> 1) & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t w[32];
          tmem_ld_32x32b_x32(lane_addr + 128 + k * 32, w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * corr);
          tmem_st_32x32b_x32(lane_addr + 128 + k * 32, w);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[st]);
    }
    if (__all_sync(0xffffffffu, ok) && mbar_wait_warp(&o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag,
                                                       ERRW_TIMEOUT_EPILOGUE)) {
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      // O (bf16) leaves through the Q tile, free once every S product has
      // completed (they precede the last PV that o_done follows): two 64-column
      // halves of 128 rows x 128 bytes, 128-byte swizzle; a warp whose 32 rows
      // all lie inside the sequences stores them with two TMA boxes, the last
      // rows go out one by one
      const int row0 = q0 + qw * 32;  // first query of this warp's rows
      const bool whole = row0 + 32 <= n_rows;
      f32x2 all = 0;  // the sum of the row's O: finite unless one of them is not (or they are as large as that)
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // columns 32k .. 32k+31
        uint32_t w[32];
        tmem_ld_32x32b_x32(lane_addr + 128 + k * 32, w);
        tmem_ld_wait();
        uint8_t* row = sQ + (k >> 1) * 16384 + r * 128;
#pragma unroll
        for (int i = 0; i < 32; i += 2) all = f2_add(all, f2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1])));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint4 u;
          u.x = pack_bf16(__uint_as_float(w[g * 8 + 0]) * inv, __uint_as_float(w[g * 8 + 1]) * inv);
          u.y = pack_bf16(__uint_as_float(w[g * 8 + 2]) * inv, __uint_as_float(w[g * 8 + 3]) * inv);
          u.z = pack_bf16(__uint_as_float(w[g * 8 + 4]) * inv, __uint_as_float(w[g * 8 + 5]) * inv);
          u.w = pack_bf16(__uint_as_float(w[g * 8 + 6]) * inv, __uint_as_float(w[g * 8 + 7]) * inv);
          const int cg = (k & 1) * 4 + g;  // 16-byte chunk within the 128-byte half row
          if (whole)
            *reinterpret_cast<uint4*>(row + ((cg ^ (r & 7)) << 4)) = u;
          else if (tq < n_rows)
            *reinterpret_cast<uint4*>(o + (long long)tq * ldo + h * 128 + k * 32 + g * 8) = u;
        }
      }
      // A row whose o is not finite, though its sum is, may owe that to rows it
      // does not see (P = 0 there, and 0 * NaN is NaN), so it is worked out again
      // from those that it sees
      float a0, a1;
      f2_unpack(all, a0, a1);
      __syncwarp();
      const unsigned again = __ballot_sync(0xffffffffu, tq < n_rows && l > 0.f && finite(l) && !finite(a0 + a1));
      if (again)
        packed_rows_alone(again, row0, kv_lo, m_used, inv, n > PF_LONG ? lo : jlo * PF_BN, min(q0 + FA_BM, n_rows) - 1, in.q + h * 128, in.ldq, in.k + kvh * 128, in.ldk, in.v + kvh * 128,
                          in.ldv, whole ? sQ + qw * 4096 : reinterpret_cast<uint8_t*>(o + row0 * ldo + h * 128),
                          whole ? 0 : ldo * 2);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && whole) {
        tma_store_2d(&tm_o, sQ + qw * 4096, h * 128, row0);
        tma_store_2d(&tm_o, sQ + 16384 + qw * 4096, h * 128 + 64, row0);
        bulk_commit_group();
        bulk_wait_read0();  // the tile's shared memory is read before the CTA ends
      }
      __syncwarp();
      if (tq < n_rows) lse[(long long)h * total + tq] = (m_used + log2f(l)) * LN2;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// zeroes the Q and dO rows of a stage whose LSE is not finite (out of the way of the loop that calls it)
__device__ __noinline__ void packed_zero_odd(uint8_t* q, uint8_t* dO, const float* lse) {
#pragma unroll 1
  for (int r = 0; r < AB2_BQ; ++r) {
    if (finite(lse[r])) continue;
    zero_tile_row(q, 8192, r);
    zero_tile_row(dO, 8192, r);
  }
  fence_proxy_async_smem();
}

// Backward.  Roles, TMEM columns and barriers as in attn_bwd_tc_kernel: 128
// keys of one kv head per CTA, a chain of steps of one query head and 64
// queries each.  A chain costs 10 us to start and end and 2 us per step, so
// where there are fewer chains than SMs a cluster of up to 8 CTAs shares each:
// every CTA takes a part of its steps, and the partial dK and dV meet through
// distributed shared memory, added in a fixed order (5 sequences of 12 to 180
// tokens, 8 query heads over 2: 47 us with one CTA per chain, 30 with 8).
//
// A query whose LSE or D is not finite (its q or dout is not, or a k or v that
// it sees) has P and dS of NaN where it sees a key: the producer makes its LSE
// NaN, and the MMA warp zeroes its Q and dO rows before the products in which
// they would meet the zeros of other keys.  A key whose row of K is not finite
// is found by the dQ warps while they wait for the first step: they zero the row
// and make that of V NaN, so that dS is NaN where a query sees the key.  None of
// this is on the softmax warps' way: with the checks there, 20 sequences of 200
// to 2048 rows take 575 us (forward and backward), so 541, and 535 without them.
constexpr int PB_CLUSTER = 8;
__global__ void __launch_bounds__(AB2_THREADS, 1)
    packed_attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                           const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                           bf16* __restrict__ dk, long long lddk, bf16* __restrict__ dv, long long lddv,
                           const float* __restrict__ lse, const float* __restrict__ Dd, float* __restrict__ dq,
                           const int32_t* __restrict__ cu, int n_seq, int total, int H, int Hkv, int window, int cs) {
  extern __shared__ uint8_t ab_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ab_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + AB2_KV_TILE;
  uint8_t* sQ = sV + AB2_KV_TILE;                  // AB2_STAGES stages
  uint8_t* sDO = sQ + AB2_STAGES * AB2_Q_TILE;     // AB2_STAGES stages
  uint8_t* sDS = sDO + AB2_STAGES * AB2_Q_TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sDS + AB2_PS_TILE);
  uint64_t* kv_full = bars + 0;
  uint64_t* qdo_full = bars + 1;                 // [AB2_STAGES] TMA bytes + one arrival after LSE / D are stored
  uint64_t* qdo_empty = bars + 1 + AB2_STAGES;   // [AB2_STAGES]
  uint64_t* s_full = bars + 1 + 2 * AB2_STAGES;
  uint64_t* s_empty = s_full + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* ds_free = s_full + 3;
  uint64_t* dq_full = s_full + 4;
  uint64_t* dq_free = s_full + 5;
  uint64_t* acc_done = s_full + 6;
  uint64_t* drain = s_full + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sLD = reinterpret_cast<float*>(bars + 32);  // [AB2_STAGES][lse*log2e 64 | D 64]

  __shared__ int s_vis[2];  // last query that sees the tile's first key; ... its last key
  __shared__ int s_odd[AB2_STAGES];  // the stage has a query whose LSE or D is not finite

  const int rank = (int)blockIdx.x % cs, chain = (int)blockIdx.x / cs;
  const int kb = chain / Hkv, kvh = chain % Hkv;
  const int G = H / Hkv;
  const int k0 = kb * AB2_BK;
  const int n_rows = packed_rows(cu, n_seq, total);
  if (k0 >= n_rows) return;  // (the whole CTA: rows behind the last sequence)
  const long long lddq = (long long)H * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int i = 0; i < AB2_STAGES; ++i) {
      mbar_init(&qdo_full[i], 2);
      mbar_init(&qdo_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_empty, 8);
    mbar_init(p_full, 8);
    mbar_init(ds_free, 1);
    mbar_init(dq_full, 1);
    mbar_init(dq_free, 8);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_dk);
    tma_prefetch_desc(&tm_dv);
    // K and V, and where the chain has one CTA the first step's Q and dO: they
    // need no lookup
    mbar_arrive_expect_tx(kv_full, 2 * AB2_KV_TILE);
    tma_load_2d(sK, &tm_k, kv_full, kvh * 128, k0);
    tma_load_2d(sK + 16384, &tm_k, kv_full, kvh * 128 + 64, k0);
    tma_load_2d(sV, &tm_v, kv_full, kvh * 128, k0);
    tma_load_2d(sV + 16384, &tm_v, kv_full, kvh * 128 + 64, k0);
    if (cs == 1) {
      const int hh = kvh * G, q0 = k0;
      mbar_arrive_expect_tx(&qdo_full[0], 2 * AB2_Q_TILE);
      tma_load_2d(sQ, &tm_q, &qdo_full[0], hh * 128, q0);
      tma_load_2d(sQ + 8192, &tm_q, &qdo_full[0], hh * 128 + 64, q0);
      tma_load_2d(sDO, &tm_do, &qdo_full[0], hh * 128, q0);
      tma_load_2d(sDO + 8192, &tm_do, &qdo_full[0], hh * 128 + 64, q0);
    }
  }
  // queries that see a softmax thread's key: [key, key + W] inside its sequence
  int q_vis_hi = -1;
  if (warp >= 2 && warp < 10) {
    const int r = (warp & 3) * 32 + lane, key = k0 + r;
    if (key < n_rows) {
      q_vis_hi = packed_seq(cu, n_seq, key, n_rows).y - 1;
      if (window >= 0) q_vis_hi = min(q_vis_hi, key + min(window, total));
    }
    if (r == 0) s_vis[0] = q_vis_hi;
    if (key == min(k0 + AB2_BK, n_rows) - 1) s_vis[1] = q_vis_hi;
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch();
  pdl_wait();  // (D, and the dQ sums set to 0)
  const int q_first = s_vis[0];
  const int qt_lo = k0 / AB2_BQ;
  const int nq = s_vis[1] / AB2_BQ - qt_lo + 1;
  // this CTA's steps: first .. first + steps - 1 of the chain's
  const int first = (int)((long long)G * nq * rank / cs);
  const int steps = (int)((long long)G * nq * (rank + 1) / cs) - first;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    for (int i = 0; i < steps && ok; ++i) {
      const int st = i % AB2_STAGES;
      const int hh = kvh * G + (first + i) / nq;
      const int q0 = (qt_lo + (first + i) % nq) * AB2_BQ;
      ok = mbar_wait_warp(&qdo_empty[st], ((i / AB2_STAGES) & 1) ^ 1u, abort_flag, ERRW_TIMEOUT_PRODUCER);
      if (!ok) break;
      // the tile loads go out first; LSE and D (plain loads, guarded at the
      // sequence end) overlap them and complete the stage with a second arrival
      if (lane == 0 && (i > 0 || cs > 1)) {
        mbar_arrive_expect_tx(&qdo_full[st], 2 * AB2_Q_TILE);
        uint8_t* q = sQ + st * AB2_Q_TILE;
        uint8_t* d = sDO + st * AB2_Q_TILE;
        tma_load_2d(q, &tm_q, &qdo_full[st], hh * 128, q0);
        tma_load_2d(q + 8192, &tm_q, &qdo_full[st], hh * 128 + 64, q0);
        tma_load_2d(d, &tm_do, &qdo_full[st], hh * 128, q0);
        tma_load_2d(d + 8192, &tm_do, &qdo_full[st], hh * 128 + 64, q0);
      }
      float* ld = sLD + st * 128;
      bool odd = false;
      for (int e = lane; e < 64; e += 32) {
        const int t = q0 + e;
        const long long li = (long long)hh * total + t;
        const float l2 = (t < n_rows) ? lse[li] * LOG2E : 0.f, d = (t < n_rows) ? Dd[li] : 0.f;
        const bool here = !(finite(l2) && finite(d));
        ld[e] = here ? NAN : l2;
        ld[64 + e] = d;
        odd |= here;
      }
      odd = __any_sync(0xffffffffu, odd);
      if (lane == 0) s_odd[st] = odd;
      if (lane == 0) mbar_arrive(&qdo_full[st]);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t ID_S = make_idesc(128, 64, false, false, false);   // S^T, dP^T
      constexpr uint32_t ID_G = make_idesc(128, 128, false, true, false);   // dV, dK (A from TMEM)
      constexpr uint32_t ID_Q = make_idesc(128, 64, true, true, false);     // dQ^T
      const uint32_t aK = smem_u32(sK), aV = smem_u32(sV), aDS = smem_u32(sDS);
      bool ok = mbar_wait(kv_full, 0, abort_flag, ERRW_TIMEOUT_MMA);
      auto grads = [&](int i) -> bool {
        const int st = i % AB2_STAGES;
        const int odd = s_odd[st];
        if (!mbar_wait(p_full, i & 1, abort_flag, ERRW_TIMEOUT_MMA)) return false;
        if (odd) packed_zero_odd(sQ + st * AB2_Q_TILE, sDO + st * AB2_Q_TILE, sLD + st * 128);
        tc_fence_after();
        const uint32_t aQ = smem_u32(sQ + st * AB2_Q_TILE), aDO = smem_u32(sDO + st * AB2_Q_TILE);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t acc = (i > 0 || k > 0) ? 1u : 0u;
          // A: P^T / dS^T in TMEM (lane = key, 8 columns per 16 queries)
          // B: dO / Q as MN-major (hd halves 8 KB apart), K step = 16 query rows
          mma_bf16_ts(tmem + 128, tmem + 448 + k * 8, smem_desc_sw128(aDO + k * 2048, 8192, 1024), ID_G, acc);
          mma_bf16_ts(tmem + 0, tmem + 480 + k * 8, smem_desc_sw128(aQ + k * 2048, 8192, 1024), ID_G, acc);
        }
        if (!mbar_wait(dq_free, i & 1, abort_flag, ERRW_TIMEOUT_MMA)) return false;  // (its first phase: K is in order)
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          // A = K^T (MN-major over hd, halves 16 KB apart), B = dS (MN-major over queries), K step = 16 keys
          mma_bf16_ss(tmem + 384, smem_desc_sw128(aK + k * 2048, 16384, 1024),
                      smem_desc_sw128(aDS + k * 2048, 8192, 1024), ID_Q, k > 0 ? 1u : 0u);
        }
        mma_commit(ds_free);
        mma_commit(&qdo_empty[st]);
        mma_commit(dq_full);
        return true;
      };
      for (int i = 0; ok && i < steps; ++i) {
        const int st = i % AB2_STAGES;
        if (!mbar_wait(&qdo_full[st], (i / AB2_STAGES) & 1, abort_flag, ERRW_TIMEOUT_MMA)) { ok = false; break; }
        if (!mbar_wait(s_empty, (i & 1) ^ 1u, abort_flag, ERRW_TIMEOUT_MMA)) { ok = false; break; }
        tc_fence_after();
        const uint32_t aQ = smem_u32(sQ + st * AB2_Q_TILE), aDO = smem_u32(sDO + st * AB2_Q_TILE);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          // K-major over hd: A rows = keys (halves 16 KB apart), B rows = queries (halves 8 KB apart)
          const uint32_t ka = (uint32_t)((k >> 2) * 16384 + (k & 3) * 32), kq = (uint32_t)((k >> 2) * 8192 + (k & 3) * 32);
          mma_bf16_ss(tmem + 256, smem_desc_sw128(aK + ka, 16, 1024), smem_desc_sw128(aQ + kq, 16, 1024), ID_S, k > 0);
          mma_bf16_ss(tmem + 320, smem_desc_sw128(aV + ka, 16, 1024), smem_desc_sw128(aDO + kq, 16, 1024), ID_S, k > 0);
        }
        mma_commit(s_full);
        if (i > 0 && !grads(i - 1)) { ok = false; break; }
      }
      if (ok && steps > 0) ok = grads(steps - 1);
      if (ok && steps == 0) mbar_arrive(acc_done);  // (nothing to wait for)
      else mma_commit(acc_done);
      if (*abort_flag) {
        mma_commit(drain);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0))
          if (globaltimer_ns() - t0 > 100000000ull) { record_error(ERRW_TIMEOUT_DRAIN); break; }
      }
    }
  } else if (warp < 10) {
    // ---------------------------------------------------- softmax backward
    const int qw = warp & 3;
    const int cb = (warp - 2) >> 2;          // queries cb*32 .. cb*32+31 of the tile
    const int r = qw * 32 + lane;            // key row within the tile
    const int key = k0 + r;
    const uint32_t lane_addr = tmem + ((uint32_t)(qw * 32) << 16);
    const float scale = rsqrtf(128.f);
    const float sl2 = LOG2E * scale;
    bool ok = true;
    for (int i = 0; i < steps && ok; ++i) {
      const int st = i % AB2_STAGES;
      const int q0 = (qt_lo + (first + i) % nq) * AB2_BQ;
      ok = mbar_wait_warp(s_full, i & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE);
      if (!ok) break;
      tc_fence_after();
      const int tq = q0 + cb * 32;  // first query of this warp's columns
      const bool need_mask = (k0 + AB2_BK - 1 > tq) || (tq + 31 > q_first) || (k0 + AB2_BK > n_rows);
      const float4* l2v = reinterpret_cast<const float4*>(sLD + st * 128 + cb * 32);
      const float4* ddv = reinterpret_cast<const float4*>(sLD + st * 128 + 64 + cb * 32);
      // P^T and dS^T for this warp's 32 queries, packed to bf16 pairs (query
      // 2j in the low half); S^T and dP^T come in with one TMEM round trip
      uint32_t pu[16], du[16];
      {
        uint32_t sv[32], dvv[32];
        tmem_ld_32x32b_x32(lane_addr + 256 + cb * 32, sv);
        tmem_ld_32x32b_x32(lane_addr + 320 + cb * 32, dvv);
        tmem_ld_wait();
        // S^T / dP^T are in registers: the next step's products may overwrite them
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 a = l2v[g], d = ddv[g];
          const float l2[4] = {a.x, a.y, a.z, a.w}, dd[4] = {d.x, d.y, d.z, d.w};
          float pe[4], de[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = tq + g * 4 + e;
            const bool vis = !need_mask || (t >= key && t <= q_vis_hi);
            pe[e] = vis ? fast_exp2(fmaf(__uint_as_float(sv[g * 4 + e]), sl2, -l2[e])) : 0.f;
            de[e] = vis ? pe[e] * (__uint_as_float(dvv[g * 4 + e]) - dd[e]) * scale : 0.f;
          }
          pu[g * 2] = pack_bf16(pe[0], pe[1]);
          pu[g * 2 + 1] = pack_bf16(pe[2], pe[3]);
          du[g * 2] = pack_bf16(de[0], de[1]);
          du[g * 2 + 1] = pack_bf16(de[2], de[3]);
        }
      }
      // the previous step's dV/dK/dQ MMAs must be done reading P^T / dS^T
      if (i > 0) {
        ok = mbar_wait_warp(ds_free, (i - 1) & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE);
        if (!ok) break;
        tc_fence_after();
      }
      tmem_st_32x32b_x16(lane_addr + 448 + cb * 16, pu);
      tmem_st_32x32b_x16(lane_addr + 480 + cb * 16, du);
      // rows behind the last sequence may hold anything (0 * NaN is NaN): the
      // K rows (read by dQ), Q rows (dK) and dO rows (dV) of this tile that lie
      // there are zeroed before the products that read them.  S^T and dP^T of
      // these rows and columns are masked, whatever they were computed from.
      if (n_rows < total) {
        if (i == 0 && cb == 0 && key >= n_rows) zero_tile_row(sK, 16384, r);
        if (cb == 1 && r < AB2_BQ && q0 + r >= n_rows) {
          zero_tile_row(sQ + st * AB2_Q_TILE, 8192, r);
          zero_tile_row(sDO + st * AB2_Q_TILE, 8192, r);
        }
      }
      uint8_t* drow = sDS + r * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int cc = cb * 4 + c;  // 16-byte chunk (8 queries) within the 128-byte row
        *reinterpret_cast<uint4*>(drow + ((cc ^ (r & 7)) << 4)) =
            make_uint4(du[c * 4], du[c * 4 + 1], du[c * 4 + 2], du[c * 4 + 3]);
      }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
    // dK, dV rows (bf16) for this CTA's keys, columns cb*64 .. cb*64+63, through
    // two 32-row x 128-byte swizzled staging tiles per warp in the (now idle) Q/dO ring
    if (__all_sync(0xffffffffu, ok) && mbar_wait_warp(acc_done, 0, abort_flag, ERRW_TIMEOUT_EPILOGUE)) {
      tc_fence_after();
      uint8_t* stg = sQ + (warp - 2) * 2 * 4096;
      const bool whole = k0 + qw * 32 + 32 <= n_rows;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint32_t v0[32], v1[32];
        tmem_ld_32x32b_x32(lane_addr + which * 128 + cb * 64, v0);
        tmem_ld_32x32b_x32(lane_addr + which * 128 + cb * 64 + 32, v1);
        tmem_ld_wait();
        if (cs > 1) {  // this CTA's part in fp32 (0 without a step): rows of 32 16-byte chunks, chunk c at c ^ (row % 32)
          float4* prow = reinterpret_cast<float4*>(sQ) + (which * 128 + r) * 32;
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            const uint32_t* w = g < 8 ? v0 + g * 4 : v1 + (g - 8) * 4;
            prow[(cb * 16 + g) ^ lane] =
                steps > 0 ? make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          continue;
        }
        uint8_t* prow = stg + which * 4096 + lane * 128;
#pragma unroll
        for (int g = 0; g < 8; ++g) {  // 16-byte chunk g: columns 8g .. 8g+7
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c0 = g * 8 + 2 * j;
            const float lo = __uint_as_float(c0 < 32 ? v0[c0] : v1[c0 - 32]);
            const float hi = __uint_as_float(c0 + 1 < 32 ? v0[c0 + 1] : v1[c0 + 1 - 32]);
            w[j] = pack_bf16(lo, hi);
          }
          if (whole)
            *reinterpret_cast<uint4*>(prow + ((g ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          else if (key < n_rows)
            *reinterpret_cast<uint4*>((which ? dv + (long long)key * lddv : dk + (long long)key * lddk) + kvh * 128 +
                                      cb * 64 + g * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && whole && cs == 1) {
        tma_store_2d(&tm_dk, stg, kvh * 128 + cb * 64, k0 + qw * 32);
        tma_store_2d(&tm_dv, stg + 4096, kvh * 128 + cb * 64, k0 + qw * 32);
        bulk_commit_group();
        bulk_wait_read0();  // the staging tiles are read before the CTA ends
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------- dQ epilogue
    // TMEM gives each thread one hd column of dQ^T (64 queries).  A 4x4
    // transpose among each group of 4 lanes (two butterfly stages of
    // shuffles) turns that into 4 consecutive hd values of one query, so one
    // 16-byte fp32 reduction per thread covers 4 rows x 128 bytes per warp:
    // a quarter of the reduction instructions of one-float-per-lane.
    const int qw = warp & 3;
    const int qh = (warp - 10) >> 2;  // queries qh*32 .. qh*32+31 of the tile
    const uint32_t lane_addr = tmem + ((uint32_t)(qw * 32) << 16);
    bool ok = mbar_wait_warp(kv_full, 0, abort_flag, ERRW_TIMEOUT_EPILOGUE);
    if (ok) {  // rows of K that are not finite: 16 rows per warp, half a row per lane
      const int row = (warp - 10) * 16 + (lane & 15);
      const auto chunk = [&](uint8_t* tile, int c) {
        return reinterpret_cast<uint4*>(tile + (lane >> 4) * 16384 + row * 128 + ((c ^ (row & 7)) << 4));
      };
      uint32_t odd = 0;  // the exponent of a NaN or infinity is all ones: one more carries into the bit above
      const auto look = [&](uint32_t u) { odd |= (u & 0x7f807f80u) + 0x00800080u; };
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 u = *chunk(sK, c);
        look(u.x);
        look(u.y);
        look(u.z);
        look(u.w);
      }
      odd |= __shfl_xor_sync(0xffffffffu, odd, 16);
      if (odd & 0x80008000u) {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          *chunk(sV, c) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
          *chunk(sK, c) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(dq_free);
    for (int i = 0; i < steps; ++i) {
      const int hh = kvh * G + (first + i) / nq;
      const int q0 = (qt_lo + (first + i) % nq) * AB2_BQ;
      ok = ok && mbar_wait_warp(dq_full, i & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE);
      uint32_t v0[32];
      if (ok) {
        tc_fence_after();
        tmem_ld_32x32b_x32(lane_addr + 384 + qh * 32, v0);
        tmem_ld_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(dq_free);
      if (ok) {
        const int m4 = lane & 3;
        const bool b1 = (m4 & 2) != 0, b0 = (m4 & 1) != 0;
        const int nv = n_rows - q0 - qh * 32;  // query rows of this half inside the sequence
        float* dst = dq + (long long)(q0 + qh * 32 + m4) * lddq + hh * 128 + qw * 32 + (lane & ~3);
#pragma unroll
        for (int qb = 0; qb < 8; ++qb) {
          // a[j]: query 4qb+j at this lane's hd  ->  a[j]: query 4qb+m4 at hd (lane&~3)+j
          float a[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = __uint_as_float(v0[qb * 4 + j]);
#pragma unroll
          for (int t = 0; t < 2; ++t) {  // swap the off-diagonal 2x2 blocks (lane bit 1)
            const float y = __shfl_xor_sync(0xffffffffu, b1 ? a[t] : a[2 + t], 2);
            if (b1) a[t] = y; else a[2 + t] = y;
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {  // transpose inside each 2x2 block (lane bit 0)
            const float y = __shfl_xor_sync(0xffffffffu, b0 ? a[2 * t] : a[2 * t + 1], 1);
            if (b0) a[2 * t] = y; else a[2 * t + 1] = y;
          }
          if (4 * qb + m4 < nv) red_add_v4_f32(dst + (long long)(4 * qb) * lddq, a[0], a[1], a[2], a[3]);
        }
      }
    }
  }
  if (cs > 1) {
    // the parts of the cluster's CTAs, added in their order: CTA `rank` does its
    // share of the rows, 8 columns at a time
    __syncwarp();
    cluster_sync_all();
    const int rows = AB2_BK / cs;
    for (int x = threadIdx.x; x < 2 * rows * 16; x += AB2_THREADS) {
      const int which = x / (rows * 16), rr = rank * rows + x / 16 % rows, c = (x & 15) * 2;
      float s[8] = {};
      for (int q = 0; q < cs; ++q) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float4 w;
          const uint32_t at = map_shared_rank(reinterpret_cast<float4*>(sQ) + (which * 128 + rr) * 32 + ((c + half) ^ (rr & 31)), q);
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
                       : "r"(at) : "memory");
          s[half * 4 + 0] += w.x;
          s[half * 4 + 1] += w.y;
          s[half * 4 + 2] += w.z;
          s[half * 4 + 3] += w.w;
        }
      }
      if (k0 + rr < n_rows)
        store8((which ? dv + (long long)(k0 + rr) * lddv : dk + (long long)(k0 + rr) * lddk) + kvh * 128 + c * 4, s);
    }
    cluster_sync_all();  // no CTA leaves while another reads its part
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Before the backward: D = rowsum(dO o) of each (row, head) and the fp32 dQ
// sums set to 0, a warp per (row, head) pair, 4 columns per lane; bound by HBM (8
// bytes per element).  o has been rounded to bf16, which moves dS = P (dP - D)
// by P dO (o rounded - o): next to what rounding dS to bf16 costs this is
// 1 / sqrt(visible keys).  So for rows that see at most PB_FEW keys D is taken
// as the sum of P dP, which needs no o: two lanes per key, by CTAs of their own.  (Without it dq and
// dk of 5 sequences of 12 to 180 tokens were 2.6e-3 off in the norm, with it
// 2.4e-3; 1.7e-3 is the rounding of the result alone.  15733 rows of 12 heads: 44
// us; forward and backward together take 5 us less without the rows of few keys.)
constexpr int PB_FEW = 16;
constexpr int PB_PRE_ROWS = 16;  // most rows of a CTA

// sum over 64 columns of two bf16 rows
__device__ __forceinline__ float dot64(const bf16* __restrict__ x, const bf16* __restrict__ y) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < 64; c += 8) {
    float a[8], b[8];
    load8(x + c, a);
    load8(y + c, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(a[k], b[k], s);
  }
  return s;
}

__global__ void __launch_bounds__(256)
    packed_attn_pre_kernel(const bf16* __restrict__ q, long long ldq, const bf16* __restrict__ k, long long ldk,
                           const bf16* __restrict__ v, long long ldv, const bf16* __restrict__ o, long long ldo,
                           const bf16* __restrict__ dO, long long lddo, const float* __restrict__ lse,
                           float* __restrict__ D, float* __restrict__ dq, const int32_t* __restrict__ cu, int n_seq,
                           int total, int H, int Hkv, int window, int rows, int few_ctas) {
  __shared__ int s_first[PB_PRE_ROWS];  // first visible row of each of the CTA's rows
  pdl_launch();  // (the main kernel's CTAs take the place of those that end)
  const int n_rows = packed_rows(cu, n_seq, total);
  if (blockIdx.x == 0) packed_check(cu, n_seq, total);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int STEP = 8, AHEAD = 4;
  const int few = (int)blockIdx.x - ((int)gridDim.x - few_ctas);  // (the last CTAs)
  if (few >= 0) {
    // the rows that see few keys: the first ones of every sequence, or all
    const bool every = window >= 0 && window < PB_FEW;
    const long long items = (every ? (long long)n_rows : (long long)n_seq * PB_FEW) * H;
#pragma unroll 1
    for (long long i = (long long)few * STEP + warp; i < items; i += (long long)few_ctas * STEP) {
      const int x = (int)(i / H), h = (int)(i - (long long)x * H);
      int t, first;
      if (every) {
        t = x;
        first = max(packed_seq(cu, n_seq, t, n_rows).x, t - window);
      } else {
        first = cu[x / PB_FEW];
        if (first < 0 || first >= n_rows) continue;  // (an empty sequence at the end; bad offsets)
        t = first + x % PB_FEW;
        if (t >= min(cu[x / PB_FEW + 1], n_rows)) continue;
      }
      const int j = first + (lane >> 1), c = (lane & 1) * 64, kvh = h / (H / Hkv);
      float acc = 0.f;
      if (j <= t) {
        float s = dot64(q + t * ldq + h * 128 + c, k + j * ldk + kvh * 128 + c);
        float dp = dot64(dO + t * lddo + h * 128 + c, v + j * ldv + kvh * 128 + c);
        const unsigned both = 3u << (lane & 30);
        s += __shfl_xor_sync(both, s, 1);
        dp += __shfl_xor_sync(both, dp, 1);
        acc = (lane & 1) ? 0.f
                         : fast_exp2(fmaf(s, LOG2E * rsqrtf(128.f), -lse[(long long)h * total + t] * LOG2E)) * dp;
      }
      acc = warp_sum(acc);
      if (lane == 0) D[(long long)h * total + t] = acc;
    }
    return;
  }
  const int r0 = (int)blockIdx.x * rows;
  if (r0 >= n_rows) return;
  if (threadIdx.x < rows && r0 + (int)threadIdx.x < n_rows) {
    const int t = r0 + threadIdx.x, first = packed_seq(cu, n_seq, t, n_rows).x;
    s_first[threadIdx.x] = window >= 0 ? max(first, t - min(window, t)) : first;
  }
  __syncthreads();
  const int n = min(rows, n_rows - r0) * H;  // (row, head) pairs, dealt out to the warps
  for (int i0 = warp; i0 < n; i0 += STEP * AHEAD) {
    uint2 a[AHEAD], b[AHEAD];
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      const int i = i0 + x * STEP;
      if (i >= n) break;
      const int t = r0 + i / H, h = i % H;
      a[x] = *reinterpret_cast<const uint2*>(o + (long long)t * ldo + h * 128 + lane * 4);
      b[x] = *reinterpret_cast<const uint2*>(dO + (long long)t * lddo + h * 128 + lane * 4);
      *reinterpret_cast<float4*>(dq + ((long long)t * H + h) * 128 + lane * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      const int i = i0 + x * STEP;
      if (i >= n) break;
      const __nv_bfloat162 *ha = reinterpret_cast<const __nv_bfloat162*>(&a[x]), *hb = reinterpret_cast<const __nv_bfloat162*>(&b[x]);
      float acc = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 u = __bfloat1622float2(ha[k]), w = __bfloat1622float2(hb[k]);
        acc = fmaf(u.x, w.x, fmaf(u.y, w.y, acc));
      }
      acc = warp_sum(acc);
      if (lane == 0 && r0 + i / H - s_first[i / H] >= PB_FEW) D[(long long)(i % H) * total + r0 + i / H] = acc;
    }
  }
}

// After it: dQ rounded to bf16, 8 columns per thread; bound by HBM (6 bytes per
// element: 15733 rows of 12 heads in 20 us, 7.2 TB/s, some of it still in L2).
__global__ void __launch_bounds__(256)
    packed_attn_dq_kernel(const float* __restrict__ acc, bf16* __restrict__ dq, long long lddq,
                          const int32_t* __restrict__ cu, int n_seq, int total, int H) {
  pdl_wait();  // (the sums)
  const int n_rows = packed_rows(cu, n_seq, total);
  const int per_row = H * 16;
  const long long n = (long long)n_rows * per_row;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const long long t = i / per_row;
    const int c = (int)(i - t * per_row) * 8;
    float v[8];
    load8(acc + i * 8, v);
    store8(dq + t * lddq + c, v);
  }
}

}  // namespace gptb
