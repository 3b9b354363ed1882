// One decode step of a batch whose sequences share prompts (bf16, hd = 128):
// attention of each sequence's newest token over the K/V rows of its group's
// prompt (the prefix, kept once for the whole group) and over its own cache.
//
//   keys of sequence b of group g: prefix rows j = 0 .. plen_g-1 at position j,
//   own rows i = 0 .. lens[b]-1 at position plen_g + i; the query stands at
//   t = plen_g + lens[b] - 1 and sees position p iff W < 0 or t - p <= W
//   o = softmax(q k^T / sqrt(hd)) v over both, lse its logarithm
//
// Bound by HBM: every visible prefix row is read once per group, not once per
// sequence, every own row once.  What makes that possible is the matrix unit:
// the query rows of a group that use one kv head (sequences x heads of the kv
// head's group, up to 128) are the M rows of one tile, so a K/V tile is read
// from shared memory once for all of them.  A sequence's own cache goes through
// the same tiles with only its few heads as rows; the padded rows cost matrix
// time that hides behind the loads, and warps without a row skip the softmax.
//
// Work: a "segment" is one (query rows, kv head, prefix or own cache); its
// keys are cut into 128-row tiles.  The tiles of all segments, laid end to end,
// are dealt out evenly and contiguously over the CTAs (every CTA computes the
// same prefix sum over the batch from lens and the offsets), so lengths that
// differ by any factor load every SM alike.  A segment that spans several CTAs
// leaves one partial softmax (max, sum, o) per CTA -- and per CTA two, as the
// even and odd tiles go to two softmax groups with an accumulator each -- and
// prefix_combine_kernel joins them.  The dealing is fixed by the lengths, so
// results do not vary from run to run.
#pragma once
#include "attention_tc.cuh"
#include "common.cuh"
#include "packed_attention.cuh"

namespace gptb {

constexpr int PD_THREADS = 320;
constexpr int PD_MAX_CTAS = 160;
constexpr int PD_TILE = FA_TILE;     // 128 rows x 128 columns, bf16: two 64-column swizzled halves
constexpr int PD_BOX = 32;           // rows per TMA box (a short last tile loads only the boxes it needs)
constexpr int PD_RING = 8;           // tile descriptors in flight (more than the K / V stages)
constexpr int PD_SMEM = 1024 + 2 * PD_TILE /*Q*/ + 4 * PD_TILE /*K, V x2*/;
constexpr int PD_REC = 132;          // floats of a partial result: o[128], max (base 2), sum, 2 unused

enum : int {
  PD_FIRST_SEG = 1, PD_LAST_SEG = 2,    // first / last tile of the segment's share in this CTA
  PD_FIRST_ACC = 4, PD_LAST_ACC = 8,    // first / last of them in its accumulator
  PD_END = 16,                          // no tile: the stream ends
  PD_CONT = 32,                         // the segment began in an earlier CTA
  PD_OWN = 64,                          // own cache (else prefix)
  PD_ODD = 128,                         // second accumulator's tiles of the segment
};
struct PdTile {
  int flags;
  int nk;     // valid keys, 1..128
  int pos;    // position of the first key
  int b0, nrows, kvh;
  int plen;   // prefix length of the group
  int pad;
};

struct PrefixArgs {
  const int32_t *cu_prefix, *cu_group, *lens;
  int total_prefix, n_groups, B, H, Hkv, T_max, window;
  int spt;       // sequences per query tile of a prefix segment (128 / G)
  int4* plan;    // [B + 1]: first tile of the sequence's segments, prefix tiles, own tiles (-1: bad length), first
                 // sequence of its query tile; [B].x = all tiles
  float* rec_a;  // [2 sources][B*H][2][PD_REC] the share of a segment that starts it
  float* rec_b;  // [CTAs][rows of a query tile][2][PD_REC] the share of the segment that a CTA goes on with
};

// the tiles of sequence b
struct PdSeq {
  int p0, plen;    // prefix rows p0 .. p0 + plen - 1
  int b0, nseq;    // its query tile: first sequence; sequences in it (0: b is not the first)
  int plo, ntp;    // first visible prefix row of the query tile, 128-key tiles (of b0's tile; 0 unless b == b0)
  int len, olo, nto;  // own rows (-1: outside the cache), first visible one, tiles
};
__device__ __forceinline__ PdSeq pd_seq(const PrefixArgs& a, int b) {
  PdSeq s;
  s.len = a.lens[b];
  if (s.len < 0 || s.len > a.T_max) s.len = -1;
  int gs = 0, ge = a.B, g = -1;
  if (a.n_groups > 0 && a.cu_group[0] <= b && b < a.cu_group[a.n_groups]) {
    int lo = 0, hi = a.n_groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_group[mid] <= b) lo = mid; else hi = mid;
    }
    g = lo;
    gs = max(0, min(a.cu_group[lo], b));
    ge = min(max(a.cu_group[hi], b + 1), a.B);
  }
  s.p0 = g >= 0 ? max(0, min(a.cu_prefix[g], a.total_prefix)) : 0;
  s.plen = g >= 0 ? max(s.p0, min(a.cu_prefix[g + 1], a.total_prefix)) - s.p0 : 0;
  s.b0 = g >= 0 ? gs + (b - gs) / a.spt * a.spt : b;
  s.nseq = s.b0 == b ? (g >= 0 ? min(a.spt, ge - b) : 1) : 0;
  s.plo = 0;
  s.ntp = 0;
  if (s.nseq > 0 && s.plen > 0) {
    if (a.window >= 0) {  // the shortest sequence of the tile sees furthest back
      int least = a.T_max;
      for (int i = 0; i < s.nseq; ++i) least = min(least, max(0, a.lens[b + i]));
      const long long lo = (long long)s.plen + least - 1 - a.window;
      s.plo = (int)max(0ll, min(lo, (long long)s.plen));
    }
    s.ntp = (s.plen - s.plo + FA_BN - 1) / FA_BN;
  }
  s.olo = (a.window >= 0 && s.len > 0) ? max(0, s.len - 1 - a.window) : 0;
  s.nto = s.len > 0 ? (s.len - s.olo + FA_BN - 1) / FA_BN : 0;
  return s;
}

// tile range of CTA c of n: [pd_begin(c), pd_begin(c + 1)); pd_owner(f): the CTA that has tile f
__device__ __forceinline__ int pd_begin(int c, int n, int W) { return (int)((long long)c * W / n); }
__device__ __forceinline__ int pd_owner(int f, int n, int W) { return (int)((((long long)f + 1) * n - 1) / W); }

__global__ void __launch_bounds__(PD_THREADS, 1)
    prefix_split_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qo,
                        const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                        const __grid_constant__ CUtensorMap tm_ko, const __grid_constant__ CUtensorMap tm_vo,
                        const PrefixArgs a) {
  extern __shared__ uint8_t pd_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pd_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;              // 2 segments' query tiles
  uint8_t* sK = sQ + 2 * PD_TILE;  // 2 stages
  uint8_t* sV = sK + 2 * PD_TILE;  // 2 stages
  __shared__ __align__(8) uint64_t bars[24];
  uint64_t* q_full = bars + 0;    // [2]
  uint64_t* q_empty = bars + 2;   // [2]
  uint64_t* k_full = bars + 4;    // [2]
  uint64_t* k_empty = bars + 6;   // [2]
  uint64_t* v_full = bars + 8;    // [2]
  uint64_t* v_empty = bars + 10;  // [2]
  uint64_t* s_full = bars + 12;   // [2 groups]
  uint64_t* p_full = bars + 14;   // [2 groups]
  uint64_t* o_done = bars + 16;   // [2 groups]
  uint64_t* o_free = bars + 18;   // [2 groups] the accumulator has been read out
  uint64_t* drain = bars + 20;
  __shared__ PdTile ring[PD_RING];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort, s_sum[PD_THREADS / 32], s_b, s_off;
  volatile int* abort_flag = &s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv;
  const int cta = blockIdx.x, nctas = gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_free[i], 4);
    }
    mbar_init(drain, 1);
    s_abort = 0;
    s_b = 0;
    s_off = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_qp);
    tma_prefetch_desc(&tm_qo);
    tma_prefetch_desc(&tm_kp);
    tma_prefetch_desc(&tm_vp);
    tma_prefetch_desc(&tm_ko);
    tma_prefetch_desc(&tm_vo);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, 512);

  // the batch's tiles, summed up: thread i has the sequences i*per .. of the batch
  const int per = (a.B + PD_THREADS - 1) / PD_THREADS;
  const int b_lo = min(a.B, (int)threadIdx.x * per), b_hi = min(a.B, b_lo + per);
  int mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const PdSeq s = pd_seq(a, b);
    mine += a.Hkv * (s.ntp + s.nto);
  }
  int inc = mine;  // inclusive sum over the warp's lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_sum[warp] = inc;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  int before = inc - mine, W = 0;
  for (int w = 0; w < PD_THREADS / 32; ++w) {
    if (w < warp) before += s_sum[w];
    W += s_sum[w];
  }
  const int f0 = pd_begin(cta, nctas, W), f1 = pd_begin(cta + 1, nctas, W);
  if (cta == 0 || (before <= f0 && f0 < before + mine)) {
    int f = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const PdSeq s = pd_seq(a, b);
      const int n = a.Hkv * (s.ntp + s.nto);
      if (f <= f0 && f0 < f + n) {  // this CTA's first tile
        s_b = b;
        s_off = f0 - f;
      }
      if (cta == 0) a.plan[b] = make_int4(f, s.ntp, s.len < 0 ? -1 : s.nto, s.b0);
      f += n;
    }
  }
  if (cta == 0) {
    if (threadIdx.x == 0) a.plan[a.B] = make_int4(W, 0, 0, 0);
    if (a.n_groups > 0) {
      packed_check(a.cu_prefix, a.n_groups, a.total_prefix);
      packed_check(a.cu_group, a.n_groups, a.B);
    }
  }
  __syncthreads();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int left = f1 - f0, b = s_b, off = s_off, n = 0, seg = 0;
      bool ok = true;
      PdSeq s;
      if (left > 0) s = pd_seq(a, b);
      while (ok && left > 0) {
        const int np = a.Hkv * s.ntp;
        const bool own = off >= np;
        const int nt = own ? s.nto : s.ntp;
        const int at = own ? off - np : off;
        if (nt == 0 || at >= a.Hkv * nt) {  // the next sequence
          if (++b >= a.B) break;
          off = 0;
          s = pd_seq(a, b);
          continue;
        }
        const int kvh = at / nt, t0 = at - kvh * nt;
        const int cnt = min(nt - t0, left);
        // the segment's query rows
        const int qs = seg & 1;
        ok = mbar_wait(&q_empty[qs], ((seg >> 1) & 1) ^ 1u, abort_flag, ERRW_TIMEOUT_PRODUCER);
        if (!ok) break;
        uint8_t* q = sQ + qs * PD_TILE;
        const CUtensorMap* mq = own ? &tm_qo : &tm_qp;
        mbar_arrive_expect_tx(&q_full[qs], 2 * 128 * G * (own ? 1 : a.spt));
        tma_load_3d(q, mq, &q_full[qs], 0, kvh * G, b);
        tma_load_3d(q + 16384, mq, &q_full[qs], 64, kvh * G, b);
        const CUtensorMap *mk = own ? &tm_ko : &tm_kp, *mv = own ? &tm_vo : &tm_vp;
        const int first = own ? s.olo : s.plo, rows = own ? s.len : s.plen;
        const int base = own ? b * a.T_max : s.p0;
        for (int j = 0; j < cnt; ++j, ++n) {
          const int st = n & 1;
          const uint32_t par = ((n >> 1) & 1) ^ 1u;
          const int r0 = first + (t0 + j) * FA_BN;
          PdTile d;
          d.nk = min(FA_BN, rows - r0);
          d.flags = (j == 0 ? PD_FIRST_SEG : 0) | (j == cnt - 1 ? PD_LAST_SEG : 0) | (j < 2 ? PD_FIRST_ACC : 0) |
                    (j >= cnt - 2 ? PD_LAST_ACC : 0) | (t0 > 0 ? PD_CONT : 0) | (own ? PD_OWN : 0) |
                    (j & 1 ? PD_ODD : 0);
          d.pos = own ? s.plen + r0 : r0;
          d.b0 = b;
          d.nrows = own ? G : s.nseq * G;
          d.kvh = kvh;
          d.plen = s.plen;
          const int boxes = (d.nk + PD_BOX - 1) / PD_BOX;
          ok = mbar_wait(&k_empty[st], par, abort_flag, ERRW_TIMEOUT_PRODUCER);
          if (!ok) break;
          // (the ring's entry was last read by the softmax of tile n - PD_RING,
          // before the PV product whose end freed the V stage of tile n - 1)
          ring[n % PD_RING] = d;
          mbar_arrive_expect_tx(&k_full[st], boxes * 2 * PD_BOX * 128);
          uint8_t* k = sK + st * PD_TILE;
          for (int x = 0; x < boxes; ++x) {
            tma_load_2d(k + x * PD_BOX * 128, mk, &k_full[st], kvh * 128, base + r0 + x * PD_BOX);
            tma_load_2d(k + 16384 + x * PD_BOX * 128, mk, &k_full[st], kvh * 128 + 64, base + r0 + x * PD_BOX);
          }
          ok = mbar_wait(&v_empty[st], par, abort_flag, ERRW_TIMEOUT_PRODUCER);
          if (!ok) break;
          mbar_arrive_expect_tx(&v_full[st], boxes * 2 * PD_BOX * 128);
          uint8_t* v = sV + st * PD_TILE;
          for (int x = 0; x < boxes; ++x) {
            tma_load_2d(v + x * PD_BOX * 128, mv, &v_full[st], kvh * 128, base + r0 + x * PD_BOX);
            tma_load_2d(v + 16384 + x * PD_BOX * 128, mv, &v_full[st], kvh * 128 + 64, base + r0 + x * PD_BOX);
          }
        }
        off += cnt;
        left -= cnt;
        ++seg;
      }
      // the end of the stream, for both softmax groups
      if (ok && mbar_wait(&k_empty[n & 1], ((n >> 1) & 1) ^ 1u, abort_flag, ERRW_TIMEOUT_PRODUCER)) {
        ring[n % PD_RING].flags = PD_END;
        ring[(n + 1) % PD_RING].flags = PD_END;
        mbar_arrive(&k_full[n & 1]);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // S_t = Q K^T of tile n (t = n % 2) is issued one tile ahead of O_t += P_t V
    if (lane == 0) {
      constexpr uint32_t IDESC_S = make_idesc(128, 128, false, false, false);
      constexpr uint32_t IDESC_O = make_idesc(128, 128, false, true, false);
      int seg = -1, used[2] = {0, 0};
      bool ok = true, end = false;
      auto issue_s = [&](int n) -> int {
        const int t = n & 1;
        ok = mbar_wait(&k_full[t], (n >> 1) & 1, abort_flag, ERRW_TIMEOUT_MMA);
        if (!ok) return 0;
        const int fl = *reinterpret_cast<volatile int*>(&ring[n % PD_RING].flags);
        if (fl & PD_END) {
          end = true;
          return fl;
        }
        if (fl & PD_FIRST_SEG) {
          ++seg;
          ok = mbar_wait(&q_full[seg & 1], (seg >> 1) & 1, abort_flag, ERRW_TIMEOUT_MMA);
          if (!ok) return 0;
        }
        tc_fence_after();
        const uint32_t aQ = smem_u32(sQ + (seg & 1) * PD_TILE), aK = smem_u32(sK + t * PD_TILE);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ss(tmem + t * 128, fa_desc_k(aQ, k), fa_desc_k(aK, k), IDESC_S, k > 0 ? 1u : 0u);
        mma_commit(&s_full[t]);
        mma_commit(&k_empty[t]);
        if (fl & PD_LAST_SEG) mma_commit(&q_empty[seg & 1]);
        return fl;
      };
      int fl = issue_s(0);
      for (int n = 0; ok && !end; ++n) {
        const int t = n & 1;
        const int fl_n = fl;
        fl = issue_s(n + 1);
        if (!ok) break;
        if (!mbar_wait(&v_full[t], (n >> 1) & 1, abort_flag, ERRW_TIMEOUT_MMA) ||
            !mbar_wait(&p_full[t], (n >> 1) & 1, abort_flag, ERRW_TIMEOUT_MMA) ||
            ((fl_n & PD_FIRST_ACC) &&
             !mbar_wait(&o_free[t], (used[t]++ & 1) ^ 1u, abort_flag, ERRW_TIMEOUT_MMA))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t aV = smem_u32(sV + t * PD_TILE);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, fa_desc_mn(aV, k), IDESC_O,
                      (k > 0 || !(fl_n & PD_FIRST_ACC)) ? 1u : 0u);
        mma_commit(&v_empty[t]);
        mma_commit(&o_done[t]);
      }
      if (ok) {  // both groups have taken their last tile: they read the end mark
        mbar_arrive(&s_full[0]);
        mbar_arrive(&s_full[1]);
      }
      if (*abort_flag) {
        mma_commit(drain);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0))
          if (globaltimer_ns() - t0 > 100000000ull) { record_error(ERRW_TIMEOUT_DRAIN); break; }
      }
    }
  } else {
    // ------------------------------------- softmax group t: tiles n % 2 == t
    const int t = (warp - 2) >> 2;
    const int qw = warp & 3;       // TMEM lane quarter
    const int r = qw * 32 + lane;  // row of the query tile
    const uint32_t lane_addr = tmem + ((uint32_t)(qw * 32) << 16);
    const uint32_t s_col = (uint32_t)(t * 128), o_col = (uint32_t)(256 + t * 128);
    const float sl2 = LOG2E / sqrtf(128.f);
    float m_used = -INFINITY, l = 0.f;
    int oldest = 0;  // the row's oldest visible position
    for (int c = 0;; ++c) {
      const int n = 2 * c + t;
      if (!mbar_wait_warp(&s_full[t], c & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE)) break;
      const volatile PdTile& dv = ring[n % PD_RING];
      const int flags = dv.flags;
      if (flags & PD_END) break;
      const int nk = dv.nk, pos = dv.pos, b0 = dv.b0, nrows = dv.nrows, kvh = dv.kvh;
      const bool active = qw * 32 < nrows;  // (the whole warp)
      const int b = b0 + r / G;
      if (flags & PD_FIRST_ACC) {
        m_used = -INFINITY;
        l = 0.f;
        if (a.window >= 0) oldest = r < nrows ? dv.plen + a.lens[b] - 1 - min(a.window, 1 << 30) : 0;
      }
      // V rows behind the last key are another sequence's, or older tiles':
      // they are zeroed (0 * NaN is NaN)
      if (nk < FA_BN) {
        if (!mbar_wait_warp(&v_full[t], c & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE)) break;
        if (r >= nk) zero_tile_row(sV + t * PD_TILE, 16384, r);
        fence_proxy_async_smem();
      }
      if (active) {
        tc_fence_after();
        uint32_t v[128];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tmem_ld_32x32b_x32(lane_addr + s_col + k * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[k * 32]));
        tmem_ld_wait();
        const int lo = a.window >= 0 ? oldest - pos : 0;  // the row sees keys lo .. nk-1 of the tile
        if (nk < FA_BN || __any_sync(0xffffffffu, lo > 0)) {
#pragma unroll
          for (int i = 0; i < 128; ++i) v[i] = (i >= lo && i < nk) ? v[i] : __float_as_uint(-INFINITY);
        }
        float mp[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mp[i] = __uint_as_float(v[i]);
#pragma unroll
        for (int i = 8; i < 128; ++i) mp[i & 7] = fmaxf(mp[i & 7], __uint_as_float(v[i]));
        const float mx = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                               fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7]))) * sl2;
        // the running max moves only when it grows by more than 8 (base 2)
        const bool grow = mx > m_used + 8.f;
        const float corr = grow ? fast_exp2(m_used - mx) : 1.f;  // 0 when m_used is -inf
        if (grow) {
          l *= corr;
          m_used = mx;
        }
        const float mu = (m_used == -INFINITY) ? 0.f : m_used;
        float lp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hq = 0; hq < 4; ++hq) {  // 32 keys (16 columns of P) at a time
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int i = hq * 32 + 2 * e;
            const float p0 = fast_exp2(fmaf(__uint_as_float(v[i]), sl2, -mu));
            const float p1 = fast_exp2(fmaf(__uint_as_float(v[i + 1]), sl2, -mu));
            lp[(2 * e) & 3] += p0;
            lp[(2 * e + 1) & 3] += p1;
            pk[e] = pack_bf16(p0, p1);
          }
          tmem_st_32x32b_x16(lane_addr + s_col + hq * 16, pk);
        }
        l += (lp[0] + lp[1]) + (lp[2] + lp[3]);
        if (!(flags & PD_FIRST_ACC) && __any_sync(0xffffffffu, grow)) {
          if (!mbar_wait_warp(&o_done[t], (c - 1) & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE)) break;
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t w[32];
            tmem_ld_32x32b_x32(lane_addr + o_col + k * 32, w);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * corr);
            tmem_st_32x32b_x32(lane_addr + o_col + k * 32, w);
          }
        }
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
      if (flags & PD_LAST_ACC) {
        if (active) {
          if (!mbar_wait_warp(&o_done[t], c & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE)) break;
          tc_fence_after();
          const int odd = flags & PD_ODD ? 1 : 0;
          float* rec;
          if (flags & PD_CONT)
            rec = a.rec_b + (((long long)cta * a.spt * G + r) * 2 + odd) * PD_REC;
          else
            rec = a.rec_a + ((((flags & PD_OWN ? 1ll : 0ll) * a.B + b) * a.H + kvh * G + r % G) * 2 + odd) * PD_REC;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t w[32];
            tmem_ld_32x32b_x32(lane_addr + o_col + k * 32, w);
            tmem_ld_wait();
            if (r < nrows) {
#pragma unroll
              for (int g = 0; g < 8; ++g)
                *reinterpret_cast<float4*>(rec + k * 32 + g * 4) =
                    make_float4(__uint_as_float(w[g * 4]), __uint_as_float(w[g * 4 + 1]),
                                __uint_as_float(w[g * 4 + 2]), __uint_as_float(w[g * 4 + 3]));
            }
          }
          if (r < nrows) *reinterpret_cast<float2*>(rec + 128) = make_float2(m_used, l);
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[t]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One warp per (sequence, head) joins its partial results: lane i takes the
// max and sum of the i-th one, then all lanes add up 4 columns each.
__global__ void __launch_bounds__(128)
    prefix_combine_kernel(const PrefixArgs a, bf16* __restrict__ o, float* __restrict__ lse, int nctas) {
  const int lane = threadIdx.x & 31;
  const long long bh = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (bh >= (long long)a.B * a.H) return;
  const int b = (int)(bh / a.H), h = (int)(bh - (long long)b * a.H);
  const int G = a.H / a.Hkv, kvh = h / G, W = a.plan[a.B].x;
  const int4 mine = a.plan[b], tile = a.plan[mine.w];
  // the segments: first tile, tiles, first and last CTA, row in its query tile
  int f[2], nt[2], c0[2], c1[2], row[2];
  nt[0] = tile.y;
  f[0] = tile.x + kvh * nt[0];
  row[0] = (b - mine.w) * G + h - kvh * G;
  nt[1] = max(mine.z, 0);
  f[1] = mine.x + a.Hkv * mine.y + kvh * nt[1];
  row[1] = h - kvh * G;
  int count = 0, split = 0;  // partial results; those of the prefix come first
  for (int s = 0; s < 2; ++s) {
    c0[s] = nt[s] > 0 ? pd_owner(f[s], nctas, W) : 0;
    c1[s] = nt[s] > 0 ? pd_owner(f[s] + nt[s] - 1, nctas, W) : -1;
    if (s == 1) split = count;
    count += 2 * (c1[s] - c0[s] + 1);
  }
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (mine.z < 0) count = 0;  // a length outside the cache
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int i = i0 + lane;
    const float* rec = nullptr;
    if (i < count) {
      const int s = i >= split ? 1 : 0, x = i - (s ? split : 0), c = c0[s] + (x >> 1), odd = x & 1;
      const int from = max(f[s], pd_begin(c, nctas, W)), to = min(f[s] + nt[s], pd_begin(c + 1, nctas, W));
      if (to - from > odd)  // the odd tiles' result exists if the CTA had two tiles
        rec = c == c0[s] ? a.rec_a + ((((long long)s * a.B + b) * a.H + h) * 2 + odd) * PD_REC
                         : a.rec_b + (((long long)c * a.spt * G + row[s]) * 2 + odd) * PD_REC;
    }
    const float mi = rec ? rec[128] : -INFINITY, li = rec ? rec[129] : 0.f;
    const float mn = fmaxf(m, warp_max(mi));
    // (a result of no visible key has sum 0; one whose scores are all NaN has sum NaN)
    const float w = mi == -INFINITY ? (li == 0.f ? 0.f : 1.f) : fast_exp2(mi - mn);
    const float old = m == -INFINITY ? 0.f : fast_exp2(m - mn);
    l = l * old + warp_sum(li * w);
    m = mn;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= old;
    const int here = min(32, count - i0);
#pragma unroll 4
    for (int j = 0; j < here; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float* rj = reinterpret_cast<const float*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rec), j));
      if (wj != 0.f) {
        const float4 u = *reinterpret_cast<const float4*>(rj + lane * 4);
        acc[0] = fmaf(wj, u.x, acc[0]);
        acc[1] = fmaf(wj, u.y, acc[1]);
        acc[2] = fmaf(wj, u.z, acc[2]);
        acc[3] = fmaf(wj, u.w, acc[3]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 u;
  u.x = pack_bf16(acc[0] * inv, acc[1] * inv);
  u.y = pack_bf16(acc[2] * inv, acc[3] * inv);
  *reinterpret_cast<uint2*>(o + bh * 128 + lane * 4) = u;
  if (lane == 0 && lse) lse[bh] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

}  // namespace gptb
