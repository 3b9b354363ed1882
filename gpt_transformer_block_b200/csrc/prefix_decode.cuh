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
// are dealt out contiguously over the CTAs by cost (every CTA computes the same
// prefix sum over the batch from lens and the offsets), so lengths that differ
// by any factor load every SM alike.  A segment that spans several CTAs leaves
// one partial softmax (max, sum, o) per CTA -- and per CTA two, as the even and
// odd tiles go to two softmax groups with an accumulator each -- and
// prefix_combine_kernel joins them.  The dealing is fixed by the lengths, so
// results do not vary from run to run.
//
// A tile's loads take 2.4 us to arrive with HBM busy, so K and V have a ring
// each, and the producer issues whichever has a free stage (in turn, K waited
// for the V stage before it: 2600 cycles per tile); and the query rows of
// several segments lie in shared memory side by side: the matrix product reads
// 128 rows from the first of them on, and what lies behind makes rows of S that
// nobody reads.  64 samples over 32000 shared tokens, 12 heads, 10 to 250 own
// tokens: 62 us with the join, 3.6 TB/s over all and 5 TB/s between start (3 us)
// and join (8 us); 128 samples of 8 prompts, 10 heads over 5: 43 us.
#pragma once
#include "attention_tc.cuh"
#include "common.cuh"
#include "packed_attention.cuh"

namespace gptb {

constexpr int PD_THREADS = 384;   // warps 0-7 softmax, 10 producer, 11 MMA issuer
// (the producer polls: on the scheduler of the warps that hold TMEM lanes 0-31,
// the only ones with rows in most segments, it would take their issue slots)
constexpr int PD_PRODUCER = 10, PD_MMA = 11;
constexpr int PD_MAX_CTAS = 160;
constexpr int PD_TILE = FA_TILE;  // 128 rows x 128 columns, bf16: two 64-column swizzled halves
constexpr int PD_BOX = 32;        // rows per TMA box (a short last tile loads only the boxes it needs)
constexpr int PD_ST = 3;          // K / V stages
constexpr int PD_RING = 8;        // tile descriptors in flight (more than the K / V stages)
constexpr int PD_QS = 8;          // segments whose query rows can be in shared memory, in 16 units of 8 rows
constexpr int PD_SMEM = 1024 + PD_TILE /*Q*/ + 2 * PD_ST * PD_TILE;
// cost of a segment: its tiles, and PD_OPEN units more (query rows to load, an
// accumulator to read out) that go with its first tile
constexpr int PD_UNIT = 4, PD_OPEN = 2;
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
  int q;      // first 8-row unit of the segment's query rows
  int row;    // first row of the tile in the prefix or the cache
};

struct PrefixArgs {
  const int32_t *cu_prefix, *cu_group, *lens;
  int total_prefix, n_groups, B, H, Hkv, T_max, window;
  int spt;       // sequences per query tile of a prefix segment (128 / G)
  const bf16 *q, *k_prefix, *v_prefix, *k_cache, *v_cache;
  long long ld_prefix;
  int4* plan;    // [B + 1]: first cost unit of the sequence's segments, prefix tiles, own tiles (-1: bad length),
                 // first sequence of its query tile; [B].x = all units
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

// units of a segment of nt tiles; the first tile whose units begin at u (relative to the segment) or later
__device__ __forceinline__ int pd_units(int nt) { return nt > 0 ? PD_UNIT * nt + PD_OPEN : 0; }
__device__ __forceinline__ int pd_tile(int u) {
  return u <= 0 ? 0 : u <= PD_OPEN + PD_UNIT ? 1 : (u - PD_OPEN + PD_UNIT - 1) / PD_UNIT;
}
// CTA c of n has the tiles that begin in the units [pd_begin(c), pd_begin(c + 1)) of U; pd_owner(u): the CTA of unit u
// (n <= PD_MAX_CTAS; a 64-bit division costs ten times a 32-bit one)
__device__ __forceinline__ int pd_begin(int c, int n, int U) {
  return U < (1 << 24) ? (int)((uint32_t)c * (uint32_t)U / (uint32_t)n) : (int)((long long)c * U / n);
}
__device__ __forceinline__ int pd_owner(int u, int n, int U) {
  return U < (1 << 24) ? (int)((((uint32_t)u + 1u) * (uint32_t)n - 1u) / (uint32_t)U)
                       : (int)((((long long)u + 1) * n - 1) / U);
}

// f(seq, b, own, kvh, j0, j1) for every segment with tiles in the units [u0,
// u1): its tiles j0 .. j1-1.  The walk starts at sequence b, whose segments
// start at unit `base`, and ends early when f returns false.  By a whole warp,
// whose lanes look up 32 sequences at once.
template <class F>
__device__ __forceinline__ bool pd_walk(const PrefixArgs& a, int b, int base, int u0, int u1, F&& f) {
  const int lane = threadIdx.x & 31;
  PdSeq block;
  for (int at_lane = 0; b < a.B && base < u1; ++b, ++at_lane) {
    if ((at_lane & 31) == 0) block = pd_seq(a, min(b + lane, a.B - 1));
    const auto get = [&](int v) { return __shfl_sync(0xffffffffu, v, at_lane & 31); };
    const PdSeq s{get(block.p0), get(block.plen), get(block.b0), get(block.nseq), get(block.plo),
                  get(block.ntp), get(block.len), get(block.olo), get(block.nto)};
    for (int own = 0; own < 2; ++own) {
      const int nt = own ? s.nto : s.ntp, len = pd_units(nt);
      if (nt == 0) continue;
      for (int kvh = u0 > base ? (u0 - base) / len : 0; kvh < a.Hkv; ++kvh) {
        const int at = base + kvh * len;
        if (at >= u1) break;
        const int j0 = pd_tile(u0 - at), j1 = min(nt, pd_tile(u1 - at));
        if (j0 < j1 && !f(s, b, own != 0, kvh, j0, j1)) return false;
      }
      base += a.Hkv * len;
    }
  }
  return true;
}

__global__ void __launch_bounds__(PD_THREADS, 1)
    prefix_split_kernel(const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qo,
                        const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                        const __grid_constant__ CUtensorMap tm_ko, const __grid_constant__ CUtensorMap tm_vo,
                        const PrefixArgs a) {
  extern __shared__ uint8_t pd_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pd_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                  // the query rows of up to PD_QS segments
  uint8_t* sK = sQ + PD_TILE;          // PD_ST stages
  uint8_t* sV = sK + PD_ST * PD_TILE;  // PD_ST stages
  __shared__ __align__(8) uint64_t bars[9 + 4 * PD_ST + 2 * PD_QS];
  uint64_t* s_full = bars + 0;             // [2 groups]
  uint64_t* p_full = bars + 2;             // [2 groups]
  uint64_t* o_done = bars + 4;             // [2 groups]
  uint64_t* o_free = bars + 6;             // [2 groups] the accumulator has been read out
  uint64_t* drain = bars + 8;
  uint64_t* k_full = bars + 9;             // [PD_ST]
  uint64_t* k_empty = k_full + PD_ST;      // [PD_ST]
  uint64_t* v_full = k_full + 2 * PD_ST;   // [PD_ST]
  uint64_t* v_empty = k_full + 3 * PD_ST;  // [PD_ST]
  uint64_t* q_full = k_full + 4 * PD_ST;   // [PD_QS]
  uint64_t* q_empty = q_full + PD_QS;      // [PD_QS]
  __shared__ PdTile ring[PD_RING];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort, s_sum[PD_THREADS / 32], s_b, s_base;
  volatile int* abort_flag = &s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hkv;
  const int cta = blockIdx.x, nctas = gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_free[i], 4);
    }
    for (int i = 0; i < PD_ST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < PD_QS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    mbar_init(drain, 1);
    s_abort = 0;
    s_b = a.B;
    s_base = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_qp);
    tma_prefetch_desc(&tm_qo);
    tma_prefetch_desc(&tm_kp);
    tma_prefetch_desc(&tm_vp);
    tma_prefetch_desc(&tm_ko);
    tma_prefetch_desc(&tm_vo);
  }
  if (warp == PD_MMA) tmem_alloc(&tmem_slot, 512);

  // the batch's cost, summed up: thread i has the sequences i*per .. of the batch
  const int per = (a.B + PD_THREADS - 1) / PD_THREADS;
  const int b_lo = min(a.B, (int)threadIdx.x * per), b_hi = min(a.B, b_lo + per);
  int mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const PdSeq s = pd_seq(a, b);
    mine += a.Hkv * (pd_units(s.ntp) + pd_units(s.nto));
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
  int before = inc - mine, U = 0;
  for (int w = 0; w < PD_THREADS / 32; ++w) {
    if (w < warp) before += s_sum[w];
    U += s_sum[w];
  }
  const int u0 = pd_begin(cta, nctas, U), u1 = pd_begin(cta + 1, nctas, U);
  if (cta == 0 || (before <= u0 && u0 < before + mine)) {
    int u = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const PdSeq s = pd_seq(a, b);
      const int n = a.Hkv * (pd_units(s.ntp) + pd_units(s.nto));
      if (u <= u0 && u0 < u + n) {  // this CTA's first unit
        s_b = b;
        s_base = u;
      }
      if (cta == 0) a.plan[b] = make_int4(u, s.ntp, s.len < 0 ? -1 : s.nto, s.b0);
      u += n;
    }
  }
  pdl_launch();  // (prefix_combine_kernel's CTAs take the place of those that end, and wait for the rest)
  if (cta == 0) {
    if (threadIdx.x == 0) a.plan[a.B] = make_int4(U, 0, 0, 0);
    if (a.n_groups > 0) {
      packed_check(a.cu_prefix, a.n_groups, a.total_prefix);
      packed_check(a.cu_group, a.n_groups, a.B);
    }
  }
  __syncthreads();

  if (warp == PD_PRODUCER) {
    // -------------------------------------------- producer (the whole warp)
    {
      int n = 0, nv = 0, seg = 0;    // K tiles, V tiles and segments so far
      int q_at = 0, q_used = 0;      // next free unit of sQ; units in use
      int q_old = 0;                 // the oldest segment in sQ
      unsigned long long q_len = 0;  // units (8 bits) of the segments q_old, q_old + 1, ... in sQ, and skipped before them
      // one tile's rows (those boxes that hold keys) into a stage, a box by each lane
      const auto load = [&](const PdTile& d, uint8_t* to, uint64_t* bar, const CUtensorMap* map) {
        const int boxes = (d.nk + PD_BOX - 1) / PD_BOX;
        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * 2 * PD_BOX * 128);
        __syncwarp();
        const int x = lane >> 1, half = lane & 1;
        if (x < boxes)
          tma_load_2d(to + half * 16384 + x * PD_BOX * 128, map, bar, d.kvh * 128 + half * 64, d.row + x * PD_BOX);
      };
      const auto ready = [&](uint64_t* bar, uint32_t parity) {  // (the same answer in all lanes)
        return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) != 0;
      };
      // the V tiles whose stages are free, up to the last K tile
      const auto pump = [&]() {
        while (nv < n && ready(&v_empty[nv % PD_ST], ((nv / PD_ST) & 1) ^ 1u)) {
          const PdTile d = ring[nv % PD_RING];
          load(d, sV + nv % PD_ST * PD_TILE, &v_full[nv % PD_ST], d.flags & PD_OWN ? &tm_vo : &tm_vp);
          ++nv;
        }
      };
      // bounded as mbar_wait, issuing V tiles meanwhile; bar NULL: until all V tiles are issued
      const auto wait = [&](uint64_t* bar, uint32_t parity) {
        unsigned long long t0 = 0;
        for (uint32_t i = 0;; ++i) {
          if (bar ? ready(bar, parity) : nv == n) return true;
          pump();
          if ((i & 255u) == 255u) {
            const unsigned long long now = __shfl_sync(0xffffffffu, globaltimer_ns(), 0);
            if (t0 == 0) t0 = now;
            const bool late = now - t0 > g_wait_limit_ns;
            if (late && lane == 0) {
              record_error(ERRW_TIMEOUT_PRODUCER);
              *abort_flag = 1;
            }
            __syncwarp();
            if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
          }
        }
      };
      const auto segment = [&](const PdSeq& s, int b, bool own, int kvh, int j0, int j1) {
        // room for its query rows, in one piece; the oldest leave first
        const int nseq = own ? 1 : a.spt, need = (nseq * G + 7) / 8;
        bool wrap;
        int skip;
        while (true) {
          if (q_used == 0) q_at = 0;
          wrap = q_at + need > 16;
          skip = wrap ? 16 - q_at : 0;
          if (q_used + skip + need <= 16 && seg - q_old < PD_QS) break;
          if (!wait(&q_empty[q_old % PD_QS], (q_old / PD_QS) & 1)) return false;
          q_used -= (int)(q_len & 255);
          q_len >>= 8;
          ++q_old;
        }
        const int at = wrap ? 0 : q_at;
        q_len |= (unsigned long long)(skip + need) << (8 * (seg - q_old));
        q_used += skip + need;
        q_at = at + need;
        uint64_t* qf = &q_full[seg % PD_QS];
        const CUtensorMap* mq = own ? &tm_qo : &tm_qp;
        if (lane == 0) mbar_arrive_expect_tx(qf, 2 * 128 * G * nseq);
        __syncwarp();
        if (lane < 2) tma_load_3d(sQ + lane * 16384 + at * 1024, mq, qf, lane * 64, kvh * G, b);
        ++seg;
        PdTile d;
        d.b0 = b;
        d.nrows = own ? G : s.nseq * G;
        d.kvh = kvh;
        d.plen = s.plen;
        d.q = at;
        const int first = own ? s.olo : s.plo, rows = own ? s.len : s.plen, base = own ? b * a.T_max : s.p0;
        for (int j = j0; j < j1; ++j) {
          const int r0 = first + j * FA_BN;
          d.nk = min(FA_BN, rows - r0);
          d.flags = (j == j0 ? PD_FIRST_SEG : 0) | (j == j1 - 1 ? PD_LAST_SEG : 0) | (j < j0 + 2 ? PD_FIRST_ACC : 0) |
                    (j >= j1 - 2 ? PD_LAST_ACC : 0) | (j0 > 0 ? PD_CONT : 0) | (own ? PD_OWN : 0) |
                    ((j - j0) & 1 ? PD_ODD : 0);
          d.pos = own ? s.plen + r0 : r0;
          d.row = base + r0;
          if (!wait(&k_empty[n % PD_ST], ((n / PD_ST) & 1) ^ 1u)) return false;
          // The ring's entry was last read by the softmax of tile n - PD_RING:
          // this stage was freed by S of tile n - PD_ST, issued after the PV
          // product of tile n - PD_ST - 2, and so after that tile's softmax
          // and the issue of its V.
          if (lane == 0) ring[n % PD_RING] = d;
          __syncwarp();
          load(d, sK + n % PD_ST * PD_TILE, &k_full[n % PD_ST], own ? &tm_ko : &tm_kp);
          ++n;
          pump();
        }
        return true;
      };
      // then the end of the stream, for both softmax groups
      if (pd_walk(a, s_b, s_base, u0, u1, segment) && wait(nullptr, 0) &&
          wait(&k_empty[n % PD_ST], ((n / PD_ST) & 1) ^ 1u)) {
        if (lane == 0) {
          ring[n % PD_RING].flags = PD_END;
          ring[(n + 1) % PD_RING].flags = PD_END;
          mbar_arrive(&k_full[n % PD_ST]);
        }
      }
    }
  } else if (warp == PD_MMA) {
    // ---------------------------------------------------------- MMA issuer
    // S_t = Q K^T of tile n (t = n % 2) is issued one tile ahead of O_t += P_t V.
    // A short tile takes the keys it has, in steps of 16.
    if (lane == 0) {
      constexpr uint32_t IDESC_S = make_idesc(128, 0, false, false, false);  // + N
      constexpr uint32_t IDESC_O = make_idesc(128, 128, false, true, false);
      int seg = -1, used[2] = {0, 0};
      bool ok = true, end = false;
      int steps = 0, q_unit = 0;  // 16-key steps of the tile whose S was issued last; its segment's query rows
      auto issue_s = [&](int n) -> int {
        const int t = n & 1, st = n % PD_ST;
        ok = mbar_wait(&k_full[st], (n / PD_ST) & 1, abort_flag, ERRW_TIMEOUT_MMA);
        if (!ok) return 0;
        const volatile PdTile& d = ring[n % PD_RING];
        // S overwrites P of tile n - 2: products of different shapes may
        // overlap, so the one that reads it has to be done
        if (n >= 2) ok = mbar_wait(&o_done[t], ((n - 2) >> 1) & 1, abort_flag, ERRW_TIMEOUT_MMA);
        if (!ok) return 0;
        const int fl = d.flags;
        if (fl & PD_END) {
          end = true;
          return fl;
        }
        if (fl & PD_FIRST_SEG) {
          ++seg;
          q_unit = d.q;
          ok = mbar_wait(&q_full[seg % PD_QS], (seg / PD_QS) & 1, abort_flag, ERRW_TIMEOUT_MMA);
          if (!ok) return 0;
        }
        steps = (d.nk + 15) >> 4;
        tc_fence_after();
        const uint32_t aQ = smem_u32(sQ + q_unit * 1024), aK = smem_u32(sK + st * PD_TILE);
        const uint32_t idesc = IDESC_S | (uint32_t)(2 * steps) << 17;  // N = 16 steps
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ss(tmem + t * 128, fa_desc_k(aQ, k), fa_desc_k(aK, k), idesc, k > 0 ? 1u : 0u);
        mma_commit(&s_full[t]);
        mma_commit(&k_empty[st]);
        if (fl & PD_LAST_SEG) mma_commit(&q_empty[seg % PD_QS]);
        return fl;
      };
      int fl = issue_s(0);
      for (int n = 0; ok && !end; ++n) {
        const int t = n & 1, st = n % PD_ST;
        const int fl_n = fl, steps_n = steps;
        fl = issue_s(n + 1);
        if (!ok) break;
        if (!mbar_wait(&v_full[st], (n / PD_ST) & 1, abort_flag, ERRW_TIMEOUT_MMA) ||
            !mbar_wait(&p_full[t], (n >> 1) & 1, abort_flag, ERRW_TIMEOUT_MMA) ||
            ((fl_n & PD_FIRST_ACC) &&
             !mbar_wait(&o_free[t], (used[t]++ & 1) ^ 1u, abort_flag, ERRW_TIMEOUT_MMA))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t aV = smem_u32(sV + st * PD_TILE);
        for (int k = 0; k < steps_n; ++k)
          mma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, fa_desc_mn(aV, k), IDESC_O,
                      (k > 0 || !(fl_n & PD_FIRST_ACC)) ? 1u : 0u);
        mma_commit(&v_empty[st]);
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
  } else if (warp < 8) {
    // ------------------------------------- softmax group t: tiles n % 2 == t
    const int t = warp >> 2;
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
      const int nk = dv.nk;
      const bool active = qw * 32 < dv.nrows;  // (the whole warp)
      if (flags & PD_FIRST_ACC) {
        m_used = -INFINITY;
        l = 0.f;
        if (a.window >= 0) oldest = r < dv.nrows ? dv.plen + a.lens[dv.b0 + r / G] - 1 - min(a.window, 1 << 30) : 0;
      }
      if (active) {
        tc_fence_after();
        const int lo = a.window >= 0 ? oldest - dv.pos : 0;  // the row sees keys lo .. nk-1 of the tile
        // 32 scores at a time, as far as the tile has keys, twice: for the
        // maximum, then for P (a whole row of 128 in registers spills, and the L1
        // beside this much shared memory is too small for that)
        uint32_t w[32];
        const auto scores = [&](int k) {
          tmem_ld_32x32b_x32(lane_addr + s_col + k, w);
          tmem_ld_wait();
          if (k + 32 > nk || __any_sync(0xffffffffu, lo > k)) {
            uint32_t seen = 0xffffffffu;  // bit i: the row sees key k + i
            if (k + 32 > nk) seen = 0xffffffffu >> (k + 32 - nk);
            if (lo > k) seen = lo - k < 32 ? seen & (0xffffffffu << (lo - k)) : 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = seen & (1u << i) ? w[i] : __float_as_uint(-INFINITY);
          }
        };
        float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int k = 0; k < nk; k += 32) {
          scores(k);
#pragma unroll
          for (int i = 0; i < 32; ++i) mp[i & 3] = fmaxf(mp[i & 3], __uint_as_float(w[i]));
        }
        const float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * sl2;
        // the running max moves only when it grows by more than 8 (base 2)
        const bool grow = mx > m_used + 8.f;
        const float corr = grow ? fast_exp2(m_used - mx) : 1.f;  // 0 when m_used is -inf
        if (grow) {
          l *= corr;
          m_used = mx;
        }
        const float mu = (m_used == -INFINITY) ? 0.f : m_used;
        // P as bf16 pairs over the first columns of S, 16 for 32 keys
        float lp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k < nk; k += 32) {
          if (nk > 32) scores(k);  // (a short tile's are still there)
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = fast_exp2(fmaf(__uint_as_float(w[2 * e]), sl2, -mu));
            const float p1 = fast_exp2(fmaf(__uint_as_float(w[2 * e + 1]), sl2, -mu));
            lp[(2 * e) & 3] += p0;
            lp[(2 * e + 1) & 3] += p1;
            pk[e] = pack_bf16(p0, p1);
          }
          tmem_st_32x32b_x16(lane_addr + s_col + k / 2, pk);
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
      // V rows behind the last key, up to its step of 16, are another
      // sequence's: they are zeroed (0 * NaN is NaN)
      if (nk & 15) {
        if (!mbar_wait_warp(&v_full[n % PD_ST], (n / PD_ST) & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE)) break;
        if (r >= nk && r < ((nk + 15) & ~15)) zero_tile_row(sV + n % PD_ST * PD_TILE, 16384, r);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
      if (flags & PD_LAST_ACC) {
        if (active) {
          if (!mbar_wait_warp(&o_done[t], c & 1, abort_flag, ERRW_TIMEOUT_EPILOGUE)) break;
          tc_fence_after();
          // (the tile's entry of the ring stays: its successor's K waits for S
          // of a tile after this group's next one)
          const int fl = dv.flags, nrows = dv.nrows, kvh = dv.kvh, b = dv.b0 + r / G;
          const int odd = fl & PD_ODD ? 1 : 0;
          float* rec;
          if (fl & PD_CONT)
            rec = a.rec_b + (((long long)cta * a.spt * G + r) * 2 + odd) * PD_REC;
          else
            rec = a.rec_a + ((((fl & PD_OWN ? 1ll : 0ll) * a.B + b) * a.H + kvh * G + r % G) * 2 + odd) * PD_REC;
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            uint32_t w[64];
            tmem_ld_32x32b_x32(lane_addr + o_col + k * 64, *reinterpret_cast<uint32_t(*)[32]>(&w[0]));
            tmem_ld_32x32b_x32(lane_addr + o_col + k * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&w[32]));
            tmem_ld_wait();
            if (r < nrows) {
#pragma unroll
              for (int g = 0; g < 16; ++g)
                *reinterpret_cast<float4*>(rec + k * 64 + g * 4) =
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
  if (warp == PD_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// o of (b, h) by one CTA from the keys that the window leaves it, in `part` as
// one sum per warp: sum of exp2(s - m) inv v, s in base 2, 4 columns per lane.
__device__ __noinline__ void prefix_alone(const PrefixArgs& a, int b, int h, float m, float inv, float (*part)[128]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane * 4, kvh = h / (a.H / a.Hkv);
  const PdSeq s = pd_seq(a, b);
  const int oldest = a.window < 0 ? 0 : (int)max(0ll, (long long)s.plen + s.len - 1 - a.window);  // position
  const auto load4 = [&](const bf16* p, float (&x)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + c);
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xffff0000u);
  };
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
  load4(a.q + ((long long)b * a.H + h) * 128, qv);
#pragma unroll 2
  for (int pos = oldest + warp; pos < s.plen + s.len; pos += 4) {
    const bool own = pos >= s.plen;
    const long long row = own ? (long long)b * a.T_max + pos - s.plen : (long long)s.p0 + pos;
    const long long at = row * (own ? (long long)a.Hkv * 128 : a.ld_prefix) + kvh * 128;
    float k[4], v[4];
    load4((own ? a.k_cache : a.k_prefix) + at, k);
    load4((own ? a.v_cache : a.v_prefix) + at, v);
    const float sc = warp_sum(fmaf(qv[0], k[0], fmaf(qv[1], k[1], fmaf(qv[2], k[2], qv[3] * k[3]))));
    const float p = fast_exp2(fmaf(sc, LOG2E / sqrtf(128.f), -m)) * inv;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(p, v[i], acc[i]);
  }
  *reinterpret_cast<float4*>(&part[warp][c]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
}

// One CTA per (sequence, head) joins its partial results, its four warps a
// quarter of them each: lane i takes the max and sum of the i-th one, then all
// lanes add up 4 columns each.
__global__ void __launch_bounds__(128)
    prefix_combine_kernel(const __grid_constant__ PrefixArgs a, bf16* __restrict__ o, float* __restrict__ lse, int nctas) {
  __shared__ float s_acc[4][128], s_m[4], s_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long bh = blockIdx.x;
  const int b = (int)(bh / a.H), h = (int)(bh - (long long)b * a.H);
  pdl_wait();  // (the partial results)
  const int G = a.H / a.Hkv, kvh = h / G, U = a.plan[a.B].x;
  const int4 mine = a.plan[b], tile = a.plan[mine.w];
  // the two segments: first unit, tiles, first and last CTA, row in its query tile
  struct Seg {
    int f, nt, c0, n, row;
  };
  const auto seg = [&](int f, int nt, int row) {
    Seg s{f, nt, 0, 0, row};
    if (nt > 0) {
      s.c0 = pd_owner(f, nctas, U);
      s.n = pd_owner(f + (nt > 1 ? PD_OPEN + PD_UNIT * (nt - 1) : 0), nctas, U) - s.c0 + 1;
    }
    return s;
  };
  const Seg pre = seg(tile.x + kvh * pd_units(tile.y), tile.y, (b - mine.w) * G + h - kvh * G);
  const Seg own = seg(mine.x + a.Hkv * pd_units(mine.y) + kvh * pd_units(max(mine.z, 0)), max(mine.z, 0), h - kvh * G);
  // partial results: two for each CTA of a segment, those of the prefix first
  int count = 2 * (pre.n + own.n);
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (mine.z < 0) count = 0;  // a length outside the cache
  for (int i0 = 0; i0 < count; i0 += 128) {
    const int i = i0 + lane * 4 + warp;
    const float* rec = nullptr;
    if (i < count) {
      const bool is_own = i >= 2 * pre.n;
      const Seg& s = is_own ? own : pre;
      const int x = i - (is_own ? 2 * pre.n : 0), c = s.c0 + (x >> 1), odd = x & 1;
      const int j0 = pd_tile(pd_begin(c, nctas, U) - s.f), j1 = min(s.nt, pd_tile(pd_begin(c + 1, nctas, U) - s.f));
      if (j1 - j0 > odd)  // the odd tiles' result exists if the CTA had two tiles
        rec = c == s.c0 ? a.rec_a + ((((is_own ? 1ll : 0ll) * a.B + b) * a.H + h) * 2 + odd) * PD_REC
                        : a.rec_b + (((long long)c * a.spt * G + s.row) * 2 + odd) * PD_REC;
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
    const int here = min(32, (count - i0 - warp + 3) / 4);
    for (int j0 = 0; j0 < here; j0 += 4) {  // four results' loads at a time, before their weights are needed
      float4 u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float* rj = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rec), (j0 + q) & 31));
        u[q] = rj && j0 + q < here ? *reinterpret_cast<const float4*>(rj + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float wj = __shfl_sync(0xffffffffu, w, (j0 + q) & 31);
        if (j0 + q < here && wj != 0.f) {
          acc[0] = fmaf(wj, u[q].x, acc[0]);
          acc[1] = fmaf(wj, u[q].y, acc[1]);
          acc[2] = fmaf(wj, u[q].z, acc[2]);
          acc[3] = fmaf(wj, u[q].w, acc[3]);
        }
      }
    }
  }
  *reinterpret_cast<float4*>(&s_acc[warp][lane * 4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  const float mm = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float sum = 0.f, x = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float w = s_m[q] == -INFINITY ? (s_l[q] == 0.f ? 0.f : 1.f) : fast_exp2(s_m[q] - mm);
    if (w != 0.f) {
      sum = fmaf(w, s_l[q], sum);
      x = fmaf(w, s_acc[q][threadIdx.x], x);
    }
  }
  float y = sum == 0.f ? 0.f : x / sum;
  // With a window the samples of a prompt see different rows of it, and a NaN or
  // infinity of V that this one does not see has met its P = 0 all the same.  (V
  // as large as 2^-8 of the type's largest may overflow before it is divided.)
  if (finite(sum) && __syncthreads_or(!finite(y))) {
    prefix_alone(a, b, h, mm, 1.f / sum, s_acc);
    __syncthreads();
    if (!finite(y)) y = (s_acc[0][threadIdx.x] + s_acc[1][threadIdx.x]) + (s_acc[2][threadIdx.x] + s_acc[3][threadIdx.x]);
  }
  o[bh * 128 + threadIdx.x] = __float2bfloat16_rn(y);
  if (threadIdx.x == 0 && lse) lse[bh] = sum == 0.f ? -INFINITY : (mm + log2f(sum)) * LN2;
}

}  // namespace gptb
