// swa_paged_fwd.cuh -- attention of packed new tokens over a paged cache, for
// sm_100a (tcgen05 MMAs, tensor-memory accumulators, TMA staging).
//
// Rows of a query tile: the G query heads of one key/value head at 128 / G
// consecutive tokens (row r is token r / G, head r % G), so a chunk of a few
// tokens fills its rows with heads, and a window of W keys is read for
// W + 128 / G positions.  A unit is two such tiles A and B on consecutive
// tokens of one sequence and one key/value head; both use the same key tiles
// but for the ends of their windows.
//
// Schedule: every unit's key tiles, one unit after another, are a list of T
// tiles (each unit counts kUnitCost more for its start and epilogue) that is
// cut into one run per CTA, so the SMs finish together whatever the lengths
// are, and a few rows over a long context are spread over all SMs.  A unit
// that a border cuts leaves unnormalised rows (output, running maximum and
// sum) that paged_fwd_merge_kernel joins.  Short units are not cut (keep_whole).
// Units are listed column by column of a matrix with one column per CTA, so CTAs that run
// at the same time read neighbouring windows, which L2 holds.
//
// Roles (384 threads):
//   warp 0    producer: Q_A, Q_B, then K and V tiles into their rings; lane i
//             looks the page of box i up a tile ahead and loads it.
//   warp 1    one thread issues every tcgen05.mma: S_X = Q_X K^T and
//             O_X += P_X V in the order PV_A(j), S_A(j+1), PV_B(j), S_B(j+1).
//             (A thread for A and one for B would decouple the two, but then their
//             MMAs and their softmaxes fall together instead of alternating: 667
//             against 460 us for a prompt of 8192 tokens.)
//   warp 2    scheduler: walks this CTA's run, 32 list entries at a time, and
//             hands the units to the other roles through a ring.
//   warp 3    zeroes the rows that no unit writes (outside the sequences, or of one that is
//             skipped), on request.
//   warps 4-7, 8-11   softmax and epilogue of tile A, tile B: a row per thread.
// Registers, tensor memory and the handshakes of S, P and O are those of
// fwd2_kernel (swa_fwd2.cuh).
//
// Slots that no query of a unit sees may hold anything.  Boxes without a
// visible slot are not read (a page out of the map's bounds loads zeros).  In
// the others an unseen key only reaches scores that the mask replaces; unseen
// value rows, which a zero weight would not silence (0 * NaN), are zeroed in
// shared memory by the softmax warps before they hand their weights over.
//
// Weights are rounded to bf16 for the second MMA (2^-9 of each on average, the price of
// its rate); scores, running maximum, sum and output stay in 32 bits.
//
// Bound: the chain S -> softmax -> PV of a tile, 1.6 us for both query tiles, where the
// MMAs and the exponentials of a step (2048 cycles each) would allow 1.1.  Measured with
// H / Hkv / d = 32 / 8 / 128: a prompt of 8192 tokens 443 us, 1240 TFLOP/s; 4 x 512 tokens
// over full 4096-key windows 134 us, 1025 (pages of 16 slots; 128 of 64 or more, 185 of 8, where a
// key tile takes 64 TMA instructions of 1 KB); 61 tokens over 130000 keys 129 us; five drafted
// tokens over 1000 keys (8 / 2 / 64) 11.2 us.  With d = 64 half the MMA work meets the same
// softmax: 4 x 512 tokens 109 us, the prompt 373.  Behind the last tile the merge takes 10.6 us
// where all borders cut a unit and 3 us where none does; a unit's start and epilogue cost
// about 5 us of its SM.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sm100.cuh"
#include "swa_epilogue.cuh"
#include "swa_fwd2.cuh"
#include "swa_paged.cuh"

namespace swa {

// Of a unit besides its key tiles, in key tiles.  (A start and epilogue take three tiles' time,
// but 2 and 3 measured like 1: within 1% on prompts, chunks and narrow windows, 2 to 4% either
// way on ragged batches.)
constexpr int kUnitCost = 1;
constexpr int kUnitRing = 4;   // units the scheduler is ahead

// n / d for n < 2^31 by a multiplication: mul = ceil(2^(31 + l) / d), l = ceil(log2 d),
// shift = 31 + l (the excess of mul adds n / 2^31 < 1 parts of 1 / d at most).
struct FastDiv {
  uint32_t mul, shift;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> shift);
  }
};

struct PagedFwdParams {
  __nv_bfloat16 *out;  // [total, H, D]
  float *lse;          // [H, total] or nullptr
  PagedCache c;
  int box_rows;  // slots per TMA box: a power of two that divides page_size, at most 128
  const int64_t *cu_seqlens, *q_start;
  int n_seq, total;
  int H, Hkv, G;
  int tpt;       // tokens per tile: 128 / G
  int g_inv;     // ceil(2^16 / G): r * g_inv >> 16 = r / G for r < 128
  FastDiv by_hkv, by_tu;  // divisions by Hkv and by a unit's 2 tpt tokens
  int n_slots;   // entries of the unit list, empty ones among them
  int W;         // clamped below 2^31 - 1024
  int n_sink, zero_rest;
  float scale_log2;
  // Partials: of a unit that starts before run c in slot 2c, of one that starts in
  // it and goes on in run c + 1 in slot 2c + 1.
  float4 *ws_o;   // [2P][2][D / 4][128]
  float2 *ws_ml;  // [2P][2][128] running maximum (base 2) and sum; sum 0: no key
  int4 *ws_run;   // [P] the unit that starts in run c and goes on: {first token, kv head,
                  //     tokens (0: none), the run after the last that holds a part}
};

template <int D>
struct PagedFwdLayout {
  static constexpr int PANELS = D / 64;
  static constexpr int NK = D == 64 ? 4 : 3, NV = D == 64 ? 4 : 2;  // K, V stages
  static constexpr uint32_t Q_BYTES = kQT * D * 2, KV_BYTES = kKT * D * 2;
  static constexpr uint32_t OFF_QA = 0, OFF_QB = Q_BYTES, OFF_K = 2 * Q_BYTES;
  static constexpr uint32_t OFF_V = OFF_K + NK * KV_BYTES;
  static constexpr uint32_t OFF_UNIT = OFF_V + NV * KV_BYTES;  // int4 [kUnitRing][4]
  static constexpr uint32_t OFF_BAR = OFF_UNIT + kUnitRing * 64;
  // q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], s_full[2], p_full[2],
  // p2_full[2], o_full[2], mma_drain, u_full[kUnitRing], u_empty[kUnitRing]
  static constexpr int NBAR = 2 + 2 * NK + 2 * NV + 9 + 2 * kUnitRing;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t ALLOC = OFF_MISC + 64 + 1024;  // + alignment
  static constexpr uint32_t TMEM_COLS = 512;
};

// One unit, as the scheduler hands it over: what its roles need, so that none of
// them computes it on its way from one unit to the next.
struct PagedUnit {
  int b, kvh, tok, ntok;  // sequence, key/value head, first packed token, tokens (0: the end)
  int qpos, t0, t1, n;    // position of the first token; the run's part [t0, t1) of n tiles
  // Key tiles in stream order: first + j, but tile 0 at j = 0 with `sink` (then first
  // is the window's first tile less one).
  int first, sink;
  int low, last;          // lowest key of any window, last position
  // Stream indices live for query tile A: t0 .. a_last (none if below t0); for B: b_first
  // (a sink tile, or the first of the rest) and b_from .. b_last (none if b_last < t0).
  int a_last, b_first, b_from, b_last;

  __device__ __forceinline__ int tile(int j) const { return sink && j == 0 ? 0 : first + j; }
  __device__ __forceinline__ bool live(int x, int j) const {
    return x == 0 ? j <= a_last : j <= b_last && (j >= b_from || j == b_first);
  }
  // after b .. n are set
  __device__ __forceinline__ void plan(const PagedFwdParams &p) {
    low = qpos - p.W + 1 > 0 ? qpos - p.W + 1 : 0;
    last = qpos + ntok - 1;
    first = low / kKT;
    sink = p.n_sink > 0 && first > 0 ? 1 : 0;
    first -= sink;
    const bool has_b = ntok > p.tpt;
    const int a_hi = has_b ? qpos + p.tpt - 1 : last;  // A's last position
    const int b_lo = qpos + p.tpt - p.W + 1;           // B's lowest key
    a_last = min(a_hi / kKT - first, t1 - 1);
    b_from = (b_lo > 0 ? b_lo : 0) / kKT - first;
    // every row of B sees the sinks, in key tile 0
    b_first = p.n_sink > 0 && tile(t0) == 0 ? t0 : max(b_from, t0);
    b_last = !has_b || b_first >= t1 ? t0 - 1 : (b_from < t1 ? t1 - 1 : b_first);
  }
};

// Whether tokens a .. e - 1 (e >= a), the first at position s, are a sequence that the call can
// compute.  An empty one may have any start: batches are padded with them.
__device__ __forceinline__ bool takes_sequence(const PagedFwdParams &p, int64_t a, int64_t e,
                                               int64_t s) {
  return a >= 0 && e <= p.total && (e == a || positions_fit(s, e - a, p.c.max_pos));
}

// Whether a sequence that the call computes holds token t (for offsets in order).
__device__ __forceinline__ bool writes_token(const PagedFwdParams &p, int64_t t) {
  if (t < p.cu_seqlens[0] || t >= p.cu_seqlens[p.n_seq]) return false;
  int lo = 0, hi = p.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_seqlens[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return takes_sequence(p, p.cu_seqlens[lo], p.cu_seqlens[lo + 1], p.q_start[lo]);
}

// Entry u of the unit list: sequence b owns the entries from base(b) * Hkv on, with
// base(b) = cu[b] / (tokens per unit) + b, which leaves room for its units on every
// key/value head without a sum over the sequences before it; what is left over
// is empty.  Sets b .. qpos and n and returns n, the unit's key tiles (0: an empty entry).
__device__ __forceinline__ int paged_unit(const PagedFwdParams &p, int u, PagedUnit &U) {
  if (u >= p.n_slots) return 0;
  const int tu = 2 * p.tpt;
  const uint32_t q = p.by_hkv(u);
  int lo = 0, hi = p.n_seq;  // the last sequence whose base is <= q, from the first on
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    // cu / tu + mid <= q  (for any cu the search stays in range)
    if (p.cu_seqlens[mid] < (static_cast<int64_t>(q) - mid + 1) * tu)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t a = p.cu_seqlens[lo], e = p.cu_seqlens[lo + 1], s = p.q_start[lo];
  if (e <= a || !takes_sequence(p, a, e, s)) return 0;
  const uint32_t b0 = p.by_tu(static_cast<uint32_t>(a)) + lo;
  if (q < b0) return 0;
  const uint32_t per = p.by_tu(static_cast<uint32_t>(e)) + lo + 1 - b0;
  const uint32_t rem = u - b0 * p.Hkv, kvh = rem / per, tok = (rem - kvh * per) * tu;
  const uint32_t len = static_cast<uint32_t>(e - a);
  if (kvh >= static_cast<uint32_t>(p.Hkv) || tok >= len) return 0;
  U.b = lo;
  U.kvh = static_cast<int>(kvh);
  U.tok = static_cast<int>(a) + static_cast<int>(tok);
  U.ntok = min(static_cast<int>(len - tok), tu);
  U.qpos = static_cast<int>(s) + static_cast<int>(tok);
  const int low = U.qpos - p.W + 1 > 0 ? U.qpos - p.W + 1 : 0, first = low / kKT;
  U.n = (U.qpos + U.ntok - 1) / kKT - first + 1 + (p.n_sink > 0 && first > 0 ? 1 : 0);
  return U.n;
}

// Whether a unit goes whole to the run in which it starts.  Cutting it balances the runs
// to a tile, but the parts of 148 cut units cost about 10 us (39 MB of partials written by
// this kernel and read by the merge, most of it behind the last tile), some 6 key tiles of an
// SM.  With units of equal cost the longest run exceeds T / P by the remainder to a whole
// unit.  Measured, cut against whole, one sequence with 32 own key/value heads (excess in
// tiles): window 512, 8191 tokens (3) 124 and 116 us, 4096 tokens (5) 70.5 and 69.3; window
// 128, 2047 tokens (2) 34 and 29; window 1024, 8191 tokens (5) 164 and 161.  Where a run is a
// tile or two (ten drafted tokens) cutting wins 11 us against 16: few parts are joined in 3 us.
//
// For units of unlike cost this is a prediction only: over 1000 random ragged batches that
// the rule takes (simulated), the longest run is more than 6 tiles above T / P in 25%, 12 at
// worst.  Measured, cut against whole, 32 sequences of 1 to 512 tokens with 32 and 8 own
// key/value heads: window 256 138 and 136 us, 100 and 101; window 512 168 and 170, 117 and
// 116; window 1024 228 and 237, 156 and 163.
constexpr int kWholeCost = 12, kWholeExcess = 6, kWholeRun = 3;
__device__ __forceinline__ bool keep_whole(int64_t T, int P, int most) {
  if (most > kWholeCost || T < kWholeRun * P || T >= (int64_t(1) << 31) || T == 0) return false;
  const uint32_t row = static_cast<uint32_t>(P) * most;
  const uint32_t rounds = (static_cast<uint32_t>(T) + row - 1) / row;
  return static_cast<int64_t>(rounds) * row - T <= kWholeExcess * P;
}

template <int D>
__global__ void __launch_bounds__(kFwd2Threads, 1)
    paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PagedFwdParams p) {
  using L = PagedFwdLayout<D>;
  constexpr int NK = L::NK, NV = L::NV;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - raw);
  const uint32_t sK = base + L::OFF_K, sV = base + L::OFF_V, bar = base + L::OFF_BAR;
  const uint32_t BAR_QF = bar, BAR_QE = bar + 8;
  const uint32_t BAR_KF = bar + 16;             // + 8 * K stage
  const uint32_t BAR_KE = BAR_KF + 8 * NK;      // + 8 * K stage
  const uint32_t BAR_VF = BAR_KE + 8 * NK;      // + 8 * V stage
  const uint32_t BAR_VE = BAR_VF + 8 * NV;      // + 8 * V stage
  const uint32_t BAR_S = BAR_VE + 8 * NV;       // + 8 * tile
  const uint32_t BAR_P = BAR_S + 16;            // + 8 * tile: first half of P stored
  const uint32_t BAR_P2 = BAR_P + 16;           // + 8 * tile: second half
  const uint32_t BAR_O = BAR_P2 + 16;           // + 8 * tile
  const uint32_t BAR_DRAIN = BAR_O + 16;        // the MMA thread's teardown
  const uint32_t BAR_UF = BAR_DRAIN + 8;        // + 8 * ring entry
  const uint32_t BAR_UE = BAR_UF + 8 * kUnitRing;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + L::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + L::OFF_MISC + 4);
  volatile int *skip_all = reinterpret_cast<volatile int *>(gbase + L::OFF_MISC + 24);
  int64_t *s_run = reinterpret_cast<int64_t *>(gbase + L::OFF_MISC + 8);  // entry, its offset
  int4 *s_unit = reinterpret_cast<int4 *>(gbase + L::OFF_UNIT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    mbar_init(BAR_QF, 1);
    mbar_init(BAR_QE, 1);
    for (int s = 0; s < NK; ++s) {
      mbar_init(BAR_KF + 8 * s, 1);
      mbar_init(BAR_KE + 8 * s, 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(BAR_VF + 8 * s, 1);
      mbar_init(BAR_VE + 8 * s, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(BAR_S + 8 * x, 1);
      mbar_init(BAR_P + 8 * x, 4 * 32);
      mbar_init(BAR_P2 + 8 * x, 4 * 32);
      mbar_init(BAR_O + 8 * x, 1);
    }
    mbar_init(BAR_DRAIN, 1);
    for (int s = 0; s < kUnitRing; ++s) {
      mbar_init(BAR_UF + 8 * s, 1);
      mbar_init(BAR_UE + 8 * s, 10);  // producer, MMA thread, eight softmax warps
    }
    *abort_flag = 0;
    *skip_all = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // This CTA's run: costs [T c / P, T (c + 1) / P) of the list, P the number of
  // CTAs or T if that is less.  List position s is column s / rows, row s % rows of
  // the matrix of units.  Every CTA sums the costs, a contiguous piece per thread.
  const int n_cols = gridDim.x, n_rows = (p.n_slots + n_cols - 1) / n_cols;
  const int n_list = n_rows * n_cols;
  auto entry = [&](int s) -> int {
    const int col = s / n_rows;
    return (s - col * n_rows) * n_cols + col;
  };
  int64_t T = 0, lo, hi;
  int P = 0;
  bool whole = false;
  {
    if (blockIdx.x == 0)  // sequences that are skipped
      for (int b = threadIdx.x; b < p.n_seq; b += kFwd2Threads) {
        const int64_t a = p.cu_seqlens[b], e = p.cu_seqlens[b + 1];
        if (e < a || !takes_sequence(p, a, e, p.q_start[b]))
          atomicOr(&g_swa_status, SWA_DEV_BADARG);
      }
    int64_t *s_warp = reinterpret_cast<int64_t *>(gbase);
    int *s_most = reinterpret_cast<int *>(gbase + 256);
    const int per = (n_list + kFwd2Threads - 1) / kFwd2Threads;
    const int s_lo = min(static_cast<int>(threadIdx.x) * per, n_list);
    const int s_hi = min(s_lo + per, n_list);
    // Two passes over one piece of code, which a launch meets cold: the sums, then the
    // entry in which this run begins (by the costs that the first pass left in shared
    // memory, as far as the K and V stages hold them).
    int *s_cost = reinterpret_cast<int *>(gbase + L::OFF_K);
    const bool stored = n_list <= static_cast<int>((NK + NV) * L::KV_BYTES / 4);
    const int col0 = s_lo / n_rows, row0 = s_lo - col0 * n_rows;
    int64_t sum = 0, at = 0;
    int most = 0;  // the largest cost of a unit
    lo = hi = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      if (pass == 0 || (hi > lo && lo >= at && lo < at + sum)) {
        int64_t acc = at;
        int col = col0, row = row0;
#pragma unroll 1
        for (int s = s_lo; s < s_hi; ++s) {
          int cost;
          if (pass && stored) {
            cost = s_cost[s];
          } else {
            PagedUnit U;
            const int n = paged_unit(p, row * n_cols + col, U);
            cost = n ? n + kUnitCost : 0;
            if (stored) s_cost[s] = cost;
            most = max(most, cost);
            if (++row == n_rows) {
              row = 0;
              ++col;
            }
          }
          if (pass && lo < acc + cost) {
            s_run[0] = s;
            s_run[1] = acc;
            break;
          }
          acc += cost;
        }
        if (pass == 0) sum = acc;
      }
      if (pass) break;
      int64_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 31) {
        s_warp[warp] = incl;
        s_most[warp] = most;
      }
      __syncthreads();
      at = incl - sum;
      for (int w = 0; w < kFwd2Threads / 32; ++w) {
        if (w < warp) at += s_warp[w];
        T += s_warp[w];
        most = max(most, s_most[w]);
      }
      const int c = blockIdx.x;
      P = T < n_cols ? static_cast<int>(T) : n_cols;
      lo = c < P ? mul_div(T, c, P) : 0;
      hi = c < P ? mul_div(T, c + 1, P) : 0;
      whole = keep_whole(T, P, most);
    }
  }
  // With offsets out of order the list loses some sequences and tokens can be in several: every
  // CTA sees it, and has no unit then.
  for (int b = threadIdx.x; b < p.n_seq; b += kFwd2Threads)
    if (p.cu_seqlens[b + 1] < p.cu_seqlens[b]) *skip_all = 1;
  // the costs above lie where copies of the async proxy write from here on
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Next unit from the scheduler; false at the end of the run.  Each warp (or
  // thread) that takes it frees it with unit_done.
  auto unit_load = [&](int it, PagedUnit &U) -> bool {
    const int4 *e = s_unit + 4 * (it % kUnitRing);
    const int4 a = e[0], c = e[1], d = e[2], f = e[3];
    U.b = a.x;
    U.kvh = a.y;
    U.tok = a.z;
    U.ntok = a.w;
    U.qpos = c.x;
    U.t0 = c.y;
    U.t1 = c.z;
    U.n = c.w;
    U.first = d.x;
    U.sink = d.y;
    U.low = d.z;
    U.last = d.w;
    U.a_last = f.x;
    U.b_first = f.y;
    U.b_from = f.z;
    U.b_last = f.w;
    return U.ntok > 0;
  };
  auto unit_bar = [&](int it) -> uint32_t { return BAR_UF + 8 * (it % kUnitRing); };
  auto unit_done = [&](int it) { mbar_arrive(BAR_UE + 8 * (it % kUnitRing)); };

  if (warp < 4) {
    warpgroup_regs_dec<kRegsControl>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      const int boxes = kKT / p.box_rows;  // per tile, at most 16
      const uint32_t q_bytes = p.tpt * p.G * 128 * L::PANELS;
      int kv = 0, q_iter = 0;
      bool k_ahead = false;  // K of tile kv issued, its V not (abort between them)
      bool ok = true;
      for (int it = 0; ok; ++it) {
        PagedUnit U;
        if (!mbar_wait_warp(unit_bar(it), (it / kUnitRing) & 1, abort_flag)) break;
        const bool any = unit_load(it, U);
        __syncwarp();
        if (lane == 0) unit_done(it);
        if (!any) break;
        const int32_t *row = p.c.table + U.b * p.c.table_stride;
        // this lane's box of tile j: its page and first slot (-1: no visible key lies there)
        auto look_up = [&](int j, int &slot) -> int {
          slot = -1;
          if (j >= U.t1 || lane >= boxes) return 0;
          const int at = U.tile(j) * kKT + lane * p.box_rows;
          if (at > U.last || (at + p.box_rows <= U.low && at >= p.n_sink)) return 0;
          const int pg = at / p.c.page_size;
          slot = at - pg * p.c.page_size;
          return row[pg];
        };
        int slot, page = look_up(U.t0, slot);
        if (lane == 0) {
          ok = q_iter == 0 || mbar_wait(BAR_QE, (q_iter - 1) & 1, abort_flag);
          if (ok) {
            const bool has_b = U.ntok > p.tpt;
            mbar_expect_tx(BAR_QF, (has_b ? 2 : 1) * q_bytes);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x == 1 && !has_b) break;
#pragma unroll
              for (int pn = 0; pn < L::PANELS; ++pn)
                tma_load_3d(base + L::OFF_QA + x * L::Q_BYTES + pn * (kQT * 128), &tm_q, BAR_QF,
                            pn * 64, U.kvh * p.G, U.tok + x * p.tpt);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        ++q_iter;
        for (int j = U.t0; j < U.t1; ++j) {
          int slot_n;
          const int page_n = look_up(j + 1, slot_n);  // a tile ahead of its use
          const int sk = kv % NK, sv = kv % NV;
          if (lane == 0) {
            ok = kv < NK || mbar_wait(BAR_KE + 8 * sk, ((kv / NK) - 1) & 1, abort_flag);
            if (ok) mbar_expect_tx(BAR_KF + 8 * sk, L::KV_BYTES);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          // a page out of the map's bounds reads as zeros
          if (slot < 0) {
            slot = 0;
            page = p.c.n_pages;
          } else if (page < 0 || page >= p.c.n_pages) {
            atomicOr(&g_swa_status, SWA_DEV_BADARG);
            page = p.c.n_pages;
          }
          const uint32_t off = lane * p.box_rows * 128;
          if (lane < boxes) {
#pragma unroll
            for (int pn = 0; pn < L::PANELS; ++pn)
              tma_load_5d(sK + sk * L::KV_BYTES + pn * (kKT * 128) + off, &tm_k, BAR_KF + 8 * sk,
                          0, slot, pn, U.kvh, page);
          }
          if (lane == 0) {
            ok = kv < NV || mbar_wait(BAR_VE + 8 * sv, ((kv / NV) - 1) & 1, abort_flag);
            if (ok) mbar_expect_tx(BAR_VF + 8 * sv, L::KV_BYTES);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) {
            k_ahead = true;
            break;
          }
          if (lane < boxes) {
#pragma unroll
            for (int pn = 0; pn < L::PANELS; ++pn)
              tma_load_5d(sV + sv * L::KV_BYTES + pn * (kKT * 128) + off, &tm_v, BAR_VF + 8 * sv,
                          0, slot, pn, U.kvh, page);
          }
          ++kv;
          page = page_n;
          slot = slot_n;
        }
      }
      // every copy issued must land before the CTA ends
      if (lane == 0) {
        if (q_iter > 0) mbar_drain(BAR_QF, (q_iter - 1) & 1);
        const int k_issued = kv + (k_ahead ? 1 : 0);
        for (int i = max(0, k_issued - NK); i < k_issued; ++i)
          mbar_drain(BAR_KF + 8 * (i % NK), (i / NK) & 1);
        for (int i = max(0, kv - NV); i < kv; ++i)
          mbar_drain(BAR_VF + 8 * (i % NV), (i / NV) & 1);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      if (elect_one()) {
        constexpr uint32_t idS = idesc_bf16_f32(kQT, kKT, false);
        constexpr uint32_t idO = idesc_bf16_f32(kQT, D, true);
        constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
        const uint32_t q_lo[2] = {sdesc_sw128_lo(base + L::OFF_QA, 16),
                                  sdesc_sw128_lo(base + L::OFF_QB, 16)};
        const uint32_t k_lo = sdesc_sw128_lo(sK, 16), v_lo = sdesc_sw128_lo(sV, kKT * 128);
        int kv = 0, q_iter = 0;
        uint32_t p_cnt[2] = {0u, 0u};
        // (the empty asm keeps the compiler from precomputing every MMA's words)
        auto issue_s = [&](int x, int st) {
          uint32_t qb = q_lo[x], kb = k_lo + st * (L::KV_BYTES >> 4), dS = tmem + x * 128;
          asm volatile("" : "+r"(qb), "+r"(kb), "+r"(dS));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (kKT * 128) + (kk & 3) * 32;
            mma_ss_w(dS, qb + (off >> 4), kb + (off >> 4), kDescHi, idS, kk > 0 ? 1u : 0u);
          }
          tc_commit(BAR_S + 8 * x);
        };
        auto issue_pv = [&](int x, int st, bool acc, int half) {
          uint32_t dO = tmem + 256 + x * D, aP = tmem + x * 128;
          uint32_t vb = v_lo + st * (L::KV_BYTES >> 4);
          asm volatile("" : "+r"(vb), "+r"(dO), "+r"(aP));
#pragma unroll
          for (int k16 = 0; k16 < kKT / 32; ++k16) {
            const int kk = half * (kKT / 32) + k16;
            mma_ts_w(dO, aP + kk * 8, vb + ((kk * 16 * 128) >> 4), kDescHi, idO,
                     (acc || kk > 0) ? 1u : 0u);
          }
        };
        auto pv_tile = [&](int x, int st, bool acc) -> bool {
          if (!mbar_wait(BAR_P + 8 * x, p_cnt[x] & 1, abort_flag)) return false;
          tc_fence_after();
          issue_pv(x, st, acc, 0);
          if (!mbar_wait(BAR_P2 + 8 * x, p_cnt[x] & 1, abort_flag)) return false;
          tc_fence_after();
          issue_pv(x, st, true, 1);
          ++p_cnt[x];
          return true;
        };
        auto k_wait = [&](int i) -> bool {
          if (!mbar_wait(BAR_KF + 8 * (i % NK), (i / NK) & 1, abort_flag)) return false;
          tc_fence_after();
          return true;
        };
        for (int it = 0;; ++it) {
          PagedUnit U;
          if (!mbar_wait(unit_bar(it), (it / kUnitRing) & 1, abort_flag)) break;
          const bool any = unit_load(it, U);
          unit_done(it);
          if (!any) break;
          if (!mbar_wait(BAR_QF, q_iter & 1, abort_flag)) break;
          tc_fence_after();
          int j = U.t0;
          bool ca = U.live(0, j), cb = U.live(1, j), have = true, has_next = ++j < U.t1;
          bool na = has_next && U.live(0, j), nb = has_next && U.live(1, j);
          if (!k_wait(kv)) break;
          if (ca) issue_s(0, kv % NK);
          if (cb) issue_s(1, kv % NK);
          // tile B starting one key tile after A: its first S now instead of behind A's
          // first softmax
          bool b_ahead = false;
          if (has_next && nb && !cb) {
            if (!k_wait(kv + 1)) break;
            issue_s(1, (kv + 1) % NK);
            b_ahead = true;
          }
          tc_commit(BAR_KE + 8 * (kv % NK));
          bool first[2] = {true, true};
          bool stop = false;  // a wait gave up: issue nothing more
          while (have) {
            if (!has_next) tc_commit(BAR_QE);  // every S of this unit is issued
            const int sv = kv % NV, skn = (kv + 1) % NK;
            if (!mbar_wait(BAR_VF + 8 * sv, (kv / NV) & 1, abort_flag)) {
              stop = true;
              break;
            }
            if (ca) {
              if (!pv_tile(0, sv, !first[0])) {
                stop = true;
                break;
              }
              first[0] = false;
              // o_full completes once per unit in which the tile had work; its next
              // completion needs that tile's softmax to hand over its next P
              if (j - 1 == U.a_last) tc_commit(BAR_O);
            }
            if (has_next) {
              if (!k_wait(kv + 1)) {
                stop = true;
                break;
              }
              if (na) issue_s(0, skn);
            }
            if (cb) {
              if (!pv_tile(1, sv, !first[1])) {
                stop = true;
                break;
              }
              first[1] = false;
              if (j - 1 == U.b_last) tc_commit(BAR_O + 8);
            }
            tc_commit(BAR_VE + 8 * sv);  // V(j) is read by both PV MMAs
            if (has_next) {
              if (nb && !b_ahead) issue_s(1, skn);
              b_ahead = false;
              tc_commit(BAR_KE + 8 * skn);
            }
            ++kv;
            ca = na;
            cb = nb;
            have = has_next;
            has_next = ++j < U.t1;
            na = has_next && U.live(0, j);
            nb = has_next && U.live(1, j);
          }
          if (stop) break;
          ++q_iter;
        }
        // every MMA issued must complete before the tensor memory is freed
        tc_commit(BAR_DRAIN);
        mbar_drain(BAR_DRAIN, 0);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------------- scheduler
      if (lane == 0) p.ws_run[blockIdx.x] = make_int4(0, 0, 0, 0);
      __syncwarp();
      int it = 0;
      bool ok = true;
      auto publish = [&](const PagedUnit &U) -> bool {
        const int r = it % kUnitRing;
        if (it >= kUnitRing &&
            !mbar_wait(BAR_UE + 8 * r, ((it / kUnitRing) - 1) & 1, abort_flag))
          return false;
        s_unit[4 * r] = make_int4(U.b, U.kvh, U.tok, U.ntok);
        s_unit[4 * r + 1] = make_int4(U.qpos, U.t0, U.t1, U.n);
        s_unit[4 * r + 2] = make_int4(U.first, U.sink, U.low, U.last);
        s_unit[4 * r + 3] = make_int4(U.a_last, U.b_first, U.b_from, U.b_last);
        mbar_arrive(BAR_UF + 8 * r);
        return true;
      };
      if (hi > lo && !*skip_all) {
        int s = static_cast<int>(s_run[0]);
        int64_t at = s_run[1];
        while (ok && at < hi && s < n_list) {
          PagedUnit U;
          const int n = s + lane < n_list ? paged_unit(p, entry(s + lane), U) : 0;
          const int cost = n ? n + kUnitCost : 0;
          int incl = cost;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
          }
          const int64_t a = at + incl - cost;  // the unit's tiles are costs [a, a + n)
          if (whole) {  // its start decides
            U.t0 = 0;
            U.t1 = a >= lo && a < hi ? n : 0;
          } else {
            U.t0 = lo - a <= 0 ? 0 : (lo - a < n ? static_cast<int>(lo - a) : n);
            U.t1 = hi - a <= 0 ? 0 : (hi - a < n ? static_cast<int>(hi - a) : n);
          }
          if (n) U.plan(p);
          uint32_t todo = __ballot_sync(0xffffffffu, n && U.t0 < U.t1);
          for (; todo && ok; todo &= todo - 1, ++it) {
            const int i = __ffs(todo) - 1;
            if (lane == i) ok = publish(U);
            ok = __shfl_sync(0xffffffffu, ok, i);
          }
          if (n && U.t0 == 0 && U.t1 > 0 && U.t1 < n)
            // run j begins inside iff floor(T j / P) < a + n iff j < (a + n) P / T
            p.ws_run[blockIdx.x] = make_int4(U.tok, U.kvh, U.ntok,
                                             static_cast<int>(((a + n) * P + T - 1) / T));
          at += __shfl_sync(0xffffffffu, incl, 31);
          s += 32;
        }
      }
      PagedUnit none = {};
      if (ok && lane == 0) publish(none);
    } else if (p.zero_rest) {
      // ---------------------------------------------------------------- rows outside
      // Tokens of padding and of skipped sequences: 32 are looked up at once, one per lane, a
      // grid apart, so that a stretch of them is spread over all CTAs.
      const int64_t apart = gridDim.x;
      for (int64_t t0 = blockIdx.x; t0 < p.total; t0 += 32 * apart) {
        const int64_t mine = t0 + lane * apart;
        const bool rest = mine < p.total && (*skip_all || !writes_token(p, mine));
        for (uint32_t m = __ballot_sync(0xffffffffu, rest); m; m &= m - 1) {
          const int64_t t = t0 + (__ffs(m) - 1) * apart;
          for (int j = lane; j < p.H * (D / 8); j += 32)
            reinterpret_cast<uint4 *>(p.out + t * p.H * D)[j] = make_uint4(0, 0, 0, 0);
          if (p.lse)
            for (int j = lane; j < p.H; j += 32) p.lse[static_cast<int64_t>(j) * p.total + t] = 0;
        }
      }
    }
  } else {
    warpgroup_regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax + epilogue
    const int x = warp < 8 ? 0 : 1;  // query tile of this warp group
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const int row_t = row * p.g_inv >> 16;  // token of the row within its tile
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off;
    const uint32_t tO = tmem + 256 + x * D + lane_off;
    uint32_t s_cnt = 0, u_iter = 0;
    int kv0 = 0;        // K/V tiles of the units before
    bool stop = false;  // a wait gave up (the whole warp): no more TMEM work or stores
    for (int it = 0;; ++it) {
      PagedUnit U;
      if (!mbar_wait_warp(unit_bar(it), (it / kUnitRing) & 1, abort_flag)) break;
      const bool any = unit_load(it, U);
      __syncwarp();
      if (lane == 0) unit_done(it);
      if (!any) break;
      const int qlo = U.qpos + x * p.tpt, qhi = min(qlo + p.tpt - 1, U.last);
      const int qrow = qlo + row_t;
      float m_run = -INFINITY, l_run = 0.f;
      int nt = 0;
      for (int j = U.t0; j < U.t1; ++j) {
        if (!U.live(x, j)) continue;
        const int k = U.tile(j);
        if (!mbar_wait_warp(BAR_S + 8 * x, s_cnt & 1, abort_flag)) {
          stop = true;
          break;
        }
        ++s_cnt;
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld128(tS, sr);
        float *s = reinterpret_cast<float *>(sr);
        const int k0 = k * kKT;
        if (k0 + kKT - 1 > qlo || k0 < qhi - p.W + 1) {
          // allowed columns of this row: key k0 + c in [q - W + 1, q] or below n_sink
          const int hi_c = qrow - k0, lo_c = hi_c - p.W + 1;
          const int sink_c = k == 0 ? min(p.n_sink - 1, qrow) : -1;
          uint32_t mw[kKT / 32];
#pragma unroll
          for (int i = 0; i < kKT / 32; ++i)
            mw[i] = range_bits(lo_c - 32 * i, hi_c - 32 * i) | range_bits(-32 * i, sink_c - 32 * i);
#pragma unroll
          for (int c = 0; c < kKT; ++c) s[c] = ((mw[c >> 5] >> (c & 31)) & 1u) ? s[c] : -INFINITY;
          if (k0 + kKT - 1 > U.last || k0 < U.low) {
            // value rows that no query of the unit sees (one row per thread, its pieces
            // in an order that spreads a warp over the banks)
            const int i = kv0 + j - U.t0;
            if (!mbar_wait_warp(BAR_VF + 8 * (i % NV), (i / NV) & 1, abort_flag)) {
              stop = true;
              break;
            }
            const int key = k0 + row;
            if (key > U.last || (key < U.low && key >= p.n_sink)) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                st_shared_v4(sV + (i % NV) * L::KV_BYTES + (c >> 3) * (kKT * 128) + row * 128 +
                                 (((c + lane) & 7) << 4),
                             0, 0, 0, 0);
            }
            fence_async_smem();
          }
        }
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = s[i];
#pragma unroll
        for (int c = 8; c + 16 <= kKT; c += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i) mx[i] = max3(mx[i], s[c + i], s[c + 8 + i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], s[kKT - 8 + i]);
        const float m_raw = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]),
                                 fmaxf(mx[6], mx[7]));
        const float m_tile = m_raw * p.scale_log2;
        const bool grow = m_tile > m_run + kLazyRescaleLog2;
        const float m_new = grow ? m_tile : m_run;
        const float alpha = grow ? ex2(m_run - m_new) : 1.f;
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        // x = s * scale * log2(e) - m, two columns per packed FMA
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nm2 = make_float2(-m_use, -m_use);
        float2 *s2 = reinterpret_cast<float2 *>(s);
#pragma unroll
        for (int c = 0; c < kKT / 2; ++c) s2[c] = __ffma2_rn(s2[c], sc2, nm2);
        // P of keys 64h .. 64h + 63 as bf16 pairs (key 2c in the low half of
        // column c) into columns 32h .. 32h + 31 of S_X; no wait
        auto store_p = [&](int h) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) pk[i] = pack_bf16(s[h * 64 + 2 * i], s[h * 64 + 2 * i + 1]);
          tmem_st32(tS + h * 32, pk);
        };
        auto rescale_o = [&](float a) {
#pragma unroll 1
          for (int cb2 = 0; cb2 < D / 32; ++cb2) {
            uint32_t o32[32];
            tmem_ld32(tO + cb2 * 32, o32);
#pragma unroll
            for (int i = 0; i < 32; ++i) o32[i] = __float_as_uint(__uint_as_float(o32[i]) * a);
            tmem_st32(tO + cb2 * 32, o32);
          }
        };
        // O_X is stable (PV_X of the previous tile was issued before this
        // S_X): rescale it before the first half of P hands PV_X the tile
        if (nt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) rescale_o(alpha);
        // exponentials on the MUFU (a masked column gives 2^-inf = 0) in two
        // halves of 64 keys; P of the first half (bf16 pairs, key 2c in the
        // low half of column c) goes to PV_X while the second is computed
        float2 sm2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sm2[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
#pragma unroll
          for (int c = h2 * 64; c < h2 * 64 + 64; ++c) s[c] = ex2(s[c]);
#pragma unroll
          for (int c = h2 * 32; c < h2 * 32 + 32; c += 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) sm2[i] = __fadd2_rn(sm2[i], s2[c + i]);
          store_p(h2);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(h2 == 0 ? BAR_P + 8 * x : BAR_P2 + 8 * x);
        }
        const float2 sa = __fadd2_rn(__fadd2_rn(sm2[0], sm2[1]), __fadd2_rn(sm2[2], sm2[3]));
        l_run = l_run * alpha + (sa.x + sa.y);
        m_run = m_new;
        ++nt;
      }
      if (stop) break;
      kv0 += U.t1 - U.t0;
      const int rows = min(p.tpt, U.ntok - x * p.tpt) * p.G;  // valid rows (<= 0: no tile B)
      const int tok0 = U.tok + x * p.tpt;
      if (nt > 0) {  // every PV of this unit is done
        if (!mbar_wait_warp(BAR_O + 8 * x, u_iter & 1, abort_flag)) break;
        ++u_iter;
        tc_fence_after();
      }
      if (U.t1 - U.t0 < U.n) {
        // a part: this row's unnormalised O with its running maximum and sum
        const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (U.t0 > 0 ? 0 : 1)) * 2 + x;
        if (nt > 0) {
          float4 *po = p.ws_o + slot * (D / 4) * kQT + row;
#pragma unroll 1
          for (int c32 = 0; c32 < D / 32; ++c32) {
            uint32_t o32[32];
            tmem_ld32(tO + c32 * 32, o32);
            if (row < rows)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                po[(c32 * 8 + i) * kQT] =
                    make_float4(__uint_as_float(o32[4 * i]), __uint_as_float(o32[4 * i + 1]),
                                __uint_as_float(o32[4 * i + 2]), __uint_as_float(o32[4 * i + 3]));
          }
        }
        if (row < rows)
          p.ws_ml[slot * kQT + row] = make_float2(m_run, nt > 0 ? l_run : 0.f);
      } else if (rows > 0) {
        const float inv_l = 1.f / l_run;
        // rows of this lane's 8-lane group: whole 128-byte segments per store
        const int grp = quad * 32 + (lane & ~7);
        __nv_bfloat16 *o0 = p.out + (static_cast<int64_t>(tok0) * p.H + U.kvh * p.G) * D +
                            8 * (lane & 7);
#pragma unroll 1
        for (int h2 = 0; h2 < D / 64; ++h2) {
          uint32_t e[32];
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
            uint32_t o32[32];
            tmem_ld32(tO + h2 * 64 + c2 * 32, o32);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              e[c2 * 16 + i] = pack_bf16(__uint_as_float(o32[2 * i]) * inv_l,
                                         __uint_as_float(o32[2 * i + 1]) * inv_l);
          }
          transpose8_pieces(e, lane);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = grp + i, t = r * p.g_inv >> 16;
            if (r < rows)
              *reinterpret_cast<uint4 *>(o0 + (static_cast<int64_t>(t) * p.H + r - t * p.G) * D +
                                         h2 * 64) =
                  make_uint4(e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3]);
          }
        }
        if (p.lse && row < rows)
          p.lse[static_cast<int64_t>(U.kvh * p.G + row - row_t * p.G) * p.total + tok0 + row_t] =
              (m_run + __log2f(l_run)) * 0.6931471805599453f;
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Joins the parts of the unit that starts in run blockIdx.x and goes on, a row per
// thread and 8 columns: run c's slot 2c + 1, then the slots 2j of the runs that
// follow.  Four parts of 8 columns are in flight per thread: two of 16 columns lose 4 us
// where a unit has ten parts (61 tokens over 130000 keys), four of 16 columns keep half as
// many threads on an SM and lose 1 to 2 us where units have two.
constexpr int kMergeThreads = 512;  // 128 rows, 32 columns
constexpr int kMergeCols = 8;
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 2) paged_fwd_merge_kernel(const PagedFwdParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int N = kMergeCols / 4, B = 4;  // float4 columns per thread; parts in flight
  const int c = blockIdx.x, x = blockIdx.y, row = threadIdx.x % kQT;
  const int col4 = (blockIdx.z * (kMergeThreads / kQT) + threadIdx.x / kQT) * N;
  const int4 run = p.ws_run[c];
  const int rows = min(p.tpt, run.z - x * p.tpt) * p.G;
  if (row >= rows) return;
  float m = -INFINITY, l = 0.f;
  float4 acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = c; j0 < run.w; j0 += B) {
    float2 ml[B];
    float4 o[B][N];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      if (j0 + u < run.w) {
        const int64_t slot = (j0 + u == c ? 2 * c + 1 : 2 * (j0 + u)) * 2 + x;
        ml[u] = p.ws_ml[slot * kQT + row];
#pragma unroll
        for (int i = 0; i < N; ++i) o[u][i] = p.ws_o[(slot * (D / 4) + col4 + i) * kQT + row];
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < B; ++u)
      if (ml[u].y != 0.f) mn = fmaxf(mn, ml[u].x);
    const float w0 = m == -INFINITY ? 0.f : ex2(m - mn);
    l *= w0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      acc[i].x *= w0;
      acc[i].y *= w0;
      acc[i].z *= w0;
      acc[i].w *= w0;
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      // the part gave this row no key: its O may not be written (a sum that is NaN stays in)
      if (ml[u].y == 0.f) continue;
      const float w = ex2(ml[u].x - mn);
      l = fmaf(ml[u].y, w, l);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        acc[i].x = fmaf(o[u][i].x, w, acc[i].x);
        acc[i].y = fmaf(o[u][i].y, w, acc[i].y);
        acc[i].z = fmaf(o[u][i].z, w, acc[i].z);
        acc[i].w = fmaf(o[u][i].w, w, acc[i].w);
      }
    }
    m = mn;
  }
  const int t = row * p.g_inv >> 16, h = run.y * p.G + row - t * p.G;
  const int64_t tok = run.x + x * p.tpt + t;
  const float inv = 1.f / l;
  uint4 *dst = reinterpret_cast<uint4 *>(p.out + (tok * p.H + h) * D + col4 * 4);
#pragma unroll
  for (int i = 0; i < N; i += 2)
    dst[i / 2] = make_uint4(pack_bf16(acc[i].x * inv, acc[i].y * inv),
                            pack_bf16(acc[i].z * inv, acc[i].w * inv),
                            pack_bf16(acc[i + 1].x * inv, acc[i + 1].y * inv),
                            pack_bf16(acc[i + 1].z * inv, acc[i + 1].w * inv));
  if (p.lse && col4 == 0)
    p.lse[static_cast<int64_t>(h) * p.total + tok] = (m + __log2f(l)) * 0.6931471805599453f;
}

}  // namespace swa
