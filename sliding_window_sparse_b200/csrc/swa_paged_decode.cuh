// swa_paged_decode.cuh -- batched single-token decode over a paged cache.
//
// The cost of a decode step is reading the visible keys and values
// (sparse-attention taxonomy page, section 1): once for up to 16 query heads
// per key/value head, ceil(G / 16) times for more, since a block of 16 heads is
// a unit of its own.  The work of a call is the list
// of 128-key tiles of every (sequence, key/value head, block of 16 query
// heads); each CTA, one per SM, takes one contiguous run of that list, so all
// of them stream the same number of bytes whatever the lengths are.  A unit
// that a run's border cuts leaves one unnormalised partial per run (output,
// running maximum and sum); paged_decode_merge_kernel joins them.
//
// Roles (288 threads): warp 8 is the producer, which looks pages up one tile
// ahead and keeps a ring of tiles in flight (TMA, 192 KB at d = 128: the loads
// cover the latency of HBM, the arithmetic only has to keep up).  Warps 0-7
// take 16 keys each of every tile, with a softmax state of their own that is
// joined at the end of a unit:
//   S [16 heads x 16 keys] = Q K^T,   O [16 heads x d] += P V
// on mma.sync m16n8k16.  A tile needs 256 of them for 64 KB, which an SM
// receives in about 2800 cycles: they take under a quarter of that time at the
// legacy rate, and unlike an M = 128 tcgen05 tile they leave scores and output
// in the registers of the warp that needs them.  Query heads beyond G fill the
// 16 rows with zeros.
//
// P goes in as two terms of 16 bits, the second one the rounding of the first,
// so a weight loses 2^-16 where one term would lose 2^-8.  Up to 8 query heads
// leave rows 8-15 free: the second terms fill them, and the two halves of O are
// added in the end.  More heads take a second MMA per fragment (384 a tile).
//
// Measured (H / Hkv / d = 32 / 8 / 128): 64 sequences of 4096-key windows in pages of
// 16 slots 171 us, 6.3 TB/s (a copy reaches 6.56); 24 sequences of up to 100000 keys with
// 64 query heads in pages of 64 slots 757 us, 7.1 TB/s; one sequence of 1000 keys 8.8 us,
// the latency of two launches, the page table, one tile and the merge (2.5 us).  The 64
// sequences with 16 heads a group 181 us, with 20 330 and with 32 337; with d = 64 92 us in
// pages of 64 slots, 5.8 TB/s, and 136 in pages of 16, whose boxes of 2 KB are bound by
// the rate of TMA instructions.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "sm100.cuh"
#include "swa_paged.cuh"

namespace swa {

constexpr int kPDThreads = 288;
constexpr int kPDWarps = 8;   // consumer warps
constexpr int kPDKeys = 128;  // keys per tile
constexpr int kPDRows = 16;   // query heads per unit

struct PagedDecodeParams {
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  float *lse;  // or nullptr
  const int64_t *pos;
  PagedCache c;
  int box_rows;  // slots per TMA box: a power of two that divides page_size, at most 128
  int B, H, Hkv, G, HB;  // HB: blocks of 16 query heads per key/value head
  int n_sink;
  int64_t W;
  float scale_log2;
  // Partials: of a unit that starts before run c in slot 2c, of one that starts in
  // it and goes on in run c + 1 in slot 2c + 1.
  float *ws_o;    // [2P][16][D]
  float2 *ws_ml;  // [2P][16] running maximum (base 2) and sum
  int2 *ws_run;   // [P] {the unit that starts in run c and goes on, or -1; the run
                  //      after the last that holds a part of it}
};

template <int D>
struct PagedDecodeLayout {
  static constexpr int PANELS = D / 64;
  static constexpr uint32_t TILE = kPDKeys * D * 2;  // K or V
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr uint32_t OFF_RED = STAGES * 2 * TILE;  // [8][16][64] or [8][8][128] fp32
  static constexpr uint32_t OFF_ML = OFF_RED + 32768;     // [8][16] float2
  static constexpr uint32_t OFF_BAR = OFF_ML + 1024;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 2 * STAGES * 8;
  static constexpr uint32_t ALLOC = OFF_MISC + 64 + 1024;  // + alignment
};

// The 128-key tiles that hold a key visible at position pos: those of the
// window, behind tile 0 if it holds sinks that the window's tiles do not.
struct PagedSpan {
  int pos, low, first, n;  // first: first window tile; n: tiles in all
  bool sink;               // tile 0 comes first
  __device__ __forceinline__ void init(int64_t pos_, int64_t W, int n_sink) {
    pos = static_cast<int>(pos_);
    low = pos_ - W + 1 > 0 ? static_cast<int>(pos_ - W + 1) : 0;
    first = low / kPDKeys;
    sink = n_sink > 0 && first > 0;
    n = pos_ < 0 ? 0 : pos / kPDKeys - first + 1 + (sink ? 1 : 0);
  }
  __device__ __forceinline__ int tile(int i) const {
    return sink ? (i == 0 ? 0 : first + i - 1) : first + i;
  }
};

__device__ __forceinline__ int64_t decode_pos(const PagedDecodeParams &p, int b) {
  const int64_t v = p.pos[b];
  return v < -1 || v >= p.c.max_pos ? -1 : v;
}

// One CTA's run of the tile list, unit by unit.
struct DecodeRun {
  int64_t left;   // tiles still to go, this unit's among them
  int b, kh;      // sequence, kvh * HB + head block
  int t0, t1;     // tiles of the unit in this run
  PagedSpan s;
  __device__ __forceinline__ bool begin(const PagedDecodeParams &p, int b0, int64_t pos0,
                                        int64_t skip, int64_t len) {
    left = len;
    if (left <= 0) return false;
    b = b0;
    s.init(pos0, p.W, p.n_sink);
    kh = skip < (int64_t(1) << 32) ? static_cast<int>(static_cast<uint32_t>(skip) / s.n)
                                   : static_cast<int>(skip / s.n);
    t0 = static_cast<int>(skip - static_cast<int64_t>(kh) * s.n);
    t1 = left < s.n - t0 ? t0 + static_cast<int>(left) : s.n;
    return true;
  }
  __device__ __forceinline__ bool next(const PagedDecodeParams &p) {
    left -= t1 - t0;
    if (left <= 0) return false;
    if (++kh == p.Hkv * p.HB) {
      kh = 0;
      do {  // left > 0: a sequence with tiles follows
        s.init(decode_pos(p, ++b), p.W, p.n_sink);
      } while (s.n == 0);
    }
    t0 = 0;
    t1 = left < s.n ? static_cast<int>(left) : s.n;
    return true;
  }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kPDThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedDecodeParams p) {
  using L = PagedDecodeLayout<D>;
  constexpr int ST = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - raw);
  const uint32_t BAR_F = base + L::OFF_BAR, BAR_E = BAR_F + 8 * ST;
  float *s_red = reinterpret_cast<float *>(gbase + L::OFF_RED);
  float2 *s_ml = reinterpret_cast<float2 *>(gbase + L::OFF_ML);
  int64_t *s_run = reinterpret_cast<int64_t *>(gbase + L::OFF_MISC);  // b0, its pos, tiles
                                                                        // to skip
  volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + L::OFF_MISC + 24);
  uint8_t *s_failed = gbase + L::OFF_MISC + 32;  // [8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, units_per_seq = p.Hkv * p.HB;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(BAR_F + 8 * s, 1);
      mbar_init(BAR_E + 8 * s, kPDWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // This run: tiles [T c / P, T (c + 1) / P) of the list of T, with P the number
  // of CTAs or T if that is less (no run is empty, the CTAs past P have none).
  // Every CTA sums the tile counts of all sequences, a contiguous piece per thread.
  int64_t total = 0, lo, hi;
  int P;
  {
    int64_t *s_warp = reinterpret_cast<int64_t *>(s_red);
    const int per = (p.B + kPDThreads - 1) / kPDThreads;
    const int b_lo = min(static_cast<int>(threadIdx.x) * per, p.B), b_hi = min(b_lo + per, p.B);
    int64_t sum = 0;
    for (int b = b_lo; b < b_hi; ++b) {
      PagedSpan s;
      s.init(decode_pos(p, b), p.W, p.n_sink);
      sum += s.n;
    }
    sum *= units_per_seq;
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < kPDThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    P = total < gridDim.x ? static_cast<int>(total) : static_cast<int>(gridDim.x);
    lo = cta < P ? mul_div(total, cta, P) : 0;
    hi = cta < P ? mul_div(total, cta + 1, P) : 0;
    int64_t at = before + incl - sum;
    if (hi > lo && lo >= at && lo < at + sum) {
      for (int b = b_lo; b < b_hi; ++b) {
        PagedSpan s;
        const int64_t pos = decode_pos(p, b);
        s.init(pos, p.W, p.n_sink);
        const int64_t n = static_cast<int64_t>(s.n) * units_per_seq;
        if (lo < at + n) {
          s_run[0] = b;
          s_run[1] = pos;
          s_run[2] = lo - at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
  }
  const int b0 = static_cast<int>(s_run[0]);
  const int64_t pos0 = s_run[1], skip = s_run[2], len = hi - lo;

  if (warp == kPDWarps) {
    // ------------------------------------------------------------------ producer
    const int boxes = kPDKeys / p.box_rows;  // per tile, at most 16
    DecodeRun r;
    int it = 0;
    bool ok = true;
    for (bool more = r.begin(p, b0, pos0, skip, len); more && ok; more = r.next(p)) {
      const int32_t *row = p.c.table + r.b * p.c.table_stride;
      const int head = r.kh / p.HB;
      // this lane's box of tile i: its page and first slot (-1: no visible key lies there)
      auto look_up = [&](int i, int &slot) -> int {
        slot = -1;
        if (i >= r.t1 || lane >= boxes) return 0;
        const int at = r.s.tile(i) * kPDKeys + lane * p.box_rows;
        if (at > r.s.pos || (at + p.box_rows <= r.s.low && at >= p.n_sink)) return 0;
        const int pg = at / p.c.page_size;
        slot = at - pg * p.c.page_size;
        return row[pg];
      };
      int slot, page = look_up(r.t0, slot);
      for (int i = r.t0; i < r.t1; ++i, ++it) {
        int slot_n;
        const int page_n = look_up(i + 1, slot_n);  // a tile ahead of its use
        const int st = it % ST;
        if (lane == 0) {
          ok = it < ST || mbar_wait(BAR_E + 8 * st, ((it / ST) - 1) & 1, abort_flag);
          if (ok) mbar_expect_tx(BAR_F + 8 * st, 2 * L::TILE);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < boxes) {
          // a page out of the map's bounds reads as zeros
          if (slot < 0) {
            slot = 0;
            page = p.c.n_pages;
          } else if (page < 0 || page >= p.c.n_pages) {
            atomicOr(&g_swa_status, SWA_DEV_BADARG);
            page = p.c.n_pages;
          }
          const uint32_t dst = base + st * 2 * L::TILE + lane * p.box_rows * (D * 2);
          tma_load_5d(dst, &tm_k, BAR_F + 8 * st, 0, slot, 0, head, page);
          tma_load_5d(dst + L::TILE, &tm_v, BAR_F + 8 * st, 0, slot, 0, head, page);
        }
        page = page_n;
        slot = slot_n;
      }
    }
    // padded rows: zero, and a log-sum-exp of -infinity (32 sequences at a look)
    for (int64_t b0 = static_cast<int64_t>(cta) * 32; b0 < p.B; b0 += gridDim.x * 32) {
      const int b = static_cast<int>(b0) + lane;
      const bool pad = b < p.B && decode_pos(p, b) < 0;
      if (pad && p.pos[b] != -1) atomicOr(&g_swa_status, SWA_DEV_BADARG);
      for (uint32_t m = __ballot_sync(0xffffffffu, pad); m; m &= m - 1) {
        const int64_t row = (b0 + __ffs(m) - 1) * p.H;
        uint4 *o = reinterpret_cast<uint4 *>(p.out + row * D);
        for (int i = lane; i < p.H * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
          for (int i = lane; i < p.H; i += 32) p.lse[row + i] = -INFINITY;
      }
    }
    // every copy issued must land before the CTA ends
    if (lane == 0)
      for (int i = max(0, it - ST); i < it; ++i) mbar_drain(BAR_F + 8 * (i % ST), (i / ST) & 1);
    return;
  }

  // -------------------------------------------------------------------- consumers
  // Fragment coordinates: rows gr and gr + 8 (query heads), keys or columns 2 gc, 2 gc + 1.
  const int gr = lane >> 2, gc = lane & 3;
  // A box of a tile lies in shared memory as [D / 64][box_rows][128 bytes], swizzled.
  // One box holds whole rows: as two boxes of 64 columns the loads of 16-slot pages were
  // bound by the rate of TMA instructions (about 50 cycles each; 200 us against 172 for
  // 64 sequences of 4096 keys).
  auto row_off = [&](int row) -> uint32_t {
    return (row & -p.box_rows) * (D * 2) + (row & (p.box_rows - 1)) * 128;
  };
  const uint32_t panel = p.box_rows * 128;
  // ldmatrix rows: K: lanes 0-7, 8-15 give dims [0,8), [8,16) of keys 0-7, lanes 16-31
  // of keys 8-15; V (transposed): lanes 0-7, 8-15 keys 0-7, 8-15 of columns [0,8), lanes
  // 16-31 of columns [8,16)
  const int k_row = warp * 16 + (lane & 7) + ((lane >> 4) << 3), k_half = (lane >> 3) & 1;
  const int v_row = warp * 16 + (lane & 15), v_half = lane >> 4;
  const uint32_t sw_k = k_row & 7, sw_v = v_row & 7;
  const uint32_t k_off = row_off(k_row), v_off = L::TILE + row_off(v_row);
  DecodeRun r;
  int it = 0;
  int2 split = make_int2(-1, 0);  // the unit to be joined by the merge kernel's block of this run
  for (bool more = r.begin(p, b0, pos0, skip, len); more; more = r.next(p)) {
    bool ok = true;
    const int kvh = r.kh / p.HB, hb = r.kh % p.HB;
    const int rows = min(kPDRows, p.G - hb * kPDRows);
    const bool few = rows <= 8;  // rows 8-15 of P: the second terms of rows 0-7
    const int64_t h0 = static_cast<int64_t>(r.b) * p.H + kvh * p.G + hb * kPDRows;
    uint32_t qa[D / 16][4];
    {
      const __nv_bfloat16 *qp = p.q + (h0 + gr) * D + 2 * gc;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = gr + 8 * (e & 1) < rows;
          qa[kk][e] = in ? *reinterpret_cast<const uint32_t *>(qp + (e & 1) * 8 * D + kk * 16 +
                                                               (e >> 1) * 8)
                         : 0u;
        }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int i = r.t0; i < r.t1; ++i, ++it) {
      const int st = it % ST;
      if (!mbar_wait_warp(BAR_F + 8 * st, (it / ST) & 1, abort_flag)) {
        ok = false;
        break;
      }
      const int key0 = r.s.tile(i) * kPDKeys + warp * 16;  // this warp's 16 keys
      const bool whole = key0 + 15 <= r.s.pos && (key0 >= r.s.low || key0 + 16 <= p.n_sink);
      const bool none = key0 > r.s.pos || (key0 + 15 < r.s.low && key0 >= p.n_sink);
      if (!none) {
        const uint32_t stage = base + st * 2 * L::TILE;
        float s[2][4];  // keys [0,8) and [8,16)
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t kb[4];
          const uint32_t c = (kk & 3) * 2 + k_half;
          ldsm4(kb, stage + (kk >> 2) * panel + k_off + ((c ^ sw_k) << 4));
          mma16816(s[0], qa[kk], kb[0], kb[1]);
          mma16816(s[1], qa[kk], kb[2], kb[3]);
        }
        uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};  // V pairs (2 gc, 2 gc + 1), + 8
        if (!whole) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            keep[nb] = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + nb * 8 + 2 * gc + e;
              const bool in = key <= r.s.pos && (key >= r.s.low || key < p.n_sink);
              if (in) keep[nb] |= 0xFFFFu << (16 * e);
              if (!in) s[nb][e] = s[nb][2 + e] = -INFINITY;
            }
          }
        }
        // running maximum per row; the output is rescaled only when it grows by
        // more than 2^8 (weights stay below that, far inside the types' range)
        float al[2];
        bool grow = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]),
                           fmaxf(s[1][2 * x], s[1][2 * x + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.scale_log2;
          const bool g = mx > m[x] + 8.f;
          al[x] = g ? ex2(m[x] - mx) : 1.f;
          if (g) m[x] = mx;
          grow |= g;
        }
        if (__any_sync(0xffffffffu, grow)) {
          l[0] *= al[0];
          l[1] *= al[1];
          if (few) al[1] = al[0];
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= al[e >> 1];
        }
        // P as the A operand (rows gr / gr + 8, keys of either half) and its rounding
        uint32_t pa[4], pb[4];
        auto weigh = [&](int x) {
          const float mu = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            const float w0 = ex2(fmaf(s[nb][2 * x], p.scale_log2, -mu));
            const float w1 = ex2(fmaf(s[nb][2 * x + 1], p.scale_log2, -mu));
            l[x] += w0 + w1;
            const uint32_t hi = pack_bf16(w0, w1);
            pa[nb * 2 + x] = hi;
            pb[nb * 2 + x] = pack_bf16(w0 - __uint_as_float(hi << 16),
                                       w1 - __uint_as_float(hi & 0xFFFF0000u));
          }
        };
        weigh(0);
        if (few) {
          pa[1] = pb[0];
          pa[3] = pb[2];
        } else {
          weigh(1);
        }
        auto add_pv = [&](const uint32_t(&pw)[4]) {
#pragma unroll
          for (int n2 = 0; n2 < D / 16; ++n2) {
            uint32_t vb[4];
            const uint32_t c = (n2 & 3) * 2 + v_half;
            ldsm4t(vb, stage + (n2 >> 2) * panel + v_off + ((c ^ sw_v) << 4));
            if (!whole) {
              vb[0] &= keep[0];
              vb[1] &= keep[1];
              vb[2] &= keep[0];
              vb[3] &= keep[1];
            }
            mma16816(o[2 * n2], pw, vb[0], vb[1]);
            mma16816(o[2 * n2 + 1], pw, vb[2], vb[3]);
          }
        };
        add_pv(pa);
        if (!few) add_pv(pb);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR_E + 8 * st);
    }

    if (few)
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] += o[n][2];
        o[n][1] += o[n][3];
      }
    // Join the eight warps' states: a common maximum per row, then sums through shared
    // memory, 8 rows x D or 16 rows x 64 columns at a time.
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (gc == 0) s_ml[warp * 16 + gr + 8 * x] = make_float2(m[x], l[x]);
    }
    if (lane == 0) s_failed[warp] = ok ? 0 : 1;
    named_bar_sync(1, kPDWarps * 32);
    // a wait gave up in some warp: all eight leave at the same barrier
    if (*reinterpret_cast<const uint64_t *>(s_failed) != 0) break;
    const bool cut_front = r.t0 > 0, cut_back = r.t1 < r.s.n;
    // run j begins before tile e iff floor(T j / P) < e iff j < e P / T
    if (cut_back && !cut_front)
      split = make_int2(r.b * units_per_seq + r.kh,
                        static_cast<int>(((hi + r.s.n - r.t1) * P + total - 1) / total));
    const int slot = 2 * cta + (cut_front ? 0 : 1);
    float mm[2], wt[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float v = -INFINITY;
#pragma unroll
      for (int w = 0; w < kPDWarps; ++w) v = fmaxf(v, s_ml[w * 16 + gr + 8 * x].x);
      mm[x] = v;
      wt[x] = m[x] == -INFINITY ? 0.f : ex2(m[x] - v);
    }
    const int halves = rows > 8 ? 2 : 1;          // row halves that hold query heads
    const int cols = rows > 8 ? 64 : D;           // columns per round
    for (int c0 = 0; c0 < D; c0 += cols) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        if (n * 8 < c0 || n * 8 >= c0 + cols) continue;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (x < halves)
            *reinterpret_cast<float2 *>(s_red + ((warp * halves + x) * 8 + gr) * cols + n * 8 - c0 +
                                        2 * gc) =
                make_float2(o[n][2 * x] * wt[x], o[n][2 * x + 1] * wt[x]);
      }
      named_bar_sync(1, kPDWarps * 32);
      for (int e = threadIdx.x; e < rows * cols / 4; e += kPDWarps * 32) {
        const int row = e / (cols / 4), col = (e % (cols / 4)) * 4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float M = -INFINITY, Ls = 0.f;
#pragma unroll
        for (int w = 0; w < kPDWarps; ++w) M = fmaxf(M, s_ml[w * 16 + row].x);
#pragma unroll
        for (int w = 0; w < kPDWarps; ++w) {
          const float2 ml = s_ml[w * 16 + row];
          // without a finite score the sum is 0, or NaN and stays so
          Ls += ml.y * (ml.x == -INFINITY ? 0.f : ex2(ml.x - M));
          const float4 v =
              *reinterpret_cast<const float4 *>(s_red + (w * halves * 8 + row) * cols + col);
          a.x += v.x;
          a.y += v.y;
          a.z += v.z;
          a.w += v.w;
        }
        if (cut_front || cut_back) {
          *reinterpret_cast<float4 *>(p.ws_o + (static_cast<int64_t>(slot) * kPDRows + row) * D +
                                      c0 + col) = a;
          if (c0 + col == 0) p.ws_ml[slot * kPDRows + row] = make_float2(M, Ls);
        } else {
          const float inv = 1.f / Ls;
          *reinterpret_cast<uint2 *>(p.out + (h0 + row) * D + c0 + col) =
              make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
          if (p.lse && c0 + col == 0)
            p.lse[h0 + row] = (M + __log2f(Ls)) * 0.6931471805599453f;
        }
      }
      named_bar_sync(1, kPDWarps * 32);
    }
  }
  if (threadIdx.x == 0) p.ws_run[cta] = split;
}

// Joins the partials of the unit that starts in run c and goes on: run c's
// slot 2c + 1, then the slots 2j of the runs that follow.
template <int D>
__global__ void __launch_bounds__(128) paged_decode_merge_kernel(const PagedDecodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const int u = p.ws_run[c].x, end = p.ws_run[c].y;
  if (u < 0) return;
  const int kh = u % (p.Hkv * p.HB), b = u / (p.Hkv * p.HB);
  const int kvh = kh / p.HB, hb = kh % p.HB, rows = min(kPDRows, p.G - hb * kPDRows);
  const int64_t h0 = static_cast<int64_t>(b) * p.H + kvh * p.G + hb * kPDRows;
  for (int e = threadIdx.x; e < rows * (D / 4); e += blockDim.x) {
    const int row = e / (D / 4), col = (e % (D / 4)) * 4;
    // eight parts in flight at a time, their maximum joined to the running one
    constexpr int N = 8;
    float M = -INFINITY, Ls = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = c; j0 < end; j0 += N) {
      float2 ml[N];
      float4 v[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int j = j0 + k, slot = j == c ? 2 * c + 1 : 2 * j;
        ml[k] = make_float2(-INFINITY, 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < end) {
          ml[k] = p.ws_ml[slot * kPDRows + row];
          v[k] = *reinterpret_cast<const float4 *>(
              p.ws_o + (static_cast<int64_t>(slot) * kPDRows + row) * D + col);
        }
      }
      float mn = M;
#pragma unroll
      for (int k = 0; k < N; ++k) mn = fmaxf(mn, ml[k].x);
      // A maximum of -infinity (all scores of the parts are that, or NaN) gives weight 0, which
      // leaves sums of 0 as they are, and NaN.
      const float w0 = M == -INFINITY ? 0.f : ex2(M - mn);
      Ls *= w0;
      a = make_float4(a.x * w0, a.y * w0, a.z * w0, a.w * w0);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float w = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - mn);
        Ls = fmaf(ml[k].y, w, Ls);
        a.x = fmaf(v[k].x, w, a.x);
        a.y = fmaf(v[k].y, w, a.y);
        a.z = fmaf(v[k].z, w, a.z);
        a.w = fmaf(v[k].w, w, a.w);
      }
      M = mn;
    }
    const float inv = 1.f / Ls;
    *reinterpret_cast<uint2 *>(p.out + (h0 + row) * D + col) =
        make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    if (p.lse && col == 0) p.lse[h0 + row] = (M + __log2f(Ls)) * 0.6931471805599453f;
  }
}

}  // namespace swa
