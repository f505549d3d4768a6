// swa_paged.cuh -- the paged cache: its address arithmetic, and the append
// kernel that rotates new keys (and queries) by their positions and writes
// keys and values into the slots of their sequence's pages.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "sm100.cuh"

namespace swa {

// Position p of sequence b: page table[b * table_stride + p / page_size], slot
// p % page_size.  Strides in elements, shared by k and v.
struct PagedCache {
  __nv_bfloat16 *k = nullptr, *v = nullptr;
  const int32_t *table = nullptr;
  int64_t page_stride = 0, head_stride = 0, slot_stride = 0, table_stride = 0;
  int n_pages = 0;
  int page_size = 0;
  int64_t max_pos = 0;  // positions a table row can map: max_pages * page_size
};

// Whether positions start .. start + n - 1 (n >= 0) lie in [0, max_pos), for any start:
// start + n could pass 2^63 and come out negative.
__host__ __device__ inline bool positions_fit(int64_t start, int64_t n, int64_t max_pos) {
  return start >= 0 && n <= max_pos && start <= max_pos - n;
}

// One lane of a converged warp.  Inside a branch on it the compiler knows that a
// single thread runs, and keeps the operands of MMA and copy instructions in
// uniform registers; inside a branch on the lane index it does not.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0u;
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, uint32_t bar, int x,
                                            int y, int z, int u, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
      : "memory");
}

// T c / P of a run's border; in 32 bits (a 64-bit division takes 500 cycles of a
// launch's start) unless the list is very long.
__device__ __forceinline__ int64_t mul_div(int64_t T, int c, int P) {
  if (T < (1 << 22)) return static_cast<uint32_t>(T) * static_cast<uint32_t>(c) / P;
  return T * c / P;
}

// ------------------------------------------------------------------ append
//
// One token per team: a warp, or the whole CTA where a call has so few tokens that
// the latency of one counts.  Bound: bytes (every input row read once, every output
// row written once), then, for few tokens, the chain of dependent loads offsets ->
// start -> table entry; the token's first rows are loaded into registers before
// that chain starts.  Measured with H = 32, Hkv = 8, d = 128: 64 tokens 4.1 us (a
// warp each: 7.0), 768 tokens 6.0 (8.1), 2048 tokens 11.5 either way; 9843 tokens 47 us
// (53 as CTAs), 5.1 TB/s; 16384 tokens with Hkv = 32 141 us, 5.7 TB/s.  Five items in
// flight per thread: with four the last takes 155 us, with six (80 registers) 4096 tokens
// take 24 instead of 20 us.
//
// The rotation of pair i turns (x, y) by a = position * inv_freq[i].  In 32
// bits a would lose its fraction of a turn for far positions (position 10^5,
// inv_freq 1: the product is rounded to 2^-8 of a radian), so the number of
// turns a / 2 pi is formed in 64 bits, its integer part dropped there, and
// only the remainder in [-1/2, 1/2] goes to the 32-bit sincospi.  One angle
// per pair and token serves all H + Hkv heads through shared memory.
constexpr int kAppendThreads = 128;
constexpr int kAppendBatch = 5;  // 16-element items a thread keeps in flight

struct AppendParams {
  const __nv_bfloat16 *k_new, *v_new, *q;
  __nv_bfloat16 *q_out;
  int64_t k_stride, v_stride, q_stride, qo_stride;  // token strides, elements
  PagedCache c;
  const int64_t *cu_seqlens, *q_start;
  int n_seq;
  int64_t total;
  int H, Hkv;  // H = 0: no queries
  int zero_rest;
  const float *inv_freq;
  const int64_t *positions;  // nullptr: the position in the sequence
  const int32_t *pair_axis;  // nullptr: axis 0
  int64_t pos_stride;
  int rot, n_axes;
};

// The number of threads of a team (the warp, or the CTA) for which `c` holds.
template <int TEAM>
__device__ __forceinline__ int team_count(bool c) {
  return TEAM == 32 ? __popc(__ballot_sync(0xffffffffu, c)) : __syncthreads_count(c);
}
template <int TEAM>
__device__ __forceinline__ void team_sync() {
  if (TEAM == 32)
    __syncwarp();
  else
    __syncthreads();
}

// The number of i in [0, n] with cu[i] <= t, for non-decreasing cu (any value
// in range otherwise): each round narrows the range by the team's size.
template <int TEAM>
__device__ __forceinline__ int64_t team_count_le(const int64_t *cu, int64_t n, int64_t t,
                                                 int rank) {
  int64_t lo = 0, len = n + 1;
  while (len > 0) {
    const int64_t step = (len + TEAM - 1) / TEAM;
    const int64_t i = lo + (rank + 1) * step - 1;
    const int c = team_count<TEAM>(i < lo + len && cu[i] <= t);
    const int64_t end = lo + len;
    lo += c * step;
    len = step - 1 < end - lo ? step - 1 : end - lo;
  }
  return lo;
}

__device__ __forceinline__ void rotate_pair(float &x, float &y, float2 cs) {
  const float a = x * cs.x - y * cs.y;
  y = y * cs.x + x * cs.y;
  x = a;
}

template <int D, bool INTERLEAVED, int TEAM>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendParams p) {
  constexpr int IPR = D / 16;  // items per row
  __shared__ float2 s_turn[kAppendThreads / TEAM][D / 2];
  float2 *s_cs = s_turn[threadIdx.x / TEAM];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / TEAM) + threadIdx.x / TEAM;
  const int tid = threadIdx.x % TEAM;
  if (t >= p.total) return;
  const int rows = p.H + 2 * p.Hkv, n_items = rows * IPR;
  const int rot16 = p.rot / 16;
  // Item i of a row is two 16-byte pieces: elements [8i, 8i+8) and their
  // partners rot/2 further on (halves), or 16 consecutive ones (interleaved
  // pairs, and whatever does not turn).
  auto piece = [&](int item, int &row, int &i, int &e0, int &e1, bool &turns) {
    row = item / IPR;
    i = item % IPR;
    turns = row < p.H + p.Hkv && i < rot16;
    e0 = !INTERLEAVED && turns ? 8 * i : 16 * i;
    e1 = !INTERLEAVED && turns ? p.rot / 2 + 8 * i : 16 * i + 8;
  };
  auto src_row = [&](int row) -> const __nv_bfloat16 * {
    if (row < p.H) return p.q + t * p.q_stride + row * D;
    if (row < p.H + p.Hkv) return p.k_new + t * p.k_stride + (row - p.H) * D;
    return p.v_new + t * p.v_stride + (row - p.H - p.Hkv) * D;
  };
  uint4 a[kAppendBatch], b[kAppendBatch];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
      const int item = base + u * TEAM + tid;
      if (item >= n_items) break;
      int row, i, e0, e1;
      bool turns;
      piece(item, row, i, e0, e1, turns);
      const __nv_bfloat16 *src = src_row(row);
      a[u] = *reinterpret_cast<const uint4 *>(src + e0);
      b[u] = *reinterpret_cast<const uint4 *>(src + e1);
    }
  };
  load(0);

  if (t == 0) {  // offsets out of order or range: flagged once
    for (int64_t i = tid; i < p.n_seq; i += TEAM)
      if (p.cu_seqlens[i] < 0 || p.cu_seqlens[i + 1] < p.cu_seqlens[i] ||
          p.cu_seqlens[i + 1] > p.total)
        atomicOr(&g_swa_status, SWA_DEV_BADARG);
  }
  const int64_t seq = team_count_le<TEAM>(p.cu_seqlens, p.n_seq, t, tid) - 1;
  int64_t pos = 0;
  int page = -1;
  if (seq >= 0 && seq < p.n_seq) {
    const int64_t begin = p.cu_seqlens[seq], end = p.cu_seqlens[seq + 1];
    const int64_t start = p.q_start[seq];
    if (begin >= 0 && t >= begin && t < end && end <= p.total) {
      if (positions_fit(start, t - begin + 1, p.c.max_pos)) {
        pos = start + (t - begin);
        page = p.c.table[seq * p.c.table_stride + pos / p.c.page_size];
      }
      if (page >= p.c.n_pages) page = -1;
      if (page < 0 && tid == 0) atomicOr(&g_swa_status, SWA_DEV_BADARG);
    }
  }
  if (page < 0) {  // no slot to write
    if (p.zero_rest)
      for (int i = tid; i < p.H * (D / 8); i += TEAM)
        *reinterpret_cast<uint4 *>(p.q_out + t * p.qo_stride + 8 * i) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t slot =
      static_cast<int64_t>(page) * p.c.page_stride + (pos % p.c.page_size) * p.c.slot_stride;

  for (int pair = tid; pair < p.rot / 2; pair += TEAM) {
    int64_t at = pos;
    if (p.positions) {
      int axis = p.pair_axis ? p.pair_axis[pair] : 0;
      if (axis < 0 || axis >= p.n_axes) {
        atomicOr(&g_swa_status, SWA_DEV_BADARG);
        axis = 0;
      }
      at = p.positions[axis * p.pos_stride + t];
    }
    const double kInv2Pi = 0.15915494309189533577;
    double turns = static_cast<double>(at) * (static_cast<double>(p.inv_freq[pair]) * kInv2Pi);
    turns -= rint(turns);
    float s, c;
    sincospif(static_cast<float>(2.0 * turns), &s, &c);
    s_cs[pair] = make_float2(c, s);
  }
  team_sync<TEAM>();

  for (int base = 0; base < n_items; base += kAppendBatch * TEAM) {
    if (base > 0) load(base);
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
      const int item = base + u * TEAM + tid;
      if (item >= n_items) break;
      int row, i, e0, e1;
      bool turns;
      piece(item, row, i, e0, e1, turns);
      if (turns) {
        uint32_t wa[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
        uint32_t wb[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 x = make_float2(__uint_as_float(wa[j] << 16), __uint_as_float(wa[j] & 0xFFFF0000u));
          float2 y = make_float2(__uint_as_float(wb[j] << 16), __uint_as_float(wb[j] & 0xFFFF0000u));
          if (INTERLEAVED) {  // pairs inside each word
            rotate_pair(x.x, x.y, s_cs[8 * i + j]);
            rotate_pair(y.x, y.y, s_cs[8 * i + 4 + j]);
          } else {
            rotate_pair(x.x, y.x, s_cs[8 * i + 2 * j]);
            rotate_pair(x.y, y.y, s_cs[8 * i + 2 * j + 1]);
          }
          wa[j] = pack_bf16(x.x, x.y);
          wb[j] = pack_bf16(y.x, y.y);
        }
        a[u] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
        b[u] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
      }
      __nv_bfloat16 *dst;
      if (row < p.H)
        dst = p.q_out + t * p.qo_stride + row * D;
      else if (row < p.H + p.Hkv)
        dst = p.c.k + slot + (row - p.H) * p.c.head_stride;
      else
        dst = p.c.v + slot + (row - p.H - p.Hkv) * p.c.head_stride;
      *reinterpret_cast<uint4 *>(dst + e0) = a[u];
      *reinterpret_cast<uint4 *>(dst + e1) = b[u];
    }
  }
}

}  // namespace swa
