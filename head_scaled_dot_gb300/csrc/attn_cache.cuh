// attn_cache.cuh - what the kernels of the attention over the 8-bit cache
// share: parameters, the list of groups that is cut into equal ranges, TMA.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "internal.h"

namespace mha {

constexpr int CA_MAX_CTAS = 192;   // of the main kernels: bounds the workspace
constexpr int CA_WARPS = 8;        // warps of the mma.sync kernel, a range each
constexpr int CA_HEADER = 8192;    // workspace: first group of every batch item

struct CacheAttnParams {
  CUtensorMap map_k;    // K as (d_h, bt, n_blocks h_kv) bytes
  CUtensorMap map_v;
  const void* Q;        // (B, h, n_q, d_h)
  const uint8_t* K;     // (n_blocks, h_kv, bt, d_h)
  const uint8_t* V;     // (n_blocks, h_kv, bt, d_vh)
  const float* Ks;      // (n_blocks, h_kv)
  const float* Vs;
  const int32_t* table; // (B, max_blocks)
  const int32_t* total; // (B)
  const int32_t* fresh; // (B) or null: new rows, n_q
  void* Z;              // (B, n_q, h d_vh)
  int32_t* first;       // workspace: (B + 1) groups before item b, per tile of rows
  float* part;          // workspace: summaries, [2 ranges][slot_rows][2], then [2 ranges][slot_rows][d_vh]
  int32_t* err;
  int B, n_q, h, h_kv, share, d_h, d_vh, n_blocks, bt, max_blocks;
  int tile_rows;        // query rows per tile: row r is new row r / share of head r % share
  int tiles;            // tiles per key/value head
  int slot_rows;        // rows of a summary slot
  int box;              // rows per TMA box
  int causal_tail;
  int ranges;           // the list of groups is cut into so many ranges
  int tile_cost;        // what a tile costs beside its groups, in groups
  int per_tile;         // tiles have groups up to what their last row sees, else all of them
  int tile_new;         // new rows per tile where heads do not cross tiles, else 0 (divisions then)
  float cl2;            // c log2(e)
  uint64_t limit_ns;    // bounded waits give up after this long
};

// Merges the summaries of the tiles that more than one range had a part of,
// and writes the rows that see no key (attn_cache.cu).
cudaError_t launch_cache_merge(const CacheAttnParams& P, mha_dtype dt, cudaStream_t s);
// Tensor-core kernels for bf16 queries and head sizes up to 128 (attn_cache_tc.cu).
mha_status launch_cache_attention_tc(CacheAttnParams& P, cudaStream_t s);
// The tensor maps of the cache, for boxes of `box` rows of `width` bytes.
bool make_cache_maps(CacheAttnParams& P, int box, int width);

// The rows of a batch item: keys in the cache and new query rows, each held
// inside its bounds.
struct Item {
  int total, fresh;
};
__device__ __forceinline__ Item item_of(const CacheAttnParams& P, int b, bool& bad) {
  const int t = __ldg(P.total + b), f = P.fresh ? __ldg(P.fresh + b) : P.n_q;
  const int most = P.max_blocks * P.bt;
  bad = t < 0 || t > most || f < 0 || f > P.n_q;
  return Item{min(max(t, 0), most), min(max(f, 0), P.n_q)};
}

// Groups of SK keys of tile rt of an item's rows, with P.per_tile: up to what
// its last row sees, none for a tile of padding. (Against all groups of the
// sequence for every tile: 512 new rows over 6000 keys 89.5 -> 78.8 us, 2048
// over 4096 72 -> 65.6; with divisions only, 83.8 and 78.)
__device__ __forceinline__ int tile_groups(const CacheAttnParams& P, int total, int fresh, int rt, int SK) {
  const int begin = P.tile_new ? rt * P.tile_new : rt * P.tile_rows / P.share;
  const int end = P.tile_new ? begin + P.tile_new : ((rt + 1) * P.tile_rows - 1) / P.share + 1;
  const int keys = total - fresh + min(end, fresh);  // (fresh is at most n_q)
  return begin >= fresh || keys <= 0 ? 0 : (unsigned)(keys + SK - 1) / SK;
}

// first[b], b = 0 .. B: groups of SK keys before batch item b, per tile of rows
// (with P.per_tile per key/value head, all its tiles together); totals[b],
// news[b] (unless null): its keys and new rows. Every CTA computes them; the
// first one leaves them in the workspace and reports lengths out of bounds. All
// threads of the CTA.
template <int THREADS, int SK, bool PT>
__device__ __forceinline__ void scan_groups(const CacheAttnParams& P, int* first, int* totals, int* news,
                                            int* warp_sums) {
  constexpr int PER = (MHA_MAX_PADDED_BATCH + THREADS - 1) / THREADS;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int n[PER], sum = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int b = threadIdx.x * PER + k;
    n[k] = 0;
    if (b < P.B) {
      bool bad;
      const Item it = item_of(P, b, bad);
      if (bad && blockIdx.x == 0 && P.err) atomicCAS(P.err, 0, MHA_ERR_INVALID_ARG);
      if (it.fresh > 0) {
        if (PT && P.per_tile)
          for (int t = 0; t < P.tiles; ++t) n[k] += tile_groups(P, it.total, it.fresh, t, SK);
        else
          n[k] = (it.total + SK - 1) / SK;
      }
      if (totals) totals[b] = it.total;
      if (news) news[b] = it.fresh;
    }
    sum += n[k];
  }
  int v = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int before = v - sum;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int b = threadIdx.x * PER + k;
    if (b <= P.B) {
      first[b] = before;
      if (blockIdx.x == 0) P.first[b] = before;
    }
    before += n[k];
  }
  if (threadIdx.x == THREADS - 1 && P.B == THREADS * PER) {
    first[P.B] = before;
    if (blockIdx.x == 0) P.first[P.B] = before;
  }
  __syncthreads();
}

// A place in the list of groups: batch item by batch item, in it tile by tile
// (tile `pr` = key/value head * tiles + tile of rows), in that group by group.
struct Cursor {
  int b, pr, gi, ng;  // ng: groups per tile of this item
};

// How the list is cut into ranges. Beginning and ending a tile costs about as
// much as P.tile_cost groups, so equal shares are of costs: a tile's groups
// come after tile_cost units of their own, and range w begins at w / ranges of
// them all. Item b has `unit` parts of first[b + 1] - first[b] groups and `cost`
// more each: its tiles, or with P.per_tile its key/value heads. (With shares of
// groups alone a CTA that got ten short tiles took 307 us where the median took
// 226.)
// PT: tiles may have groups of their own number (P.per_tile), of SK keys.
template <bool PT, int SK>
struct Ranges {
  int unit, cost, n, per, more;  // the first `more` ranges have per + 1 units
  __device__ __forceinline__ Ranges(const CacheAttnParams& P, int groups)
      : unit(PT && P.per_tile ? P.h_kv : P.h_kv * P.tiles),
        cost(PT && P.per_tile ? P.tile_cost * P.tiles : P.tile_cost),
        n(P.ranges) {
    const int all = groups * unit + cost * unit * P.B;
    per = all / n;
    more = all - per * n;
  }
  // The first group of range w: its cursor, and its number in the list. (w = n:
  // the end.) totals and news with PT only.
  __device__ __forceinline__ int begin(const CacheAttnParams& P, int w, const int* first, const int* totals,
                                       const int* news, Cursor& c) const {
    const int at = w * per + min(w, more), B = P.B;
    int lo = 0, hi = B;  // the last item that starts at or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if ((first[mid] + cost * mid) * unit <= at) lo = mid; else hi = mid - 1;
    }
    const int item = lo;
    while (lo < B && first[lo + 1] == first[lo]) ++lo;  // (in an empty one: on to the next group)
    c.b = lo;
    c.pr = c.gi = 0;
    c.ng = lo < B ? first[lo + 1] - first[lo] : 1;
    if (lo == B) return first[B] * unit;
    const int size = c.ng + cost;
    int in = lo == item ? at - (first[lo] + cost * lo) * unit : 0;
    if (!(PT && P.per_tile)) {
      if (in > 0) {
        c.pr = in / size;
        c.gi = max(0, in - c.pr * size - cost);
      }
      return first[lo] * unit + c.pr * c.ng + c.gi;
    }
    // along the head's tiles; from a place in an empty one on to the next group
    const int kv = in / size;
    int number = first[lo] * unit + kv * c.ng;
    in -= kv * size;
    for (int t = 0; t < P.tiles; ++t) {
      const int g = tile_groups(P, totals[lo], news[lo], t, SK);
      if (g > 0 && in < P.tile_cost + g) {
        c.pr = kv * P.tiles + t;
        c.gi = max(0, in - P.tile_cost);
        c.ng = g;
        return number + c.gi;
      }
      in = max(0, in - P.tile_cost - g);
      number += g;
    }
    c.pr = (kv + 1) * P.tiles - 1;  // past the head's last group
    c.gi = 0;
    c.ng = 1;
    next_tile(P, c, first, totals, news);
    return number;
  }
  // Where the tile's first group is in the costs; g: its groups.
  __device__ __forceinline__ int place(const CacheAttnParams& P, const int* first, const Item& it, int b, int pr,
                                       int& g) const {
    const int ng = first[b + 1] - first[b], at = (first[b] + cost * b) * unit;
    g = ng;
    if (!(PT && P.per_tile)) return at + pr * (ng + cost) + cost;
    const int kv = pr / P.tiles, rt = pr - kv * P.tiles;
    int before = 0;
    for (int t = 0; t < rt; ++t) before += P.tile_cost + tile_groups(P, it.total, it.fresh, t, SK);
    g = ng > 0 ? tile_groups(P, it.total, it.fresh, rt, SK) : 0;
    return at + kv * (ng + cost) + before + P.tile_cost;
  }
  // The range that has unit `at` of the costs.
  __device__ __forceinline__ int owner(int at) const {
    const int big = more * (per + 1);
    return at < big ? at / (per + 1) : more + (at - big) / per;
  }
  // On to the next tile that has groups.
  static __device__ __forceinline__ void next_tile(const CacheAttnParams& P, Cursor& c, const int* first,
                                                   const int* totals, const int* news) {
    c.gi = 0;
#pragma unroll 1
    do {
      if (++c.pr == P.h_kv * P.tiles) {
        c.pr = 0;
        do {
          ++c.b;
        } while (c.b < P.B && first[c.b + 1] == first[c.b]);
      }
      c.ng = c.b >= P.B         ? 1
             : PT && P.per_tile ? tile_groups(P, totals[c.b], news[c.b], c.pr % P.tiles, SK)
                                : first[c.b + 1] - first[c.b];
    } while (c.ng == 0);
  }
};

// True when the cursor has moved to another tile.
template <class R>
__device__ __forceinline__ bool advance(const CacheAttnParams& P, Cursor& c, const int* first,
                                        const int* totals = nullptr, const int* news = nullptr) {
  if (++c.gi < c.ng) return false;
  R::next_tile(P, c, first, totals, news);
  return true;
}

__device__ __forceinline__ void tma_load_3d_at(uint32_t dst, const CUtensorMap* m, uint64_t* bar,
                                               int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// The bounded wait, kept short: a kernel whose warps have different roles waits
// in many places, and its code has to stay in the instruction cache. (Not out
// of line: a call keeps the caller's values in local memory, which shared
// memory has taken the cache of.) Once any wait of the CTA has given up, all
// others return at once.
__device__ __forceinline__ bool cache_wait(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  for (uint32_t it = 1; it != 0; ++it) {
    if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
    if (*w.abort) return false;
    if (globaltimer_ns() - t0 > w.limit_ns) break;
  }
  report_error(w, MHA_ERR_DEVICE_TIMEOUT);
  return false;
}

// Waits, with a limit of its own, until a barrier phase has completed although
// a wait has been given up: for copies or products still in flight.
__device__ __forceinline__ void wait_in_flight(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  for (uint32_t it = 1; it != 0; ++it) {
    if (mbar_try_wait_sleep(bar, parity, 20000)) return;
    if (globaltimer_ns() - t0 > 100000000ull) return;
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Two e4m3 numbers (the low or high half of w) as two fp16 numbers, exactly.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// Two floats as fp16.
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace mha
