// attn_cache_tc.cu - attention over the 8-bit cache on the fifth-generation
// tensor cores: bf16 queries, head sizes up to 128.
//
// The bytes of the cache go from HBM to the tensor cores as they are: TMA puts
// tiles of 128 keys into shared memory, and both products are tcgen05.mma of
// kind f8f6f4 with the key and value tiles as e4m3 operands and fp32 sums in
// tensor memory. What is multiplied with them is written as a sum of two e4m3
// numbers, x = hi + lo / 16:
//   queries  a row is scaled by a power of two to a largest element in
//            [2^7, 2^8). bf16's 8 bits are exactly the 4 of hi and the 4 of
//            lo, down to 2^-13 of the row's largest element.
//   weights  p = 2^{s - m}, times 2^8 vs / vref: 8 bits, down to 2^-18 of the
//            weight of the row's reference m.
// Each hi and lo is an operand row of its own, so the sums are exact fp32
// additions of the two accumulator rows.
//
// Two forms, by the rows of a tile (new rows times the query heads that share
// a key/value head):
//   narrow, 16 rows. An MMA has 128 operand rows. Its four groups of 32 (the
//     tensor-memory lanes of one warp each) all hold the same 16 rows, hi in
//     the first 16 lanes and lo in the others; warp q takes keys 32 q ..
//     32 q + 31 of a tile from its own lanes, keeps its own summary (m, l, z)
//     of them, and writes zeros as its weights of the other keys. So four warps share a tile of 16 rows without ever meeting, until the
//     four summaries are merged at the end.
//   wide, 128 rows, one per lane: hi and lo of the queries go into the same
//     accumulator (lo is not scaled there: exact down to 2^-9 of the largest
//     element, off by at most 2^-17 of it below), those of the weights into
//     two.
//
// Bound. Narrow: reading the cache. One 32 KB stage takes about 1500 cycles of
// its SM's share of HBM, 540 of tensor work and 500 of its softmax warps. Wide:
// 4 x 128^3 multiply-adds at the 8-bit rate, 1070 cycles per tile of 128 keys,
// beside the softmax step of eight warps.
//
// Pipeline of a CTA (one per SM, persistent over its range of the list of
// groups): warps 0, 2 and 3 fill the ring of stages, warp 1 issues the
// products (the scores of the next group before the value product of the
// current one), the softmax warps turn scores into weights, which go over the scores in tensor
// memory as the value product's other operand. z stays in tensor memory; it is
// rescaled only where a row's reference is raised or the values' scale moves.
//
// Measured against the mma.sync kernel of attn_cache.cu, which this one
// replaced for these types: its m16n8k16 products alone took 512 cycles per 32
// keys and SM on the profiler, more than HBM's share of 370.
#include "attn_cache.cuh"

namespace mha {
namespace {

constexpr int KEYS = 128;               // keys per group
constexpr int ROW = 128;                // bytes of a row in shared memory
constexpr int SIDE = KEYS * ROW;        // one side of a stage
constexpr int STAGE = 2 * SIDE;
constexpr int STAGES = 4;
constexpr int OPERAND = 128 * ROW;      // 128 operand rows of e4m3
constexpr int TMEM_COLS = 512;
constexpr int S_COL = 0;                // two score tiles of 128 columns; the weights over them
constexpr int Z_COL = 256;              // z; wide: hi, and lo at Z_COL + 128
constexpr float RAISE = 0.75f;          // p at most 2^0.75 (448 = 1.75 2^8)

// Beside a stage: scales of its eight groups of 16 keys, which of them there
// are, the largest vs, and whether all vs are within 2^2 of it.
struct Meta {
  float ks[8], vs[8];
  uint32_t found;
  float top;
  uint32_t single;
  uint32_t pad;
};

template <bool WIDE>
struct Form {
  static constexpr int SOFTMAX_WARPS = WIDE ? 8 : 4;
  static constexpr int THREADS = 128 + 32 * SOFTMAX_WARPS;
  static constexpr int ROWS = WIDE ? 128 : 16;
  static constexpr int PIECES = WIDE ? 2 : 1;      // operand tiles of Q and of P
  static constexpr int SUBS = WIDE ? 4 : 1;        // groups of 16 keys per lane
  // shared memory
  static constexpr int Q_AT = STAGES * STAGE;
  static constexpr int M_AT = Q_AT + PIECES * OPERAND;      // narrow: four summaries' z
  static constexpr int META_AT = M_AT + (WIDE ? 0 : 4 * 16 * 128 * 4);
  static constexpr int NAN_AT = META_AT + STAGES * (int)sizeof(Meta);
  static constexpr int LIM_AT = NAN_AT + ROWS * 16;
  static constexpr int QF_AT = LIM_AT + ROWS * 4;
  static constexpr int ML_AT = QF_AT + ROWS * 4;            // narrow: m, l of four summaries
  static constexpr int FIRST_AT = ML_AT + 4 * 16 * 2 * 4;
  static constexpr int BAR_AT = FIRST_AT + (MHA_MAX_PADDED_BATCH + 8) * 4;
  static constexpr int SMEM = 1024 + BAR_AT + 256;
};

// D[tmem] (+)= A * B, e4m3 operands in shared memory, fp32 sums.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A in tensor memory, four elements per column.
__device__ __forceinline__ void umma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind f8f6f4: e4m3 A (K-major) and B, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Half-split load of 16 columns: lane i < 16 gets columns [0, 16) of TMEM lane
// i, lane i + 16 those at OFF of the same TMEM lane.
template <int OFF>
__device__ __forceinline__ void tmem_ld_x2_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16], %17;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr), "n"(OFF));
}

// Half-split stores: lane i < 16 to the columns from taddr on of TMEM lane i,
// lane i + 16 to those at OFF of the same TMEM lane.
template <int OFF>
__device__ __forceinline__ void tmem_st_x2_4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x32bx2.x4.b32 [%0], %1, {%2, %3, %4, %5};" ::"r"(taddr),
               "n"(OFF), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
template <int OFF>
__device__ __forceinline__ void tmem_st_x2_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, {%2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17};" ::"r"(taddr),
      "n"(OFF), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15])
      : "memory");
}
// Zeros in eight columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_zero8(uint32_t taddr) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(
                   taddr),
               "r"(0)
               : "memory");
}

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// Four values x (at most 448) as hi and lo of x = hi + lo / 2^SHIFT, four
// e4m3 numbers each. fp16 in between holds 11 bits.
template <int SHIFT>
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t& hi,
                                       uint32_t& lo) {
  const uint32_t h0 = pack_half(a, b), h1 = pack_half(c, d);
  uint32_t e;
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(e)
      : "r"(h0), "r"(h1));
  hi = e;
  const __half2 k = __float2half2_rn((float)(1 << SHIFT));
  const uint32_t g0 = e4m3_lo(e), g1 = e4m3_hi(e);
  const __half2 r0 = __hmul2(__hsub2(reinterpret_cast<const __half2&>(h0), reinterpret_cast<const __half2&>(g0)), k);
  const __half2 r1 = __hmul2(__hsub2(reinterpret_cast<const __half2&>(h1), reinterpret_cast<const __half2&>(g1)), k);
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(lo)
      : "r"(reinterpret_cast<const uint32_t&>(r0)), "r"(reinterpret_cast<const uint32_t&>(r1)));
}

// Byte offset of 16-byte piece c of operand or tile row r (128-byte swizzle).
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return (uint32_t)(r * ROW + ((c ^ (r & 7)) << 4));
}

// Groups of 16 keys whose values go into the next product: those of `todo`
// within 2^2 of its largest scale `top` (and those without a positive scale,
// so that every round takes at least one).
__device__ __forceinline__ uint32_t take_of(const Meta* m, uint32_t todo, float& top) {
  top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (todo >> i & 1) top = fmaxf(top, m->vs[i]);
  uint32_t take = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((todo >> i & 1) && !(m->vs[i] > 0.f && m->vs[i] < 0.25f * top)) take |= 1u << i;
  return take;
}

template <bool WIDE>
__global__ void __launch_bounds__(Form<WIDE>::THREADS, 1)
    cache_attention_tc_kernel(const __grid_constant__ CacheAttnParams P) {
  using F = Form<WIDE>;
  constexpr int NST = 32 * F::SOFTMAX_WARPS;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Meta* metas = reinterpret_cast<Meta*>(smem + F::META_AT);
  int* first = reinterpret_cast<int*>(smem + F::FIRST_AT);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::BAR_AT);  // [STAGES] tiles and scales there
  uint64_t* empty = full + STAGES;    // [STAGES] both products done
  uint64_t* s_full = empty + STAGES;  // [2] scores there
  uint64_t* q_full = s_full + 2;      // the tile's queries there
  uint64_t* p_full = q_full + 1;      // weights there
  uint64_t* p_free = p_full + 1;      // value product done
  uint64_t* done = p_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  __shared__ int warp_sums[F::THREADS / 32];
  __shared__ int abort_flag;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 3);  // key tiles, value tiles, scales
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(s_full + s, 1);
    mbar_init(q_full, F::SOFTMAX_WARPS);
    mbar_init(p_full, F::SOFTMAX_WARPS);
    mbar_init(p_free, 1);
    mbar_init(done, 1);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&P.map_k);
    tma_prefetch_desc(&P.map_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  grid_dep_wait();
  grid_dep_launch_dependents();
  scan_groups<F::THREADS, KEYS>(P, first, warp_sums);

  const int unit = P.h_kv * P.tiles;
  const long long G = (long long)first[P.B] * unit;
  const long long g0 = blockIdx.x * G / P.ranges, g1 = (blockIdx.x + 1) * G / P.ranges;
  const int steps = (int)(g1 - g0);
  const WaitCtl ctl{P.err, &abort_flag, P.limit_ns};

  if (steps > 0 && warp < 4 && warp != 1) {
    // ---- the ring: warp 0 the key tiles, warp 2 the value tiles, warp 3 the
    // scales, each walking the groups for itself ----
    // A lane has one box of a tile (warp 3: 16 keys of it): its entry j of the
    // block table and its row in that block, moved on by 128 keys a step.
    // Entries come from two windows of 32, the second asked for ahead of use.
    const int span = warp == 3 ? 16 : P.box;
    const bool mine = lane < KEYS / span;
    const int dj = KEYS / P.bt, drow = KEYS % P.bt;
    Cursor lc = cursor_at(first, P.B, unit, g0);
    int j, row, kv, total, win, win_id, next_id;
    auto table_entry = [&](int i) {
      return i < P.max_blocks ? __ldg(P.table + (long long)lc.b * P.max_blocks + i) : -1;
    };
    auto place = [&]() {
      bool bad;
      const int k = lc.gi * KEYS + (mine ? lane * span : 0);
      total = item_of(P, lc.b, bad).total;
      kv = lc.pr / P.tiles;
      j = k / P.bt;
      row = k - j * P.bt;
      win = __shfl_sync(0xffffffffu, j, 0);
      win_id = table_entry(win + lane);
      next_id = table_entry(win + 32 + lane);
    };
    place();
    const CUtensorMap* map = warp == 0 ? &P.map_k : &P.map_v;
    const uint32_t tiles = smem_u32(smem) + (warp == 0 ? 0 : SIDE) + lane * span * ROW;
    bool ok = true;
    int n = 0;
    for (; n < steps; ++n) {
      const int stage = n % STAGES;
      const int j0 = __shfl_sync(0xffffffffu, j, 0);
      if (j0 + 8 >= win + 32) {  // lane i takes entry j0 + i of the two windows
        const int at = lane + j0 - win;
        const int x = __shfl_sync(0xffffffffu, win_id, at & 31);
        const int y = __shfl_sync(0xffffffffu, next_id, at & 31);
        win_id = at < 32 ? x : y;
        win = j0;
        next_id = table_entry(win + 32 + lane);
      }
      const int id = __shfl_sync(0xffffffffu, win_id, j - win);
      const bool used = mine && lc.gi * KEYS + lane * span < total;
      const bool there = used && id >= 0 && id < P.n_blocks;
      const int blk = id * P.h_kv + kv;
      if (warp == 3) {
        // the scales are on their way while the stage is waited for
        const float ks = there ? __ldg(P.Ks + blk) : 0.f, vs = there ? __ldg(P.Vs + blk) : 0.f;
        const uint32_t found = __ballot_sync(0xffffffffu, there);
        if (n >= STAGES) ok = __all_sync(0xffffffffu, mbar_wait(empty + stage, (n / STAGES - 1) & 1, ctl));
        if (!ok) break;
        float top = there ? vs : 0.f, least = there ? vs : 3.4e38f;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
        }
        Meta* m = metas + stage;
        if (mine) {
          m->ks[lane] = ks;
          m->vs[lane] = vs;
        }
        if (lane == 0) {
          m->found = found;
          m->top = top;
          m->single = !(least < 0.25f * top);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full + stage);
      } else {
        if (used && !there && P.err) atomicCAS(P.err, 0, MHA_ERR_INVALID_ARG);
        const uint32_t load = __ballot_sync(0xffffffffu, there);
        if (n >= STAGES) ok = __all_sync(0xffffffffu, mbar_wait(empty + stage, (n / STAGES - 1) & 1, ctl));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(full + stage, __popc(load) * span * ROW);
        __syncwarp();
        if (there) tma_load_3d_at(tiles + stage * STAGE, map, full + stage, 0, row, blk);
      }
      if (advance(lc, first, P.B, unit)) {
        if (n + 1 < steps) place();
      } else {
        j += dj;
        row += drow;
        if (row >= P.bt) {
          row -= P.bt;
          ++j;
        }
      }
    }
    if (!ok && warp != 3)  // gave up: the copies in flight are waited for before the CTA ends
      for (int k = n > STAGES ? n - STAGES : 0; k < n; ++k)
        wait_in_flight(full + k % STAGES, (k / STAGES) & 1);
  } else if (steps > 0 && warp == 1 && lane == 0) {
    // ---- products ----
    constexpr uint32_t idesc_s = idesc_e4m3_f32(128, KEYS, 0);
    const uint32_t idesc_z = idesc_e4m3_f32(128, P.d_vh, 1);
    const int slices = (P.d_h + 31) / 32;
    const uint32_t base = smem_u32(smem);
    const uint64_t q_desc = sdesc_sw128(base + F::Q_AT, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(base, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(base + SIDE, 16384, 1024);
    Cursor cc = cursor_at(first, P.B, unit, g0);
    bool ok = true, begins = true;
    int tile = 0, pv = 0;
    auto issue_s = [&](int n) {
      const int stage = n % STAGES, b = n & 1;
      // The scores go over the weights of group n - 2, whose value product is
      // ahead of them in this thread's order.
      ok = ok && mbar_wait(full + stage, (n / STAGES) & 1, ctl);
      if (!ok) return;
      tc_fence_after();
      const uint64_t kd = k_desc + (uint64_t)(stage * STAGE >> 4);
#pragma unroll
      for (int p = 0; p < F::PIECES; ++p) {
        for (int k = 0; k < slices; ++k)
          umma_f8(tmem + S_COL + b * KEYS, q_desc + (uint64_t)((p * OPERAND + k * 32) >> 4),
                  kd + (uint64_t)(k * 32 >> 4), idesc_s, p + k > 0);
      }
      umma_commit(s_full + b);
    };
    for (int n = 0; ok && n < steps; ++n) {
      const int stage = n % STAGES;
      const bool ends = cc.gi == cc.ng - 1 || n == steps - 1;
      if (begins) {
        ok = mbar_wait(q_full, tile & 1, ctl);
        ++tile;
        issue_s(n);
      }
      if (!ends) issue_s(n + 1);
      if (!ok) break;
      const Meta* m = metas + stage;
      uint32_t todo = m->single ? 0u : m->found;
      bool fresh = begins;
      do {
        if (todo) {
          float top;
          todo &= ~take_of(m, todo, top);
        }
        if (!mbar_wait(p_full, pv & 1, ctl)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t vd = v_desc + (uint64_t)(stage * STAGE >> 4);
#pragma unroll
        for (int p = 0; p < F::PIECES; ++p) {
#pragma unroll
          for (int k = 0; k < KEYS / 32; ++k)
            umma_f8_ts(tmem + Z_COL + p * 128, tmem + S_COL + (n & 1) * KEYS + p * 32 + k * 8,
                       vd + (uint64_t)(k * 32 * ROW >> 4), idesc_z, !fresh || k > 0);
        }
        umma_commit(p_free);
        fresh = false;
        ++pv;
      } while (todo);
      if (!ok) break;
      umma_commit(empty + stage);
      begins = ends;
      advance(cc, first, P.B, unit);
    }
    umma_commit(done);  // the products in flight end before tensor memory is given back
    wait_in_flight(done, 0);
  } else if (steps > 0 && warp >= 4) {
    // ---- softmax ----
    // Lane i < 16 of a warp holds the first half of row i's keys, lane i + 16
    // the other: 16 keys each of the warp's 32 (narrow) or 64 each (wide).
    const int q = warp & 3, hh = (warp - 4) >> 2, half = lane >> 4;
    const int tid = threadIdx.x - 128;
    const int row = WIDE ? 32 * q + 16 * hh + (lane & 15) : lane & 15;
    const uint32_t lanes = static_cast<uint32_t>(WIDE ? 32 * q + 16 * hh : 32 * q) << 16;
    const uint32_t lo_lanes = 16u << 16;  // narrow: from a row's hi to its lo
    uint32_t* nan_map = reinterpret_cast<uint32_t*>(smem + F::NAN_AT);
    int* lim_s = reinterpret_cast<int*>(smem + F::LIM_AT);
    float* qf_s = reinterpret_cast<float*>(smem + F::QF_AT);
    const uint32_t q_base = smem_u32(smem) + F::Q_AT;
    Cursor cc = cursor_at(first, P.B, unit, g0);
    bool ok = true, begins = true;
    int pv = 0, start_gi = 0;
    int limit = -1, lim_all = 0, lim_any = -1;
    float qf = 0.f, m = -INFINITY, l = 0.f, vref = 1.f, vtop = 0.f;

    // The tile's queries as operand rows, and its rows' limits.
    auto begin_tile = [&]() {
      const int kv = cc.pr / P.tiles, rt = cc.pr - kv * P.tiles;
      bool bad;
      const Item it = item_of(P, cc.b, bad);
      const int rows = P.n_q * P.share;
      {
        constexpr int TPR = WIDE ? 2 : 8;     // threads per row
        constexpr int PPT = 8 / TPR;          // 16-element pieces per thread
        const int r = tid / TPR, part = tid % TPR;
        const int rr = rt * F::ROWS + r, i = rr / P.share;
        const bool in = rr < rows && i < it.fresh;
        const int head = kv * P.share + (rr - i * P.share);
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(P.Q) +
                                   (((long long)cc.b * P.h + head) * P.n_q + i) * P.d_h;
        uint4 raw[PPT][2];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
          const int col = (part * PPT + k) * 16;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            raw[k][e] = make_uint4(0u, 0u, 0u, 0u);
            if (in && col < P.d_h) raw[k][e] = __ldg(reinterpret_cast<const uint4*>(src + col) + e);
            const uint32_t x[4] = {raw[k][e].x, raw[k][e].y, raw[k][e].z, raw[k][e].w};
#pragma unroll
            for (int f = 0; f < 4; ++f)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[f] << 16)),
                                     fabsf(__uint_as_float(x[f] & 0xffff0000u))));
          }
        }
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^(7 - E) for a largest element in [2^E, 2^(E + 1))
        int E = (int)(__float_as_uint(top) >> 23) - 127;
        E = E > 127 || top == 0.f ? 7 : max(E, -100);
        const float up = __uint_as_float((uint32_t)(7 - E + 127) << 23);
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const uint4 u = raw[k][f / 2];
            const uint32_t x0 = f % 2 ? u.z : u.x, x1 = f % 2 ? u.w : u.y;
            split4<WIDE ? 0 : 4>(__uint_as_float(x0 << 16) * up, __uint_as_float(x0 & 0xffff0000u) * up,
                                 __uint_as_float(x1 << 16) * up, __uint_as_float(x1 & 0xffff0000u) * up,
                                 hi[f], lo[f]);
          }
          const uint4 h4 = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          const uint4 l4 = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          const int c = part * PPT + k;
          if constexpr (WIDE) {
            sts128(q_base + swz(r, c), h4);
            sts128(q_base + OPERAND + swz(r, c), l4);
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              sts128(q_base + swz(32 * w + r, c), h4);
              sts128(q_base + swz(32 * w + 16 + r, c), l4);
            }
          }
        }
        if (part == 0) {
          qf_s[r] = P.cl2 * __uint_as_float((uint32_t)(E - 7 + 127) << 23);
          lim_s[r] = !in ? -1 : P.causal_tail ? max(-1, it.total - it.fresh + i) : it.total - 1;
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      softmax_sync<NST>();
      for (int e = tid; e < F::ROWS * 4; e += NST) nan_map[e] = 0u;  // the last tile's was read
      softmax_sync<NST>();
      qf = qf_s[row];
      limit = lim_s[row];
      // the limits of the tile's first and last row that see a key
      const int i0 = rt * F::ROWS / P.share;
      const int i1 = min((min(rows, (rt + 1) * F::ROWS) - 1) / P.share, it.fresh - 1);
      const int back = it.total - it.fresh;
      lim_any = i1 < i0 ? -1 : P.causal_tail ? back + i1 : it.total - 1;
      lim_all = P.causal_tail ? max(0, back + i0) : it.total - 1;
      m = -INFINITY;
      l = 0.f;
      vref = 1.f;
      vtop = 0.f;
      start_gi = cc.gi;
    };

    // z of this warp's rows times f (f may differ from row to row).
    auto scale_z = [&](float f) {
      tc_fence_after();
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t at = tmem + lanes + Z_COL + (WIDE ? p * 128u : p * lo_lanes);
#pragma unroll
        for (int cb = 0; cb < 2; ++cb) {
          uint32_t o[32];
          tmem_ld_x2_32<64>(at + 32 * cb, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tmem_st_x2_32<64>(at + 32 * cb, o);
        }
      }
      tmem_wait_st();
    };

    for (int n = 0; n < steps; ++n) {
      const int stage = n % STAGES, b = n & 1;
      const bool ends = cc.gi == cc.ng - 1 || n == steps - 1;
      if (begins) begin_tile();
      ok = ok && mbar_wait(full + stage, (n / STAGES) & 1, ctl);
      ok = ok && mbar_wait(s_full + b, (n >> 1) & 1, ctl);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        const Meta* meta = metas + stage;
        const int kb = cc.gi * KEYS;
        const uint32_t found = meta->found;
        const bool masked = kb + KEYS - 1 > lim_all || found != 0xffu;
        float s[F::SUBS][16];
        {
          const uint32_t at = tmem + lanes + S_COL + b * KEYS;
          if constexpr (WIDE) {
            uint32_t x[64];
            tmem_ld_x2_64<64>(at, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 64; ++k) s[k / 16][k % 16] = __uint_as_float(x[k]);
          } else {
            uint32_t x[16], y[16];
            tmem_ld_x2_16<16>(at + 32 * q, x);
            tmem_ld_x2_16<16>(at + 32 * q + lo_lanes, y);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              s[0][k] = fmaf(__uint_as_float(y[k]), 0.0625f, __uint_as_float(x[k]));
          }
        }
        const int sub0 = WIDE ? 4 * half : 2 * q + half;  // this lane's groups of 16 keys
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < F::SUBS; ++i) {
          const float f = qf * meta->ks[sub0 + i];
          const int seen = found >> (sub0 + i) & 1 ? limit - kb - 16 * (sub0 + i) : -1;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            s[i][k] *= f;
            if (masked && k > seen) s[i][k] = -INFINITY;
            mx = fmaxf(mx, s[i][k]);
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        // a row's reference is raised only where a weight would pass 2^0.75
        float alpha = 1.f;
        if (mx > m + RAISE) {
          alpha = ex2_approx(m - mx);
          m = mx;
          l *= alpha;
        }
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < F::SUBS; ++i) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            s[i][k] = ex2_approx(s[i][k] - base);
            l += s[i][k];
          }
        }
        if (masked && tid < KEYS) {
          // Value rows that not every row sees, or none: their NaN bytes are
          // zeroed, and noted for the rows that do see them.
          const uint32_t src = smem_u32(smem) + stage * STAGE + SIDE;
          const bool there = found >> (tid >> 4) & 1;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            const uint32_t at = src + swz(tid, c);
            const uint4 u = lds128(at);
            uint32_t x[4] = {u.x, u.y, u.z, u.w}, any = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t hit = ((x[w] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              any |= hit;
              if (hit && there && kb + tid <= lim_any) {
                for (int byte = 0; byte < 4; ++byte) {
                  if (!(hit >> (8 * byte + 7) & 1)) continue;
                  const int d = 16 * c + 4 * w + byte;
                  for (int r = 0; r < F::ROWS; ++r)
                    if (kb + tid <= lim_s[r]) atomicOr(nan_map + r * 4 + (d >> 5), 1u << (d & 31));
                }
              }
              x[w] &= ~((hit >> 7) * 0xffu);
            }
            if (any) sts128(at, make_uint4(x[0], x[1], x[2], x[3]));
          }
        }
        // Weights, times 2^8 vs / vref with vs / vref in [2^-4, 1]. vref
        // follows vs, a smaller one down to 2^-60 of the largest only, so
        // that z cannot overflow. Blocks further apart go one after another.
        uint32_t todo = meta->single ? 0u : found;
        bool fresh = begins;  // z holds nothing yet
        bool again = false;   // a further round
        const uint32_t p_at = tmem + lanes + S_COL + b * KEYS;
        do {
          float top = meta->top;
          uint32_t take = found;
          if (todo) {
            take = take_of(meta, todo, top);
            todo &= ~take;
          }
          const float seen = vtop;
          vtop = fmaxf(vtop, top);
          float by = 1.f;
          if (top > 0.f && (top > vref || top < 0.25f * vref)) {
            const float to = fmaxf(top, vtop * 8.6736173798840355e-19f);  // 2^-60
            if (seen > 0.f) by = vref / to;
            vref = to;
          }
          // z may be changed, and weights of this group replaced, only behind
          // the products so far (all but the last one are: the scores of this
          // group came after them)
          const float f = alpha * by;
          const bool scales = !fresh && __any_sync(0xffffffffu, f != 1.f);
          if (scales || again) {
            ok = __all_sync(0xffffffffu, mbar_wait(p_free, (pv - 1) & 1, ctl));
            if (!ok) break;
            if (scales) scale_z(f);
          }
          alpha = 1.f;
          fresh = false;
          again = true;
          uint32_t hi[4 * F::SUBS], lo[4 * F::SUBS];
#pragma unroll
          for (int i = 0; i < F::SUBS; ++i) {
            const float r = take >> (sub0 + i) & 1 ? 256.f * (meta->vs[sub0 + i] / vref) : 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              split4<4>(s[i][4 * k] * r, s[i][4 * k + 1] * r, s[i][4 * k + 2] * r, s[i][4 * k + 3] * r,
                        hi[4 * i + k], lo[4 * i + k]);
          }
          if constexpr (WIDE) {
            tmem_st_x2_16<16>(p_at, hi);
            tmem_st_x2_16<16>(p_at + 32, lo);
          } else {
            tmem_st_x2_4<4>(p_at + 8 * q, hi);
            tmem_st_x2_4<4>(p_at + 8 * q + lo_lanes, lo);
            // no weight for the other warps' keys
            tmem_zero8(p_at + ((8 * q + 8) & 31));
            tmem_zero8(p_at + ((8 * q + 16) & 31));
            tmem_zero8(p_at + ((8 * q + 24) & 31));
          }
          tmem_wait_st();
          if (masked) fence_async_shared();  // value rows may have been mended
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full);
          ++pv;
        } while (todo);
      }
      if (ends) {
        // ---- the summary of the keys [start_gi, cc.gi] of the tile ----
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(p_free, (pv - 1) & 1, ctl));
        tc_fence_after();
        const bool whole = start_gi == 0 && cc.gi == cc.ng - 1;
        const int kv = cc.pr / P.tiles, rt = cc.pr - kv * P.tiles;
        const long long slot = 2ll * blockIdx.x + (start_gi == 0 ? 1 : 0);
        float* const pz = P.part + 4ll * P.ranges * P.slot_rows;
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const bool none = limit < 0 || l == 0.f;
        // columns [c, c + 16) of row r: v = z sum, to Z or to the workspace
        auto store = [&](int r, int c, const float (&v)[16], float scale) {
          const int rr = rt * F::ROWS + r;
          if (rr >= P.n_q * P.share || c >= P.d_vh) return;
          const int i = rr / P.share, head = kv * P.share + (rr - i * P.share);
          const uint32_t bad = nan_map[r * 4 + (c >> 5)] >> (c & 31);
          float o[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = bad >> k & 1 ? __int_as_float(0x7fffffff) : v[k] * scale;
          if (whole) {
            uint4* z = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.Z) +
                                                ((long long)cc.b * P.n_q + i) * P.h * P.d_vh +
                                                (long long)head * P.d_vh + c);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              z[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
          } else {
            float4* z = reinterpret_cast<float4*>(pz + (slot * P.slot_rows + r) * P.d_vh + c);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              z[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        };
        if constexpr (WIDE) {
          const float scale = none ? 0.f : 0.00390625f * (whole ? 1.f / l : 1.f);  // 2^-8
          if (ok && !whole && half == 0 && rt * F::ROWS + row < P.n_q * P.share) {
            P.part[2 * (slot * P.slot_rows + row)] = none ? -INFINITY : m;
            P.part[2 * (slot * P.slot_rows + row) + 1] = none ? 0.f : l;
          }
#pragma unroll
          for (int cb = 0; cb < 2; ++cb) {
            if (!ok) continue;
            uint32_t x[32], y[32];
            tmem_ld_x2_32<64>(tmem + lanes + Z_COL + 32 * cb, x);
            tmem_ld_x2_32<64>(tmem + lanes + Z_COL + 128 + 32 * cb, y);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; c += 16) {
              float v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k)
                v[k] = none ? 0.f : fmaf(__uint_as_float(y[c + k]), 0.0625f, __uint_as_float(x[c + k])) * vref;
              store(row, 64 * half + 32 * cb + c, v, scale);
            }
          }
        } else {
          // four warps' summaries of the same rows, merged in shared memory
          float* mz = reinterpret_cast<float*>(smem + F::M_AT);   // [4][16][128], pieces of 4 swizzled
          float* ml = reinterpret_cast<float*>(smem + F::ML_AT);  // [4][16][2]
          if (half == 0) {
            ml[(q * 16 + row) * 2] = none ? -INFINITY : m;
            ml[(q * 16 + row) * 2 + 1] = none ? 0.f : l;
          }
#pragma unroll
          for (int cb = 0; cb < 2; ++cb) {
            if (!ok) continue;
            uint32_t x[32], y[32];
            tmem_ld_x2_32<64>(tmem + lanes + Z_COL + 32 * cb, x);
            tmem_ld_x2_32<64>(tmem + lanes + lo_lanes + Z_COL + 32 * cb, y);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                v[k] = none ? 0.f
                            : fmaf(__uint_as_float(y[c + k]), 0.0625f, __uint_as_float(x[c + k])) * 0.00390625f * vref;
              const int piece = (64 * half + 32 * cb + c) >> 2;
              *reinterpret_cast<float4*>(mz + (q * 16 + row) * 128 + ((piece ^ (row & 7)) << 2)) =
                  make_float4(v[0], v[1], v[2], v[3]);
            }
          }
          softmax_sync<NST>();
          const int r = tid >> 3, c = (tid & 7) * 16;
          float mm = -INFINITY, ll = 0.f, w4[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml[(w * 16 + r) * 2]);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float mw = ml[(w * 16 + r) * 2], lw = ml[(w * 16 + r) * 2 + 1];
            // the empty summary weighs nothing; a NaN one has no m but an l
            w4[w] = mw == mm ? 1.f : ex2_approx(mw - mm);
            if (mw == -INFINITY && lw == 0.f) w4[w] = 0.f;
            ll += w4[w] * lw;
          }
          float v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (w4[w] == 0.f) continue;
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 u = *reinterpret_cast<const float4*>(mz + (w * 16 + r) * 128 +
                                                               ((((c + k) >> 2) ^ (r & 7)) << 2));
              v[k] = fmaf(w4[w], u.x, v[k]);
              v[k + 1] = fmaf(w4[w], u.y, v[k + 1]);
              v[k + 2] = fmaf(w4[w], u.z, v[k + 2]);
              v[k + 3] = fmaf(w4[w], u.w, v[k + 3]);
            }
          }
          if (ok) {
            if (!whole && (tid & 7) == 0 && rt * F::ROWS + r < P.n_q * P.share) {
              P.part[2 * (slot * P.slot_rows + r)] = mm;
              P.part[2 * (slot * P.slot_rows + r) + 1] = ll;
            }
            store(r, c, v, whole ? (ll == 0.f ? 0.f : 1.f / ll) : 1.f);
          }
        }
        tc_fence_before();
      }
      begins = ends;
      advance(cc, first, P.B, unit);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <bool WIDE>
cudaError_t launch(const CacheAttnParams& P, int ctas, cudaStream_t s) {
  auto* kernel = cache_attention_tc_kernel<WIDE>;
  if (!ensure_smem_limit(reinterpret_cast<const void*>(kernel), Form<WIDE>::SMEM))
    return cudaErrorUnknown;
  return launch_dependent(kernel, dim3(ctas), dim3(Form<WIDE>::THREADS), Form<WIDE>::SMEM, s, P);
}

}  // namespace

mha_status launch_cache_attention_tc(CacheAttnParams& P, cudaStream_t s) {
  int box = KEYS;  // the largest box that blocks are made of
  while (P.bt % box) box /= 2;
  if (!make_cache_maps(P, box, ROW)) return MHA_ERR_CUDA;
  const int ctas = num_sms() < CA_MAX_CTAS ? num_sms() : CA_MAX_CTAS;
  P.ranges = ctas;
  cudaError_t e = P.tile_rows == 16 ? launch<false>(P, ctas, s) : launch<true>(P, ctas, s);
  if (e == cudaSuccess) e = launch_cache_merge(P, MHA_DTYPE_BF16, s);
  count_launch(2);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // namespace mha
