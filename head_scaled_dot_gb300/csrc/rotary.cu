// rotary.cu - rotary positions with several axes, applied to head-split
// queries and keys.
//
// Row t of batch item b has one position per axis (time, height, width, ...).
// Pair i of a row's first 2 P columns turns by the angle
//   theta = position(axis(i), b, t) * w_i,
//   (x, y) -> (x cos theta - y sin theta, x sin theta + y cos theta);
// the inverse turns by -theta, which is also the gradient: a rotation's
// transpose is its inverse.
//
// Angles. w_i comes as the 64-bit fraction F_i = round(w_i / (2 pi) * 2^64) of
// a turn, so position * F_i mod 2^64 is the angle's fraction of a turn with
// the whole turns already gone: the range reduction is one exact integer
// product, and a position of 2^20 turns as exactly as a position of 1. The
// top 32 bits, as a signed number, are the angle in units of pi / 2^31, and
// sincospi takes it from there. In fp32 the product position * w alone would
// be off by 2^-24 of the angle, 0.06 radians at position 10^6.
//
// The work is bound by memory: every value is read once and written once.
// A thread holds the sines and cosines of one vector of pairs of one row and
// walks over heads with them, so each angle is computed once per row and
// group of heads, not once per head.
#include <cuda_bf16.h>

#include "device_common.cuh"
#include "internal.h"

namespace mha {
namespace {

constexpr int ROT_THREADS = 256;

struct RotaryParams {
  const void* x[2];  // Q, K
  void* y[2];
  int heads[2];
  const int32_t* positions;  // (n_axes, B, T)
  const uint64_t* steps;     // one per pair
  int cut[MHA_MAX_ROTARY_AXES];  // first pair of axis a + 1
  int n_axes;
  int T, d, pairs;
  long long rows;   // B T
  int chunks;       // vectors of a row: the rotated ones, then the copied rest
  int rot_chunks;
  int group;        // heads per thread
  int inverse;
};

// N elements of T as one aligned load or store of N * sizeof(T) bytes.
template <typename T, int N>
struct alignas(N * sizeof(T)) Pack {
  T v[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// One thread: vector `chunk` of row `row`, for `group` heads of Q and K
// (numbered Q first). Half-split pairing (i, i + P): N pairs are two vectors
// of N elements; interleaved pairing (2i, 2i + 1): one vector of N elements
// holds N / 2 pairs (N = 1 when pairs cannot be read as one vector).
template <typename T, int N, bool INTERLEAVED>
__global__ void __launch_bounds__(ROT_THREADS, 4) rotary_kernel(const __grid_constant__ RotaryParams P) {
  constexpr int NP = INTERLEAVED ? N / 2 : N;  // pairs per thread
  using V = Pack<T, N>;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const long long e = (long long)blockIdx.x * ROT_THREADS + threadIdx.x;
  const long long row = e / P.chunks;
  if (row >= P.rows) return;
  const int chunk = (int)(e - row * P.chunks);
  const int b = (int)(row / P.T), t = (int)(row % P.T);
  const bool rotated = chunk < P.rot_chunks;

  float cs[NP], sn[NP];
  if (rotated) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int i = chunk * NP + j;
      int axis = 0;
#pragma unroll
      for (int a = 0; a + 1 < MHA_MAX_ROTARY_AXES; ++a) axis += a + 1 < P.n_axes && i >= P.cut[a];
      const long long pos = __ldg(P.positions + axis * P.rows + row);
      const uint64_t turn = (uint64_t)pos * __ldg(P.steps + i);
      sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sn[j], &cs[j]);  // 2^-31
      if (P.inverse) sn[j] = -sn[j];
    }
  }
  // first element of the vector (of the second one: + P.pairs)
  const int col = !rotated ? 2 * P.pairs + (chunk - P.rot_chunks) * N : chunk * N;
  // Heads in batches of HB, whose loads are all under way before the first
  // store: an output may be its own input, so the compiler cannot move a load
  // above the store before it. 64 bytes a thread; more, or a fourth CTA's
  // registers taken away, is slower: 16,384 rows of 2 x 16 heads of 128 in bf16
  // take 49 us so, 59 us head by head, 55 with two heads and any number of
  // registers, 67 with four (a copy of the same bytes: 43).
  constexpr int HB = INTERLEAVED ? 4 : 2;
  const int h0 = blockIdx.y * P.group, h1 = min(h0 + P.group, P.heads[0] + P.heads[1]);
  const long long stride = (long long)P.T * P.d, in_head = (long long)t * P.d + col;
  for (int hb = h0; hb < h1; hb += HB) {
    V u[HB], w[INTERLEAVED ? 1 : HB];
    auto place = [&](int hh, int& which) {
      which = hh >= P.heads[0];
      return ((long long)b * P.heads[which] + (which ? hh - P.heads[0] : hh)) * stride + in_head;
    };
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      if (hb + k < h1) {
        int which;
        const long long at = place(hb + k, which);
        const T* x = static_cast<const T*>(P.x[which]) + at;
        u[k] = *reinterpret_cast<const V*>(x);
        if constexpr (!INTERLEAVED) {
          if (rotated) w[k] = *reinterpret_cast<const V*>(x + P.pairs);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      if (hb + k < h1) {
        int which;
        const long long at = place(hb + k, which);
        T* y = static_cast<T*>(P.y[which]) + at;
        if (rotated) {
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const float p = to_f(u[k].v[2 * j]), q = to_f(u[k].v[2 * j + 1]);
              from_f(u[k].v[2 * j], p * cs[j] - q * sn[j]);
              from_f(u[k].v[2 * j + 1], p * sn[j] + q * cs[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const float p = to_f(u[k].v[j]), q = to_f(w[k].v[j]);
              from_f(u[k].v[j], p * cs[j] - q * sn[j]);
              from_f(w[k].v[j], p * sn[j] + q * cs[j]);
            }
            *reinterpret_cast<V*>(y + P.pairs) = w[k];
          }
        }
        *reinterpret_cast<V*>(y) = u[k];
      }
    }
  }
}

template <typename T, int N>
cudaError_t launch(RotaryParams& P, bool interleaved, cudaStream_t s) {
  P.rot_chunks = (interleaved ? 2 * P.pairs : P.pairs) / N;
  // the columns past the pairs are copied, unless they are in place already
  P.chunks = P.rot_chunks;
  if (P.x[0] != P.y[0] || (P.heads[1] && P.x[1] != P.y[1]))
    P.chunks += (P.d - 2 * P.pairs) / N;
  const long long threads = P.rows * P.chunks;
  const int heads = P.heads[0] + P.heads[1];
  // as many heads per thread as leave every SM its threads (four CTAs' worth)
  const long long want = (long long)num_sms() * 1024;
  long long groups = (want + threads - 1) / threads;
  if (groups > heads) groups = heads;
  P.group = (int)((heads + groups - 1) / groups);
  const dim3 grid((unsigned)((threads + ROT_THREADS - 1) / ROT_THREADS),
                  (unsigned)((heads + P.group - 1) / P.group));
  if (interleaved) {
    if constexpr (N > 1)
      return launch_dependent(rotary_kernel<T, N, true>, grid, dim3(ROT_THREADS), 0, s, P);
    else
      return cudaErrorInvalidValue;
  }
  return launch_dependent(rotary_kernel<T, N, false>, grid, dim3(ROT_THREADS), 0, s, P);
}

template <typename T>
cudaError_t launch_type(RotaryParams& P, bool interleaved, cudaStream_t s) {
  // the widest vector that every row, both halves and the rest are made of
  auto fits = [&](int n) {
    return P.d % n == 0 && (interleaved ? 2 * P.pairs % n == 0 : P.pairs % n == 0) &&
           (P.d - 2 * P.pairs) % n == 0;
  };
  constexpr int W = 16 / (int)sizeof(T);
  if (fits(W)) return launch<T, W>(P, interleaved, s);
  if (fits(W / 2)) return launch<T, W / 2>(P, interleaved, s);
  if constexpr (W / 4 >= 2) {
    if (fits(W / 4)) return launch<T, W / 4>(P, interleaved, s);
  }
  return launch<T, 1>(P, interleaved, s);
}

}  // namespace

mha_status rotary(const RotaryArgs& a, mha_dtype dt, cudaStream_t s) {
  RotaryParams P{};
  P.x[0] = a.Q;
  P.x[1] = a.K;
  P.y[0] = a.Q_out;
  P.y[1] = a.K_out;
  P.heads[0] = a.h;
  P.heads[1] = a.K ? a.h_kv : 0;
  P.positions = a.positions;
  P.steps = a.steps;
  P.n_axes = a.n_axes;
  P.T = a.T;
  P.d = a.d;
  P.rows = (long long)a.B * a.T;
  P.inverse = a.inverse;
  for (int i = 0; i < a.n_axes; ++i) {
    P.pairs += a.sections[i];
    P.cut[i] = P.pairs;
  }
  const cudaError_t e = dt == MHA_DTYPE_F32 ? launch_type<float>(P, a.interleaved, s)
                                            : launch_type<__nv_bfloat16>(P, a.interleaved, s);
  count_launch();
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // namespace mha
