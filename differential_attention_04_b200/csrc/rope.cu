// Rotary positions outside the projections: queries and keys rotated at given
// positions (forward, and the inverse that is its gradient), and the same
// rotation fused with the write of keys and values into a paged cache.
//
// Rotary embedding as in RoFormer (cited on page "Differential Transformer",
// "Builds on"): the pair (a, b) of channels with frequency theta_j becomes
//   a' = m (a cos - b sin),  b' = m (a sin + b cos)   at the angle n theta_j
// with m = 1 unless the table is a scaled one.  The map is m times a rotation,
// so its transpose (what a gradient needs) is the same with sin negated.
// Pairs are channels (2j, 2j + 1) ("interleaved") or (j, j + rot / 2)
// ("half"); channels from rot on are copied.
//
// HBM-bound: every element is read once and written once.  A CTA takes one
// token at a time; a thread keeps one unit of channels (16 bytes, or the two
// 16-byte halves of the same pairs) and walks the token's head rows with it,
// so cos and sin are read once per thread rather than once per row.  The rows
// are those of q, then of k, then (cache write) of v, each d wide: the two
// maps of a head are two rows, and a head's 2d values are two rows too.
// Rotation in float32, one rounding to the storage type at the end.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace diffattn {

namespace {

constexpr int kRopeThreads = 256;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T x[VEC];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ void record_bounds(int* status) { atomicCAS(status, 0, 6); }

// VEC elements a load; HALF: pairs (j, j + rot/2), a unit holds both ends.
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const RopeParams p) {
  const int half = p.rot / 2;
  const int rot_units = HALF ? half / VEC : p.rot / VEC;
  const int units = rot_units + (p.d - p.rot) / VEC;
  const int q_rows = 2 * p.H, k_rows = 2 * p.H_kv;
  const int rows = q_rows + k_rows + (p.v ? k_rows : 0);
  const int lanes = kRopeThreads / units > 0 ? kRopeThreads / units : 1;  // rows side by side
  using V = Vec<T, VEC>;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int pos = p.table ? p.positions[t] : 0;
    if (pos < 0) continue;  // a padding row
    if (p.table && pos >= p.n_pos) {
      if (threadIdx.x == 0) record_bounds(p.status);
      continue;
    }
    // rows of this token's keys and values: its own, or its slot of the cache
    long long kv_row = t;
    bool kv_ok = true;
    if (p.slots) {
      const int slot = p.slots[t];
      kv_ok = slot >= 0 && slot < p.num_slots;
      if (slot >= p.num_slots && threadIdx.x == 0) record_bounds(p.status);
      kv_row = slot;
    }
    for (int i = threadIdx.x; i < units * lanes; i += kRopeThreads) {
      const int u = i % units;
      const bool rotated = u < rot_units;
      const int c0 = HALF ? (rotated ? u * VEC : p.rot + (u - rot_units) * VEC) : u * VEC;
      constexpr int NP = HALF ? VEC : VEC / 2;  // pairs of a unit
      float cs[NP], sn[NP];
      if (rotated && p.table) {
        const float2* tb = reinterpret_cast<const float2*>(p.table) + static_cast<size_t>(pos) * half +
                           (HALF ? c0 : c0 / 2);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const float2 x = __ldg(tb + j);
          cs[j] = x.x;
          sn[j] = p.inverse ? -x.y : x.y;
        }
      }
      for (int r = i / units; r < rows; r += lanes) {
        const T* src;
        T* dst;
        bool turn = rotated && p.table;
        if (r < q_rows) {
          const size_t at = (static_cast<size_t>(t) * q_rows + r) * p.d;
          src = static_cast<const T*>(p.q) + at;
          dst = static_cast<T*>(p.q_out) + at;
        } else {
          if (!kv_ok) break;
          const bool is_v = r >= q_rows + k_rows;
          const int rr = r - q_rows - (is_v ? k_rows : 0);
          src = static_cast<const T*>(is_v ? p.v : p.k) + (static_cast<size_t>(t) * k_rows + rr) * p.d;
          dst = static_cast<T*>(is_v ? p.v_out : p.k_out) + (static_cast<size_t>(kv_row) * k_rows + rr) * p.d;
          if (is_v) turn = false;
        }
        V a = *reinterpret_cast<const V*>(src + c0);
        if constexpr (HALF) {
          V b;
          if (rotated) b = *reinterpret_cast<const V*>(src + c0 + half);
          if (turn) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              const float x = to_f(a.x[j]), y = to_f(b.x[j]);
              a.x[j] = from_f<T>(fmaf(x, cs[j], -y * sn[j]));
              b.x[j] = from_f<T>(fmaf(x, sn[j], y * cs[j]));
            }
          }
          *reinterpret_cast<V*>(dst + c0) = a;
          if (rotated) *reinterpret_cast<V*>(dst + c0 + half) = b;
        } else {
          if (turn) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const float x = to_f(a.x[2 * j]), y = to_f(a.x[2 * j + 1]);
              a.x[2 * j] = from_f<T>(fmaf(x, cs[j], -y * sn[j]));
              a.x[2 * j + 1] = from_f<T>(fmaf(x, sn[j], y * cs[j]));
            }
          }
          *reinterpret_cast<V*>(dst + c0) = a;
        }
      }
    }
  }
}

// Frequencies of the scaled tables, in double precision:
//   linear: theta / s;  NTK: base * s^(rot/(rot-2));  YaRN (Peng et al. 2023):
//   theta (g + (1 - g) / s) with g rising from 0 to 1 as the turns that the
//   original length makes of theta go from beta_slow to beta_fast, and cos and
//   sin times 0.1 ln s + 1.
__global__ void rope_table_scaled_kernel(int seq_len, int rot, double base, int scaling, double factor, int orig_len,
                                         double beta_fast, double beta_slow, float2* table) {
  const int half = rot / 2;
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<long long>(seq_len) * half) return;
  const int n = static_cast<int>(i / half), j = static_cast<int>(i % half);
  if (scaling == 2) base *= pow(factor, static_cast<double>(rot) / (rot - 2));
  double f = pow(base, -2.0 * j / rot), m = 1.0;
  if (scaling == 1) f /= factor;
  if (scaling == 3) {
    const double turns = orig_len * f / 6.283185307179586476925286766559;
    const double g = fmin(1.0, fmax(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
    f = f * g + f / factor * (1.0 - g);
    m = 0.1 * log(factor) + 1.0;
  }
  double s, c;
  sincos(n * f, &s, &c);
  table[i] = make_float2(static_cast<float>(c * m), static_cast<float>(s * m));
}

template <typename T, int FULL>
cudaError_t launch_rows(const RopeParams& p, int layout, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.T);
  // 16-byte units where the pairs allow it; else one pair at a time
  const bool wide = layout == 0 ? p.rot % FULL == 0 : (p.rot / 2) % FULL == 0;
  if (layout == 0) {
    if (wide)
      rope_rows_kernel<T, FULL, false><<<grid, kRopeThreads, 0, stream>>>(p);
    else
      rope_rows_kernel<T, 2, false><<<grid, kRopeThreads, 0, stream>>>(p);
  } else {
    if (wide)
      rope_rows_kernel<T, FULL, true><<<grid, kRopeThreads, 0, stream>>>(p);
    else
      rope_rows_kernel<T, 1, true><<<grid, kRopeThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_rows(const RopeParams& p, int bf16, int layout, cudaStream_t stream) {
  return bf16 ? launch_rows<__nv_bfloat16, 8>(p, layout, stream) : launch_rows<float, 4>(p, layout, stream);
}

cudaError_t launch_rope_table_scaled(int seq_len, int rot, double base, int scaling, double factor, int orig_len,
                                     double beta_fast, double beta_slow, float* table, cudaStream_t stream) {
  const long long n = static_cast<long long>(seq_len) * (rot / 2);
  rope_table_scaled_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(
      seq_len, rot, base, scaling, factor, orig_len, beta_fast, beta_slow, reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

}  // namespace diffattn
