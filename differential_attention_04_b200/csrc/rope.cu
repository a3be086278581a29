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
// HBM-bound: every element is read once and written once.  A thread keeps one
// unit of channels (16 bytes, or the two 16-byte ends of the same pairs) of
// one token and takes a few of the token's head rows at a time with it, so cos
// and sin are read once per thread rather than once per row, and 64 bytes are
// in flight that wait neither for the position nor for the table.
// The rows are those of q, then of k, then (cache write) of v, each d wide:
// the two maps of a head are two rows, and a head's 2d values are two rows
// too.  A block of 256 threads is units x rows side by side x tokens.
// Rotation in float32, one rounding to the storage type at the end.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace diffattn {

namespace {

constexpr int kRopeThreads = 256;

// VEC channels as they lie in memory, in 32-bit words where they fill one (a
// 16-bit element in a register of its own would halve the rows in flight).
template <typename T, int VEC, bool WORDS = (sizeof(T) * VEC >= 4)>
struct alignas(sizeof(T) * VEC) Unit {
  uint32_t w[sizeof(T) * VEC / 4];
};
template <typename T, int VEC>
struct Unit<T, VEC, false> {
  T w[VEC];
};

__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
  return make_float2(fmaf(a, c, -b * s), fmaf(a, s, b * c));
}

// Pairs (2j, 2j + 1) of a unit.
template <typename T, int VEC>
__device__ __forceinline__ void turn_unit(Unit<T, VEC>& u, const float2 (&cs)[VEC / 2]) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    if constexpr (sizeof(T) == 2) {
      const float2 y = turn(bf16lo_to_f32(u.w[j]), bf16hi_to_f32(u.w[j]), cs[j].x, cs[j].y);
      u.w[j] = pack_bf16x2(y.x, y.y);
    } else {
      const float2 y = turn(__uint_as_float(u.w[2 * j]), __uint_as_float(u.w[2 * j + 1]), cs[j].x, cs[j].y);
      u.w[2 * j] = __float_as_uint(y.x);
      u.w[2 * j + 1] = __float_as_uint(y.y);
    }
  }
}
// Pairs of a channel of `a` and the same one of `b`.
template <typename T, int VEC>
__device__ __forceinline__ void turn_ends(Unit<T, VEC>& a, Unit<T, VEC>& b, const float2 (&cs)[VEC]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float2 y = turn(__uint_as_float(a.w[j]), __uint_as_float(b.w[j]), cs[j].x, cs[j].y);
      a.w[j] = __float_as_uint(y.x);
      b.w[j] = __float_as_uint(y.y);
    }
  } else if constexpr (VEC == 1) {
    const float2 y = turn(__bfloat162float(a.w[0]), __bfloat162float(b.w[0]), cs[0].x, cs[0].y);
    a.w[0] = __float2bfloat16_rn(y.x);
    b.w[0] = __float2bfloat16_rn(y.y);
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const float2 y0 = turn(bf16lo_to_f32(a.w[j]), bf16lo_to_f32(b.w[j]), cs[2 * j].x, cs[2 * j].y);
      const float2 y1 = turn(bf16hi_to_f32(a.w[j]), bf16hi_to_f32(b.w[j]), cs[2 * j + 1].x, cs[2 * j + 1].y);
      a.w[j] = pack_bf16x2(y0.x, y1.x);
      b.w[j] = pack_bf16x2(y0.y, y1.y);
    }
  }
}

__device__ __forceinline__ void record_bounds(int* status) { atomicCAS(status, 0, 6); }

// 64 bytes of a thread in flight: four rows of one vector or two of two.
template <bool HALF>
constexpr int kRopeBatch = HALF ? 2 : 4;

struct RopeGrid {
  int units, lanes, tokens;  // of a block: units of a row, rows side by side, tokens
};

// VEC elements a load; HALF: a unit is two loads, both ends of the pairs
// (j, j + rot/2) or two neighbours of the channels that are copied.
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_rows_kernel(const RopeParams p, const RopeGrid g) {
  const int half = p.rot / 2;
  const int rot_units = HALF ? half / VEC : p.rot / VEC;
  const int q_rows = 2 * p.H, k_rows = 2 * p.H_kv;
  const int rows = q_rows + k_rows + (p.v ? k_rows : 0);
  using V = Unit<T, VEC>;
  const int u = threadIdx.x % g.units, side = threadIdx.x / g.units;
  const int lane = side % g.lanes, tk = side / g.lanes;
  const int t = blockIdx.x * g.tokens + tk;
  if (tk >= g.tokens || t >= p.T) return;
  const bool rotated = u < rot_units;
  constexpr int kBatch = kRopeBatch<HALF>;
  const int c0 = HALF ? (rotated ? u * VEC : p.rot + (u - rot_units) * 2 * VEC) : u * VEC;
  const int second = rotated ? half : VEC;  // of a unit's two loads, behind the first
  const bool has_b = HALF && c0 + second < p.d;
  constexpr int NP = HALF ? VEC : VEC / 2;  // pairs of a unit
  // debug builds: the unit lies in its row, and its pairs in the table's
  if (!DA_CHECK(p.status, c0 + VEC <= p.d && (!has_b || c0 + second + VEC <= p.d) &&
                              (!rotated || (HALF ? c0 : c0 / 2) + NP <= half)))
    return;
  const int pos = p.table ? p.positions[t] : 0;
  // rows of this token's keys and values: its own, or its slot of the cache
  const int slot = p.slots ? p.slots[t] : t;
  for (int r0 = lane; r0 < rows; r0 += g.lanes * kBatch) {
    V a[kBatch], b[HALF ? kBatch : 1];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * g.lanes;
      if (r < rows) {
        const bool is_v = r >= q_rows + k_rows;
        const T* src = r < q_rows ? static_cast<const T*>(p.q) + (static_cast<size_t>(t) * q_rows + r) * p.d
                                  : static_cast<const T*>(is_v ? p.v : p.k) +
                                        (static_cast<size_t>(t) * k_rows + r - q_rows - (is_v ? k_rows : 0)) * p.d;
        a[i] = *reinterpret_cast<const V*>(src + c0);
        if constexpr (HALF) {
          if (has_b) b[i] = *reinterpret_cast<const V*>(src + c0 + second);
        }
      }
    }
    if (pos < 0 || (p.table && pos >= p.n_pos)) {  // a padding row, or one without an angle: left as it is, or zeros
      if (pos >= 0) record_bounds(p.status);
      if (!p.pad_zero) return;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * g.lanes;
        if (r >= rows || (r >= q_rows && p.slots)) continue;  // (a cache's rows are left)
        T* dst = r < q_rows ? static_cast<T*>(p.q_out) + (static_cast<size_t>(t) * q_rows + r) * p.d
                            : static_cast<T*>(p.k_out) + (static_cast<size_t>(t) * k_rows + r - q_rows) * p.d;
        *reinterpret_cast<V*>(dst + c0) = V{};
        if (has_b) *reinterpret_cast<V*>(dst + c0 + second) = V{};
      }
      continue;
    }
    if (p.slots && slot >= p.num_slots) record_bounds(p.status);
    const bool kv_ok = !p.slots || (slot >= 0 && slot < p.num_slots);
    float2 cs[NP];
    if (rotated && p.table) {
      const float2* tb = reinterpret_cast<const float2*>(p.table) + static_cast<size_t>(pos) * half +
                         (HALF ? c0 : c0 / 2);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        cs[j] = __ldg(tb + j);
        if (p.inverse) cs[j].y = -cs[j].y;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * g.lanes;
      const bool is_v = r >= q_rows + k_rows;
      if (r >= rows || (r >= q_rows && !kv_ok)) continue;
      T* dst = r < q_rows ? static_cast<T*>(p.q_out) + (static_cast<size_t>(t) * q_rows + r) * p.d
                          : static_cast<T*>(is_v ? p.v_out : p.k_out) +
                                (static_cast<size_t>(slot) * k_rows + r - q_rows - (is_v ? k_rows : 0)) * p.d;
      const bool turned = rotated && p.table && !is_v;
      if constexpr (HALF) {
        if (turned) turn_ends<T, VEC>(a[i], b[i], cs);
        *reinterpret_cast<V*>(dst + c0) = a[i];
        if (has_b) *reinterpret_cast<V*>(dst + c0 + second) = b[i];
      } else {
        if (turned) turn_unit<T, VEC>(a[i], cs);
        *reinterpret_cast<V*>(dst + c0) = a[i];
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

template <typename T, int VEC, bool HALF>
cudaError_t launch_units(const RopeParams& p, cudaStream_t stream) {
  const int rows = 2 * p.H + 2 * p.H_kv * (p.v ? 2 : 1);
  RopeGrid g;
  g.units = HALF ? p.rot / 2 / VEC + (p.d - p.rot + 2 * VEC - 1) / (2 * VEC) : p.d / VEC;
  // the split of a block's threads that leaves the fewest of them idle: rows
  // side by side such that a thread takes k batches of a token
  const int room = kRopeThreads / g.units;
  int used = 0;
  for (int k = 1; k <= 4; ++k) {
    const int want = (rows + kRopeBatch<HALF> * k - 1) / (kRopeBatch<HALF> * k), lanes = want < room ? want : room;
    const int tokens = room / lanes;
    if (lanes * tokens > used) {
      used = lanes * tokens;
      g.lanes = lanes;
      g.tokens = tokens;
    }
  }
  rope_rows_kernel<T, VEC, HALF>
      <<<static_cast<unsigned>((p.T + g.tokens - 1) / g.tokens), kRopeThreads, 0, stream>>>(p, g);
  return cudaGetLastError();
}

template <typename T, int FULL>
cudaError_t launch_rows(const RopeParams& p, int layout, cudaStream_t stream) {
  // 16-byte units where the pairs allow it; else one pair at a time
  if (layout == 0)
    return p.rot % FULL == 0 ? launch_units<T, FULL, false>(p, stream) : launch_units<T, 2, false>(p, stream);
  return (p.rot / 2) % FULL == 0 ? launch_units<T, FULL, true>(p, stream) : launch_units<T, 1, true>(p, stream);
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
