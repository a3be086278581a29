// Attention of requests with more than 8 query rows per key head over a paged
// cache: one block per row, float32 throughout.
#include <math.h>

#include "common.cuh"
#include "extend.cuh"

namespace diffattn {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) extend_wide_kernel(const ExtendArgs a, int max_keys, int* status) {
  constexpr int E = 2 * D / 32;  // elements of a row per lane
  const int G = a.n.H / a.n.H_kv, hk = blockIdx.y, r = blockIdx.z;
  if (!plan_fits(a.plan, a.n, status)) return;
  const PlanView pv = plan_view(a.plan, a.n, 1);
  if (blockIdx.x >= pv.head->tiles) return;
  const WideTile w = pv.wide[blockIdx.x];
  if (r >= w.ntok * G) return;
  const int t = w.tok0 + r / G, h = hk * G + r % G;
  const int L = min(w.L, max_keys);
  if (w.L > max_keys && threadIdx.x == 0) atomicCAS(status, 0, 6);
  const int last = min(w.lim0 + (pv.head->causal ? r / G : 0), L - 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, map = lane >> 4;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(t) * a.n.H + h) * 2 * D;
  float qf[E], o[2][E], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qf[i] = __bfloat162float(q[E * lane + i]) * (kLog2e * rsqrtf(static_cast<float>(D)));
    o[0][i] = o[1][i] = 0.f;
  }
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.k_cache);
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.v_cache);
  for (int key = warp; key <= last; key += kWarps) {
    const int page = a.block_table[static_cast<size_t>(w.s) * a.max_pages + key / a.page_size];
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok) atomicCAS(status, 0, 6);
    const size_t row = ((static_cast<size_t>(ok ? page : 0) * a.page_size + key % a.page_size) * a.n.H_kv + hk) * 2 * D;
    float s = 0.f, v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      s = fmaf(qf[i], ok ? __bfloat162float(kc[row + E * lane + i]) : 0.f, s);
      v[i] = ok ? __bfloat162float(vc[row + E * lane + i]) : 0.f;
    }
#pragma unroll
    for (int off = 8; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float other = __shfl_xor_sync(0xffffffffu, s, 16);
    const float sc[2] = {map ? other : s, map ? s : other};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float mn = fmaxf(m[j], sc[j]), al = fast_exp2(m[j] - mn), p = fast_exp2(sc[j] - mn);
      m[j] = mn;
      l[j] = l[j] * al + p;
#pragma unroll
      for (int i = 0; i < E; ++i) o[j][i] = fmaf(o[j][i], al, p * v[i]);
    }
  }
  __shared__ float sm_m[kWarps][2], sm_l[kWarps][2], sm_o[kWarps][2][2 * D], red[kWarps];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (lane == 0) {
      sm_m[warp][j] = m[j];
      sm_l[warp][j] = l[j];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) sm_o[warp][j][E * lane + i] = o[j][i];
  }
  __syncthreads();
  const float c2 = map2_coefficient(a.mode, *a.lambda);
  float y[2 * D / (kWarps * 32)], ss = 0.f;
#pragma unroll
  for (int i = 0; i < 2 * D / (kWarps * 32); ++i) {
    const int c = threadIdx.x + i * kWarps * 32;
    float ov = 0.f;
    for (int j = 0; j < 2; ++j) {
      float M = -INFINITY, sum = 0.f, y0 = 0.f;
      for (int g = 0; g < kWarps; ++g) M = fmaxf(M, sm_m[g][j]);
      for (int g = 0; g < kWarps; ++g) {
        const float f = M == -INFINITY ? 0.f : fast_exp2(sm_m[g][j] - M);
        sum = fmaf(f, sm_l[g][j], sum);
        y0 = fmaf(f, sm_o[g][j][c], y0);
      }
      ov += sum > 0.f ? (j ? c2 : 1.f) * y0 / sum : 0.f;
    }
    y[i] = ov;
    ss = fmaf(ov, ov, ss);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  ss = red[0] + red[1] + red[2] + red[3];
  const float gsc = (1.f - a.lambda_init) * rsqrtf(ss / (2 * D) + a.eps);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + (static_cast<size_t>(t) * a.n.H + h) * 2 * D;
#pragma unroll
  for (int i = 0; i < 2 * D / (kWarps * 32); ++i) {
    const int c = threadIdx.x + i * kWarps * 32;
    out[c] = __float2bfloat16_rn(y[i] * gsc * a.rms_w[c]);
  }
}
}  // namespace

cudaError_t launch_extend_wide(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream) {
  (void)recs;
  const long long keys = static_cast<long long>(a.max_pages) * a.page_size;
  const int max_keys = keys < kMaxKeys ? static_cast<int>(keys) : kMaxKeys;
  const dim3 grid(plan_layout(a.n).max_tiles, a.n.H_kv, kWideRows);
  if (a.n.d == 128) extend_wide_kernel<128><<<grid, kWarps * 32, 0, stream>>>(a, max_keys, ctl.status);
  else extend_wide_kernel<64><<<grid, kWarps * 32, 0, stream>>>(a, max_keys, ctl.status);
  return cudaGetLastError();
}

}  // namespace diffattn
