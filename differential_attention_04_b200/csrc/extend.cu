// Differential attention of new tokens over a paged cache, d in {64, 128},
// bf16 in and out, float32 arithmetic: the schedule of a step and the plain
// kernel.
//
// Query i of a request with n new tokens and L cached ones (the new ones
// included) sees keys 0 .. L - n + i (causal) or all L; a row that sees no key
// gives zeros.  Per head it is the DiffAttn equation (peer review
// "Differential Transformer", Summary, Eq. 1), the headwise RMSNorm and the
// (1 - lambda_init) scale (Eq. 3).
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace diffattn {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;

__device__ __forceinline__ void note_bounds(int* status) { atomicCAS(status, 0, 6); }

// Per token: (request, last visible key); request -1 for rows behind the last one.
__global__ void extend_plan_kernel(const int* __restrict__ cu, const int* __restrict__ kvl, ExtendShape n, int causal,
                                   int2* tok, int* status) {
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= n.T) return;
  int2 e = make_int2(-1, -1);
  if (t < cu[n.S]) {
    int lo = 0, hi = n.S - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (cu[m] <= t) lo = m;
      else hi = m - 1;
    }
    const int nq = cu[lo + 1] - cu[lo], L = kvl[lo];
    if (nq > n.max_new || L < 0) note_bounds(status);
    else e = make_int2(lo, causal ? L - nq + (t - cu[lo]) : L - 1);
  }
  tok[t] = e;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) extend_plain_kernel(const ExtendArgs a, int* status) {
  constexpr int E = 2 * D / 32;  // elements of a row per lane
  const int t = blockIdx.x, h = blockIdx.y, hk = h / (a.n.H / a.n.H_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, map = lane >> 4;
  const int2 e = static_cast<const int2*>(a.plan)[t];
  if (e.x < 0) return;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<size_t>(t) * a.n.H + h) * 2 * D;
  float qf[E], o[2][E], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qf[i] = __bfloat162float(q[E * lane + i]) * (kLog2e * rsqrtf(static_cast<float>(D)));
    o[0][i] = o[1][i] = 0.f;
  }
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.k_cache);
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.v_cache);
  for (int key = warp; key <= e.y; key += kWarps) {
    const int j = key / a.page_size;
    const int page = j < a.max_pages ? a.block_table[static_cast<size_t>(e.x) * a.max_pages + j] : -1;
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok) note_bounds(status);
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
    for (int w = 0; w < 2; ++w) {
      const float mn = fmaxf(m[w], sc[w]), al = fast_exp2(m[w] - mn), p = fast_exp2(sc[w] - mn);
      m[w] = mn;
      l[w] = l[w] * al + p;
#pragma unroll
      for (int i = 0; i < E; ++i) o[w][i] = fmaf(o[w][i], al, p * v[i]);
    }
  }
  __shared__ float sm_m[kWarps][2], sm_l[kWarps][2], sm_o[kWarps][2][2 * D], red[kWarps];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (lane == 0) {
      sm_m[warp][w] = m[w];
      sm_l[warp][w] = l[w];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) sm_o[warp][w][E * lane + i] = o[w][i];
  }
  __syncthreads();
  const float c2 = map2_coefficient(a.mode, *a.lambda);
  float y[2 * D / (kWarps * 32)], ss = 0.f;
#pragma unroll
  for (int i = 0; i < 2 * D / (kWarps * 32); ++i) {
    const int c = threadIdx.x + i * kWarps * 32;
    float ov = 0.f;
    for (int w = 0; w < 2; ++w) {
      float M = -INFINITY, L = 0.f, x = 0.f;
      for (int g = 0; g < kWarps; ++g) M = fmaxf(M, sm_m[g][w]);
      for (int g = 0; g < kWarps; ++g) {
        const float f = M == -INFINITY ? 0.f : fast_exp2(sm_m[g][w] - M);
        L = fmaf(f, sm_l[g][w], L);
        x = fmaf(f, sm_o[g][w][c], x);
      }
      ov += L > 0.f ? (w ? c2 : 1.f) * x / L : 0.f;
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

size_t extend_plan_bytes(const ExtendShape& n) { return static_cast<size_t>(n.T > 0 ? n.T : 1) * sizeof(int2) + 16; }
size_t extend_workspace_bytes(const ExtendShape&) { return 0; }

cudaError_t launch_extend_plan(const int* cu_q, const int* kv_lens, const ExtendShape& n, int causal, void* plan,
                               DevCtl ctl, cudaStream_t stream) {
  if (n.T == 0) return cudaSuccess;
  extend_plan_kernel<<<(n.T + 255) / 256, 256, 0, stream>>>(cu_q, kv_lens, n, causal, static_cast<int2*>(plan),
                                                            ctl.status);
  return cudaGetLastError();
}

cudaError_t launch_extend(const ExtendArgs& a, DevCtl ctl, cudaStream_t stream) {
  const dim3 grid(a.n.T, a.n.H);
  if (a.n.d == 128) extend_plain_kernel<128><<<grid, kWarps * 32, 0, stream>>>(a, ctl.status);
  else extend_plain_kernel<64><<<grid, kWarps * 32, 0, stream>>>(a, ctl.status);
  return cudaGetLastError();
}

}  // namespace diffattn
