// Attention of requests with at most 8 query rows per key head (single tokens,
// drafted tokens, small groups of shared heads) over a paged cache.
//
// HBM-bound: 8 d bytes of K and V per key and key head against 12 d flops per
// row.  All 8 rows go through the matrix units at once, so the arithmetic does
// not grow with the rows: with keys and channels as the M dimension of
// m16n8k16 (S^T = K Q^T, O^T = V^T P^T) the rows are the N = 8 columns.  The
// warp-level instruction is taken on purpose: tcgen05 has M = 128 and would
// put P through shared memory, and the kernel needs less than a fifth of the
// warp-level rate (48 instructions per 16 keys at d = 128) to run at the
// speed of memory.
//
// A CTA of four warps per SM takes a contiguous range of the step's units of
// 128 keys (extend.cuh).  Within a unit warp w takes keys 16 w .. 16 w + 15
// and 64 more on; a slice of 16 keys lies in one page.  Each warp streams its
// slices through its own ring of stages with 16-byte cp.async (one page
// lookup a slice; rows behind the cached ones are filled with zeros, so what
// the page holds there never enters), without any barrier between the warps:
// 128 KB are in flight per SM.  The loads run ahead across the borders of
// items.  Per slice: scores, online softmax in the log2 domain with a lazy
// rescale (only when the maximum has grown by more than 2^8), P rounded to
// bf16 for the product (its relative error of 2^-8 is that of the output's own
// rounding), V^T P^T.  S^T's accumulators become P^T's operand by one 8x8
// transposition in registers (movmatrix).  At the end of an item the warps'
// states are merged through shared memory and the row is finished here, or
// its unnormalised sums go to a record if the item is split.
#include <math.h>

#include "common.cuh"
#include "extend.cuh"

namespace diffattn {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSlice = 16;
constexpr float kLazy = 8.0f;  // log2 units

template <int D>
struct Narrow {
  static constexpr int DV = 2 * D;
  static constexpr int ROW = 4 * D;                     // bytes of a K or a V row
  static constexpr int STAGE = kSlice * 2 * ROW;        // K rows, then V rows
  static constexpr int STAGES = D == 128 ? 3 : 6;       // 48 KB a warp
  static constexpr int PITCH = DV + 4;                  // floats of a row of the merge buffer (no bank conflicts)
  static constexpr int OFF_BUF = kWarps * STAGES * STAGE;
  static constexpr int SMEM = OFF_BUF + kWarps * kNarrowRows * PITCH * 4;
  static_assert(SMEM + 1024 <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A position on the line of units: the item and the unit in it.
struct Cursor {
  NarrowReq rq;
  int at, hk, unit, units;
  __device__ void open(const NarrowReq* list) {
    rq = list[at];
    units = rq.L <= 0 ? 1 : (rq.L - 1) / kUnit + 1;
  }
  // The item behind this one (only called while the worker has units left).
  __device__ void next(const NarrowReq* list, int H_kv) {
    unit = 0;
    if (++hk == H_kv) {
      hk = 0;
      ++at;
      open(list);
    }
  }
};

// one_unit: the block table holds at most kUnit keys, so a unit behind an
// item's first has none, and the first is the whole item.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) extend_narrow_kernel(const ExtendArgs a, float* recs, int page_shift,
                                                                    int max_keys, int one_unit, int* status) {
  using C = Narrow<D>;
  constexpr int DV = C::DV, KS = D / 16, CT = DV / 16, R8 = kNarrowRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][2][R8], s_l[kWarps][2][R8], s_inv[2][R8], s_ss[kWarps][R8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  if (!plan_fits(a.plan, a.n, status)) return;
  const PlanView pv = plan_view(a.plan, a.n, 0);
  const WorkStart st = pv.starts[blockIdx.x];
  if (st.count == 0) return;
  const int causal = pv.head->causal;
  const int H = a.n.H, H_kv = a.n.H_kv, G = H / H_kv;
  const uint32_t ring = smem_u32(smem) + warp * C::STAGES * C::STAGE;
  float* buf = reinterpret_cast<float*>(smem + C::OFF_BUF);
  const char* kc = static_cast<const char*>(a.k_cache);
  const char* vc = static_cast<const char*>(a.v_cache);

  // ------------------------------------------------------------- the loads --
  Cursor ld{};
  ld.at = st.at;
  ld.hk = st.hk;
  ld.unit = st.unit;
  ld.open(pv.narrow);
  const int slices = 2 * st.count;
  int issued = 0;
  auto issue = [&]() {
    if (issued < slices) {
      if (issued > 0 && !(issued & 1) && ++ld.unit == ld.units) ld.next(pv.narrow, H_kv);
      const int L = min(ld.rq.L, max_keys);
      const int key0 = ld.unit * kUnit + (issued & 1) * 64 + warp * kSlice;
      if (key0 < L) {
        const int page = a.block_table[static_cast<size_t>(ld.rq.s) * a.max_pages + (key0 >> page_shift)];
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok) atomicCAS(status, 0, 6);
        const size_t row0 = (static_cast<size_t>(ok ? page : 0) << page_shift) + (key0 & ((1 << page_shift) - 1));
        const uint32_t dst = ring + (issued % C::STAGES) * C::STAGE;
        const size_t pitch = static_cast<size_t>(H_kv) * C::ROW;
        const size_t off = row0 * pitch + static_cast<size_t>(ld.hk) * C::ROW;
        const int rows = ok ? min(kSlice, L - key0) : 0;  // the rest is filled with zeros
        constexpr int CH = C::ROW / 16;                   // 16-byte chunks of a row
        const int ch = lane % CH;
        if constexpr (CH == 32) {
#pragma unroll
          for (int i = 0; i < kSlice; ++i) {
            const size_t src = off + (i < rows ? i : 0) * pitch + 16 * ch;
            const uint32_t to = dst + i * C::ROW + ((ch ^ (i & 7)) << 4);
            cp16(to, kc + src, i < rows ? 16 : 0);
            cp16(to + kSlice * C::ROW, vc + src, i < rows ? 16 : 0);
          }
        } else {
          const char* from = lane < CH ? kc : vc;
          const uint32_t to0 = dst + (lane < CH ? 0 : kSlice * C::ROW);
#pragma unroll
          for (int i = 0; i < kSlice; ++i)
            cp16(to0 + i * C::ROW + ((ch ^ (i & 7)) << 4), from + off + (i < rows ? i : 0) * pitch + 16 * ch,
                 i < rows ? 16 : 0);
        }
      }
    }
    ++issued;
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) issue();

  // ------------------------------------------------------------ the items --
  const float sc = kLog2e * rsqrtf(static_cast<float>(D));
  const float c2 = map2_coefficient(a.mode, *a.lambda);
  Cursor cur{};
  cur.at = st.at;
  cur.hk = st.hk;
  cur.unit = st.unit;
  cur.open(pv.narrow);
  int slice = 0;
  for (int left = st.count; left > 0;) {
    const int take = min(left, cur.units - cur.unit);
    const bool begins = cur.unit == 0, whole = begins && (take == cur.units || one_unit);
    const int R = cur.rq.n * G;
    const int L = min(cur.rq.L, max_keys);
    if (cur.rq.L > max_keys && tid == 0) atomicCAS(status, 0, 6);
    // this thread's two rows (columns of S^T and O^T) and the last keys that they see
    int lim[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * (lane & 3) + j;
      lim[j] = causal && r < R ? min(cur.rq.L - cur.rq.n + r / G, L - 1) : L - 1;
    }
    const int lim_min = causal ? min(cur.rq.L - cur.rq.n, L - 1) : L - 1;
    uint32_t qf[2][KS][2];
    {
      const int r = lane >> 2;
      const uint32_t* qp = static_cast<const uint32_t*>(a.q) +
                           ((static_cast<size_t>(cur.rq.q0 + (r < R ? r / G : 0)) * H + cur.hk * G + r % G) * DV) / 2 +
                           (lane & 3);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[m][k][0] = r < R ? qp[(m * D + 16 * k) / 2] : 0u;
          qf[m][k][1] = r < R ? qp[(m * D + 16 * k + 8) / 2] : 0u;
        }
    }
    float o[2][CT][4], mx[2][2], l[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      mx[m][0] = mx[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][c][i] = 0.f;
    }
    for (int i = 0; i < 2 * take; ++i, ++slice) {
      issue();  // into the stage that the slice before this one has left
      cp_wait<C::STAGES - 1>();
      __syncwarp();
      const int key0 = (cur.unit + (i >> 1)) * kUnit + (i & 1) * 64 + warp * kSlice;
      if (key0 < L) {
        const uint32_t kb = ring + (slice % C::STAGES) * C::STAGE, vb = kb + kSlice * C::ROW;
        const int lr = lane & 7, mi = lane >> 3;
        // S^T: keys x rows
        float s[2][4];
        {
          const uint32_t base = kb + (lr + (mi & 1) * 8) * C::ROW;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float e[2][4] = {};  // two chains of products
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t f[4];
              ldsm4(f, base + (((m * (D / 8) + 2 * k + (mi >> 1)) ^ lr) << 4));
              mma(e[k & 1], f, qf[m][k][0], qf[m][k][1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[m][j] = (e[0][j] + e[1][j]) * sc;
          }
        }
        const int k_lo = key0 + (lane >> 2);
        if (key0 + kSlice - 1 > lim_min) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (k_lo + (j >> 1) * 8 > lim[j & 1]) s[0][j] = s[1][j] = -INFINITY;
          }
        }
        float t[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[m][j], s[m][j + 2]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            t[m][j] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          }
        const bool grow = t[0][0] > mx[0][0] + kLazy || t[0][1] > mx[0][1] + kLazy || t[1][0] > mx[1][0] + kLazy ||
                          t[1][1] > mx[1][1] + kLazy;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float al[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float mn = fmaxf(mx[m][j], t[m][j]);
              al[j] = mn == -INFINITY ? 1.f : fast_exp2(mx[m][j] - mn);
              mx[m][j] = mn;
              l[m][j] *= al[j];
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
#pragma unroll
              for (int j = 0; j < 4; ++j) o[m][c][j] *= al[j & 1];
            }
          }
        }
        uint32_t pb[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float ref = mx[m][j & 1];
            p[j] = fast_exp2(s[m][j] - (ref == -INFINITY ? 0.f : ref));
            l[m][j & 1] += p[j];
          }
          pb[m][0] = transpose8x8(pack_bf16x2(p[0], p[1]));
          pb[m][1] = transpose8x8(pack_bf16x2(p[2], p[3]));
        }
        // O^T += V^T P^T: channels x rows, the V operand shared by the maps
        const uint32_t base = vb + (lr + (mi >> 1) * 8) * C::ROW;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          uint32_t f[4];
          ldsm4t(f, base + (((2 * c + (mi & 1)) ^ lr) << 4));
          mma(o[0][c], f, pb[0][0], pb[0][1]);
          mma(o[1][c], f, pb[1][0], pb[1][1]);
        }
      }
      __syncwarp();  // every lane has read the stage
    }

    // ------------------------------------------------- merge of the warps --
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[m][j];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (lane < 4) {
          s_l[warp][m][2 * lane + j] = x;
          s_m[warp][m][2 * lane + j] = mx[m][j];
        }
      }
    __syncthreads();
    if (tid < 2 * R8) {
      const int m = tid / R8, r = tid % R8;
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][m][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum = fmaf(M == -INFINITY ? 0.f : fast_exp2(s_m[w][m][r] - M), s_l[w][m][r], sum);
      s_inv[m][r] = whole ? (sum > 0.f ? (m ? c2 : 1.f) / sum : 0.f) : sum;
      if (!whole && r < R && !(one_unit && !begins)) {
        float* ml = recs + (2 * blockIdx.x + (begins ? 1 : 0)) * record_floats(R8, D) + 4 * r + 2 * m;
        ml[0] = M;
        ml[1] = sum;
      }
    }
    constexpr int E = DV / kThreads;  // channels a thread finishes
    float y[R8][E];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 2 * (lane & 3) + j;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][m][r]);
        f[j] = M == -INFINITY ? 0.f : fast_exp2(mx[m][j] - M);
      }
      if (m) __syncthreads();  // the buffer's first map has been read
      float* mine = buf + static_cast<size_t>(warp) * R8 * C::PITCH;
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 2 * (lane & 3) + (j & 1);
          if (r < R) mine[r * C::PITCH + 16 * c + (lane >> 2) + (j >> 1) * 8] = o[m][c][j] * f[j & 1];
        }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R8; ++r) {
        if (r < R) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float* b = buf + r * C::PITCH + tid + e * kThreads;
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x += b[w * R8 * C::PITCH];
            if (whole) {
              y[r][e] = m ? fmaf(x, s_inv[1][r], y[r][e]) : x * s_inv[0][r];
            } else if (!(one_unit && !begins)) {
              recs[(2 * blockIdx.x + (begins ? 1 : 0)) * record_floats(R8, D) + 4 * R8 +
                   static_cast<size_t>(r) * 2 * DV + m * DV + tid + e * kThreads] = x;
            }
          }
        }
      }
    }
    if (whole) {  // the same for the whole CTA
#pragma unroll
      for (int r = 0; r < R8; ++r) {
        if (r < R) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) ss = fmaf(y[r][e], y[r][e], ss);
#pragma unroll
          for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          if (lane == 0) s_ss[warp][r] = ss;
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R8; ++r) {
        if (r < R) {
          const float ss = (s_ss[0][r] + s_ss[1][r]) + (s_ss[2][r] + s_ss[3][r]);
          const float gsc = (1.f - a.lambda_init) * rsqrtf(ss / DV + a.eps);
          const size_t row = static_cast<size_t>(cur.rq.q0 + r / G) * H + cur.hk * G + r % G;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int ch = tid + e * kThreads;
            static_cast<__nv_bfloat16*>(a.o)[row * DV + ch] =
                __float2bfloat16_rn(y[r][e] * gsc * __ldg(a.rms_w + ch));
          }
        }
      }
    }
    __syncthreads();  // the merge's shared memory is free again
    left -= take;
    if (left > 0) cur.next(pv.narrow, H_kv);
  }
  cp_wait<0>();
}

template <int D>
cudaError_t launch_d(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream) {
  static unsigned long long set_ctx[64] = {};
  if (ctl.dev < 0 || ctl.dev >= 64) return cudaErrorInvalidDevice;
  if (ctl.ctx == 0 || set_ctx[ctl.dev] != ctl.ctx) {
    const cudaError_t e = cudaFuncSetAttribute(extend_narrow_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Narrow<D>::SMEM);
    if (e != cudaSuccess) return e;
    set_ctx[ctl.dev] = ctl.ctx;
  }
  int shift = 0;
  while ((1 << shift) < a.page_size) ++shift;
  const long long keys = static_cast<long long>(a.max_pages) * a.page_size;
  const int max_keys = keys < kMaxKeys ? static_cast<int>(keys) : kMaxKeys;
  extend_narrow_kernel<D><<<kNarrowWorkers, kThreads, Narrow<D>::SMEM, stream>>>(
      a, recs, shift, max_keys, keys <= kUnit && !wide_possible(a.n), ctl.status);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_extend_narrow(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream) {
  return a.n.d == 128 ? launch_d<128>(a, recs, ctl, stream) : launch_d<64>(a, recs, ctl, stream);
}

}  // namespace diffattn
