// Attention of requests with at most 8 query rows per key head (single tokens,
// drafted tokens, small groups of shared heads) over a paged cache.
//
// HBM-bound: 8 d bytes of K and V per key and key head against 12 d flops per
// row.  All 8 rows go through the matrix units at once, so the arithmetic does
// not grow with the rows: with keys and channels as the M dimension of
// m16n8k16 (S^T = K Q^T, O^T = V^T P^T) the rows are the N = 8 columns.  The
// warp-level instruction is taken on purpose: tcgen05 has M = 128 and would
// put P through shared memory, and the kernel needs a fraction of the
// warp-level rate to run at the speed of memory.
//
// P enters as the sum of two bf16, the rounded weight and the remainder of the
// rounding: one bf16 alone adds as much error to the output as the output's own
// rounding (relative 2-norm 0.0026 against 0.0017).  With up to four rows the
// remainders take the four free columns, at no cost; with five to eight they
// are a second product into the same sums.
//
// A CTA of four pairs of warps per SM takes a contiguous range of the step's
// units of 128 keys (extend.cuh).  Within a unit pair w takes keys 16 w ..
// 16 w + 15 and the same 64 on; a slice of 16 keys lies in one page.  One warp
// of a pair computes map 1 and loads the keys, the other map 2 and the values:
// two warps per scheduler hide each other's latencies (one warp with both
// maps: 1943 us against TWO_WARPS for 64 requests of 1K to 32K tokens, 12 heads,
// d 128).  A pair streams its slices through its own ring of stages with
// 16-byte cp.async (one page lookup a slice; rows behind the cached ones are
// filled with zeros, so what the page holds there never enters) and meets at
// one barrier a slice; pairs do not wait for each other.  128 KB are in flight
// per SM, and the loads run ahead across the borders of items.  Per slice:
// scores, online softmax in the log2 domain with a lazy rescale (only when the
// maximum has grown by more than 2^8), V^T P^T.  S^T's accumulators become
// P^T's operand by one 8x8 transposition in registers (movmatrix).  At the end
// of an item the pairs' states are merged through shared memory and the row is
// finished here, or its unnormalised sums go to a record if the item is split.
#include <math.h>

#include "common.cuh"
#include "extend.cuh"

namespace diffattn {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPairs = 4;
constexpr int kThreads = 2 * kPairs * 32;
constexpr int kSlice = 16;
constexpr float kLazy = 8.0f;  // log2 units

template <int D>
struct Narrow {
  static constexpr int DV = 2 * D;
  static constexpr int ROW = 4 * D;                     // bytes of a K or a V row
  static constexpr int STAGE = kSlice * 2 * ROW;        // K rows, then V rows
  static constexpr int STAGES = D == 128 ? 3 : 6;       // 48 KB a pair
  static constexpr int PITCH = DV + 4;                  // floats of a row of the merge buffer (no bank conflicts)
  static constexpr int OFF_BUF = kPairs * STAGES * STAGE;
  static constexpr int SMEM = OFF_BUF + kPairs * kNarrowRows * PITCH * 4;
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
  __shared__ float s_m[kPairs][2][R8], s_l[kPairs][2][R8], s_f[2][R8], s_ss[2 * kPairs][R8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pair = warp & (kPairs - 1), map = warp / kPairs;
  if (!plan_fits(a.plan, a.n, status)) return;
  const PlanView pv = plan_view(a.plan, a.n, 0);
  const WorkStart st = pv.starts[blockIdx.x];
  if (st.count == 0) return;
  const int causal = pv.head->causal;
  const int H = a.n.H, H_kv = a.n.H_kv, G = H / H_kv;
  const uint32_t ring = smem_u32(smem) + pair * C::STAGES * C::STAGE;
  float* buf = reinterpret_cast<float*>(smem + C::OFF_BUF);

  // ------------------------------------------------------------- the loads --
  const char* cache = static_cast<const char*>(map ? a.v_cache : a.k_cache);
  const uint32_t mine = ring + (map ? kSlice * C::ROW : 0);
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
      const int key0 = ld.unit * kUnit + (issued & 1) * 64 + pair * kSlice;
      if (key0 < L) {
        const int page = a.block_table[static_cast<size_t>(ld.rq.s) * a.max_pages + (key0 >> page_shift)];
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok) atomicCAS(status, 0, 6);
        constexpr int CH = C::ROW / 16, RPI = 32 / CH;  // 16-byte chunks of a row, rows an instruction
        const int ch = lane % CH, r0 = lane / CH;
        const size_t row0 = (static_cast<size_t>(ok ? page : 0) << page_shift) + (key0 & ((1 << page_shift) - 1));
        const size_t pitch = static_cast<size_t>(H_kv) * C::ROW;
        const char* src = cache + row0 * pitch + static_cast<size_t>(ld.hk) * C::ROW + 16 * ch;
        const uint32_t dst = mine + (issued % C::STAGES) * C::STAGE;
        const int rows = ok ? min(kSlice, L - key0) : 0;  // the rest is filled with zeros
#pragma unroll
        for (int i = 0; i < kSlice / RPI; ++i) {
          const int r = i * RPI + r0;
          cp16(dst + r * C::ROW + ((ch ^ (r & 7)) << 4), src + (r < rows ? r : 0) * pitch, r < rows ? 16 : 0);
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
    const bool dup = R <= R8 / 2;  // columns 4 .. 7 hold rows 0 .. 3 again, with the remainders of their weights
    const int L = min(cur.rq.L, max_keys);
    if (cur.rq.L > max_keys && tid == 0) atomicCAS(status, 0, 6);
    // this thread's two columns of S^T and O^T and the last keys that their rows see
    int lim[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = (2 * (lane & 3) + j) & (dup ? 3 : 7);
      lim[j] = causal && r < R ? min(cur.rq.L - cur.rq.n + r / G, L - 1) : L - 1;
    }
    const int lim_min = causal ? min(cur.rq.L - cur.rq.n, L - 1) : L - 1;
    const bool rest = dup && (lane & 2);  // this thread's columns are remainders
    uint32_t qf[KS][2];
    {
      const int r = (lane >> 2) & (dup ? 3 : 7);
      const uint32_t* qp =
          static_cast<const uint32_t*>(a.q) +
          ((static_cast<size_t>(cur.rq.q0 + (r < R ? r / G : 0)) * H + cur.hk * G + r % G) * DV + map * D) / 2 +
          (lane & 3);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][0] = r < R ? qp[8 * k] : 0u;
        qf[k][1] = r < R ? qp[8 * k + 4] : 0u;
      }
    }
    float o[CT][4], mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][i] = 0.f;
    for (int i = 0; i < 2 * take; ++i, ++slice) {
      cp_wait<C::STAGES - 2>();
      named_bar_sync(1 + pair, 64);  // both halves of the slice are here, and the slice before it has been read
      issue();                       // into that one's stage
      const int key0 = (cur.unit + (i >> 1)) * kUnit + (i & 1) * 64 + pair * kSlice;
      if (key0 < L) {
        const uint32_t kb = ring + (slice % C::STAGES) * C::STAGE, vb = kb + kSlice * C::ROW;
        const int lr = lane & 7, mi = lane >> 3;
        // S^T: keys x rows
        float s[4];
        {
          const uint32_t base = kb + (lr + (mi & 1) * 8) * C::ROW;
          float e[2][4] = {};  // two chains of products
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t f[4];
            ldsm4(f, base + (((map * (D / 8) + 2 * k + (mi >> 1)) ^ lr) << 4));
            mma(e[k & 1], f, qf[k][0], qf[k][1]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) s[j] = (e[0][j] + e[1][j]) * sc;
        }
        if (key0 + kSlice - 1 > lim_min) {
          const int k_lo = key0 + (lane >> 2);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (k_lo + (j >> 1) * 8 > lim[j & 1]) s[j] = -INFINITY;
        }
        float t[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(s[j], s[j + 2]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          t[j] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        }
        if (__any_sync(0xffffffffu, t[0] > mx[0] + kLazy || t[1] > mx[1] + kLazy)) {
          float al[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mn = fmaxf(mx[j], t[j]);
            al[j] = mn == -INFINITY ? 1.f : fast_exp2(mx[j] - mn);
            mx[j] = mn;
            l[j] *= al[j];
          }
#pragma unroll
          for (int c = 0; c < CT; ++c) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[c][j] *= al[j & 1];
          }
        }
        uint32_t pb[2], pl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p0 = fast_exp2(s[2 * j] - (mx[0] == -INFINITY ? 0.f : mx[0]));
          const float p1 = fast_exp2(s[2 * j + 1] - (mx[1] == -INFINITY ? 0.f : mx[1]));
          l[0] += p0;
          l[1] += p1;
          const uint32_t hi = pack_bf16x2(p0, p1);
          const uint32_t lo = pack_bf16x2(p0 - bf16lo_to_f32(hi), p1 - bf16hi_to_f32(hi));
          pb[j] = transpose8x8(rest ? lo : hi);
          pl[j] = lo;
        }
        // O^T += V^T P^T: channels x rows
        const uint32_t base = vb + (lr + (mi >> 1) * 8) * C::ROW;
        if (dup) {
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            uint32_t f[4];
            ldsm4t(f, base + (((2 * c + (mi & 1)) ^ lr) << 4));
            mma(o[c], f, pb[0], pb[1]);
          }
        } else {
          pl[0] = transpose8x8(pl[0]);
          pl[1] = transpose8x8(pl[1]);
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            uint32_t f[4];
            ldsm4t(f, base + (((2 * c + (mi & 1)) ^ lr) << 4));
            mma(o[c], f, pb[0], pb[1]);
            mma(o[c], f, pl[0], pl[1]);
          }
        }
      }
    }

    // ------------------------------------------------- merge of the pairs --
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x = l[j];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      if (lane < 4) {
        s_l[pair][map][2 * lane + j] = x;
        s_m[pair][map][2 * lane + j] = mx[j];
      }
    }
    __syncthreads();
    // The item's record, for a part of it that the joining kernel reads.
    float* rec = recs + (2 * blockIdx.x + (begins ? 1 : 0)) * record_floats(R8, D);
    const bool part = !whole && !(one_unit && !begins);
    if (tid < 2 * R8) {
      const int m = tid / R8, r = tid % R8;
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kPairs; ++w) M = fmaxf(M, s_m[w][m][r]);
#pragma unroll
      for (int w = 0; w < kPairs; ++w)
        sum = fmaf(M == -INFINITY ? 0.f : fast_exp2(s_m[w][m][r] - M), s_l[w][m][r], sum);
      s_f[m][r] = sum > 0.f ? (m ? c2 : 1.f) / sum : 0.f;
      if (part && r < R) {
        rec[4 * r + 2 * m] = M;
        rec[4 * r + 2 * m + 1] = sum;
      }
    }
    float f[2];  // this warp's sums to the common maximum
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = 2 * (lane & 3) + j;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kPairs; ++w) M = fmaxf(M, s_m[w][map][c]);
      f[j] = M == -INFINITY ? 0.f : fast_exp2(mx[j] - M);
    }
    // a thread finishes channel ch of every NG-th row
    constexpr int NG = kThreads / DV, NR = R8 / NG;
    const int ch = tid % DV, rg = tid / DV;
    float y[NR];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (m) __syncthreads();  // the buffer's first map has been read
      if (map == m) {
        float* to = buf + static_cast<size_t>(pair) * R8 * C::PITCH;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 2 * (lane & 3) + (j & 1);
            if ((r & (dup ? 3 : 7)) < R) to[r * C::PITCH + 16 * c + (lane >> 2) + (j >> 1) * 8] = o[c][j] * f[j & 1];
          }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int r = rg + k * NG;
        if (r < R) {
          const float* b = buf + r * C::PITCH + ch;
          float x = 0.f;
#pragma unroll
          for (int w = 0; w < kPairs; ++w) x += b[w * R8 * C::PITCH] + (dup ? b[(w * R8 + 4) * C::PITCH] : 0.f);
          if (part) rec[4 * R8 + static_cast<size_t>(r) * 2 * DV + m * DV + ch] = x;
          y[k] = m ? fmaf(x, s_f[1][r], y[k]) : x * s_f[0][r];
        }
      }
    }
    if (whole) {  // the same for the whole CTA
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int r = rg + k * NG;
        if (r < R) {  // the same for a whole warp
          float ss = y[k] * y[k];
#pragma unroll
          for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          if (lane == 0) s_ss[warp][r] = ss;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int r = rg + k * NG;
        if (r < R) {
          float ss = 0.f;
#pragma unroll
          for (int w = 0; w < DV / 32; ++w) ss += s_ss[rg * (DV / 32) + w][r];
          const float gsc = (1.f - a.lambda_init) * rsqrtf(ss / DV + a.eps);
          const size_t row = static_cast<size_t>(cur.rq.q0 + r / G) * H + cur.hk * G + r % G;
          static_cast<__nv_bfloat16*>(a.o)[row * DV + ch] = __float2bfloat16_rn(y[k] * gsc * __ldg(a.rms_w + ch));
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
