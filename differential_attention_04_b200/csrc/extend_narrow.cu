// Attention of requests with at most 16 query rows per key head (single tokens,
// drafted tokens, small groups of shared heads) over a paged cache.
//
// HBM-bound: 8 d bytes of K and V per key and key head against 12 d flops per
// row.  Eight rows go through the matrix units at once, so the arithmetic hardly
// grows with the rows: with keys and channels as the M dimension of
// m16n8k16 (S^T = K Q^T, O^T = V^T P^T) the rows are the N = 8 columns.  The
// warp-level instruction is taken on purpose: tcgen05 has M = 128 and would
// put P through shared memory, and the kernel needs a fraction of the
// warp-level rate to run at the speed of memory.
//
// P enters as the sum of two bf16, the rounded weight and the remainder of the
// rounding: one bf16 alone adds as much error to the output as the output's own
// rounding (relative 2-norm 0.0026 against 0.0017).  With up to four rows the
// remainders take the four free columns, at no cost; with more they are a second
// product into the same sums.  Nine to sixteen rows take two column tiles, in
// steps that have no more (narrow_rows in extend.cuh).  As tiles of 128 rows on
// the tensor cores, 16 rows over 32 x 2000 tokens and 16 heads took 250 us at
// d = 128 and 147 at d = 64; here 205 and 124.
//
// Two CTAs of two pairs of warps per SM take a contiguous range of the step's
// units of 128 keys each (extend.cuh).  Within a unit the pairs take turns of
// 16 keys; a slice of 16 keys lies in one page.  One warp of a pair computes
// map 1 and loads the keys, the other map 2 and the values: two warps per
// scheduler hide each other's latencies (one warp with both maps and the
// product for the remainders: 2272 us for 64 requests of 1K to 32K tokens, 12
// heads, d 128; two warps: 1845).  A pair streams its slices through its own
// ring of stages with 16-byte cp.async (one page lookup a slice; rows behind
// the cached ones are filled with zeros, so what the page holds there never
// enters) and meets at one barrier a step; pairs do not wait for each other.
// 128 KB are in flight per SM, and the loads run ahead across the borders of
// items.  Per step: scores, online softmax in the log2 domain with a lazy
// rescale (only when the maximum has grown by more than 2^8), V^T P^T.  S^T's
// accumulators become P^T's operand by one 8x8 transposition in registers
// (movmatrix).  At the end of an item the pairs' states are merged through
// shared memory and the row is finished here, or its unnormalised sums go to a
// record if the item is split.  The second CTA of an SM loads and computes
// under the first one's merge: one CTA of four pairs took 141 us for 256
// requests of 80 tokens over 16 heads where this takes 80, and 386 us for 24 x 5
// drafted tokens where this takes 355 (a lone request of 1000 tokens: 14 and 17
// us).
//
// Measured (d 128), over several GPUs: the 64 requests above 1717 to 1814 us, 6.8
// to 7.2 TB/s (12.3 GB); the drafted tokens 335 to 355 us, 6.1 to 6.4 TB/s.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "extend.cuh"

namespace diffattn {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPairs = 2;
constexpr int kThreads = 2 * kPairs * 32;
constexpr int kSlice = 16;
constexpr float kLazy = 8.0f;  // log2 units

template <int D>
struct Narrow {
  static constexpr int DV = 2 * D;
  static constexpr int ROW = 4 * D;                     // bytes of a K or a V row
  static constexpr int SL = D == 128 ? 1 : 2;           // slices a step: 16 KB of keys and values
  static constexpr int SLICE = kSlice * 2 * ROW;        // K rows, then V rows
  static constexpr int STAGE = SL * SLICE;
  static constexpr int STAGES = 3;                      // 48 KB a pair
  static constexpr int PITCH = DV + 4;                  // floats of a row of the merge buffer (no bank conflicts)
  static constexpr int OFF_BUF = kPairs * STAGES * STAGE;
  static constexpr int SMEM = OFF_BUF + kPairs * 8 * PITCH * 4;  // 8 rows of one map, or 4 of both, at a time
  static_assert(2 * (SMEM + 1024 + 512) <= 233472, "shared memory of two CTAs");
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
  __device__ void count_units() { units = rq.L <= 0 ? 1 : (rq.L - 1) / kUnit + 1; }
  __device__ explicit Cursor(const WorkStart& st) : rq(st.rq), at(st.at), hk(st.hk), unit(st.unit) { count_units(); }
  // The item behind this one (only called while the worker has units left).
  __device__ void next(const NarrowReq* list, const ExtendShape& n, int* status) {
    unit = 0;
    if (++hk == n.H_kv) {
      hk = 0;
      rq = narrow_at(list, ++at, n, status);
      count_units();
    }
  }
};

// one_unit: the block table holds at most kUnit keys, so a unit behind an
// item's first has none, and the first is the whole item.
// NT: columns of 8 rows that an item may have (the host's bound of new tokens
// says which; a kernel for 16 rows has no registers to spare).
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2) extend_narrow_kernel(const ExtendArgs a, float* recs, int page_shift,
                                                                    int max_keys, int one_unit, UnitLimits most,
                                                                    int* status) {
  using C = Narrow<D>;
  constexpr int DV = C::DV, KS = D / 16, CT = DV / 16, RT = 8 * NT, SL = C::SL;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kPairs][2][RT], s_l[kPairs][2][RT], s_ss[2 * kPairs][RT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pair = warp & (kPairs - 1), map = warp / kPairs;
  const PlanView pv = plan_view(a.plan, a.n, 0);
  const WorkStart st = pv.starts[blockIdx.x];  // read beside the header: the first loads are one chain of trips to L2
  if (!plan_fits(a.plan, a.n, most, status)) return;
  if (st.count == 0) return;
#ifdef DIFFATTN_DEBUG
  {  // the range begins in the request that its entry names
    const NarrowReq r = narrow_at(pv.narrow, st.at, a.n, status);
    const Cursor c(st);
    if (!da_check(status, st.count > 0 && st.count <= pv.head->units[0] && r.q0 == st.rq.q0 && r.n == st.rq.n &&
                              r.L == st.rq.L && r.s == st.rq.s && st.hk >= 0 && st.hk < a.n.H_kv && st.unit >= 0 &&
                              st.unit < c.units))
      return;
  }
#endif
  const int causal = pv.head->causal;
  const int H = a.n.H, H_kv = a.n.H_kv, G = H / H_kv;
  const uint32_t ring = smem_u32(smem) + pair * C::STAGES * C::STAGE;
  float* buf = reinterpret_cast<float*>(smem + C::OFF_BUF);

  // ------------------------------------------------------------- the loads --
  const char* cache = static_cast<const char*>(map ? a.v_cache : a.k_cache);
  const uint32_t mine = ring + (map ? kSlice * C::ROW : 0);
  Cursor ld(st);
  constexpr int SPU = kUnit / (kPairs * kSlice * SL);  // steps a unit
  // where step i's slice x of this pair begins in the unit
  auto slice_at = [&](int i, int x) { return ((i % SPU * SL + x) * kPairs + pair) * kSlice; };
  const int steps = SPU * st.count;
  int issued = 0;
  auto issue = [&]() {
    if (issued < steps) {
      if (issued > 0 && issued % SPU == 0 && ++ld.unit == ld.units) ld.next(pv.narrow, a.n, status);
      const int L = min(ld.rq.L, max_keys);
#pragma unroll
      for (int x = 0; x < SL; ++x) {
        const int key0 = ld.unit * kUnit + slice_at(issued, x);
        if (key0 < L) {
          const int page = a.block_table[static_cast<size_t>(ld.rq.s) * a.max_pages + (key0 >> page_shift)];
          const bool ok = page >= 0 && page < a.num_pages;
          if (!ok) atomicCAS(status, 0, 6);
          constexpr int CH = C::ROW / 16, RPI = 32 / CH;  // 16-byte chunks of a row, rows an instruction
          const int ch = lane % CH, r0 = lane / CH;
          const size_t row0 = (static_cast<size_t>(ok ? page : 0) << page_shift) + (key0 & ((1 << page_shift) - 1));
          const size_t pitch = static_cast<size_t>(H_kv) * C::ROW;
          const char* src = cache + row0 * pitch + static_cast<size_t>(ld.hk) * C::ROW + 16 * ch;
          const uint32_t dst = mine + (issued % C::STAGES) * C::STAGE + x * C::SLICE;
          const int rows = ok ? min(kSlice, L - key0) : 0;  // the rest is filled with zeros
#pragma unroll
          for (int i = 0; i < kSlice / RPI; ++i) {
            const int r = i * RPI + r0;
            cp16(dst + r * C::ROW + ((ch ^ (r & 7)) << 4), src + (r < rows ? r : 0) * pitch, r < rows ? 16 : 0);
          }
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
  Cursor cur(st);
  // the queries of an item as the operand of S^T (this map's)
  uint32_t qf[NT][KS][2];
  auto load_q = [&](const Cursor& it) {
    const int R = it.rq.n * G;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + ((lane >> 2) & (R <= 4 ? 3 : 7));
      const uint32_t* qp =
          static_cast<const uint32_t*>(a.q) +
          ((static_cast<size_t>(it.rq.q0 + (r < R ? r / G : 0)) * H + it.hk * G + r % G) * DV + map * D) / 2 + (lane & 3);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[t][k][0] = r < R ? qp[8 * k] : 0u;
        qf[t][k][1] = r < R ? qp[8 * k + 4] : 0u;
      }
    }
  };
  load_q(cur);
  int step = 0;
  for (int left = st.count; left > 0;) {
    const int take = min(left, cur.units - cur.unit);
    const bool begins = cur.unit == 0, whole = begins && (take == cur.units || one_unit);
    const int R = cur.rq.n * G;
    const bool dup = R <= 4;  // columns 4 .. 7 hold rows 0 .. 3 again, with the remainders of their weights
    const int L = min(cur.rq.L, max_keys);
    if (cur.rq.L > max_keys && tid == 0) atomicCAS(status, 0, 6);
    // the item behind this one: its request is read now and its queries before the merge, so that neither is waited for
    Cursor nx = cur;
    const bool more = left > take;
    if (more) nx.next(pv.narrow, a.n, status);
    // this thread's columns of S^T and O^T and the last keys that their rows see
    int lim[NT][2];
    float o[NT][CT][4], mx[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * t + ((2 * (lane & 3) + j) & (dup ? 3 : 7));
        lim[t][j] = causal && r < R ? min(cur.rq.L - cur.rq.n + r / G, L - 1) : L - 1;
        mx[t][j] = -INFINITY;
        l[t][j] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][c][i] = 0.f;
    }
    const int lim_min = causal ? min(cur.rq.L - cur.rq.n, L - 1) : L - 1;
    const bool rest = dup && (lane & 2);  // this thread's columns are remainders
    // one loop for each way, so that none carries another's registers
    auto steps_of = [&](auto dup_c, auto nt_c) {
      constexpr bool DUP = decltype(dup_c)::value;
      constexpr int NN = decltype(nt_c)::value;
      for (int i = 0; i < SPU * take; ++i, ++step) {
        cp_wait<C::STAGES - 2>();
        named_bar_sync(1 + pair, 64);  // both halves of the step are here, and the step before it has been read
        issue();                       // into that one's stage
        const int first = (cur.unit + i / SPU) * kUnit + slice_at(i, 0);
        if (first < L) {  // (a second slice without keys holds stale data: its scores are masked, and its V is not read)
          const uint32_t kb = ring + (step % C::STAGES) * C::STAGE;
          const int lr = lane & 7, mi = lane >> 3;
          // S^T: keys x rows
          float s[SL][NN][4], tm[NN][2];
#pragma unroll
          for (int t = 0; t < NN; ++t) tm[t][0] = tm[t][1] = -INFINITY;
#pragma unroll
          for (int x = 0; x < SL; ++x) {
            const uint32_t base = kb + x * C::SLICE + (lr + (mi & 1) * 8) * C::ROW;
            float e[2][NN][4] = {};  // two chains of products
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t f[4];
              ldsm4(f, base + (((map * (D / 8) + 2 * k + (mi >> 1)) ^ lr) << 4));
#pragma unroll
              for (int t = 0; t < NN; ++t) mma(e[k & 1][t], f, qf[t][k][0], qf[t][k][1]);
            }
            const int key0 = first + kPairs * kSlice * x, k_lo = key0 + (lane >> 2);
            const bool mask = key0 + kSlice - 1 > lim_min;
#pragma unroll
            for (int t = 0; t < NN; ++t) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                s[x][t][j] = (e[0][t][j] + e[1][t][j]) * sc;
                if (mask && k_lo + (j >> 1) * 8 > lim[t][j & 1]) s[x][t][j] = -INFINITY;
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) tm[t][j] = fmaxf(tm[t][j], fmaxf(s[x][t][j], s[x][t][j + 2]));
            }
          }
          bool grow = false;
#pragma unroll
          for (int t = 0; t < NN; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float& m = tm[t][j];
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              grow |= m > mx[t][j] + kLazy;
            }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int t = 0; t < NN; ++t) {
              float al[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float mn = fmaxf(mx[t][j], tm[t][j]);
                al[j] = mn == -INFINITY ? 1.f : fast_exp2(mx[t][j] - mn);
                mx[t][j] = mn;
                l[t][j] *= al[j];
              }
#pragma unroll
              for (int c = 0; c < CT; ++c) {
#pragma unroll
                for (int j = 0; j < 4; ++j) o[t][c][j] *= al[j & 1];
              }
            }
          }
#pragma unroll
          for (int x = 0; x < SL; ++x) {
            if (x > 0 && first + kPairs * kSlice * x >= L) break;
            uint32_t pb[NN][2], pl[NN][2];
#pragma unroll
            for (int t = 0; t < NN; ++t)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float p0 = fast_exp2(s[x][t][2 * j] - (mx[t][0] == -INFINITY ? 0.f : mx[t][0]));
                const float p1 = fast_exp2(s[x][t][2 * j + 1] - (mx[t][1] == -INFINITY ? 0.f : mx[t][1]));
                l[t][0] += p0;
                l[t][1] += p1;
                const uint32_t hi = pack_bf16x2(p0, p1);
                const uint32_t lo = pack_bf16x2(p0 - bf16lo_to_f32(hi), p1 - bf16hi_to_f32(hi));
                pb[t][j] = transpose8x8(DUP && rest ? lo : hi);
                if constexpr (!DUP) pl[t][j] = transpose8x8(lo);
              }
            // O^T += V^T P^T: channels x rows
            const uint32_t base = kb + x * C::SLICE + (kSlice + lr + (mi >> 1) * 8) * C::ROW;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              uint32_t f[4];
              ldsm4t(f, base + (((2 * c + (mi & 1)) ^ lr) << 4));
#pragma unroll
              for (int t = 0; t < NN; ++t) {
                mma(o[t][c], f, pb[t][0], pb[t][1]);
                if constexpr (!DUP) mma(o[t][c], f, pl[t][0], pl[t][1]);
              }
            }
          }
        }
      }
    };
    using One = std::integral_constant<int, 1>;
    if (dup)
      steps_of(std::true_type{}, One{});
    else if (NT == 1 || R <= 8)
      steps_of(std::false_type{}, One{});
    else
      steps_of(std::false_type{}, std::integral_constant<int, NT>{});
    if (more) load_q(nx);

    // ------------------------------------------------- merge of the pairs --
    // Every warp leaves its maxima, sums and unnormalised O^T; the thread that
    // finishes a channel takes the pairs' to their common maximum itself.  With
    // up to four rows both maps fit the buffer (rows 0 .. 3 and 4 .. 7) and one
    // barrier does; with more, eight rows of a map go through it at a time.
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[t][j];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (lane < 4) {
          s_l[pair][map][8 * t + 2 * lane + j] = x;
          s_m[pair][map][8 * t + 2 * lane + j] = mx[t][j];
        }
      }
    // The item's record, for a part of it that the joining kernel reads.
    float* rec = recs + (2 * blockIdx.x + (begins ? 1 : 0)) * record_floats(RT, D);
    const bool part = !whole && !(one_unit && !begins);
    // a thread finishes channels tid, tid + kThreads, ... of every row
    constexpr int E = DV / kThreads;
    float y[RT][E];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) y[r][e] = 0.f;
    auto leave = [&](const float (&x)[CT][4], int row0, int rows) {  // this thread's columns below `rows`, from row0 on
      float* to = buf + static_cast<size_t>(pair * 8 + row0) * C::PITCH + (lane >> 2);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 2 * (lane & 3) + j;
        if (r < rows) {
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            to[r * C::PITCH + 16 * c] = x[c][j];
            to[r * C::PITCH + 16 * c + 8] = x[c][j + 2];
          }
        }
      }
    };
    auto finish = [&](float (&z)[E], int r, int m, int at) {  // row r of map m, at row `at` of the buffer
      float M = -INFINITY, sum = 0.f, f[kPairs];
#pragma unroll
      for (int w = 0; w < kPairs; ++w) M = fmaxf(M, s_m[w][m][r]);
#pragma unroll
      for (int w = 0; w < kPairs; ++w) {
        f[w] = M == -INFINITY ? 0.f : fast_exp2(s_m[w][m][r] - M);
        sum = fmaf(f[w], s_l[w][m][r], sum);
      }
      const float scale = sum > 0.f ? (m ? c2 : 1.f) / sum : 0.f;
      if (part && tid == 0) *reinterpret_cast<float2*>(rec + 4 * r + 2 * m) = make_float2(M, sum);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float* b = buf + at * C::PITCH + tid + e * kThreads;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kPairs; ++w) x = fmaf(f[w], b[w * 8 * C::PITCH], x);
        if (part) rec[4 * RT + static_cast<size_t>(r) * 2 * DV + m * DV + tid + e * kThreads] = x;
        z[e] = fmaf(x, scale, z[e]);
      }
    };
    if (dup) {
      // the weights' and their remainders' products
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[0][c][j] += __shfl_xor_sync(0xffffffffu, o[0][c][j], 2);
      leave(o[0], 4 * map, R);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r < R) {
          finish(y[r], r, 0, r);
          finish(y[r], r, 1, 4 + r);
        }
      }
    } else {
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (8 * t < R) {
            if (m + t > 0) __syncthreads();  // the rows before these have been read
            if (map == m) leave(o[t], 0, R - 8 * t);
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (8 * t + r < R) finish(y[8 * t + r], 8 * t + r, m, r);
          }
        }
      }
    }
    if (whole) {  // the same for the whole CTA
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (r < R) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) ss = fmaf(y[r][e], y[r][e], ss);
#pragma unroll
          for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          if (lane == 0) s_ss[warp][r] = ss;
        }
      }
    }
    // the merge's buffers are free for the next item (its sums of squares come behind its own barrier)
    __syncthreads();
    if (whole) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (r < R) {
          float ss = 0.f;
#pragma unroll
          for (int w = 0; w < 2 * kPairs; ++w) ss += s_ss[w][r];
          const float gsc = norm_factor(ss / DV, a.eps, a.lambda_init);
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
    left -= take;
    cur = nx;
  }
  cp_wait<0>();
}

template <int D, int NT>
cudaError_t launch_d(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream) {
  static unsigned long long set_ctx[64] = {};
  if (ctl.dev < 0 || ctl.dev >= 64) return cudaErrorInvalidDevice;
  if (ctl.ctx == 0 || set_ctx[ctl.dev] != ctl.ctx) {
    const cudaError_t e = cudaFuncSetAttribute(extend_narrow_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Narrow<D>::SMEM);
    if (e != cudaSuccess) return e;
    set_ctx[ctl.dev] = ctl.ctx;
  }
  int shift = 0;
  while ((1 << shift) < a.page_size) ++shift;
  const long long keys = static_cast<long long>(a.max_pages) * a.page_size;
  const int max_keys = keys_of_table(a.max_pages, a.page_size);
  extend_narrow_kernel<D, NT><<<kNarrowWorkers, kThreads, Narrow<D>::SMEM, stream>>>(
      a, recs, shift, max_keys, keys <= kUnit && !wide_possible(a.n), unit_limits(a.n, max_keys), ctl.status);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_extend_narrow(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream) {
  const bool few = narrow_rows(a.n) == 8;
  if (a.n.d == 128) return few ? launch_d<128, 1>(a, recs, ctl, stream) : launch_d<128, 2>(a, recs, ctl, stream);
  return few ? launch_d<64, 1>(a, recs, ctl, stream) : launch_d<64, 2>(a, recs, ctl, stream);
}

}  // namespace diffattn
