// The page bookkeeping of one serving step, on the device: from each request's
// cached and new token counts, the block table's new entries (pages taken from
// a ring of free pages), finished requests' pages returned to the ring, and
// per new token its position and its slot in the cache.
//
// With c_s cached tokens, n_s new ones, pages of P tokens, old_s = ceil(c_s/P)
// and want_s = ceil((c_s + n_s)/P): request s takes want_s - old_s pages, the
// first one base_s = sum of the earlier requests' needs behind the ring's head.
// A finished request (n_s = -1) appends its old_s pages behind the ring's tail.
// Nothing that the step reads is written by it (pages returned in a step are
// free from the next one on), so no part waits for another.
//
// Latency-bound: a few bytes per token.  One launch: every CTA scans the
// requests itself (2 S integers from L2, cheaper than a second launch), keeps
// the prefix sums in shared memory, then takes its share of the tokens (each
// found by binary search) and of the table entries.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"

namespace diffattn {

namespace {

constexpr int kStepThreads = 512;
constexpr int kMaxS = kPagedStepMaxRequests;

struct StepParams {
  const int *ctx, *nlen;
  int S;
  int* bt;
  int max_pages;
  int* ring;
  int F;
  const int* pool;
  int* pool_out;
  int P, T;
  int *cu_q, *kv, *pos, *slots, *info;
};

struct Sums {
  long long tok, need, rel;
};

// Exclusive block scan of three sums; `total` gets the block's sums.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* sm, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x.tok, off), b = __shfl_up_sync(0xffffffffu, x.need, off),
                    c = __shfl_up_sync(0xffffffffu, x.rel, off);
    if (lane >= off) {
      x.tok += a;
      x.need += b;
      x.rel += c;
    }
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  Sums before{0, 0, 0};
  total = Sums{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kStepThreads / 32; ++w) {
    if (w == warp) before = total;
    total.tok += sm[w].tok;
    total.need += sm[w].need;
    total.rel += sm[w].rel;
  }
  __syncthreads();  // sm is reused
  return Sums{before.tok + x.tok - v.tok, before.need + x.need - v.need, before.rel + x.rel - v.rel};
}

__global__ void __launch_bounds__(kStepThreads) paged_step_kernel(const StepParams p) {
  extern __shared__ int sm_dyn[];
  int* tok0 = sm_dyn;                // [S + 1] first token of each request
  int* need0 = sm_dyn + p.S + 1;     // [S] pages taken before it
  int* rel0 = need0 + p.S;           // [S] pages returned before it
  __shared__ Sums warp_sums[kStepThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // Every request's needs; sums in 64 bits, and a step whose sums do not fit
  // 32 bits fails the checks below before any of them is used.
  Sums carry{0, 0, 0};
  int bad = 0;
  for (int base = 0; base < p.S; base += kStepThreads) {
    const int s = base + tid;
    Sums v{0, 0, 0};
    if (s < p.S) {
      const int c = p.ctx[s], n = p.nlen[s];
      if (c < 0 || n < -1 || static_cast<long long>(c) + n > 0x7fffffffll) {
        bad |= 8;
      } else {
        const int old = static_cast<int>((static_cast<long long>(c) + p.P - 1) / p.P);
        if (old > p.max_pages) bad |= 2;
        if (n < 0) {
          v.rel = old;
        } else {
          const int want = static_cast<int>((static_cast<long long>(c) + n + p.P - 1) / p.P);
          if (want > p.max_pages) bad |= 2;
          v.tok = n;
          v.need = want - old;
        }
      }
    }
    Sums total;
    const Sums at = block_scan(v, warp_sums, total);
    if (s < p.S) {
      tok0[s] = static_cast<int>(carry.tok + at.tok);
      need0[s] = static_cast<int>(carry.need + at.need);
      rel0[s] = static_cast<int>(carry.rel + at.rel);
    }
    carry.tok += total.tok;
    carry.need += total.need;
    carry.rel += total.rel;
  }
  const int head = p.pool[0], count = p.pool[1];
  if (tid == 0) {
    if (carry.need > count) bad |= 1;
    if (carry.tok > p.T) bad |= 4;
    if (head < 0 || head >= p.F || count < 0 || count + carry.rel > p.F) bad |= 16;
    tok0[p.S] = static_cast<int>(carry.tok);
  }
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  const int status = s_bad;
  const bool ok = status == 0;
  const int total = ok ? static_cast<int>(carry.tok) : 0;
  const int gtid = blockIdx.x * kStepThreads + tid, gsize = gridDim.x * kStepThreads;

  if (gtid == 0) {
    p.info[0] = static_cast<int>(min(carry.tok, 0x7fffffffll));
    p.info[1] = static_cast<int>(min(carry.need, 0x7fffffffll));
    p.info[2] = static_cast<int>(min(carry.rel, 0x7fffffffll));
    p.info[3] = status;
    // pool and pool_out may be one buffer, and other CTAs may still have to
    // read it: the launch with one CTA writes it here, else a second kernel
  }
  // the requests' offsets and lengths
  for (int s = gtid; s <= p.S; s += gsize) {
    p.cu_q[s] = ok ? tok0[s] : 0;
    if (s < p.S) {
      const int n = p.nlen[s];
      p.kv[s] = ok && n >= 0 ? p.ctx[s] + n : 0;
    }
  }
  // pages: one request per warp
  if (ok) {
    const int lane = tid & 31;
    for (int s = gtid >> 5; s < p.S; s += gsize >> 5) {
      const int c = p.ctx[s], n = p.nlen[s];
      const int old = static_cast<int>((static_cast<long long>(c) + p.P - 1) / p.P);
      int* row = p.bt + static_cast<size_t>(s) * p.max_pages;
      if (n < 0) {
        for (int j = lane; j < old; j += 32)
          p.ring[(static_cast<long long>(head) + count + rel0[s] + j) % p.F] = row[j];
      } else {
        const int want = static_cast<int>((static_cast<long long>(c) + n + p.P - 1) / p.P);
        for (int j = old + lane; j < want; j += 32)
          row[j] = p.ring[(static_cast<long long>(head) + need0[s] + j - old) % p.F];
      }
    }
  }
  // tokens: a page that was there before comes from the table, a new one from the ring
  for (int t = gtid; t < p.T; t += gsize) {
    int pos = -1, slot = -1;
    if (t < total) {
      int lo = 0, hi = p.S - 1;  // the last request with tok0 <= t
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (tok0[m] <= t) lo = m;
        else hi = m - 1;
      }
      const int c = p.ctx[lo];
      pos = c + t - tok0[lo];
      const int old = static_cast<int>((static_cast<long long>(c) + p.P - 1) / p.P);
      const int j = pos / p.P;
      const int page = j < old ? p.bt[static_cast<size_t>(lo) * p.max_pages + j]
                               : p.ring[(static_cast<long long>(head) + need0[lo] + j - old) % p.F];
      // a page number that is no page's stays out of every cache's range
      slot = page < 0 ? -1 : static_cast<int>(min(static_cast<long long>(page) * p.P + pos % p.P, 0x7fffffffll));
    }
    p.pos[t] = pos;
    p.slots[t] = slot;
  }
}

// The ring's new head and count, once every CTA of the step has read the old ones.
__global__ void paged_step_pool_kernel(const int* pool, int F, const int* info, int* pool_out) {
  const int head = pool[0], count = pool[1];
  const bool ok = info[3] == 0;
  pool_out[0] = ok ? static_cast<int>((static_cast<long long>(head) + info[1]) % F) : head;
  pool_out[1] = ok ? count - info[1] + info[2] : count;
}

}  // namespace

cudaError_t launch_paged_step(const int* ctx_lens, const int* new_lens, int S, int* block_table, int max_pages,
                              int* free_pages, int ring_size, const int* pool, int* pool_out, int page_size, int T,
                              int* cu_q, int* kv_lens, int* positions, int* slots, int* info, cudaStream_t stream) {
  StepParams p = {ctx_lens, new_lens, S,    block_table, max_pages, free_pages, ring_size, pool,
                  pool_out, page_size, T,   cu_q,        kv_lens,   positions,  slots,     info};
  const size_t smem = static_cast<size_t>(3 * S + 1) * sizeof(int);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(paged_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>((3 * kMaxS + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  const int work = T > S * 32 ? T : S * 32;
  int grid = (work + kStepThreads - 1) / kStepThreads;
  if (grid > 148) grid = 148;
  paged_step_kernel<<<grid, kStepThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  paged_step_pool_kernel<<<1, 1, 0, stream>>>(pool, ring_size, info, pool_out);
  return cudaGetLastError();
}

}  // namespace diffattn
