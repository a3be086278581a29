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
// Latency-bound: a few bytes per token.  One launch (a second, of one thread,
// only where the new pool replaces the old one in place and several CTAs read
// it): every CTA scans the requests itself (2 S integers from L2, cheaper than a second launch), keeps
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
  int write_pool;
  int* status;  // debug builds
};

struct Sums {
  long long tok, need, rel;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.tok + b.tok, a.need + b.need, a.rel + b.rel};
}
__device__ __forceinline__ Sums operator-(const Sums& a, const Sums& b) {
  return Sums{a.tok - b.tok, a.need - b.need, a.rel - b.rel};
}

// Inclusive scan over the first `width` lanes of a warp.
template <int WIDTH>
__device__ __forceinline__ Sums warp_scan(Sums x, int lane) {
#pragma unroll
  for (int off = 1; off < WIDTH; off <<= 1) {
    const Sums o{__shfl_up_sync(0xffffffffu, x.tok, off), __shfl_up_sync(0xffffffffu, x.need, off),
                 __shfl_up_sync(0xffffffffu, x.rel, off)};
    if (lane >= off) x = x + o;
  }
  return x;
}

// Exclusive block scan; `total` gets the block's sums.  The warps' totals are
// scanned by every warp for itself.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* sm, Sums& total) {
  constexpr int kWarps = kStepThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Sums x = warp_scan<32>(v, lane);
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  const Sums w = warp_scan<kWarps>(sm[lane & (kWarps - 1)], lane);
  auto of = [&](const Sums& s, int from) {
    return Sums{__shfl_sync(0xffffffffu, s.tok, from), __shfl_sync(0xffffffffu, s.need, from),
                __shfl_sync(0xffffffffu, s.rel, from)};
  };
  total = of(w, kWarps - 1);
  const Sums before = of(w, max(warp - 1, 0));
  return (warp ? before + x : x) - v;
}

// ceil(tokens / P); tokens and P are at most 2^31 - 1, so the sum fits 32 bits unsigned.
__device__ __forceinline__ int pages_of(int tokens, int P) {
  return static_cast<int>((static_cast<unsigned>(tokens) + static_cast<unsigned>(P) - 1u) / static_cast<unsigned>(P));
}
// at mod F for at < 2 F.
__device__ __forceinline__ unsigned in_ring(unsigned at, unsigned F) { return at >= F ? at - F : at; }

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
  const int head = p.pool[0], count = p.pool[1];
  // Every request's needs, a run of requests per thread; sums in 64 bits, and a
  // step whose sums do not fit 32 bits fails the checks below before any of
  // them is used.
  const int per = (p.S + kStepThreads - 1) / kStepThreads;
  const int s_lo = min(tid * per, p.S), s_hi = min(s_lo + per, p.S);
  int bad = 0;
  auto needs = [&](int s) {
    Sums v{0, 0, 0};
    const int c = p.ctx[s], n = p.nlen[s];
    if (c < 0 || n < -1 || static_cast<long long>(c) + n > 0x7fffffffll) {
      bad |= 8;
      return v;
    }
    const int old = pages_of(c, p.P);
    if (old > p.max_pages) bad |= 2;
    if (n < 0) {
      v.rel = old;
    } else {
      const int want = pages_of(c + n, p.P);
      if (want > p.max_pages) bad |= 2;
      v.tok = n;
      v.need = want - old;
    }
    return v;
  };
  Sums mine{0, 0, 0}, carry;
  for (int s = s_lo; s < s_hi; ++s) mine = mine + needs(s);
  Sums at = block_scan(mine, warp_sums, carry);
  for (int s = s_lo; s < s_hi; ++s) {
    tok0[s] = static_cast<int>(at.tok);
    need0[s] = static_cast<int>(at.need);
    rel0[s] = static_cast<int>(at.rel);
    at = at + needs(s);
  }
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
  // unsigned: tokens and pages may number 2^31 - 1, and an index takes one more step than there are
  const unsigned gtid = blockIdx.x * kStepThreads + tid, gsize = gridDim.x * kStepThreads;

  if (gtid == 0) {
    p.info[0] = static_cast<int>(min(carry.tok, 0x7fffffffll));
    p.info[1] = static_cast<int>(min(carry.need, 0x7fffffffll));
    p.info[2] = static_cast<int>(min(carry.rel, 0x7fffffffll));
    p.info[3] = status;
    // Where pool and pool_out share words, other CTAs may still have to read
    // them: then a second kernel writes the result.
    if (p.write_pool) {
      p.pool_out[0] = ok ? static_cast<int>((head + carry.need) % p.F) : head;
      p.pool_out[1] = ok ? static_cast<int>(count - carry.need + carry.rel) : count;
    }
  }
  // the requests' offsets and lengths
  for (int s = static_cast<int>(gtid); s <= p.S; s += static_cast<int>(gsize)) {
    p.cu_q[s] = ok ? tok0[s] : 0;
    if (s < p.S) {
      const int n = p.nlen[s];
      p.kv[s] = ok && n >= 0 ? p.ctx[s] + n : 0;
    }
  }
  // the request of entry e: the last one whose entries begin at or before it
  auto owner = [&](const int* first, int e) {
    int lo = 0, hi = p.S - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (first[m] <= e) lo = m;
      else hi = m - 1;
    }
    return lo;
  };
  // pages, an entry a thread: a finished request may return thousands, and a
  // warp that walked its row alone would take a trip to memory per 32 of them
  // (14.7 us against 6.5 us in all for 700 requests of up to 32K tokens)
  if (ok) {
    const unsigned taken = static_cast<unsigned>(carry.need), back = static_cast<unsigned>(carry.rel);
    for (unsigned e = gtid; e < back; e += gsize) {
      const int s = owner(rel0, static_cast<int>(e));
      const unsigned to = in_ring(static_cast<unsigned>(head) + count + e, p.F), col = e - rel0[s];
      if (DA_CHECK(p.status, to < static_cast<unsigned>(p.F) && col < static_cast<unsigned>(p.max_pages)))
        p.ring[to] = p.bt[static_cast<size_t>(s) * p.max_pages + col];
    }
    for (unsigned e = gtid; e < taken; e += gsize) {
      const int s = owner(need0, static_cast<int>(e));
      const unsigned from = in_ring(static_cast<unsigned>(head) + e, p.F), col = pages_of(p.ctx[s], p.P) + (e - need0[s]);
      if (DA_CHECK(p.status, from < static_cast<unsigned>(p.F) && col < static_cast<unsigned>(p.max_pages)))
        p.bt[static_cast<size_t>(s) * p.max_pages + col] = p.ring[from];
    }
  }
  // tokens: a page that was there before comes from the table, a new one from the ring
  for (unsigned t = gtid; t < static_cast<unsigned>(p.T); t += gsize) {
    int pos = -1, slot = -1;
    if (t < static_cast<unsigned>(total)) {
      const int lo = owner(tok0, static_cast<int>(t));
      const int c = p.ctx[lo];
      pos = c + (static_cast<int>(t) - tok0[lo]);
      const int old = pages_of(c, p.P), j = pos / p.P;
      const unsigned from = in_ring(static_cast<unsigned>(head) + need0[lo] + max(j - old, 0), p.F);
      const bool fits = DA_CHECK(p.status, pos >= c && (j < old ? j < p.max_pages : from < static_cast<unsigned>(p.F)));
      const int page = !fits ? -1 : j < old ? p.bt[static_cast<size_t>(lo) * p.max_pages + j] : p.ring[from];
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
                  pool_out, page_size, T,   cu_q,        kv_lens,   positions,  slots,     info,       0,
                  debug_status()};
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
  const bool apart = pool_out + 2 <= pool || pool + 2 <= pool_out;
  p.write_pool = grid == 1 || apart;
  paged_step_kernel<<<grid, kStepThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.write_pool) return e;
  paged_step_pool_kernel<<<1, 1, 0, stream>>>(pool, ring_size, info, pool_out);
  return cudaGetLastError();
}

}  // namespace diffattn
