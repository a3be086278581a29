// Differential attention of new tokens over a paged cache: the schedule of a
// step, the joining of split rows, and the launches.
//
// Query i of a request with n new tokens and L cached ones (the new ones
// included) sees keys 0 .. L - n + i (causal) or all L; a row that sees no key
// gives zeros.  Per head it is the DiffAttn equation (peer review
// "Differential Transformer", Summary, Eq. 1), the headwise RMSNorm and the
// (1 - lambda_init) scale (Eq. 3).
#include <math.h>

#include "extend_wide.cuh"

namespace diffattn {

namespace {

constexpr int kPlanThreads = 1024;

struct PlanSums {
  long long units;
  int reqs, tiles, top;  // top: the largest offset so far (a maximum, not a sum)
};

__device__ __forceinline__ PlanSums plan_add(const PlanSums& a, const PlanSums& b) {
  return PlanSums{a.units + b.units, a.reqs + b.reqs, a.tiles + b.tiles, max(a.top, b.top)};
}

// Exclusive scan over the block (identity: zeros and the smallest int); `total`
// gets the block's.  Every warp scans the warps' totals for itself.
__device__ __forceinline__ PlanSums plan_scan(PlanSums v, PlanSums* sm, PlanSums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto inclusive = [&](PlanSums x) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const PlanSums o{__shfl_up_sync(0xffffffffu, x.units, off), __shfl_up_sync(0xffffffffu, x.reqs, off),
                       __shfl_up_sync(0xffffffffu, x.tiles, off), __shfl_up_sync(0xffffffffu, x.top, off)};
      if (lane >= off) x = plan_add(o, x);
    }
    return x;
  };
  auto of = [](const PlanSums& x, int from) {
    return PlanSums{__shfl_sync(0xffffffffu, x.units, from), __shfl_sync(0xffffffffu, x.reqs, from),
                    __shfl_sync(0xffffffffu, x.tiles, from), __shfl_sync(0xffffffffu, x.top, from)};
  };
  const PlanSums none{0, 0, 0, static_cast<int>(0x80000000)};
  const PlanSums x = inclusive(v);
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  static_assert(kPlanThreads == 1024, "one total a lane");
  const PlanSums w = inclusive(sm[lane]);
  __syncthreads();  // sm is reused
  total = of(w, 31);
  const PlanSums last = of(w, max(warp - 1, 0)), prev = of(x, max(lane - 1, 0));
  const PlanSums before = warp ? last : none;
  return lane ? plan_add(before, prev) : before;
}

__device__ __forceinline__ int units_of(long long keys) {
  return keys <= 0 ? 1 : static_cast<int>((keys + kUnit - 1) / kUnit);
}

// The last i < n with pre[i] <= u (pre[0] = 0, non-decreasing).
template <class F>
__device__ __forceinline__ int last_at_most(int lo, int hi, long long u, F pre) {
  while (lo < hi) {
    const int m = static_cast<int>((static_cast<long long>(lo) + hi + 1) >> 1);
    if (pre(m) <= u) lo = m;
    else hi = m - 1;
  }
  return lo;
}

// One CTA: it reads each length once, and the two lists are short.  Latency-
// bound (block scans and, per worker, two binary searches in L2); a step pays
// it once for all layers.
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const int* __restrict__ cu,
                                                                   const int* __restrict__ kvl, ExtendShape n,
                                                                   int causal, char* plan, int* status) {
  __shared__ PlanSums sm[kPlanThreads / 32];
  const PlanLayout lay = plan_layout(n);
  PlanHeader* head = reinterpret_cast<PlanHeader*>(plan);
  NarrowReq* narrow = reinterpret_cast<NarrowReq*>(plan + lay.narrow);
  WideTile* wide = reinterpret_cast<WideTile*>(plan + lay.wide);
  long long* npre = reinterpret_cast<long long*>(plan + lay.narrow_pre);
  long long* wpre = reinterpret_cast<long long*>(plan + lay.wide_pre);
  WideItem* items = reinterpret_cast<WideItem*>(plan + lay.items);
  __shared__ long long cut[2][kNarrowWorkers + 1];  // where the workers' ranges begin on the lines
  __shared__ long long whole_cost[kNarrowWorkers];  // of a wide worker's whole items
  __shared__ int s_rounds;
  const int tid = threadIdx.x, lane = tid & 31;
  const int G = n.H / n.H_kv, tpt = kWideRows / G;

  // the requests, into the two lists
  PlanSums carry{0, 0, 0, 0};
  for (int base = 0; base < n.S; base += kPlanThreads) {
    const int s = base + tid;
    int q0 = 0, nq = 0, L = 0;
    bool mine = s < n.S;
    PlanSums v{0, 0, 0, static_cast<int>(0x80000000)};
    if (mine) {
      q0 = cu[s];
      const long long end = cu[s + 1];
      L = kvl[s];
      // offsets must not fall below an earlier one: then no two requests share rows, and
      // the row tiles fit their list
      v.top = q0;
      const bool fits = q0 >= 0 && end >= q0 && end <= n.T && L >= 0 && L <= kMaxKeys && end - q0 <= n.max_new;
      nq = fits ? static_cast<int>(end - q0) : -1;
    }
    // whether it fits is only known with the largest earlier offset, so that is scanned first
    PlanSums total;
    const PlanSums before = plan_scan(v, sm, total);
    if (mine && (nq < 0 || q0 < max(carry.top, before.top))) {
      atomicCAS(status, 0, 6);
      nq = -1;
    }
    carry.top = max(carry.top, total.top);
    const bool is_wide = static_cast<long long>(nq) * G > narrow_rows(n);
    v = PlanSums{0, 0, 0, static_cast<int>(0x80000000)};
    if (nq > 0 && !is_wide) {
      v.reqs = 1;
      v.units = static_cast<long long>(units_of(L)) * n.H_kv;
    }
    if (is_wide) v.tiles = (nq + tpt - 1) / tpt;
    const PlanSums at = plan_scan(v, sm, total);
    const int i = carry.reqs + at.reqs;
    if (v.reqs && DA_CHECK(status, i < n.S)) {
      narrow[i] = NarrowReq{q0, nq, L, s};
      npre[i] = carry.units + at.units;
    }
    // a warp writes the row tiles of one request at a time
    for (unsigned todo = __ballot_sync(0xffffffffu, v.tiles > 0); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const int first = __shfl_sync(0xffffffffu, carry.tiles + at.tiles, from);
      const int cnt = __shfl_sync(0xffffffffu, v.tiles, from), fq = __shfl_sync(0xffffffffu, q0, from);
      const int fn = __shfl_sync(0xffffffffu, nq, from), fL = __shfl_sync(0xffffffffu, L, from);
      const int fs = __shfl_sync(0xffffffffu, s, from);
      for (int i = lane; i < cnt && first + i < lay.max_tiles; i += 32) {
        WideTile w;
        w.tok0 = fq + i * tpt;
        w.ntok = min(tpt, fn - i * tpt);
        w.lim0 = causal ? fL - fn + i * tpt : fL - 1;
        w.units = units_of(causal ? static_cast<long long>(w.lim0) + w.ntok : fL);
        w.L = fL;
        w.s = fs;
        w.first = first;
        w.count = cnt;
        wide[first + i] = w;
      }
    }
    carry.reqs += total.reqs;
    carry.tiles += total.tiles;
    carry.units += total.units;
  }
  const int nreqs = carry.reqs, ntiles = min(carry.tiles, lay.max_tiles);
  const long long nunits = carry.units;
  __syncthreads();  // the tiles are read by other threads
  long long wunits = 0;  // per key head
  for (int base = 0; base < ntiles; base += kPlanThreads) {
    const int x = base + tid;
    const PlanSums v{x < ntiles ? wide[x].units : 0, 0, 0, 0};
    PlanSums total;
    const PlanSums at = plan_scan(v, sm, total);
    if (x < ntiles) wpre[x] = wunits + at.units;
    wunits += total.units;
  }
  if (tid == 0) {
    npre[nreqs] = nunits;
    wpre[ntiles] = wunits;
  }
  __syncthreads();
  const int wc = wide_cost(n.d);
  const long long U[2] = {nunits + static_cast<long long>(nreqs) * n.H_kv * kNarrowCost,
                          (wunits + static_cast<long long>(ntiles) * wc) * n.H_kv};
  const int W[2] = {static_cast<int>(min(U[0], static_cast<long long>(kNarrowWorkers))),
                    static_cast<int>(min(U[1], static_cast<long long>(wide_workers(n.d))))};
  auto wide_line = [&](int k) { return wpre[k] + static_cast<long long>(k) * wc; };  // of one key head
  // the wide items in order, and how many rounds of whole ones leave every worker at least one unit of its share
  auto item_index = [&](const WideTile& t, int x, int hk) {
    return static_cast<long long>(t.first) * n.H_kv + static_cast<long long>(hk) * t.count + (x - t.first);
  };
  for (int x = tid; x < ntiles; x += kPlanThreads) {
    const WideTile t = wide[x];
    for (int hk = 0; hk < n.H_kv; ++hk)
      if (DA_CHECK(status, item_index(t, x, hk) >= 0 &&
                               item_index(t, x, hk) < static_cast<long long>(lay.max_tiles) * n.H_kv))
        items[item_index(t, x, hk)] = WideItem{t.tok0, t.ntok, t.lim0, t.units, t.L, t.s, hk, x};
  }
  const long long nitems = static_cast<long long>(ntiles) * n.H_kv;
  if (tid == 0) s_rounds = W[1] > 0 ? static_cast<int>(nitems / W[1]) : 0;
  __syncthreads();
  // A worker's whole items of rounds 0 .. limit - 1 while they cost at most `most`: their number, and their cost.
  auto whole_items = [&](int limit, long long most, long long& cost) {
    cost = 0;
    int r = 0;
    while (r < limit) {
      int u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = r + i < limit ? items[static_cast<long long>(r + i) * W[1] + tid].units : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r < limit) {
          if (cost + u[i] + wc > most) return r;
          cost += u[i] + wc;
          ++r;
        }
      }
    }
    return r;
  };
  if (tid < W[1]) {
    long long cost;
    const int r = whole_items(static_cast<int>(nitems / W[1]), U[1] / W[1] - 1, cost);
    atomicMin(&s_rounds, r);
  }
  __syncthreads();
  const int rounds = s_rounds;
  if (tid < W[1]) {
    long long cost;
    whole_items(rounds, U[1], cost);
    whole_cost[tid] = cost;
  }
  if (tid < W[0]) cut[0][tid] = tid * U[0] / W[0];
  __syncthreads();
  if (tid < W[1]) {
    // the line behind the whole items, cut where the workers' shares are used up
    long long at = U[1], used = 0;
    const long long done = static_cast<long long>(rounds) * W[1];
    if (done < nitems) {
      const WideItem it = items[done];
      const int first = wide[it.tile].first, cnt = wide[it.tile].count;
      at = wide_line(first) * n.H_kv + it.hk * (wide_line(first + cnt) - wide_line(first)) + wide_line(it.tile) -
           wide_line(first);
    }
    for (int v = 0; v < tid; ++v) used += whole_cost[v];
    cut[1][tid] = at + tid * U[1] / W[1] - used;
  }
  if (tid == 0) *head = PlanHeader{{W[0], W[1]}, causal, ntiles, n, kPlanMagic, rounds, {nunits, wunits}};
  __syncthreads();
  // the workers: where each begins, and the item that it leaves unfinished
  for (int i = tid; i < kNarrowWorkers + wide_workers(n.d); i += kPlanThreads) {
    const int c = i >= kNarrowWorkers, w = c ? i - kNarrowWorkers : i;
    WorkStart st{};
    WorkTail tl{0, 0, 0, 0};
    if (w < W[c]) {
      const int ic = c ? wc : kNarrowCost;
      // the item at u on the line of costs, its first unit and the one behind its last (counted over all
      // items), and the unit of it that u means
      struct Spot {
        int at, hk;
        long long cost, b, e;  // where the item begins on the line; its first unit and the one behind its last
        long long unit;
      };
      auto spot = [&](long long u) -> Spot {
        Spot r;
        if (c == 0) {
          auto cost = [&](int k) { return npre[k] + static_cast<long long>(k) * n.H_kv * ic; };
          r.at = last_at_most(0, nreqs - 1, u, cost);
          const long long per = (npre[r.at + 1] - npre[r.at]) / n.H_kv, off = u - cost(r.at);
          r.hk = static_cast<int>(off / (per + ic));
          r.cost = cost(r.at) + r.hk * (per + ic);
          r.b = npre[r.at] + r.hk * per;
          r.e = r.b + per;
        } else {
          auto cost = wide_line;
          const int any = last_at_most(0, ntiles - 1, u, [&](int k) { return cost(wide[k].first) * n.H_kv; });
          const int first = wide[any].first, cnt = wide[any].count;
          const long long c0 = cost(first), per = cost(first + cnt) - c0, off = u - c0 * n.H_kv;
          r.hk = static_cast<int>(off / per);
          const long long in = off - r.hk * per;
          r.at = last_at_most(first, first + cnt - 1, in, [&](int k) { return cost(k) - c0; });
          r.cost = c0 * n.H_kv + r.hk * per + cost(r.at) - c0;
          r.b = wpre[first] * n.H_kv + r.hk * (wpre[first + cnt] - wpre[first]) + wpre[r.at] - wpre[first];
          r.e = r.b + wpre[r.at + 1] - wpre[r.at];
        }
        r.unit = max(0ll, u - r.cost - ic);
        return r;
      };
      const bool last = w + 1 == W[c], none = cut[c][w] >= U[c];
      if (!none) {
        const Spot x0 = spot(cut[c][w]);
        const Spot x1 = last ? x0 : spot(min(cut[c][w + 1], U[c] - 1));
        const long long all = c ? wunits * n.H_kv : nunits;
        const long long u0 = x0.b + x0.unit, u1 = last || cut[c][w + 1] >= U[c] ? all : x1.b + x1.unit;
        auto index = [&](const Spot& x) { return c ? static_cast<int>(item_index(wide[x.at], x.at, x.hk)) : x.at; };
        if (u1 > u0)
          st = WorkStart{index(x0), x0.hk, static_cast<int>(x0.unit), static_cast<int>(u1 - u0),
                         c ? NarrowReq{} : narrow[x0.at]};
        // The item that the range ends in is split if the next worker begins
        // inside it.  Its owner is the last worker that begins at or before
        // its first unit.
        if (u1 < all && x1.unit > 0) {
          const int owner = last_at_most(0, w, x1.cost + ic, [&](int v) { return cut[c][v]; });
          const int end =
              last_at_most(w + 1, W[c] - 1, x1.cost + ic + x1.e - x1.b - 1, [&](int v) { return cut[c][v]; });
          tl = WorkTail{index(x1), x1.hk, end - owner + 1, w - owner};
        }
      }
    }
    reinterpret_cast<WorkStart*>(plan + lay.starts[c])[w] = st;
    reinterpret_cast<WorkTail*>(plan + lay.tails[c])[w] = tl;
  }
}

// Joins the rows that were split.  An item of P parts is joined by the blocks
// of the workers that have nothing but it at the end of their range (its owner
// and all but the last of the others): a warp a row where there are few parts,
// a block a row where there are many.  The parts are taken to the common
// maximum and added in the order of the keys (many parts: within eight groups,
// then group by group), then comes the epilogue of a whole row.  Reads 16 d
// bytes a part and row; with one block a row for every worker it took 48 us
// where this takes 15 (a mixed step of 20 over 4 heads, d 128).
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinFew = kJoinWarps;  // parts up to which a warp takes a row alone
constexpr int kJoinWideBlocks = kWideRows / kJoinWarps;  // blocks of a wide worker (a narrow one has one)

template <int D>
__global__ void __launch_bounds__(kJoinThreads) extend_join_kernel(const ExtendArgs a, const float* nrecs,
                                                                   const float* wrecs, UnitLimits most, int* status) {
  constexpr int DV = 2 * D;
  constexpr int NV = 2 * DV / 128;  // float4 of a lane: first map 1's channels, then the same of map 2
  if (!plan_fits(a.plan, a.n, most, status)) return;
  const bool is_wide = blockIdx.x >= kNarrowWorkers;
  const int bi = is_wide ? blockIdx.x - kNarrowWorkers : blockIdx.x;
  const int blocks = is_wide ? kJoinWideBlocks : 1;
  const int w = bi / blocks;
  const PlanView pv = plan_view(a.plan, a.n, is_wide);
  const WorkTail tl = pv.tails[w];
  if (tl.parts == 0) return;
  const int G = a.n.H / a.n.H_kv;
  // debug builds: the parts' records are the class's workers', and the rows a request's
  if (!DA_CHECK(status, tl.parts > 1 && tl.member >= 0 && tl.member < tl.parts - 1 && w >= tl.member &&
                            w - tl.member + tl.parts <= (is_wide ? wide_workers(a.n.d) : kNarrowWorkers) &&
                            tl.hk >= 0 && tl.hk < a.n.H_kv))
    return;
  const int tok0 = is_wide ? wide_at(pv.wide, tl.at, a.n, status).tok0 : narrow_at(pv.narrow, tl.at, a.n, status).q0;
  const int R = (is_wide ? wide_at(pv.wide, tl.at, a.n, status).ntok : narrow_at(pv.narrow, tl.at, a.n, status).n) * G;
  const int rows = is_wide ? kWideRows : narrow_rows(a.n);
  const float* recs = is_wide ? wrecs : nrecs;
  const size_t rec = record_floats(rows, D);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int owner = w - tl.member, team = tl.member * blocks + bi % blocks, teams = (tl.parts - 1) * blocks;
  // part p: the owner's last record, then the first records of the workers behind it
  auto part = [&](int p) { return recs + (p == 0 ? 2 * owner + 1 : 2 * (owner + p)) * rec; };
  auto max_of = [](float x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
  };
  auto sum_of = [](float x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
  };
  const float c2 = map2_coefficient(a.mode, *a.lambda);
  auto out_row = [&](int r) {
    return static_cast<__nv_bfloat16*>(a.o) +
           (static_cast<size_t>(tok0 + r / G) * a.n.H + static_cast<size_t>(tl.hk) * G + r % G) * DV;
  };
  float4 x[NV];
  auto add_part = [&](int p, int r, float f1, float f2) {
    const float4* o = reinterpret_cast<const float4*>(part(p) + 4 * rows + static_cast<size_t>(r) * 2 * DV);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float4 v = __ldg(o + 32 * i + lane);
      const float f = i < NV / 2 ? f1 : f2;
      x[i].x = fmaf(f, v.x, x[i].x);
      x[i].y = fmaf(f, v.y, x[i].y);
      x[i].z = fmaf(f, v.z, x[i].z);
      x[i].w = fmaf(f, v.w, x[i].w);
    }
  };

  if (tl.parts <= kJoinFew) {
    for (int r = team * kJoinWarps + warp; r < R; r += teams * kJoinWarps) {
      float4 ml = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      if (lane < tl.parts) ml = *reinterpret_cast<const float4*>(part(lane) + 4 * r);
      const float M1 = max_of(ml.x), M2 = max_of(ml.z);
      const float f1 = M1 == -INFINITY ? 0.f : fast_exp2(ml.x - M1), f2 = M2 == -INFINITY ? 0.f : fast_exp2(ml.z - M2);
      const float l1 = sum_of(f1 * ml.y), l2 = sum_of(f2 * ml.w);
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int p = 0; p < tl.parts; ++p)
        add_part(p, r, __shfl_sync(0xffffffffu, f1, p), __shfl_sync(0xffffffffu, f2, p));
      const float i1 = l1 > 0.f ? 1.f / l1 : 0.f, i2 = l2 > 0.f ? c2 / l2 : 0.f;
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        float4& y = x[i];
        const float4& z = x[i + NV / 2];
        y.x = fmaf(y.x, i1, z.x * i2);
        y.y = fmaf(y.y, i1, z.y * i2);
        y.z = fmaf(y.z, i1, z.z * i2);
        y.w = fmaf(y.w, i1, z.w * i2);
        ss += y.x * y.x + y.y * y.y + y.z * y.z + y.w * y.w;
      }
      const float gsc = norm_factor(sum_of(ss) / DV, a.eps, a.lambda_init);
      __nv_bfloat16* o = out_row(r);
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        const int ch = 128 * i + 4 * lane;
        const float* rw = a.rms_w + ch;
        *reinterpret_cast<uint2*>(o + ch) = make_uint2(pack_bf16x2(x[i].x * gsc * rw[0], x[i].y * gsc * rw[1]),
                                                       pack_bf16x2(x[i].z * gsc * rw[2], x[i].w * gsc * rw[3]));
      }
    }
    return;
  }

  __shared__ float2 f[kNarrowWorkers];  // factors of a part's two maps
  __shared__ float red[4][kJoinWarps];
  __shared__ float acc[kJoinWarps][2 * DV];
  constexpr int PT = (kNarrowWorkers + kJoinThreads - 1) / kJoinThreads;  // parts of a thread
  for (int r = team; r < R; r += teams) {
    float4 ml[PT];
    float M1 = -INFINITY, M2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int p = tid + i * kJoinThreads;
      ml[i] = p < tl.parts ? *reinterpret_cast<const float4*>(part(p) + 4 * r)
                           : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      M1 = fmaxf(M1, ml[i].x);
      M2 = fmaxf(M2, ml[i].z);
    }
    M1 = max_of(M1);
    M2 = max_of(M2);
    if (lane == 0) {
      red[0][warp] = M1;
      red[1][warp] = M2;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kJoinWarps; ++g) {
      M1 = fmaxf(M1, red[0][g]);
      M2 = fmaxf(M2, red[1][g]);
    }
    float l1 = 0.f, l2 = 0.f;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int p = tid + i * kJoinThreads;
      const float f1 = M1 == -INFINITY ? 0.f : fast_exp2(ml[i].x - M1);
      const float f2 = M2 == -INFINITY ? 0.f : fast_exp2(ml[i].z - M2);
      if (p < tl.parts) f[p] = make_float2(f1, f2);
      l1 = fmaf(f1, ml[i].y, l1);
      l2 = fmaf(f2, ml[i].w, l2);
    }
    l1 = sum_of(l1);
    l2 = sum_of(l2);
    if (lane == 0) {
      red[2][warp] = l1;
      red[3][warp] = l2;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int p = warp; p < tl.parts; p += kJoinWarps) add_part(p, r, f[p].x, f[p].y);
#pragma unroll
    for (int i = 0; i < NV; ++i) *reinterpret_cast<float4*>(&acc[warp][4 * (32 * i + lane)]) = x[i];
    __syncthreads();
    float y = 0.f;
    if (tid < DV) {
      float o1 = 0.f, o2 = 0.f;
      l1 = l2 = 0.f;
#pragma unroll
      for (int g = 0; g < kJoinWarps; ++g) {
        o1 += acc[g][tid];
        o2 += acc[g][DV + tid];
        l1 += red[2][g];
        l2 += red[3][g];
      }
      y = (l1 > 0.f ? o1 / l1 : 0.f) + c2 * (l2 > 0.f ? o2 / l2 : 0.f);
    }
    const float part_ss = sum_of(y * y);
    if (lane == 0) red[0][warp] = part_ss;
    __syncthreads();
    float ss = 0.f;
#pragma unroll
    for (int g = 0; g < kJoinWarps; ++g) ss += red[0][g];
    if (tid < DV) {
      const float gsc = norm_factor(ss / DV, a.eps, a.lambda_init);
      out_row(r)[tid] = __float2bfloat16_rn(y * gsc * a.rms_w[tid]);
    }
    __syncthreads();  // the next row reuses the shared memory
  }
}

size_t narrow_record_bytes(const ExtendShape& n) {
  return 2 * kNarrowWorkers * record_floats(narrow_rows(n), n.d) * sizeof(float);
}
}  // namespace

bool extend_wide_possible(const ExtendShape& n) { return wide_possible(n); }
size_t extend_plan_bytes(const ExtendShape& n) { return plan_layout(n).bytes; }

size_t extend_workspace_bytes(const ExtendShape& n) {
  size_t b = narrow_record_bytes(n);
  if (wide_possible(n)) b += 2 * wide_workers(n.d) * record_floats(kWideRows, n.d) * sizeof(float);
  return b;
}

cudaError_t launch_extend_plan(const int* cu_q, const int* kv_lens, const ExtendShape& n, int causal, void* plan,
                               DevCtl ctl, cudaStream_t stream) {
  extend_plan_kernel<<<1, kPlanThreads, 0, stream>>>(cu_q, kv_lens, n, causal ? 1 : 0, static_cast<char*>(plan),
                                                     ctl.status);
  return cudaGetLastError();
}

cudaError_t launch_extend(const ExtendArgs& a, DevCtl ctl, cudaStream_t stream) {
  float* nrecs = static_cast<float*>(a.workspace);
  float* wrecs = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + narrow_record_bytes(a.n));
  const bool wide = wide_possible(a.n);
  cudaError_t e = launch_extend_narrow(a, nrecs, ctl, stream);
  if (e != cudaSuccess) return e;
  if (wide)
    e = a.n.d == 64 ? launch_extend_wide64(a, wrecs, ctl, stream) : launch_extend_wide128(a, wrecs, ctl, stream);
  if (e != cudaSuccess) return e;
  // no item can be split where every request's keys fit one unit
  if (!wide && static_cast<long long>(a.max_pages) * a.page_size <= kUnit) return cudaSuccess;
  const UnitLimits most = unit_limits(a.n, keys_of_table(a.max_pages, a.page_size));
  const unsigned grid = kNarrowWorkers + (wide ? wide_workers(a.n.d) * kJoinWideBlocks : 0);
  if (a.n.d == 128)
    extend_join_kernel<128><<<grid, kJoinThreads, 0, stream>>>(a, nrecs, wrecs, most, ctl.status);
  else
    extend_join_kernel<64><<<grid, kJoinThreads, 0, stream>>>(a, nrecs, wrecs, most, ctl.status);
  return cudaGetLastError();
}

}  // namespace diffattn
