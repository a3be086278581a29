// Schedule of a serving step's attention, shared by the plan kernel, the two
// attention kernels and the kernel that joins split rows.
//
// A request's query rows are its new tokens times the G = H / H_kv query heads
// that share a key head.  Requests of at most narrow_rows rows are "narrow"
// (extend_narrow.cu: memory-bound), the others "wide" (extend_wide*.cu: tiles of
// up to 128 rows on the tensor cores).  An item is one (request, key head) of
// the narrow class or one (row tile, key head) of the wide class; its work is
// its number of units, blocks of kUnit keys that its last row can see (at
// least one, so that rows without keys are written too), and a fixed number
// more for what it costs once (the start of its pipeline, its epilogue).
//
// The items of a class are in order of requests, then key heads, then row
// tiles, and lie end to end on a line of costs.  W workers get the same share
// of it (to one unit) whatever the lengths:
//   * Wide class only: in each of the first R rounds, worker w takes the whole
//     item round * W + w.  So the row tiles of a key head run side by side and
//     read its keys and values at about the same time, once from memory for
//     all of them.  R is the most rounds that leave no worker above its share.
//   * The rest of the line is cut where the workers' shares are used up.  Only
//     a worker's first and last items there can be split: their unnormalised
//     sums go to the workspace records 2 w (the item began before the worker's
//     range) and 2 w + 1 (it began inside it and goes on behind it), which the
//     joining kernel adds up in order.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace diffattn {

constexpr int kUnit = 128;
constexpr int kWideRows = 128;
// What an item costs beside its units, in units, from times of 74 requests of
// 128 rows over 128 and 640 keys: 12 and 20 thousand cycles against 3.7 and 2.8
// thousand a unit (ten ragged chunks and prompts, d = 128: 165 us with 3, 138
// with 7).  A narrow item's end is hidden by the loads that run ahead.
constexpr int kNarrowCost = 0;
__host__ __device__ constexpr int wide_cost(int d) { return d == 64 ? 3 : 7; }
constexpr int kNarrowWorkers = 296;  // two CTAs per SM
// One CTA per SM (both maps), or one CTA pair per two SMs (a map each): two
// output tiles of 2 d = 128 columns fit tensor memory, two of 256 do not.
__host__ __device__ constexpr int wide_workers(int d) { return d == 64 ? 148 : 74; }

struct PlanHeader {
  int workers[2];      // workers of the narrow and the wide class
  int causal;
  int tiles;           // entries of the list of row tiles
  ExtendShape shape;   // the sizes that the plan was made for
  int magic;
  int rounds;          // whole items of a wide worker
  long long units[2];  // of the narrow class, and of the wide class per key head
};
constexpr int kPlanMagic = 0x64706c6e;
constexpr int kMaxKeys = 0x7fffff00;  // keys of a request: a unit behind the last one still has a 32-bit index
static_assert(sizeof(PlanHeader) == 64, "the sections behind the header are 16-byte aligned");

struct NarrowReq {
  int q0, n, L, s;  // first row, new tokens, cached tokens, request
};
struct WideTile {  // a row tile, while the schedule is made
  int tok0, ntok, lim0, units;
  int L, s, first, count;  // first row tile of its request and their number
};
struct WideItem {
  int tok0, ntok;  // its tokens' rows
  int lim0;        // last key its first token sees (causal: one more per token)
  int units;
  int L, s, hk;    // cached tokens, request, key head
  int tile;        // in the schedule's list of row tiles
};
// Where a worker's range begins: item (list index, and key head and request of
// a narrow one), its unit, and how many units it takes.
struct WorkStart {
  int at, hk, unit, count;
  NarrowReq rq;
};
// The split item that the range ends in and that goes on behind it, in how
// many parts (0: there is none), and which of them the worker has.
struct WorkTail {
  int at, hk, parts, member;
};

struct PlanLayout {
  size_t starts[2], tails[2], narrow, narrow_pre, wide, wide_pre, items, bytes;
  int max_tiles;  // row tiles of the wide class there can be
};

// The most rows of a request that the host's bound allows.
__host__ __device__ inline long long most_rows(const ExtendShape& n) {
  return static_cast<long long>(n.max_new) * (n.H / n.H_kv);
}
// Rows of the narrow class.  Two column tiles (9 to 16 rows) are 20% faster
// than a 128-row tile, but the kernel that has them takes 7 to 10 us longer over
// the single tokens of a step with chunks (mixed step 48 against 55 us), so they
// are for steps that need no wide kernel.  It goes by the bound of new tokens, since
// the lengths are on the device.  With a wide bound, requests of 10 and of 16 rows
// over 32 x 2000 tokens and 16 heads take 260 and 262 us in place of 213 and 219 (d
// 64: 148 and 150 in place of 129 and 133), and 64 single tokens over 2000 take 340
// in place of 332 (194, 184), for a wide kernel that finds no work.
__host__ __device__ inline int narrow_rows(const ExtendShape& n) {
  return most_rows(n) > 8 && most_rows(n) <= 16 ? 16 : 8;
}
__host__ __device__ inline bool wide_possible(const ExtendShape& n) { return most_rows(n) > 16; }

__host__ __device__ inline PlanLayout plan_layout(const ExtendShape& n) {
  PlanLayout l;
  const int tpt = kWideRows / (n.H / n.H_kv);
  l.max_tiles = wide_possible(n) ? n.T / tpt + (n.S < n.T ? n.S : n.T) : 0;  // a request has a token at least
  size_t at = sizeof(PlanHeader);
  const int workers[2] = {kNarrowWorkers, wide_workers(n.d)};
  for (int c = 0; c < 2; ++c) {
    l.starts[c] = at;
    at += workers[c] * sizeof(WorkStart);
    l.tails[c] = at;
    at += workers[c] * sizeof(WorkTail);
  }
  l.narrow = at;
  at += static_cast<size_t>(n.S) * sizeof(NarrowReq);
  l.wide = at;
  at += static_cast<size_t>(l.max_tiles) * sizeof(WideTile);
  l.narrow_pre = at;
  at += (static_cast<size_t>(n.S) + 1) * sizeof(long long);
  l.wide_pre = at;
  at += (static_cast<size_t>(l.max_tiles) + 1) * sizeof(long long);
  at = (at + 15) & ~static_cast<size_t>(15);
  l.items = at;
  at += static_cast<size_t>(l.max_tiles) * n.H_kv * sizeof(WideItem);
  l.bytes = (at + 15) & ~static_cast<size_t>(15);
  return l;
}

// What a row is multiplied with behind its norm.  A row of zeros (one that sees no
// key) stays one with eps = 0 too, where 1 / sqrt(0) would make it NaN.
__device__ __forceinline__ float norm_factor(float mean_square, float eps, float lambda_init) {
  const float x = mean_square + eps;
  return x > 0.f ? (1.f - lambda_init) * rsqrtf(x) : x;  // (x: 0, or a NaN that stays one)
}

// A record: (m1, l1, m2, l2) of every row, then per row both maps' sums over 2d channels.
__host__ __device__ inline size_t record_floats(int rows, int d) {
  return static_cast<size_t>(rows) * (4 + 4 * d);
}

// The most keys of a request that a block table can hold.
inline int keys_of_table(int max_pages, int page_size) {
  const long long keys = static_cast<long long>(max_pages) * page_size;
  return keys < kMaxKeys ? static_cast<int>(keys) : kMaxKeys;
}

struct PlanView {
  const PlanHeader* head;
  const WorkStart* starts;
  const WorkTail* tails;
  const NarrowReq* narrow;
  const WideItem* wide;
};
// The most units that a call works off (PlanHeader::units): what the block table
// can hold, and some more.  A length costs its time even where its keys do not
// enter, and 64 uninitialised ones of 2^30 keys would take seconds.  Below the
// limit a worker's units and steps fit 32 bits.
struct UnitLimits {
  long long units[2];
};
inline UnitLimits unit_limits(const ExtendShape& n, int max_keys) {
  constexpr long long kSpare = 1 << 14, kMost = 1ll << 36;
  const long long per = max_keys / kUnit + 1, narrow = (n.S * per + kSpare) * n.H_kv;
  const long long wide = plan_layout(n).max_tiles * per + kSpare;
  return UnitLimits{{narrow < kMost ? narrow : kMost, wide < kMost / n.H_kv ? wide : kMost / n.H_kv}};
}
// Whether the buffer holds a plan of these sizes within the limits; the kernels
// do nothing otherwise.
__device__ inline bool plan_fits(const void* plan, const ExtendShape& n, const UnitLimits& most, int* status) {
  const PlanHeader* h = static_cast<const PlanHeader*>(plan);
  const ExtendShape& p = h->shape;
  const bool ok = h->magic == kPlanMagic && p.S == n.S && p.T == n.T && p.H == n.H && p.H_kv == n.H_kv &&
                  p.d == n.d && p.max_new == n.max_new &&
                  h->units[0] <= most.units[0] && h->units[1] <= most.units[1];
  if (!ok) atomicCAS(status, 0, 6);
  // debug builds: what its lists and ranges are indexed with
  return ok && DA_CHECK(status, h->tiles >= 0 && h->tiles <= plan_layout(n).max_tiles && h->workers[0] >= 0 &&
                                    h->workers[0] <= kNarrowWorkers && h->workers[1] >= 0 &&
                                    h->workers[1] <= wide_workers(n.d) && h->rounds >= 0 &&
                                    static_cast<long long>(h->rounds) * h->workers[1] <=
                                        static_cast<long long>(h->tiles) * n.H_kv);
}
// Entries of a plan's lists.  Debug builds check the index and everything that is
// computed from the entry (rows of q and o, of the block table, a key head); one
// that is out of range counts as an entry without rows and keys.
__device__ __forceinline__ NarrowReq narrow_at(const NarrowReq* list, int at, const ExtendShape& n, int* status) {
  if (!DA_CHECK(status, at >= 0 && at < n.S)) return NarrowReq{0, 0, 0, 0};
  const NarrowReq r = list[at];
  return DA_CHECK(status, r.q0 >= 0 && r.n >= 0 && r.n <= n.T - r.q0 &&
                              static_cast<long long>(r.n) * (n.H / n.H_kv) <= narrow_rows(n) && r.L >= 0 &&
                              r.L <= kMaxKeys && r.s >= 0 && r.s < n.S)
             ? r
             : NarrowReq{0, 0, 0, 0};
}
__device__ __forceinline__ WideItem wide_at(const WideItem* list, int at, const ExtendShape& n, int* status) {
  if (!DA_CHECK(status, at >= 0 && at < static_cast<long long>(plan_layout(n).max_tiles) * n.H_kv))
    return WideItem{0, 0, -1, 1, 0, 0, 0, 0};
  const WideItem t = list[at];
  return DA_CHECK(status, t.tok0 >= 0 && t.ntok >= 0 && t.ntok <= n.T - t.tok0 &&
                              static_cast<long long>(t.ntok) * (n.H / n.H_kv) <= kWideRows && t.units >= 1 &&
                              t.units <= kMaxKeys / kUnit + 1 && t.L >= 0 && t.L <= kMaxKeys && t.s >= 0 &&
                              t.s < n.S && t.hk >= 0 && t.hk < n.H_kv)
             ? t
             : WideItem{0, 0, -1, 1, 0, 0, 0, 0};
}
__device__ inline PlanView plan_view(const void* plan, const ExtendShape& n, int cls) {
  const PlanLayout l = plan_layout(n);
  const char* p = static_cast<const char*>(plan);
  return PlanView{reinterpret_cast<const PlanHeader*>(p), reinterpret_cast<const WorkStart*>(p + l.starts[cls]),
                  reinterpret_cast<const WorkTail*>(p + l.tails[cls]),
                  reinterpret_cast<const NarrowReq*>(p + l.narrow), reinterpret_cast<const WideItem*>(p + l.items)};
}

cudaError_t launch_extend_narrow(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream);


}  // namespace diffattn
