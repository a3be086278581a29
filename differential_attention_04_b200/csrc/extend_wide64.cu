// Attention of requests with more than 16 query rows per key head over a paged
// cache, on the tensor cores, d = 64: one CTA computes both maps.
//
// Rows, pages, schedule and records are those of extend_wide.cu.  At d = 64
// both maps' outputs (2 x 128 float32 columns) fit tensor memory beside both
// maps' scores, so a CTA needs no partner: V is loaded once for both maps, the
// maps are combined without a cluster, and the two maps' chains
//   S_m = Q_m K_m^T  ->  softmax (warpgroup m)  ->  O_m += P_m V
// alternate on the tensor cores, one map's products under the other's softmax.
// (As a cluster of two CTAs with a map each, extend_wide.cu's way, ragged
// prompts of 8 K tokens over 16 heads took 365 us with all launches, this way 218.)
//
// Tensor memory: the scores of map m are taken 64 keys at a time into two
// buffers, at 128 m and 128 m + 64; O_m (128 columns) is at 256 + 128 m.  P_m
// (bf16, 32 columns) takes the first half of its scores' columns: a thread
// owns its row's lane, so it may overwrite scores that it has read.  With one
// buffer of 128 keys a map's scores, softmax and product ran one after the
// other and a tile of 128 keys took 4300 cycles.
//
// Order of a map's products (one thread, an in-order pipe), t counting 64 keys:
//   S(0) | S(t+1) PV(t) | ...
// PV(t) waits for p_full, which also says that S(t) has been read, so S(t+2)
// needs no barrier of its own; it overwrites P(t) behind the product that
// reads it.  Each map has an issuing thread: commits and waits take as long as
// the products, and one thread's fall under the other's products (one thread
// for both maps: 299 us against 241 for 2048 tokens behind 6K over 16 heads).
//
// Warp roles (384 threads): warp 0 loads Q and K (both maps), warp 2 loads V,
// warps 1 and 3 issue a map's MMAs each (warp 1 owns tensor memory), warps 4-7
// and 8-11 are the maps' softmax and epilogue, one query row per thread.  In the epilogue the
// two threads of a row swap halves of their normalised sums through shared
// memory (a barrier between the two warps of a row quarter, none over the
// CTA), so each finishes 64 of the 128 channels.
//
// A tile of 128 x 128 and both maps takes about 3500 cycles: 2200 of
// exponentials and packing (one pipe, shared by the two warpgroups), about as
// many of products (S at N = 64 costs 70 cycles an instruction, 35 of them
// work), and the hand-overs between them.  Scores are scaled and weights added
// in pairs (F2), and the maximum is formed in four chains: 223 us against 236
// with single ones and eight chains (pairs alone 229); one vote a tile instead
// of two: 219.  A polynomial in place of an eighth of the exponentials takes
// 2% more.  Measured: 823 TFLOP/s for 2048 tokens behind 6K over 16 heads (219
// us).
#include "extend_wide.cuh"

namespace diffattn {

namespace {

constexpr int D = 64;
constexpr int kThreads = 384;
constexpr int kBM = kWideRows;
constexpr int kBN = kUnit;
constexpr int kHalf = kBN / 2;  // keys of a step of the softmax

struct C {
  static constexpr int DV = 2 * D;
  static constexpr int BLK_BYTES = 128 * 128;     // one [128 rows][128 bytes] block
  static constexpr int MAP_BYTES = BLK_BYTES;     // a map's Q or K tile
  static constexpr int VBLK = DV / 64;
  static constexpr int V_BYTES = VBLK * BLK_BYTES;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * MAP_BYTES;
  static constexpr int OFF_V = OFF_K + 2 * 2 * MAP_BYTES;  // two stages of both maps
  static constexpr int OFF_SWAP = OFF_V + 2 * V_BYTES;     // float[2][128][64]: the halves that the maps swap
  static constexpr int OFF_BAR = OFF_SWAP + 2 * kBM * D * 4;
  static constexpr int OFF_SS = OFF_BAR + 256;             // float[2][128]: sums of squares
  static constexpr int SMEM = OFF_SS + 1024;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[2], k_empty[2];
  uint64_t v_full[2], v_empty[2];
  uint64_t v_land;      // a ragged V tile has landed; the rows behind the last key are still to be zeroed
  uint64_t s_full[2][2];  // per map and buffer: 64 keys' scores are there
  uint64_t p_full[2][2];  // their weights are there (and the scores have been read)
  // their product is done (a barrier per buffer: with one per map, a wait could
  // take the phase before the last for the one that it means)
  uint64_t pv_done[2][2];
  uint64_t o_free[2];     // per map and segment: O has been read
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barriers");

__global__ void __launch_bounds__(kThreads, 1)
    extend_wide64_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const WideParams p) {
  if (!plan_fits(p.plan, p.n, p.most, p.status)) return;
  const PlanView pv = plan_view(p.plan, p.n, 1);
  Walk wk;
  if (!wk.begin(pv, blockIdx.x, p)) return;
  const int causal = pv.head->causal;
  const int H = p.n.H, G = H / p.n.H_kv, tpt = kBM / G;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {  // the swizzled tiles need it; there is no room to align by hand
    if (threadIdx.x == 0) atomicCAS(p.status, 0, 6);
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 2);  // both maps' products have read it, as for K and V
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->s_full[i][b], 1);
        mbar_init(&bars->p_full[i][b], 4);  // one arrival per softmax warp
        mbar_init(&bars->pv_done[i][b], 1);
      }
      mbar_init(&bars->o_free[i], 4);
    }
    mbar_init(&bars->v_land, 1);
    mbar_init(&bars->mma_done, 2);
    bars->abort = 0;
    fence_mbarrier_init();
  }
  // query rows that no box writes (128 is not a multiple of G): zeros, so that they stay finite
  for (int i = tid; i < (kBM - tpt * G) * 8 * 2; i += kThreads) {
    const int map = i / ((kBM - tpt * G) * 8), j = i % ((kBM - tpt * G) * 8);
    *reinterpret_cast<uint4*>(sQ + map * C::MAP_BYTES + tpt * G * 128 + j * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  const WaitCtl wc{p.status, &bars->abort, p.limit_ns};
  // Drains (after a normal run these return at once) ignore the abort flag.
  int drain_abort = 0;
  const WaitCtl wdrain{p.status, &drain_abort, 1000000000ull};
  const TileBoxes box(p);

  // The block's 384 x 168 registers, split anew as 128 x 40 + 256 x 232 (short
  // prompts: 131 us against 147).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ---------------------------------------------------- Q / K producer --
      int gk = 0, gq = 0;  // K tiles and Q tiles issued
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int L = min(wk.t.L, p.max_keys);
        if (wk.t.L > p.max_keys && lane == 0) atomicCAS(p.status, 0, 6);
        // Q of this segment replaces the last one's once that one's S products have read it
        if (k > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_empty, (k - 1) & 1, wc)))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full, 2 * G * tpt * 128);
#pragma unroll
          for (int m = 0; m < 2; ++m)
            tma_load_4d(sQ + m * C::MAP_BYTES, &tq, &bars->q_full, 0, m, wk.t.hk * G, wk.t.tok0);
        }
        ++gq;
        for (int j = 0; j < wk.take; ++j, ++gk) {
          const int st = gk & 1, key0 = (wk.unit + j) * kBN;
          const int boxes = box.count(key0, L), row = box.row(p, wk.t, key0, boxes, lane);
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_empty[st], ((gk >> 1) & 1) ^ 1, wc)))) break;
          if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[st], 2 * boxes * box.rows * 128);
          __syncwarp();
          if (lane < boxes) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
              tma_load_4d(sK + (2 * st + m) * C::MAP_BYTES + lane * box.rows * 128, &tk, &bars->k_full[st], 0,
                          2 * wk.t.hk + m, row, 0);
          }
        }
        if (!ok || !wk.next(pv, p)) break;
      }
      // nothing may still be landing in shared memory when the CTA exits (after an
      // abort no product may have waited for the last Q either)
      mbar_wait(&bars->q_full, (gq - 1) & 1, wdrain);
      for (int j = max(0, gk - 2); j < gk; ++j) mbar_wait(&bars->k_full[j & 1], (j >> 1) & 1, wdrain);
      __syncwarp();
    } else if (warp == 2) {
      // -------------------------------------------------------- V producer --
      int gv = 0, ragged = 0;  // V tiles issued; ragged ones among them
      bool ok = true;
      while (ok) {
        const int L = min(wk.t.L, p.max_keys);
        for (int j = 0; j < wk.take; ++j, ++gv) {
          const int st = gv & 1, key0 = (wk.unit + j) * kBN;
          const int boxes = box.count(key0, L), row = box.row(p, wk.t, key0, boxes, lane);
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_empty[st], ((gv >> 1) & 1) ^ 1, wc)))) break;
          const bool full = key0 + kBN <= L;
          uint64_t* bar = full ? &bars->v_full[st] : &bars->v_land;
          uint8_t* dst = sV + st * C::V_BYTES;
          if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box.rows * 128 * C::VBLK);
          __syncwarp();
          if (lane < boxes) {
#pragma unroll
            for (int blk = 0; blk < C::VBLK; ++blk)
              tma_load_4d(dst + blk * C::BLK_BYTES + lane * box.rows * 128, &tv, bar, blk * 64, wk.t.hk, row, 0);
          }
          if (!full) {
            mbar_wait(&bars->v_land, ragged & 1, wdrain);
            ++ragged;
            clear_v_rows(dst, C::VBLK, max(0, L - key0), lane);
            if (lane == 0) mbar_arrive(&bars->v_full[st]);
          }
        }
        if (!ok || !wk.next(pv, p)) break;
      }
      for (int j = max(0, gv - 2); j < gv; ++j) mbar_wait(&bars->v_full[j & 1], (j >> 1) & 1, wdrain);
      __syncwarp();
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------- MMA issuers, one for each map --
      if (lane == 0) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, kHalf, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, C::DV, false, true);
        const int m = warp >> 1;
        const uint32_t sQa = smem_u32(sQ) + m * C::MAP_BYTES, sKa = smem_u32(sK) + m * C::MAP_BYTES, sVa = smem_u32(sV);
        const uint32_t t_s = tmem + C::TM_S + 128 * m, t_o = tmem + C::TM_O + 128 * m;
        int gs = 0;  // halves of tiles whose S products have been issued
        int gp = 0;  // and whose PV products have
        // S for half gs & 1 of tile gs / 2
        auto issue_s = [&](bool last) -> bool {
          const int st = (gs >> 1) & 1, b = gs & 1;
          if (b == 0 && !mbar_wait(&bars->k_full[st], (gs >> 2) & 1, wc)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // each instruction takes 32 bytes of every row
            umma_ss(t_s + kHalf * b, smem_desc_sw128(sQa + kk * 32, 16, 1024),
                    smem_desc_sw128(sKa + 2 * st * C::MAP_BYTES + b * kHalf * 128 + kk * 32, 16, 1024), idesc_s,
                    kk > 0 ? 1u : 0u);
          umma_commit(&bars->s_full[m][b]);
          if (b == 1) umma_commit(&bars->k_empty[st]);
          if (last) umma_commit(&bars->q_empty);
          ++gs;
          return true;
        };
        bool ok = true;
        for (int k = 0; ok; ++k) {
          const int n = 2 * wk.take;
          ok = mbar_wait(&bars->q_full, k & 1, wc) && issue_s(false);
          for (int t = 0; ok && t < n; ++t, ++gp) {
            if (t + 1 < n && !(ok = issue_s(t + 2 == n))) break;
            const int st = (gp >> 1) & 1, b = gp & 1;
            if (!(ok = mbar_wait(&bars->p_full[m][b], (gp >> 1) & 1, wc))) break;
            if (b == 0 && !(ok = mbar_wait(&bars->v_full[st], (gp >> 2) & 1, wc))) break;
            // a new segment's O replaces the last one's once that has been read
            if (t == 0 && k > 0 && !(ok = mbar_wait(&bars->o_free[m], (k - 1) & 1, wc))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kHalf / 16; ++kk)
              umma_ts(t_o, t_s + kHalf * b + 8 * kk,
                      smem_desc_sw128(sVa + st * C::V_BYTES + (b * (kHalf / 16) + kk) * 2048, C::BLK_BYTES, 1024),
                      idesc_pv, (t > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&bars->pv_done[m][b]);
            if (b == 1) umma_commit(&bars->v_empty[st]);
          }
          if (!ok || !wk.next(pv, p)) break;
        }
        // drain: every issued MMA has completed before tensor memory is read or freed
        umma_commit(&bars->mma_done);
        mbar_wait(&bars->mma_done, 0, wdrain);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ------------------------------------------------ softmax + epilogue --
    const int quarter = warp & 3, map = (warp >> 2) - 1;
    const int r = quarter * 32 + lane;  // query row within the tile (= TMEM lane)
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + C::TM_S + 128 * map, t_o = tmem + lanes + C::TM_O + 128 * map;
    const float coef = map ? map2_coefficient(p.mode, *p.lambda) : 1.f;  // c in softmax(S1) + c softmax(S2)
    const float sc = kLog2e * rsqrtf(static_cast<float>(D));
    float* swap = reinterpret_cast<float*>(smem + C::OFF_SWAP);
    float* ssx = reinterpret_cast<float*>(smem + C::OFF_SS);
    int g = 0;  // halves of tiles consumed
    bool sm_ok = true;
    do {
      const int L = min(wk.t.L, p.max_keys);
      const int lim = min(wk.t.lim0 + (causal ? r / G : 0), L - 1);  // last key that this row sees
      const bool live = r < wk.t.ntok * G;
      float m_run = -INFINITY, l_run = 0.f;
      const int n = 2 * wk.take, g_end = g + n;
      // O *= alpha (the whole warp takes part; alpha = 1 leaves a row as it is)
      auto rescale_o = [&](float alpha) {
#pragma unroll
        for (int c = 0; c < C::DV / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32_sync(t_o + 32 * c, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
          tmem_st32(t_o + 32 * c, ov);
        }
        tmem_st_wait();
        l_run *= alpha;
      };
      for (int t = 0; sm_ok && t < n; ++t, ++g) {
        const int b = g & 1;
        // every exit is taken by the whole warp (a wait may end differently in its lanes)
        if (!(sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[map][b], (g >> 1) & 1, wc)))) break;
        tc_fence_after();
        uint32_t su[kHalf];
        tmem_ld64_sync(t_s + kHalf * b, su);
        float x[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) x[i] = __uint_as_float(su[i]);
        const int last = lim - wk.unit * kBN - t * kHalf;  // last visible one of these keys
        if (last < kHalf - 1) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i)
            if (i > last) x[i] = -INFINITY;
        }
        auto max8 = [](const float (&mk)[8]) {
          return fmaxf(fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])), fmaxf(fmaxf(mk[4], mk[5]), fmaxf(mk[6], mk[7])));
        };
        if (t == 0) {  // the first keys set the reference maximum
          float mk[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mk[c] = x[c];
#pragma unroll
          for (int i = 8; i < kHalf; i += 8) {
#pragma unroll
            for (int c = 0; c < 8; ++c) mk[c] = fmaxf(mk[c], x[i + c]);
          }
          m_run = max8(mk) * sc;
        }
        // P = exp2(s*c - m_run), taken relative to the reference maximum m_run
        // as it stands; the maximum of these keys is formed alongside.  A row
        // without keys keeps the maximum -inf: all its P are 0.  P is rounded to
        // bf16, as in the dense prefill: the remainders would be a second
        // product (see extend_narrow.cu, where it is free).
        float lsum = 0.f, t_mx = -INFINITY;
        auto make_p = [&](bool with_max) {
          const float mneg = m_run == -INFINITY ? 0.f : -m_run;
          const F2 sc2(sc, sc), mneg2(mneg, mneg);
          F2 acc[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
          float mk[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mk[c] = -INFINITY;
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float a0 = x[2 * i], a1 = x[2 * i + 1];
            if (with_max) mk[i & 3] = fmaxf(mk[i & 3], fmaxf(a0, a1));
            float p0, p1;
            fma2(F2(a0, a1), sc2, mneg2).get(p0, p1);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            acc[i & 1] = add2(acc[i & 1], F2(p0, p1));
            pk[i] = pack_bf16x2(p0, p1);
          }
          tmem_st32(t_s + kHalf * b, pk);
          float l0, l1;
          add2(acc[0], acc[1]).get(l0, l1);
          lsum = l0 + l1;
          if (with_max) t_mx = fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])) * sc;
        };
        make_p(true);
        // A jump of the maximum by more than 2^64 would overflow P: rescale O
        // to the new maximum (after the previous PV has completed) and redo P.
        // (`grown`: one vote a tile where the maximum has hardly grown, the usual case)
        const bool grown = __any_sync(0xffffffffu, t_mx > m_run + kRescaleThreshold);
        const bool hard = t > 0 && t_mx > m_run + kOverflowGuard;
        if (grown && __any_sync(0xffffffffu, hard)) {
          tmem_st_wait();
          if (!(sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[map][(g - 1) & 1], ((g - 1) >> 1) & 1, wc)))) break;
          tc_fence_after();
          rescale_o(hard ? fast_exp2(m_run - t_mx) : 1.0f);
          if (hard) m_run = t_mx;
          make_p(false);
        }
        l_run += lsum;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[map][b]);
        // Lazy rescale: keep the reference within 2^8 of the running maximum.
        // O is rescaled once this PV (which used the old reference) has completed.
        const bool need = t_mx > m_run + kRescaleThreshold;
        if (grown && __any_sync(0xffffffffu, need)) {
          if (!(sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[map][b], (g >> 1) & 1, wc)))) break;
          tc_fence_after();
          rescale_o(need ? fast_exp2(m_run - t_mx) : 1.0f);
          if (need) m_run = t_mx;
          tc_fence_before();
        }
      }
      g = g_end;  // the loop may stop early after an abort: keep the tile count in step

      // ------------------------------------------------------ epilogue --
      // O is complete once the segment's last PV (and with it every earlier MMA) has.
      if (sm_ok) sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[map][(g - 1) & 1], ((g - 1) >> 1) & 1, wc));
      tc_fence_after();
      if (!wk.whole()) {
        // a part of the row's keys: this map's sums to the worker's record
        float* rec = p.recs + (2 * blockIdx.x + (wk.begins() ? 1 : 0)) * record_floats(kBM, D);
        float* orow = rec + 4 * kBM + static_cast<size_t>(r) * 2 * C::DV + map * C::DV;
#pragma unroll 1
        for (int c = 0; c < C::DV / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32_sync(t_o + 32 * c, ov);
          if (live) {
#pragma unroll
            for (int f = 0; f < 8; ++f)
              *reinterpret_cast<uint4*>(orow + 32 * c + 4 * f) =
                  make_uint4(ov[4 * f + 0], ov[4 * f + 1], ov[4 * f + 2], ov[4 * f + 3]);
          }
        }
        if (live) *reinterpret_cast<float2*>(rec + 4 * r + 2 * map) = make_float2(m_run, l_run);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->o_free[map]);
        continue;
      }
      // Map 1's thread of a row finishes channels 0 .. 63, map 2's the others: each hands over the other
      // half of its own sums.  A warp only ever touches its quarter's rows of the buffers.
      const float inv = l_run > 0.f ? coef / l_run : 0.f;
      constexpr int NC = D / 4;  // float4 chunks of a handed row
      float* give = swap + (map * kBM + r) * D;
      const float* take = swap + ((map ^ 1) * kBM + r) * D;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t ov[32];
        tmem_ld32_sync(t_o + (map ? 0 : D) + 32 * c, ov);
#pragma unroll
        for (int f = 0; f < 8; ++f)
          *reinterpret_cast<float4*>(give + (((c * 8 + f) ^ (r % NC)) * 4)) =
              make_float4(__uint_as_float(ov[4 * f + 0]) * inv, __uint_as_float(ov[4 * f + 1]) * inv,
                          __uint_as_float(ov[4 * f + 2]) * inv, __uint_as_float(ov[4 * f + 3]) * inv);
      }
      float y[D];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t ov[32];
        tmem_ld32_sync(t_o + (map ? D : 0) + 32 * c, ov);
#pragma unroll
        for (int i = 0; i < 32; ++i) y[32 * c + i] = __uint_as_float(ov[i]) * inv;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_free[map]);
      named_bar_sync(1 + quarter, 64);  // both warps' halves are there
      float ss = 0.f;
#pragma unroll
      for (int f = 0; f < NC; ++f) {
        const float4 o = *reinterpret_cast<const float4*>(take + ((f ^ (r % NC)) * 4));
        const float os[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[4 * f + e] += os[e];
          ss = fmaf(y[4 * f + e], y[4 * f + e], ss);
        }
      }
      ssx[map * kBM + r] = ss;
      named_bar_sync(1 + quarter, 64);  // and both sums of squares; both buffers have been read
      ss += ssx[(map ^ 1) * kBM + r];
      const float gsc = norm_factor(ss / static_cast<float>(C::DV), p.eps, p.lambda_init);
      // The warp's 32 rows of 64 channels as bf16 through its part of the buffer, to be written row by row.
      const uint32_t out = smem_u32(swap + (map * kBM + quarter * 32) * D);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        uint32_t w4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = map * D + 8 * i + 2 * e;
          w4[e] = pack_bf16x2(y[8 * i + 2 * e] * gsc * __ldg(p.rms_w + c), y[8 * i + 2 * e + 1] * gsc * __ldg(p.rms_w + c + 1));
        }
        st_shared_v4(out + lane * 128 + ((i ^ (lane & 7)) << 4), w4[0], w4[1], w4[2], w4[3]);
      }
      __syncwarp();
      const int chunk = lane & 7;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int lr = 4 * i + (lane >> 3), row = quarter * 32 + lr;
        uint32_t v[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(out + lr * 128 + ((chunk ^ (lr & 7)) << 4))
                     : "memory");
        if (row < wk.t.ntok * G) {
          const size_t at = static_cast<size_t>(wk.t.tok0 + row / G) * H + wk.t.hk * G + row % G;
          *reinterpret_cast<uint4*>(p.o + at * C::DV + map * D + 8 * chunk) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      __syncwarp();  // the buffer is read before the next segment's sums replace it
    } while (wk.next(pv, p));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}
}  // namespace

cudaError_t launch_extend_wide64(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream) {
  static unsigned long long set_ctx[64] = {};
  if (ctl.dev < 0 || ctl.dev >= 64) return cudaErrorInvalidDevice;
  if (ctl.ctx == 0 || set_ctx[ctl.dev] != ctl.ctx) {
    const cudaError_t e =
        cudaFuncSetAttribute(extend_wide64_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    set_ctx[ctl.dev] = ctl.ctx;
  }
  extend_wide64_kernel<<<wide_workers(D), kThreads, C::SMEM, stream>>>(a.tq, a.tk, a.tv, wide_params(a, recs, ctl));
  return cudaGetLastError();
}

}  // namespace diffattn
