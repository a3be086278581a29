// Attention of requests with more than 16 query rows per key head (chunks of
// prompts, whole prompts, many heads sharing a key head) over a paged cache,
// on the tensor cores, d = 128.
//
// The arithmetic of a tile is that of the dense prefill (prefill_sm100.cu): a
// cluster of two CTAs takes a tile of up to 128 query rows, CTA rank i
// computes map i + 1 (S = Q_i K_i^T with tcgen05 into tensor memory, online
// softmax with a lazy rescale, O_i += P V with P read from tensor memory), and
// the pair combines the maps at the end through distributed shared memory.
// What differs:
//   * Rows are (token, query head of the group) pairs of one request, token by
//     token, 128 / G tokens a tile: the heads that share a key head share its
//     K and V loads and fill the 128 rows.  One TMA box of G heads x 128 / G
//     tokens brings a tile's queries; rows of other requests behind the last
//     token are computed and not written.
//   * Keys come page by page: one lane per page issues its boxes (a whole page,
//     or 128 rows of a larger one).  A bad page is a box outside the tensor,
//     which TMA fills with zeros.  Keys behind the cached ones are masked in S;
//     their V rows are overwritten with zeros in shared memory before the
//     product, so that nothing that a page holds there can enter as 0 * NaN.
//   * Work is dealt as equal ranges of 128-key units (extend.cuh), so an item
//     may begin or end inside a row's keys.  Such a segment writes its
//     unnormalised O_i, maximum and sum to a record instead of combining.
//   * The output tile is copied out by warp 3 row by row (a TMA store could not
//     stop at the end of a request).
//
// Warp roles (256 threads): warp 0 loads Q_i and K_i, warp 2 loads V, warp 1
// owns tensor memory and issues the MMAs, warp 3 copies finished tiles out,
// warps 4-7 do softmax and epilogue, one query row per thread.  Pipeline and
// barriers are the prefill's; barrier phases count segments (epi_free), tiles
// (K, V, S, P) or combined segments (the exchange and the hand-over to warp 3).
// After a wait that ran out the softmax warps leave together at the start of the
// next epilogue, and every other role at its next wait.
//
// Bound: as the prefill, the softmax warps and the serial issue of products
// (about 2500 cycles a 128-key tile against 1540 of tensor work) for long
// chunks; memory for few rows over many keys; and about 20 thousand cycles an
// item for its exchange and refill, which short prompts feel (74 x 128 tokens
// over 12 heads: 147 us).  Measured: 2048 tokens behind 30K cached ones over 12
// heads 900 us in single calls with pauses (1300 TFLOP/s), 1030 us in a loop under
// the power cap; 2048 behind 6K 237 us (239 without the pairs of F2).  Two
// softmax warpgroups with 64 keys each were not faster here (chunk 1285 against 1280 us, mixed step 136 against 132).
#include "extend_wide.cuh"

namespace diffattn {

namespace {

constexpr int kThreads = 256;
constexpr int kBM = kWideRows;
constexpr int kBN = kUnit;
constexpr int D = 128;

struct C {
  static constexpr int DV = 2 * D;
  static constexpr int HALF = D;                // output columns finished by each CTA
  static constexpr int QBLK = D / 64;           // 128-byte swizzle blocks per Q/K row
  static constexpr int VBLK = DV / 64;          // and per V row
  static constexpr int BLK_BYTES = 128 * 128;   // one [128 rows][128 bytes] block
  static constexpr int Q_BYTES = kBM * D * 2;
  static constexpr int K_BYTES = kBN * D * 2;
  static constexpr int V_BYTES = kBN * DV * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + Q_BYTES;
  static constexpr int OFF_V = OFF_K + 2 * K_BYTES;
  static constexpr int OFF_BAR = OFF_V + 2 * V_BYTES;
  static constexpr int OFF_SSX = OFF_BAR + 256;  // float[128]: the partner's sums of squares
  static constexpr int SMEM_USED = OFF_SSX + 512;
  static constexpr int SMEM = SMEM_USED + 1024;  // slack for 1024-byte alignment
  static constexpr int EXCH_BYTES = kBM * HALF * 4;
  static constexpr uint32_t TM_S = 0, TM_P = 128, TM_O = 256, TM_COLS = 512;
  static_assert(EXCH_BYTES <= V_BYTES && SMEM <= 232448, "shared memory per CTA");
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[2], k_empty[2];
  uint64_t v_full[2], v_empty[2];
  uint64_t v_land;  // a ragged V tile has landed; the rows behind the last key are still to be zeroed
  uint64_t s_full, s_free;
  uint64_t p_full[2], p_empty[2];
  uint64_t mma_done;
  uint64_t exch_full, peer_ready, ss_full, epi_free;
  uint64_t tile_full;  // per combined segment: its output tile is staged
  uint32_t tmem_base;
  volatile int abort;
};
static_assert(sizeof(Bars) <= 256, "barriers");

__global__ void __launch_bounds__(kThreads, 1)
    extend_wide_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const WideParams p) {
  if (!plan_fits(p.plan, p.n, p.most, p.status)) return;  // the same for both CTAs of the cluster
  const PlanView pv = plan_view(p.plan, p.n, 1);
  Walk wk;
  if (!wk.begin(pv, blockIdx.x >> 1, p)) return;  // and this too
  const int causal = pv.head->causal;
  const int H = p.n.H, G = H / p.n.H_kv, tpt = kBM / G;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  float* ssx = reinterpret_cast<float*>(smem + C::OFF_SSX);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();  // 0: map 1, 1: map 2
  const uint32_t partner = rank ^ 1u;

  if (tid == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 1);
      mbar_init(&bars->p_full[i], 4);  // one arrival per softmax warp
      mbar_init(&bars->p_empty[i], 1);
    }
    mbar_init(&bars->v_land, 1);
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->s_free, 4);
    mbar_init(&bars->mma_done, 1);
    mbar_init(&bars->exch_full, 1);
    mbar_init(&bars->peer_ready, 1);
    mbar_init(&bars->ss_full, 1);
    mbar_init(&bars->epi_free, 1);
    mbar_init(&bars->tile_full, 4);  // one arrival per softmax warp
    bars->abort = 0;
    fence_mbarrier_init();
  }
  // query rows that no box writes (128 is not a multiple of G): zeros, so that they stay finite
  for (int i = tid; i < (kBM - tpt * G) * 8 * C::QBLK; i += kThreads) {
    const int blk = i / ((kBM - tpt * G) * 8), j = i % ((kBM - tpt * G) * 8);
    *reinterpret_cast<uint4*>(sQ + blk * C::BLK_BYTES + tpt * G * 128 + j * 16) = make_uint4(0, 0, 0, 0);
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
  cluster_sync_all();  // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  const WaitCtl wc{p.status, &bars->abort, p.limit_ns};
  // Drains (after a normal run these return at once) ignore the abort flag.
  int drain_abort = 0;
  const WaitCtl wdrain{p.status, &drain_abort, 1000000000ull};

  const TileBoxes box(p);

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
        mbar_arrive_expect_tx(&bars->q_full, G * tpt * 128 * C::QBLK);
#pragma unroll
        for (int blk = 0; blk < C::QBLK; ++blk)
          tma_load_4d(sQ + blk * C::BLK_BYTES, &tq, &bars->q_full, blk * 64, static_cast<int>(rank), wk.t.hk * G,
                      wk.t.tok0);
      }
      ++gq;
      for (int j = 0; j < wk.take; ++j, ++gk) {
        const int st = gk & 1, key0 = (wk.unit + j) * kBN;
        const int boxes = box.count(key0, L), row = box.row(p, wk.t, key0, boxes, lane);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_empty[st], ((gk >> 1) & 1) ^ 1, wc)))) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[st], boxes * box.rows * 128 * C::QBLK);
        __syncwarp();
        if (lane < boxes) {
#pragma unroll
          for (int blk = 0; blk < C::QBLK; ++blk)
            tma_load_4d(sK + st * C::K_BYTES + blk * C::BLK_BYTES + lane * box.rows * 128, &tk, &bars->k_full[st],
                        blk * 64, 2 * wk.t.hk + static_cast<int>(rank), row, 0);
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
    for (int k = 0; ok; ++k) {
      const int L = min(wk.t.L, p.max_keys);
      // the previous segment's epilogue uses both V stages for its exchange
      if (k > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(&bars->epi_free, (k - 1) & 1, wc)))) break;
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
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer --
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, C::DV, false, true);
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK), sVa = smem_u32(sV);
      int gs = 0;  // S products issued
      int gp = 0;  // PV products issued
      // O (+)= P V for the next tile; `first` starts a new segment's O
      auto issue_pv = [&](bool first) -> bool {
        const int bb = gp & 1;
        const uint32_t ph = (gp >> 1) & 1;
        if (!mbar_wait(&bars->v_full[bb], ph, wc)) return false;
        if (!mbar_wait(&bars->p_full[bb], ph, wc)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk) {
          const uint32_t a_tmem = tmem + C::TM_P + 64 * bb + 8 * kk;
          const uint64_t bd = smem_desc_sw128(sVa + bb * C::V_BYTES + kk * 2048, C::BLK_BYTES, 1024);
          umma_ts(tmem + C::TM_O, a_tmem, bd, idesc_pv, (!first || kk > 0) ? 1u : 0u);
        }
        umma_commit(&bars->v_empty[bb]);
        umma_commit(&bars->p_empty[bb]);
        ++gp;
        return true;
      };
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!(ok = mbar_wait(&bars->q_full, k & 1, wc))) break;
        for (int j = 0; ok && j < wk.take; ++j, ++gs) {
          const int st = gs & 1;
          // S overwrites the previous S tile: every softmax warp must have read it
          if (gs > 0 && !(ok = mbar_wait(&bars->s_free, (gs - 1) & 1, wc))) break;
          if (!(ok = mbar_wait(&bars->k_full[st], (gs >> 1) & 1, wc))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // each instruction takes 32 bytes of every row
            const int blk = kk >> 2;
            const uint32_t koff = (kk & 3) * 32;
            const uint64_t ad = smem_desc_sw128(sQa + blk * C::BLK_BYTES + koff, 16, 1024);
            const uint64_t bd = smem_desc_sw128(sKa + st * C::K_BYTES + blk * C::BLK_BYTES + koff, 16, 1024);
            umma_ss(tmem + C::TM_S, ad, bd, idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bars->k_empty[st]);
          umma_commit(&bars->s_full);
          if (j == wk.take - 1) umma_commit(&bars->q_empty);  // the segment's S products are all issued
          if (j > 0) ok = issue_pv(j == 1);
        }
        if (ok) ok = issue_pv(wk.take == 1);
        if (!ok || !wk.next(pv, p)) break;
      }
      // drain: every issued MMA has completed before tensor memory is read or freed
      umma_commit(&bars->mma_done);
      mbar_wait(&bars->mma_done, 0, wdrain);
    }
    __syncwarp();
  } else if (warp == 3) {
    // --------------------------------------------------- output copy --
    // Per finished tile: once the softmax warps have staged it as bf16 (V
    // stage 1), copy its rows out and free both V stages for the next segment.
    const uint32_t tile = smem_u32(sV + C::V_BYTES);
    const int own0 = (rank == 0) ? 0 : C::HALF;
    int kt = 0;                    // tiles copied
    unsigned long long tiles = 2;  // of keys since the last one, and the epilogue's share
    do {
      tiles += wk.take;
      if (!wk.whole()) continue;
      // The keys before a tile may take longer than one wait may: each of their
      // tiles has the limit for itself, so this wait has it as often.
      const WaitCtl wt{p.status, &bars->abort, __umul64hi(p.limit_ns, tiles) ? ~0ull : p.limit_ns * tiles};
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->tile_full, kt & 1, wt))) break;
      ++kt;
      tiles = 2;
      const int rows = wk.t.ntok * G, chunk = lane & 7;
#pragma unroll
      for (int blk = 0; blk < C::HALF / 64; ++blk) {
#pragma unroll 4
        for (int r = lane >> 3; r < rows; r += 4) {
          uint32_t x[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(tile + blk * C::BLK_BYTES + r * 128 + ((chunk ^ (r & 7)) << 4))
                       : "memory");
          const size_t row = static_cast<size_t>(wk.t.tok0 + r / G) * H + wk.t.hk * G + r % G;
          *reinterpret_cast<uint4*>(p.o + row * C::DV + own0 + 64 * blk + 8 * chunk) =
              make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->epi_free);
    } while (wk.next(pv, p));
  }

  if (warp >= 4) {
    // ------------------------------------------------ softmax + epilogue --
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // query row within the tile (= TMEM lane)
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float coef2 = map2_coefficient(p.mode, *p.lambda);  // c in softmax(S1) + c softmax(S2)
    const float sc = kLog2e * rsqrtf(static_cast<float>(D));
    constexpr int HALF = C::HALF;
    constexpr int NC = HALF / 4;  // float4 chunks per exchanged row
    float* recv = reinterpret_cast<float*>(sV);                // V stage 0: the partner's half
    float* stage = reinterpret_cast<float*>(sV + C::V_BYTES);  // V stage 1: the half sent, then the output
    const uint32_t own0 = (rank == 0) ? 0 : HALF;   // columns this CTA finishes
    const uint32_t send0 = (rank == 0) ? HALF : 0;  // columns it hands to the partner
    int g = 0;   // S / P tiles consumed
    int ke = 0;  // segments combined
    bool sm_ok = true;
    do {
      const int L = min(wk.t.L, p.max_keys);
      const int lim = min(wk.t.lim0 + (causal ? r / G : 0), L - 1);  // last key that this row sees
      const bool live = r < wk.t.ntok * G;
      float m_run = -INFINITY, l_run = 0.f;
      // O and l *= alpha (the whole warp takes part; alpha = 1 leaves a row as it is)
      auto rescale_o = [&](float alpha) {
#pragma unroll
        for (int c = 0; c < C::DV / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32_sync(tl + C::TM_O + 32 * c, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
          tmem_st32(tl + C::TM_O + 32 * c, ov);
        }
        tmem_st_wait();
        l_run *= alpha;
      };
      const int g_end = g + wk.take;
      for (int j = 0; sm_ok && j < wk.take; ++j, ++g) {
        const int bb = g & 1;
        // every exit is taken by the whole warp (a wait may end differently in its lanes)
        if (!(sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full, g & 1, wc)))) break;
        // S_g has completed, and with it every MMA issued before it, PV_{g-2}
        // included: P buffer b is free.
        tc_fence_after();
        uint32_t su[128];
        tmem_ld128_sync(tl + C::TM_S, su);
        // S is in registers: the next S tile may overwrite the buffer
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free);
        float x[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) x[i] = __uint_as_float(su[i]);
        const int last = lim - (wk.unit + j) * kBN;  // last visible key of the tile
        if (last < kBN - 1) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i > last) x[i] = -INFINITY;
        }
        if (j == 0) {  // the first tile sets the reference maximum
          float mk[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mk[c] = x[c];
#pragma unroll
          for (int i = 8; i < 128; i += 8) {
#pragma unroll
            for (int c = 0; c < 8; ++c) mk[c] = fmaxf(mk[c], x[i + c]);
          }
          m_run = fmaxf(fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])), fmaxf(fmaxf(mk[4], mk[5]), fmaxf(mk[6], mk[7]))) * sc;
        }
        // P = exp2(s*c - m_run) into P[b], taken relative to the reference
        // maximum m_run as it stands; the tile's own maximum is formed
        // alongside.  A row without keys keeps the maximum -inf: all its P are 0.
        float lsum = 0.f, t_mx = -INFINITY;
        auto make_p = [&](bool with_max) {
          const float mneg = m_run == -INFINITY ? 0.f : -m_run;
          const F2 sc2(sc, sc), mneg2(mneg, mneg);
          F2 acc[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
          float mk[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mk[c] = -INFINITY;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float a0 = x[64 * half + 2 * i], a1 = x[64 * half + 2 * i + 1];
              if (with_max) mk[i & 3] = fmaxf(mk[i & 3], fmaxf(a0, a1));
              float p0, p1;
              fma2(F2(a0, a1), sc2, mneg2).get(p0, p1);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              acc[i & 1] = add2(acc[i & 1], F2(p0, p1));
              pk[i] = pack_bf16x2(p0, p1);
            }
            tmem_st32(tl + C::TM_P + 64 * bb + 32 * half, pk);
          }
          float l0, l1;
          add2(acc[0], acc[1]).get(l0, l1);
          lsum = l0 + l1;
          if (with_max) t_mx = fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])) * sc;
        };
        make_p(true);
        // A jump of the maximum by more than 2^64 would overflow P: rescale O
        // to the new maximum (after the previous tile's PV has completed) and redo P.
        const bool hard = j > 0 && t_mx > m_run + kOverflowGuard;
        if (__any_sync(0xffffffffu, hard)) {
          tmem_st_wait();
          if (!(sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->p_empty[(g - 1) & 1], ((g - 1) >> 1) & 1, wc))))
            break;
          tc_fence_after();
          rescale_o(hard ? fast_exp2(m_run - t_mx) : 1.0f);
          if (hard) m_run = t_mx;
          make_p(false);
        }
        tmem_st_wait();
        l_run += lsum;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[bb]);
        // Lazy rescale: keep the reference within 2^8 of the running maximum.
        // O is rescaled once this tile's PV (which used the old reference) has completed.
        const bool need = t_mx > m_run + kRescaleThreshold;
        if (__any_sync(0xffffffffu, need)) {
          if (!(sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->p_empty[bb], (g >> 1) & 1, wc)))) break;
          tc_fence_after();
          rescale_o(need ? fast_exp2(m_run - t_mx) : 1.0f);
          if (need) m_run = t_mx;
        }
      }
      g = g_end;  // the loop may stop early after an abort: keep the tile count in step

      // ------------------------------------------------------ epilogue --
      // O is complete once the segment's last PV (and with it every earlier MMA) has.
      // (A vote, as at every wait: its lanes may see it end differently after an abort.)
      if (sm_ok) sm_ok = __all_sync(0xffffffffu, mbar_wait(&bars->p_empty[(g - 1) & 1], ((g - 1) >> 1) & 1, wc));
      tc_fence_after();
      // After an abort nothing is exchanged, recorded or handed over any more:
      // the four warps leave the walk together, and warp 3 by itself.
      if (named_bar_or(1, 128, !sm_ok || bars->abort)) break;
      if (!wk.whole()) {
        // a part of the row's keys: this map's sums to the worker's record
        float* rec = p.recs + (2 * (blockIdx.x >> 1) + (wk.begins() ? 1 : 0)) * record_floats(kBM, D);
        float* orow = rec + 4 * kBM + static_cast<size_t>(r) * 2 * C::DV + rank * C::DV;
#pragma unroll 1
        for (int c = 0; c < C::DV / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32_sync(tl + C::TM_O + 32 * c, ov);
          if (live) {
#pragma unroll
            for (int f = 0; f < 8; ++f)
              *reinterpret_cast<uint4*>(orow + 32 * c + 4 * f) =
                  make_uint4(ov[4 * f + 0], ov[4 * f + 1], ov[4 * f + 2], ov[4 * f + 3]);
          }
        }
        if (live) *reinterpret_cast<float2*>(rec + 4 * r + 2 * rank) = make_float2(m_run, l_run);
        tc_fence_before();
        named_bar_sync(1, 128);  // every row's tensor-memory reads are done
        if (tid == 128) mbar_arrive(&bars->epi_free);  // the next segment's first PV may overwrite O
        __syncwarp();
        continue;
      }
      // Both V stages are free of this segment's PV products: announce that
      // this CTA's receive buffer is ready, with the exchange barrier armed first.
      if (tid == 128) {
        mbar_arrive_expect_tx(&bars->exch_full, C::EXCH_BYTES);
        mbar_arrive_expect_tx(&bars->ss_full, kBM * 4);  // the partner's sums of squares, by st.async
        mbar_arrive_remote(map_to_cta(smem_u32(&bars->peer_ready), partner));
      }
      const float inv = l_run > 0.f ? ((rank == 0) ? 1.0f / l_run : coef2 / l_run) : 0.f;
      float* srow = stage + r * HALF;
#pragma unroll
      for (int c = 0; c < HALF / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32_sync(tl + C::TM_O + send0 + 32 * c, ov);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          const int chunk = (c * 8 + f) ^ (r % NC);
          *reinterpret_cast<float4*>(srow + chunk * 4) =
              make_float4(__uint_as_float(ov[4 * f + 0]) * inv, __uint_as_float(ov[4 * f + 1]) * inv,
                          __uint_as_float(ov[4 * f + 2]) * inv, __uint_as_float(ov[4 * f + 3]) * inv);
        }
      }
      fence_proxy_async_smem();  // the staged rows are read by the bulk copy (async proxy)
      __syncwarp();
      // the partner's receive buffer must be free before this CTA writes into it
      const bool peer_ok = __all_sync(0xffffffffu, mbar_wait_acq_cluster(&bars->peer_ready, ke & 1, wc));
      if (lane == 0 && peer_ok) {
        const int off = quarter * 32 * HALF;  // this warp's 32 rows, contiguous
        bulk_copy_s2cluster(map_to_cta(smem_u32(recv + off), partner), stage + off, 32 * HALF * 4,
                            map_to_cta(smem_u32(&bars->exch_full), partner));
        bulk_commit_group();
      }
      // the partner's half has landed (waited for even after an abort: a copy may be on its way)
      const bool got_half = mbar_wait(&bars->exch_full, ke & 1, wdrain);
      float y[HALF];
      float ss = 0.f;
      const float* rrow = recv + r * HALF;
#pragma unroll
      for (int c = 0; c < HALF / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32_sync(tl + C::TM_O + own0 + 32 * c, ov);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          const int chunk = (c * 8 + f) ^ (r % NC);
          const float4 xr = *reinterpret_cast<const float4*>(rrow + chunk * 4);
          const float xs[4] = {xr.x, xr.y, xr.z, xr.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float val = fmaf(__uint_as_float(ov[4 * f + e]), inv, xs[e]);
            y[32 * c + 4 * f + e] = val;
            ss = fmaf(val, val, ss);
          }
        }
      }
      // this row's half of the sum of squares to the partner: an asynchronous
      // store that completes on the partner's barrier (armed before its
      // receive buffer was announced)
      if (peer_ok)
        st_async_f32(map_to_cta(smem_u32(ssx + r), partner), ss, map_to_cta(smem_u32(&bars->ss_full), partner));
      if (lane == 0 && peer_ok) bulk_wait_group_read0();  // the outgoing copy has left the staging rows
      __syncwarp();
      named_bar_sync(1, 128);  // every warp's outgoing copy is done with the rows the output tile reuses
      // a partner that is gone sends nothing: this CTA leaves at the next vote, before its barriers are armed again
      if (!mbar_wait_acq_cluster(&bars->ss_full, ke & 1, wdrain) || !got_half) bars->abort = 1;
      const float gsc = norm_factor((ss + ssx[r]) / static_cast<float>(C::DV), p.eps, p.lambda_init);
      // bf16 tile [64-column block][128 rows][64 columns], 128-byte swizzle, in the staging stage
      const uint32_t sout = smem_u32(stage);
#pragma unroll
      for (int c8 = 0; c8 < HALF / 8; ++c8) {
        uint32_t w4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 8 * c8 + 2 * e;
          w4[e] = pack_bf16x2(y[c] * gsc * __ldg(p.rms_w + own0 + c), y[c + 1] * gsc * __ldg(p.rms_w + own0 + c + 1));
        }
        const uint32_t a = sout + (c8 / 8) * C::BLK_BYTES + r * 128 + (((c8 % 8) ^ (r & 7)) << 4);
        st_shared_v4(a, w4[0], w4[1], w4[2], w4[3]);
      }
      ++ke;
      // hand the staged tile to warp 3, which copies it out and frees the V
      // stages, and go on with the next segment.  (An mbarrier, which waits with
      // a limit and counts an arrival a phase: on a named barrier, warps that
      // went through aborted segments could arrive twice before warp 3 did once,
      // complete the barrier without it and leave it waiting for good.)
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->tile_full);
    } while (wk.next(pv, p));
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no remote access to either CTA remains
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

}  // namespace

WideParams wide_params(const ExtendArgs& a, float* recs, DevCtl ctl) {
  WideParams p = {};
  p.plan = a.plan;
  p.n = a.n;
  p.block_table = a.block_table;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
  p.max_keys = keys_of_table(a.max_pages, a.page_size);
  p.most = unit_limits(a.n, p.max_keys);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.recs = recs;
  p.lambda = a.lambda;
  p.lambda_init = a.lambda_init;
  p.rms_w = a.rms_w;
  p.eps = a.eps;
  p.mode = a.mode;
  p.status = ctl.status;
  p.limit_ns = ctl.limit_ns;
  return p;
}

cudaError_t launch_extend_wide128(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream) {
  static unsigned long long set_ctx[64] = {};
  if (ctl.dev < 0 || ctl.dev >= 64) return cudaErrorInvalidDevice;
  if (ctl.ctx == 0 || set_ctx[ctl.dev] != ctl.ctx) {
    const auto fn = extend_wide_kernel;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(fn, cudaFuncAttributeRequiredClusterWidth, 2)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(fn, cudaFuncAttributeRequiredClusterHeight, 1)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(fn, cudaFuncAttributeRequiredClusterDepth, 1)) != cudaSuccess)
      return e;
    set_ctx[ctl.dev] = ctl.ctx;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * wide_workers(D), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, extend_wide_kernel, a.tq, a.tk, a.tv, wide_params(a, recs, ctl));
}

}  // namespace diffattn
