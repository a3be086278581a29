// What the two kernels for many query rows share (extend_wide.cu: d = 128,
// extend_wide64.cu: d = 64): their parameters, a worker's walk over its
// segments, and the boxes that bring a tile of keys from its pages.
#pragma once

#include <math.h>

#include "common.cuh"
#include "extend.cuh"

namespace diffattn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kOverflowGuard = 64.0f;    // log2 units

struct WideParams {
  const void* plan;
  ExtendShape n;
  const int* block_table;
  int max_pages, num_pages, page_shift, max_keys;
  __nv_bfloat16* o;
  float* recs;
  const float* lambda;
  float lambda_init;
  const float* rms_w;
  float eps;
  int mode;
  int* status;
  unsigned long long limit_ns;
};

// A worker's walk over its segments: units unit .. unit + take - 1 of (row tile at, key head hk).
struct Walk {
  WideTile t;
  int at, hk, unit, take, left;
  __device__ void open(const WideTile* list) {
    t = list[at];
    take = min(left, t.units - unit);
  }
  __device__ bool next(const WideTile* list, int H_kv) {  // false: the range is done
    left -= take;
    if (left <= 0) return false;
    unit = 0;
    if (++at == t.first + t.count) {
      if (++hk < H_kv) {
        at = t.first;
      } else {
        hk = 0;
      }
    }
    open(list);
    return true;
  }
  __device__ bool begins() const { return unit == 0; }
  __device__ bool whole() const { return unit == 0 && take == t.units; }
};

// Rows of a page's box, boxes of a tile, and (in lane b of a warp) the first
// row of box b of the tile at key0: outside the tensor for a page out of range.
struct TileBoxes {
  int rows, shift;
  __device__ explicit TileBoxes(const WideParams& p) : rows(min(1 << p.page_shift, kUnit)), shift(min(p.page_shift, 7)) {}
  __device__ int count(int key0, int L) const { return L <= key0 ? 0 : (min(kUnit, L - key0) + rows - 1) >> shift; }
  __device__ int row(const WideParams& p, const WideTile& t, int key0, int boxes, int lane) const {
    if (lane >= boxes) return 0;
    const int key = key0 + (lane << shift);
    const int page = p.block_table[static_cast<size_t>(t.s) * p.max_pages + (key >> p.page_shift)];
    if (page < 0 || page >= p.num_pages) {
      atomicCAS(p.status, 0, 6);
      return -kUnit;
    }
    return (page << p.page_shift) + (key & ((1 << p.page_shift) - 1));
  }
};

// Zeros over the rows of a V tile ([64-channel block][128 rows][128 bytes])
// behind its live ones, by one warp; the product reads them through the async proxy.
__device__ __forceinline__ void clear_v_rows(uint8_t* tile, int blocks, int live, int lane) {
  const int chunks = (kUnit - live) * 8;  // 16-byte chunks to clear in a block
  for (int i = lane; i < chunks * blocks; i += 32)
    *reinterpret_cast<uint4*>(tile + (i / chunks) * (kUnit * 128) + live * 128 + (i % chunks) * 16) =
        make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

WideParams wide_params(const ExtendArgs& a, float* recs, DevCtl ctl);
cudaError_t launch_extend_wide128(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream);
cudaError_t launch_extend_wide64(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream);

}  // namespace diffattn
