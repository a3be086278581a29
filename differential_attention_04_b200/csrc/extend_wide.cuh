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
  UnitLimits most;
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

// Two float32 in one register pair: Blackwell's packed instructions take the
// pair in one issue slot.
struct F2 {
  uint64_t v;
  __device__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 fma2(F2 a, const F2& b, const F2& c) {
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.v) : "l"(b.v), "l"(c.v));
  return a;
}
__device__ __forceinline__ F2 add2(F2 a, const F2& b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
  return a;
}

// A worker's walk over its segments: units unit .. unit + take - 1 of an item,
// first its whole items (every workers-th up to `whole_end`), then its range of
// the line.
struct Walk {
  WideItem t;
  int at, unit, take, left;  // left: units of the range from this segment on
  int worker, workers, whole_end;
  __device__ WideItem item(const PlanView& pv, const WideParams& p) const { return wide_at(pv.wide, at, p.n, p.status); }
  __device__ bool begin(const PlanView& pv, int w, const WideParams& p) {  // false: there is no work
    worker = w;
    workers = pv.head->workers[1];
    whole_end = pv.head->rounds * workers;
    left = pv.starts[w].count;
    if (!DA_CHECK(p.status, left <= pv.head->units[1] * p.n.H_kv)) left = 0;
    if (w >= workers || whole_end == 0) return open_range(pv, p);
    at = w;
    open_whole(pv, p);
    return true;
  }
  __device__ void open_whole(const PlanView& pv, const WideParams& p) {
    t = item(pv, p);
    unit = 0;
    take = t.units;
  }
  __device__ bool open_range(const PlanView& pv, const WideParams& p) {
    whole_end = 0;
    if (left <= 0) return false;
    const WorkStart st = pv.starts[worker];
    at = st.at;
    unit = st.unit;
    t = item(pv, p);
    if (!DA_CHECK(p.status, unit >= 0 && unit < t.units)) return false;
    take = min(left, t.units - unit);
    return true;
  }
  __device__ bool next(const PlanView& pv, const WideParams& p) {  // false: that was the last segment
    if (whole_end) {
      at += workers;
      if (at >= whole_end) return open_range(pv, p);
      open_whole(pv, p);
      return true;
    }
    left -= take;
    if (left <= 0) return false;
    ++at;
    t = item(pv, p);
    unit = 0;
    take = min(left, t.units);
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
  __device__ int row(const WideParams& p, const WideItem& t, int key0, int boxes, int lane) const {
    if (lane >= boxes) return 0;
    const int key = key0 + (lane << shift);
    if (!DA_CHECK(p.status, (key >> p.page_shift) < p.max_pages)) return -kUnit;
    const int page = p.block_table[static_cast<size_t>(t.s) * p.max_pages + (key >> p.page_shift)];
    if (page < 0 || page >= p.num_pages) {
      atomicCAS(p.status, 0, 6);
      return -kUnit;
    }
    return (page << p.page_shift) + (key & ((1 << p.page_shift) - 1));
  }
};

// Barrier over `count` threads that tells all of them whether any brought `x`.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t count, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(id), "r"(count), "r"(x ? 1u : 0u)
      : "memory");
  return y != 0;
}

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

// 32 lanes x 64 consecutive columns, waited for: loads and wait are one
// statement, so that no register can be moved or spilled before its value is there.
__device__ __forceinline__ void tmem_ld64_sync(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
}

// 32 lanes x 128 consecutive columns, waited for: loads and wait are one
// statement, so that no register can be moved or spilled before its value is there.
__device__ __forceinline__ void tmem_ld128_sync(uint32_t taddr, uint32_t (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
        "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
        "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
        "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
        "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
        "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
        "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
        "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
        "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(taddr), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
      : "memory");
}

WideParams wide_params(const ExtendArgs& a, float* recs, DevCtl ctl);
cudaError_t launch_extend_wide128(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream);
cudaError_t launch_extend_wide64(const ExtendArgs& a, float* recs, DevCtl ctl, cudaStream_t stream);

}  // namespace diffattn
