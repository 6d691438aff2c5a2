// What the 8-bit operators share: E4M3 blocks of 128 with an fp32 scale, and the place of a unit of
// rows among the groups of a row plan.
#pragma once
#include "qf_device.h"
#include "qf_kernels.h"

#include <type_traits>

namespace qf {

constexpr int FB = QF_FP8_BLOCK;
constexpr float F8_TOP = 448.0f;                  // largest E4M3 value
constexpr float F8_LIVE = 0x1p-100f;              // blocks below are all zero: 448 / amax must stay finite

// Scale of a block whose largest magnitude has the fp32 bits `top`, and the factor of its codes.
// A block with a NaN or an infinity gets a NaN scale, which whatever reads the block then is.
struct F8Scale {
  float scale, inv;
};
__device__ __forceinline__ F8Scale f8_scale(uint32_t top) {
  const float a = __uint_as_float(top);
  const bool live = a >= F8_LIVE;
  F8Scale o = {live ? a / F8_TOP : 0.0f, live ? F8_TOP / a : 0.0f};
  if (top >= 0x7F800000u) o.scale = __uint_as_float(0x7FC00000u);
  return o;
}

// Four codes of y[0..3] (already times inv, so at most a rounding past 448, which rounds back to it):
// v_cvt_pk_fp8_f32, to nearest even.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return (uint32_t)v;
}

// Unit `u` of the groups' rows, each group cut into units of `unit` rows from its own first row:
// the group (-1: there are fewer units), the unit's first position, its rows, its index in the group.
struct GroupUnit {
  int group, first, rows, index;
};

// The sum of v over the lanes below this one, and over all.
__device__ __forceinline__ uint32_t wave_before(uint32_t v, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    if (lane >= (uint32_t)d) x += y;
  }
  *total = __shfl(x, 63);
  return x - v;
}
// Offset i of the plan, inside [0, n].
__device__ __forceinline__ int group_offset(const int32_t* offsets, int i, int n) {
  const int v = offsets[i];
  return v < 0 ? 0 : v > n ? n : v;
}
__device__ __forceinline__ uint32_t units_of(int lo, int hi, int unit) {
  return hi > lo ? (uint32_t)(hi - lo + unit - 1) / (uint32_t)unit : 0u;
}
// Called by whole waves; every wave finds it for itself.  Up to 64 groups a pass; more take a first
// pass over runs of groups.
__device__ __forceinline__ GroupUnit find_unit(const int32_t* offsets, int n_ids, int n, int unit, uint32_t u) {
  const int lane = threadIdx.x & 63;
  const int per = (n_ids + 63) / 64;             // groups per lane, 1..16
  int g0 = 0;                                    // first group of the run that holds the unit
  uint32_t total, left = u;
  if (per > 1) {
    uint32_t mine = 0;
    int lo = group_offset(offsets, min(lane * per, n_ids), n);
    for (int j = 0; j < per; ++j) {
      const int hi = group_offset(offsets, min(lane * per + j + 1, n_ids), n);
      mine += units_of(lo, hi, unit);
      lo = hi;
    }
    const uint32_t before = wave_before(mine, &total);
    const uint64_t hit = __ballot(u >= before && u - before < mine);
    if (!hit) return GroupUnit{-1, 0, 0, 0};
    const int at = __ffsll((unsigned long long)hit) - 1;
    g0 = at * per;
    left = u - (uint32_t)__builtin_amdgcn_readlane((int)before, at);
  }
  const int g = g0 + lane;
  const bool in = lane < per * (per > 1 ? 1 : 64) && g < n_ids;
  const int lo = in ? group_offset(offsets, g, n) : 0, hi = in ? group_offset(offsets, g + 1, n) : 0;
  const uint32_t mine = units_of(lo, hi, unit);
  const uint32_t before = wave_before(mine, &total);
  const uint64_t hit = __ballot(left >= before && left - before < mine);
  if (!hit) return GroupUnit{-1, 0, 0, 0};
  const int at = __ffsll((unsigned long long)hit) - 1;
  const int index = (int)(left - (uint32_t)__builtin_amdgcn_readlane((int)before, at));
  const int first = __builtin_amdgcn_readlane(lo, at) + index * unit;
  const int last = __builtin_amdgcn_readlane(hi, at);
  return GroupUnit{g0 + at, first, min(unit, last - first), index};
}
// The same for workgroups that ask for many units: the groups' offsets and unit counts stay in LDS.
struct GroupTable {
  int32_t off[QF_ROW_MAX_IDS + 1];      // the plan's offsets
  uint32_t pre[QF_ROW_MAX_IDS + 1];     // units of the groups before
  uint32_t sums[16];                    // of each wave, while the table is built
};
// Fills the table with the whole workgroup (of `waves` waves, at least four).
__device__ __forceinline__ void group_table(GroupTable& t, const int32_t* offsets, int n_ids, int n, int unit, int waves) {
  const int threads = waves * 64, per = (n_ids + threads - 1) / threads, g0 = (int)threadIdx.x * per;
  uint32_t mine[4] = {0, 0, 0, 0}, sum = 0, total;
  int lo = group_offset(offsets, min(g0, n_ids), n);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < per && g0 + j < n_ids) {
      const int hi = group_offset(offsets, g0 + j + 1, n);
      t.off[g0 + j] = lo;
      if (g0 + j + 1 == n_ids) t.off[n_ids] = hi;
      mine[j] = units_of(lo, hi, unit);
      sum += mine[j];
      lo = hi;
    }
  uint32_t before = wave_before(sum, &total);
  if ((threadIdx.x & 63) == 0) t.sums[threadIdx.x >> 6] = total;
  __syncthreads();
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) before += t.sums[w];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < per && g0 + j < n_ids) {
      t.pre[g0 + j] = before;
      before += mine[j];
      if (g0 + j + 1 == n_ids) t.pre[n_ids] = before;
    }
  __syncthreads();
}
__device__ __forceinline__ GroupUnit unit_at(const GroupTable& t, int n_ids, int unit, uint32_t u) {
  const int lane = threadIdx.x & 63, per = (n_ids + 63) / 64;
  int g = 0;
  if (per > 1) {                                     // runs of groups first
    const uint64_t upto = __ballot(t.pre[min(lane * per, n_ids)] <= u && lane * per < n_ids);
    g = (63 - __clzll((unsigned long long)upto)) * per;
  }
  // the last group of the run that begins at or before u, empty ones behind it left out
  const bool in = (per == 1 || lane < per) && g + lane < n_ids;
  const uint32_t lo = in ? t.pre[g + lane] : 0, hi = in ? t.pre[g + lane + 1] : 0;
  const uint64_t hit = __ballot(lo <= u && u < hi);
  if (!hit) return GroupUnit{-1, 0, 0, 0};
  const int at = __ffsll((unsigned long long)hit) - 1;
  const int index = (int)(u - (uint32_t)__builtin_amdgcn_readlane((int)lo, at));
  g += at;
  const int first = __builtin_amdgcn_readfirstlane(t.off[g]) + index * unit;
  return GroupUnit{g, first, min(unit, __builtin_amdgcn_readfirstlane(t.off[g + 1]) - first), index};
}

// 16 bytes, past the caches (NT) where they will not be read from there again.
template <bool NT>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  u32x4_t* q = (u32x4_t*)p;
  if constexpr (NT) __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), q);
  else *q = __builtin_bit_cast(u32x4_t, v);
}
__device__ __forceinline__ uint4 load16(const void* p) { return *(const uint4*)p; }
__device__ __forceinline__ uint4 load16_nt(const void* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4_t*)p));
}
// Outputs of this many bytes and more are stored past the caches: the 256 MiB behind the L2s hold what comes
// after them better.  Codes and sums of rows, through the caches / past them: 8192 x 4096 codes to 4 experts each (134 MB)
// 39.2 / 37.9 us, half of that 20.6 / 18.8, 16.8 MB 9.3 / 9.3; panels of 134 MB 77.5 / 63.3, of 67 MB 34.0 / 32.9, of
// 17 MB 13 / 10.3 but 118 / 123 with the product that reads them.
constexpr int64_t NT_BYTES = 64 << 20;
// bf16 rows are larger and the next kernel reads them, so they stay in the caches as long as they fit.  The rows'
// gradients of a mixture with their quantization: called over and over 97 / 115 us at 134 MB, 132 / 146 at 196, 166 / 168
// at 229, 226 / 206 at 268; after other work 123 / 146, 156 / 197, 182 / 217, 224 / 253.  A captured step of a mixture,
// forward and backward, with rows of 67, 98, 134 and 537 MB: 1.175 / 1.189, 1.505 / 1.518, 2.03 / 2.03 and, all sides past the
// caches at this size, 6.77 ms against 6.80 with none.
constexpr int64_t NT_ROWS_BYTES = 224 << 20;
// Calls f(std::true_type) or f(std::false_type).
template <typename F>
void with_nt(bool nt, F f) {
  if (nt) f(std::integral_constant<bool, true>());
  else f(std::integral_constant<bool, false>());
}

// Positions that a row is written to by one set of lanes; a row with more is read again.
constexpr uint32_t SPREAD_MOST = 16;

inline bool misaligned(const void* p, size_t a) { return (uintptr_t)p % a != 0; }
inline bool plan_sizes_ok(int64_t n, int n_ids) { return n >= 0 && n < QF_ROW_MAX_ROWS && n_ids >= 1 && n_ids <= QF_ROW_MAX_IDS; }

}  // namespace qf
