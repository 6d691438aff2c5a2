// Row plan: rows grouped by an id (a request's adapter, a routed expert), in order.
//
// A stable counting sort.  Each workgroup owns a contiguous run of rows and each of its waves
// a contiguous part of it; waves count their ids in LDS, counts are prefixed over ids,
// workgroups and waves, and every wave then places its rows 64 at a time: lanes with the same
// id find each other by comparing the id's bits with ballots, a lane's rank is the number of
// such lanes below it.  Nothing depends on the order of atomics (they only count), so the
// result is the one stable order.
//
// Up to RP_ONE rows take one workgroup and one launch; more take a counting launch first,
// whose per-workgroup counts every workgroup of the second launch sums for itself (at most
// RP_MAX_WG rows of counts, read from L2).  Bounded by launch and LDS latency, not by bytes.
#include "qf_kernels.h"

namespace qf {

constexpr int RP_WAVES = 8, RP_WG = RP_WAVES * 64;
constexpr int RP_IDS = QF_ROW_MAX_IDS;
static_assert(RP_IDS == 2 * RP_WG, "the prefix sum handles two ids per thread");

// Rows per workgroup and workgroups of a plan of n rows.
int row_plan_wgs(int64_t n, int64_t* rows_per_wg) {
  int64_t per = RP_ONE;
  if (n > RP_ONE) {
    per = (n + RP_MAX_WG - 1) / RP_MAX_WG;
    per = (per + RP_WG - 1) / RP_WG * RP_WG;
    if (per < RP_MIN_PER_WG) per = RP_MIN_PER_WG;
  }
  *rows_per_wg = per;
  return n > 0 ? (int)((n + per - 1) / per) : 1;
}

__device__ __forceinline__ void rp_count(const int32_t* ids, int64_t lo, int64_t hi, uint32_t n_ids, uint32_t* cnt) {
  for (int64_t i = lo + (threadIdx.x & 63); i < hi; i += 64) {
    const uint32_t id = (uint32_t)ids[i];
    if (id < n_ids) atomicAdd(&cnt[id], 1u);
  }
}

__global__ __launch_bounds__(RP_WG) void k_row_hist(const int32_t* __restrict__ ids, int64_t n, int64_t per,
                                                    uint32_t n_ids, uint32_t* __restrict__ hist) {
  __shared__ uint32_t cnt[RP_IDS];
  for (uint32_t i = threadIdx.x; i < n_ids; i += RP_WG) cnt[i] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * per, hi = lo + per < n ? lo + per : n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += RP_WG) {
    const uint32_t id = (uint32_t)ids[i];
    if (id < n_ids) atomicAdd(&cnt[id], 1u);
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < n_ids; i += RP_WG) hist[(int64_t)blockIdx.x * n_ids + i] = cnt[i];
}

// Exclusive prefix sums of two values per id, ids 2 * thread and 2 * thread + 1.
__device__ __forceinline__ uint2 rp_scan(uint32_t a, uint32_t b, uint2* wave_sum) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = a, y = b;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t u = __shfl_up(x, d), v = __shfl_up(y, d);
    if (lane >= (uint32_t)d) {
      x += u;
      y += v;
    }
  }
  if (lane == 63) wave_sum[wave] = uint2{x, y};
  __syncthreads();
  uint2 base = {x - a, y - b};
  for (uint32_t w = 0; w < wave; ++w) {
    base.x += wave_sum[w].x;
    base.y += wave_sum[w].y;
  }
  return base;
}

__global__ __launch_bounds__(RP_WG) void k_row_plan(RowPlanArgs a) {
  __shared__ uint32_t cnt[RP_WAVES][RP_IDS];       // counts, then the next position, per wave and id
  __shared__ uint32_t off[RP_IDS + 1], toff[RP_IDS + 1];
  __shared__ uint2 wave_sum[RP_WAVES];
  const uint32_t n_ids = (uint32_t)a.n_ids, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t i = threadIdx.x; i < n_ids * RP_WAVES; i += RP_WG) cnt[i / n_ids][i % n_ids] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * a.per, hi = lo + a.per < a.n ? lo + a.per : a.n;
  const int64_t part = a.per / RP_WAVES, wlo = lo + wave * part;      // per is a multiple of 8 x 64
  const int64_t whi = wlo + part < hi ? wlo + part : hi;
  rp_count(a.ids, wlo, whi, n_ids, cnt[wave]);
  __syncthreads();

  uint32_t before[2] = {0, 0}, total[2] = {0, 0}, tiles[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t id = threadIdx.x * 2 + j;
    if (id < n_ids) {
      if (gridDim.x == 1) {
        for (int w = 0; w < RP_WAVES; ++w) total[j] += cnt[w][id];
      } else {
#pragma unroll 8
        for (uint32_t b = 0; b < gridDim.x; ++b) {
          const uint32_t h = a.hist[(int64_t)b * n_ids + id];
          total[j] += h;
          if (b < blockIdx.x) before[j] += h;
        }
      }
    }
    tiles[j] = (total[j] + QF_ROW_TILE - 1) / QF_ROW_TILE;
  }
  const uint2 base = rp_scan(total[0] + total[1], tiles[0] + tiles[1], wave_sum);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t id = threadIdx.x * 2 + j;
    if (id < n_ids) {
      const uint32_t o = base.x + (j ? total[0] : 0), t = base.y + (j ? tiles[0] : 0);
      off[id] = o;
      toff[id] = t;
      if (id == n_ids - 1) {
        off[n_ids] = o + total[j];
        toff[n_ids] = t + tiles[j];
      }
      uint32_t next = o + before[j];
      for (int w = 0; w < RP_WAVES; ++w) {
        const uint32_t c = cnt[w][id];
        cnt[w][id] = next;
        next += c;
      }
    }
  }
  __syncthreads();

  // place the rows: a wave's own counters, so no other wave's work is waited for
  int bits = 0;
  while ((1u << bits) < n_ids) ++bits;
  for (int64_t i0 = wlo; i0 < whi; i0 += 64) {
    const int64_t i = i0 + lane;
    const uint32_t id = i < whi ? (uint32_t)a.ids[i] : 0xFFFFFFFFu;
    const bool in = id < n_ids;
    uint64_t peers = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((id >> b) & 1u);
      peers &= ((id >> b) & 1u) ? set : ~set;
    }
    const uint32_t rank = __popcll(peers & ((1ull << lane) - 1ull));
    uint32_t at = 0;
    if (in && rank == 0) at = atomicAdd(&cnt[wave][id], (uint32_t)__popcll(peers));
    at = __shfl(at, in ? __ffsll((unsigned long long)peers) - 1 : 0) + rank;
    if (in) a.order[at] = (int32_t)i;
  }

  // the rest, spread over the grid: offsets, the tile table, the unused end of order
  const int64_t tid = (int64_t)blockIdx.x * RP_WG + threadIdx.x, step = (int64_t)gridDim.x * RP_WG;
  for (int64_t i = tid; i <= n_ids; i += step) a.offsets[i] = (int32_t)off[i];
  for (int64_t i = off[n_ids] + tid; i < a.n; i += step) a.order[i] = -1;
  const uint32_t used = toff[n_ids];
  for (int64_t t = tid; t < a.n_tiles; t += step) {
    int32_t e = -1, first = 0;
    if (t < used) {
      uint32_t l = 0, r = n_ids;                    // last id whose first tile is at or before t
      while (r - l > 1) {
        const uint32_t m = (l + r) / 2;
        if (toff[m] <= t) l = m; else r = m;
      }
      e = (int32_t)l;
      first = (int32_t)(off[l] + QF_ROW_TILE * ((uint32_t)t - toff[l]));
    }
    reinterpret_cast<int2*>(a.tiles)[t] = int2{e, first};
  }
}

hipError_t launch_row_plan(RowPlanArgs a, hipStream_t s) {
  int64_t per;
  const int wgs = row_plan_wgs(a.n, &per);
  a.per = per;
  if (wgs > 1) {
    k_row_hist<<<wgs, RP_WG, 0, s>>>(a.ids, a.n, per, (uint32_t)a.n_ids, a.hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_row_plan<<<wgs, RP_WG, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace qf

extern "C" {

int64_t qf_row_plan_tiles(int64_t n, int n_ids) {
  if (n < 0 || n >= QF_ROW_MAX_ROWS || n_ids < 1 || n_ids > QF_ROW_MAX_IDS) return 0;
  return (n + QF_ROW_TILE - 1) / QF_ROW_TILE + (n < n_ids ? n : n_ids);
}

size_t qf_row_plan_workspace(int64_t n, int n_ids) {
  if (n < 0 || n >= QF_ROW_MAX_ROWS || n_ids < 1 || n_ids > QF_ROW_MAX_IDS) return 0;
  int64_t per;
  const int wgs = qf::row_plan_wgs(n, &per);
  return wgs > 1 ? (size_t)wgs * n_ids * 4 : 0;
}

qf_status qf_row_plan(const int32_t* ids, int64_t n, int n_ids, int32_t* offsets, int32_t* order, int32_t* tiles,
                      void* ws, size_t ws_bytes, void* stream) {
  if (n < 0 || n >= QF_ROW_MAX_ROWS) return QF_ERR_SHAPE;
  if (n_ids < 1 || n_ids > QF_ROW_MAX_IDS) return QF_ERR_ARG;
  if (!offsets || (n > 0 && (!ids || !order || !tiles))) return QF_ERR_NULL;
  if (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)order | (uintptr_t)ws) % 4 || (uintptr_t)tiles % 8)
    return QF_ERR_ALIGN;
  const size_t need = qf_row_plan_workspace(n, n_ids);
  if (need > 0 && (!ws || ws_bytes < need)) return QF_ERR_WORKSPACE;
  qf::RowPlanArgs a;
  a.ids = ids;
  a.n = n;
  a.per = 0;
  a.n_ids = n_ids;
  a.offsets = offsets;
  a.order = order;
  a.tiles = tiles;
  a.n_tiles = qf_row_plan_tiles(n, n_ids);
  a.hist = (uint32_t*)ws;
  return qf::status_of(qf::launch_row_plan(a, (hipStream_t)stream));
}

}  // extern "C"
