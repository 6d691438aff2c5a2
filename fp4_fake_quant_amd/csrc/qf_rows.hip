// Row plan: rows grouped by an id (a request's adapter, a routed expert), in order.
//
// A stable counting sort.  Each workgroup owns a contiguous run of rows and each of its waves
// a contiguous part of it; waves count their ids in LDS, counts are prefixed over ids,
// workgroups and waves, and every wave then places its rows 64 at a time: lanes with the same
// id find each other by comparing the id's bits with ballots, a lane's rank is the number of
// such lanes below it.  Nothing depends on the order of atomics (they only count), so the
// result is the one stable order.
//
// Up to RP_ONE_LAUNCH rows every workgroup counts all rows for itself (one launch; reading 4 n
// bytes from L2 is shorter than a second launch); more take a counting launch first, whose
// per-workgroup counts every workgroup of the second launch sums.  Bounded by launch, load and
// LDS latency, not by bytes: 61 rows of 40 ids take 4.0 us, 16384 rows 11, 262144 rows of 256 ids
// (2 MB) 3.5 + 10.2 in the two launches.
#include "qf_operators.h"

namespace qf {

constexpr int RP_WAVES = 8, RP_WG = RP_WAVES * 64;
constexpr int RP_IDS = QF_ROW_MAX_IDS;
constexpr int RP_HELD = 4;                 // ids per lane kept in registers between counting and placing
static_assert(RP_IDS == 2 * RP_WG, "the prefix sum handles two ids per thread");

// Rows per workgroup and workgroups of a plan of n rows.
int row_plan_wgs(int64_t n, int64_t* rows_per_wg) {
  int64_t per = (n + RP_MAX_WG - 1) / RP_MAX_WG;
  per = (per + RP_WG - 1) / RP_WG * RP_WG;
  if (per < RP_MIN_PER_WG) per = RP_MIN_PER_WG;
  *rows_per_wg = per;
  return n > 0 ? (int)((n + per - 1) / per) : 1;
}
// Row length of the counts: even, so that two ids load together.
__host__ __device__ inline uint32_t rp_pitch(uint32_t n_ids) { return (n_ids + 1) & ~1u; }

// The lanes of the wave with a valid id, and whether they all have the same one.
struct RpWave {
  uint64_t in;
  bool one;
};
__device__ __forceinline__ RpWave rp_wave(uint32_t id, uint32_t n_ids) {
  RpWave o;
  o.in = __ballot(id < n_ids);
  const int lane = o.in ? __ffsll((unsigned long long)o.in) - 1 : 0;
  const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)id, lane);
  o.one = __ballot(id < n_ids && id != first) == 0;
  return o;
}

// Counts one id per lane (called by whole waves); a wave with a single id adds once, where 64
// additions to one word would queue up.
__device__ __forceinline__ void rp_add(uint32_t* cnt, uint32_t id, uint32_t n_ids) {
  const RpWave w = rp_wave(id, n_ids);
  if (w.one) {
    if (w.in && (threadIdx.x & 63) == (uint32_t)__ffsll((unsigned long long)w.in) - 1)
      atomicAdd(&cnt[id], (uint32_t)__popcll(w.in));
  } else if (id < n_ids) {
    atomicAdd(&cnt[id], 1u);
  }
}

// The lanes with this lane's id.
__device__ __forceinline__ uint64_t rp_peers(uint32_t id, uint32_t n_ids, int bits) {
  const RpWave w = rp_wave(id, n_ids);
  uint64_t peers = w.in;
  if (!w.one)
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((id >> b) & 1u);
      peers &= ((id >> b) & 1u) ? set : ~set;
    }
  return peers;
}
// Writes row i at its id's next position, one per peer, in lane order.
__device__ __forceinline__ void rp_place(uint32_t* next, uint32_t id, uint32_t n_ids, uint64_t peers, uint32_t lane,
                                         int64_t i, int32_t* order) {
  const bool in = id < n_ids;
  const uint32_t rank = __popcll(peers & ((1ull << lane) - 1ull));
  uint32_t at = 0;
  if (in && rank == 0) at = atomicAdd(&next[id], (uint32_t)__popcll(peers));
  at = __shfl(at, in ? __ffsll((unsigned long long)peers) - 1 : 0) + rank;
  if (in) order[at] = (int32_t)i;
}

// Counts rows [lo, hi) into cnt with the whole workgroup.
__device__ __forceinline__ void rp_count_all(const int32_t* ids, int64_t lo, int64_t hi, uint32_t n_ids, uint32_t* cnt) {
  for (int64_t i0 = lo; i0 < hi; i0 += 16 * RP_WG) {
    uint32_t id[16];                         // sixteen loads in flight
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t i = i0 + j * RP_WG + threadIdx.x;
      id[j] = i < hi ? (uint32_t)ids[i] : 0xFFFFFFFFu;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (i0 + j * RP_WG < hi) rp_add(cnt, id[j], n_ids);
  }
}

__global__ __launch_bounds__(RP_WG) void k_row_hist(const int32_t* __restrict__ ids, int64_t n, int64_t per,
                                                    uint32_t n_ids, uint32_t* __restrict__ hist) {
  __shared__ uint32_t cnt[RP_IDS];
  for (uint32_t i = threadIdx.x; i < rp_pitch(n_ids); i += RP_WG) cnt[i] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * per, hi = lo + per < n ? lo + per : n;
  rp_count_all(ids, lo, hi, n_ids, cnt);
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < rp_pitch(n_ids); i += RP_WG) hist[(int64_t)blockIdx.x * rp_pitch(n_ids) + i] = cnt[i];
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
  __shared__ uint32_t all[RP_IDS], prior[RP_IDS];  // rows of an id: in all, in the workgroups before this one
  __shared__ uint32_t off[RP_IDS + 1], toff[RP_IDS + 1];
  __shared__ uint2 wave_sum[RP_WAVES];
  const uint32_t n_ids = (uint32_t)a.n_ids, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t i = threadIdx.x; i < RP_IDS; i += RP_WG) {
    all[i] = 0;
    prior[i] = 0;
#pragma unroll
    for (int w = 0; w < RP_WAVES; ++w) cnt[w][i] = 0;
  }
  const int64_t lo = (int64_t)blockIdx.x * a.per, hi = lo + a.per < a.n ? lo + a.per : a.n;
  const int64_t part = a.per / RP_WAVES, wlo = lo + wave * part;      // per is a multiple of 8 x 64
  const int64_t whi = wlo + part < hi ? wlo + part : hi;
  uint32_t held[RP_HELD];                                             // the wave's first rows
#pragma unroll
  for (int j = 0; j < RP_HELD; ++j) {
    const int64_t i = wlo + j * 64 + lane;
    held[j] = i < whi ? (uint32_t)a.ids[i] : 0xFFFFFFFFu;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < RP_HELD; ++j)
    if (wlo + j * 64 < whi) rp_add(cnt[wave], held[j], n_ids);
  for (int64_t i0 = wlo + RP_HELD * 64; i0 < whi; i0 += 64)
    rp_add(cnt[wave], i0 + lane < whi ? (uint32_t)a.ids[i0 + lane] : 0xFFFFFFFFu, n_ids);
  if (a.hist) {
    // two ids per thread and, where there are fewer ids than that, several parts of the workgroups
    uint32_t pairs = 1;
    while (pairs * 2 < n_ids) pairs *= 2;
    const uint32_t id = (threadIdx.x & (pairs - 1)) * 2, pitch = rp_pitch(n_ids);
    if (id < n_ids) {
      uint2 s = {0, 0}, p = {0, 0};
      for (uint32_t b0 = threadIdx.x / pairs; b0 < gridDim.x; b0 += 32 * (RP_WG / pairs)) {
        uint2 h[32];                         // all loads in flight: the counts come from other XCDs' caches
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint32_t b = b0 + j * (RP_WG / pairs);
          h[j] = b < gridDim.x ? *reinterpret_cast<const uint2*>(a.hist + (int64_t)b * pitch + id) : uint2{0, 0};
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const bool earlier = b0 + j * (RP_WG / pairs) < blockIdx.x;
          s.x += h[j].x;
          s.y += h[j].y;
          p.x += earlier ? h[j].x : 0;
          p.y += earlier ? h[j].y : 0;
        }
      }
      atomicAdd(&all[id], s.x);
      atomicAdd(&prior[id], p.x);
      if (id + 1 < n_ids) {
        atomicAdd(&all[id + 1], s.y);
        atomicAdd(&prior[id + 1], p.y);
      }
    }
  } else {
    rp_count_all(a.ids, 0, lo, n_ids, prior);
    rp_count_all(a.ids, hi, a.n, n_ids, all);          // the later ones; the rest is added below
  }
  __syncthreads();

  uint32_t before[2] = {0, 0}, total[2] = {0, 0}, tiles[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t id = threadIdx.x * 2 + j;
    if (id < n_ids) {
      before[j] = prior[id];
      total[j] = all[id];
      if (!a.hist) {
        total[j] += before[j];
#pragma unroll
        for (int w = 0; w < RP_WAVES; ++w) total[j] += cnt[w][id];
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
#pragma unroll
      for (int w = 0; w < RP_WAVES; ++w) {
        const uint32_t c = cnt[w][id];
        cnt[w][id] = next;
        next += c;
      }
    }
  }
  __syncthreads();

  // place the rows: a wave's own counters, so no other wave's work is waited for; the held rows'
  // peers are found side by side
  int bits = 0;
  while ((1u << bits) < n_ids) ++bits;
  uint64_t peers[RP_HELD];
#pragma unroll
  for (int j = 0; j < RP_HELD; ++j) peers[j] = rp_peers(held[j], n_ids, bits);
#pragma unroll
  for (int j = 0; j < RP_HELD; ++j)
    if (wlo + j * 64 < whi) rp_place(cnt[wave], held[j], n_ids, peers[j], lane, wlo + j * 64 + lane, a.order);
  for (int64_t i0 = wlo + RP_HELD * 64; i0 < whi; i0 += 64) {
    const uint32_t id = i0 + lane < whi ? (uint32_t)a.ids[i0 + lane] : 0xFFFFFFFFu;
    rp_place(cnt[wave], id, n_ids, rp_peers(id, n_ids, bits), lane, i0 + lane, a.order);
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
  if (a.n > RP_ONE_LAUNCH) {
    k_row_hist<<<wgs, RP_WG, 0, s>>>(a.ids, a.n, per, (uint32_t)a.n_ids, a.hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else {
    a.hist = nullptr;
  }
  k_row_plan<<<wgs, RP_WG, 0, s>>>(a);
  return hipGetLastError();
}

size_t row_plan_hist_bytes(int64_t n, int n_ids) {
  if (n <= RP_ONE_LAUNCH) return 0;
  int64_t per;
  return (size_t)row_plan_wgs(n, &per) * rp_pitch((uint32_t)n_ids) * 4;
}

}  // namespace qf

extern "C" {

int64_t qf_row_plan_tiles(int64_t n, int n_ids) {
  if (n < 0 || n >= QF_ROW_MAX_ROWS || n_ids < 1 || n_ids > QF_ROW_MAX_IDS) return 0;
  return (n + QF_ROW_TILE - 1) / QF_ROW_TILE + (n < n_ids ? n : n_ids);
}

size_t qf_row_plan_workspace(int64_t n, int n_ids) {
  if (n < 0 || n >= QF_ROW_MAX_ROWS || n_ids < 1 || n_ids > QF_ROW_MAX_IDS) return 0;
  return qf::row_plan_hist_bytes(n, n_ids);
}

qf_status qf_row_plan(const int32_t* ids, int64_t n, int n_ids, int32_t* offsets, int32_t* order, int32_t* tiles,
                      void* ws, size_t ws_bytes, void* stream) {
  if (n < 0 || n >= QF_ROW_MAX_ROWS) return QF_ERR_SHAPE;
  if (n_ids < 1 || n_ids > QF_ROW_MAX_IDS) return QF_ERR_ARG;
  if (!offsets || (n > 0 && (!ids || !order || !tiles))) return QF_ERR_NULL;
  const size_t need = qf_row_plan_workspace(n, n_ids);
  if (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)order) % 4 || (uintptr_t)tiles % 8 || (need > 0 && (uintptr_t)ws % 8))
    return QF_ERR_ALIGN;
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
