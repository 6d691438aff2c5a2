// Low-rank adapters of many requests beside one shared projection:
//   Y[i] += scale[e] * B_e (A_e X[i / rows_per_x]),  e the adapter of row i.
// This is the unmerged form of the adapters that the merge kernels fold into the weights: a
// rollout batch holds rows of many adapters, and the shared (packed) weight stays as it is.
//
// Two steps, S = X A^T (fp32) and Y += (scale S) B^T, in one of two forms:
//   rows   few rows: a workgroup per row (and part of K or of N), vector FMAs; the adapters'
//          bytes are the work, and a decode step's rows rarely share an adapter.
//   tiles  otherwise: the row plan's tiles of up to 32 rows of one adapter, on the bf16 matrix
//          cores (32x32x16).  X is read once; the second step accumulates onto Y in fp32 and
//          rounds once.  S enters the matrix cores as the sum of two bf16 (hi + lo, relative
//          error below 2^-16), so its rounding stays far under Y's own.
// Both are bounded by memory: X and Y pass once, 4 r flops per X element and per Y element.
// K is split over workgroups when there are few rows; the parts of S are summed in a fixed
// order by the second step (no atomics: same inputs, same bits).
#include <algorithm>
#include <string.h>

#include "qf_device.h"
#include "qf_kernels.h"

namespace qf {

typedef __bf16 la_bf16x8 __attribute__((ext_vector_type(8)));
typedef float la_f32x16 __attribute__((ext_vector_type(16)));

constexpr int LA_WG = 256, LA_WAVES = LA_WG / 64;
constexpr int LA_KSTEP = 64;                       // K per wave and step: 128 bytes of every row
constexpr int LA_ROW_RANKS = 16;                   // adapter rows per workgroup of the rows form
constexpr int LA_ROW_K = LA_WG * 8;                // K per pass of a rows-form workgroup

__device__ __forceinline__ float la_wave_sum(float v) {
  v += __uint_as_float(dpp_xor1(__float_as_uint(v)));
  v += __uint_as_float(dpp_xor2(__float_as_uint(v)));
  v += __uint_as_float(dpp_hmirror(__float_as_uint(v)));
  v += __uint_as_float(dpp_mirror(__float_as_uint(v)));
  v += __uint_as_float(swz_xor16(__float_as_uint(v)));
  return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ void la_unpack8(uint4 w, float (&f)[8]) {
  f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x);
  f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z);
  f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}

// Eight consecutive bf16 of a row of r (from k; those at or past r read as zero).
template <bool VEC>
__device__ __forceinline__ uint4 la_rank8(const uint16_t* row, int k, int r) {
  uint4 o = {0, 0, 0, 0};
  if (VEC) {                                       // r a multiple of 8, rows 16-byte aligned
    if (k < r) o = *reinterpret_cast<const uint4*>(row + k);
    return o;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < r) w[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
  return uint4{w[0], w[1], w[2], w[3]};
}

// ---------------------------------------------------------------- rows form ----
__global__ __launch_bounds__(LA_WG) void k_lora_row_down(LoraApplyArgs a) {
  __shared__ float part[LA_WAVES][LA_ROW_RANKS];
  const int row = blockIdx.x, r0 = blockIdx.y * LA_ROW_RANKS, split = blockIdx.z;
  const int e = a.ids[row];
  if ((uint32_t)e >= (uint32_t)a.n_adapters) return;
  const uint16_t* x = a.X + (int64_t)(row / a.rows_per_x) * a.ldx;
  const uint16_t* A = a.A + ((int64_t)e * a.r + r0) * a.K;
  const int nr = a.r - r0 < LA_ROW_RANKS ? a.r - r0 : LA_ROW_RANKS;
  float acc[LA_ROW_RANKS];
#pragma unroll
  for (int j = 0; j < LA_ROW_RANKS; ++j) acc[j] = 0.0f;
  for (int k = split * LA_ROW_K + threadIdx.x * 8; k < a.K; k += a.splits * LA_ROW_K) {
    float xf[8];
    la_unpack8(*reinterpret_cast<const uint4*>(x + k), xf);
    uint4 w[LA_ROW_RANKS];
#pragma unroll
    for (int j = 0; j < LA_ROW_RANKS; ++j)
      if (j < nr) w[j] = *reinterpret_cast<const uint4*>(A + (int64_t)j * a.K + k);
#pragma unroll
    for (int j = 0; j < LA_ROW_RANKS; ++j) {
      if (j < nr) {
        float f[8];
        la_unpack8(w[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j] = __builtin_fmaf(xf[i], f[i], acc[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < LA_ROW_RANKS; ++j) acc[j] = la_wave_sum(acc[j]);
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int j = 0; j < LA_ROW_RANKS; ++j) part[threadIdx.x >> 6][j] = acc[j];
  __syncthreads();
  if ((int)threadIdx.x < nr)
    a.S[((int64_t)split * a.rows + row) * a.r + r0 + threadIdx.x] =
        (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}

template <bool VEC>
__global__ __launch_bounds__(LA_WG) void k_lora_row_up(LoraApplyArgs a) {
  __shared__ float s[QF_LORA_APPLY_MAX_R];
  const int row = blockIdx.y;
  const int e = a.ids[row];
  if ((uint32_t)e >= (uint32_t)a.n_adapters) return;
  const float scale = a.scale ? a.scale[e] : 1.0f;
  if ((int)threadIdx.x < QF_LORA_APPLY_MAX_R) {
    float v = 0.0f;
    if ((int)threadIdx.x < a.r)
      for (int p = 0; p < a.splits; ++p) v += a.S[((int64_t)p * a.rows + row) * a.r + threadIdx.x];
    s[threadIdx.x] = v * scale;                    // zero past r
  }
  __syncthreads();
  const int n = blockIdx.x * LA_WG + threadIdx.x;
  if (n >= a.N) return;
  const uint16_t* b = a.B + ((int64_t)e * a.N + n) * a.r;
  uint16_t* y = a.Y + (int64_t)row * a.ldy + n;
  float acc = __uint_as_float((uint32_t)*y << 16);
  for (int k = 0; k < a.r; k += 8) {
    float f[8];
    la_unpack8(la_rank8<VEC>(b, k, a.r), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = __builtin_fmaf(f[i], s[k + i], acc);
  }
  *y = (uint16_t)pack_bf16x2(acc, 0.0f);
}

// --------------------------------------------------------------- tiles form ----
// One tile's adapter, rows and positions; a plan that does not fit the call gives no tile.
struct LaTile {
  int e, first, count;
};
__device__ __forceinline__ bool la_tile(const LoraApplyArgs& a, int t, LaTile& o) {
  const int2 w = reinterpret_cast<const int2*>(a.tiles)[t];
  if ((uint32_t)w.x >= (uint32_t)a.n_ids || w.y < 0) return false;
  o.e = w.x;
  o.first = w.y;
  o.count = std::min(std::min(a.offsets[w.x + 1], a.rows) - w.y, (int)QF_ROW_TILE);
  return o.count > 0;
}
__device__ __forceinline__ int la_row(const LoraApplyArgs& a, const LaTile& t, int i) {
  if (i >= t.count) return -1;
  const int row = a.order[t.first + i];
  return (uint32_t)row < (uint32_t)a.rows ? row : -1;
}

// S of one tile and K part: 32 rows x 32 NB adapter rows.  Lane (i = lane & 31, h = lane >> 5)
// holds 8 bf16 of X row i and of adapter row i per matrix instruction; a 64-wide K step takes
// the 64 bytes h * 64 .. of both, 16 at a time (the order of K inside a step is free).
template <int NB>
__global__ __launch_bounds__(LA_WG) void k_lora_tile_down(LoraApplyArgs a) {
  __shared__ float buf[QF_ROW_TILE][NB * 32 + 1];
  LaTile t;
  if (!la_tile(a, blockIdx.x, t)) return;
  const int split = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 31, h = lane >> 5;
  const int row = la_row(a, t, i);
  const uint16_t* x = a.X + (int64_t)((row < 0 ? 0 : row) / a.rows_per_x) * a.ldx;
  const uint16_t* A = a.A + ((int64_t)t.e * a.r + i) * a.K;
  la_f32x16 acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[b][j] = 0.0f;
  for (int k0 = (split * LA_WAVES + wave) * LA_KSTEP; k0 < a.K; k0 += a.splits * LA_WAVES * LA_KSTEP) {
    uint4 xv[4], av[NB][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + h * 32 + j * 8;
      xv[j] = uint4{0, 0, 0, 0};
      if (row >= 0 && k < a.K) xv[j] = *reinterpret_cast<const uint4*>(x + k);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        av[b][j] = uint4{0, 0, 0, 0};
        if (b * 32 + i < a.r && k < a.K) av[b][j] = *reinterpret_cast<const uint4*>(A + (int64_t)b * 32 * a.K + k);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(la_bf16x8, xv[j]),
                                                         __builtin_bit_cast(la_bf16x8, av[b][j]), acc[b], 0, 0, 0);
  }
  // the waves' parts, added in order; register j of a lane is row 8 (j / 4) + 4 h + j % 4, column i
  for (int w = 0; w < LA_WAVES; ++w) {
    if (wave == w) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float* c = &buf[8 * (j >> 2) + 4 * h + (j & 3)][b * 32 + i];
          *c = w == 0 ? acc[b][j] : *c + acc[b][j];
        }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < t.count * a.r; c += LA_WG)
    a.S[((int64_t)split * a.rows + t.first + c / a.r) * a.r + c % a.r] = buf[c / a.r][c % a.r];
}

// Y of one tile and N part.  The matrix instruction's rows are outputs n and its columns the
// tile's rows; its row m stands for n = n0 + 16 (m / 8) + 8 ((m / 4) % 2) + 4 half + m % 4 of a
// 64-wide step, so that a lane ends up with 8 consecutive n of its row in two instructions'
// registers: 16-byte accesses of Y.
template <int RB, bool VEC_B, bool VEC_Y>
__global__ __launch_bounds__(LA_WG) void k_lora_tile_up(LoraApplyArgs a) {
  LaTile t;
  if (!la_tile(a, blockIdx.x, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 31, h = lane >> 5;
  const int row = la_row(a, t, i);
  const float scale = a.scale ? a.scale[t.e] : 1.0f;
  uint4 hi[RB], lo[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = b * 16 + h * 8 + j;
      v[j] = 0.0f;
      if (i < t.count && k < a.r)
        for (int p = 0; p < a.splits; ++p) v[j] += a.S[((int64_t)p * a.rows + t.first + i) * a.r + k];
      v[j] *= scale;
    }
    uint32_t wh[4], wl[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wh[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      wl[j] = pack_bf16x2(v[2 * j] - bf16_lo(wh[j]), v[2 * j + 1] - bf16_hi(wh[j]));
    }
    hi[b] = uint4{wh[0], wh[1], wh[2], wh[3]};
    lo[b] = uint4{wl[0], wl[1], wl[2], wl[3]};
  }
  const uint16_t* B = a.B + (int64_t)t.e * a.N * a.r;
  uint16_t* y = a.Y + (int64_t)(row < 0 ? 0 : row) * a.ldy;
  const int end = std::min(a.N, (int)(blockIdx.y + 1) * a.n_part);
  for (int n0 = blockIdx.y * a.n_part + wave * 64; n0 < end; n0 += LA_WAVES * 64) {
    la_f32x16 acc[2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = n0 + 16 * q + 8 * h;
      uint32_t w[4] = {0, 0, 0, 0};
      if (row >= 0) {
        if (VEC_Y && n + 8 <= a.N) {
          const uint4 u = *reinterpret_cast<const uint4*>(y + n);
          w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n + j < a.N) w[j >> 1] |= (uint32_t)y[n + j] << (16 * (j & 1));
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j >> 2][4 * q + (j & 3)] = j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int n = n0 + 16 * (i >> 3) + 8 * ((i >> 2) & 1) + 4 * half + (i & 3);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        uint4 bv = {0, 0, 0, 0};
        if (n < a.N) bv = la_rank8<VEC_B>(B + (int64_t)n * a.r, b * 16 + h * 8, a.r);
        acc[half] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(la_bf16x8, bv),
                                                            __builtin_bit_cast(la_bf16x8, hi[b]), acc[half], 0, 0, 0);
        acc[half] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(la_bf16x8, bv),
                                                            __builtin_bit_cast(la_bf16x8, lo[b]), acc[half], 0, 0, 0);
      }
    }
    if (row >= 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + 16 * q + 8 * h;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = pack_bf16x2(acc[j >> 1][4 * q + 2 * (j & 1)], acc[j >> 1][4 * q + 2 * (j & 1) + 1]);
        if (VEC_Y && n + 8 <= a.N) {
          *reinterpret_cast<uint4*>(y + n) = uint4{w[0], w[1], w[2], w[3]};
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n + j < a.N) y[n + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
      }
    }
  }
}

namespace {
template <int RB>
void launch_up(const LoraApplyArgs& a, dim3 g, bool vb, bool vy, hipStream_t s) {
  if (vb && vy) k_lora_tile_up<RB, true, true><<<g, LA_WG, 0, s>>>(a);
  else if (vb) k_lora_tile_up<RB, true, false><<<g, LA_WG, 0, s>>>(a);
  else if (vy) k_lora_tile_up<RB, false, true><<<g, LA_WG, 0, s>>>(a);
  else k_lora_tile_up<RB, false, false><<<g, LA_WG, 0, s>>>(a);
}
}  // namespace

// K parts: enough workgroups to fill the chip when there are few rows or tiles, each wave
// keeping at least one step.
int lora_apply_splits(bool tiles, int64_t units, int K, int r) {
  const int64_t wgs = tiles ? units : units * ((r + LA_ROW_RANKS - 1) / LA_ROW_RANKS);
  const int per = tiles ? LA_WAVES * LA_KSTEP : LA_ROW_K;
  const int most = std::min((K + per - 1) / per, LORA_APPLY_MAX_SPLITS);
  int s = 1;
  while (s * 2 <= most && wgs * s < 512) s *= 2;
  return s;
}

hipError_t launch_lora_apply(LoraApplyArgs a, bool tiles, int64_t n_tiles, hipStream_t s) {
  const bool vb = a.r % 8 == 0 && (uintptr_t)a.B % 16 == 0;
  const bool vy = a.ldy % 8 == 0 && (uintptr_t)a.Y % 16 == 0;
  if (!tiles) {
    const dim3 g1((unsigned)a.rows, (unsigned)((a.r + LA_ROW_RANKS - 1) / LA_ROW_RANKS), (unsigned)a.splits);
    k_lora_row_down<<<g1, LA_WG, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 g2((unsigned)((a.N + LA_WG - 1) / LA_WG), (unsigned)a.rows);
    if (vb) k_lora_row_up<true><<<g2, LA_WG, 0, s>>>(a);
    else k_lora_row_up<false><<<g2, LA_WG, 0, s>>>(a);
    return hipGetLastError();
  }
  const dim3 g1((unsigned)n_tiles, (unsigned)a.splits);
  if (a.r <= 32) k_lora_tile_down<1><<<g1, LA_WG, 0, s>>>(a);
  else if (a.r <= 64) k_lora_tile_down<2><<<g1, LA_WG, 0, s>>>(a);
  else k_lora_tile_down<4><<<g1, LA_WG, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // N parts: whole passes of the four waves, about 1024 outputs, fewer for few tiles
  int parts = (a.N + 1023) / 1024;
  const int most = (a.N + LA_WAVES * 64 - 1) / (LA_WAVES * 64);
  while (parts * 2 <= most && n_tiles * parts < 1024) parts *= 2;
  a.n_part = ((a.N + parts - 1) / parts + LA_WAVES * 64 - 1) / (LA_WAVES * 64) * (LA_WAVES * 64);
  const dim3 g2((unsigned)n_tiles, (unsigned)((a.N + a.n_part - 1) / a.n_part));
  if (a.r <= 16) launch_up<1>(a, g2, vb, vy, s);
  else if (a.r <= 32) launch_up<2>(a, g2, vb, vy, s);
  else if (a.r <= 64) launch_up<4>(a, g2, vb, vy, s);
  else launch_up<8>(a, g2, vb, vy, s);
  return hipGetLastError();
}

}  // namespace qf

namespace {

int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

bool sizes_ok(int64_t rows, int64_t K, int64_t N, int r, int n_adapters) {
  return rows >= 0 && rows < QF_LORA_APPLY_MAX_ROWS && K >= 8 && K % 8 == 0 && K < (1 << 22) && N >= 1 &&
         N < (1 << 22) && r >= 1 && r <= QF_LORA_APPLY_MAX_R && n_adapters >= 1 && n_adapters <= QF_ROW_MAX_IDS;
}

bool row_form(int64_t rows) { return rows <= qf::LORA_APPLY_ROW_FORM; }

// The workspace's parts: S, then the plan that a call without one makes for itself.
struct Space {
  int64_t S, offsets, order, tiles, hist, total;
};
Space space_of(int64_t rows, int64_t K, int r, int n_adapters, bool planned) {
  Space o;
  memset(&o, 0, sizeof(o));
  const bool tiles = planned || !row_form(rows);
  const int64_t n_tiles = qf_row_plan_tiles(rows, n_adapters);
  const int splits = qf::lora_apply_splits(tiles, tiles ? n_tiles : rows, (int)K, r);
  int64_t at = up256(rows * r * 4 * splits);
  if (tiles && !planned) {
    o.offsets = at;
    at += up256((int64_t)(n_adapters + 1) * 4);
    o.order = at;
    at += up256(rows * 4);
    o.tiles = at;
    at += up256(n_tiles * 8);
    o.hist = at;
    at += up256((int64_t)qf_row_plan_workspace(rows, n_adapters));
  }
  o.total = at;
  return o;
}

bool bad(const void* p, uintptr_t a) { return ((uintptr_t)p % a) != 0; }

qf_status apply(const uint16_t* X, int64_t ldx, int64_t rows_per_x, const uint16_t* A, const uint16_t* B,
                const float* scale, int n_adapters, const int32_t* ids, const int32_t* offsets, const int32_t* order,
                const int32_t* tiles, int n_ids, bool planned, uint16_t* Y, int64_t ldy, int64_t rows, int64_t N,
                int64_t K, int r, void* ws, size_t ws_bytes, void* stream) {
  if (r < 1 || r > QF_LORA_APPLY_MAX_R || n_adapters < 1 || n_adapters > QF_ROW_MAX_IDS || rows_per_x < 1 ||
      rows_per_x > QF_LORA_APPLY_MAX_ROWS)
    return QF_ERR_ARG;
  if (planned && (n_ids < 1 || n_ids > n_adapters)) return QF_ERR_ARG;
  if (!sizes_ok(rows, K, N, r, n_adapters) || ldx < K || ldy < N) return QF_ERR_SHAPE;
  if (rows == 0) return QF_OK;
  if (!X || !A || !B || !Y || (planned ? !offsets || !order || !tiles : !ids)) return QF_ERR_NULL;
  if (bad(X, 16) || ldx % 8 || bad(A, 16) || bad(B, 2) || bad(Y, 2) || bad(scale, 4) || bad(ids, 4) ||
      bad(offsets, 4) || bad(order, 4) || bad(tiles, 8))
    return QF_ERR_ALIGN;
  const Space sp = space_of(rows, K, r, n_adapters, planned);
  if (!ws || ws_bytes < (size_t)sp.total) return QF_ERR_WORKSPACE;
  if (bad(ws, 16)) return QF_ERR_ALIGN;
  const bool tiled = planned || !row_form(rows);
  char* base = (char*)ws;
  if (tiled && !planned) {
    int32_t* o = (int32_t*)(base + sp.offsets);
    int32_t* p = (int32_t*)(base + sp.order);
    int32_t* q = (int32_t*)(base + sp.tiles);
    const qf_status st = qf_row_plan(ids, rows, n_adapters, o, p, q, base + sp.hist, ws_bytes - sp.hist, stream);
    if (st != QF_OK) return st;
    offsets = o;
    order = p;
    tiles = q;
    n_ids = n_adapters;
  }
  qf::LoraApplyArgs a;
  memset(&a, 0, sizeof(a));
  a.X = X;
  a.A = A;
  a.B = B;
  a.scale = scale;
  a.Y = Y;
  a.ldx = ldx;
  a.ldy = ldy;
  a.ids = ids;
  a.offsets = offsets;
  a.order = order;
  a.tiles = tiles;
  a.S = (float*)base;
  a.rows = (int)rows;
  a.rows_per_x = (int)rows_per_x;
  a.K = (int)K;
  a.N = (int)N;
  a.r = r;
  a.n_adapters = n_adapters;
  a.n_ids = n_ids;
  const int64_t n_tiles = tiled ? qf_row_plan_tiles(rows, n_ids) : 0;
  a.splits = qf::lora_apply_splits(tiled, tiled ? qf_row_plan_tiles(rows, n_adapters) : rows, a.K, r);
  return qf::status_of(qf::launch_lora_apply(a, tiled, n_tiles, (hipStream_t)stream));
}

}  // namespace

extern "C" {

size_t qf_lora_apply_workspace(int64_t rows, int64_t K, int r, int n_adapters, int planned) {
  if (!sizes_ok(rows, K, 1, r, n_adapters)) return 0;
  return (size_t)space_of(rows, K, r, n_adapters, planned != 0).total;
}

qf_status qf_lora_apply(const uint16_t* X, int64_t ldx, int64_t rows_per_x, const uint16_t* A, const uint16_t* B,
                        const float* d_scale, int n_adapters, const int32_t* ids, uint16_t* Y, int64_t ldy,
                        int64_t rows, int64_t N, int64_t K, int r, void* ws, size_t ws_bytes, void* stream) {
  return apply(X, ldx, rows_per_x, A, B, d_scale, n_adapters, ids, nullptr, nullptr, nullptr, 0, false, Y, ldy, rows, N,
               K, r, ws, ws_bytes, stream);
}

qf_status qf_lora_apply_planned(const uint16_t* X, int64_t ldx, int64_t rows_per_x, const uint16_t* A,
                                const uint16_t* B, const float* d_scale, int n_adapters, const int32_t* offsets,
                                const int32_t* order, const int32_t* tiles, int n_ids, uint16_t* Y, int64_t ldy,
                                int64_t rows, int64_t N, int64_t K, int r, void* ws, size_t ws_bytes, void* stream) {
  return apply(X, ldx, rows_per_x, A, B, d_scale, n_adapters, nullptr, offsets, order, tiles, n_ids, true, Y, ldy, rows,
               N, K, r, ws, ws_bytes, stream);
}

}  // extern "C"
