// Low-rank adapters of many requests beside one shared projection:
//   Y[i] += scale[e] * B_e (A_e X[i / rows_per_x]),  e the adapter of row i.
// This is the unmerged form of the adapters that the merge kernels fold into the weights: a
// rollout batch holds rows of many adapters, and the shared (packed) weight stays as it is.
//
// Two steps, S = X A^T (fp32) and Y += (scale S) B^T, in one of two forms:
//   rows   few rows: one launch, a workgroup per row and part of N, vector FMAs; the adapters'
//          bytes are the work, and a decode step's rows rarely share an adapter.
//   tiles  otherwise: the row plan's tiles of up to 32 rows of one adapter, on the bf16 matrix
//          cores (16x16x32).  X is read once; the second step accumulates onto Y in fp32 and
//          rounds once.  S enters the matrix cores as the sum of two bf16 (hi + lo, relative
//          error below 2^-16), so its rounding stays far under Y's own.
// Both are bounded by memory: X and Y pass once, 4 r flops per X element and per Y element.  16384
// rows of 24 adapters, 4096 -> 6144, rank 16: S 32 us (4.2 TB/s), Y 83 (4.9 TB/s read and written).
// K is split over workgroups when there are few tiles; the parts of S are summed in a fixed
// order by the second step (no atomics: same inputs, same bits).
#include <algorithm>
#include <string.h>

#include "qf_device.h"
#include "qf_operators.h"

namespace qf {

typedef __bf16 la_bf16x8 __attribute__((ext_vector_type(8)));
typedef float la_f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t la_u32x4 __attribute__((ext_vector_type(4)));

constexpr int LA_WG = 256, LA_WAVES = LA_WG / 64;
constexpr int LA_KSTEP = 128;                      // K per wave and step, at most
constexpr int LA_NSTEP = 64;                       // N per wave and step: 128 bytes of every row
constexpr int LR_WG = 1024, LR_WAVES = LR_WG / 64; // the rows form

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

// Lanes i and i ^ 8 of a 16-lane row exchange: lanes below 8 give v1 and get the other's v0.
// Two registers that hold the 64-byte halves of a lane's own row become halves of two rows such
// that one access of the wave covers whole 128-byte lines of 8 rows; applied again, it goes back.
__device__ __forceinline__ void la_swap8(uint4& v0, uint4& v1, bool low) {
  uint32_t a[4] = {v0.x, v0.y, v0.z, v0.w}, b[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t give = low ? b[j] : a[j];
    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0x128, 0xF, 0xF, true);   // row_ror:8
    if (low) b[j] = got; else a[j] = got;
  }
  v0 = uint4{a[0], a[1], a[2], a[3]};
  v1 = uint4{b[0], b[1], b[2], b[3]};
}

// Two values of S as bf16 pairs {high parts, low parts}.  The high part stays finite, or its difference
// to S would be infinity less infinity: S past the largest bf16 is that and the rest, an infinite or NaN
// S is in the low part.
__device__ __forceinline__ uint2 la_split2(float a, float b) {
  constexpr float MOST = 0x1.fep127f;
  const uint32_t hi = pack_bf16x2(__builtin_amdgcn_fmed3f(a, -MOST, MOST), __builtin_amdgcn_fmed3f(b, -MOST, MOST));
  return uint2{hi, pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi))};
}

// ---------------------------------------------------------------- rows form ----
// A workgroup per row and part of N, both steps in one launch: every part computes the row's S
// again, which is shorter than a second launch.  Rows are dealt to the 8 XCDs in turn, all parts of
// a row to one, so that its adapter's A comes from that L2 after the first (64 rows of 40 adapters,
// 4096 -> 6144, rank 16: 9.4 -> 8.4 us; 64 adapters, 4096 -> 4096, rank 32: 16.0 -> 10.1).
// The waves split K (kw of them, each lane 8 columns at a time) and, where K has fewer than 16
// waves' columns, the adapter rows; their sums meet in LDS in a fixed order.  The first outputs'
// B rows and Y are loaded before S is there.  RANKS: adapter rows per wave and pass (all their
// loads in flight at once); C: groups of 8 of B's columns loaded at once.
template <int RANKS, int C, bool VEC>
__global__ __launch_bounds__(LR_WG) void k_lora_rows(LoraApplyArgs a) {
  __shared__ float part[LR_WAVES * QF_LORA_APPLY_FEW_R];
  __shared__ float s[QF_LORA_APPLY_FEW_R];
  const int row = blockIdx.x, lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int e = a.ids[row];
  if ((uint32_t)e >= (uint32_t)a.n_adapters) return;
  const uint16_t* x = a.X + (int64_t)(row / a.rows_per_x) * a.ldx;
  const uint16_t* A = a.A + (int64_t)e * a.r * a.K;
  const uint16_t* B = a.B + (int64_t)e * a.N * a.r;
  const int n1 = std::min(a.N, (int)(blockIdx.y + 1) * a.n_part);
  int n = blockIdx.y * a.n_part + threadIdx.x;
  uint4 b[C];
  uint32_t y0 = 0;
  auto load_b = [&](int k) {
#pragma unroll
    for (int c = 0; c < C; ++c) b[c] = la_rank8<VEC>(B + (int64_t)n * a.r, k + 8 * c, a.r);
  };
  if (n < n1) {
    y0 = a.Y[(int64_t)row * a.ldy + n];
    load_b(0);
  }

  int kw = 1;
  while (kw < LR_WAVES && kw * 512 < a.K) kw *= 2;
  const int groups = LR_WAVES / kw, per = (a.r + groups - 1) / groups;
  const int kwave = wave & (kw - 1), r0 = wave / kw * per, r1 = std::min(a.r, r0 + per);
  for (int rc = r0; rc < r1; rc += RANKS) {
    float acc[RANKS];
#pragma unroll
    for (int j = 0; j < RANKS; ++j) acc[j] = 0.0f;
    for (int k = (kwave * 64 + lane) * 8; k < a.K; k += kw * 512) {
      const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
      uint4 w[RANKS];
#pragma unroll
      for (int j = 0; j < RANKS; ++j) w[j] = *reinterpret_cast<const uint4*>(A + (int64_t)std::min(rc + j, r1 - 1) * a.K + k);
      float xf[8];
      la_unpack8(xv, xf);
#pragma unroll
      for (int j = 0; j < RANKS; ++j) {
        float f[8];
        la_unpack8(w[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j] = __builtin_fmaf(xf[i], f[i], acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < RANKS; ++j) {
      acc[j] = la_wave_sum(acc[j]);
      if (lane == 0 && rc + j < r1) part[kwave * a.r + rc + j] = acc[j];
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < QF_LORA_APPLY_FEW_R) {
    float v = 0.0f;
    if ((int)threadIdx.x < a.r) {
      for (int w = 0; w < kw; ++w) v += part[w * a.r + threadIdx.x];
      v *= a.scale ? a.scale[e] : 1.0f;
    }
    s[threadIdx.x] = v;                            // zero past r
  }
  __syncthreads();
  while (n < n1) {
    float acc = __uint_as_float(y0 << 16);
    for (int k = 0; k < a.r; k += 8 * C) {
      if (k > 0) load_b(k);
#pragma unroll
      for (int c = 0; c < C; ++c) {                // zero past r on both sides
        float f[8];
        la_unpack8(b[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = __builtin_fmaf(f[i], s[k + 8 * c + i], acc);
      }
    }
    a.Y[(int64_t)row * a.ldy + n] = (uint16_t)pack_bf16x2(acc, 0.0f);
    n += LR_WG;
    if (n < n1) {
      y0 = a.Y[(int64_t)row * a.ldy + n];
      load_b(0);
    }
  }
}

// --------------------------------------------------------------- tiles form ----
// The tile of a workgroup: workgroups go to the 8 XCDs in turn, tiles of one adapter follow each
// other, so every block of 64 tiles is dealt out in runs of 8: an adapter's A and B then pass
// through few of the XCDs' caches (all 8 would read 63 MB more for 24 adapters of 4096 x 16 and
// 6144 x 16, next to 134 MB of X and 200 of Y).
__device__ __forceinline__ int la_tile_of(unsigned wg, unsigned n) {
  const unsigned base = wg & ~63u, r = wg & 63u;
  return (int)(base + 64u <= n ? base + (r & 7u) * 8u + (r >> 3) : wg);
}

// One tile's adapter, positions, and the rows of this lane's two 16-row blocks (-1: none).  A plan
// that does not fit the call gives no tile or no row.  The loads of a tile depend on each other
// (tile, then order and offsets, then X or Y), so they are issued as early as they can be.
struct LaTile {
  int e, first, count, row[2];
};
__device__ __forceinline__ bool la_tile(const LoraApplyArgs& a, int t, int i, LaTile& o) {
  const int2 w = reinterpret_cast<const int2*>(a.tiles)[t];
  if ((uint32_t)w.x >= (uint32_t)a.n_ids || (uint32_t)w.y >= (uint32_t)a.rows) return false;
  o.e = w.x;
  o.first = w.y;
#pragma unroll
  for (int b = 0; b < 2; ++b) o.row[b] = a.order[std::min(w.y + 16 * b + i, a.rows - 1)];
  const int end = std::min(a.offsets[w.x + 1], a.rows);
  o.count = end > w.y ? std::min(end - w.y, (int)QF_ROW_TILE) : 0;      // compared first: end may be any number
#pragma unroll
  for (int b = 0; b < 2; ++b)
    if (16 * b + i >= o.count || (uint32_t)o.row[b] >= (uint32_t)a.rows) o.row[b] = -1;
  return o.count > 0;
}

// S of one tile and K part: 32 rows x 16 NB adapter rows, two 16-row blocks of the 16x16x32
// matrix instruction.  Lane (i = lane & 15, g = lane >> 4) holds 8 bf16 of X row i and of adapter
// row i: the four lanes of a row read 64 contiguous bytes per load, two loads a 128-byte line.
// Steps of 32 J columns, the next step's loads in flight during this one's products; the waves
// take steps in turn and join their parts in LDS as (0 + 2) + (1 + 3).  Lanes without a row read
// row 0 (their results are not stored); adapter rows past r are stored as zero.
template <int NB>
__global__ __launch_bounds__(LA_WG) void k_lora_tile_down(LoraApplyArgs a) {
  constexpr int J = NB <= 2 ? LA_KSTEP / 32 : 2, STEP = 32 * J;
  __shared__ la_f32x4 part[2][2 * NB][64];
  const int split = blockIdx.y, lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  LaTile t;
  if (!la_tile(a, la_tile_of(blockIdx.x, gridDim.x), i, t)) return;
  const uint16_t* x[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) x[b] = a.X + (int64_t)(std::max(t.row[b], 0) / a.rows_per_x) * a.ldx + g * 8;
  const uint16_t* A[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n)
    A[n] = a.A + ((int64_t)t.e * a.r + std::min(n * 16 + i, a.r - 1)) * a.K + g * 8;
  la_f32x4 acc[2][NB];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[b][n] = la_f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  uint4 xv[J][2], av[J][NB];
  auto load = [&](int k0) {
    if (k0 + STEP <= a.K) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int b = 0; b < 2; ++b) xv[j][b] = *reinterpret_cast<const uint4*>(x[b] + k0 + j * 32);
#pragma unroll
        for (int n = 0; n < NB; ++n) av[j][n] = *reinterpret_cast<const uint4*>(A[n] + k0 + j * 32);
      }
    } else {
      const uint4 zero = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool in = k0 + j * 32 + g * 8 < a.K;
#pragma unroll
        for (int b = 0; b < 2; ++b) xv[j][b] = in ? *reinterpret_cast<const uint4*>(x[b] + k0 + j * 32) : zero;
#pragma unroll
        for (int n = 0; n < NB; ++n) av[j][n] = in ? *reinterpret_cast<const uint4*>(A[n] + k0 + j * 32) : zero;
      }
    }
  };
  const int stride = a.splits * LA_WAVES * STEP;
  int k0 = (split * LA_WAVES + wave) * STEP;
  if (k0 < a.K) load(k0);
  while (k0 < a.K) {
    uint4 xc[J][2], ac[J][NB];
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int b = 0; b < 2; ++b) xc[j][b] = xv[j][b];
#pragma unroll
      for (int n = 0; n < NB; ++n) ac[j][n] = av[j][n];
    }
    k0 += stride;
    if (k0 < a.K) load(k0);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int n = 0; n < NB; ++n)
          acc[b][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(la_bf16x8, xc[j][b]),
                                                              __builtin_bit_cast(la_bf16x8, ac[j][n]), acc[b][n], 0, 0, 0);
  }
#pragma unroll
  for (int from = 2; from > 0; from >>= 1) {
    if (wave >= from && wave < 2 * from)
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) part[wave - from][c][lane] = acc[c / NB][c % NB];
    __syncthreads();
    if (wave < from)
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) acc[c / NB][c % NB] += part[wave][c][lane];
    __syncthreads();
  }
  if (wave != 0) return;
  // register j of a lane: row 4 g + j of the block, adapter row i
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = 16 * b + 4 * g + j;
      if (at < t.count)
#pragma unroll
        for (int n = 0; n < NB; ++n)
          if (n * 16 < a.rpad)
            a.S[((int64_t)split * a.rows + t.first + at) * a.rpad + n * 16 + i] = n * 16 + i < a.r ? acc[b][n][j] : 0.0f;
    }
}

// Y of one tile and N part.  The matrix instruction's rows are outputs n and its columns the
// tile's rows (two blocks of 16).  Row m of instruction `half` stands for n = n0 + 8 (m / 4) +
// 4 half + m % 4 of a 32-wide step q, so that a lane's two results are 8 consecutive n of its row
// and the four lanes of a row hold 64 contiguous bytes; the steps q = 0, 1 are the halves of a
// 128-byte line, exchanged between lanes so that Y is accessed in whole lines.  S is summed over
// the K parts, scaled and split into its two bf16 once per workgroup, in LDS.  Up to rank 16 the
// instruction's 32 products are 16 adapter rows twice, S's high part in the first 16, its low part
// in the others, B the same in both; above, 32 adapter rows, one instruction for each part.  The
// next step's Y (and B) is loaded during this one's products.  RK: blocks of 32 adapter rows (0: rank 16).
// NT_Y: Y with the non-temporal policy.
template <int RK, bool VEC_B, bool VEC_Y, bool NT_Y>
__global__ __launch_bounds__(LA_WG) void k_lora_tile_up(LoraApplyArgs a) {
  static_assert(LA_NSTEP == 64, "a step of the wave is one 128-byte line of every row");
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const bool low = i < 8;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  LaTile t;
  if (!la_tile(a, la_tile_of(blockIdx.x, gridDim.x), i, t)) return;
  const int end = std::min(a.N, (int)(blockIdx.y + 1) * a.n_part), step = LA_WAVES * LA_NSTEP;
  // An XCD's tiles start at different steps: rows are a multiple of 256 bytes apart as a rule, and all
  // its tiles at one column would share a few cache channels (16384 rows, N 6144: 6 us of 141).
  const int begin = blockIdx.y * a.n_part + wave * LA_NSTEP;
  const int steps = begin < end ? (end - begin + step - 1) / step : 0;
  int left = steps, n0 = begin + (steps > 0 ? (int)((blockIdx.x >> 3) % (unsigned)steps) * step : 0);
  // accesses v = 0, 1 of block b: rows (i & 7) + 8 v of the block, half i / 8 of the line
  int row[2][2];
  uint16_t* y[2][2];
  const int off = 32 * (i >> 3) + 8 * g;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int other = __builtin_amdgcn_mov_dpp(t.row[b], 0x128, 0xF, 0xF, true);   // the row of lane i ^ 8
    row[b][0] = low ? t.row[b] : other;
    row[b][1] = low ? other : t.row[b];
#pragma unroll
    for (int v = 0; v < 2; ++v) y[b][v] = a.Y + (int64_t)std::max(row[b][v], 0) * a.ldy + off;
  }
  constexpr int RP = RK == 0 ? 16 : 32 * RK, NS = RK == 0 ? 1 : 2, NK = RK == 0 ? 1 : RK;
  const uint16_t* B = a.B + (int64_t)t.e * a.N * a.r;
  const int col = RK == 0 ? (g & 1) * 8 : g * 8;       // the lane's 8 adapter rows of block k
  // The step's B is loaded with its Y, one step ahead: loads return in order, so B loaded for the step
  // at hand would wait for the next step's Y too.  Above rank 32 the registers for it cost more (4096 ->
  // 4096, 1000 rows of rank 64 21.6 -> 24.5 us, 8192 rows of rank 128 143 -> 152).
  constexpr bool AHEAD = RK < 2;
  uint4 yv[2][2], bv[2][2][NK];
  auto b_at = [&](int at, int q, int half, int k) {
    // rows past N repeat the last one (not stored), columns past r the last ones (S is zero there)
    const int m = std::min(at + 32 * q + 8 * (i >> 2) + 4 * half + (i & 3), a.N - 1), c = k * 32 + col;
    return la_rank8<VEC_B>(B + (int64_t)m * a.r, VEC_B ? std::min(c, a.r - 8) : c, a.r);
  };
  auto load_b = [&](int at) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < NK; ++k) bv[q][half][k] = b_at(at, q, half, k);
  };
  auto load_y = [&](int at) {
    if (VEC_Y && at + LA_NSTEP <= a.N) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const la_u32x4* p = reinterpret_cast<const la_u32x4*>(y[b][v] + at);
          yv[b][v] = __builtin_bit_cast(uint4, NT_Y ? __builtin_nontemporal_load(p) : *p);
        }
      return;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + off + j < a.N) w[j >> 1] |= (uint32_t)y[b][v][at + j] << (16 * (j & 1));
        yv[b][v] = uint4{w[0], w[1], w[2], w[3]};
      }
  };
  if (left > 0) {
    load_y(n0);
    if (AHEAD) load_b(n0);
  }

  const float scale = a.scale ? a.scale[t.e] : 1.0f;
  __shared__ __align__(16) uint2 sp[2][QF_ROW_TILE][RP / 4 + 2];   // high and low parts; rows 16 bytes apart in banks
  for (int c = threadIdx.x; c < QF_ROW_TILE * RP / 4; c += LA_WG) {
    const int at = c / (RP / 4), k = c % (RP / 4) * 4;
    const float* p = a.S + (int64_t)(t.first + std::min(at, t.count - 1)) * RP + k;
    float4 v = *reinterpret_cast<const float4*>(p);
    for (int q = 1; q < a.splits; ++q) {
      const float4 u = *reinterpret_cast<const float4*>(p + (int64_t)q * a.rows * RP);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    v.x *= scale; v.y *= scale; v.z *= scale; v.w *= scale;
    const uint2 p0 = la_split2(v.x, v.y), p1 = la_split2(v.z, v.w);
    sp[0][at][k / 4] = uint2{p0.x, p1.x};
    sp[1][at][k / 4] = uint2{p0.y, p1.y};
  }
  __syncthreads();
  uint4 sv[NS][2][NK];
#pragma unroll
  for (int h = 0; h < NS; ++h)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int k = 0; k < NK; ++k)
        sv[h][b][k] = *reinterpret_cast<const uint4*>(&sp[RK == 0 ? g >> 1 : h][16 * b + i][(k * 32 + col) / 4]);
  while (left > 0) {
    const int at = n0;
    uint4 yc[2][2], bc[2][2][NK];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < NK; ++k)
          if (AHEAD) bc[q][half][k] = bv[q][half][k];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 2; ++v) yc[b][v] = yv[b][v];
    n0 = n0 + step < end ? n0 + step : begin;
    if (--left > 0) {
      load_y(n0);
      if (AHEAD) load_b(n0);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) la_swap8(yc[b][0], yc[b][1], low);    // now this lane's row, steps q = 0, 1
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      la_f32x4 acc[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        acc[b][0] = la_f32x4{bf16_lo(yc[b][q].x), bf16_hi(yc[b][q].x), bf16_lo(yc[b][q].y), bf16_hi(yc[b][q].y)};
        acc[b][1] = la_f32x4{bf16_lo(yc[b][q].z), bf16_hi(yc[b][q].z), bf16_lo(yc[b][q].w), bf16_hi(yc[b][q].w)};
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const uint4 bw = AHEAD ? bc[q][half][k] : b_at(at, q, half, k);
#pragma unroll
          for (int h = 0; h < NS; ++h)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              acc[b][half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(la_bf16x8, bw), __builtin_bit_cast(la_bf16x8, sv[h][b][k]), acc[b][half], 0, 0, 0);
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
        yc[b][q] = uint4{pack_bf16x2(acc[b][0][0], acc[b][0][1]), pack_bf16x2(acc[b][0][2], acc[b][0][3]),
                         pack_bf16x2(acc[b][1][0], acc[b][1][1]), pack_bf16x2(acc[b][1][2], acc[b][1][3])};
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) la_swap8(yc[b][0], yc[b][1], low);
    const bool whole = VEC_Y && at + LA_NSTEP <= a.N;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        if (row[b][v] < 0) continue;
        if (whole) {
          la_u32x4* p = reinterpret_cast<la_u32x4*>(y[b][v] + at);
          if (NT_Y) __builtin_nontemporal_store(__builtin_bit_cast(la_u32x4, yc[b][v]), p);
          else *p = __builtin_bit_cast(la_u32x4, yc[b][v]);
        } else {
          const uint32_t w[4] = {yc[b][v].x, yc[b][v].y, yc[b][v].z, yc[b][v].w};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (at + off + j < a.N) y[b][v][at + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
      }
  }
}

namespace {
// Y beyond the caches is accessed non-temporally.  Microseconds without / with it, rank 16 and
// one adapter: Y of 201 MB 133 / 126 (plan and 24 adapters), of 101 MB 49 / 58.
constexpr int64_t LA_NT_BYTES = 160ll << 20;

template <int RK>
void launch_up(const LoraApplyArgs& a, dim3 g, bool vb, bool vy, hipStream_t s) {
  if (vb && vy && (int64_t)a.rows * a.N * 2 > LA_NT_BYTES) k_lora_tile_up<RK, true, true, true><<<g, LA_WG, 0, s>>>(a);
  else if (vb && vy) k_lora_tile_up<RK, true, true, false><<<g, LA_WG, 0, s>>>(a);
  else if (vb) k_lora_tile_up<RK, true, false, false><<<g, LA_WG, 0, s>>>(a);
  else if (vy) k_lora_tile_up<RK, false, true, false><<<g, LA_WG, 0, s>>>(a);
  else k_lora_tile_up<RK, false, false, false><<<g, LA_WG, 0, s>>>(a);
}
}  // namespace

// K parts of the tiles form: enough workgroups to fill the chip when there are few tiles, each
// wave keeping at least one step.
int lora_apply_splits(int64_t tiles, int K) {
  const int most = std::min((K + LA_WAVES * LA_KSTEP - 1) / (LA_WAVES * LA_KSTEP), LORA_APPLY_MAX_SPLITS);
  int s = 1;
  while (s * 2 <= most && tiles * s < 1024) s *= 2;
  return s;
}

hipError_t launch_lora_apply(LoraApplyArgs a, bool tiles, int64_t n_tiles, hipStream_t s) {
  const bool vb = a.r % 8 == 0 && (uintptr_t)a.B % 16 == 0;
  const bool vy = a.ldy % 8 == 0 && (uintptr_t)a.Y % 16 == 0;
  if (!tiles) {
    // parts of N: about one workgroup per CU, each with at least one output per thread
    const int most = (a.N + LR_WG - 1) / LR_WG;
    const int parts = std::min(most, std::max(1, 256 / a.rows));
    a.n_part = ((a.N + parts - 1) / parts + 63) / 64 * 64;
    const dim3 g((unsigned)(a.rows + 7) / 8 * 8, (unsigned)((a.N + a.n_part - 1) / a.n_part));
    if (a.r <= 16 && vb) k_lora_rows<8, 2, true><<<g, LR_WG, 0, s>>>(a);
    else if (a.r <= 16) k_lora_rows<8, 2, false><<<g, LR_WG, 0, s>>>(a);
    else if (vb) k_lora_rows<16, 4, true><<<g, LR_WG, 0, s>>>(a);
    else k_lora_rows<16, 4, false><<<g, LR_WG, 0, s>>>(a);
    return hipGetLastError();
  }
  const dim3 g1((unsigned)n_tiles, (unsigned)a.splits);
  if (a.r <= 16) k_lora_tile_down<1><<<g1, LA_WG, 0, s>>>(a);
  else if (a.r <= 32) k_lora_tile_down<2><<<g1, LA_WG, 0, s>>>(a);
  else if (a.r <= 64) k_lora_tile_down<4><<<g1, LA_WG, 0, s>>>(a);
  else k_lora_tile_down<8><<<g1, LA_WG, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // N parts: whole passes of the four waves; enough workgroups to fill the chip once (each pays for its
  // tile's rows and S before its first product), twice where a part keeps more than two passes.
  // Microseconds once / twice, rank 16: 16384 rows of 24 adapters, N 6144 (24 passes) 136 / 120; 2048
  // rows of 40, N 8192 (3 passes at once) 27 / 24; 1024 rows of 16, N 6144 (2 passes) 16.2 / 17.0.
  const int most = (a.N + LA_WAVES * LA_NSTEP - 1) / (LA_WAVES * LA_NSTEP);
  int parts = (int)std::min<int64_t>(most, std::max<int64_t>(1, 1024 / n_tiles));
  if (parts * 2 < most) parts = (int)std::min<int64_t>(most, std::max<int64_t>(1, 2048 / n_tiles));
  a.n_part = ((a.N + parts - 1) / parts + LA_WAVES * LA_NSTEP - 1) / (LA_WAVES * LA_NSTEP) * (LA_WAVES * LA_NSTEP);
  const dim3 g2((unsigned)n_tiles, (unsigned)((a.N + a.n_part - 1) / a.n_part));
  if (a.r <= 16) launch_up<0>(a, g2, vb, vy, s);
  else if (a.r <= 32) launch_up<1>(a, g2, vb, vy, s);
  else if (a.r <= 64) launch_up<2>(a, g2, vb, vy, s);
  else launch_up<4>(a, g2, vb, vy, s);
  return hipGetLastError();
}

}  // namespace qf

namespace {

int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

bool sizes_ok(int64_t rows, int64_t K, int64_t N, int r, int n_adapters) {
  return rows >= 0 && rows < QF_LORA_APPLY_MAX_ROWS && K >= 8 && K % 8 == 0 && K < (1 << 22) && N >= 1 &&
         N < (1 << 22) && r >= 1 && r <= QF_LORA_APPLY_MAX_R && n_adapters >= 1 && n_adapters <= QF_ROW_MAX_IDS;
}

bool row_form(int64_t rows, int r) { return rows <= qf::lora_apply_few(r); }

// The workspace's parts: S, then the plan that a call without one makes for itself.
struct Space {
  int64_t S, offsets, order, tiles, hist, total;
};
Space space_of(int64_t rows, int64_t K, int r, int n_adapters, bool planned) {
  Space o;
  memset(&o, 0, sizeof(o));
  if (!planned && row_form(rows, r)) return o;
  const int64_t n_tiles = qf_row_plan_tiles(rows, n_adapters);
  int64_t at = up256(rows * qf::lora_apply_rpad(r) * 4 * qf::lora_apply_splits(n_tiles, (int)K));
  if (!planned) {
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
  if (r < 1 || r > QF_LORA_APPLY_MAX_R || n_adapters < 1 || n_adapters > QF_ROW_MAX_IDS || rows_per_x < 1) return QF_ERR_ARG;
  if (planned && (n_ids < 1 || n_ids > n_adapters)) return QF_ERR_ARG;
  if (!sizes_ok(rows, K, N, r, n_adapters) || ldx < K || ldy < N) return QF_ERR_SHAPE;
  if (rows == 0) return QF_OK;
  if (!X || !A || !B || !Y || (planned ? !offsets || !order || !tiles : !ids)) return QF_ERR_NULL;
  if (bad(X, 16) || ldx % 8 || bad(A, 16) || bad(B, 2) || bad(Y, 2) || bad(scale, 4) || bad(ids, 4) ||
      bad(offsets, 4) || bad(order, 4) || bad(tiles, 8))
    return QF_ERR_ALIGN;
  const Space sp = space_of(rows, K, r, n_adapters, planned);
  if (sp.total > 0 && (!ws || ws_bytes < (size_t)sp.total)) return QF_ERR_WORKSPACE;
  if (sp.total > 0 && bad(ws, 16)) return QF_ERR_ALIGN;
  const bool tiled = planned || !row_form(rows, r);
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
  a.rows_per_x = (int)std::min(rows_per_x, rows);      // one row of X for all of Y from there on
  a.K = (int)K;
  a.N = (int)N;
  a.r = r;
  a.rpad = qf::lora_apply_rpad(r);
  a.n_adapters = n_adapters;
  a.n_ids = n_ids;
  const int64_t n_tiles = tiled ? qf_row_plan_tiles(rows, n_ids) : 0;
  a.splits = tiled ? qf::lora_apply_splits(qf_row_plan_tiles(rows, n_adapters), a.K) : 1;
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
