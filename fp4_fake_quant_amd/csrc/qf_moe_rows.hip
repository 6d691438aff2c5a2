// Rows into expert order and back: dispatch, combine (a weighted sum over a token's experts) and the
// gradients of both.
//
// Nothing is computed that matters for time: each kernel reads every row once and writes every row
// once, 16 bytes a lane.  All go by token through the plan's positions (the inverse of its order), so
// that a token's row is read once for all its experts, a token's sum is formed in registers in a
// fixed order, and no atomics are needed.
//
// Rows of 4096, 8 of 64 experts: 8192 tokens combined in 96 us (593 MB, 6.1 TB/s; 123 with one row at a time in flight,
// 103 with eight, 97 with stores past the caches), the gradients of 4099 tokens of 6 in 89 us (436 MB, 4.9 TB/s; 98 at first;
// 80 past the caches, which the reader of these rows then pays for).
// A decode step takes what its call takes (7.8 us from Python, kernel 3.5).
#include "qf_fp8.h"

namespace qf {
namespace {

constexpr int MR_WG = 256;
constexpr int64_t MR_MAX_GRID = 1 << 22;        // a launch holds below 2^32 lanes; the rest is looped over

struct MoeRowsArgs {
  const uint16_t* x;        // dispatch: X; combine: R; backward: dY
  const uint16_t* r;        // backward: R
  uint16_t* y;              // dispatch: out; combine: Y; backward: dR (null: not wanted)
  int64_t ldx, ldr, ldy;
  const int32_t* index;     // positions
  const float* w;           // null: all 1
  float* dw;                // backward, null: not wanted
  int64_t n;                // rows in expert order
  int64_t tokens;
  uint32_t per, chunks;     // rows per token; 16-byte chunks per row
  uint32_t lane_bits;       // log2 of the lanes that share a row
};

// Lanes of a row of X: read once, written to each position that it has.
template <bool NT>
__global__ __launch_bounds__(MR_WG) void k_moe_dispatch(MoeRowsArgs a) {
  const uint32_t lanes = 1u << a.lane_bits, rows = MR_WG >> a.lane_bits;
  const uint32_t first = threadIdx.x & (lanes - 1);
  const uint32_t parts = (a.per + SPREAD_MOST - 1) / SPREAD_MOST;
  const int64_t total = a.tokens * parts;
  for (int64_t u0 = (int64_t)blockIdx.x * rows; u0 < total; u0 += (int64_t)gridDim.x * rows) {
    const int64_t u = u0 + (threadIdx.x >> a.lane_bits);
    if (u >= total) continue;
    const int64_t t = parts == 1 ? u : u / parts, i0 = t * a.per + (u - t * parts) * SPREAD_MOST;
    const int64_t end = min((t + 1) * (int64_t)a.per, a.n);
    const uint32_t mine = end <= i0 ? 0u : (uint32_t)min(end - i0, (int64_t)SPREAD_MOST);
    const uint16_t* src = a.x + t * a.ldx;
    for (uint32_t c0 = first; c0 < a.chunks; c0 += 4 * lanes) {
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c0 + q * lanes < a.chunks) v[q] = load16(src + 8 * (c0 + q * lanes));
      for (uint32_t j = 0; j < mine; ++j) {
        const uint32_t p = (uint32_t)a.index[i0 + j];
        if (p >= (uint32_t)a.n) continue;                   // in no group
        uint16_t* dst = a.y + (int64_t)p * a.ldy;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c0 + q * lanes < a.chunks) store16<NT>(dst + 8 * (c0 + q * lanes), v[q]);
      }
    }
  }
}

template <bool NT>
__global__ __launch_bounds__(MR_WG) void k_moe_combine(MoeRowsArgs a) {
  constexpr int DEEP = 8;                                   // rows loaded before the first is added
  const int64_t total = a.tokens * a.chunks;
  for (int64_t u = (int64_t)blockIdx.x * MR_WG + threadIdx.x; u < total; u += (int64_t)gridDim.x * MR_WG) {
    const int64_t t = u / a.chunks;
    const uint32_t c = (uint32_t)(u - t * a.chunks);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t j0 = 0; j0 < a.per; j0 += DEEP) {
      uint32_t p[DEEP];
      float w[DEEP];
      uint4 v[DEEP];
#pragma unroll
      for (int j = 0; j < DEEP; ++j) {
        const int64_t i = t * a.per + j0 + j;
        p[j] = j0 + j < a.per ? (uint32_t)a.index[i] : 0xFFFFFFFFu;
        w[j] = j0 + j < a.per && a.w ? a.w[i] : 1.0f;
      }
#pragma unroll
      for (int j = 0; j < DEEP; ++j)
        if (p[j] < (uint32_t)a.n) v[j] = load16_nt(a.x + (int64_t)p[j] * a.ldx + 8 * c);
#pragma unroll
      for (int j = 0; j < DEEP; ++j) {
        if (p[j] >= (uint32_t)a.n) continue;                // no expert: adds nothing, whatever its weight
        const uint32_t q[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[2 * e] = __builtin_fmaf(w[j], bf16_lo(q[e]), acc[2 * e]);
          acc[2 * e + 1] = __builtin_fmaf(w[j], bf16_hi(q[e]), acc[2 * e + 1]);
        }
      }
    }
    store16<NT>(a.y + t * a.ldy + 8 * c, make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7])));
  }
}

// Lanes of one pair (token, expert) after another; a pair's dot product is joined between its lanes.
template <bool NT>
__global__ __launch_bounds__(MR_WG) void k_moe_combine_backward(MoeRowsArgs a) {
  constexpr int DEEP = 4;
  const uint32_t lanes = 1u << a.lane_bits, rows = MR_WG >> a.lane_bits;
  const uint32_t first = threadIdx.x & (lanes - 1);
  for (int64_t i0 = (int64_t)blockIdx.x * rows; i0 < a.n; i0 += (int64_t)gridDim.x * rows) {
    const int64_t i = i0 + (threadIdx.x >> a.lane_bits);
    const uint32_t p = i < a.n ? (uint32_t)a.index[i] : 0xFFFFFFFFu;
    const bool in = p < (uint32_t)a.n;
    float dot = 0.0f;
    if (in) {
      const float w = a.w ? a.w[i] : 1.0f;
      const uint16_t* dy = a.x + (int64_t)((uint32_t)i / a.per) * a.ldx;
      const uint16_t* r = a.r + (int64_t)p * a.ldr;
      uint16_t* y = a.y + (int64_t)p * a.ldy;
      for (uint32_t c0 = first; c0 < a.chunks; c0 += DEEP * lanes) {
        uint4 g[DEEP], v[DEEP];
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
          const uint32_t c = c0 + d * lanes;
          g[d] = v[d] = make_uint4(0, 0, 0, 0);
          if (c < a.chunks) {
            g[d] = load16(dy + 8 * c);
            if (a.dw) v[d] = load16_nt(r + 8 * c);
          }
        }
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
          const uint32_t c = c0 + d * lanes;
          const uint32_t q[4] = {g[d].x, g[d].y, g[d].z, g[d].w}, s[4] = {v[d].x, v[d].y, v[d].z, v[d].w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dot = __builtin_fmaf(bf16_lo(q[e]), bf16_lo(s[e]), dot);
            dot = __builtin_fmaf(bf16_hi(q[e]), bf16_hi(s[e]), dot);
            o[e] = pack_bf16x2(w * bf16_lo(q[e]), w * bf16_hi(q[e]));
          }
          if (a.y && c < a.chunks) store16<NT>(y + 8 * c, make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
    }
    if (a.dw) {
      for (uint32_t d = 1; d < lanes; d <<= 1) dot += __shfl_xor(dot, d);
      if (first == 0 && i < a.n) a.dw[i] = dot;
    }
  }
}

// Up to four chunks a lane.  The gradients of 65536 tokens of 4 (16384 of rows of 2048) with 4 / 8 / 16 / 32 / 64 lanes a row:
// rows of 64 17.6 / 21 / 35 / 62 / 114 us, 128 32 / 29 / 39 / 66 / 118, 256 65 / 49 / 51 / 75 / 131, 512 148 / 99 / 94 / 98 / 150,
// 2048 214 / 144 / 122 / 104 / 100; dispatch goes the same way, and with few rows all are alike or 64 the best.
uint32_t lane_bits_of(uint32_t chunks) { return chunks > 64 ? 6 : chunks > 16 ? 4 : chunks > 8 ? 3 : 2; }
dim3 grid_of(int64_t units) { return dim3((unsigned)(units < MR_MAX_GRID ? units : MR_MAX_GRID)); }
bool bad_rows(int64_t H, int64_t ld) { return H < 1 || H % 8 != 0 || H >= QF_MOE_MAX_COLS || ld < H; }
bool bad_mat(const void* p, int64_t ld) { return misaligned(p, 16) || ld % 8 != 0; }

}  // namespace
}  // namespace qf

using namespace qf;

extern "C" {

qf_status qf_moe_dispatch(const uint16_t* X, int64_t ldx, int64_t rows_per_x, const int32_t* positions, int64_t n, int64_t H,
                          uint16_t* out, int64_t ldo, void* stream) {
  if (n < 0 || n >= QF_ROW_MAX_ROWS || bad_rows(H, ldx) || ldo < H) return QF_ERR_SHAPE;
  if (rows_per_x < 1) return QF_ERR_ARG;
  if (n == 0) return QF_OK;
  if (!X || !positions || !out) return QF_ERR_NULL;
  if (bad_mat(X, ldx) || bad_mat(out, ldo) || misaligned(positions, 4)) return QF_ERR_ALIGN;
  MoeRowsArgs a = {};
  a.x = X;
  a.ldx = ldx;
  a.index = positions;
  a.n = n;
  a.per = (uint32_t)(rows_per_x < n ? rows_per_x : n);
  a.tokens = (n + a.per - 1) / a.per;
  a.chunks = (uint32_t)(H / 8);
  a.lane_bits = lane_bits_of(a.chunks);
  a.y = out;
  a.ldy = ldo;
  const int64_t rows = MR_WG >> a.lane_bits;
  const int64_t units = a.tokens * ((a.per + SPREAD_MOST - 1) / SPREAD_MOST);
  with_nt(n * H * 2 >= NT_ROWS_BYTES, [&](auto nt) {
    k_moe_dispatch<decltype(nt)::value><<<grid_of((units + rows - 1) / rows), MR_WG, 0, (hipStream_t)stream>>>(a);
  });
  return status_of(hipGetLastError());
}

static qf_status combine_args(int64_t tokens, int64_t k, int64_t H, int64_t ldr, int64_t ldt) {
  if (tokens < 0 || tokens >= QF_ROW_MAX_ROWS || bad_rows(H, ldr) || ldt < H) return QF_ERR_SHAPE;
  if (k < 1 || k >= QF_ROW_MAX_ROWS) return QF_ERR_ARG;
  if (tokens * k >= QF_ROW_MAX_ROWS) return QF_ERR_SHAPE;
  return QF_OK;
}

qf_status qf_moe_combine(const uint16_t* R, int64_t ldr, const int32_t* positions, const float* weights, int64_t tokens,
                         int64_t k, int64_t H, uint16_t* Y, int64_t ldy, void* stream) {
  const qf_status st = combine_args(tokens, k, H, ldr, ldy);
  if (st != QF_OK || tokens == 0) return st;
  if (!R || !positions || !Y) return QF_ERR_NULL;
  if (bad_mat(R, ldr) || bad_mat(Y, ldy) || misaligned(positions, 4) || misaligned(weights, 4)) return QF_ERR_ALIGN;
  MoeRowsArgs a = {};
  a.x = R;
  a.ldx = ldr;
  a.index = positions;
  a.w = weights;
  a.n = tokens * k;
  a.tokens = tokens;
  a.per = (uint32_t)k;
  a.chunks = (uint32_t)(H / 8);
  a.y = Y;
  a.ldy = ldy;
  with_nt(tokens * H * 2 >= NT_BYTES, [&](auto nt) {
    k_moe_combine<decltype(nt)::value><<<grid_of((tokens * a.chunks + MR_WG - 1) / MR_WG), MR_WG, 0, (hipStream_t)stream>>>(a);
  });
  return status_of(hipGetLastError());
}

qf_status qf_moe_combine_backward(const uint16_t* dY, int64_t lddy, const uint16_t* R, int64_t ldr, const int32_t* positions,
                                  const float* weights, int64_t tokens, int64_t k, int64_t H, uint16_t* dR, int64_t lddr,
                                  float* dW, void* stream) {
  qf_status st = combine_args(tokens, k, H, lddy, lddy);
  if (st != QF_OK) return st;
  if ((dW && ldr < H) || (dR && lddr < H)) return QF_ERR_SHAPE;
  if (tokens == 0 || (!dR && !dW)) return QF_OK;
  if (!dY || !positions || (dW && !R)) return QF_ERR_NULL;
  if (bad_mat(dY, lddy) || (dW && bad_mat(R, ldr)) || (dR && bad_mat(dR, lddr)) || misaligned(positions, 4) ||
      misaligned(weights, 4) || misaligned(dW, 4))
    return QF_ERR_ALIGN;
  MoeRowsArgs a = {};
  a.x = dY;
  a.ldx = lddy;
  a.r = R;
  a.ldr = ldr;
  a.index = positions;
  a.w = weights;
  a.n = tokens * k;
  a.tokens = tokens;
  a.per = (uint32_t)k;
  a.chunks = (uint32_t)(H / 8);
  a.lane_bits = lane_bits_of(a.chunks);
  a.y = dR;
  a.ldy = lddr;
  a.dw = dW;
  const int64_t rows = MR_WG >> a.lane_bits;
  with_nt(a.n * H * 2 >= NT_ROWS_BYTES, [&](auto nt) {
    k_moe_combine_backward<decltype(nt)::value><<<grid_of((a.n + rows - 1) / rows), MR_WG, 0, (hipStream_t)stream>>>(a);
  });
  return status_of(hipGetLastError());
}

}  // extern "C"
