// Block quantization to E4M3 with one fp32 scale per 128 elements, and the gated activation in front
// of it: rows (1 x 128 along a row, gathered into expert order or not), panels (128 rows of one
// group in a column, transposed for a reduction over rows) and tiles (128 x 128, with the transpose).
//
// All are streams: each element is read once and leaves as one byte.  The scales lie block-major
// ([block][row]) because the product reads the scales of many rows of one block at a time; a row
// workgroup therefore takes 32 rows, whose scales of a block fill one cache line, except where rows are spread
// over experts: there a wave takes eight blocks of a row.
//
// Bound by bytes, at the rate of a copy (5.1 TB/s on the card of these figures): 8192 rows of 4096 to 8 experts each 66 us
// (340 MB; 127 when every copy read and quantized its row, 101 by row, 87 with a wave per row, 66 with stores past
// the caches); 32768 rows of 4096 in panels 77 us (405 MB; 83 through the caches); the gate of 65536 x 2048 134 us (675 MB),
// its gradient 114 us (671 MB).
#include "qf_fp8.h"

namespace qf {
namespace {

constexpr int Q8_WG = 256;
constexpr int64_t Q8_MAX_GRID = 1 << 22;         // a launch holds below 2^32 lanes; the rest is looped over

// ------------------------------------------------------------------- rows ---
constexpr int RQ_LANES = 8;                       // lanes of a block of 128, 16 elements each
constexpr int RQ_ROWS = Q8_WG / RQ_LANES;         // rows of a workgroup
constexpr int RQ_DEEP = 4;                        // blocks loaded before the first is encoded

struct RowQuantArgs {
  const uint16_t* x;
  int64_t ldx;
  const int32_t* positions; // where each row of x goes (null: row p to p)
  const int32_t* used;      // null, or the rows in use
  int64_t rows, n;          // rows (of x, times parts); positions
  uint32_t per, parts;      // positions per row of x, and in how many parts it is taken
  uint32_t cols, blocks, part;   // part: blocks of a workgroup
  uint8_t* codes;
  int64_t ldc;
  float* scales;
  int64_t lds;
  uint16_t* y;              // the activation in bf16 (null: not wanted)
  int64_t ldy;
};

// 16 fp32 values of a block from its lane's chunks.
__device__ __forceinline__ void f32_of(uint4 w, float* v) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = bf16_lo(q[e]);
    v[2 * e + 1] = bf16_hi(q[e]);
  }
}
__device__ __forceinline__ uint32_t max8lanes(uint32_t m) {
  m = umax(m, dpp_xor1(m));
  m = umax(m, dpp_xor2(m));
  return umax(m, dpp_hmirror(m));
}

// 1 / (1 + exp(-g)) of a bf16 g.  log2 e is taken in two parts, the first of 16 bits, so that its product
// with g is exact, and cut off rather than rounded, so that the second part's correction m of exp(-g)
// (1 + m, |m| < 2^-10 where the result is neither 0 nor 1) is not negative where exp(-g) is infinite.  Where
// exp(-g) is 0, m is kept finite (g may be infinite).
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float HI = 0x1.7154p0f;
  constexpr float LO = (float)((1.44269504088896340736 - (double)HI) * 0.69314718055994530942);
  static_assert(LO > 0.0f, "cut off, not rounded");
  const float e = __builtin_amdgcn_exp2f(-g * HI), m = fmaxf(-g * LO, -1.0f);       // (a NaN stays one in e)
  return __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, m, e));
}

// SPREAD: row t of x has the `per` positions from positions[t * per] on; it is quantized once and written to
// each.
template <bool GATED, bool SPREAD, bool NT>
__global__ __launch_bounds__(Q8_WG) void k_quant8_rows(RowQuantArgs a) {
  // a wave's eight units: one block of eight rows, whose scales lie side by side, or eight blocks of one row, whose
  // copies then leave in runs of 1 KiB
  constexpr uint32_t WIDE = SPREAD ? 8 : 1, ROWS = RQ_ROWS / WIDE;
  const uint32_t l = threadIdx.x & (RQ_LANES - 1), unit = threadIdx.x / RQ_LANES / WIDE, side = threadIdx.x / RQ_LANES % WIDE;
  const int64_t rows = a.used ? (int64_t)min((uint32_t)max(*a.used, 0), (uint32_t)a.rows) : a.rows;
  const uint32_t b0 = blockIdx.y * a.part, b1 = min(b0 + a.part, a.blocks);
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < rows; r0 += (int64_t)gridDim.x * ROWS) {
    int64_t row = r0 + unit, i0 = 0;
    if (row >= rows) continue;                    // whole units leave, so the eight lanes of a block stay together
    uint32_t mine = 1;
    if constexpr (SPREAD) {
      const int64_t t = a.parts == 1 ? row : row / a.parts;
      i0 = t * a.per + (row - t * a.parts) * SPREAD_MOST;
      const int64_t end = min((t + 1) * (int64_t)a.per, a.n);
      mine = end <= i0 ? 0u : (uint32_t)min(end - i0, (int64_t)SPREAD_MOST);
      row = t;
    }
    const uint16_t* x = a.x + row * a.ldx;
    for (uint32_t bb = b0; bb < b1; bb += RQ_DEEP * WIDE) {
      const uint32_t b = bb + side;
      uint4 w[RQ_DEEP][2], u[GATED ? RQ_DEEP : 1][2];
#pragma unroll
      for (int j = 0; j < RQ_DEEP; ++j) {
        const uint32_t c = (b + j * WIDE) * FB + l * 16;
        const bool in = b + j * WIDE < b1 && c < a.cols;
        w[j][0] = in ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
        w[j][1] = in ? *reinterpret_cast<const uint4*>(x + c + 8) : make_uint4(0, 0, 0, 0);
        if constexpr (GATED) {
          u[j][0] = in ? *reinterpret_cast<const uint4*>(x + a.cols + c) : make_uint4(0, 0, 0, 0);
          u[j][1] = in ? *reinterpret_cast<const uint4*>(x + a.cols + c + 8) : make_uint4(0, 0, 0, 0);
        }
      }
      float scale[RQ_DEEP];
#pragma unroll
      for (int j = 0; j < RQ_DEEP; ++j) {
        const uint32_t c = (b + j * WIDE) * FB + l * 16;
        float v[16];
        f32_of(w[j][0], v);
        f32_of(w[j][1], v + 8);
        uint32_t top;
        if constexpr (GATED) {
          float up[16];
          f32_of(u[j][0], up);
          f32_of(u[j][1], up + 8);
          float most = 0.0f;                       // (a NaN stays)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v[e] = up[e] * (v[e] * sigmoid(v[e]));
            most = __builtin_elementwise_maximum(most, fabsf(v[e]));
          }
          top = __float_as_uint(most) & 0x7FFFFFFFu;
        } else {
          top = umax(amax_bits8(w[j][0]), amax_bits8(w[j][1])) << 16;
        }
        const F8Scale s = f8_scale(max8lanes(top));
        scale[j] = s.scale;
        if constexpr (GATED) {
          if (a.y && b + j * WIDE < b1 && c < a.cols) {
            uint4* y = reinterpret_cast<uint4*>(a.y + row * a.ldy + c);
            y[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            y[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]), pack_bf16x2(v[14], v[15]));
          }
        }
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = f8_pack4(v[4 * e] * s.inv, v[4 * e + 1] * s.inv, v[4 * e + 2] * s.inv, v[4 * e + 3] * s.inv);
        w[j][0] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      for (uint32_t k = 0; k < mine; ++k) {
        int64_t p = row;
        if constexpr (SPREAD) {
          const uint32_t at = (uint32_t)a.positions[i0 + k];
          if (at >= (uint32_t)a.n) continue;      // in no group
          p = at;
        }
        uint8_t* codes = a.codes + p * a.ldc;
#pragma unroll
        for (int j = 0; j < RQ_DEEP; ++j) {
          const uint32_t c = (b + j * WIDE) * FB + l * 16;
          if (b + j * WIDE < b1 && c < a.cols) store16<NT>(codes + c, w[j][0]);
          if (b + j * WIDE < b1 && l == 0) a.scales[(int64_t)(b + j * WIDE) * a.lds + p] = scale[j];
        }
      }
    }
  }
}

hipError_t launch_rows(RowQuantArgs a, bool gated, hipStream_t s) {
  a.blocks = (a.cols + FB - 1) / FB;
  const int wide = a.positions ? 8 : 1;
  const int64_t rows = RQ_ROWS / wide, tiles = (a.rows + rows - 1) / rows;
  // few rows: their blocks over several workgroups, until there are 2048
  int64_t parts = (2048 + tiles - 1) / tiles;
  const int64_t most = (a.blocks + RQ_DEEP * wide - 1) / (RQ_DEEP * wide);
  parts = parts < 1 ? 1 : parts > most ? most : parts;
  a.part = (uint32_t)((most + parts - 1) / parts * RQ_DEEP * wide);
  const dim3 g((unsigned)(tiles < Q8_MAX_GRID / parts ? tiles : Q8_MAX_GRID / parts), (a.blocks + a.part - 1) / a.part);
  with_nt((a.positions ? a.n : a.rows) * (int64_t)a.cols >= NT_BYTES, [&](auto nt) {
    constexpr bool NT = decltype(nt)::value;
    if (gated) k_quant8_rows<true, false, NT><<<g, Q8_WG, 0, s>>>(a);
    else if (a.positions) k_quant8_rows<false, true, NT><<<g, Q8_WG, 0, s>>>(a);
    else k_quant8_rows<false, false, NT><<<g, Q8_WG, 0, s>>>(a);
  });
  return hipGetLastError();
}

// -------------------------------------------------------- gradient of the gate ---
struct GateArgs {
  const uint16_t *h, *da;
  uint16_t* dh;
  int64_t ldh, ldda, lddh, rows;
  const int32_t* used;
  uint32_t cols, chunks;
};

template <bool NT>
__global__ __launch_bounds__(Q8_WG) void k_swiglu_backward(GateArgs a) {
  const int64_t rows = a.used ? (int64_t)min((uint32_t)max(*a.used, 0), (uint32_t)a.rows) : a.rows;
  const int64_t total = rows * a.chunks;
  for (int64_t t = (int64_t)blockIdx.x * Q8_WG + threadIdx.x; t < total; t += (int64_t)gridDim.x * Q8_WG) {
    const int64_t row = t / a.chunks;
    const uint32_t c = (uint32_t)(t - row * a.chunks) * 8;
    const uint16_t* h = a.h + row * a.ldh + c;
    float g[8], u[8], d[8];
    f32_of(*reinterpret_cast<const uint4*>(h), g);
    f32_of(*reinterpret_cast<const uint4*>(h + a.cols), u);
    f32_of(*reinterpret_cast<const uint4*>(a.da + row * a.ldda + c), d);
    uint32_t dg[4], du[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sigmoid(g[e]);
      const float m = g[e] * s;
      const float f = s * (1.0f + (g[e] - m)), du = d[e] * u[e];
      // da u past the range with a finite u: a small f comes first (it loses nothing: both factors are above 1, or da is
      // infinite)
      const bool past = !(fabsf(du) < __builtin_inff()) && fabsf(u[e]) < __builtin_inff();
      g[e] = past ? (d[e] * f) * u[e] : du * f;
      u[e] = d[e] * m;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dg[e] = pack_bf16x2(g[2 * e], g[2 * e + 1]);
      du[e] = pack_bf16x2(u[2 * e], u[2 * e + 1]);
    }
    uint16_t* o = a.dh + row * a.lddh + c;
    store16<NT>(o, make_uint4(dg[0], dg[1], dg[2], dg[3]));
    store16<NT>(o + a.cols, make_uint4(du[0], du[1], du[2], du[3]));
  }
}

// -------------------------------------------------- panels and tiles: 128 x 128 ---
// A workgroup holds a 128 x 128 square: thread (rg, ch) rows 8 rg .. 8 rg + 7 of the 16-byte chunk ch.
// The transposed codes go through LDS, [col][128] bytes; the 8-byte unit rg of a column lies at
// rg ^ (col / 8), so that the 16 chunks of one store instruction hit distinct banks.
constexpr int SQ_PAD = 16;

struct Square {
  uint4 w[8];
};
// Codes of the transposed square from the threads' values to LDS.  inv: factor of the thread's column c.
template <typename Inv>
__device__ __forceinline__ void square_to_lds(const Square& q, Inv inv, uint8_t* t, uint32_t rg, uint32_t ch) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {                   // columns 2p, 2p + 1 of the chunk
    float lo[8], hi[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint32_t w = p == 0 ? q.w[r].x : p == 1 ? q.w[r].y : p == 2 ? q.w[r].z : q.w[r].w;
      lo[r] = bf16_lo(w) * inv(2 * p);
      hi[r] = bf16_hi(w) * inv(2 * p + 1);
    }
    const uint32_t col = ch * 8 + 2 * p, at = (rg ^ ch) * 8;
    *reinterpret_cast<uint2*>(t + col * FB + at) = make_uint2(f8_pack4(lo[0], lo[1], lo[2], lo[3]), f8_pack4(lo[4], lo[5], lo[6], lo[7]));
    *reinterpret_cast<uint2*>(t + (col + 1) * FB + at) = make_uint2(f8_pack4(hi[0], hi[1], hi[2], hi[3]), f8_pack4(hi[4], hi[5], hi[6], hi[7]));
  }
}
// 16 codes (rows 16 q .. 16 q + 15) of a column back from LDS.
__device__ __forceinline__ uint4 square_from_lds(const uint8_t* t, uint32_t col, uint32_t q) {
  const uint32_t ch = col >> 3;
  const uint4 v = *reinterpret_cast<const uint4*>(t + col * FB + ((2 * q) ^ (ch & ~1u)) * 8);
  return ch & 1 ? make_uint4(v.z, v.w, v.x, v.y) : v;
}

struct PanelArgs {
  const uint16_t* x;
  int64_t ldx;
  const int32_t *order, *offsets;
  int64_t n;
  uint32_t per, cols, col_tiles;
  int64_t blocks;           // at most
  int32_t n_ids;
  uint8_t* codes;           // [blocks][cols][128]
  float* scales;            // [blocks][cols]
};

template <bool NT>
__global__ __launch_bounds__(Q8_WG) void k_quant8_panels(PanelArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t t[FB * FB];
  __shared__ uint32_t part[4][64];                // column pairs' maxima of each wave
  __shared__ float inv[FB];
  const uint32_t rg = threadIdx.x >> 4, ch = threadIdx.x & 15, wave = threadIdx.x >> 6;
  const int64_t total = a.blocks * a.col_tiles;
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int64_t block = u / a.col_tiles;
    const uint32_t c0 = (uint32_t)(u - block * a.col_tiles) * FB;
    GroupUnit g;
    if (a.offsets) {
      g = find_unit(a.offsets, a.n_ids, (int)a.n, FB, (uint32_t)block);
      if (g.group < 0) return;                    // blocks come in order: none is left
    } else {
      g.first = (int)(block * FB);
      g.rows = (int)(a.n - g.first < FB ? a.n - g.first : FB);
    }
    const uint32_t c = c0 + ch * 8;
    Square q;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int row = (int)(rg * 8) + r;
      q.w[r] = make_uint4(0, 0, 0, 0);
      if (row < g.rows && c < a.cols) {
        int64_t src = g.first + row;
        if (a.order) {
          const uint32_t i = (uint32_t)a.order[src];
          src = i < (uint32_t)a.n ? (int64_t)(i / a.per) : -1;
        }
        if (src >= 0) q.w[r] = *reinterpret_cast<const uint4*>(a.x + src * a.ldx + c);
      }
    }
    // column maxima: 8 rows here, 4 row groups of the wave, 4 waves
    u16x2_t m[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      m[p] = u16x2_t{0, 0};
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t w = p == 0 ? q.w[r].x : p == 1 ? q.w[r].y : p == 2 ? q.w[r].z : q.w[r].w;
        m[p] = __builtin_elementwise_max(m[p], __builtin_bit_cast(u16x2_t, w & 0x7FFF7FFFu));
      }
#pragma unroll
      for (int d = 16; d < 64; d <<= 1)
        m[p] = __builtin_elementwise_max(m[p], __builtin_bit_cast(u16x2_t, (uint32_t)__shfl_xor((int)__builtin_bit_cast(uint32_t, m[p]), d)));
    }
    if ((rg & 3) == 0)
#pragma unroll
      for (int p = 0; p < 4; ++p) part[wave][ch * 4 + p] = __builtin_bit_cast(uint32_t, m[p]);
    __syncthreads();
    if (threadIdx.x < FB) {
      uint32_t top = 0;
      for (int w = 0; w < 4; ++w) top = umax(top, (part[w][threadIdx.x >> 1] >> (16 * (threadIdx.x & 1))) & 0xFFFFu);
      const F8Scale s = f8_scale(top << 16);
      inv[threadIdx.x] = s.inv;
      if (c0 + threadIdx.x < a.cols) a.scales[block * a.cols + c0 + threadIdx.x] = s.scale;
    }
    __syncthreads();
    square_to_lds(q, [&](int e) { return inv[ch * 8 + e]; }, t, rg, ch);
    __syncthreads();
    uint8_t* out = a.codes + (block * a.cols + c0) * FB;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = j * Q8_WG + threadIdx.x, col = at >> 3;
      if (c0 + col < a.cols) store16<NT>(out + at * 16, square_from_lds(t, col, at & 7));
    }
    __syncthreads();
  }
}

struct TileArgs {
  const uint16_t* x;        // [count][rows][ldx]
  int64_t ldx, rows, cols, count;
  uint32_t row_tiles, col_tiles;
  uint8_t *codes, *codes_t; // [count][rows][cols], [count][cols][rows] (either may be null)
  float *scales, *scales_t; // [count][row tiles][col tiles], [count][col tiles][row tiles]
};

__global__ __launch_bounds__(Q8_WG) void k_quant8_tiles(TileArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t t[FB * FB];
  __shared__ uint32_t part[4];
  const uint32_t rg = threadIdx.x >> 4, ch = threadIdx.x & 15;
  const int64_t per = (int64_t)a.row_tiles * a.col_tiles, total = a.count * per;
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int64_t e = u / per;
    const uint32_t in_e = (uint32_t)(u - e * per), rt = in_e / a.col_tiles, ct = in_e - rt * a.col_tiles;
    const int64_t r0 = (int64_t)rt * FB + rg * 8, c = (int64_t)ct * FB + ch * 8;
    const uint16_t* x = a.x + (e * a.rows + r0) * a.ldx + c;
    Square q;
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      q.w[r] = r0 + r < a.rows && c < a.cols ? *reinterpret_cast<const uint4*>(x + r * a.ldx) : make_uint4(0, 0, 0, 0);
      top = umax(top, amax_bits8(q.w[r]));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = umax(top, (uint32_t)__shfl_xor((int)top, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    const F8Scale s = f8_scale(umax(umax(part[0], part[1]), umax(part[2], part[3])) << 16);
    if (threadIdx.x == 0) {
      if (a.scales) a.scales[e * per + in_e] = s.scale;
      if (a.scales_t) a.scales_t[e * per + (int64_t)ct * a.row_tiles + rt] = s.scale;
    }
    if (a.codes && c < a.cols) {
      uint8_t* o = a.codes + (e * a.rows + r0) * a.cols + c;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        float v[8];
        f32_of(q.w[r], v);
        if (r0 + r < a.rows)
          *reinterpret_cast<uint2*>(o + r * a.cols) = make_uint2(f8_pack4(v[0] * s.inv, v[1] * s.inv, v[2] * s.inv, v[3] * s.inv),
                                                                 f8_pack4(v[4] * s.inv, v[5] * s.inv, v[6] * s.inv, v[7] * s.inv));
      }
    }
    if (a.codes_t) {
      square_to_lds(q, [&](int) { return s.inv; }, t, rg, ch);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = j * Q8_WG + threadIdx.x, col = at >> 3, row = (at & 7) * 16;
        if ((int64_t)ct * FB + col < a.cols && (int64_t)rt * FB + row < a.rows)
          *reinterpret_cast<uint4*>(a.codes_t + (e * a.cols + (int64_t)ct * FB + col) * a.rows + (int64_t)rt * FB + row) =
              square_from_lds(t, col, at & 7);
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ argument checks ---
bool bad_cols(int64_t cols, int64_t step) { return cols < 1 || cols % step != 0 || cols >= QF_FP8_MAX_COLS; }
unsigned grid_of(int64_t units) { return (unsigned)(units < Q8_MAX_GRID ? units : Q8_MAX_GRID); }

qf_status rows_args(const RowQuantArgs& a, int64_t rows, int64_t cols, int64_t wide, int64_t rows_per_x) {
  if (rows < 0 || rows >= QF_ROW_MAX_ROWS || bad_cols(cols, 16) || a.ldx < wide || a.ldc < cols || a.lds < rows)
    return QF_ERR_SHAPE;
  if (a.positions && rows_per_x < 1) return QF_ERR_ARG;
  if (rows == 0) return QF_OK;
  if (!a.x || !a.codes || !a.scales) return QF_ERR_NULL;
  if (misaligned(a.x, 16) || a.ldx % 8 || misaligned(a.codes, 16) || a.ldc % 16 || misaligned(a.scales, 4) ||
      misaligned(a.positions, 4) || misaligned(a.used, 4))
    return QF_ERR_ALIGN;
  return QF_OK;
}

}  // namespace
}  // namespace qf

using namespace qf;

extern "C" {

qf_status qf_quant_fp8(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols, const int32_t* positions,
                       int64_t rows_per_x, const int32_t* d_rows, uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                       void* stream) {
  RowQuantArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.positions = positions;
  a.used = positions ? nullptr : d_rows;
  a.codes = codes;
  a.ldc = ldc;
  a.scales = scales;
  a.lds = lds;
  const qf_status st = rows_args(a, rows, cols, cols, rows_per_x);
  if (st != QF_OK || rows == 0) return st;
  a.n = rows;
  a.per = (uint32_t)(positions && rows_per_x < rows ? rows_per_x : positions ? rows : 1);
  a.parts = (a.per + SPREAD_MOST - 1) / SPREAD_MOST;
  a.rows = (rows + a.per - 1) / a.per * a.parts;
  a.cols = (uint32_t)cols;
  return status_of(launch_rows(a, false, (hipStream_t)stream));
}

qf_status qf_swiglu_quant_fp8(const uint16_t* h, int64_t ldh, int64_t rows, int64_t cols, const int32_t* d_rows,
                              uint8_t* codes, int64_t ldc, float* scales, int64_t lds, uint16_t* y, int64_t ldy,
                              void* stream) {
  RowQuantArgs a = {};
  a.x = h;
  a.ldx = ldh;
  a.used = d_rows;
  a.codes = codes;
  a.ldc = ldc;
  a.scales = scales;
  a.lds = lds;
  const qf_status st = rows_args(a, rows, cols, 2 * cols, 1);
  if (st != QF_OK) return st;
  if (y && ldy < cols) return QF_ERR_SHAPE;
  if (rows == 0) return QF_OK;
  if (y && (misaligned(y, 16) || ldy % 8)) return QF_ERR_ALIGN;
  a.y = y;
  a.ldy = ldy;
  a.rows = rows;
  a.cols = (uint32_t)cols;
  a.per = 1;
  return status_of(launch_rows(a, true, (hipStream_t)stream));
}

qf_status qf_swiglu_backward(const uint16_t* h, int64_t ldh, const uint16_t* da, int64_t ldda, int64_t rows, int64_t cols,
                             const int32_t* d_rows, uint16_t* dh, int64_t lddh, void* stream) {
  if (rows < 0 || rows >= QF_ROW_MAX_ROWS || bad_cols(cols, 8) || ldh < 2 * cols || ldda < cols || lddh < 2 * cols)
    return QF_ERR_SHAPE;
  if (rows == 0) return QF_OK;
  if (!h || !da || !dh) return QF_ERR_NULL;
  if (misaligned(h, 16) || ldh % 8 || misaligned(da, 16) || ldda % 8 || misaligned(dh, 16) || lddh % 8 || misaligned(d_rows, 4))
    return QF_ERR_ALIGN;
  GateArgs a = {h, da, dh, ldh, ldda, lddh, rows, d_rows, (uint32_t)cols, (uint32_t)(cols / 8)};
  // past the caches where twice NT_BYTES leave: 35.3 through / 35.1 past at 98 MB (67 / 70 with a quantization that reads
  // them), 58.4 / 46.8 at 134 MB (100 / 99), 71.7 / 56.4 at 163 MB (125 / 118)
  with_nt(rows * cols * 4 >= 2 * NT_BYTES, [&](auto nt) {
    k_swiglu_backward<decltype(nt)::value><<<grid_of((rows * a.chunks + Q8_WG - 1) / Q8_WG), Q8_WG, 0, (hipStream_t)stream>>>(a);
  });
  return status_of(hipGetLastError());
}

int64_t qf_fp8_panels(int64_t n, int n_ids) {
  if (!plan_sizes_ok(n, n_ids)) return 0;
  return n_ids == 1 ? (n + FB - 1) / FB : (n + FB - 1) / FB + (n < n_ids ? n : n_ids);
}

qf_status qf_quant_fp8_panels(const uint16_t* x, int64_t ldx, int64_t rows, int64_t cols, const int32_t* order,
                              int64_t rows_per_x, const int32_t* offsets, int n_ids, uint8_t* codes, float* scales,
                              void* stream) {
  if (rows < 0 || rows >= QF_ROW_MAX_ROWS || bad_cols(cols, 8) || ldx < cols) return QF_ERR_SHAPE;
  if (n_ids < 1 || n_ids > QF_ROW_MAX_IDS || (!offsets && n_ids != 1) || (order && rows_per_x < 1)) return QF_ERR_ARG;
  if (rows == 0) return QF_OK;
  if (!x || !codes || !scales) return QF_ERR_NULL;
  if (misaligned(x, 16) || ldx % 8 || misaligned(codes, 16) || misaligned(scales, 4) || misaligned(order, 4) || misaligned(offsets, 4))
    return QF_ERR_ALIGN;
  PanelArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.order = order;
  a.offsets = offsets;
  a.n = rows;
  a.per = (uint32_t)(rows_per_x < rows ? rows_per_x : rows);
  a.cols = (uint32_t)cols;
  a.col_tiles = (a.cols + FB - 1) / FB;
  a.blocks = qf_fp8_panels(rows, n_ids);
  a.n_ids = n_ids;
  a.codes = codes;
  a.scales = scales;
  with_nt(rows * cols >= NT_BYTES, [&](auto nt) {
    k_quant8_panels<decltype(nt)::value><<<grid_of(a.blocks * a.col_tiles), Q8_WG, 0, (hipStream_t)stream>>>(a);
  });
  return status_of(hipGetLastError());
}

qf_status qf_quant_fp8_tiles(const uint16_t* x, int64_t ldx, int64_t count, int64_t rows, int64_t cols, uint8_t* codes,
                             float* scales, uint8_t* codes_t, float* scales_t, void* stream) {
  if (count < 0 || rows < 0 || rows >= QF_FP8_MAX_COLS || bad_cols(cols, 16) || ldx < cols || ldx >= QF_FP8_MAX_COLS)
    return QF_ERR_SHAPE;
  if (codes_t && rows % 16 != 0) return QF_ERR_SHAPE;
  if (count > QF_ROW_MAX_IDS || (!codes) != (!scales) || (!codes_t) != (!scales_t)) return QF_ERR_ARG;
  if (count == 0 || rows == 0) return QF_OK;
  if (!x || (!codes && !codes_t)) return QF_ERR_NULL;
  if (misaligned(x, 16) || ldx % 8 || misaligned(codes, 16) || misaligned(codes_t, 16) || misaligned(scales, 4) || misaligned(scales_t, 4))
    return QF_ERR_ALIGN;
  TileArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.count = count;
  a.row_tiles = (uint32_t)((rows + FB - 1) / FB);
  a.col_tiles = (uint32_t)((cols + FB - 1) / FB);
  a.codes = codes;
  a.scales = scales;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  k_quant8_tiles<<<grid_of(count * a.row_tiles * a.col_tiles), Q8_WG, 0, (hipStream_t)stream>>>(a);
  return status_of(hipGetLastError());
}

}  // extern "C"
