// Products of E4M3 operands with an fp32 scale per block of 128 along the reduction:
//   y[m, n] = sum_b sx[m, b] sw(n, b) P_b[m, n],   P_b[m, n] = sum_(k in b) x[m, k] w[n, k],
// dense, over the rows of each group of a row plan (its own w), or over a group's blocks of rows
// (weight gradients: both operands are panels and sw has a scale per column).
//
// P_b is one v_mfma_f32_16x16x128_f8f6f4 from zero per 16 x 16 outputs, and is then added to the
// accumulators times its scale in fp32.  The instruction's lane l holds 32 consecutive bytes of row
// l % 16 of each operand, from byte 32 (l / 16) of the block; both operands are laid out alike, so
// which element the hardware pairs with which inside the block does not matter.  Its result has
// column l % 16 of the second operand and rows 4 (l / 16) + 0..3 of the first: x is the second, so
// that a lane's row of x, and its scale, are one.
//
// Accuracy of the instruction, measured with pairs and triples of planted products (the K = 32 and
// 32 x 32 FP8 forms behave alike): eight products at a time are aligned to the largest exponent E among
// them and cut below 2^(E - 13), and the sums of these groups are added in fp32.  Codes drawn from the
// whole range lose up to 2^-13 of the terms' magnitudes, quantized normal values 2^-19 at the root mean square.
#include "qf_fp8.h"

namespace qf {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int64_t G8_MAX_WGS = 1 << 22;

// An operand: rows of `row` bytes pitch, blocks of 128 at `blk` bytes pitch.
struct Gemm8Args {
  const uint8_t *x, *w;
  int64_t x_row, x_blk, w_row, w_blk, w_group;
  const float *xs, *ws;
  int64_t xs_blk;                        // scales of x: [block][rows]
  int64_t ws_tile, ws_blk, ws_group;     // of w: tile scales [tile][block], or [block][rows] with ws_blk
  uint16_t* y;
  int64_t ldy, y_group;
  const int32_t* offsets;
  int32_t n_ids, n;                      // groups and rows of the plan
  int32_t M, N, K;                       // K: elements of a row-major row (panels: 0, every block whole)
  int32_t blocks;                        // blocks of the reduction (grouped over blocks: from the offsets)
  int32_t tiles_m, tiles_n;
};
enum { G8_DENSE, G8_ROWS, G8_BLOCKS };   // over what the groups go

__device__ __forceinline__ f32x4_t mfma_f8(i32x8_t a, i32x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------------ tiles ---
// 128 x 128 outputs by 4 waves of 64 x 64.
template <int MODE>
__global__ __launch_bounds__(256) void k_gemm8(Gemm8Args a) {
  constexpr int BM = 128, BN = 128, TM = 4, TN = 4;
  constexpr bool WROWS = MODE == G8_BLOCKS;                  // w has a scale per row and block
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t frow = lane & 15, fk = lane >> 4;
  const int tn = blockIdx.x % a.tiles_n;
  int tm = blockIdx.x / a.tiles_n;
  int m0, rows, group = 0, block0 = 0, blocks = a.blocks;
  if (MODE == G8_ROWS) {
    const GroupUnit g = find_unit(a.offsets, a.n_ids, a.n, BM, (uint32_t)tm);
    if (g.group < 0) return;
    group = g.group;
    m0 = g.first;
    rows = g.rows;
  } else {
    if (MODE == G8_BLOCKS) {
      group = tm / a.tiles_m;
      tm -= group * a.tiles_m;
      if (a.offsets) {
        block0 = (int)units_before(a.offsets, group, a.n, FB);
        blocks = (int)units_of(group_offset(a.offsets, group, a.n), group_offset(a.offsets, group + 1, a.n), FB);
      }
    }
    m0 = tm * BM;
    rows = min(BM, a.M - m0);
  }
  const int n0 = tn * BN, cols = min(BN, a.N - n0);
  const uint32_t wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const uint8_t* x = a.x + (int64_t)m0 * a.x_row + (int64_t)block0 * a.x_blk;
  const uint8_t* w = a.w + (int64_t)group * (WROWS ? 0 : a.w_group) + (int64_t)n0 * a.w_row + (int64_t)block0 * a.w_blk;
  const float* xs = a.xs + m0 + (int64_t)block0 * a.xs_blk;
  const float* ws = WROWS ? a.ws + n0 + (int64_t)block0 * a.ws_blk : a.ws + (int64_t)group * a.ws_group + (n0 / FB) * a.ws_tile;

  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  const i32x8_t zero = {0, 0, 0, 0, 0, 0, 0, 0};

  for (int b = 0; b < blocks; ++b) {
    const int left = a.K ? a.K - b * FB - (int)fk * 32 : 32;     // bytes of the row from the lane's place on
    auto load = [&](const uint8_t* p, int64_t row_pitch, int64_t blk, int row, int n) {
      i32x8_t v = zero;
      const uint8_t* q = p + (int64_t)row * row_pitch + (int64_t)b * blk + fk * 32;
      if (row < n && left > 0) {
        const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(q);
        const i32x4_t hi = left > 16 ? *reinterpret_cast<const i32x4_t*>(q + 16) : i32x4_t{0, 0, 0, 0};
        v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
      return v;
    };
    i32x8_t fx[TM], fw[TN];
    float sx[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r = (int)(wm + 16 * i + frow);
      fx[i] = load(x, a.x_row, a.x_blk, r, rows);
      sx[i] = r < rows ? xs[(int64_t)b * a.xs_blk + r] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) fw[j] = load(w, a.w_row, a.w_blk, (int)(wn + 16 * j + frow), cols);
    const float sw = WROWS ? 1.0f : ws[(int64_t)b * a.ws_blk];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      f32x4_t swr = {1, 1, 1, 1};
      if constexpr (WROWS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = (int)(wn + 16 * j + 4 * fk) + e;
          swr[e] = r < cols ? ws[(int64_t)b * a.ws_blk + r] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const f32x4_t p = mfma_f8(fw[j], fx[i], f32x4_t{0, 0, 0, 0});
        const float s = sx[i] * sw;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(WROWS ? p[e] * swr[e] : p[e], s, acc[i][j][e]);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = (int)(wm + 16 * i + frow);
    if (r >= rows) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int c = (int)(wn + 16 * j + 4 * fk);
      const int64_t at = (MODE == G8_BLOCKS ? (int64_t)group * a.y_group : 0) + (int64_t)(m0 + r) * a.ldy + n0 + c;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c + e < cols) a.y[at + e] = (uint16_t)pack_bf16x2(acc[i][j][e], 0.0f);
      }
    }
  }
}

bool bad_codes(int64_t K, int64_t ld) { return K < 1 || K % 16 != 0 || ld < K || ld >= QF_FP8_MAX_COLS; }
constexpr int64_t G8_MAX_N = 1 << 22;

hipError_t launch(const Gemm8Args& a, int mode, int64_t wgs, hipStream_t s) {
  const dim3 g((unsigned)wgs);
  if (mode == G8_DENSE) k_gemm8<G8_DENSE><<<g, 256, 0, s>>>(a);
  else if (mode == G8_ROWS) k_gemm8<G8_ROWS><<<g, 256, 0, s>>>(a);
  else k_gemm8<G8_BLOCKS><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

// The forward product: rows of x (all, or those of a plan's groups) against w or each group's w.
qf_status forward(const uint8_t* Xc, int64_t ldx, const float* Xs, int64_t ldxs, const uint8_t* Wc, int64_t ldw,
                  const float* Ws, const int32_t* offsets, const int32_t* tiles, int n_ids, bool grouped, uint16_t* Y,
                  int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  if (M < 0 || M >= QF_ROW_MAX_ROWS || N < 0 || N >= G8_MAX_N || bad_codes(K, ldx) || bad_codes(K, ldw) || ldxs < M || ldy < N)
    return QF_ERR_SHAPE;
  if (grouped && (n_ids < 1 || n_ids > QF_ROW_MAX_IDS)) return QF_ERR_ARG;
  if (M == 0 || N == 0) return QF_OK;
  if (!Xc || !Xs || !Wc || !Ws || !Y || (grouped && (!offsets || !tiles))) return QF_ERR_NULL;
  if (misaligned(Xc, 16) || ldx % 16 || misaligned(Wc, 16) || ldw % 16 || misaligned(Xs, 4) || misaligned(Ws, 4) ||
      misaligned(Y, 2) || misaligned(offsets, 4) || misaligned(tiles, 8))
    return QF_ERR_ALIGN;
  Gemm8Args a = {};
  a.x = Xc;
  a.x_row = ldx;
  a.x_blk = FB;
  a.xs = Xs;
  a.xs_blk = ldxs;
  a.w = Wc;
  a.w_row = ldw;
  a.w_blk = FB;
  a.w_group = N * ldw;
  a.ws = Ws;
  a.blocks = (int32_t)((K + FB - 1) / FB);
  a.ws_tile = a.blocks;
  a.ws_blk = 1;
  a.ws_group = (N + FB - 1) / FB * a.blocks;
  a.y = Y;
  a.ldy = ldy;
  a.offsets = offsets;
  a.n_ids = n_ids;
  a.n = (int32_t)M;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  a.tiles_m = (int32_t)((M + 127) / 128 + (grouped ? (M < n_ids ? M : n_ids) : 0));
  a.tiles_n = (int32_t)((N + 127) / 128);
  const int64_t wgs = (int64_t)a.tiles_m * a.tiles_n;
  if (wgs > G8_MAX_WGS) return QF_ERR_SHAPE;
  return status_of(launch(a, grouped ? G8_ROWS : G8_DENSE, wgs, s));
}

}  // namespace
}  // namespace qf

using namespace qf;

extern "C" {

qf_status qf_gemm_fp8(const uint8_t* Xc, int64_t ldx, const float* Xs, int64_t ldxs, const uint8_t* Wc, int64_t ldw,
                      const float* Ws, uint16_t* Y, int64_t ldy, int64_t M, int64_t N, int64_t K, void* stream) {
  return forward(Xc, ldx, Xs, ldxs, Wc, ldw, Ws, nullptr, nullptr, 1, false, Y, ldy, M, N, K, (hipStream_t)stream);
}

qf_status qf_gemm_fp8_grouped(const uint8_t* Xc, int64_t ldx, const float* Xs, int64_t ldxs, const uint8_t* Wc, int64_t ldw,
                              const float* Ws, const int32_t* offsets, const int32_t* tiles, int n_ids, uint16_t* Y,
                              int64_t ldy, int64_t rows, int64_t N, int64_t K, void* stream) {
  return forward(Xc, ldx, Xs, ldxs, Wc, ldw, Ws, offsets, tiles, n_ids, true, Y, ldy, rows, N, K, (hipStream_t)stream);
}

qf_status qf_gemm_fp8_wgrad(const uint8_t* Dc, const float* Ds, const uint8_t* Xc, const float* Xs, const int32_t* offsets,
                            int n_ids, int64_t rows, uint16_t* dW, int64_t N, int64_t K, void* stream) {
  if (rows < 0 || rows >= QF_ROW_MAX_ROWS || N < 0 || N >= G8_MAX_N || K < 0 || K >= G8_MAX_N || N % 8 || K % 8) return QF_ERR_SHAPE;
  if (n_ids < 1 || n_ids > QF_ROW_MAX_IDS || (!offsets && n_ids != 1)) return QF_ERR_ARG;
  if (N == 0 || K == 0) return QF_OK;
  if (!dW || (rows > 0 && (!Dc || !Ds || !Xc || !Xs))) return QF_ERR_NULL;
  if (misaligned(Dc, 16) || misaligned(Xc, 16) || misaligned(Ds, 4) || misaligned(Xs, 4) || misaligned(dW, 16) || misaligned(offsets, 4))
    return QF_ERR_ALIGN;
  Gemm8Args a = {};
  a.x = Dc;
  a.x_row = FB;
  a.x_blk = N * FB;
  a.xs = Ds;
  a.xs_blk = N;
  a.w = Xc;
  a.w_row = FB;
  a.w_blk = K * FB;
  a.ws = Xs;
  a.ws_blk = K;
  a.y = dW;
  a.ldy = K;
  a.y_group = N * K;
  a.offsets = rows > 0 ? offsets : nullptr;
  a.n_ids = n_ids;
  a.n = (int32_t)rows;
  a.M = (int32_t)N;
  a.N = (int32_t)K;
  a.blocks = (int32_t)((rows + FB - 1) / FB);
  a.tiles_m = (int32_t)((N + 127) / 128);
  a.tiles_n = (int32_t)((K + 127) / 128);
  const int64_t wgs = (int64_t)n_ids * a.tiles_m * a.tiles_n;
  if (wgs > G8_MAX_WGS) return QF_ERR_SHAPE;
  return status_of(launch(a, G8_BLOCKS, wgs, (hipStream_t)stream));
}

}  // extern "C"
