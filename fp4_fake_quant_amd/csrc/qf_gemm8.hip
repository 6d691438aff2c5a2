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

constexpr int64_t G8_MAX_TILES = 1 << 22;
constexpr int G8_CUS = 256;
constexpr int G8_RUN = 4;                // tile rows that share their columns' w in a cache

// An operand: rows of `row` bytes pitch, blocks of 128 at `blk` bytes pitch.
struct Gemm8Args {
  const uint8_t *x, *w;
  int64_t x_row, x_blk, w_row, w_blk, w_group;
  const float *xs, *ws;
  int64_t xs_blk;                        // scales of x: [block][rows]
  int64_t ws_tile, ws_blk, ws_group;     // of w: tile scales [tile][block], or [block][rows] with ws_blk
  uint16_t* y;
  int64_t ldy, y_group;
  const int32_t *offsets, *tiles;
  int32_t n_ids, n;                      // groups and rows of the plan
  int32_t M, N, K;                       // K: elements of a row-major row (panels: 0, every block whole)
  int32_t blocks;                        // blocks of the reduction (grouped over blocks: from the offsets)
  int32_t tiles_m, tiles_n;
  int32_t most;                          // blocks that the panels hold, or tiles that a plan's groups make, at most
  int32_t y_vec;                         // rows of y take whole stores of 16 bytes (few rows: of 8); 2: past the caches
};
enum { G8_DENSE, G8_ROWS, G8_BLOCKS };   // over what the groups go

__device__ __forceinline__ f32x4_t mfma_f8(i32x8_t a, i32x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------------ tiles ---
// BM x BN outputs by WM x WN waves of 16 TM x 16 TN each.  A step is one block of 128: its codes go from
// memory straight into LDS (buffer loads that write LDS, 16 bytes a lane: a wave's instruction fills
// eight rows of 128 bytes), with the block's scales of the tile's rows behind them.  Two stages: while
// one is computed from, the next is on its way, and its place is refilled as soon as every wave has read
// its last fragments.
//
// 256 x 256 (two stages of 66 KiB, one workgroup per CU, two waves per SIMD, 228 to 255 registers): per step and wave
// 32 products, 128 sums (256 where w has a scale per row) and 24 reads of 16 bytes.  32768 x 14336 x 4096 takes 1.70 ms
// (2.26 PFLOP/s; 1.68 to 1.81 by card; a library product with one scale per tensor 1.27 ms): the matrix cores are busy 54% of 1.96 GHz,
// which is what the card's power leaves of 2.4, and the 940 MB of results, which all workgroups write at the same time, take
// 0.18 ms of it (1.52 ms per 4096 of K without).  On the way: fragments straight from memory 6.99 ms; LDS with two
// barriers a step 2.07; sums between the products and reads without conflicts 1.99; one barrier 1.89; workgroups that stay
// 1.72.  Runs of 4 tile rows: 1 / 2 / 4 / 8 / 16 / 32 take 1.88 / 1.84 / 1.82 / 1.83 / 1.86 / 1.92 ms (before the last step).
// 64 groups of about 512 rows, 4096 -> 4096, take 0.70 ms (1.57 PFLOP/s): a group's last tile is half empty.  Weight
// gradients of 64 groups, 2048 x 2048, take 0.27 to 0.30 ms: 4 or 5 steps a tile, then 537 MB of results.
// 128 x 128 (four waves, two workgroups per CU) is for products of fewer than 1024 such tiles, which 256 x 256 would leave
// CUs without: the large product takes 2.07 ms in it, 512 x 2048 x 2048 14 us.
template <int BM, int BN>
struct Stage {
  static constexpr int W = BM * FB, XS = W + BN * FB, WS = XS + BM * 4, BYTES = WS + BN * 4;
};
// The 16-byte chunk c of a row lies at c ^ (row / 2) % 8, so that 16 lanes reading one chunk of 16 rows meet
// 16 different places of 256 bytes.
__device__ __forceinline__ uint32_t g8_chunk(uint32_t row, uint32_t c) { return row * FB + ((c ^ ((row >> 1) & 7u)) << 4); }

// Waits until at most n vector-memory operations of this wave are in flight, and for its LDS reads.
#define G8_WAIT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (0 << 8))
// Workgroup barrier that leaves loads in flight (a __syncthreads() would wait for all); the empty asm
// keeps the compiler from moving LDS accesses across it.
#define G8_BARRIER()                 \
  do {                               \
    asm volatile("" ::: "memory");   \
    __builtin_amdgcn_s_barrier();    \
    asm volatile("" ::: "memory");   \
  } while (0)

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// Values that are the same in all lanes, kept in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)uniform((int)v) | ((int64_t)uniform((int)(v >> 32)) << 32);
}
template <typename T>
__device__ __forceinline__ T* uniform(T* p) { return (T*)uniform((int64_t)p); }

// A tile of outputs: its first row and column, how many of each there are, its group.
struct TileAt {
  int m0, rows, n0, cols, group, blocks;
};

// Workgroups stay: each takes tiles of its XCD's run one after another, and the blocks of all its tiles are
// one stream of steps, so that the next tile's first operands are on their way while a tile's last
// products are formed and its results leave through LDS (the stage that the last step has freed).
template <int MODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_gemm8(Gemm8Args a) {
  constexpr int WAVES = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr bool WROWS = MODE == G8_BLOCKS;                  // w has a scale per row and block
  constexpr int XW = BM / 8 / WAVES, WW = BN / 8 / WAVES;    // LDS windows (eight rows) that a wave fills per step
  static_assert(BM / 64 + BN / 64 == WAVES, "one window of 64 scales per wave");
  static_assert(XW % 2 == 0 && WW % 2 == 0, "the parity of a window is that of its index in the wave");
  using S = Stage<BM, BN>;
  constexpr int PASSES = (BM * BN * 2 + S::BYTES - 1) / S::BYTES;      // in which a tile leaves through a stage
  static_assert(PASSES == 1 || PASSES == WM, "a pass takes the rows of one row of waves, or all");
  // (one array: with a second one the compiler waits for all loads in flight before it reads either)
  constexpr int LDS = 2 * S::BYTES + (MODE == G8_DENSE ? 0 : (int)sizeof(GroupTable));
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  GroupTable& table = *reinterpret_cast<GroupTable*>(lds + (MODE == G8_DENSE ? 0 : 2 * S::BYTES));

  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t frow = lane & 15, fk = lane >> 4;
  const uint32_t wm = wave / WN, wn = wave % WN;

  // tiles of this workgroup: t, t + step, ... below end, inside its XCD's run
  uint32_t tiles_m = (uint32_t)a.tiles_m, tiles_n = (uint32_t)a.tiles_n;
  if (MODE != G8_DENSE && a.offsets) {
    group_table(table, a.offsets, a.n_ids, a.n, MODE == G8_ROWS ? BM : FB, WAVES);
    if (MODE == G8_ROWS) tiles_m = min((uint32_t)uniform((int)table.pre[a.n_ids]), (uint32_t)a.most);
  }
  const uint32_t total = tiles_m * tiles_n * (MODE == G8_BLOCKS ? (uint32_t)a.n_ids : 1u);
  const uint32_t xcd = blockIdx.x & 7;
  const uint32_t first = xcd * (total >> 3) + min(xcd, total & 7u);
  const uint32_t end = first + (total >> 3) + (xcd < (total & 7u) ? 1u : 0u);
  const uint32_t step = (gridDim.x - xcd + 7) >> 3;
  auto tile_at = [&](uint32_t t, int& block0) {
    TileAt o;
    o.group = 0;
    block0 = 0;
    int blocks = a.blocks;
    if (MODE == G8_BLOCKS) {
      o.group = (int)(t / (tiles_m * tiles_n));
      t -= (uint32_t)o.group * tiles_m * tiles_n;
      if (a.offsets) {
        block0 = min(uniform((int)table.pre[o.group]), a.most);
        blocks = min(uniform((int)table.pre[o.group + 1]), a.most) - block0;
      }
    }
    // runs of G8_RUN tile rows, column by column
    const uint32_t run = t / (G8_RUN * tiles_n), in_run = t - run * (G8_RUN * tiles_n);
    const uint32_t deep = min(tiles_m - run * G8_RUN, (uint32_t)G8_RUN);
    const uint32_t tn = in_run / deep, tm = run * G8_RUN + in_run - tn * deep;
    o.m0 = (int)tm * BM;
    o.rows = min(BM, a.M - o.m0);
    if (MODE == G8_ROWS) {
      const GroupUnit g = unit_at(table, a.n_ids, BM, tm);
      o.group = g.group;
      o.m0 = g.first;
      o.rows = g.rows;
    }
    o.n0 = uniform((int)tn * BN);
    o.cols = uniform(min(BN, a.N - o.n0));
    o.m0 = uniform(o.m0);
    o.rows = uniform(o.rows);
    o.group = uniform(o.group);
    o.blocks = uniform(blocks);
    return o;
  };
  auto out_of = [&](const TileAt& o) {
    return a.y + (MODE == G8_BLOCKS ? (int64_t)o.group * a.y_group : 0) + (int64_t)o.m0 * a.ldy + o.n0;
  };

  // ---- loads: a cursor that runs two blocks ahead of the products ----
  // the lane's place in window i of its wave: row lane / 8 of its eight, chunk (lane % 8) ^ swizzle, which
  // goes by the parity of the window
  const uint32_t xrow = (8 * XW * wave + (lane >> 3)) * (uint32_t)a.x_row, wrow = (8 * WW * wave + (lane >> 3)) * (uint32_t)a.w_row;
  const uint32_t chunk = ((lane & 7) ^ (lane >> 4)) * 16;      // even windows; odd ones: chunk ^ 64
  // scales: wave i fills window i of 64 of the BM + BN words behind the codes: x's rows, then w's rows, or
  // w's tiles (in the first of these windows alone)
  const bool for_x = wave < BM / 64;
  const uint32_t sr = for_x ? 64 * wave : 64 * wave - BM;
  const uint32_t soff = for_x || WROWS ? (sr + lane) * 4 : sr == 0 && lane < BN / FB ? lane * (uint32_t)a.ws_tile * 4 : BUF_OOR;
  const int64_t sstep = for_x ? a.xs_blk : a.ws_blk;
  uint32_t next_t = first + (blockIdx.x >> 3);
  const uint8_t *x = nullptr, *w = nullptr;
  const float* sbase = nullptr;
  int64_t xbytes = 0, wbytes = 0, sbytes = 0;
  int at = 0, last = 0;                                       // blocks of the cursor's tile: next one, behind the last
  // tiles begun and not yet stored: the products' own and, at most, the one behind it (the last one opened:
  // a tile is stored before the second one behind it is begun)
  int n_m0 = 0, n_rows = 0, n_n0 = 0, n_cols = 0, n_group = 0, n_blocks = 0;
  int held = 0;
  // the next tile with blocks, if there is one; tiles without (a group without rows) become zeros at once
  auto open = [&]() {
    while (next_t < end) {
      int block0;
      const TileAt o = tile_at(next_t, block0);
      next_t = (uint32_t)uniform((int)(next_t + step));
      if (MODE == G8_BLOCKS && o.blocks == 0) {
        uint16_t* y = out_of(o);
        for (int i = threadIdx.x; i < o.rows * (BN / 4); i += 64 * WAVES) {
          const int r = i / (BN / 4), c = i % (BN / 4) * 4;
          if (c < o.cols) *reinterpret_cast<uint2*>(y + (int64_t)r * a.ldy + c) = make_uint2(0, 0);
        }
        continue;
      }
      x = uniform(a.x + (int64_t)o.m0 * a.x_row + (int64_t)block0 * a.x_blk);
      w = uniform(a.w + (WROWS ? 0 : (int64_t)o.group * a.w_group) + (int64_t)o.n0 * a.w_row + (int64_t)block0 * a.w_blk);
      const float* xs = a.xs + o.m0 + (int64_t)block0 * a.xs_blk;
      const float* ws = WROWS ? a.ws + o.n0 + (int64_t)block0 * a.ws_blk
                              : a.ws + (int64_t)o.group * a.ws_group + (int64_t)(o.n0 / FB) * a.ws_tile;
      sbase = uniform(for_x ? xs : ws);
      sbytes = for_x ? (int64_t)o.rows * 4 : WROWS ? (int64_t)o.cols * 4 : ((int64_t)((o.cols - 1) / FB) * a.ws_tile + 1) * 4;
      // a row of a row-major operand ends at K, inside the last block; what lies behind must read as zeros
      xbytes = (int64_t)(o.rows - 1) * a.x_row + (WROWS ? FB : a.K);
      wbytes = (int64_t)(o.cols - 1) * a.w_row + (WROWS ? FB : a.K);
      at = 0;
      last = o.blocks;
      n_m0 = o.m0;
      n_rows = o.rows;
      n_n0 = o.n0;
      n_cols = o.cols;
      n_group = o.group;
      n_blocks = o.blocks;
      ++held;
      return;
    }
  };
  auto issue = [&](uint8_t* st) {
    if (at == last) open();
    if (at == last) return;                                   // no tile is left
    const int64_t bx = WROWS ? 0 : (int64_t)at * FB;          // what a row-major row has behind it
    const uint32_t left = WROWS ? (uint32_t)FB : (uint32_t)(a.K - at * FB);
    const __amdgpu_buffer_rsrc_t rx = make_buf(x + (int64_t)at * a.x_blk, xbytes - bx);
    const __amdgpu_buffer_rsrc_t rw = make_buf(w + (int64_t)at * a.w_blk, wbytes - bx);
    const __amdgpu_buffer_rsrc_t rs = make_buf(sbase + (int64_t)at * sstep, sbytes);
    ++at;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(st + S::XS + wave * 256), 4, soff, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < XW; ++i) {
      const uint32_t c = chunk ^ (i & 1 ? 64 : 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(st + (XW * wave + i) * 1024), 16,
                                               c < left ? xrow + c + i * 8 * (uint32_t)a.x_row : BUF_OOR, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < WW; ++i) {
      const uint32_t c = chunk ^ (i & 1 ? 64 : 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(st + S::W + (WW * wave + i) * 1024), 16,
                                               c < left ? wrow + c + i * 8 * (uint32_t)a.w_row : BUF_OOR, 0, 0, 0);
    }
  };

  // ---- products ----
  auto frag = [&](const uint8_t* base, uint32_t row) {
    const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(base + g8_chunk(row, fk));
    const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(base + g8_chunk(row, fk + 4));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto read_w = [&](const uint8_t* st, int j) { return frag(st + S::W, (wn * TN + j) * 16 + frow); };
  auto read_x = [&](const uint8_t* st, int i) { return frag(st, (wm * TM + i) * 16 + frow); };
  auto read_sx = [&](const uint8_t* st, int i) { return *reinterpret_cast<const float*>(st + S::XS + ((wm * TM + i) * 16 + frow) * 4); };
  auto read_sw = [&](const uint8_t* st) { return WROWS ? 1.0f : *reinterpret_cast<const float*>(st + S::WS + (wn * TN * 16 / FB) * 4); };

  issue(lds);
  if (held == 0) return;
  int c_m0 = n_m0, c_rows = n_rows, c_n0 = n_n0, c_cols = n_cols, c_group = n_group, left = n_blocks;
  issue(lds + S::BYTES);
  G8_WAIT(0);
  G8_BARRIER();
  i32x8_t fw[TN], fx[2];
  f32x4_t acc[TM][TN], p[TN], swr[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    fw[j] = read_w(lds, j);
    p[j] = swr[j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[i][j] = f32x4_t{0, 0, 0, 0};
  }
  fx[0] = read_x(lds, 0);
  float sw = read_sw(lds), sx = read_sx(lds, 0), before = 0.0f;        // before: scale of the row before
  auto add = [&](int i, int j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(WROWS ? p[j][e] * swr[j][e] : p[j][e], before, acc[i][j][e]);
    asm volatile("" : "+v"(acc[i][j]));                      // the sum stays here, beside the next products
  };
  uint32_t parity = 0;
  // Row i of the wave's tiles: its products (operands read a row earlier), and beside each the sum of the
  // row before, whose products are done by then.  The last row of a step waits for the next stage, passes
  // the step's one barrier (this stage is read, the next has landed), refills this stage and reads the
  // next step's first operands, so that the matrix cores go on over the step's end.
#pragma unroll 1
  while (true) {
    uint8_t* st;
#pragma unroll 1
    do {
    st = lds + parity * S::BYTES;
    const uint8_t* next = lds + (parity ^ 1) * S::BYTES;
    --left;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const float s = sx * sw;
      if (i == TM - 1) {
        G8_WAIT(0);
        G8_BARRIER();
        if (left > 0) issue(st);
      }
      fx[(i + 1) & 1] = i + 1 < TM ? read_x(st, i + 1) : read_x(next, 0);
      sx = i + 1 < TM ? read_sx(st, i + 1) : read_sx(next, 0);
      if (i == TM - 1) sw = read_sw(next);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        add((i + TM - 1) % TM, j);
        p[j] = mfma_f8(fw[j], fx[i & 1], f32x4_t{0, 0, 0, 0});
        if (i == TM - 1) fw[j] = read_w(next, j);
        if constexpr (WROWS)
          if (i == 0) swr[j] = *reinterpret_cast<const f32x4_t*>(st + S::WS + ((wn * TN + j) * 16 + 4 * fk) * 4);
        __builtin_amdgcn_sched_barrier(0);
      }
      before = s;
    }
    parity ^= 1;
    } while (left > 0);

    // ---- the tile is done ----
    // (the lane's number is made anew, so that no address of the epilogue takes a register in the loop)
    uint32_t tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const uint32_t erow = tid & 15, ek = (tid >> 4) & 3;
#pragma unroll
    for (int j = 0; j < TN; ++j) add(TM - 1, j);
    const TileAt o = {c_m0, c_rows, c_n0, c_cols, c_group, 0};
    uint16_t* y = out_of(o);
    // 16-byte chunk c of a row lies at c ^ row: rows written by one instruction, and the chunks of a row
    // read back, meet different banks.  (The accesses are written out: the compiler would let each of them
    // wait for the stores before it, as it does not tell those from loads that write LDS.)
    constexpr uint32_t CH = BN / 8, ROWS = BM / PASSES, EACH = ROWS * CH / (64 * WAVES);
    static_assert(EACH == 8, "read back by one instruction sequence");
    const __amdgpu_buffer_rsrc_t ry = make_buf(y, ((int64_t)(o.rows - 1) * a.ldy + o.cols) * 2);
    const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr_t)st;
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      if (PASSES == 1 || (int)wm == pass) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const uint32_t r = (PASSES == 1 ? wm * TM * 16 : 0) + i * 16 + erow;
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const uint32_t c = (wn * TN + j) * 2 + (ek >> 1);
            const uint2 v = make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
            asm volatile("ds_write_b64 %0, %1" ::"v"(base + r * (BN * 2) + ((c ^ (r & (CH - 1))) << 4) + (ek & 1) * 8),
                         "v"(__builtin_bit_cast(uint64_t, v))
                         : "memory");
          }
        }
      }
      G8_WAIT(63);
      G8_BARRIER();
      // thread u of the workgroup: chunk u % CH of rows u / CH + k 64 WAVES / CH; the row's swizzle goes with k only
      // above CH
      const uint32_t r0 = tid / CH, c0 = tid % CH;
      constexpr uint32_t DOWN = 64 * WAVES / CH;
      u32x4_t v[EACH];
      uint32_t from[EACH];
#pragma unroll
      for (uint32_t k = 0; k < EACH; ++k) {
        const uint32_t r = r0 + k * DOWN;
        from[k] = base + r * (BN * 2) + ((c0 ^ (r & (CH - 1))) << 4);
      }
      asm volatile(
          "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\tds_read_b128 %3, %11\n\t"
          "ds_read_b128 %4, %12\n\tds_read_b128 %5, %13\n\tds_read_b128 %6, %14\n\tds_read_b128 %7, %15\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
          : "v"(from[0]), "v"(from[1]), "v"(from[2]), "v"(from[3]), "v"(from[4]), "v"(from[5]), "v"(from[6]), "v"(from[7])
          : "memory");
      const int c = (int)(8 * c0);
      if (a.y_vec) {
        auto store = [&](auto nt) {
#pragma unroll
          for (uint32_t k = 0; k < EACH; ++k) {
            const uint32_t row = pass * ROWS + r0 + k * DOWN;
            const uint32_t at = (int)row < o.rows && c < o.cols ? (row * (uint32_t)a.ldy + (uint32_t)c) * 2 : BUF_OOR;
            __builtin_amdgcn_raw_buffer_store_b128(v[k], ry, (int)at, 0, decltype(nt)::value ? 2 : 0);
          }
        };
        if (a.y_vec == 2) store(std::true_type());
        else store(std::false_type());
      } else {                                                // rows off 16 bytes, or of any length
#pragma unroll
        for (uint32_t k = 0; k < EACH; ++k) {
          const uint32_t row = pass * ROWS + r0 + k * DOWN;
          uint16_t* yr = y + (int64_t)row * a.ldy + c;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((int)row < o.rows && c + e < o.cols) yr[e] = (uint16_t)(v[k][e >> 1] >> (16 * (e & 1)));
        }
      }
      G8_BARRIER();
    }
    if (--held == 0) return;
    c_m0 = n_m0, c_rows = n_rows, c_n0 = n_n0, c_cols = n_cols, c_group = n_group;
    left = n_blocks;
    issue(st);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      p[j] = swr[j] = f32x4_t{0, 0, 0, 0};                    // (the scales too: 0 times a NaN of this tile is one in the next)
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[i][j] = f32x4_t{0, 0, 0, 0};
    }
    before = 0.0f;
  }
}

// --------------------------------------------------------------- few rows ---
// Up to 16 MT rows: the product streams w once, so the work is split over its columns (16 NJ a workgroup)
// and over the blocks of the reduction, which the workgroup's waves take in turn and join in LDS in a
// fixed order.  Operands go from memory into registers, several blocks ahead.  Bound by the bytes of w where
// there are enough of them (61 tokens to 8 of 128 experts of 2048 -> 1536: 64 us, 6.2 TB/s; 16 rows of 4096 -> 28672 26 us,
// 4.4 TB/s), else by the call (7 rows of 4096 -> 6144: 8.4 to 8.7 us, kernel 7.7 to 8.1 traced), and with more rows by x, which every
// workgroup reads from the caches.
constexpr int FEW_WAVES = 8;

template <int MT, int NJ>
__device__ __forceinline__ void few_rows(const Gemm8Args& a, int group, int m0, int rows, float* lds) {
  constexpr int DEEP = MT + NJ <= 2 ? 4 : MT + NJ <= 4 ? 3 : 2;        // blocks in flight: 8 (MT + NJ) registers each
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t frow = lane & 15, fk = lane >> 4;
  const int n0 = (int)blockIdx.x * 16 * NJ, cols = min(16 * NJ, a.N - n0);
  const uint8_t* x = a.x + (int64_t)m0 * a.x_row;
  const uint8_t* w = a.w + (int64_t)group * a.w_group + (int64_t)n0 * a.w_row;
  const __amdgpu_buffer_rsrc_t rx = make_buf(x, (int64_t)(rows - 1) * a.x_row + a.K);
  const __amdgpu_buffer_rsrc_t rw = make_buf(w, (int64_t)(cols - 1) * a.w_row + a.K);
  const float* ws = a.ws + (int64_t)group * a.ws_group + (int64_t)(n0 / FB) * a.ws_tile;
  f32x4_t acc[MT][NJ];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};

  for (int b0 = (int)wave; b0 < a.blocks; b0 += FEW_WAVES * DEEP) {
    i32x8_t fw[DEEP][NJ], fx[DEEP][MT];
    float sx[DEEP][MT], sw[DEEP];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int b = b0 + d * FEW_WAVES;
      // chunks fk and fk + 4 of the row's 128 bytes; what lies behind K (and every block behind the last) reads as zeros
      const uint32_t k0 = (uint32_t)b * FB + fk * 16, k1 = k0 + 64;
      auto load = [&](__amdgpu_buffer_rsrc_t r, uint32_t row) {
        const uint4 lo = buf_load16(r, k0 < (uint32_t)a.K ? row + k0 : BUF_OOR), hi = buf_load16(r, k1 < (uint32_t)a.K ? row + k1 : BUF_OOR);
        return __builtin_shufflevector(__builtin_bit_cast(i32x4_t, lo), __builtin_bit_cast(i32x4_t, hi), 0, 1, 2, 3, 4, 5, 6, 7);
      };
#pragma unroll
      for (int j = 0; j < NJ; ++j) fw[d][j] = load(rw, (16 * j + frow) * (uint32_t)a.w_row);
#pragma unroll
      for (int i = 0; i < MT; ++i) fx[d][i] = load(rx, (16 * i + frow) * (uint32_t)a.x_row);
      const int bs = min(b, a.blocks - 1);
      sw[d] = ws[bs * a.ws_blk];
#pragma unroll
      for (int i = 0; i < MT; ++i) sx[d][i] = a.xs[(int64_t)bs * a.xs_blk + m0 + min((int)(16 * i + frow), rows - 1)];
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      if (b0 + d * FEW_WAVES >= a.blocks) break;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const float s = sx[d][i] * sw[d];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const f32x4_t p = mfma_f8(fw[d][j], fx[d][i], f32x4_t{0, 0, 0, 0});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], s, acc[i][j][e]);
        }
      }
    }
  }
  // [wave][tile][lane]; the tiles are then dealt to the waves
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      *reinterpret_cast<f32x4_t*>(lds + ((wave * MT * NJ + i * NJ + j) * 64 + lane) * 4) = acc[i][j];
  __syncthreads();
  for (int u = (int)wave; u < MT * NJ; u += FEW_WAVES) {
    f32x4_t y = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < FEW_WAVES; ++v) y += *reinterpret_cast<const f32x4_t*>(lds + ((v * MT * NJ + u) * 64 + lane) * 4);
    const int r = 16 * (u / NJ) + (int)frow, c = 16 * (u % NJ) + 4 * (int)fk;
    uint16_t* o = a.y + (int64_t)(m0 + r) * a.ldy + n0 + c;
    const uint32_t lo = pack_bf16x2(y[0], y[1]), hi = pack_bf16x2(y[2], y[3]);
    if (r >= rows) continue;
    if (a.y_vec && c + 3 < cols) {
      *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
    } else {
      const uint16_t v[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < cols) o[e] = v[e];
    }
  }
}

// MT: 16-row tiles at most (grouped: of the plan's tiles of QF_ROW_TILE rows; those with up to 16 rows take
// half).
template <int MODE, int MT, int NJ>
__global__ __launch_bounds__(64 * FEW_WAVES, 2) void k_gemm8_few(Gemm8Args a) {
  __shared__ __attribute__((aligned(16))) float lds[FEW_WAVES * MT * NJ * 256];
  if (MODE == G8_DENSE) {
    const int m0 = (int)blockIdx.y * 16 * MT;
    few_rows<MT, NJ>(a, 0, m0, min(16 * MT, a.M - m0), lds);
    return;
  }
  const int group = uniform(a.tiles[2 * (int64_t)blockIdx.y]), m0 = uniform(a.tiles[2 * (int64_t)blockIdx.y + 1]);
  if (group < 0 || group >= a.n_ids || m0 < 0) return;
  const int rows = uniform(min(QF_ROW_TILE, group_offset(a.offsets, group + 1, a.n) - m0));
  if (rows <= 0) return;
  if (MT > 1 && rows > 16) few_rows<MT, NJ>(a, group, m0, rows, lds);
  else few_rows<1, NJ>(a, group, m0, rows, lds);
}

bool bad_codes(int64_t K, int64_t ld) { return K < 1 || K % 16 != 0 || ld < K || ld >= QF_FP8_MAX_COLS; }
constexpr int64_t G8_MAX_N = 1 << 22;

template <int BM, int BN, int WM, int WN>
hipError_t launch_tiles(Gemm8Args a, int mode, hipStream_t s) {
  a.tiles_m = (int32_t)((a.M + BM - 1) / BM);
  a.tiles_n = (int32_t)((a.N + BN - 1) / BN);
  // at most as many workgroups as the chip holds at once
  if (mode == G8_ROWS) a.most = a.tiles_m + (a.M < a.n_ids ? a.M : a.n_ids);
  const int64_t tiles = (mode == G8_ROWS ? a.most : a.tiles_m) * (int64_t)a.tiles_n * (mode == G8_BLOCKS ? a.n_ids : 1);
  const int64_t most = G8_CUS * (160 * 1024 / (2 * Stage<BM, BN>::BYTES));
  const dim3 g((unsigned)(tiles < most ? tiles : most)), wg(64 * WM * WN);
  if (mode == G8_DENSE) k_gemm8<G8_DENSE, BM, BN, WM, WN><<<g, wg, 0, s>>>(a);
  else if (mode == G8_ROWS) k_gemm8<G8_ROWS, BM, BN, WM, WN><<<g, wg, 0, s>>>(a);
  else k_gemm8<G8_BLOCKS, BM, BN, WM, WN><<<g, wg, 0, s>>>(a);
  return hipGetLastError();
}

// 128 x 128 tiles of a product (of all its groups together, at most).
int64_t small_tiles(const Gemm8Args& a, int mode) {
  const int64_t m = (a.M + 127) / 128 + (mode == G8_ROWS ? (a.M < a.n_ids ? a.M : a.n_ids) : 0);
  return m * ((a.N + 127) / 128) * (mode == G8_BLOCKS ? a.n_ids : 1);
}

template <int MODE, int MT>
hipError_t launch_few(Gemm8Args a, int64_t tiles, int64_t likely, int nj, hipStream_t s) {
  a.y_vec = a.ldy % 4 == 0 && (uintptr_t)a.y % 8 == 0;
  // wide workgroups read x less often; narrower ones share the work out as long as each has a CU to itself (the next
  // one on a CU waits for the first's loads).  Microseconds with 16 / 32 / 64 columns, w from memory: 16 rows of 4096 -> 4096
  // (256 / 128 / 64 workgroups) 7.5 / 9.2 / 12.8, -> 5120 (320 / 160 / 80) 11.4 / 9.4 / 12.9, -> 8192 12.0 / 10.9 / 13.3,
  // -> 10240 14.6 / 15.9 / 13.7, -> 28672 31.9 / 30.3 / 27.5; 64 rows -> 4096 12.9 / 15.1 / 19.2, -> 5120 22.6 / 15.3 / 19.4,
  // -> 10240 31.5 / 26.5 / 20.2; 14336 -> 5120 with 16 rows 31.5 / 25.2 / 36.8; 8 groups of 16 rows of 2048 -> 512 5.0 / 6.0 /
  // 7.7, -> 1024 7.8 / 6.7 / 8.3, -> 1536 9.3 / 9.5 / 8.4.  (One row alone, 4096 -> 5120: 8.3 / 8.6 / 11.8.)
  while (nj > 1 && (a.N + 8 * nj - 1) / (8 * nj) * likely <= G8_CUS) nj /= 2;
  const dim3 g((unsigned)((a.N + 16 * nj - 1) / (16 * nj)), (unsigned)tiles), wg(64 * FEW_WAVES);
  if (nj == 4) k_gemm8_few<MODE, MT, 4><<<g, wg, 0, s>>>(a);
  else if (nj == 2) k_gemm8_few<MODE, MT, 2><<<g, wg, 0, s>>>(a);
  else k_gemm8_few<MODE, MT, 1><<<g, wg, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch(Gemm8Args a, int mode, hipStream_t s) {
  // Few rows stream w with columns and blocks split, 64 rows at a time; more take tiles, which need about a microsecond
  // a block however few they are.  Microseconds few / tiles: 64 rows of 4096 -> 6144 15.0 / 31.5, 14336 -> 4096 35 / 106; 128
  // rows of 4096 -> 6144 19 / 31, 192 35 / 32, 128 of 4096 -> 28672 72 / 38; 256 of 14336 -> 4096 55 / 106, 512 106 / 106; 512
  // of 2048 -> 2048 11.3 / 14.4; 128 groups of 2048 -> 1536 with 16 rows each 78 / 93, with 32 109 / 97; groups with 4 rows
  // in 16 / 32 / 64 columns a workgroup 73 / 66 / 70, with 16 rows 106 / 88 / 78.
  // From 33 rows on the border lies where the workgroups of 64 columns no longer fit the CUs: over one round a CU for
  // several parts (128 rows of 4096 -> 8192 20.0 / 33.9, -> 10240 36.1 / 34.4, of 14336 59 / 110, 109 / 111), over two for
  // 33 to 64 rows (64 rows of 2048 -> 16384 12.2 / 19.1, -> 28672 22.3 / 20.8, -> 45056 32.4 / 25.3, -> 65536 43.4 / 30.3; of
  // 4096 -> 16384 21.9 / 35.2, -> 32768 41.0 / 42.3, -> 45056 59.4 / 49.9, -> 65536 79.6 / 69.4; of 14336 -> 32768 122 / 125, ->
  // 45056 175 / 145).  Up to 32 rows they stay ahead (32 rows of 2048 -> 65536 30.8 / 29.6, 4096 -> 65536 59 / 68).
  if (mode == G8_DENSE) {
    const int64_t parts = (a.M + 63) / 64, wgs = parts * ((a.N + 63) / 64);
    if (a.M <= 16) return launch_few<G8_DENSE, 1>(a, 1, 1, 4, s);
    if (a.M <= 32) return launch_few<G8_DENSE, 2>(a, 1, 1, 4, s);
    if (parts <= 8 && wgs <= (parts == 1 ? 2 : 1) * G8_CUS) return launch_few<G8_DENSE, 4>(a, parts, parts, 4, s);
  }
  // Groups go by their mean, as their sizes are on the device: few / tiles of 1536 rows of 2048 -> 4096 evenly in 64 groups
  // 117 / 137, with half of them in one 132 / 161, with all 73 / 32; 2048 rows of 2048 -> 1536 in 128 groups 80 / 102, 93 / 123, 39 / 31.
  const int64_t groups = a.M < a.n_ids ? a.M : a.n_ids;
  if (mode == G8_ROWS && a.M <= 24 * (int64_t)a.n_ids)
    return launch_few<G8_ROWS, 2>(a, (a.M + QF_ROW_TILE - 1) / QF_ROW_TILE + groups, groups, a.M < 8 * (int64_t)a.n_ids ? 2 : 4, s);
  a.y_vec = a.ldy % 8 == 0 && (uintptr_t)a.y % 16 == 0 && a.N % 8 == 0 && a.ldy < QF_FP8_MAX_COLS;
  // through the caches / past them: 32768 x 14336 x 4096 1.73 / 1.70 ms; 32768 rows of 2048 -> 4096 for 16 groups 305 / 287 us
  // (with the sum over a token's four rows that follows 360 / 341), half the rows 166 / 154 (188 / 185), a quarter 92 / 91 (107 / 109)
  if (a.y_vec && (int64_t)a.M * a.N * 2 * (mode == G8_BLOCKS ? a.n_ids : 1) >= NT_ROWS_BYTES) a.y_vec = 2;
  // 128 / 256, codes drawn evenly: weight gradients of 64 groups of 512 rows, 2048 x 2048, 244 / 210 us, of 128 rows 113 / 109,
  // of 64 groups of 1024 x 1024 61 / 62, one of 8192 rows, 4096 x 4096 (1024 tiles), 166 / 150, 512 rows, 14336 x 4096, 54 / 56;
  // rows of 64 groups 4096 -> 4096, 512 a group 680 / 544, 300 494 / 498, 200 352 / 290, but 128 248 / 269; 8 groups of 256 rows
  // 2048 -> 2048 (384 tiles) 19 / 32
  if (small_tiles(a, mode) >= 1024) return launch_tiles<256, 256, 2, 4>(a, mode, s);
  return launch_tiles<128, 128, 2, 2>(a, mode, s);
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
  a.tiles = tiles;
  a.n_ids = n_ids;
  a.n = (int32_t)M;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  const int mode = grouped ? G8_ROWS : G8_DENSE;
  if (small_tiles(a, mode) > G8_MAX_TILES) return QF_ERR_SHAPE;
  return status_of(launch(a, mode, s));
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
  a.most = (int32_t)qf_fp8_panels(rows, n_ids);
  if (small_tiles(a, G8_BLOCKS) > G8_MAX_TILES) return QF_ERR_SHAPE;
  return status_of(launch(a, G8_BLOCKS, (hipStream_t)stream));
}

}  // extern "C"
