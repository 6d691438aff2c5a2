// Host launch interface of the operators around the quantized layer: AdamW, row plans, adapters
// beside a product, routing.
#pragma once
#include "qf_kernels.h"

namespace qf {

// ----------------------------------------------------------------- AdamW ---
constexpr int AW_TENSORS = 48;      // tensors per launch: the descriptors stay below 4 KiB of kernel arguments
constexpr int AW_FEW = 8;           // up to this many take a shorter argument block

struct AdamwTensor {
  float* p;
  const void* g;          // fp32 or bf16
  void* m;                // fp32, or E4M3 codes with a scale per block in ms
  void* v;                // fp32, or E4M3 codes of sqrt(v) with a scale per block in vs
  float* ms;
  float* vs;
  uint16_t* p16;          // bf16 copy of p (null: none)
  double weight_decay;
  uint32_t n;
};

// What follows from the learning rate and the step number.
struct AdamwScalars {
  double lr;
  float size;             // lr / (1 - beta1^step)
  float root;             // 1 / sqrt(1 - beta2^step)
  uint32_t key;           // of the stochastic rounding's hash
};

struct AdamwCommon {
  double beta1, beta2, eps;
  int64_t step;
  uint32_t seed;
  AdamwScalars s;               // used unless d_lr or d_step is given
  const float* d_lr;
  const int64_t* d_step;
  const float* d_grad_scale;
  const uint32_t* skip;
};
template <int N>
struct AdamwArgs : AdamwCommon {
  static constexpr int TENSORS = N;
  uint32_t begin[N];            // first workgroup of each tensor; 0xFFFFFFFF past the last
  AdamwTensor t[N];
};
// The same for any number of tensors, in device memory.
struct AdamwTableArgs : AdamwCommon {
  const AdamwTensor* t;
  const uint32_t* begin;
  int n;
};

// -------------------------------------------------------------- row plan ---
constexpr int RP_ONE_LAUNCH = 16384;  // rows up to which every workgroup counts all of them itself
constexpr int RP_MAX_WG = 128;        // workgroups of a plan, at most
constexpr int RP_MIN_PER_WG = 2048;   // rows per workgroup, at least

struct RowPlanArgs {
  const int32_t* ids;
  int64_t n, per;          // rows, and rows per workgroup
  int32_t n_ids;
  int32_t* offsets;        // [n_ids + 1]
  int32_t* order;          // [n]
  int32_t* tiles;          // [n_tiles][2]
  int64_t n_tiles;
  uint32_t* hist;          // workspace [workgroups][n_ids rounded up to even] (null: one launch)
};
hipError_t launch_row_plan(RowPlanArgs a, hipStream_t s);

// ------------------------------------------------- adapters beside a product ---
// Rows up to which a call without a plan goes row by row: the whole adapter is read again for
// every row, so fewer of higher ranks, and none past rank 64 (an adapter then takes one workgroup
// longer than two more launches).  Microseconds row by row / plan and tiles, for 1 and for 64
// adapters: 4096 -> 6144 rank 16, 256 rows 9.2 / 15.0 and 13.6 / 18.9; rank 32, 128 rows, 4096 ->
// 4096 11.1 / 15.7 and 13.6 / 19.4, 4096 -> 14336 16.9 / 16.5 and 24.5 / 25.1 (256 rows 24.7 / 17.6
// and 39 / 28); 4096 -> 4096, rank 64, 64 rows 19.3 / 19.8 and 21.2 / 27.2, 96 rows 22.5 / 19.4 and
// 27.2 / 28.9; rank 128, 4 rows 28.8 / 23.5.
inline int lora_apply_few(int r) {
  return r > QF_LORA_APPLY_FEW_R ? 0 : r > 16 ? 16 * QF_LORA_APPLY_FEW / r : QF_LORA_APPLY_FEW;
}
constexpr int LORA_APPLY_MAX_SPLITS = 4;    // K parts

struct LoraApplyArgs {
  const uint16_t* X;
  const uint16_t* A;        // [n_adapters][r][K]
  const uint16_t* B;        // [n_adapters][N][r]
  const float* scale;       // [n_adapters] (null: 1)
  uint16_t* Y;
  int64_t ldx, ldy;
  const int32_t* ids;       // rows form
  const int32_t* offsets;   // tiles form: the row plan
  const int32_t* order;
  const int32_t* tiles;
  float* S;                 // tiles form: workspace [splits][positions][rpad]
  int32_t rows, rows_per_x, K, N, r, rpad, n_adapters, n_ids, splits, n_part;
};
inline int lora_apply_rpad(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }   // S's row length
int lora_apply_splits(int64_t tiles, int K);
hipError_t launch_lora_apply(LoraApplyArgs a, bool tiles, int64_t n_tiles, hipStream_t s);

// ----------------------------------------------------------------- routing ---
struct RouteArgs {
  const void* logits;       // fp32 or bf16 [T, ld]
  int64_t ld, T;
  const float* bias;
  int32_t* indices;         // [T, k]
  float* weights;           // [T, k]
  const float* dweights;    // backward
  void* dlogits;
  int64_t ldd;
  float scale;
  int32_t E, k, scoring, renorm, n_group, topk_group, group_top2;
};
hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t s);

}  // namespace qf
