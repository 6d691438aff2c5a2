// Routing of tokens to experts: scores, selection, weights, and their gradient.
//
// A row (token) is held by L lanes of one wave, V consecutive logits each, so that an index
// order is a lane order, and one wave works on 64 / L rows.
//
// What is compared decides the chosen experts, and a tie decided by rounding would choose
// differently from one implementation to the next.  Without a bias (and with groups ranked by
// their best expert) both scorings are increasing in the logit, so the logits themselves are
// compared: exact.  Otherwise scores plus bias are compared as if in 64 bits.
//
// Both are done twice at most.  The fast pass orders 31-bit integer keys: the leading bits of
// the fp32 value, and below them the place in the lane, so that the largest key below the
// last choice takes one subtraction and half a maximum per logit and nothing has to be
// removed.  It knows when it cannot tell: two neighbours in the order whose values are closer
// than the key's truncation and the fp32 score's error bound.  Only then does the wave select
// again, on the fp32 logits themselves or on 64-bit scores.  bf16 logits fit a key with their
// index and need no second pass.  The selection is bounded by vector instructions (k + 1 rounds
// of about 40), the rest by memory: 32768 rows of 256 experts with bias, 4 of 8 groups and top 8
// take 26.5 us (36 MB), 17 of them before any second pass; 7 rows of 128 experts 3.2, 32768 rows of 128
// experts without bias or groups 9.5 (bf16 7.0).
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "qf_device.h"
#include "qf_operators.h"

namespace qf {

constexpr int RT_WAVE = 64;
constexpr int RT_WAVES = 4;       // waves per workgroup (they share nothing: fewer workgroups to start)
constexpr float RT_INF = __builtin_inff();

// Reductions over the L lanes of a row.
template <int L>
__device__ __forceinline__ float rt_row_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp_xor1(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_xor2(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_hmirror(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_mirror(__float_as_uint(v))));
  if (L > 16) v = fmaxf(v, __uint_as_float(swz_xor16(__float_as_uint(v))));
  return v;
}
template <int CTRL>
__device__ __forceinline__ double rt_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int L>
__device__ __forceinline__ double rt_row_max(double v) {
  v = fmax(v, rt_dpp<0xB1>(v));        // lane ^ 1, lane ^ 2, then mirrors as for float
  v = fmax(v, rt_dpp<0x4E>(v));
  v = fmax(v, rt_dpp<0x141>(v));
  v = fmax(v, rt_dpp<0x140>(v));
  if (L > 16) v = fmax(v, __shfl_xor(v, 16));
  return v;
}
template <int L, typename T>
__device__ __forceinline__ T rt_row_sum(T v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float rt_logit(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float rt_logit(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }

// V consecutive logits from e0 of a row; past E minus infinity.
template <int V, bool VEC>
__device__ __forceinline__ void rt_load(const float* row, int e0, int E, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (VEC) {
      const float4 v = e0 + i < E ? *reinterpret_cast<const float4*>(row + e0 + i) : float4{-RT_INF, -RT_INF, -RT_INF, -RT_INF};
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i + j] = e0 + i + j < E ? row[e0 + i + j] : -RT_INF;
    }
  }
}
template <int V, bool VEC>
__device__ __forceinline__ void rt_load(const uint16_t* row, int e0, int E, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (VEC) {
      const uint2 v = e0 + i < E ? *reinterpret_cast<const uint2*>(row + e0 + i) : uint2{0xFF80FF80u, 0xFF80FF80u};
      x[i] = bf16_lo(v.x); x[i + 1] = bf16_hi(v.x); x[i + 2] = bf16_lo(v.y); x[i + 3] = bf16_hi(v.y);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[i + j] = e0 + i + j < E ? __uint_as_float((uint32_t)row[e0 + i + j] << 16) : -RT_INF;
    }
  }
}

// Orders a wave's own LDS accesses: its lanes exchange through LDS, waves do not.
__device__ __forceinline__ void rt_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Groups: none, each a power of two of whole lanes (WHOLE), or any.
enum { RT_NO_GROUPS = 0, RT_WHOLE = 1, RT_ANY = 2 };

// LDS of the group ranking, per row.
template <int L, int V, int GROUPS, typename K>
struct RtGroups {
  K keys[GROUPS == RT_ANY ? RT_WAVES * RT_WAVE * V : 1];
  K score[RT_WAVES * RT_WAVE / L * QF_ROUTE_MAX_GROUPS];
  uint8_t keep[RT_WAVES * RT_WAVE / L * QF_ROUTE_MAX_GROUPS];
};

__device__ __forceinline__ void rt_top2(double& m1, double& m2, double v) {
  m2 = fmax(m2, fmin(m1, v));
  m1 = fmax(m1, v);
}
__device__ __forceinline__ void rt_top2(float& m1, float& m2, float v) {
  m2 = __builtin_amdgcn_fmed3f(m1, m2, v);
  m1 = fmaxf(m1, v);
}

// Keeps only the experts of the best groups: the others' keys become minus infinity.  False
// where a kept and a dropped group differ by no more than margin.
template <int L, int V, int GROUPS, typename K>
__device__ __forceinline__ bool rt_groups(const RouteArgs& a, int sub, int lane, K (&key)[V], RtGroups<L, V, GROUPS, K>& s,
                                          K margin) {
  const int size = a.E / a.n_group;
  const K none = -(K)RT_INF;
  K* keys = s.keys + (GROUPS == RT_ANY ? sub * (L * V) : 0);
  K* score = s.score + sub * QF_ROUTE_MAX_GROUPS;
  uint8_t* keep = s.keep + sub * QF_ROUTE_MAX_GROUPS;
  const int lanes = size / V;
  if (GROUPS == RT_WHOLE) {                    // a group's two best by exchange
    K m1 = none, m2 = none;
#pragma unroll
    for (int i = 0; i < V; ++i) rt_top2(m1, m2, key[i]);
    for (int d = 1; d < lanes; d <<= 1) {
      const K o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
      m2 = m1 > o1 ? (m2 > o1 ? m2 : o1) : (m1 > o2 ? m1 : o2);
      m1 = m1 > o1 ? m1 : o1;
    }
    if (lane % lanes == 0 && lane * V < a.E) score[lane / lanes] = a.group_top2 && m2 > none ? m1 + m2 : m1;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i < a.E) keys[lane * V + i] = key[i];
    rt_wave_sync();
    for (int g = lane; g < a.n_group; g += L) {
      K m1 = none, m2 = none;
      for (int i = 0; i < size; ++i) rt_top2(m1, m2, keys[g * size + i]);
      score[g] = a.group_top2 && m2 > none ? m1 + m2 : m1;
    }
  }
  rt_wave_sync();
  K worst = (K)RT_INF, best = none;            // of the kept, of the dropped
  for (int g = lane; g < a.n_group; g += L) {
    const K mine = score[g];
    int rank = 0;
    for (int o = 0; o < a.n_group; ++o) {
      const K v = score[o];
      rank += v > mine || (v == mine && o < g);
    }
    const bool in = rank < a.topk_group;
    keep[g] = in;
    if (in) worst = mine < worst ? mine : worst;
    else best = mine > best ? mine : best;
  }
  rt_wave_sync();
  worst = -rt_row_max<L>(-worst);
  best = rt_row_max<L>(best);
  if (GROUPS == RT_WHOLE) {
    const bool in = lane * V < a.E && keep[lane / lanes];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = in ? key[i] : none;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < a.E && !keep[e / size]) key[i] = none;
    }
  }
  return !(best > none) || worst - best > margin;
}

// Selection by comparing keys of type K (ties to the lower index); minus infinity is never
// chosen.
template <int L, int V, typename K>
__device__ __forceinline__ void rt_select(const RouteArgs& a, int lane, uint64_t seg, K (&key)[V], int32_t* chosen) {
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    K best = key[0];
    int slot = 0;
#pragma unroll
    for (int i = 1; i < V; ++i) {
      const bool up = key[i] > best;
      best = up ? key[i] : best;
      slot = up ? i : slot;
    }
    const K mx = rt_row_max<L>(best);
    const uint64_t who = __ballot(best == mx) & seg;
    if (who == 0) {                                          // NaN keys of a poisoned row
      if (lane == 0) chosen[j] = -1;
    } else if ((int)(threadIdx.x & 63) == __ffsll((unsigned long long)who) - 1) {
      chosen[j] = mx > -(K)RT_INF ? lane * V + slot : -1;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == slot) key[i] = -(K)RT_INF;
    }
  }
}

__device__ __forceinline__ uint32_t rt_order(float v) {      // increasing with v
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float rt_unorder(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}
template <int L>
__device__ __forceinline__ uint32_t rt_row_umax(uint32_t v) {
  v = umax(v, dpp_xor1(v));
  v = umax(v, dpp_xor2(v));
  v = umax(v, dpp_hmirror(v));
  v = umax(v, dpp_mirror(v));
  if (L > 16) v = umax(v, swz_xor16(v));
  return v;
}

// Fast selection by keys below 2^31: each round takes the largest key below the last one,
// which is the largest of key - last as an unsigned number (all keys above wrap to small
// differences).  The j-th key ends up in lane j % L, register j / L, and unless places[] is null
// the lane that holds it writes its index there.  Where nothing is left the keys are below
// `least`, minus infinity's.  False if two lanes of a row hold an equal valid key (only one
// counts then).
template <int L, int V, int P>
__device__ __forceinline__ bool rt_select_keys(int rounds, int lane, const uint32_t (&key)[V], uint32_t least, int top_index,
                                               uint32_t low, int32_t* places, uint32_t (&held)[P]) {
  uint32_t last = 0x80000000u;
  int holders = 0, valid = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    held[p] = 0;
    for (int i = 0; i < L && p * L + i < rounds; ++i) {
      uint32_t mine = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) mine = umax(mine, key[v] - last);
      const uint32_t row = rt_row_umax<L>(mine);
      last = (last + row) & (uint32_t)((int32_t)row >> 31);      // 0 when nothing is below
      held[p] = lane == i ? last : held[p];
      const bool ok = last >= least;
      if (places != nullptr && mine == row && ok) {
        places[p * L + i] = top_index - (int)(last & low);
        ++holders;
      }
      valid += ok;
    }
  }
  return places == nullptr || rt_row_sum<L>(holders) == valid;
}

constexpr int rt_log2(int v) { return v <= 1 ? 0 : 1 + rt_log2(v / 2); }

// exp in 64 bits for x <= 709: x = n ln 2 + r with ln 2 in two parts (Cody and Waite's reduction),
// |r| <= ln 2 / 2, and r's Taylor polynomial (the term after the last is below 2^-57); about two
// units of rounding.  The second pass is rare and its code cold, so it is short.
__device__ __forceinline__ double rt_exp64(double x) {
  x = fmax(x, -746.0);                               // from there on exp is 0 in 64 bits
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = __builtin_fma(n, -0x1.62e42fefa39efp-1, x);
  r = __builtin_fma(n, -0x1.abc9e3b39803fp-56, r);
  double p = 1.0 / 6227020800.0;                     // 1 / 13!
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}
// 1 / d for d in [1, 2]: the hardware's approximation and two Newton steps.
__device__ __forceinline__ double rt_rcp64(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

// Below this logit 1 + exp(x) is 1 to 2^-28, so a sigmoid is exp(x); expf(-x) there comes near its
// overflow.  A row whose chosen logits are all below it has the sums of a softmax over them.
constexpr float RT_LOW = -20.0f;

__device__ __forceinline__ float rt_fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// SCORES: choose by scores plus bias, else by logits.
template <int L, int V, typename X, bool SCORES, bool VEC, int GROUPS>
__global__ __launch_bounds__(RT_WAVE * RT_WAVES) void k_route(RouteArgs a) {
  constexpr int ROWS = RT_WAVE * RT_WAVES / L;
  constexpr bool IN_ROW = !SCORES && sizeof(X) == 2;       // logit and index fit a key
  using K2 = typename std::conditional<SCORES, double, float>::type;   // the second pass's keys
  __shared__ int32_t chosen[ROWS][QF_ROUTE_MAX_K + 1];
  __shared__ typename std::conditional<GROUPS != 0, RtGroups<L, V, GROUPS, K2>, char>::type gs2;
  __shared__ typename std::conditional<GROUPS != 0 && SCORES, RtGroups<L, V, GROUPS, float>, char>::type gs1;
  const int lane = threadIdx.x % L, sub = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * ROWS + sub;
  const bool live = t < a.T;
  const X* row = static_cast<const X*>(a.logits) + (live ? t : 0) * a.ld;
  float x[V];
  rt_load<V, VEC>(row, lane * V, live ? a.E : 0, x);

  float top = -RT_INF, total = 0.0f;       // softmax: the sum of exp(x - top), when it is needed
  const bool softmax = a.scoring == QF_ROUTE_SOFTMAX;
  float v[V];                      // what is compared (-0 + 0 = +0: one key for both zeros)
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = x[i] + 0.0f;
  if (softmax && (SCORES || !a.renorm)) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
    top = rt_row_max<L>(top);
    if (top == -RT_INF) top = 0.0f;        // nothing but masked experts: every exp is 0
    float e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      e[i] = rt_fast_exp(x[i] - top);
      total += e[i];
    }
    total = rt_row_sum<L>(total);
    if (SCORES) {
      const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = e[i] * inv;
    }
  } else if (SCORES) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __builtin_amdgcn_rcpf(1.0f + rt_fast_exp(-x[i]));
  }
  float bias[V];
  if (SCORES) {
    if (a.bias) {
      rt_load<V, VEC>(a.bias, lane * V, a.E, bias);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += bias[i];
  }
  // a NaN or plus infinity (in a masked expert's bias too) poisons its row: as integers, positive ones
  // are the largest signed numbers, and negative NaN lies above minus infinity among the unsigned
  int32_t most = INT32_MIN;
  uint32_t mostu = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    most = std::max(most, (int32_t)__float_as_uint(v[i]));
    if (SCORES) most = std::max(most, (int32_t)__float_as_uint(x[i]));
    mostu = umax(mostu, __float_as_uint(v[i]));
    if (SCORES) v[i] = x[i] == -RT_INF ? -RT_INF : v[i];
  }
  const uint64_t seg = ((1ull << L) - 1ull) << ((threadIdx.x & 63) / L * L);
  const bool bad = (__ballot(most >= 0x7F800000 || mostu > 0xFF800000u) & seg) != 0;

  // The fp32 score's error: sigmoid, 5 units of 2^-24 (exp2 and its argument, sum, reciprocal,
  // each weighed by s or s (1 - s)); softmax, 32 units of the largest score (the sum's
  // roundings most of all); the bias adds half a unit of the key.  Twice that for a pair.
  const float err = SCORES ? (softmax ? 0x1p-18f * (total > 0.0f ? 1.0f / total : 0.0f) : 0x1p-20f) : 0.0f;
  bool sure = true;
  if constexpr (GROUPS != 0) {
    if constexpr (SCORES) {
      float big = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) big = fmaxf(big, v[i] > -RT_INF ? __builtin_fabsf(v[i]) : 0.0f);
      sure = rt_groups<L, V, GROUPS, float>(a, sub, lane, v, gs1, 2.0f * err + 0x1p-21f * rt_row_max<L>(big));
    } else {
      rt_groups<L, V, GROUPS, float>(a, sub, lane, v, gs2, 0.0f);
    }
  }
  uint32_t key[V];
  constexpr int IDX = IN_ROW ? 10 : rt_log2(V);
  constexpr uint32_t LOW = (1u << IDX) - 1u;
#pragma unroll
  for (int i = 0; i < V; ++i)
    key[i] = IN_ROW ? ((rt_order(v[i]) >> 16) << IDX | (LOW - (uint32_t)(lane * V + i)))
                    : ((rt_order(v[i]) >> 1) & ~LOW) | (LOW - (uint32_t)i);
  // the smallest finite value's key: minus infinity is the one before it in order
  constexpr uint32_t least = IN_ROW ? (0x0080u << IDX) : (0x00800000u >> 1);
  constexpr int P = (QF_ROUTE_MAX_K + 1 + L - 1) / L, PER = (QF_ROUTE_MAX_K + L - 1) / L;
  uint32_t held[P];
  // one round more than choices: the next key decides the last choice
  const int rounds = IN_ROW ? a.k : a.k + 1;
  sure = rt_select_keys<L, V, P>(rounds, lane, key, least, lane * V + V - 1, LOW, IN_ROW ? nullptr : chosen[sub], held) && sure;
  int id[PER];
  if constexpr (IN_ROW) {
#pragma unroll
    for (int p = 0; p < PER; ++p) id[p] = held[p] >= least ? (int)(LOW - (held[p] & LOW)) : -1;
  } else {
    // neighbours in the order, each pair in the first one's lane
#pragma unroll
    for (int p = 0; p < P; ++p) {
      uint32_t next = __shfl_down(held[p], 1, L);
      if (p + 1 < P) {
        const uint32_t wrap = __shfl(held[p + 1 < P ? p + 1 : p], 0, L);
        next = lane == L - 1 ? wrap : next;
      }
      if (lane + p * L < a.k && next >= least) {
        bool close = (held[p] & ~LOW) == (next & ~LOW);
        if (SCORES) {
          const float hi = rt_unorder((held[p] & ~LOW) << 1), lo = rt_unorder((next & ~LOW) << 1);
          // truncation takes up to 2^(IDX + 1) units of 2^-23 of a value
          close = !(hi - lo > err + fmaxf(__builtin_fabsf(hi), __builtin_fabsf(lo)) * (0x1p-22f * (1 << IDX) + 0x1p-22f));
        }
        sure = sure && !close;
      }
    }
    rt_wave_sync();
#pragma unroll
    for (int p = 0; p < PER; ++p) id[p] = held[p] >= least && lane + p * L < a.k ? chosen[sub][lane + p * L] : -1;
  }

  if constexpr (!IN_ROW) {
    if (__ballot(!sure && !bad && live) != 0) {
      K2 key2[V];
      if constexpr (SCORES) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // a masked logit's score does not matter below; sigmoids from exp(-|x|), which cannot overflow
          key2[i] = rt_exp64(softmax ? (double)x[i] - (double)top : -fabs((double)x[i]));
          sum += key2[i];
        }
        if (softmax) sum = rt_row_sum<L>(sum);
        const double inv = softmax ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          key2[i] = softmax ? key2[i] * inv : rt_rcp64(1.0 + key2[i]) * (x[i] < 0.0f ? key2[i] : 1.0);
          key2[i] = x[i] > -RT_INF ? key2[i] + (double)bias[i] : -(double)RT_INF;
        }
        if constexpr (GROUPS != 0) rt_groups<L, V, GROUPS, K2>(a, sub, lane, key2, gs2, 0.0);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key2[i] = v[i];          // the groups' choice was exact
      }
      rt_select<L, V, K2>(a, lane, seg, key2, chosen[sub]);
      rt_wave_sync();
#pragma unroll
      for (int p = 0; p < PER; ++p) id[p] = lane + p * L < a.k ? chosen[sub][lane + p * L] : -1;
    }
  }

  // weights: lane j (and j + L) of a row has its j-th choice
  float u[PER], xs[PER];
  bool low = false;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int j = lane + p * L;
    if (!live || bad || j >= a.k) id[p] = -1;
    xs[p] = id[p] >= 0 ? rt_logit(row, id[p]) : -RT_INF;
    low |= id[p] >= 0 && xs[p] < RT_LOW;
  }
  float scale = a.scale;
  float sum = 0.0f;
  if (!softmax && __ballot(low) == 0) {       // sigmoids without a low one in the wave
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      u[p] = id[p] < 0 ? 0.0f : 1.0f / (1.0f + expf(-xs[p]));
      sum += u[p];
    }
  } else {
    bool exps = softmax;
    if (a.renorm) {       // relative to the largest chosen logit: the row's other scores cancel
      float first = -RT_INF;
#pragma unroll
      for (int p = 0; p < PER; ++p) first = fmaxf(first, xs[p]);
      first = rt_row_max<L>(first);
      exps = softmax || first < RT_LOW;
      if (first == -RT_INF) first = 0.0f;
      top = first;
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const bool exp = exps || xs[p] < RT_LOW;
      const float t = expf(exps ? xs[p] - top : exp ? xs[p] : -xs[p]);
      u[p] = id[p] < 0 ? 0.0f : exp ? t : 1.0f / (1.0f + t);
      sum += u[p];
    }
  }
  if (a.renorm) total = rt_row_sum<L>(sum);
  const bool divide = a.renorm || softmax;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int j = lane + p * L;
    if (!live || j >= a.k) continue;
    float w = divide ? (total > 0.0f ? u[p] / total : 0.0f) : u[p];
    a.indices[t * a.k + j] = id[p];
    a.weights[t * a.k + j] = bad ? __builtin_nanf("") : w * scale;
  }
}

// Gradient of the weights with respect to the logits.  With p_j = u_j / sum u:
//   renormalised, softmax:  dx[i_j] = c p_j (g_j - sum g p);   sigmoid: times (1 - u_j)
//   plain, sigmoid: dx[i_j] = c g_j u_j (1 - u_j);  softmax: dx[e] = c s_e (g_e - sum g u)
// with 1 - u of a sigmoid as exp(-x) u for positive x, and as 1 below RT_LOW.
// Lanes and logits are laid out as in the forward pass; the chosen ones (two per lane where k is
// over L) meet the row in LDS, so that the gradient leaves as one dense, coalesced row.  Bounded
// by the dense write (and the read, for plain softmax): 32768 x 128 bf16 6.4 us, 4099 x 128 fp32 4.1,
// of which an empty launch is 2.5.
template <int V, bool VEC>
__device__ __forceinline__ void rt_store(float* row, int e0, int E, const float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (VEC) {
      if (e0 + i < E) *reinterpret_cast<float4*>(row + e0 + i) = float4{x[i], x[i + 1], x[i + 2], x[i + 3]};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e0 + i + j < E) row[e0 + i + j] = x[i + j];
    }
  }
}
template <int V, bool VEC>
__device__ __forceinline__ void rt_store(uint16_t* row, int e0, int E, const float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const uint2 w = {pack_bf16x2(x[i], x[i + 1]), pack_bf16x2(x[i + 2], x[i + 3])};
    if (VEC) {
      if (e0 + i < E) *reinterpret_cast<uint2*>(row + e0 + i) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e0 + i + j < E) row[e0 + i + j] = (uint16_t)((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
    }
  }
}

template <int L, int V, typename X, bool VEC>
__global__ __launch_bounds__(RT_WAVE * RT_WAVES) void k_route_backward(RouteArgs a) {
  constexpr int ROWS = RT_WAVE / L, PER = (QF_ROUTE_MAX_K + L - 1) / L;
  __shared__ float4 d4[RT_WAVES * ROWS][L * V / 4];
  const int lane = threadIdx.x % L, sub = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * (RT_WAVES * ROWS) + sub;
  const bool live = t < a.T;
  const X* row = static_cast<const X*>(a.logits) + (live ? t : 0) * a.ld;
  float* d = reinterpret_cast<float*>(d4[sub]);
  const bool softmax = a.scoring == QF_ROUTE_SOFTMAX, dense = softmax && !a.renorm;
  int id[PER];
  float g[PER], x[PER], u[PER], rest[PER];       // rest: 1 - u of a sigmoid
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int j = lane + p * L;
    id[p] = live && j < a.k ? a.indices[t * a.k + j] : -1;
    g[p] = live && j < a.k ? a.dweights[t * a.k + j] : 0.0f;
    if ((uint32_t)id[p] >= (uint32_t)a.E) id[p] = -1;
  }
  float v[V];
  if (dense) rt_load<V, VEC>(row, lane * V, live ? a.E : 0, v);
#pragma unroll
  for (int i = 0; i < V; i += 4) d4[sub][(lane * V + i) / 4] = float4{0.0f, 0.0f, 0.0f, 0.0f};
  float top = -RT_INF;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    x[p] = id[p] >= 0 && !dense ? rt_logit(row, id[p]) : -RT_INF;
    g[p] = id[p] >= 0 ? g[p] * a.scale : 0.0f;
    top = fmaxf(top, x[p]);
  }
  if (!dense) {
    if (softmax) {
      top = rt_row_max<L>(top);
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        u[p] = id[p] >= 0 && top > -RT_INF ? expf(x[p] - top) : 0.0f;
        rest[p] = 1.0f;
      }
    } else {
      bool low = false;
#pragma unroll
      for (int p = 0; p < PER; ++p) low |= id[p] >= 0 && x[p] < RT_LOW;
      const bool any = __ballot(low) != 0;       // in the wave
      if (any && a.renorm) top = rt_row_max<L>(top);
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const float t = expf(-x[p]);
        u[p] = id[p] < 0 ? 0.0f : 1.0f / (1.0f + t);
        rest[p] = x[p] > 0.0f ? t * u[p] : 1.0f - u[p];      // 1 - u would lose the digits that u's rounding drops
        if (any && x[p] < RT_LOW) {
          u[p] = x[p] == -RT_INF ? 0.0f : expf(a.renorm && top < RT_LOW ? x[p] - top : x[p]);
          rest[p] = 1.0f;
        }
      }
    }
    if (a.renorm) {
      float total = 0.0f, mean = 0.0f;
#pragma unroll
      for (int p = 0; p < PER; ++p) total += u[p];
      total = rt_row_sum<L>(total);
      // divided, not times a reciprocal: a lone choice has p = 1 and a gradient of exactly 0
      float q[PER];
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        q[p] = total > 0.0f ? u[p] / total : 0.0f;
        mean += g[p] * q[p];
      }
      mean = rt_row_sum<L>(mean);
#pragma unroll
      for (int p = 0; p < PER; ++p) g[p] = q[p] * (g[p] - mean) * rest[p];
    } else {
#pragma unroll
      for (int p = 0; p < PER; ++p) g[p] *= u[p] * rest[p];
    }
  }
  rt_wave_sync();
  // an index given twice adds up: the choices one after another
#pragma unroll
  for (int p = 0; p < PER; ++p)
    for (int j = 0; j < L && p * L + j < a.k; ++j) {
      if (lane == j && id[p] >= 0) d[id[p]] += g[p];
      rt_wave_sync();              // the next lane's sum starts from this one's
    }
  float o[V];
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 w = d4[sub][(lane * V + i) / 4];
    o[i] = w.x; o[i + 1] = w.y; o[i + 2] = w.z; o[i + 3] = w.w;
  }
  if (dense) {
    int any = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) any |= id[p] >= 0;
    any = rt_row_sum<L>(any);
    float most = -RT_INF, total = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) most = fmaxf(most, v[i]);
    most = rt_row_max<L>(most);
    if (most == -RT_INF) most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = expf(v[i] - most);
      total += v[i];
      dot += v[i] * o[i];
    }
    total = rt_row_sum<L>(total);
    dot = rt_row_sum<L>(dot);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;       // a NaN stays
    const float mean = dot * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = any ? v[i] * inv * (o[i] - mean) : 0.0f;
  }
  if (live) rt_store<V, VEC>(static_cast<X*>(a.dlogits) + t * a.ldd, lane * V, a.E, o);
}

namespace {
template <int L, int V, typename X, bool S>
void route_go(const RouteArgs& a, bool vec, hipStream_t s) {
  constexpr int ROWS = RT_WAVE * RT_WAVES / L;
  const unsigned grid = (unsigned)((a.T + ROWS - 1) / ROWS);
  const int size = a.E / a.n_group, lanes = size / V;
  if (a.n_group > 1 && vec && size % V == 0 && (lanes & (lanes - 1)) == 0) {
    k_route<L, V, X, S, true, RT_WHOLE><<<grid, RT_WAVE * RT_WAVES, 0, s>>>(a);
  } else if (a.n_group > 1) {
    if (vec) k_route<L, V, X, S, true, RT_ANY><<<grid, RT_WAVE * RT_WAVES, 0, s>>>(a);
    else k_route<L, V, X, S, false, RT_ANY><<<grid, RT_WAVE * RT_WAVES, 0, s>>>(a);
  } else {
    if (vec) k_route<L, V, X, S, true, RT_NO_GROUPS><<<grid, RT_WAVE * RT_WAVES, 0, s>>>(a);
    else k_route<L, V, X, S, false, RT_NO_GROUPS><<<grid, RT_WAVE * RT_WAVES, 0, s>>>(a);
  }
}
// Few lanes with many logits each: a round's work over the lanes' logits is shared by more rows.
template <typename X, bool S>
void route_size(const RouteArgs& a, bool vec, hipStream_t s) {
  if (a.E <= 64) route_go<16, 4, X, S>(a, vec, s);
  else if (a.E <= 128) route_go<16, 8, X, S>(a, vec, s);
  else if (a.E <= 256) route_go<16, 16, X, S>(a, vec, s);
  else if (a.E <= 512) route_go<32, 16, X, S>(a, vec, s);
  else route_go<32, 32, X, S>(a, vec, s);
}
}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t s) {
  const bool scores = a.bias != nullptr || (a.n_group > 1 && a.group_top2);
  const int64_t sz = bf16 ? 2 : 4;
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && (uintptr_t)a.logits % (4 * sz) == 0 &&
                   (uintptr_t)a.bias % 16 == 0;
  if (bf16) {
    if (scores) route_size<uint16_t, true>(a, vec, s);
    else route_size<uint16_t, false>(a, vec, s);
  } else {
    if (scores) route_size<float, true>(a, vec, s);
    else route_size<float, false>(a, vec, s);
  }
  return hipGetLastError();
}

namespace {
template <int L, int V, typename X>
void route_back_go(const RouteArgs& a, bool vec, hipStream_t s) {
  constexpr int ROWS = RT_WAVE / L * RT_WAVES;
  const unsigned grid = (unsigned)((a.T + ROWS - 1) / ROWS);
  if (vec) k_route_backward<L, V, X, true><<<grid, RT_WAVE * RT_WAVES, 0, s>>>(a);
  else k_route_backward<L, V, X, false><<<grid, RT_WAVE * RT_WAVES, 0, s>>>(a);
}
template <typename X>
void route_back_size(const RouteArgs& a, bool vec, hipStream_t s) {
  if (a.E <= 64) route_back_go<16, 4, X>(a, vec, s);
  else if (a.E <= 128) route_back_go<16, 8, X>(a, vec, s);
  else if (a.E <= 256) route_back_go<16, 16, X>(a, vec, s);
  else if (a.E <= 512) route_back_go<32, 16, X>(a, vec, s);
  else route_back_go<32, 32, X>(a, vec, s);
}
}  // namespace

hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t s) {
  const int64_t sz = bf16 ? 2 : 4;
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && a.ldd % 4 == 0 && (uintptr_t)a.logits % (4 * sz) == 0 &&
                   (uintptr_t)a.dlogits % (4 * sz) == 0;
  if (bf16) route_back_size<uint16_t>(a, vec, s);
  else route_back_size<float>(a, vec, s);
  return hipGetLastError();
}

}  // namespace qf

namespace {

bool bad_align(const void* p, uintptr_t a) { return ((uintptr_t)p % a) != 0; }

// Checks what both directions read of a description, and fills the kernels' arguments.
qf_status route_args(const qf_route_desc* d, qf::RouteArgs& a) {
  if (!d) return QF_ERR_NULL;
  if (d->logits_bf16 != 0 && d->logits_bf16 != 1) return QF_ERR_ARG;
  if (d->scoring != QF_ROUTE_SOFTMAX && d->scoring != QF_ROUTE_SIGMOID) return QF_ERR_ARG;
  if (d->renorm != 0 && d->renorm != 1) return QF_ERR_ARG;
  if (!(d->scale >= -FLT_MAX && d->scale <= FLT_MAX)) return QF_ERR_ARG;      // written so that a NaN fails
  if (d->experts < 1 || d->experts > QF_ROUTE_MAX_EXPERTS || d->tokens < 0 || d->tokens > QF_ROUTE_MAX_TOKENS)
    return QF_ERR_SHAPE;
  if (d->ld < d->experts) return QF_ERR_SHAPE;
  if (d->k < 1 || d->k > QF_ROUTE_MAX_K || d->k > d->experts) return QF_ERR_ARG;
  a = qf::RouteArgs{};
  a.logits = d->logits;
  a.ld = d->ld;
  a.T = d->tokens;
  a.E = d->experts;
  a.k = d->k;
  a.scoring = d->scoring;
  a.renorm = d->renorm;
  a.scale = d->scale;
  a.n_group = 1;
  if (d->tokens > 0 && !d->logits) return QF_ERR_NULL;
  if (bad_align(d->logits, d->logits_bf16 ? 2 : 4)) return QF_ERR_ALIGN;
  return QF_OK;
}

}  // namespace

extern "C" {

qf_status qf_moe_route(const qf_route_desc* d, int32_t* indices, float* weights, void* stream) {
  qf::RouteArgs a;
  const qf_status st = route_args(d, a);
  if (st != QF_OK) return st;
  if (d->n_group < 1 || d->n_group > QF_ROUTE_MAX_GROUPS || d->experts % d->n_group || d->topk_group < 1 ||
      d->topk_group > d->n_group || d->k > d->experts / d->n_group * d->topk_group)
    return QF_ERR_ARG;
  if (d->group_rule != QF_ROUTE_GROUP_MAX && d->group_rule != QF_ROUTE_GROUP_TOP2) return QF_ERR_ARG;
  if (d->tokens > 0 && (!indices || !weights)) return QF_ERR_NULL;
  if (bad_align(indices, 4) || bad_align(weights, 4) || bad_align(d->bias, 4)) return QF_ERR_ALIGN;
  if (d->tokens == 0) return QF_OK;
  a.bias = d->bias;
  a.n_group = d->topk_group == d->n_group ? 1 : d->n_group;      // every group kept: no groups
  a.topk_group = d->topk_group;
  a.group_top2 = d->group_rule == QF_ROUTE_GROUP_TOP2;
  a.indices = indices;
  a.weights = weights;
  return qf::status_of(qf::launch_route(a, d->logits_bf16 == 1, (hipStream_t)stream));
}

qf_status qf_moe_route_backward(const qf_route_desc* d, const int32_t* indices, const float* d_weights, void* d_logits,
                                int64_t ldd, void* stream) {
  qf::RouteArgs a;
  const qf_status st = route_args(d, a);
  if (st != QF_OK) return st;
  if (ldd < d->experts) return QF_ERR_SHAPE;
  if (d->tokens > 0 && (!indices || !d_weights || !d_logits)) return QF_ERR_NULL;
  if (bad_align(indices, 4) || bad_align(d_weights, 4) || bad_align(d_logits, d->logits_bf16 ? 2 : 4)) return QF_ERR_ALIGN;
  if (d->tokens == 0) return QF_OK;
  a.indices = const_cast<int32_t*>(indices);
  a.dweights = d_weights;
  a.dlogits = d_logits;
  a.ldd = ldd;
  return qf::status_of(qf::launch_route_backward(a, d->logits_bf16 == 1, (hipStream_t)stream));
}

}  // extern "C"
