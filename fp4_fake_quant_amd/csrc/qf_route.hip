// Routing of tokens to experts: scores, selection, weights, and their gradient.
//
// A row (token) is held by L lanes of one wave, V consecutive logits each, so that an index
// order is a lane order.  Selection repeats k times: the lane's best (lowest index on ties),
// the row's best over its L lanes (cross-lane max), the lowest lane that holds it.
//
// What is compared decides the chosen experts, and a tie decided by rounding would choose
// differently from one implementation to the next.  Without a bias (and with groups ranked by
// their best expert) both scorings are increasing in the logit, so the logits themselves are
// compared: exact.  Otherwise scores plus bias are compared in 64 bits.
#include "qf_device.h"
#include "qf_kernels.h"

namespace qf {

constexpr int RT_WAVE = 64;       // one wave per workgroup: rows share nothing
constexpr float RT_INF = __builtin_inff();

__device__ __forceinline__ float rt_max_xor(float v, int d) { return fmaxf(v, __shfl_xor(v, d)); }

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
template <int L>
__device__ __forceinline__ double rt_row_max(double v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v = fmax(v, __shfl_xor(v, d));
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

template <typename K> __device__ __forceinline__ K rt_exp(K x);
template <> __device__ __forceinline__ float rt_exp<float>(float x) { return expf(x); }
template <> __device__ __forceinline__ double rt_exp<double>(double x) { return exp(x); }

// Keeps only the experts of the best groups: the others' keys become minus infinity.
template <int L, int V, typename K>
__device__ __forceinline__ void rt_groups(const RouteArgs& a, int sub, int lane, K (&key)[V], K* keys, K* score, uint8_t* keep) {
  const int size = a.E / a.n_group;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (lane * V + i < a.E) keys[sub * (L * V) + lane * V + i] = key[i];
  __syncthreads();
  for (int g = lane; g < a.n_group; g += L) {
    K m1 = -(K)RT_INF, m2 = -(K)RT_INF;
    for (int i = 0; i < size; ++i) {
      const K v = keys[sub * (L * V) + g * size + i];
      m2 = v > m1 ? m1 : (v > m2 ? v : m2);
      m1 = v > m1 ? v : m1;
    }
    score[sub * QF_ROUTE_MAX_GROUPS + g] = a.group_top2 && m2 > -(K)RT_INF ? m1 + m2 : m1;
  }
  __syncthreads();
  for (int g = lane; g < a.n_group; g += L) {
    const K mine = score[sub * QF_ROUTE_MAX_GROUPS + g];
    int rank = 0;
    for (int o = 0; o < a.n_group; ++o) {
      const K v = score[sub * QF_ROUTE_MAX_GROUPS + o];
      rank += v > mine || (v == mine && o < g);
    }
    keep[sub * QF_ROUTE_MAX_GROUPS + g] = rank < a.topk_group;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    if (e < a.E && !keep[sub * QF_ROUTE_MAX_GROUPS + e / size]) key[i] = -(K)RT_INF;
  }
}

// K: float compares logits, double compares scores plus bias.
template <int L, int V, typename X, typename K, bool VEC, bool GROUPS>
__global__ __launch_bounds__(RT_WAVE) void k_route(RouteArgs a) {
  constexpr int ROWS = RT_WAVE / L;
  constexpr bool SCORES = sizeof(K) == 8;
  __shared__ int32_t chosen[ROWS][QF_ROUTE_MAX_K];
  __shared__ K keys[GROUPS ? ROWS * L * V : 1], gscore[GROUPS ? ROWS * QF_ROUTE_MAX_GROUPS : 1];
  __shared__ uint8_t keep[GROUPS ? ROWS * QF_ROUTE_MAX_GROUPS : 1];
  const int lane = threadIdx.x % L, sub = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * ROWS + sub;
  const bool live = t < a.T;
  const X* row = static_cast<const X*>(a.logits) + (live ? t : 0) * a.ld;
  float x[V];
  rt_load<V, VEC>(row, lane * V, live ? a.E : 0, x);

  // a NaN or plus infinity poisons its row
  bool bad = false;
  float top = -RT_INF;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= !(x[i] < RT_INF);
    top = fmaxf(top, x[i]);
  }
  K key[V];
  float total = 0.0f;              // softmax: the sum of exp(x - top), when the weights need it
  const bool softmax = a.scoring == QF_ROUTE_SOFTMAX;
  if (softmax && (SCORES || !a.renorm)) {
    top = rt_row_max<L>(top);
    if (top == -RT_INF) top = 0.0f;        // nothing but masked experts: every exp is 0
  }
  if (SCORES) {
    K sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = softmax ? rt_exp<K>((K)x[i] - (K)top) : (K)1 / ((K)1 + rt_exp<K>(-(K)x[i]));
      sum += key[i];
    }
    if (softmax) {
      sum = rt_row_sum<L>(sum);
      total = (float)sum;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (softmax) key[i] = key[i] / sum;
      if (a.bias && e < a.E) key[i] += (K)a.bias[e];
      if (e >= a.E || x[i] == -RT_INF) key[i] = -(K)RT_INF;
      bad |= !(key[i] < (K)RT_INF);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = x[i];
    if (softmax && !a.renorm) {
#pragma unroll
      for (int i = 0; i < V; ++i) total += expf(x[i] - top);
      total = rt_row_sum<L>(total);
    }
  }
  const uint64_t seg = (L == 64 ? ~0ull : (1ull << L) - 1ull) << (sub * L);
  bad = (__ballot(bad) & seg) != 0;
  if (GROUPS) rt_groups<L, V, K>(a, sub, lane, key, keys, gscore, keep);

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
    const bool win = (int)threadIdx.x == __ffsll((unsigned long long)who) - 1;
    if (win) {
      chosen[sub][j] = mx > -(K)RT_INF ? lane * V + slot : -1;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == slot) key[i] = -(K)RT_INF;
    }
    if (who == 0 && lane == 0) chosen[sub][j] = -1;      // NaN keys of a poisoned row
  }
  __syncthreads();

  // weights: lane j (and j + L) of a row has its j-th choice
  constexpr int PER = (QF_ROUTE_MAX_K + L - 1) / L;
  int id[PER];
  float u[PER], xs[PER];
  float first = -RT_INF;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int j = lane + p * L;
    id[p] = live && !bad && j < a.k ? chosen[sub][j] : -1;
    xs[p] = id[p] >= 0 ? rt_logit(row, id[p]) : -RT_INF;
    first = fmaxf(first, xs[p]);
  }
  float scale = a.scale;
  if (softmax && a.renorm) {       // relative to the largest chosen logit: the row's other scores cancel
    first = rt_row_max<L>(first);
    if (first == -RT_INF) first = 0.0f;
    top = first;
  }
  float sum = 0.0f;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    u[p] = id[p] < 0 ? 0.0f : softmax ? expf(xs[p] - top) : 1.0f / (1.0f + expf(-xs[p]));
    sum += u[p];
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
// A row's gradient is assembled in LDS and leaves in whole lines.
template <typename X>
__device__ __forceinline__ void rt_store(X* p, float v);
template <> __device__ __forceinline__ void rt_store<float>(float* p, float v) { *p = v; }
template <> __device__ __forceinline__ void rt_store<uint16_t>(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }

template <typename X>
__global__ __launch_bounds__(RT_WAVE) void k_route_backward(RouteArgs a) {
  __shared__ float d[QF_ROUTE_MAX_EXPERTS];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const X* row = static_cast<const X*>(a.logits) + t * a.ld;
  X* out = static_cast<X*>(a.dlogits) + t * a.ldd;
  const bool softmax = a.scoring == QF_ROUTE_SOFTMAX;
  for (int e = lane; e < a.E; e += RT_WAVE) d[e] = 0.0f;
  const int id0 = lane < a.k ? a.indices[t * a.k + lane] : -1;
  const int id = (uint32_t)id0 < (uint32_t)a.E ? id0 : -1;
  const bool any = __ballot(id >= 0) != 0;
  const float g = id >= 0 ? a.dweights[t * a.k + lane] * a.scale : 0.0f;
  const float x = id >= 0 ? rt_logit(row, id) : -RT_INF;
  float dx = 0.0f;
  if (a.renorm || !softmax) {
    float u;
    if (softmax) {
      float top = rt_row_max<32>(x);
      top = rt_max_xor(top, 32);
      u = id >= 0 && top > -RT_INF ? expf(x - top) : 0.0f;
    } else {
      u = id >= 0 ? 1.0f / (1.0f + expf(-x)) : 0.0f;
    }
    if (a.renorm) {
      const float total = rt_row_sum<64>(u);
      const float p = total > 0.0f ? u / total : 0.0f;
      const float mean = rt_row_sum<64>(g * p);
      dx = p * (g - mean);
      if (!softmax) dx *= 1.0f - u;
    } else {
      dx = g * u * (1.0f - u);
    }
  } else {
    dx = g;                       // the score's gradient; the row's part follows
  }
  __syncthreads();
  for (int j = 0; j < a.k; ++j)   // in order, so that an index given twice adds up
    if (lane == j && id >= 0) d[id] += dx;
  __syncthreads();
  if (softmax && !a.renorm && any) {
    float top = -RT_INF;
    for (int e = lane; e < a.E; e += RT_WAVE) top = fmaxf(top, rt_logit(row, e));
    top = rt_row_max<32>(top);
    top = rt_max_xor(top, 32);
    if (top == -RT_INF) top = 0.0f;
    float total = 0.0f, dot = 0.0f;
    for (int e = lane; e < a.E; e += RT_WAVE) {
      const float s = expf(rt_logit(row, e) - top);
      total += s;
      dot += s * d[e];
    }
    total = rt_row_sum<64>(total);
    dot = rt_row_sum<64>(dot);
    const float mean = total > 0.0f ? dot / total : 0.0f;
    for (int e = lane; e < a.E; e += RT_WAVE) {
      const float s = total > 0.0f ? expf(rt_logit(row, e) - top) / total : 0.0f;
      rt_store(out + e, s * (d[e] - mean));
    }
    return;
  }
  for (int e = lane; e < a.E; e += RT_WAVE) rt_store(out + e, d[e]);
}

namespace {
template <int L, int V, typename X, typename K>
void route_go(const RouteArgs& a, bool vec, hipStream_t s) {
  constexpr int ROWS = RT_WAVE / L;
  const unsigned grid = (unsigned)((a.T + ROWS - 1) / ROWS);
  if (a.n_group > 1) {
    if (vec) k_route<L, V, X, K, true, true><<<grid, RT_WAVE, 0, s>>>(a);
    else k_route<L, V, X, K, false, true><<<grid, RT_WAVE, 0, s>>>(a);
  } else {
    if (vec) k_route<L, V, X, K, true, false><<<grid, RT_WAVE, 0, s>>>(a);
    else k_route<L, V, X, K, false, false><<<grid, RT_WAVE, 0, s>>>(a);
  }
}
template <typename X, typename K>
void route_size(const RouteArgs& a, bool vec, hipStream_t s) {
  if (a.E <= 64) route_go<16, 4, X, K>(a, vec, s);
  else if (a.E <= 128) route_go<16, 8, X, K>(a, vec, s);
  else if (a.E <= 256) route_go<16, 16, X, K>(a, vec, s);
  else if (a.E <= 512) route_go<32, 16, X, K>(a, vec, s);
  else route_go<32, 32, X, K>(a, vec, s);
}
}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t s) {
  const bool scores = a.bias != nullptr || (a.n_group > 1 && a.group_top2);
  const int64_t sz = bf16 ? 2 : 4;
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && (uintptr_t)a.logits % (4 * sz) == 0;
  if (bf16) {
    if (scores) route_size<uint16_t, double>(a, vec, s);
    else route_size<uint16_t, float>(a, vec, s);
  } else {
    if (scores) route_size<float, double>(a, vec, s);
    else route_size<float, float>(a, vec, s);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t s) {
  if (bf16) k_route_backward<uint16_t><<<(unsigned)a.T, RT_WAVE, 0, s>>>(a);
  else k_route_backward<float><<<(unsigned)a.T, RT_WAVE, 0, s>>>(a);
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
  if (!(d->scale >= -3e38f && d->scale <= 3e38f)) return QF_ERR_ARG;
  if (d->experts < 1 || d->experts > QF_ROUTE_MAX_EXPERTS || d->tokens < 0 || d->tokens >= (1ll << 30)) return QF_ERR_SHAPE;
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
