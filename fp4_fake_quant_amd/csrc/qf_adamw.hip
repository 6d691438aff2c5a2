// AdamW over many tensors: the step that turns the fp32 gradients of the straight-through
// estimator and of the adapters into the next latent weights and their bf16 copies.
//
// Arithmetic (include/qf.h): separate fp32 roundings in the stated order (the build never
// contracts a product and a sum), IEEE division and square root, so that a plain sequence of
// elementwise fp32 operations gives the same bits.  8-bit states are E4M3 codes with an fp32
// scale per 256-element block, stochastically rounded: with round-to-nearest a slow moving
// average stands still (b2 = 0.999 moves sqrt(v) by 0.05% a step, half an E4M3 step is up to
// 6%), with 16 random bits its expectation is right to 2^-16 of a step.
//
// One wave owns whole 256-element blocks, 4 consecutive elements per lane: every fp32 load
// and store instruction of a wave covers 1 KiB of contiguous memory, and a block's largest
// magnitude is one cross-lane reduction.  Every byte passes once (30 per element with fp32
// states, fp32 gradient and bf16 copy; 16 with 8-bit states and bf16 gradient), so all of it is
// accessed with the non-temporal policy.  Measured on 218 M elements: see aw_per_wave.
#include <algorithm>
#include <string.h>

#include "qf_device.h"
#include "qf_operators.h"

namespace qf {

constexpr int AW_WG = 256;
constexpr int AW_BLOCK = QF_ADAMW_BLOCK;           // elements per 8-bit block: 64 lanes x 4
// Blocks in flight per wave.  More give a wave more loads to wait for at once, fewer give small
// tensors more waves.  Microseconds for 1 / 2 / 4 blocks: fp32 states, 1.1 M elements 7.8 / 8.0 /
// 8.9 and 218 M 1120 / 1164 / 1113; 8-bit states, 22 M elements in 120 tensors 83 / 87 / 94 and
// 218 M 637 / 606 / 605 (and without the non-temporal policy, 4 blocks: 1214, 687).
constexpr int aw_per_wave(int bits) { return bits == 8 ? 2 : 1; }
constexpr int aw_chunk(int bits) { return AW_WG / 64 * aw_per_wave(bits) * AW_BLOCK; }
constexpr float AW_MIN_MAX = 7.888609052210118e-31f;   // 2^-100: smaller block maxima store zeros

static_assert(AW_BLOCK == 256, "a wave of 64 lanes holds one block, 4 elements per lane");

// 32-bit finaliser: xor-shifts and two odd multipliers, the constants of Wellons's published search
// for integer hashes of low bias (2018).
__host__ __device__ inline uint32_t aw_hash(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// b^t by repeated squaring in 64 bits.
__host__ __device__ inline double aw_pow(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

__host__ __device__ inline void aw_scalars(AdamwScalars& s, double lr, double beta1, double beta2, int64_t step,
                                           uint32_t seed) {
  if (step < 1) step = 1;
  s.lr = lr;
  s.size = (float)(lr / (1.0 - aw_pow(beta1, step)));
  s.root = (float)(1.0 / __builtin_sqrt(1.0 - aw_pow(beta2, step)));
  s.key = aw_hash(seed ^ aw_hash((uint32_t)step));
}

__device__ __forceinline__ uint32_t aw_wave_max(uint32_t v) {
  v = umax(v, dpp_xor1(v));
  v = umax(v, dpp_xor2(v));
  v = umax(v, dpp_hmirror(v));
  v = umax(v, dpp_mirror(v));
  v = umax(v, swz_xor16(v));
  return umax((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 32));
}

// E4M3 magnitude code of y in [0, 448 (1 + 2^-21)], rounded up with probability (distance to the
// code below) / step: rnd holds 16 random bits, added below the kept mantissa bits.  512 y and
// rnd / 65536 are exact, so the one rounding of the fused sum is the sum's; y just above 448 has
// too few bits there for rnd to carry.
__device__ __forceinline__ uint32_t aw_e4m3_stochastic(float y, uint32_t rnd) {
  const uint32_t small = (uint32_t)__builtin_fmaf(y, 512.0f, (float)rnd * 0x1p-16f);   // truncates: floor
  const uint32_t large = ((__float_as_uint(y) + (rnd << 4)) >> 20) - 960u;
  return y < 0.015625f ? small : large;
}

// The correctly rounded square root of v >= 0 that is 0 or at least 2^-96 (below, the residuals
// underflow): the hardware's, which is at most one unit off, and its two neighbours tested by
// the sign of v - s s' (Tuckerman's rounding test; Agarwal and others, IBM J. Res. Dev. 30, 1986).
__device__ __forceinline__ float aw_sqrt(float v) {
  float s = __builtin_amdgcn_sqrtf(v);
  const float down = __uint_as_float(__float_as_uint(s) - 1u), up = __uint_as_float(__float_as_uint(s) + 1u);
  const float rd = __builtin_fmaf(-down, s, v), ru = __builtin_fmaf(-up, s, v);
  s = rd <= 0.0f ? down : s;
  return ru > 0.0f ? up : s;
}

struct AwScale {
  float scale, inv;
};
__device__ __forceinline__ AwScale aw_block_scale(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits);
  const bool dead = top < AW_MIN_MAX;               // false for a NaN: it stays visible in the scale
  AwScale o;
  o.scale = dead ? 0.0f : top * (1.0f / 448.0f);
  o.inv = dead ? 0.0f : 1.0f / o.scale;
  return o;
}

typedef float aw_f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t aw_u32x2 __attribute__((ext_vector_type(2)));

// Four consecutive elements of an array; unless FULL only `left` of them exist (the others read
// as zero and are not written).
template <bool FULL>
__device__ __forceinline__ float4 aw_load4(const float* p, uint32_t left) {
  if (FULL || left >= 4) {
    const aw_f32x4 q = __builtin_nontemporal_load(reinterpret_cast<const aw_f32x4*>(p));
    return float4{q.x, q.y, q.z, q.w};
  }
  float4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (left > 0) o.x = p[0];
  if (left > 1) o.y = p[1];
  if (left > 2) o.z = p[2];
  return o;
}
template <bool FULL>
__device__ __forceinline__ float4 aw_load4(const uint16_t* p, uint32_t left) {
  aw_u32x2 w = {0u, 0u};
  if (FULL || left >= 4) {
    w = __builtin_nontemporal_load(reinterpret_cast<const aw_u32x2*>(p));
  } else {
    if (left > 0) w.x = p[0];
    if (left > 1) w.x |= (uint32_t)p[1] << 16;
    if (left > 2) w.y = p[2];
  }
  return {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
}
template <bool FULL>
__device__ __forceinline__ uint32_t aw_load4(const uint8_t* p, uint32_t left) {
  if (FULL || left >= 4) return __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  uint32_t w = 0;
  if (left > 0) w = p[0];
  if (left > 1) w |= (uint32_t)p[1] << 8;
  if (left > 2) w |= (uint32_t)p[2] << 16;
  return w;
}
template <bool FULL>
__device__ __forceinline__ void aw_store4(float* p, const float (&v)[4], uint32_t left) {
  if (FULL || left >= 4) {
    __builtin_nontemporal_store(aw_f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<aw_f32x4*>(p));
    return;
  }
  for (uint32_t i = 0; i < 3; ++i)
    if (i < left) p[i] = v[i];
}
template <bool FULL>
__device__ __forceinline__ void aw_store4(uint16_t* p, const float (&v)[4], uint32_t left) {
  const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
  if (FULL || left >= 4) {
    __builtin_nontemporal_store(aw_u32x2{lo, hi}, reinterpret_cast<aw_u32x2*>(p));
    return;
  }
  if (left > 0) p[0] = (uint16_t)lo;
  if (left > 1) p[1] = (uint16_t)(lo >> 16);
  if (left > 2) p[2] = (uint16_t)hi;
}
template <bool FULL>
__device__ __forceinline__ void aw_store4(uint8_t* p, uint32_t w, uint32_t left) {
  if (FULL || left >= 4) {
    __builtin_nontemporal_store(w, reinterpret_cast<uint32_t*>(p));
    return;
  }
  for (uint32_t i = 0; i < 3; ++i)
    if (i < left) p[i] = (uint8_t)(w >> (8 * i));
}

// The wave's blocks from b0 of one tensor; FULL: all of their elements exist.
template <int BITS, typename G, bool FULL, typename Args>
__device__ __forceinline__ void aw_blocks(const Args& a, const AdamwTensor& t, uint32_t b0, uint32_t lane) {
  constexpr int PER = aw_per_wave(BITS);
  // uniform bases: the lane's part of every address is a small offset
  const uint64_t first = (uint64_t)b0 * AW_BLOCK;
  float* const tp = t.p + first;
  const G* const tg = static_cast<const G*>(t.g) + first;
  uint16_t* const tp16 = t.p16 ? t.p16 + first : nullptr;
  float* const tm = static_cast<float*>(t.m) + (BITS == 8 ? 0 : first);
  float* const tv = static_cast<float*>(t.v) + (BITS == 8 ? 0 : first);
  uint8_t* const tmc = static_cast<uint8_t*>(t.m) + (BITS == 8 ? first : 0);
  uint8_t* const tvc = static_cast<uint8_t*>(t.v) + (BITS == 8 ? first : 0);
  const uint32_t n = FULL ? PER * AW_BLOCK : (uint32_t)(t.n - first);

  float4 p[PER], g[PER], m[PER], v[PER];
  uint32_t mc[PER], vc[PER];
  float ms[PER], vs[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const uint32_t at = j * AW_BLOCK + lane * 4;
    const uint32_t left = at < n ? n - at : 0;
    p[j] = aw_load4<FULL>(tp + at, left);
    g[j] = aw_load4<FULL>(tg + at, left);
    if (BITS == 8) {
      mc[j] = aw_load4<FULL>(tmc + at, left);
      vc[j] = aw_load4<FULL>(tvc + at, left);
      const bool in = FULL || j * AW_BLOCK < n;
      ms[j] = in ? t.ms[b0 + j] : 0.0f;
      vs[j] = in ? t.vs[b0 + j] : 0.0f;
    } else {
      m[j] = aw_load4<FULL>(tm + at, left);
      v[j] = aw_load4<FULL>(tv + at, left);
    }
  }

  AdamwScalars s = a.s;
  if (a.d_lr || a.d_step)      // while the loads are in flight
    aw_scalars(s, a.d_lr ? (double)*a.d_lr : s.lr, a.beta1, a.beta2, a.d_step ? *a.d_step : a.step, a.seed);
  const float keep = (float)(1.0 - s.lr * t.weight_decay);
  const float b1 = (float)a.beta1, c1 = (float)(1.0 - a.beta1);
  const float b2 = (float)a.beta2, c2 = (float)(1.0 - a.beta2);
  const float eps = (float)a.eps;

  float ms_out[PER], vs_out[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (!FULL && j * AW_BLOCK >= n) break;                      // uniform over the wave
    const uint32_t at = j * AW_BLOCK + lane * 4;
    const uint32_t left = at < n ? n - at : 0;
    if (BITS == 8) {
      const f32x2_t m01 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[j], false);
      const f32x2_t m23 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[j], true);
      const f32x2_t r01 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[j], false);
      const f32x2_t r23 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[j], true);
      m[j] = float4{m01.x * ms[j], m01.y * ms[j], m23.x * ms[j], m23.y * ms[j]};
      const float4 r = {r01.x * vs[j], r01.y * vs[j], r23.x * vs[j], r23.y * vs[j]};
      v[j] = float4{r.x * r.x, r.y * r.y, r.z * r.z, r.w * r.w};
    }
    const float pi[4] = {p[j].x, p[j].y, p[j].z, p[j].w};
    const float mi[4] = {m[j].x, m[j].y, m[j].z, m[j].w}, vi[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
    float gi[4] = {g[j].x, g[j].y, g[j].z, g[j].w};
    if (a.d_grad_scale) {
      const float gs = *a.d_grad_scale;
#pragma unroll
      for (int e = 0; e < 4; ++e) gi[e] *= gs;
    }
    float po[4], mo[4], vo[4], ro[4];
    uint32_t tiny = 0xFFFFFFFFu;                                // least v > 0; zeros wrap to the top
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      mo[e] = mi[e] * b1 + gi[e] * c1;
      vo[e] = vi[e] * b2 + (gi[e] * c2) * gi[e];
      tiny = umin(tiny, __float_as_uint(vo[e]) - 1u);
    }
    if (__builtin_expect(__ballot(tiny < 0x0F800000u - 1u) != 0, 0)) {   // some v below 2^-96
#pragma unroll
      for (int e = 0; e < 4; ++e) ro[e] = __builtin_sqrtf(vo[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) ro[e] = aw_sqrt(vo[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) po[e] = pi[e] * keep - (mo[e] / (ro[e] * s.root + eps)) * s.size;
    aw_store4<FULL>(tp + at, po, left);
    if (tp16) aw_store4<FULL>(tp16 + at, po, left);
    if (BITS == 8) {
      uint32_t mm = 0, rm = 0;                                  // non-negative floats order like their bits
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mm = umax(mm, __float_as_uint(mo[e]) & 0x7FFFFFFFu);
        rm = umax(rm, __float_as_uint(ro[e]));
      }
      const AwScale sm = aw_block_scale(aw_wave_max(mm)), sv = aw_block_scale(aw_wave_max(rm));
      ms_out[j] = sm.scale;
      vs_out[j] = sv.scale;
      uint32_t mw = 0, vw = 0;
      const uint32_t key = s.key + (uint32_t)first + at;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h = aw_hash(key + e);
        const float my = __builtin_fabsf(mo[e]) * sm.inv, vy = ro[e] * sv.inv;
        const uint32_t sign = (__float_as_uint(mo[e]) >> 24) & 0x80u;
        const uint32_t cm = aw_e4m3_stochastic(my, h & 0xFFFFu) | sign;
        // no zero for v > 0: it would let the next step divide by a far too small root
        const uint32_t cv = umax(aw_e4m3_stochastic(vy, h >> 16), umin(__float_as_uint(vy), 1u));
        mw |= cm << (8 * e);
        vw |= cv << (8 * e);
      }
      aw_store4<FULL>(tmc + at, mw, left);
      aw_store4<FULL>(tvc + at, vw, left);
    } else {
      aw_store4<FULL>(tm + at, mo, left);
      aw_store4<FULL>(tv + at, vo, left);
    }
  }
  if (BITS == 8) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if ((FULL || j * AW_BLOCK < n) && lane == (uint32_t)j) {
        t.ms[b0 + j] = ms_out[j];
        t.vs[b0 + j] = vs_out[j];
      }
    }
  }
}

// The tensor of workgroup wg: the last one that begins at or before it.  In the arguments all
// beginnings are compared at once (scalar); in a table the wave's lanes compare 64 at a time, every
// stride-th one first.
template <int N>
__device__ __forceinline__ const AdamwTensor& aw_find(const AdamwArgs<N>& a, uint32_t wg, uint32_t lane, uint32_t& begin) {
  int ti = -1;
#pragma unroll
  for (int i = 0; i < N; ++i) ti += wg >= a.begin[i];
  begin = a.begin[ti];
  return a.t[ti];
}
__device__ __forceinline__ const AdamwTensor& aw_find(const AdamwTableArgs& a, uint32_t wg, uint32_t lane, uint32_t& begin) {
  int lo = 0, len = a.n;
  while (len > 1) {
    const int stride = (len + 63) / 64, i = (int)lane * stride;
    const uint64_t in = __ballot(i < len && wg >= a.begin[lo + (i < len ? i : 0)]);    // bit 0 always
    lo += (__popcll(in) - 1) * stride;
    len = stride < a.n - lo ? stride : a.n - lo;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  begin = a.begin[lo];
  return a.t[lo];
}

template <int BITS, typename G, typename Args>
__global__ __launch_bounds__(AW_WG) void k_adamw(Args a) {
  if (a.skip && *a.skip) return;
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t begin;
  const AdamwTensor& t = aw_find(a, blockIdx.x, lane, begin);
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  constexpr int PER = aw_per_wave(BITS);
  const uint32_t b0 = ((blockIdx.x - begin) * (AW_WG / 64) + wave) * PER;   // first block of the wave
  if ((uint64_t)(b0 + PER) * AW_BLOCK <= t.n)
    aw_blocks<BITS, G, true>(a, t, b0, lane);
  else if ((uint64_t)b0 * AW_BLOCK < t.n)
    aw_blocks<BITS, G, false>(a, t, b0, lane);
}

uint32_t adamw_chunks(int64_t n, int bits) { return (uint32_t)((n + aw_chunk(bits) - 1) / aw_chunk(bits)); }

void adamw_host_scalars(AdamwScalars& s, double lr, double beta1, double beta2, int64_t step, uint32_t seed) {
  aw_scalars(s, lr, beta1, beta2, step, seed);
}

template <typename Args>
static hipError_t launch(const Args& a, uint32_t grid, int bits, bool g_bf16, hipStream_t s) {
  if (bits == 8) {
    if (g_bf16)
      k_adamw<8, uint16_t, Args><<<grid, AW_WG, 0, s>>>(a);
    else
      k_adamw<8, float, Args><<<grid, AW_WG, 0, s>>>(a);
  } else {
    if (g_bf16)
      k_adamw<32, uint16_t, Args><<<grid, AW_WG, 0, s>>>(a);
    else
      k_adamw<32, float, Args><<<grid, AW_WG, 0, s>>>(a);
  }
  return hipGetLastError();
}

// The arguments of a launch travel with it: a few tensors take the short form.
hipError_t launch_adamw(const AdamwArgs<AW_TENSORS>& a, int n, uint32_t grid, int bits, bool g_bf16, hipStream_t s) {
  if (n > AW_FEW) return launch(a, grid, bits, g_bf16, s);
  AdamwArgs<AW_FEW> f;
  static_cast<AdamwCommon&>(f) = a;
  memcpy(f.t, a.t, sizeof(f.t));
  memcpy(f.begin, a.begin, sizeof(f.begin));
  return launch(f, grid, bits, g_bf16, s);
}

hipError_t launch_adamw_table(const AdamwTableArgs& a, uint32_t grid, int bits, bool g_bf16, hipStream_t s) {
  return launch(a, grid, bits, g_bf16, s);
}

}  // namespace qf

namespace {
constexpr uint32_t AW_MAX_GRID = (1u << 24) - 1;   // a launch holds below 2^32 lanes: 256 per workgroup

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) != 0; }

qf_status check_hyper(const qf_adamw_hyper* h) {
  // written so that a NaN fails
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0 && h->beta2 >= 0.0 && h->beta2 < 1.0 && h->eps >= 0.0)) return QF_ERR_ARG;
  if (!h->d_step && h->step < 1) return QF_ERR_ARG;
  if (!h->d_lr && !(h->lr >= 0.0 && h->lr <= 1e30)) return QF_ERR_ARG;
  if (misaligned(h->d_lr, 4) || misaligned(h->d_step, 8) || misaligned(h->d_grad_scale, 4) || misaligned(h->d_skip, 4))
    return QF_ERR_ALIGN;
  return QF_OK;
}

qf_status check_tensors(const qf_adamw_tensor* t, int n, int state_bits) {
  for (int i = 0; i < n; ++i) {
    const qf_adamw_tensor& d = t[i];
    if (d.n < 0 || d.n >= (1ll << 31)) return QF_ERR_SHAPE;
    if (d.g_bf16 != 0 && d.g_bf16 != 1) return QF_ERR_ARG;
    if (!(d.weight_decay >= 0.0 && d.weight_decay <= 1e30)) return QF_ERR_ARG;
    if (d.n == 0) continue;
    if (!d.p || !d.g || !d.m || !d.v) return QF_ERR_NULL;
    if (state_bits == 8 && (!d.m_scale || !d.v_scale)) return QF_ERR_NULL;
    if (misaligned(d.p, 16) || misaligned(d.g, 16) || misaligned(d.m, 16) || misaligned(d.v, 16) ||
        misaligned(d.p16, 16) || misaligned(d.m_scale, 4) || misaligned(d.v_scale, 4))
      return QF_ERR_ALIGN;
  }
  return QF_OK;
}

void fill(qf::AdamwTensor& o, const qf_adamw_tensor& d) {
  o.p = d.p;
  o.g = d.g;
  o.m = d.m;
  o.v = d.v;
  o.ms = d.m_scale;
  o.vs = d.v_scale;
  o.p16 = d.p16;
  o.n = (uint32_t)d.n;
  o.weight_decay = d.weight_decay;
}

void common(qf::AdamwCommon& a, const qf_adamw_hyper* h) {
  a.beta1 = h->beta1;
  a.beta2 = h->beta2;
  a.eps = h->eps;
  a.step = h->step;
  a.seed = h->seed;
  a.d_lr = h->d_lr;
  a.d_step = h->d_step;
  a.d_grad_scale = h->d_grad_scale;
  a.skip = h->d_skip;
  qf::adamw_host_scalars(a.s, h->lr, h->beta1, h->beta2, h->step, h->seed);
}

size_t table_begin(int n) { return sizeof(qf::AdamwTensor) * (size_t)n; }
}  // namespace

extern "C" {

qf_status qf_adamw_step(const qf_adamw_tensor* t, int n, int state_bits, const qf_adamw_hyper* h, void* stream) {
  if (n < 0 || (state_bits != 32 && state_bits != 8)) return QF_ERR_ARG;
  if (!h || (n > 0 && !t)) return QF_ERR_NULL;
  qf_status st = check_hyper(h);
  if (st == QF_OK) st = check_tensors(t, n, state_bits);
  if (st != QF_OK) return st;
  qf::AdamwArgs<qf::AW_TENSORS> a;
  common(a, h);
  for (int bf = 0; bf < 2; ++bf) {          // one run of launches per gradient type
    int k = 0;
    uint32_t grid = 0;
    for (int i = 0; i <= n; ++i) {
      const bool mine = i < n && t[i].n > 0 && t[i].g_bf16 == bf;
      const uint32_t more = mine ? qf::adamw_chunks(t[i].n, state_bits) : 0;
      if (k > 0 && (i == n || k == qf::AW_TENSORS || grid + more > AW_MAX_GRID)) {
        for (int j = k; j < qf::AW_TENSORS; ++j) a.begin[j] = 0xFFFFFFFFu;   // no workgroup reaches these
        const hipError_t e = qf::launch_adamw(a, k, grid, state_bits, bf == 1, (hipStream_t)stream);
        if (e != hipSuccess) return qf::status_of(e);
        k = 0;
        grid = 0;
      }
      if (mine) {
        fill(a.t[k], t[i]);
        a.begin[k++] = grid;
        grid += more;
      }
    }
  }
  return QF_OK;
}

size_t qf_adamw_table_bytes(int n) { return n <= 0 ? 0 : table_begin(n) + sizeof(uint32_t) * (size_t)n; }

qf_status qf_adamw_table(const qf_adamw_tensor* t, int n, int state_bits, void* table, size_t bytes, qf_adamw_plan* plan) {
  if (n < 0 || (state_bits != 32 && state_bits != 8)) return QF_ERR_ARG;
  if (!plan || (n > 0 && (!t || !table))) return QF_ERR_NULL;
  if (bytes < qf_adamw_table_bytes(n)) return QF_ERR_WORKSPACE;
  const qf_status st = check_tensors(t, n, state_bits);
  if (st != QF_OK) return st;
  *plan = qf_adamw_plan{};
  plan->state_bits = state_bits;
  plan->capacity = n;
  int at = 0;
  for (int bf = 0; bf < 2; ++bf) {
    uint64_t grid = 0;
    const int first = at;
    for (int i = 0; i < n; ++i) {
      if (t[i].n == 0 || t[i].g_bf16 != bf) continue;
      qf::AdamwTensor o{};
      fill(o, t[i]);
      const uint32_t begin = (uint32_t)grid;
      memcpy((char*)table + sizeof(o) * at, &o, sizeof(o));
      memcpy((char*)table + table_begin(n) + sizeof(begin) * at, &begin, sizeof(begin));
      ++at;
      grid += qf::adamw_chunks(t[i].n, state_bits);
      if (grid > AW_MAX_GRID) return QF_ERR_SHAPE;
    }
    plan->tensors[bf] = at - first;
    plan->workgroups[bf] = (uint32_t)grid;
  }
  return QF_OK;
}

qf_status qf_adamw_step_table(const qf_adamw_plan* plan, const void* d_table, const qf_adamw_hyper* h, void* stream) {
  if (!plan || !h) return QF_ERR_NULL;
  if (plan->state_bits != 32 && plan->state_bits != 8) return QF_ERR_ARG;
  if (plan->tensors[0] < 0 || plan->tensors[1] < 0 || plan->capacity < 0 ||
      (int64_t)plan->tensors[0] + plan->tensors[1] > plan->capacity)
    return QF_ERR_ARG;
  const qf_status st = check_hyper(h);
  if (st != QF_OK) return st;
  if (plan->tensors[0] + plan->tensors[1] > 0 && !d_table) return QF_ERR_NULL;
  if (misaligned(d_table, 8)) return QF_ERR_ALIGN;
  qf::AdamwTableArgs a;
  common(a, h);
  int at = 0;
  for (int bf = 0; bf < 2; ++bf) {
    if (plan->tensors[bf] == 0) continue;
    a.t = (const qf::AdamwTensor*)d_table + at;
    a.begin = (const uint32_t*)((const char*)d_table + table_begin(plan->capacity)) + at;
    a.n = plan->tensors[bf];
    at += a.n;
    const hipError_t e = qf::launch_adamw_table(a, plan->workgroups[bf], plan->state_bits, bf == 1, (hipStream_t)stream);
    if (e != hipSuccess) return qf::status_of(e);
  }
  return QF_OK;
}

}  // extern "C"
