// head_norm.cu - per-head norms around a recurrent layer's state update:
//
//   qk_norm_rotary   x / sqrt(mean x^2 + eps) w  (or x / sqrt(sum x^2 + eps) w)
//                    for every head of q and k, then the pairs of its first
//                    rot components turned by theta_i = position inv_freq_i
//   head_norm_gated  y / sqrt(mean y^2 + eps) w SiLU(z) for every head of y
//
// Bound: HBM (each value read once and written once).  A group of G = d / 8
// lanes (8, 16 or 32) holds a head, 8 values per lane, so the sum is a butterfly.
// A lane's values are two runs of four, for pairs in halves the four of the low
// half and their partners in the high half: a turn stays inside the lane, and the
// lane needs the cosines and sines of four pairs (a lane of eight neighbours would
// need eight, and its partners through shuffles).  A group keeps its token's
// cosines and sines in registers and goes over the heads with them.
//
// Angles: position inv_freq loses its low bits in f32 (at position 10^6 the
// product's rounding is 0.03 rad), so the lane holds inv_freq as a 64-bit
// fraction of a turn and multiplies in integers: whole turns overflow out of
// the word exactly, for either sign, and its high half is the angle to 2^-32
// turns.  The table entry's own error is 2^-64 turns times the position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_math.cuh"
#include "launch.h"

namespace mamba {
namespace {

// Threads and resident CTAs per SM of the two vector kernels: small CTAs, several
// heads' loads each, and as many CTAs as the registers allow.  32768 tokens, d = 128:
// 24 heads of q and k 70.9 us (256 threads, 4 heads, 3 CTAs: 78.6), a norm of 40
// heads 160 us (256 threads, 4 heads, 3 CTAs: 215).
constexpr int kQkThreads = 128, kQkCtas = 7;
constexpr int kHnThreads = 64, kHnCtas = 16;

// inv_freq (radians per position) as a 2^-64 fraction of a turn: its 24-bit
// significand times 2^64 / (2 pi), shifted by its exponent.  Whole turns per
// position do not matter, positions being integers, and fall off the top.
__device__ __forceinline__ uint64_t turns_per_position(float inv_freq) {
  constexpr uint64_t kInv2Pi = 2935890503282001226ull;  // 2^64 / (2 pi), to the nearest
  const uint32_t bits = __float_as_uint(inv_freq);
  const int field = (int)((bits >> 23) & 255);
  const uint32_t m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);
  const int right = 150 - (field ? field : 1);  // inv_freq = m 2^-right
  const uint64_t lo = (uint64_t)m * (uint32_t)kInv2Pi, hi = (uint64_t)m * (uint32_t)(kInv2Pi >> 32) + (lo >> 32);
  // the product is hi 2^32 + (lo mod 2^32), 86 bits
  const uint64_t low = (hi << 32) | (uint32_t)lo, high = hi >> 32;
  uint64_t t;
  if (right >= 64)
    t = right < 128 ? high >> (right - 64) : 0;
  else if (right > 0)
    t = (low >> right) | (high << (64 - right));
  else
    t = right > -64 ? low << -right : 0;
  return (bits >> 31) ? 0 - t : t;
}

// Cosine and sine of position x turns.  The product's high word is the angle to
// 2^-32 of a turn; its nearest quarter is taken off as an integer, and what is
// left, at most an eighth of a turn either way, goes through the Taylor series
// (the first terms left out are below 2^-25).
__device__ __forceinline__ float2 cos_sin(int64_t position, uint64_t turns) {
  const uint32_t hi = (uint32_t)(((uint64_t)position * turns) >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const float t = (float)(int32_t)(hi - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
  const float t2 = t * t;
  float s = fmaf(t2, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, -1/7!
  s = fmaf(t2, s, 8.3333333e-3f);
  s = fmaf(t2, s, -1.6666667e-1f);
  s = fmaf(t2 * t, s, t);
  float c = fmaf(t2, 2.4801587e-5f, -1.3888889e-3f);  // 1/8!, -1/6!
  c = fmaf(t2, c, 4.1666667e-2f);
  c = fmaf(t2, c, -0.5f);
  c = fmaf(t2, c, 1.0f);
  const float x = (quarter & 1) ? s : c, y = (quarter & 1) ? c : s;
  return make_float2(((quarter + 1) & 2) ? -x : x, (quarter & 2) ? -y : y);
}

// The turn of `position` by a frequency; NaN for one that is NaN or infinite
__device__ __forceinline__ float2 turn(int64_t position, float inv_freq) {
  const float2 a = cos_sin(position, turns_per_position(inv_freq));
  const float zero = inv_freq - inv_freq;  // or NaN
  return make_float2(a.x + zero, a.y + zero);
}

template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* p2) {
    const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(p2);
    raw = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) { load(p, p + 4); }
  __device__ __forceinline__ void load(const float* p, const float* p2) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p2);
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) { *reinterpret_cast<uint4*>(p) = pack8(f); }
__device__ __forceinline__ void store8(__nv_bfloat16* p, __nv_bfloat16* p2, const float (&f)[8]) {
  const uint4 w = pack8(f);
  *reinterpret_cast<uint2*>(p) = make_uint2(w.x, w.y);
  *reinterpret_cast<uint2*>(p2) = make_uint2(w.z, w.w);
}
__device__ __forceinline__ void store8(float* p, float* p2, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p2) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) { store8(p, p + 4, f); }

// One group of G lanes: one token, heads [h0, h0 + per_group) of the Hq + Hk.
// kHeads heads' loads are in flight together.  The weights of the lane's 8
// components are re-read per head (L1) rather than held for both q and k.
// HALVES: pairs (i, rot / 2 + i); else neighbours, or no turns.
template <typename IN, typename OUT, int G, bool HALVES>
__global__ void __launch_bounds__(kQkThreads, kQkCtas) qk_norm_kernel(const QkNormArgs g, int per_group, int slices, float inv_n) {
  grid_dependency_begin();
  constexpr int kHeads = sizeof(IN) == 2 ? 6 : 3;
  constexpr int kGroups = kQkThreads / G;
  const int lane = threadIdx.x % G;
  const int64_t unit = (int64_t)blockIdx.x * kGroups + threadIdx.x / G;
  const int64_t rows = g.B * g.T;
  const int64_t row_raw = slices == 1 ? unit : unit / slices;
  const bool live = row_raw < rows;
  const int64_t row = live ? row_raw : rows - 1;  // idle groups stay for the shuffles
  const int heads = g.Hq + g.Hk;
  const int h0 = slices == 1 ? 0 : (int)(unit % slices) * per_group;
  const int h1 = h0 + per_group < heads ? h0 + per_group : heads;
  const bool in = 8 * lane < g.d;          // d % 8 == 0
  const bool turned = 8 * lane < g.rot;    // rot % 8 == 0
  const int c = HALVES && turned ? 4 * lane : 8 * lane;
  const int c2 = HALVES && turned ? g.rot / 2 + c : c + 4;

  // this token's turns for the lane's four pairs
  float cs[4], sn[4];
  if (g.rot > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 a = make_float2(1.0f, 0.0f);
      if (turned) a = turn(g.positions ? g.positions[row] : row % g.T, g.inv_freq[4 * lane + i]);
      cs[i] = a.x, sn[i] = a.y;
    }
  }
  const IN* q = reinterpret_cast<const IN*>(g.q) + row * g.ld_q;
  const IN* k = reinterpret_cast<const IN*>(g.k) + row * g.ld_k - (int64_t)g.Hq * g.d;
  OUT* q_out = reinterpret_cast<OUT*>(g.q_out) + row * g.ld_qo;
  OUT* k_out = reinterpret_cast<OUT*>(g.k_out) + row * g.ld_ko - (int64_t)g.Hq * g.d;

  for (int h = h0; h < h1; h += kHeads) {
    Vec8<IN> raw[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int hh = h + j < h1 ? h + j : h1 - 1;
      const IN* p = (hh < g.Hq ? q : k) + hh * g.d;
      if (in) {
        if constexpr (HALVES)
          raw[j].load(p + c, p + c2);
        else
          raw[j].load(p + c);
      }
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (h + j >= h1) break;  // uniform in the group; the shuffles below stay inside it
      float f[8];
      if (in) {
        raw[j].unpack(f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
      }
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      const unsigned mask = G == 32 ? 0xffffffffu : ((1u << G) - 1) << ((threadIdx.x % 32) / G * G);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float inv = rsqrtf(fmaf(ss, inv_n, g.eps));
      const bool is_q = h + j < g.Hq;
      const float* w = is_q ? g.q_weight : g.k_weight;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= inv;
      if (w && in) {
        const float4 lo = __ldg(reinterpret_cast<const float4*>(w + c)), hi = __ldg(reinterpret_cast<const float4*>(w + c2));
        f[0] *= lo.x, f[1] *= lo.y, f[2] *= lo.z, f[3] *= lo.w;
        f[4] *= hi.x, f[5] *= hi.y, f[6] *= hi.z, f[7] *= hi.w;
      }
      if (g.rot > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& a = f[HALVES ? i : 2 * i];
          float& b = f[HALVES ? 4 + i : 2 * i + 1];
          const float x = a, y = b;
          a = fmaf(-y, sn[i], x * cs[i]);
          b = fmaf(x, sn[i], y * cs[i]);
        }
      }
      if (in && live) {
        OUT* p = (is_q ? q_out : k_out) + (h + j) * g.d;
        if constexpr (HALVES)
          store8(p + c, p + c2, f);
        else
          store8(p + c, f);
      }
    }
  }
}

constexpr int kMaxD = 256;
constexpr int kAnyWarps = 4;

// Any d <= 256, any alignment, any even rot: one warp per (token, head), the
// head staged in shared memory for the rotation's partners.
template <typename IN, typename OUT>
__global__ void __launch_bounds__(32 * kAnyWarps) qk_norm_any_kernel(const QkNormArgs g) {
  grid_dependency_begin();
  __shared__ float stage[kAnyWarps][kMaxD];
  const int lane = threadIdx.x % 32;
  float* x = stage[threadIdx.x / 32];
  const int heads = g.Hq + g.Hk;
  const int64_t unit = (int64_t)blockIdx.x * kAnyWarps + threadIdx.x / 32;
  if (unit >= g.B * g.T * heads) return;
  const int64_t row = unit / heads;
  const int h = (int)(unit % heads);
  const bool is_q = h < g.Hq;
  const IN* p = is_q ? reinterpret_cast<const IN*>(g.q) + row * g.ld_q + (int64_t)h * g.d
                     : reinterpret_cast<const IN*>(g.k) + row * g.ld_k + (int64_t)(h - g.Hq) * g.d;
  OUT* o = is_q ? reinterpret_cast<OUT*>(g.q_out) + row * g.ld_qo + (int64_t)h * g.d
                : reinterpret_cast<OUT*>(g.k_out) + row * g.ld_ko + (int64_t)(h - g.Hq) * g.d;
  const float* w = is_q ? g.q_weight : g.k_weight;
  float ss = 0.0f;
  for (int c = lane; c < g.d; c += 32) {
    x[c] = to_f32(p[c]);
    ss = fmaf(x[c], x[c], ss);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
  const float inv = rsqrtf((g.l2 ? ss : ss / (float)g.d) + g.eps);
  for (int c = lane; c < g.d; c += 32) x[c] = x[c] * inv * (w ? w[c] : 1.0f);
  __syncwarp();
  const int64_t pos = g.positions ? g.positions[row] : row % g.T;
  const int half = g.rot / 2;
  for (int c = lane; c < g.d; c += 32) {
    float v = x[c];
    if (c < g.rot) {
      const int pair = g.interleaved ? c / 2 : c % half;
      const bool low = g.interleaved ? c % 2 == 0 : c < half;
      const float other = x[g.interleaved ? c ^ 1 : low ? c + half : c - half];
      const float2 a = turn(pos, g.inv_freq[pair]);
      v = fmaf(other, low ? -a.y : a.y, v * a.x);
    }
    o[c] = from_f32<OUT>(v);
  }
}

template <typename IN, typename OUT, int G>
__global__ void __launch_bounds__(kHnThreads, kHnCtas) head_norm_kernel(const HeadNormArgs g, int64_t units, int per_group) {
  grid_dependency_begin();
  constexpr int kHeads = sizeof(IN) == 2 ? 2 : 1;
  constexpr int kGroups = kHnThreads / G;
  const int lane = threadIdx.x % G;
  const int c = 8 * lane;
  const bool in = c < g.d;
  const unsigned mask = G == 32 ? 0xffffffffu : ((1u << G) - 1) << ((threadIdx.x % 32) / G * G);
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = g.weight && in ? __ldg(g.weight + c + i) : 1.0f;
  // unit u is head u % H of token u / H; a CTA takes per_group strides of kGroups
  // units, so one division a group and then a step from unit to unit
  const int64_t base = (int64_t)blockIdx.x * kGroups * per_group + threadIdx.x / G;
  int64_t row = base < 0x7fffffff ? (int64_t)((uint32_t)base / (uint32_t)g.H) : base / g.H;
  uint32_t h = (uint32_t)(base - row * g.H);  // below 2^31, and a step more below 2^32
  for (int s = 0; s < per_group; s += kHeads) {
    Vec8<IN> ry[kHeads], rz[kHeads];
    int64_t rows[kHeads];
    uint32_t hs[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      rows[j] = row, hs[j] = h;
      if (s + j < per_group && base + (int64_t)(s + j) * kGroups < units && in) {
        ry[j].load(reinterpret_cast<const IN*>(g.y) + row * g.ld_y + (int64_t)h * g.d + c);
        if (g.z) rz[j].load(reinterpret_cast<const IN*>(g.z) + row * g.ld_z + (int64_t)h * g.d + c);
      }
      h += kGroups;
      while (h >= (uint32_t)g.H) h -= g.H, ++row;
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (s + j >= per_group || base + (int64_t)(s + j) * kGroups >= units) break;  // uniform in the group
      float f[8];
      if (in) {
        ry[j].unpack(f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
      }
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float inv = rsqrtf(ss / (float)g.d + g.eps);
      if (in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv * w[i];
        if (g.z) {
          float z[8];
          rz[j].unpack(z);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= silu_f(z[i]);
        }
        store8(reinterpret_cast<OUT*>(g.out) + rows[j] * g.ld_out + (int64_t)hs[j] * g.d + c, f);
      }
    }
  }
}

// any d, any alignment: one warp per head, read twice (the second time from L1)
template <typename IN, typename OUT>
__global__ void __launch_bounds__(32 * kAnyWarps) head_norm_any_kernel(const HeadNormArgs g, int64_t units) {
  grid_dependency_begin();
  const int lane = threadIdx.x % 32;
  const int64_t u = (int64_t)blockIdx.x * kAnyWarps + threadIdx.x / 32;
  if (u >= units) return;
  const int64_t row = u / g.H, h = u % g.H;
  const IN* y = reinterpret_cast<const IN*>(g.y) + row * g.ld_y + h * g.d;
  const IN* z = g.z ? reinterpret_cast<const IN*>(g.z) + row * g.ld_z + h * g.d : nullptr;
  OUT* o = reinterpret_cast<OUT*>(g.out) + row * g.ld_out + h * g.d;
  float ss = 0.0f;
  for (uint32_t c = lane; c < (uint32_t)g.d; c += 32) {
    const float v = to_f32(y[c]);
    ss = fmaf(v, v, ss);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
  const float inv = rsqrtf(ss / (float)g.d + g.eps);
  for (uint32_t c = lane; c < (uint32_t)g.d; c += 32) {
    float v = to_f32(y[c]) * (inv * (g.weight ? g.weight[c] : 1.0f));
    if (z) v *= silu_f(to_f32(z[c]));
    o[c] = from_f32<OUT>(v);
  }
}

// 8-value accesses: base, row stride and head size keep every head's groups aligned
bool vec8(const void* p, int64_t ld, int d, int es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0 && d % 8 == 0);
}

template <typename IN, typename OUT, int G>
cudaError_t launch_qk_g(const QkNormArgs& a, int sms, cudaStream_t stream) {
  const int heads = a.Hq + a.Hk;
  const int64_t rows = a.B * a.T;
  // heads per group: all of a token's heads once there are enough tokens to
  // give every SM its threads, else fewer, so that a decode step's few tokens
  // still spread over the SMs
  const int64_t groups = (int64_t)sms * 1024 / G;
  int64_t slices = rows > 0 ? (groups + rows - 1) / rows : 1;
  if (slices > (heads + 3) / 4) slices = rows * ((heads + 3) / 4) * 2 > groups ? (heads + 3) / 4 : heads;
  if (slices < 1) slices = 1;
  const int per_group = (int)((heads + slices - 1) / slices);
  slices = (heads + per_group - 1) / per_group;
  const int64_t ctas = (rows * slices + kQkThreads / G - 1) / (kQkThreads / G);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)ctas), block(kQkThreads);
  const float inv_n = a.l2 ? 1.0f : 1.0f / (float)a.d;
  if (a.interleaved || a.rot == 0)
    return launch_pdl(true, qk_norm_kernel<IN, OUT, G, false>, grid, block, 0, stream, a, per_group, (int)slices, inv_n);
  return launch_pdl(true, qk_norm_kernel<IN, OUT, G, true>, grid, block, 0, stream, a, per_group, (int)slices, inv_n);
}

template <typename IN, typename OUT>
cudaError_t launch_qk_t(const QkNormArgs& a, int sms, cudaStream_t stream) {
  const int ei = sizeof(IN), eo = sizeof(OUT);
  const bool vec = vec8(a.Hq ? a.q : nullptr, a.ld_q, a.d, ei) && vec8(a.Hk ? a.k : nullptr, a.ld_k, a.d, ei) &&
                   vec8(a.Hq ? a.q_out : nullptr, a.ld_qo, a.d, eo) &&
                   vec8(a.Hk ? a.k_out : nullptr, a.ld_ko, a.d, eo) && vec8(a.q_weight, 0, a.d, 4) &&
                   vec8(a.k_weight, 0, a.d, 4) && a.d % 8 == 0 && a.rot % 8 == 0;
  if (!vec) {
    const int64_t ctas = (a.B * a.T * (a.Hq + a.Hk) + kAnyWarps - 1) / kAnyWarps;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(true, qk_norm_any_kernel<IN, OUT>, dim3((unsigned)ctas), dim3(32 * kAnyWarps), 0, stream, a);
  }
  if (a.d <= 64) return launch_qk_g<IN, OUT, 8>(a, sms, stream);
  if (a.d <= 128) return launch_qk_g<IN, OUT, 16>(a, sms, stream);
  return launch_qk_g<IN, OUT, 32>(a, sms, stream);
}

template <typename IN, typename OUT, int G>
cudaError_t launch_hn_g(const HeadNormArgs& a, int sms, cudaStream_t stream) {
  const int64_t units = a.rows * a.H;
  constexpr int kGroups = kHnThreads / G;
  // eight heads per group once that still fills every SM
  const int per_group = units >= (int64_t)sms * kHnCtas * kGroups * 8 ? 8 : 1;
  const int64_t ctas = (units + kGroups * per_group - 1) / (kGroups * per_group);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(true, head_norm_kernel<IN, OUT, G>, dim3((unsigned)ctas), dim3(kHnThreads), 0, stream, a, units,
                    per_group);
}

template <typename IN, typename OUT>
cudaError_t launch_hn_t(const HeadNormArgs& a, int sms, cudaStream_t stream) {
  const int ei = sizeof(IN), eo = sizeof(OUT);
  const bool vec = vec8(a.y, a.ld_y, a.d, ei) && vec8(a.z, a.ld_z, a.d, ei) && vec8(a.out, a.ld_out, a.d, eo) &&
                   a.d <= kMaxD;
  const int64_t units = a.rows * a.H;
  if (!vec) {
    const int64_t ctas = (units + kAnyWarps - 1) / kAnyWarps;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(true, head_norm_any_kernel<IN, OUT>, dim3((unsigned)ctas), dim3(32 * kAnyWarps), 0, stream, a,
                      units);
  }
  if (a.d <= 64) return launch_hn_g<IN, OUT, 8>(a, sms, stream);
  if (a.d <= 128) return launch_hn_g<IN, OUT, 16>(a, sms, stream);
  return launch_hn_g<IN, OUT, 32>(a, sms, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rotary(const QkNormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.B <= 0 || a.T <= 0 || a.Hq + a.Hk <= 0 || a.d <= 0) return cudaSuccess;
  if (a.in_bf16)
    return a.out_bf16 ? launch_qk_t<__nv_bfloat16, __nv_bfloat16>(a, dev.sm_count, stream)
                      : launch_qk_t<__nv_bfloat16, float>(a, dev.sm_count, stream);
  return a.out_bf16 ? launch_qk_t<float, __nv_bfloat16>(a, dev.sm_count, stream)
                    : launch_qk_t<float, float>(a, dev.sm_count, stream);
}

cudaError_t launch_head_norm_gated(const HeadNormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.rows <= 0 || a.H <= 0 || a.d <= 0) return cudaSuccess;
  if (a.in_bf16)
    return a.out_bf16 ? launch_hn_t<__nv_bfloat16, __nv_bfloat16>(a, dev.sm_count, stream)
                      : launch_hn_t<__nv_bfloat16, float>(a, dev.sm_count, stream);
  return a.out_bf16 ? launch_hn_t<float, __nv_bfloat16>(a, dev.sm_count, stream)
                    : launch_hn_t<float, float>(a, dev.sm_count, stream);
}

}  // namespace mamba
