// block_norm.cu - the residual stream between two blocks, in one pass:
//
//   n    = y, or y / sqrt(mean_j y_j^2 + eps) post_j     (the norm after a block)
//   x'   = x + scale gate . n                            (its gate and residual scale)
//   out  = x' / sqrt(mean_j x'_j^2 + eps) pre_j          (the norm before the next block)
//
// Bound: HBM.  A row's x and y are read once and stay in registers through both
// sums; x' and out are written once: 12 bytes an element with bf16 y and out
// (32768 rows of 2560: 158 us, 6.4 TB/s; 128 rows of 768: 1.65 us, a launch's own time).
// One CTA per row, 8 elements per thread and turn (16-byte accesses).  A row
// over the registers' size, or with rows off the 16-byte boundary, runs a loop that keeps
// nothing and reads y (and the x' it wrote) again.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_math.cuh"
#include "launch.h"

namespace mamba {
namespace {

constexpr int kVec = 8;
constexpr int kMaxThreads = 512;
constexpr int kMaxTurns = 4;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// the sum over the CTA, in an order that does not depend on the row; `slot` has room for 32
__device__ __forceinline__ float cta_sum(float v, float* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x / 32;
  if (threadIdx.x % 32 == 0) slot[threadIdx.x / 32] = v;
  __syncthreads();
  float s = slot[0];
  for (int w = 1; w < warps; ++w) s += slot[w];
  return s;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const void* p, int64_t row, int64_t ld) {
  return static_cast<const T*>(p) + row * ld;
}

template <typename TY, typename TO, typename TG, int TURNS>
__global__ void __launch_bounds__(kMaxThreads) block_norm_rows_kernel(const BlockNormArgs a) {
  __shared__ float slots[2][32];
  const int64_t row = blockIdx.x;
  const int D = (int)a.D;
  grid_dependency_begin();
  const float* x = a.x + row * a.ld_x;
  const TY* y = row_of<TY>(a.y, row, a.ld_y);
  const TG* gate = a.gate ? row_of<TG>(a.gate, a.gate_rows ? row / a.gate_rows : 0, a.ld_gate) : nullptr;
  float xv[TURNS][kVec], yv[TURNS][kVec];
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int j = (i * blockDim.x + threadIdx.x) * kVec;
    if (j < D) {
      load8(x + j, xv[i]);
      load8(y + j, yv[i]);
    }
  }
  float inv = 1.0f;
  if (a.post) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < TURNS; ++i)
      if ((i * (int)blockDim.x + (int)threadIdx.x) * kVec < D)
#pragma unroll
        for (int e = 0; e < kVec; ++e) ss = fmaf(yv[i][e], yv[i][e], ss);
    inv = rsqrtf(cta_sum(ss, slots[0]) / (float)D + a.eps);
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int j = (i * blockDim.x + threadIdx.x) * kVec;
    if (j >= D) continue;
    if (a.post) {
      float w[kVec];
      load8(a.post + j, w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) yv[i][e] = yv[i][e] * inv * w[e];
    }
    if (gate) {
      float w[kVec];
      load8(gate + j, w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) yv[i][e] *= w[e];
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      xv[i][e] = fmaf(a.scale, yv[i][e], xv[i][e]);
      ss = fmaf(xv[i][e], xv[i][e], ss);
    }
    store8(a.x_out + row * a.ld_xo + j, xv[i]);
  }
  if (!a.out) return;
  inv = rsqrtf(cta_sum(ss, slots[1]) / (float)D + a.eps);
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int j = (i * blockDim.x + threadIdx.x) * kVec;
    if (j >= D) continue;
    float w[kVec];
    load8(a.pre + j, w);
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[e] = xv[i][e] * inv * w[e];
    store8(static_cast<TO*>(a.out) + row * a.ld_out + j, w);
  }
}

// any length, stride and alignment: nothing kept between the passes (each thread
// reads again only what it wrote itself)
template <typename TY, typename TO, typename TG>
__global__ void __launch_bounds__(kMaxThreads) block_norm_any_kernel(const BlockNormArgs a) {
  __shared__ float slots[2][32];
  const int64_t row = blockIdx.x;
  grid_dependency_begin();
  const float* x = a.x + row * a.ld_x;
  float* xo = a.x_out + row * a.ld_xo;
  const TY* y = row_of<TY>(a.y, row, a.ld_y);
  const TG* gate = a.gate ? row_of<TG>(a.gate, a.gate_rows ? row / a.gate_rows : 0, a.ld_gate) : nullptr;
  float inv = 1.0f;
  if (a.post) {
    float ss = 0.0f;
    for (int64_t j = threadIdx.x; j < a.D; j += blockDim.x) {
      const float v = to_f32(y[j]);
      ss = fmaf(v, v, ss);
    }
    inv = rsqrtf(cta_sum(ss, slots[0]) / (float)a.D + a.eps);
  }
  float ss = 0.0f;
  for (int64_t j = threadIdx.x; j < a.D; j += blockDim.x) {
    float n = to_f32(y[j]);
    if (a.post) n = n * inv * a.post[j];
    if (gate) n *= to_f32(gate[j]);
    const float v = fmaf(a.scale, n, x[j]);
    xo[j] = v;
    ss = fmaf(v, v, ss);
  }
  if (!a.out) return;
  inv = rsqrtf(cta_sum(ss, slots[1]) / (float)a.D + a.eps);
  TO* out = static_cast<TO*>(a.out) + row * a.ld_out;
  for (int64_t j = threadIdx.x; j < a.D; j += blockDim.x) out[j] = from_f32<TO>(xo[j] * inv * a.pre[j]);
}

bool aligned(const void* p, int64_t ld, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0;
}

template <typename TY, typename TO, typename TG>
cudaError_t launch_typed(const BlockNormArgs& a, int sms, cudaStream_t stream) {
  const dim3 grid((unsigned)a.M);
  const bool vec = a.D % kVec == 0 && aligned(a.x, a.ld_x, 4) && aligned(a.x_out, a.ld_xo, 4) &&
                   aligned(a.y, a.ld_y, sizeof(TY)) && aligned(a.out, a.ld_out, sizeof(TO)) &&
                   aligned(a.gate, a.ld_gate, sizeof(TG)) && aligned(a.pre, 0, 4) && aligned(a.post, 0, 4);
  const int64_t vecs = a.D / kVec;
  if (!vec || vecs > kMaxThreads * kMaxTurns) {
    const int threads = a.D >= kMaxThreads * 4 ? kMaxThreads : 128;
    return launch_pdl(true, block_norm_any_kernel<TY, TO, TG>, grid, dim3(threads), 0, stream, a);
  }
  // two turns a thread, four for a row over 512 threads; one for a short row, and where a
  // few rows leave the SMs idle (2560 components, us: one row 2.3 against 3.0, 32768 rows 175
  // against 158)
  const bool one = vecs <= 128 || (vecs <= kMaxThreads && a.M <= 4 * (int64_t)sms);
  const int turns = one ? 1 : (vecs <= 2 * kMaxThreads ? 2 : 4);
  const int threads = (int)((vecs + turns - 1) / turns + 31) / 32 * 32;
  if (turns == 1) return launch_pdl(true, block_norm_rows_kernel<TY, TO, TG, 1>, grid, dim3(threads), 0, stream, a);
  if (turns == 2) return launch_pdl(true, block_norm_rows_kernel<TY, TO, TG, 2>, grid, dim3(threads), 0, stream, a);
  return launch_pdl(true, block_norm_rows_kernel<TY, TO, TG, 4>, grid, dim3(threads), 0, stream, a);
}

template <typename TY, typename TO>
cudaError_t launch_gate(const BlockNormArgs& a, int sms, cudaStream_t s) {
  return a.gate_bf16 ? launch_typed<TY, TO, __nv_bfloat16>(a, sms, s) : launch_typed<TY, TO, float>(a, sms, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.M <= 0 || a.D <= 0) return cudaSuccess;
  const int sms = dev.sm_count;
  if (a.y_bf16)
    return a.out_bf16 ? launch_gate<__nv_bfloat16, __nv_bfloat16>(a, sms, stream)
                      : launch_gate<__nv_bfloat16, float>(a, sms, stream);
  return a.out_bf16 ? launch_gate<float, __nv_bfloat16>(a, sms, stream) : launch_gate<float, float>(a, sms, stream);
}

}  // namespace mamba
