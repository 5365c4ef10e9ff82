// gated_delta_step.cu - the gated delta rule token by token (formulas in
// gated_delta.cuh): the batched decode step (T = 1, state in place) and short
// prefills.  The same code runs both, so a T = 1 prefill is one step bit for bit.
//
// The rows of S do not see each other: with row s (dk values) of value
// component n,
//   r = s.k,  c = s.q,  u = beta (v_n - alpha r),  s' = alpha s + u k,
//   y_n = scale (alpha c + u (k.q))
// so one pass over the row gives both products, and the update needs no second
// reduction.  16 lanes hold a row (kV values per lane, four at a time with
// 16-byte accesses), a group of 16 lanes kR rows in registers, and the state is
// read and written once however many tokens the call has.
//
// Bound (step): HBM, the state read and written once.  4096 heads of 128 x 128:
// 80.6 us, 6650 GB/s.  What that takes is bytes in flight (six CTAs of 128 threads
// per SM, 128 bytes a thread: 80.6 us against 103.6 with the four that the registers
// of an unbounded kernel allow) and stores that leave the cache first (85 us without).
#include "gated_delta.cuh"

namespace mamba {
namespace {

constexpr int kGroup = 16;    // lanes per row
constexpr int kThreads = 128;
constexpr int kCtas = 6;      // per SM

template <typename T>
__device__ __forceinline__ float ld_in(const void* p, int64_t i) {
  return to_f32(reinterpret_cast<const T*>(p)[i]);
}

// this lane's kV values of a dk-vector: component 64 j + 4 lane + i
template <typename T, int kV, bool VEC>
__device__ __forceinline__ void load_vec(float (&out)[kV], const T* p, int lane, int dk) {
#pragma unroll
  for (int j = 0; j < kV / 4; ++j) {
    const int c = 64 * j + 4 * lane;
    if (VEC) {
      if (c < dk) {
        if constexpr (sizeof(T) == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p + c);
          out[4 * j] = x.x, out[4 * j + 1] = x.y, out[4 * j + 2] = x.z, out[4 * j + 3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(p + c);
          out[4 * j] = __uint_as_float(x.x << 16), out[4 * j + 1] = __uint_as_float(x.x & 0xffff0000u);
          out[4 * j + 2] = __uint_as_float(x.y << 16), out[4 * j + 3] = __uint_as_float(x.y & 0xffff0000u);
        }
      } else {
        out[4 * j] = out[4 * j + 1] = out[4 * j + 2] = out[4 * j + 3] = 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[4 * j + i] = c + i < dk ? to_f32(p[c + i]) : 0.0f;
    }
  }
}

// IN: activation type; kV: values per lane (dk <= 16 kV); VEC: dk % 4 == 0 and
// q, k rows aligned to four values
template <typename IN, int kV, int kR, bool VEC>
__global__ void __launch_bounds__(kThreads, kCtas) recurrent_kernel(const GatedDeltaArgs g) {
  grid_dependency_begin();
  const int lane = threadIdx.x % kGroup, group = threadIdx.x / kGroup;
  const int n_tiles = (g.dv + (kThreads / kGroup) * kR - 1) / ((kThreads / kGroup) * kR);
  // value tile fastest: the CTAs of one head share its k and q
  const int64_t bh = blockIdx.x / n_tiles;
  const int h = (int)(bh % g.Hv);
  const int64_t b = bh / g.Hv;
  const int n0 = ((int)(blockIdx.x % n_tiles) * (kThreads / kGroup) + group) * kR;
  const int hk = h / (g.Hv / g.Hk);

  float s[kR][kV];
  const int64_t s_off = (bh * g.dv + n0) * g.dk;
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    if (g.state_in && n0 + r < g.dv) {
      load_vec<float, kV, VEC>(s[r], g.state_in + s_off + (int64_t)r * g.dk, lane, g.dk);
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j) s[r][j] = 0.0f;
    }
  }
  const float neg_A = -expf(g.A_log[h]);
  const float dt_bias = g.dt_bias ? g.dt_bias[h] : 0.0f;

  for (int64_t t = 0; t < g.T; ++t) {
    const int64_t row = b * g.T + t;
    float k[kV], q[kV], v[kR];
    load_vec<IN, kV, VEC>(k, reinterpret_cast<const IN*>(g.k) + row * g.ld_k + (int64_t)hk * g.dk, lane, g.dk);
    load_vec<IN, kV, VEC>(q, reinterpret_cast<const IN*>(g.q) + row * g.ld_q + (int64_t)hk * g.dk, lane, g.dk);
#pragma unroll
    for (int r = 0; r < kR; ++r)
      v[r] = n0 + r < g.dv ? ld_in<IN>(g.v, row * g.ld_v + (int64_t)h * g.dv + n0 + r) : 0.0f;
    const float alpha = expf(gdr_log_alpha(ld_in<IN>(g.a, row * g.ld_a + h), dt_bias, neg_A));
    const float beta = gdr_beta(ld_in<IN>(g.b, row * g.ld_b + h));

    float sk[kR], sq[kR], kq = 0.0f;
#pragma unroll
    for (int j = 0; j < kV; ++j) kq = fmaf(k[j], q[j], kq);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      sk[r] = 0.0f, sq[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        sk[r] = fmaf(s[r][j], k[j], sk[r]);
        sq[r] = fmaf(s[r][j], q[j], sq[r]);
      }
    }
#pragma unroll
    for (int o = kGroup / 2; o > 0; o >>= 1) {
      kq += __shfl_xor_sync(0xffffffffu, kq, o);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        sk[r] += __shfl_xor_sync(0xffffffffu, sk[r], o);
        sq[r] += __shfl_xor_sync(0xffffffffu, sq[r], o);
      }
    }
    float out = 0.0f;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const float u = beta * (v[r] - alpha * sk[r]);
#pragma unroll
      for (int j = 0; j < kV; ++j) s[r][j] = fmaf(u, k[j], alpha * s[r][j]);
      const float yr = g.scale * fmaf(u, kq, alpha * sq[r]);
      if (lane == r) out = yr;
    }
    if (lane < kR && n0 + lane < g.dv)
      store_out(g.y, row * g.ld_y + (int64_t)h * g.dv + n0 + lane, g.y_bf16, out);
  }

  if (g.state_out) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (n0 + r >= g.dv) break;
      float* dst = g.state_out + s_off + (int64_t)r * g.dk;
#pragma unroll
      for (int j = 0; j < kV / 4; ++j) {
        const int c = 64 * j + 4 * lane;
        if (VEC) {
          if (c < g.dk)
            __stcs(reinterpret_cast<float4*>(dst + c),
                   make_float4(s[r][4 * j], s[r][4 * j + 1], s[r][4 * j + 2], s[r][4 * j + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < g.dk) dst[c + i] = s[r][4 * j + i];
        }
      }
    }
  }
}

template <typename IN, int kV, int kR, bool VEC>
cudaError_t launch_r(const GatedDeltaArgs& a, cudaStream_t stream) {
  constexpr int rows = (kThreads / kGroup) * kR;
  const int64_t ctas = a.B * a.Hv * ((a.dv + rows - 1) / rows);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(a.T == 1, recurrent_kernel<IN, kV, kR, VEC>, dim3((unsigned)ctas), dim3(kThreads), 0, stream, a);
}

// 32 values of the state per lane, or half of that where the rows are few: 8 heads
// of 128 x 128 2.9 us against 3.4, 4096 heads 82.3 against 80.6 (with dk = 64 65.4
// against 47.4).  A row's arithmetic is the same.
template <typename IN, int kV, bool VEC>
cudaError_t launch_v(const GatedDeltaArgs& a, int sms, cudaStream_t stream) {
  constexpr int kR = 32 / kV;
  if (a.B * a.Hv * a.dv < (int64_t)sms * (kThreads / kGroup) * kR) return launch_r<IN, kV, kR / 2, VEC>(a, stream);
  return launch_r<IN, kV, kR, VEC>(a, stream);
}

template <typename IN>
cudaError_t launch_in(const GatedDeltaArgs& a, int sms, cudaStream_t stream) {
  constexpr int al = 4 * sizeof(IN);
  auto ok = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % al == 0 && ld % 4 == 0; };
  auto ok_s = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = a.dk % 4 == 0 && ok(a.q, a.ld_q) && ok(a.k, a.ld_k) && ok_s(a.state_in) && ok_s(a.state_out);
  if (a.dk <= 64) return vec ? launch_v<IN, 4, true>(a, sms, stream) : launch_v<IN, 4, false>(a, sms, stream);
  if (a.dk <= 128) return vec ? launch_v<IN, 8, true>(a, sms, stream) : launch_v<IN, 8, false>(a, sms, stream);
  return vec ? launch_v<IN, 16, true>(a, sms, stream) : launch_v<IN, 16, false>(a, sms, stream);
}

}  // namespace

cudaError_t launch_gated_delta_recurrent(const GatedDeltaArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.B <= 0 || a.Hv <= 0 || a.dv <= 0) return cudaSuccess;
  return a.in_bf16 ? launch_in<__nv_bfloat16>(a, dev.sm_count, stream) : launch_in<float>(a, dev.sm_count, stream);
}

}  // namespace mamba
