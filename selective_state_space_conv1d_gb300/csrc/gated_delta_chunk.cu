// gated_delta_chunk.cu - the gated delta rule over long sequences, 64 tokens at
// a time on the tensor cores (formulas in gated_delta.cuh).
//
// With G_i the running sum of log alpha inside a chunk, K, Q, V its rows and S
// [dv][dk] the state before it, the chunk's corrections u_i = beta_i (v_i -
// alpha_i S_{i-1} k_i) solve a unit lower triangular system:
//
//   A_ij = beta_i e^{G_i - G_j} k_i.k_j (j < i),   T = (I + A)^-1
//   P_ij = e^{G_i - G_j} q_i.k_j (j <= i)
//   R    = beta (V - e^G K S^T)                    [64][dv]
//   U    = T R,   Y = scale (e^G Q S^T + (P T) R)
//   S'   = e^{G_63} S + U^T diag(e^{G_63 - G}) K
//
// T and P T do not depend on the state: one back substitution X (I + A) = [I; P],
// a thread a row, gives both while the previous chunk is still in flight.  What
// remains on the path from state to state is three products and their epilogues,
// all held transposed, a tensor-memory lane per value component n:
//
//   D1 = S [K; Q]^T   128 x 128 x dk     R^T  = D1's K half, gated  (epilogue 1)
//   D2 = R^T [T; PT]^T  128 x 128 x 64   U^T  = D2's T half         (epilogue 2)
//   D3 = U^T K          128 x dk x 64    S'   = e^G S + D3          (epilogue 3)
//
// S, R^T and U^T go back to tensor memory as the A operands of the next product:
// nothing of the chain touches shared memory, and a value component's power of
// two scale is a number per thread.  The f32 state stays in registers.
//
// Precision: every operand is f16 with a power-of-two scale per row, S, R, U, T
// and P T (and f32 inputs) as two halves hi + lo (22 bits; lo.lo products are
// dropped), bf16 keys and queries as one (exact).  Two halves in bf16 would hold
// 16 bits: measured in simulation 4e-6 of the state, against 2e-7 here and 1e-7
// for plain f32.  The scales keep every operand below 2^14 whatever the inputs'
// magnitudes: S by its largest value, R by the bound max|v| + max_i(beta_i
// e^{G_i} |k_i|_1) max|S|, U by that times the largest row sum of |T|.
//
// One CTA per (sequence, value head, 128 value components), warps specialised:
//   0-7   epilogues 1-3, output, the state in registers (lane = component; two
//         warps per lane quarter, each half the columns)
//   8-11  prepare: gates x products, back substitution, [T; PT] to shared memory
//   12-14 load: K, Q rows to scaled f16, V by cp.async, the gates
//   15    issues the MMAs
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/mamba_ssm.h"
#include "async_copy.cuh"
#include "gated_delta.cuh"
#include "tcgen05.cuh"

namespace mamba {
namespace {

constexpr int kC = 64;            // tokens per chunk
constexpr int kM = 128;           // value components per CTA
constexpr int kThreads = 16 * 32;
constexpr int kLoadWarps = 3, kLoadThreads = 32 * kLoadWarps, kMmaWarp = 15;
constexpr int kGateSlots = 4;
constexpr long long kWaitLimit = 1ll << 31;  // SM cycles (about a second)

__device__ int g_delta_faults = 0;

// per-chunk scalars and vectors, written by the load and prepare warps
struct Gates {
  float col_hi[kC], col_lo[kC];          // G_j + ek_j as two floats
  float row_hi[2 * kC], row_lo[2 * kC];  // G_i - ek_i (keys), G_i - eq_i (queries)
  float beta[kC];
  float fx[kC];    // beta_i e^{G_i} 2^{-ek_i}
  float fd[kC];    // e^{G_63 - G_i} 2^{-ek_i}
  float fq[kC];    // scale e^{G_i} 2^{-eq_i}
  float fu[kC];    // fd_i / T's row scale                     (prepare warps)
  float fp[kC];    // scale / (P T)'s row scale                (prepare warps)
  float total;     // e^{G_63}
  float k_bound;   // max_i beta_i e^{G_i} |k_i|_1 (bound)
  float u_bound[2];  // max_i fd_i sum_j |T_ij|, one of each prepare warp
};

template <int DK, bool F32>
struct Smem {
  static constexpr int kTerms = F32 ? 2 : 1;          // halves of K and Q
  static constexpr int kBlocks = DK / 64;
  static constexpr int kKqTerm = kBlocks * 16384;     // [K; Q]: 128 rows x 64 f16 per block
  static constexpr int kKq = kTerms * kKqTerm;
  static constexpr int kKqStages = F32 ? 2 : 3;
  static constexpr int kTp = 2 * 16384;               // [T; PT] hi, lo: 128 rows x 64 f16
  static constexpr int kTpStages = F32 ? 1 : 2;
  static constexpr int kV = kC * kM * (F32 ? 4 : 2);
  static constexpr int kVStages = F32 ? 1 : 2;
  static constexpr int kOffTp = kKqStages * kKq;
  static constexpr int kOffV = kOffTp + kTpStages * kTp;
  static constexpr int kOffA = kOffV + kVStages * kV;  // A, f32 [64][64]
  static constexpr int kOffGates = kOffA + kC * kC * 4;
  static constexpr int kOffMax = kOffGates + kGateSlots * (int)sizeof(Gates);  // [2][2][128] f32
  static constexpr int kOffExp = kOffMax + 2 * 2 * kM * 4;                     // [2][128] int
  static constexpr int kOffBar = kOffExp + 2 * 2 * kC * 4;
  static constexpr int kBars = 2 * kKqStages + 2 * kVStages + 2 * kTpStages + 2 + 7;
  static constexpr int kBytes = kOffBar + 8 * kBars + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(sizeof(Gates) % 16 == 0, "gate slots must keep 16-byte alignment");
  static_assert(kAlloc <= 232448, "shared memory over the opt-in limit");
};

// tensor memory columns
constexpr uint32_t kColX = 0, kColQ = 64, kColU = 128, kColO = 192, kColS = 256, kColD0 = 384, kTmemCols = 512;

// kind::f16, f16 A and B, f32 accumulator, M = 128; b_mn: B is MN-major
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory: lane = row, a 32-bit column = two values of K
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// floor(log2 x) of a positive float (-127 for zero and denormals, 128 for inf)
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255) - 127; }
// 2^e, e clamped to the normal range
__device__ __forceinline__ float pow2(int e) {
  e = e < -126 ? -126 : (e > 127 ? 127 : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// (a, b) as f16 pairs hi + lo
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 bytes global -> shared, zeros if !valid
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
// this thread's arrival on bar once its cp.async copies have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Eight values of a row as f32; zeros past `valid` of them
template <bool F32>
__device__ __forceinline__ void load8(float (&f)[8], const void* row, int64_t at, int valid, bool vec) {
  if (F32) {
    const float* p = reinterpret_cast<const float*>(row) + at;
    if (vec && valid >= 8) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < valid ? p[i] : 0.0f;
  } else {
    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(row) + at;
    if (vec && valid >= 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < valid ? __bfloat162float(p[i]) : 0.0f;
  }
}

template <int DK, bool F32>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const GatedDeltaArgs g, int vec_kq, int vec_v) {
  using L = Smem<DK, F32>;
  using In = typename std::conditional<F32, float, __nv_bfloat16>::type;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023) & ~1023u;  // 1024-byte aligned for the 128-byte swizzle
  unsigned char* gbase = smem_raw + (base - raw);
  uint32_t bar_at = base + L::kOffBar;
  auto next_bars = [&](int n) {
    const uint32_t b = bar_at;
    bar_at += 8 * n;
    return b;
  };
  const uint32_t kq_full = next_bars(L::kKqStages), kq_empty = next_bars(L::kKqStages);
  const uint32_t v_full = next_bars(L::kVStages), v_empty = next_bars(L::kVStages);
  const uint32_t tp_full = next_bars(L::kTpStages), tp_empty = next_bars(L::kTpStages);
  const uint32_t d0_full = next_bars(1), d0_empty = next_bars(1);
  const uint32_t s_ready = next_bars(1), x_full = next_bars(1), r_ready = next_bars(1), u_full = next_bars(1),
                 u_ready = next_bars(1), o_full = next_bars(1), s_full = next_bars(1);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(gbase + L::kOffBar + 8 * L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
  Gates* gates = reinterpret_cast<Gates*>(gbase + L::kOffGates);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tiles = (g.dv + kM - 1) / kM;
  const int tile = blockIdx.x % tiles;
  const int64_t bh = blockIdx.x / tiles;
  const int h = (int)(bh % g.Hv);
  const int64_t b = bh / g.Hv;
  const int hk = h / (g.Hv / g.Hk);
  const int n_chunks = (int)((g.T + kC - 1) / kC);

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kKqStages; ++s) mbar_init(kq_full + 8 * s, kLoadThreads), mbar_init(kq_empty + 8 * s, 1);
    for (int s = 0; s < L::kVStages; ++s) mbar_init(v_full + 8 * s, kLoadThreads), mbar_init(v_empty + 8 * s, 8);
    for (int s = 0; s < L::kTpStages; ++s) mbar_init(tp_full + 8 * s, 4), mbar_init(tp_empty + 8 * s, 1);
    mbar_init(d0_full, 1), mbar_init(d0_empty, 4);
    mbar_init(s_ready, 8), mbar_init(x_full, 1), mbar_init(r_ready, 8), mbar_init(u_full, 1);
    mbar_init(u_ready, 8), mbar_init(o_full, 1), mbar_init(s_full, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_ptr)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *tmem_ptr;

  // A wait that runs out sets the fault and abort flags; every role then runs
  // on through its loop without waiting, so that all named barriers are met and
  // the CTA ends.
  auto wait = [&](uint32_t bar, int phase) {
    if (*abort_flag) return;
    if (!mbar_wait(bar, (uint32_t)(phase & 1), kWaitLimit)) {
      atomicOr(&g_delta_faults, MAMBA_FAULT_DELTA_WAIT);
      *abort_flag = 1;
    }
  };

  if (warp < 8) {
    // ---------------------------------------------------------- epilogues ----
    constexpr int HK = DK / 2;  // key components per thread
    const int quad = warp & 3, half = warp >> 2;
    const int lane_n = quad * 32 + lane;
    const int n = tile * kM + lane_n;
    const bool live = n < g.dv;
    const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
    float* max_v = reinterpret_cast<float*>(gbase + L::kOffMax);  // [half][128]
    float* max_s = max_v + 2 * kM;
    float s[HK];
#pragma unroll
    for (int j = 0; j < HK; ++j) s[j] = 0.0f;
    if (g.state_in && live) {
      const float* p = g.state_in + (bh * g.dv + n) * g.dk + half * HK;
#pragma unroll
      for (int j = 0; j < HK; ++j)
        if (half * HK + j < g.dk) s[j] = p[j];
    }
    float s_max = 0.0f;
    int s_exp = 0;  // S is held as 2^{s_exp} S
    // this lane's state to tensor memory, scaled, in two halves: HK / 2 columns
    // of hi, HK / 2 of lo, then the other warp's
    auto put_state = [&]() {
      float mx = 0.0f;
#pragma unroll
      for (int j = 0; j < HK; ++j) mx = fmaxf(mx, fabsf(s[j]));
      if (mx > 3.4e38f) mx = 1.0f;  // not finite: the component is lost, any scale will do
      max_s[half * kM + lane_n] = mx;
      named_barrier(3 + quad, 64);
      s_max = fmaxf(mx, max_s[(1 - half) * kM + lane_n]);
      s_exp = 13 - exponent_of(s_max);
      s_exp = s_exp > 120 ? 120 : s_exp;
      const float c = pow2(s_exp);
#pragma unroll
      for (int j0 = 0; j0 < HK; j0 += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) split2(s[j0 + 2 * j] * c, s[j0 + 2 * j + 1] * c, hi[j], lo[j]);
        tmem_st16(t_lane + kColS + (uint32_t)(half * HK + j0 / 2), hi);
        tmem_st16(t_lane + kColS + (uint32_t)(half * HK + HK / 2 + j0 / 2), lo);
      }
      tmem_wait_st();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_ready);
    };
    put_state();

    for (int c = 0; c < n_chunks; ++c) {
      const Gates& gt = gates[c % kGateSlots];
      const int vs = c % L::kVStages;
      const In* v_tile = reinterpret_cast<const In*>(gbase + L::kOffV + vs * L::kV) + (half * 32) * kM + lane_n;
      const int i0 = half * 32;  // this thread's tokens
      // scale of R from its bound; the largest |v| of the lane needs the partner's tokens
      wait(v_full + 8 * vs, c / L::kVStages);
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(to_f32(v_tile[i * kM])));
      if (mx > 3.4e38f) mx = 1.0f;
      max_v[half * kM + lane_n] = mx;
      named_barrier(3 + quad, 64);
      mx = fmaxf(mx, max_v[(1 - half) * kM + lane_n]);
      wait(kq_full + 8 * (c % L::kKqStages), c / L::kKqStages);  // the gates
      int r_exp = 13 - exponent_of(fmaf(gt.k_bound, s_max, mx));
      r_exp = r_exp > 120 ? 120 : r_exp;
      {  // epilogue 1: R^T = beta V - fx D1
        const float cv = pow2(r_exp), cx = pow2(r_exp - s_exp);
        uint32_t x[32];
        wait(x_full, c);
        tcgen05_fence_after();
        tmem_ld32(t_lane + kColX + (uint32_t)i0, x);
        tmem_wait(x);
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 be = *reinterpret_cast<const float4*>(&gt.beta[i0 + i]);
          const float4 fx = *reinterpret_cast<const float4*>(&gt.fx[i0 + i]);
          float r[4];
          const float bes[4] = {be.x, be.y, be.z, be.w}, fxs[4] = {fx.x, fx.y, fx.z, fx.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            r[j] = bes[j] * (to_f32(v_tile[(i + j) * kM]) * cv) - fxs[j] * (__uint_as_float(x[i + j]) * cx);
          split2(r[0], r[1], hi[i / 2], lo[i / 2]);
          split2(r[2], r[3], hi[i / 2 + 1], lo[i / 2 + 1]);
        }
        tmem_st16(t_lane + kColX + (uint32_t)i0, hi);
        tmem_st16(t_lane + kColX + (uint32_t)(i0 + 16), lo);
        tmem_wait_st();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(r_ready), mbar_arrive(v_empty + 8 * vs);
      }
      int u_exp;  // epilogue 2: U^T, decayed to the chunk's end
      {
        uint32_t x[32];
        wait(u_full, c);
        tcgen05_fence_after();
        tmem_ld32(t_lane + kColU + (uint32_t)i0, x);
        u_exp = exponent_of(fmaxf(gt.u_bound[0], gt.u_bound[1])) + 1;
        const float cu = pow2(-u_exp);
        tmem_wait(x);
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 fu = *reinterpret_cast<const float4*>(&gt.fu[i0 + i]);
          split2(__uint_as_float(x[i]) * (fu.x * cu), __uint_as_float(x[i + 1]) * (fu.y * cu), hi[i / 2], lo[i / 2]);
          split2(__uint_as_float(x[i + 2]) * (fu.z * cu), __uint_as_float(x[i + 3]) * (fu.w * cu), hi[i / 2 + 1],
                 lo[i / 2 + 1]);
        }
        tmem_st16(t_lane + kColU + (uint32_t)i0, hi);
        tmem_st16(t_lane + kColU + (uint32_t)(i0 + 16), lo);
        tmem_wait_st();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(u_ready);
      }
      {  // output, while D3 is in flight
        wait(o_full, c);
        tcgen05_fence_after();
        const float cq = pow2(-s_exp), cp = pow2(-r_exp);
        const int64_t row0 = b * g.T + (int64_t)c * kC + i0;
        const int left = (int)(g.T - (int64_t)c * kC) - i0;  // tokens of this half inside the sequence
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
          uint32_t xq[16], xo[16];
          tmem_ld16(t_lane + kColQ + (uint32_t)(i0 + i), xq);
          tmem_ld16(t_lane + kColO + (uint32_t)(i0 + i), xo);
          tmem_wait(xq);
          tmem_wait(xo);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float o = gt.fq[i0 + i + j] * (__uint_as_float(xq[j]) * cq) +
                            gt.fp[i0 + i + j] * (__uint_as_float(xo[j]) * cp);
            if (live && i + j < left)
              store_out(g.y, (row0 + i + j) * g.ld_y + (int64_t)h * g.dv + n, g.y_bf16, o);
          }
        }
      }
      {  // epilogue 3: S = e^G S + D3
        const float total = gt.total, cd = pow2(u_exp - r_exp);
        wait(s_full, c);
        tcgen05_fence_after();
#pragma unroll
        for (int j0 = 0; j0 < HK; j0 += 16) {
          uint32_t x[16];
          tmem_ld16(t_lane + kColS + (uint32_t)(half * HK + j0), x);
          tmem_wait(x);
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j0 + j] = fmaf(total, s[j0 + j], __uint_as_float(x[j]) * cd);
        }
        if (c + 1 < n_chunks) put_state();
      }
    }
    if (g.state_out && live) {
      float* p = g.state_out + (bh * g.dv + n) * g.dk + half * HK;
#pragma unroll
      for (int j = 0; j < HK; ++j)
        if (half * HK + j < g.dk) p[j] = s[j];
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ prepare ----
    const int quad = warp & 3;
    const int row = quad * 32 + lane;       // row of [K; Q] and of [T; PT]
    const bool is_t = quad < 2;             // warp-uniform
    const int i = row & (kC - 1);           // token
    const uint32_t t_d0 = tmem + ((uint32_t)(quad * 32) << 16) + kColD0;
    float* a_s = reinterpret_cast<float*>(gbase + L::kOffA);
    for (int c = 0; c < n_chunks; ++c) {
      Gates& gt = gates[c % kGateSlots];
      const int st = c % L::kTpStages;
      float2 x[32];  // this row, pairs of columns
      wait(kq_full + 8 * (c % L::kKqStages), c / L::kKqStages);  // the gates
      wait(d0_full, c);
      tcgen05_fence_after();
      {
        const float rh = gt.row_hi[row], rl = gt.row_lo[row];
        const float scale_row = is_t ? gt.beta[i] : 1.0f;
        const int last = is_t ? i - 1 : i;  // A is strictly lower, P lower
#pragma unroll
        for (int j0 = 0; j0 < kC; j0 += 32) {
          uint32_t d[32];
          tmem_ld32(t_d0 + (uint32_t)j0, d);
          tmem_wait(d);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 ch = *reinterpret_cast<const float4*>(&gt.col_hi[j0 + j]);
            const float4 cl = *reinterpret_cast<const float4*>(&gt.col_lo[j0 + j]);
            const float chs[4] = {ch.x, ch.y, ch.z, ch.w}, cls[4] = {cl.x, cl.y, cl.z, cl.w};
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float w = ex2_approx((rh - chs[e]) + (rl - cls[e]));
              v[e] = j0 + j + e <= last ? __uint_as_float(d[j + e]) * w * scale_row : 0.0f;
            }
            x[(j0 + j) / 2] = make_float2(v[0], v[1]);
            x[(j0 + j) / 2 + 1] = make_float2(v[2], v[3]);
          }
        }
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d0_empty);
      }
      // A to shared memory (16-byte granule q of row i at q ^ (i % 8)), once
      // the previous chunk's substitution has read its own
      named_barrier(1, 128);
      if (is_t) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          *reinterpret_cast<float4*>(a_s + i * kC + 4 * (q ^ (i & 7))) =
              make_float4(x[2 * q].x, x[2 * q].y, x[2 * q + 1].x, x[2 * q + 1].y);
          x[2 * q] = make_float2(4 * q == i ? 1.0f : 0.0f, 4 * q + 1 == i ? 1.0f : 0.0f);
          x[2 * q + 1] = make_float2(4 * q + 2 == i ? 1.0f : 0.0f, 4 * q + 3 == i ? 1.0f : 0.0f);
        }
      }
      named_barrier(1, 128);
      // X (I + A) = [I; P], columns from the last: x_k is final once every
      // column after it has been taken off; rows 0-31 have nothing past column 31
      auto eliminate = [&](int k) {
        const float xk = (k & 1) ? x[k / 2].y : x[k / 2].x;
        const float2 nx = make_float2(-xk, -xk);
#pragma unroll
        for (int q = 0; q < (k + 3) / 4; ++q) {
          const float4 a = *reinterpret_cast<const float4*>(a_s + k * kC + 4 * (q ^ (k & 7)));
          x[2 * q] = __ffma2_rn(nx, make_float2(a.x, a.y), x[2 * q]);
          if (4 * q + 2 < k) x[2 * q + 1] = __ffma2_rn(nx, make_float2(a.z, a.w), x[2 * q + 1]);
        }
      };
      if (quad & 1) {
#pragma unroll
        for (int k = kC - 1; k >= 32; --k) eliminate(k);
      }
#pragma unroll
      for (int k = 31; k >= 1; --k) eliminate(k);
      // row scale, two halves, to shared memory
      float sum = 0.0f;
#pragma unroll
      for (int q = 0; q < 32; ++q) sum += fabsf(x[q].x) + fabsf(x[q].y);
      const int e = 13 - exponent_of(sum);
      const float cs = pow2(e), inv = pow2(-(e < -126 ? -126 : (e > 127 ? 127 : e)));
      if (c >= L::kTpStages) wait(tp_empty + 8 * st, c / L::kTpStages + 1);
      if (is_t) {
        gt.fu[i] = gt.fd[i] * inv;
        const float bound = gt.fd[i] * sum;
        const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(bound));
        if (lane == 0) gt.u_bound[quad] = __uint_as_float(top);
      } else {
        gt.fp[i] = g.scale * inv;
      }
      const uint32_t dst = base + L::kOffTp + st * L::kTp + (uint32_t)(row * 128);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split2(x[4 * q + j].x * cs, x[4 * q + j].y * cs, hi[j], lo[j]);
        const uint32_t at = dst + (uint32_t)((q ^ (row & 7)) << 4);
        st_shared16(at, hi[0], hi[1], hi[2], hi[3]);
        st_shared16(at + 16384, lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(tp_full + 8 * st);
    }
  } else if (warp < kMmaWarp) {
    // --------------------------------------------------------------- load ----
    const int lw = warp - 12, lt = threadIdx.x - 12 * 32;
    constexpr int kLanes = DK / 8;           // lanes per row
    constexpr int kRowsPer = 32 / kLanes;    // rows per warp and pass
    const int sub = lane / kLanes, col = (lane % kLanes) * 8;
    const float neg_A = -expf(g.A_log[h]);
    const float dt_bias = g.dt_bias ? g.dt_bias[h] : 0.0f;
    const int valid = g.dk - col;            // of this lane's eight components
    for (int c = 0; c < n_chunks; ++c) {
      const int ks = c % L::kKqStages, vs = c % L::kVStages;
      const int64_t t0 = (int64_t)c * kC;
      const int left = (int)(g.T - t0 < kC ? g.T - t0 : kC);
      const int64_t row0 = b * g.T + t0;
      int* exps = reinterpret_cast<int*>(gbase + L::kOffExp) + (c & 1) * 2 * kC;
      if (c >= L::kKqStages) wait(kq_empty + 8 * ks, c / L::kKqStages + 1);
      // K (rows 0-63) and Q (64-127), each row scaled to [2^13, 2^14)
      constexpr int kBatch = F32 ? 4 : 8;
      constexpr int kStep = kLoadWarps * kRowsPer;  // rows per pass
#pragma unroll 1
      for (int p0 = 0; p0 * kStep < 2 * kC; p0 += kBatch) {
        float f[kBatch][8];
#pragma unroll
        for (int p = 0; p < kBatch; ++p) {
          const int r = (p0 + p) * kStep + lw * kRowsPer + sub;
          const int i = r & (kC - 1);
          const bool in = i < left && valid > 0 && r < 2 * kC;
          const void* src = r < kC ? g.k : g.q;
          const int64_t ld = r < kC ? g.ld_k : g.ld_q;
          load8<F32>(f[p], src, in ? (row0 + i) * ld + (int64_t)hk * g.dk + col : 0, in ? valid : 0, vec_kq);
        }
#pragma unroll
        for (int p = 0; p < kBatch; ++p) {
          const int r = (p0 + p) * kStep + lw * kRowsPer + sub;
          float mx = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(f[p][j]));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          int e = 13 - exponent_of(mx);
          e = e > 120 ? 120 : e;  // a zero row: 120, so that its bound below is nothing
          if (r >= 2 * kC) continue;  // a lane past the last row; the shuffles are behind it
          if (col == 0) exps[r] = e;
          const float cs = pow2(e);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (F32) {
              split2(f[p][2 * j] * cs, f[p][2 * j + 1] * cs, hi[j], lo[j]);
            } else {
              const __half2 t = __floats2half2_rn(f[p][2 * j] * cs, f[p][2 * j + 1] * cs);
              hi[j] = *reinterpret_cast<const uint32_t*>(&t);
            }
          }
          const uint32_t at = base + ks * L::kKq + (uint32_t)((col / 64) * 16384 + r * 128 +
                                                              ((((col & 63) / 8) ^ (r & 7)) << 4));
          st_shared16(at, hi[0], hi[1], hi[2], hi[3]);
          if (F32) st_shared16(at + L::kKqTerm, lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      named_barrier(2, kLoadThreads);  // every row's exponent is there
      if (lw == 0) {
        // the gates of tokens lane and lane + 32: base-2 logarithms, summed in 64
        // bits and kept as two floats, so that differences of far-decayed tokens
        // keep 32-bit accuracy.  alpha below 2^-256 is 0 in f32 all the same.
        Gates& gt = gates[c % kGateSlots];
        double G[2];
        float be[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = lane + 32 * u;
          const bool in = i < left;
          const float a = in ? to_f32(reinterpret_cast<const In*>(g.a)[(row0 + i) * g.ld_a + h]) : 0.0f;
          const float bb = in ? to_f32(reinterpret_cast<const In*>(g.b)[(row0 + i) * g.ld_b + h]) : 0.0f;
          const float la = gdr_log_alpha(a, dt_bias, neg_A);
          G[u] = in ? (double)(la < -200.0f ? -200.0f : la) * 1.4426950408889634 : 0.0;
          be[u] = in ? gdr_beta(bb) : 0.0f;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double t = __shfl_up_sync(0xffffffffu, G[u], o);
            if (lane >= o) G[u] += t;
          }
        }
        G[1] += __shfl_sync(0xffffffffu, G[0], 31);
        const double last = __shfl_sync(0xffffffffu, G[1], 31);
        float kb = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = lane + 32 * u;
          const int ek = exps[i], eq = exps[kC + i];
          const double cj = G[u] + (double)ek, rk = G[u] - (double)ek, rq = G[u] - (double)eq;
          const float eg = ex2_approx((float)G[u]);
          gt.col_hi[i] = (float)cj, gt.col_lo[i] = (float)(cj - (double)(float)cj);
          gt.row_hi[i] = (float)rk, gt.row_lo[i] = (float)(rk - (double)(float)rk);
          gt.row_hi[kC + i] = (float)rq, gt.row_lo[kC + i] = (float)(rq - (double)(float)rq);
          gt.beta[i] = be[u];
          gt.fx[i] = be[u] * eg * pow2(-ek);
          gt.fd[i] = ex2_approx((float)(last - G[u])) * pow2(-ek);
          gt.fq[i] = g.scale * eg * pow2(-eq);
          // |k|_1 <= DK max|k| < DK 2^{14 - ek}
          kb = fmaxf(kb, be[u] * eg * (float)DK * pow2(14 - ek));
        }
        const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(kb));
        if (lane == 0) gt.k_bound = __uint_as_float(top), gt.total = ex2_approx((float)last);
      }
      mbar_arrive(kq_full + 8 * ks);
      // V: straight to shared memory
      if (c >= L::kVStages) wait(v_empty + 8 * vs, c / L::kVStages + 1);
      {
        const uint32_t dst = base + L::kOffV + vs * L::kV;
        const In* src = reinterpret_cast<const In*>(g.v) + (int64_t)h * g.dv + tile * kM;
        const int cols = g.dv - tile * kM < kM ? g.dv - tile * kM : kM;
        constexpr int kPer = 16 / (int)sizeof(In);  // values per granule
        constexpr int kGr = kM / kPer;
        if (vec_v) {
#pragma unroll 4
          for (int e = lt; e < kC * kGr; e += kLoadThreads) {
            const int r = e / kGr, q = e % kGr;
            const bool in = r < left && q * kPer < cols;
            cp_async16(dst + (uint32_t)(e * 16), in ? src + (row0 + r) * g.ld_v + q * kPer : src, in);
          }
          cp_async_arrive(v_full + 8 * vs);
        } else {
          In* d = reinterpret_cast<In*>(gbase + L::kOffV + vs * L::kV);
          for (int e = lt; e < kC * kM; e += kLoadThreads) {
            const int r = e / kM, q = e % kM;
            d[e] = r < left && q < cols ? src[(row0 + r) * g.ld_v + q] : from_f32<In>(0.0f);
          }
          mbar_arrive(v_full + 8 * vs);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // --------------------------------------------------------------- MMAs ----
    if (lane == 0) {
      constexpr uint32_t id64 = idesc_f16(64, false), id3 = idesc_f16(DK, true);
      constexpr int HK = DK / 2;
      // column of S's values 16 ks ..: half by half, hi then lo
      auto s_col = [](int ks, int lo) { return (uint32_t)((16 * ks / HK) * HK + (16 * ks % HK) / 2 + lo * (HK / 2)); };
      auto r_col = [](int ks, int lo) { return (uint32_t)((ks / 2) * 32 + (ks % 2) * 8 + lo * 16); };
      // [K; Q] K^T of chunk c, for the prepare warps
      auto issue_d0 = [&](int c) {
        const int ks = c % L::kKqStages;
        const uint32_t kq = base + ks * L::kKq;
        wait(kq_full + 8 * ks, c / L::kKqStages);
        if (c > 0) wait(d0_empty, c - 1);
        tcgen05_fence_after();
        uint32_t acc = 0;
#pragma unroll
        for (int term = 0; term < (F32 ? 3 : 1); ++term) {
          const int a_lo = term == 1, b_lo = term == 2;
#pragma unroll
          for (int k = 0; k < DK / 16; ++k) {
            const uint64_t ad = smem_desc(kq + a_lo * L::kKqTerm + (k / 4) * 16384) + 2 * (k % 4);
            const uint64_t bd = smem_desc(kq + b_lo * L::kKqTerm + (k / 4) * 16384) + 2 * (k % 4);
            mma_ss(tmem + kColD0, ad, bd, id64, acc);
            acc = 1;
          }
        }
        mma_commit(d0_full);
      };
      issue_d0(0);
      for (int c = 0; c < n_chunks; ++c) {
        const int ks = c % L::kKqStages, st = c % L::kTpStages;
        const uint32_t kq = base + ks * L::kKq, tp = base + L::kOffTp + st * L::kTp;
        wait(s_ready, c);
        tcgen05_fence_after();
        // D1: S_hi K_hi + S_lo K_hi (+ S_hi K_lo); keys first, the queries'
        // half runs under epilogue 1
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t acc = 0;
#pragma unroll
          for (int term = 0; term < (F32 ? 3 : 2); ++term) {
            const int s_lo = term == 1, k_lo = term == 2;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
              const uint64_t bd =
                  smem_desc(kq + k_lo * L::kKqTerm + (k / 4) * 16384 + part * 8192) + 2 * (k % 4);
              mma_ts(tmem + (part ? kColQ : kColX), tmem + kColS + s_col(k, s_lo), bd, id64, acc);
              acc = 1;
            }
          }
          if (part == 0) mma_commit(x_full);
        }
        // one chunk ahead; the prepare warps have long read this chunk's
        if (c + 1 < n_chunks) issue_d0(c + 1);
        wait(tp_full + 8 * st, c / L::kTpStages);
        wait(r_ready, c);
        tcgen05_fence_after();
        // D2: R_hi T_hi + R_hi T_lo + R_lo T_hi; T's half first
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t acc = 0;
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            const int r_lo = term == 2, t_lo = term == 1;
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {
              const uint64_t bd = smem_desc(tp + t_lo * 16384 + part * 8192) + 2 * k;
              mma_ts(tmem + (part ? kColO : kColU), tmem + kColX + r_col(k, r_lo), bd, id64, acc);
              acc = 1;
            }
          }
          mma_commit(part ? o_full : u_full);
        }
        mma_commit(tp_empty + 8 * st);
        wait(u_ready, c);
        tcgen05_fence_after();
        // D3: U_hi K_hi + U_lo K_hi (+ U_hi K_lo); K's rows are the contraction
        {
          uint32_t acc = 0;
#pragma unroll
          for (int term = 0; term < (F32 ? 3 : 2); ++term) {
            const int u_lo = term == 1, k_lo = term == 2;
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {
              const uint64_t bd = smem_desc(kq + k_lo * L::kKqTerm + k * 2048, 16384);
              mma_ts(tmem + kColS, tmem + kColU + r_col(k, u_lo), bd, id3, acc);
              acc = 1;
            }
          }
        }
        mma_commit(s_full);
        mma_commit(kq_empty + 8 * ks);
      }
      // the last commit has arrived (and with it every MMA is done) before
      // tensor memory is freed and the barriers go away
      const int last = n_chunks - 1;
      if (!mbar_wait(kq_empty + 8 * (last % L::kKqStages), (uint32_t)(last / L::kKqStages) & 1, kWaitLimit))
        atomicOr(&g_delta_faults, MAMBA_FAULT_DELTA_WAIT);
    }
    __syncwarp();
  }
  tcgen05_fence_before();
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <int DK, bool F32>
cudaError_t launch_chunk(const GatedDeltaArgs& a, cudaStream_t stream) {
  auto kern = chunk_kernel<DK, F32>;
  constexpr int smem = Smem<DK, F32>::kAlloc;
  static int configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!__atomic_load_n(&configured[dev], __ATOMIC_RELAXED)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    __atomic_store_n(&configured[dev], 1, __ATOMIC_RELAXED);
  }
  const int es = F32 ? 4 : 2;
  auto rows16 = [&](const void* p, int64_t ld, int d) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0 && (d * es) % 16 == 0;
  };
  const int vec_kq = rows16(a.k, a.ld_k, a.dk) && rows16(a.q, a.ld_q, a.dk) && a.dk % 8 == 0;
  const int vec_v = rows16(a.v, a.ld_v, a.dv);
  const int64_t ctas = a.B * a.Hv * ((a.dv + kM - 1) / kM);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  kern<<<(unsigned)ctas, kThreads, smem, stream>>>(a, vec_kq, vec_v);
  return cudaGetLastError();
}

}  // namespace

bool gated_delta_takes_chunks(const GatedDeltaArgs& a) { return a.dk <= 128 && a.T > 16; }

cudaError_t launch_gated_delta_chunk(const GatedDeltaArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  (void)dev;
  if (a.B <= 0 || a.Hv <= 0 || a.dv <= 0) return cudaSuccess;
  if (a.dk <= 64) return a.in_bf16 ? launch_chunk<64, false>(a, stream) : launch_chunk<64, true>(a, stream);
  return a.in_bf16 ? launch_chunk<128, false>(a, stream) : launch_chunk<128, true>(a, stream);
}

int read_delta_faults(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_delta_faults, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_delta_faults, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace mamba
