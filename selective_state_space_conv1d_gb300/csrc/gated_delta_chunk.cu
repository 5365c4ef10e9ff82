// gated_delta_chunk.cu - the gated delta rule over long sequences, 64 tokens at
// a time on the tensor cores (formulas in gated_delta.cuh).
//
// With G_i the running sum of log alpha inside a chunk, K, Q, V its rows and S
// [dv][dk] the state before it, the chunk's corrections u_i = beta_i (v_i -
// alpha_i S_{i-1} k_i) solve a unit lower triangular system:
//
//   A_ij = beta_i e^{G_i - G_j} k_i.k_j (j < i),   T = (I + A)^-1 diag(beta)
//   P_ij = e^{G_i - G_j} q_i.k_j (j <= i),         W = P T
//   R    = V - e^G K S^T                           [64][dv]
//   U    = diag(e^{G_63 - G}) T R,   Y = scale (e^G Q S^T + W R)
//   S'   = e^{G_63} S + U^T K
//
// T and W do not depend on the state: X (I + A) = [I; P] gives both while the
// previous chunk is still in flight, solved in blocks of 16 columns: the
// diagonal blocks of I + A are inverted by substitution (a lane a row), the
// products with them and with the blocks beside them are warp-level tensor-core
// products in three TF32 terms.  (A thread a row for the whole substitution read
// A 64 times over from shared memory, 7-8 us a chunk.)  What remains on the path
// from state to state is three products and their epilogues, all held
// transposed, a tensor-memory lane per value component n:
//
//   D1 = S [K; Q]^T     128 x 128 x dk   R^T = V^T - D1's K half    (epilogue 1)
//   D2 = R^T [T; W]^T   128 x 128 x 64   U^T = D2's T half          (epilogue 2)
//   D3 = U^T K          128 x dk x 64    S'  = e^G S + D3           (epilogue 3)
//
// S, R^T and U^T go back to tensor memory as the A operands of the next product:
// nothing of the chain touches shared memory, and a value component's power of
// two scale is a number per thread.  The f32 state stays in registers.
//
// Precision: every operand is f16 with power-of-two scales (per row of K, Q, S
// and R; one for T and one for W), S, R, U, T and W (and f32 inputs) as two
// halves hi + lo (22 bits; lo.lo products are dropped), bf16 keys and queries as
// one (exact).  Two halves in bf16 would hold
// 16 bits: measured in simulation 4e-6 of the state, against 2e-7 here and 1e-7
// for plain f32.  The scales keep every operand below 2^14 whatever the inputs'
// magnitudes: S and R by their largest values (per value component), T and W by
// their largest row sum, which bounds U.
//
// One CTA per (sequence, value head, 128 value components), warps specialised:
//   0-7   epilogues 1-3, output, the state in registers (lane = component; two
//         warps per lane quarter, each half the columns)
//   8-11  prepare: A and P from [K; Q] K^T and the gates, T and W to shared memory
//   12-13 load: tensor copies of K, Q, V tiles, K and Q to scaled f16
//   14    the gates
//   15    issues the MMAs
// Every warp runs straight through its part of a chunk once, so the loop bodies
// are kept rolled where registers allow it: with everything unrolled the code
// was 177 KB and a chunk took 17-21 us, waiting for instructions.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <atomic>
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
constexpr int kLoadWarps = 2, kLoadThreads = 32 * kLoadWarps, kGateWarp = 14, kMmaWarp = 15;
constexpr int kGateSlots = 4;
constexpr long long kWaitLimit = 1ll << 31;  // SM cycles (about a second)

__device__ int g_delta_faults = 0;

constexpr int kLdA = kC + 4;      // row stride of A and P in shared memory, floats

// per-chunk scalars and vectors, written by the gate and prepare warps
struct Gates {
  float col_hi[kC], col_lo[kC];          // G_j + ek_j as two floats
  float row_hi[2 * kC], row_lo[2 * kC];  // G_i - ek_i (keys), G_i - eq_i (queries)
  float beta[kC];
  float fx[kC];    // e^{G_i} 2^{-ek_i}
  float fd[kC];    // e^{G_63 - G_i} 2^{-ek_i}
  float fq[kC];    // scale e^{G_i} 2^{-eq_i}
  float past[32];  // e^{G_31 - G_j} 2^{-ek_j}, j < 32
  float since[2][32];  // -beta_i e^{G_i - G_31} 2^{-ek_i}, e^{G_i - G_31} 2^{-eq_i}, i = 32 ..
  float total;     // e^{G_63}
  int t_exp, w_exp;  // T and W are held as 2^{t_exp} T, 2^{w_exp} W   (prepare warps)
  float pad;
  float sum_t[4], sum_w[4];  // largest row sums, one per prepare warp
};

template <int DK, bool F32>
struct Smem {
  static constexpr int kTerms = F32 ? 2 : 1;          // halves of K and Q
  static constexpr int kBlocks = DK / 64;
  static constexpr int kKqTerm = kBlocks * 16384;     // [K; Q]: 128 rows x 64 f16 per block
  static constexpr int kKq = kTerms * kKqTerm;
  static constexpr int kKqStages = F32 ? 2 : 3;
  static constexpr int kTp = 2 * 16384;               // [T; W] hi, lo: 128 rows x 64 f16
  static constexpr int kV = F32 ? 0 : kC * kM * 2;    // f32 values are read where they are used
  static constexpr int kRaw = F32 ? 0 : 2 * kC * DK * 2;  // K and Q rows as stored (bf16)
  static constexpr int kOffTp = kKqStages * kKq;
  static constexpr int kOffV = kOffTp + kTp;
  static constexpr int kOffRaw = kOffV + kV;
  static constexpr int kOffA = kOffRaw + kRaw;         // A and P, f32 [64][kLdA] each
  static constexpr int kOffGates = kOffA + 2 * kC * kLdA * 4;
  static constexpr int kOffMax = kOffGates + kGateSlots * (int)sizeof(Gates);  // [2][2][128] f32
  static constexpr int kOffExp = kOffMax + 2 * 2 * kM * 4;                     // [2][128] int
  static constexpr int kOffBar = kOffExp + 2 * 2 * kC * 4;
  static constexpr int kBars = 2 * kKqStages + 2 + 1 + 2 + 4 + 7;
  static constexpr int kBytes = kOffBar + 8 * kBars + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(sizeof(Gates) % 16 == 0, "gate slots must keep 16-byte alignment");
  static_assert(kAlloc <= 232448, "shared memory over the opt-in limit");
};

// tensor memory columns (two D0 buffers)
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
  hi = *reinterpret_cast<const uint32_t*>(&h);
  float ra, rb;  // hi - value, exact
  asm("{\n"
      "  .reg .f16 l, h;\n"
      "  mov.b32 {l, h}, %2;\n"
      "  sub.rn.f32.f16 %0, l, %3;\n"
      "  sub.rn.f32.f16 %1, h, %4;\n"
      "}\n"
      : "=f"(ra), "=f"(rb)
      : "r"(hi), "f"(a), "f"(b));
  const __half2 l = __floats2half2_rn(-ra, -rb);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// four 8 x 8 matrices of 16-bit values, lane l holding two of row l / 4 of each
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// A wait that did not succeed at once.  One that runs out sets the fault and
// abort flags; every role then runs on through its loop without waiting, so
// that all named barriers are met and the CTA ends.
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (*abort_flag) return;
  if (!mbar_wait(bar, parity, kWaitLimit)) {
    atomicOr(&g_delta_faults, MAMBA_FAULT_DELTA_WAIT);
    *abort_flag = 1;
  }
}

// a box of a three-dimensional tensor map to shared memory
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// x as two TF32 terms (11 bits each; the tensor cores ignore the bits below)
struct Tf32x2 {
  uint32_t hi, lo;
  __device__ __forceinline__ void set(float x) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
  }
};
// D[16][8] += A[16][8] B[8][8], f32 accumulators.  The 8 values of the
// contraction are taken in the order 0 2 4 6 1 3 5 7 on both sides: then the
// accumulator of one product is the A operand of the next as it stands.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A operand (hi, lo) from an accumulator
__device__ __forceinline__ void tf32_operand(uint32_t (&hi)[4], uint32_t (&lo)[4], const float (&c)[4]) {
  const float v[4] = {c[0], c[2], c[1], c[3]};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Tf32x2 t;
    t.set(v[i]);
    hi[i] = t.hi, lo[i] = t.lo;
  }
}

__device__ __forceinline__ void unpack8(float (&f)[8], uint4 a) {  // bf16
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

// A number as the unevaluated sum of two floats
struct Two {
  float h, l;
};
// log2(e) la
__device__ __forceinline__ Two two_log2(float la) {
  const float p = la * 1.44269502f;  // log2(e) is 1.44269502 + 1.92596299e-8
  return Two{p, fmaf(la, 1.44269502f, -p) + la * 1.92596299e-8f};
}
__device__ __forceinline__ Two two_add(Two a, Two b) {
  const float s = a.h + b.h, t = s - a.h;
  const float e = (a.h - (s - t)) + (b.h - t) + (a.l + b.l);
  const float h = s + e;
  return Two{h, e - (h - s)};
}
__device__ __forceinline__ Two two_shfl_up(Two a, int o) {
  return Two{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
}
__device__ __forceinline__ Two two_shfl(Two a, int lane) {
  return Two{__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}
// 2^(a - b)
__device__ __forceinline__ float two_exp2(Two a, Two b) { return ex2_approx((a.h - b.h) + (a.l - b.l)); }

template <int DK, bool F32>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const GatedDeltaArgs g, const __grid_constant__ CUtensorMap map_k,
                                                            const __grid_constant__ CUtensorMap map_q,
                                                            const __grid_constant__ CUtensorMap map_v, int vec_kq,
                                                            int vec_v) {
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
  const uint32_t v_full = next_bars(1), v_empty = next_bars(1);
  const uint32_t raw_full = next_bars(1), tp_full = next_bars(1), tp_empty = next_bars(1);
  const uint32_t d0_full = next_bars(2), d0_empty = next_bars(2);
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
    for (int s = 0; s < L::kKqStages; ++s) mbar_init(kq_full + 8 * s, kLoadThreads + 32), mbar_init(kq_empty + 8 * s, 1);
    mbar_init(v_full, vec_v ? 1 : kLoadThreads), mbar_init(v_empty, 8);
    mbar_init(raw_full, 1), mbar_init(tp_full, 4), mbar_init(tp_empty, 1);
    for (int s = 0; s < 2; ++s) mbar_init(d0_full + 8 * s, 1), mbar_init(d0_empty + 8 * s, 4);
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

  auto wait = [&](uint32_t bar, int phase) {
    if (!mbar_try_wait(bar, (uint32_t)(phase & 1))) wait_slow(bar, (uint32_t)(phase & 1), abort_flag);
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
    const int64_t s_at = (bh * g.dv + n) * g.dk + half * HK;
    const bool vec_s = g.dk % 4 == 0 && ((reinterpret_cast<uintptr_t>(g.state_in) | reinterpret_cast<uintptr_t>(g.state_out)) & 15) == 0;
    float s[HK];
#pragma unroll
    for (int j = 0; j < HK; j += 4) {
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (g.state_in && live) {
        const float* p = g.state_in + s_at + j;
        const int left = g.dk - half * HK - j;
        if (vec_s) {
          if (left > 0) x = *reinterpret_cast<const float4*>(p);
        } else {
          if (left > 0) x.x = p[0];
          if (left > 1) x.y = p[1];
          if (left > 2) x.z = p[2];
          if (left > 3) x.w = p[3];
        }
      }
      s[j] = x.x, s[j + 1] = x.y, s[j + 2] = x.z, s[j + 3] = x.w;
    }
    int s_exp = 0;  // S is held as 2^{s_exp} S
    // this lane's state to tensor memory, scaled, in two halves: of every 16
    // columns 8 of hi, 8 of lo
    auto put_state = [&]() {
      float mx = 0.0f;
#pragma unroll
      for (int j = 0; j < HK; ++j) mx = fmaxf(mx, fabsf(s[j]));
      if (mx > 3.4e38f) mx = 1.0f;  // not finite: the component is lost, any scale will do
      max_s[half * kM + lane_n] = mx;
      named_barrier(3 + quad, 64);
      s_exp = 13 - exponent_of(fmaxf(mx, max_s[(1 - half) * kM + lane_n]));
      s_exp = s_exp > 120 ? 120 : s_exp;
      const float2 c = make_float2(pow2(s_exp), pow2(s_exp));
#pragma unroll
      for (int j0 = 0; j0 < HK; j0 += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = __fmul2_rn(make_float2(s[j0 + 2 * j], s[j0 + 2 * j + 1]), c);
          split2(v.x, v.y, hi[j], lo[j]);
        }
        tmem_st8(t_lane + kColS + (uint32_t)(half * HK + j0), hi);
        tmem_st8(t_lane + kColS + (uint32_t)(half * HK + j0 + 8), lo);
      }
      tmem_wait_st();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_ready);
    };
    put_state();

    const int i0 = half * 32;  // this thread's tokens of a chunk
    const uint32_t y_step = (uint32_t)g.ld_y * (g.y_bf16 ? 2 : 4);  // bytes; a chunk's rows fit 32 bits
    char* y_at = reinterpret_cast<char*>(g.y) +
                 ((b * g.T + i0) * g.ld_y + (int64_t)h * g.dv + n) * (g.y_bf16 ? 2 : 4);
    for (int c = 0; c < n_chunks; ++c) {
      const Gates& gt = gates[c % kGateSlots];
      const int left = (int)(g.T - (int64_t)c * kC < kC ? g.T - (int64_t)c * kC : kC);
      // this lane's value of token i0 + i
      const In* v_tile = reinterpret_cast<const In*>(gbase + L::kOffV) + i0 * kM + lane_n;
      const In* v_global = reinterpret_cast<const In*>(g.v) + (b * g.T + (int64_t)c * kC + i0) * g.ld_v + (int64_t)h * g.dv + n;
      auto value = [&](int i) {
        if (!F32) return to_f32(v_tile[i * kM]);
        return live && i0 + i < left ? to_f32(v_global[i * g.ld_v]) : 0.0f;
      };
      int r_exp;  // R is held as 2^{r_exp} R
      {  // epilogue 1: R^T = V^T - fx D1; of every 16 columns 8 of hi, 8 of lo
        wait(kq_full + 8 * (c % L::kKqStages), c / L::kKqStages);  // the gates
        if (!F32) wait(v_full, c);
        const float cx = pow2(-s_exp);
        float2 r[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = make_float2(value(2 * j), value(2 * j + 1));
        wait(x_full, c);
        tcgen05_fence_after();
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
          uint32_t x[16];
          tmem_ld16(t_lane + kColX + (uint32_t)(i0 + i), x);
          tmem_wait(x);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 fx = *reinterpret_cast<const float4*>(&gt.fx[i0 + i + j]);
            const float2 f[2] = {make_float2(fx.x, fx.y), make_float2(fx.z, fx.w)};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float2& t = r[(i + j) / 2 + e];
              t = __ffma2_rn(__fmul2_rn(f[e], make_float2(-cx, -cx)),
                             make_float2(__uint_as_float(x[j + 2 * e]), __uint_as_float(x[j + 2 * e + 1])), t);
              mx = fmaxf(fmaxf(mx, fabsf(t.x)), fabsf(t.y));
            }
          }
        }
        if (mx > 3.4e38f) mx = 1.0f;
        max_v[half * kM + lane_n] = mx;
        named_barrier(3 + quad, 64);  // the other 32 tokens of the lane
        r_exp = 9 - exponent_of(fmaxf(mx, max_v[(1 - half) * kM + lane_n]));
        r_exp = r_exp > 120 ? 120 : r_exp;
        const float cr = pow2(r_exp);
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 t = __fmul2_rn(r[i / 2 + j], make_float2(cr, cr));
            split2(t.x, t.y, hi[j], lo[j]);
          }
          tmem_st8(t_lane + kColX + (uint32_t)(i0 + i), hi);
          tmem_st8(t_lane + kColX + (uint32_t)(i0 + i + 8), lo);
        }
        tmem_wait_st();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(r_ready);
          if (!F32) mbar_arrive(v_empty);
        }
      }
      {  // epilogue 2: U^T, already decayed to the chunk's end
        wait(u_full, c);
        tcgen05_fence_after();
#pragma unroll 1
        for (int i = i0; i < i0 + 32; i += 16) {
          uint32_t x[16], hi[8], lo[8];
          tmem_ld16(t_lane + kColU + (uint32_t)i, x);
          tmem_wait(x);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            split2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]), hi[j], lo[j]);
          tmem_st8(t_lane + kColU + (uint32_t)i, hi);
          tmem_st8(t_lane + kColU + (uint32_t)(i + 8), lo);
        }
        tmem_wait_st();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(u_ready);
      }
      {  // output, while D3 is in flight
        wait(o_full, c);
        tcgen05_fence_after();
        const float cq = pow2(-s_exp), cw = g.scale * pow2(-r_exp - gt.w_exp);
        const int rows = live ? left - i0 : 0;  // of this thread's 32 tokens
#pragma unroll 1
        for (int i = 0; i < 32; i += 8) {
          uint32_t xq[8], xo[8];
          tmem_ld8(t_lane + kColQ + (uint32_t)(i0 + i), xq);
          tmem_ld8(t_lane + kColO + (uint32_t)(i0 + i), xo);
          float2 o[4];
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 fq = *reinterpret_cast<const float4*>(&gt.fq[i0 + i + j]);
            o[j / 2] = __fmul2_rn(make_float2(fq.x, fq.y), make_float2(cq, cq));
            o[j / 2 + 1] = __fmul2_rn(make_float2(fq.z, fq.w), make_float2(cq, cq));
          }
          tmem_wait(xq);
          tmem_wait(xo);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = __ffma2_rn(make_float2(__uint_as_float(xo[2 * j]), __uint_as_float(xo[2 * j + 1])), make_float2(cw, cw),
                              __fmul2_rn(o[j], make_float2(__uint_as_float(xq[2 * j]), __uint_as_float(xq[2 * j + 1]))));
          uint32_t at = (uint32_t)i * y_step;
          if (g.y_bf16) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const __nv_bfloat162 w = __floats2bfloat162_rn(o[j / 2].x, o[j / 2].y);
              if (i + j < rows) *reinterpret_cast<__nv_bfloat16*>(y_at + at) = w.x;
              at += y_step;
              if (i + j + 1 < rows) *reinterpret_cast<__nv_bfloat16*>(y_at + at) = w.y;
              at += y_step;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (i + j < rows) *reinterpret_cast<float*>(y_at + at) = (j & 1) ? o[j / 2].y : o[j / 2].x;
              at += y_step;
            }
          }
        }
        y_at += (int64_t)kC * y_step;
      }
      {  // epilogue 3: S = e^G S + D3
        const float total = gt.total, cd = pow2(-r_exp - gt.t_exp);
        wait(s_full, c);
        tcgen05_fence_after();
#pragma unroll
        for (int j0 = 0; j0 < HK; j0 += 16) {
          uint32_t x[16];
          tmem_ld16(t_lane + kColS + (uint32_t)(half * HK + j0), x);
          tmem_wait(x);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float2 t = __ffma2_rn(
                make_float2(total, total), make_float2(s[j0 + j], s[j0 + j + 1]),
                __fmul2_rn(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), make_float2(cd, cd)));
            s[j0 + j] = t.x, s[j0 + j + 1] = t.y;
          }
        }
        if (c + 1 < n_chunks) put_state();
      }
    }
    if (g.state_out && live) {
#pragma unroll
      for (int j = 0; j < HK; j += 4) {
        float* p = g.state_out + s_at + j;
        const int left = g.dk - half * HK - j;
        if (vec_s) {
          if (left > 0) *reinterpret_cast<float4*>(p) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        } else {
          if (left > 0) p[0] = s[j];
          if (left > 1) p[1] = s[j + 1];
          if (left > 2) p[2] = s[j + 2];
          if (left > 3) p[3] = s[j + 3];
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ prepare ----
    const int quad = warp & 3;
    const int row = quad * 32 + lane;       // row of [K; Q]
    const bool is_t = quad < 2;             // warp-uniform
    const bool upper = quad & 1;            // tokens 32-63: the rows with columns past 31
    const int i = row & (kC - 1);           // token
    float* a_s = reinterpret_cast<float*>(gbase + L::kOffA);
    float* p_s = a_s + kC * kLdA;
    // of [T; W] this warp solves rows 16 rt .. of T and rows 16 rw .. of W: the
    // work of a row block grows with its index, the two together do not
    const int rt = quad, rw = 3 - quad;
    const int fr = lane / 4, fc = 2 * (lane % 4);  // accumulator fragment: rows fr, fr + 8, columns fc, fc + 1
    for (int c = 0; c < n_chunks; ++c) {
      Gates& gt = gates[c % kGateSlots];
      const uint32_t t_d0 = tmem + ((uint32_t)(quad * 32) << 16) + kColD0 + (uint32_t)(64 * (c & 1));
      wait(kq_full + 8 * (c % L::kKqStages), c / L::kKqStages);  // the gates
      wait(d0_full + 8 * (c & 1), c / 2);
      tcgen05_fence_after();
      named_barrier(1, 128);  // the previous chunk's A and P are read
      {
        // -A and P to shared memory, a row per thread
        float* dst = (is_t ? a_s : p_s) + i * kLdA;
        const uint32_t t_diag = t_d0 + (upper ? 32 : 0);
        uint32_t d[32];
        if (upper) {
          // the 32 columns before these rows' own: the decay factors at token 31
          const float since = gt.since[is_t ? 0 : 1][lane];
          tmem_ld32(t_d0, d);
          tmem_wait(d);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 past = *reinterpret_cast<const float4*>(&gt.past[j]);
            const float2 lo = __fmul2_rn(__fmul2_rn(make_float2(past.x, past.y), make_float2(since, since)),
                                         make_float2(__uint_as_float(d[j]), __uint_as_float(d[j + 1])));
            const float2 hi = __fmul2_rn(__fmul2_rn(make_float2(past.z, past.w), make_float2(since, since)),
                                         make_float2(__uint_as_float(d[j + 2]), __uint_as_float(d[j + 3])));
            *reinterpret_cast<float4*>(dst + j) = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
          dst += 32;
        }
        tmem_ld32(t_diag, d);
        const float rh = gt.row_hi[row], rl = gt.row_lo[row];
        const float scale_row = is_t ? -gt.beta[i] : 1.0f;
        const int last = is_t ? lane - 1 : lane;  // A is strictly lower, P lower
        const float* col_hi = gt.col_hi + (upper ? 32 : 0);
        const float* col_lo = gt.col_lo + (upper ? 32 : 0);
        tmem_wait(d);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 ch = *reinterpret_cast<const float4*>(col_hi + j), cl = *reinterpret_cast<const float4*>(col_lo + j);
          const float chs[4] = {ch.x, ch.y, ch.z, ch.w}, cls[4] = {cl.x, cl.y, cl.z, cl.w};
          float o[4];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 w = __fadd2_rn(__fadd2_rn(make_float2(rh, rh), make_float2(-chs[e], -chs[e + 1])),
                                        __fadd2_rn(make_float2(rl, rl), make_float2(-cls[e], -cls[e + 1])));
            const float2 v = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(d[j + e]), __uint_as_float(d[j + e + 1])),
                                                   make_float2(ex2_approx(w.x), ex2_approx(w.y))),
                                        make_float2(scale_row, scale_row));
            o[e] = j + e <= last ? v.x : 0.0f;
            o[e + 1] = j + e + 1 <= last ? v.y : 0.0f;
          }
          *reinterpret_cast<float4*>(dst + j) = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
      tcgen05_fence_before();
      named_barrier(1, 128);
      if (lane == 0) mbar_arrive(d0_empty + 8 * (c & 1));
      {
        // the inverse of diagonal block `quad` of I + A over the block itself, a
        // lane a row (16-31 repeat 0-15): X (I + A) = I, columns from the last
        float* blk = a_s + 16 * quad * (kLdA + 1);
        const int r = lane & 15;
        float2 x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = make_float2(2 * q == r ? 1.0f : 0.0f, 2 * q + 1 == r ? 1.0f : 0.0f);
#pragma unroll
        for (int k = 15; k >= 1; --k) {
          const float xk = (k & 1) ? x[k / 2].y : x[k / 2].x;
#pragma unroll
          for (int q = 0; q < (k + 3) / 4; ++q) {
            const float4 a = *reinterpret_cast<const float4*>(blk + k * kLdA + 4 * q);
            x[2 * q] = __ffma2_rn(make_float2(xk, xk), make_float2(a.x, a.y), x[2 * q]);
            if (4 * q + 2 < k) x[2 * q + 1] = __ffma2_rn(make_float2(xk, xk), make_float2(a.z, a.w), x[2 * q + 1]);
          }
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(blk + r * kLdA + 4 * q) =
                make_float4(x[2 * q].x, x[2 * q].y, x[2 * q + 1].x, x[2 * q + 1].y);
        }
      }
      named_barrier(1, 128);
      // X (I + A) = [I; P] by blocks of 16 columns, the last first: X_k = B_k D_k,
      // then B_j += X_k (-A_kj) for the blocks before it
      float t[8][4], w[8][4];
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) t[nt][e] = 0.0f, w[nt][e] = 0.0f;
        if (nt / 2 <= rw) {
          const float2 lo = *reinterpret_cast<const float2*>(p_s + (16 * rw + fr) * kLdA + 8 * nt + fc);
          const float2 hi = *reinterpret_cast<const float2*>(p_s + (16 * rw + fr + 8) * kLdA + 8 * nt + fc);
          w[nt][0] = lo.x, w[nt][1] = lo.y, w[nt][2] = hi.x, w[nt][3] = hi.y;
        }
        if (nt / 2 == rt) {  // the identity times D
          const float2 lo = *reinterpret_cast<const float2*>(a_s + (16 * rt + fr) * kLdA + 8 * nt + fc);
          const float2 hi = *reinterpret_cast<const float2*>(a_s + (16 * rt + fr + 8) * kLdA + 8 * nt + fc);
          t[nt][0] = lo.x, t[nt][1] = lo.y, t[nt][2] = hi.x, t[nt][3] = hi.y;
        }
      }
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        const bool do_t = k <= rt, do_w = k <= rw;  // warp-uniform
        if (!do_t && !do_w) continue;
        uint32_t th[2][4], tl[2][4], wh[2][4], wl[2][4];
#pragma unroll
        for (int j = k; j >= 0; --j) {  // j == k: times the inverse of the diagonal block
          Tf32x2 bm[2][2][2];  // [k8][n8][row pair]
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int nn = 0; nn < 2; ++nn)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                bm[kk][nn][e].set(a_s[(16 * k + 8 * kk + fc + e) * kLdA + 16 * j + 8 * nn + fr]);
          auto product = [&](float (&x)[8][4], uint32_t (&xh)[2][4], uint32_t (&xl)[2][4], bool solved) {
            float acc[2][4];
#pragma unroll
            for (int nn = 0; nn < 2; ++nn)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nn][e] = j < k ? x[2 * j + nn][e] : 0.0f;
            if (j == k) {
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) tf32_operand(xh[kk], xl[kk], x[2 * k + kk]);
            }
            if (j < k || !solved) {
#pragma unroll
              for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int nn = 0; nn < 2; ++nn) {
                  mma_tf32(acc[nn], xl[kk], bm[kk][nn][0].hi, bm[kk][nn][1].hi);
                  mma_tf32(acc[nn], xh[kk], bm[kk][nn][0].lo, bm[kk][nn][1].lo);
                  mma_tf32(acc[nn], xh[kk], bm[kk][nn][0].hi, bm[kk][nn][1].hi);
                }
#pragma unroll
              for (int nn = 0; nn < 2; ++nn)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[2 * j + nn][e] = acc[nn][e];
              if (j == k) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) tf32_operand(xh[kk], xl[kk], x[2 * k + kk]);
              }
            }
          };
          if (do_t) product(t, th, tl, k == rt);
          if (do_w) product(w, wh, wl, false);
        }
      }
      // T's columns times beta, its rows decayed to the chunk's end; one scale for
      // T and one for W, from the largest row sum of each
      {
        const float d0 = gt.fd[16 * rt + fr], d1 = gt.fd[16 * rt + fr + 8];
        float st0 = 0.0f, st1 = 0.0f, sw0 = 0.0f, sw1 = 0.0f;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          const float2 be = *reinterpret_cast<const float2*>(&gt.beta[8 * nt + fc]);
          t[nt][0] *= be.x * d0, t[nt][1] *= be.y * d0, t[nt][2] *= be.x * d1, t[nt][3] *= be.y * d1;
          w[nt][0] *= be.x, w[nt][1] *= be.y, w[nt][2] *= be.x, w[nt][3] *= be.y;
          st0 += fabsf(t[nt][0]) + fabsf(t[nt][1]), st1 += fabsf(t[nt][2]) + fabsf(t[nt][3]);
          sw0 += fabsf(w[nt][0]) + fabsf(w[nt][1]), sw1 += fabsf(w[nt][2]) + fabsf(w[nt][3]);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          st0 += __shfl_xor_sync(0xffffffffu, st0, o), st1 += __shfl_xor_sync(0xffffffffu, st1, o);
          sw0 += __shfl_xor_sync(0xffffffffu, sw0, o), sw1 += __shfl_xor_sync(0xffffffffu, sw1, o);
        }
        const unsigned mt = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(st0, st1)));
        const unsigned mw = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(sw0, sw1)));
        if (lane == 0) gt.sum_t[quad] = __uint_as_float(mt), gt.sum_w[quad] = __uint_as_float(mw);
      }
      named_barrier(1, 128);
      {
        const float4 a = *reinterpret_cast<const float4*>(gt.sum_t), d = *reinterpret_cast<const float4*>(gt.sum_w);
        int te = 3 - exponent_of(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)));
        int we = 3 - exponent_of(fmaxf(fmaxf(d.x, d.y), fmaxf(d.z, d.w)));
        te = te > 100 ? 100 : te, we = we > 100 ? 100 : we;
        if (c > 0) wait(tp_empty, c - 1);
        if (quad == 0 && lane == 0) gt.t_exp = te, gt.w_exp = we;
        const float ct = pow2(te), cw = pow2(we);
        // lane l addresses row l % 8 of matrix l / 8: rows 0-7 and 8-15 of one
        // granule of 8 columns, then of the next; granule q of row r at q ^ (r % 8)
        const uint32_t at = base + L::kOffTp + (uint32_t)((((lane >> 3) & 1) * 8 + (lane & 7)) * 128 +
                                                          ((((lane >> 4) & 1) ^ (lane & 7)) << 4));
        const uint32_t at_t = at + rt * 2048, at_w = at + 8192 + rw * 2048;
#pragma unroll
        for (int nt = 0; nt < 8; nt += 2) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = __fmul2_rn(make_float2(t[nt + e / 2][2 * (e & 1)], t[nt + e / 2][2 * (e & 1) + 1]),
                                        make_float2(ct, ct));
            split2(v.x, v.y, hi[e], lo[e]);
          }
          stmatrix4(at_t ^ (uint32_t)(nt << 4), hi);
          stmatrix4((at_t ^ (uint32_t)(nt << 4)) + 16384, lo);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = __fmul2_rn(make_float2(w[nt + e / 2][2 * (e & 1)], w[nt + e / 2][2 * (e & 1) + 1]),
                                        make_float2(cw, cw));
            split2(v.x, v.y, hi[e], lo[e]);
          }
          stmatrix4(at_w ^ (uint32_t)(nt << 4), hi);
          stmatrix4((at_w ^ (uint32_t)(nt << 4)) + 16384, lo);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(tp_full);
    }
  } else if (warp < kGateWarp) {
    // --------------------------------------------------------------- load ----
    const int lw = warp - 12, lt = threadIdx.x - 12 * 32;
    constexpr int kLanes = DK / 8;           // lanes per row
    constexpr int kRowsPer = 32 / kLanes;    // rows per warp and pass
    constexpr int kStep = kLoadWarps * kRowsPer;  // rows per pass
    const int sub = lane / kLanes, col = (lane % kLanes) * 8;
    const int valid = g.dk - col;            // of this lane's eight components
    const In* k_base = reinterpret_cast<const In*>(g.k) + b * g.T * g.ld_k + (int64_t)hk * g.dk;
    const In* q_base = reinterpret_cast<const In*>(g.q) + b * g.T * g.ld_q + (int64_t)hk * g.dk;
    const In* v_base = reinterpret_cast<const In*>(g.v) + b * g.T * g.ld_v + (int64_t)h * g.dv + tile * kM;
    const bool staged = !F32 && vec_kq;      // K and Q through tensor copies
    auto tokens = [&](int c) { return (int)(g.T - (int64_t)c * kC < kC ? g.T - (int64_t)c * kC : kC); };
    // K and Q rows of chunk c (tokens past the end read as zero)
    auto copy_kq = [&](int c) {
      if (lane == 0) {
        mbar_arrive_expect_tx(raw_full, 2 * kC * DK * 2);
        tma_load_3d(base + L::kOffRaw, &map_k, hk * g.dk, c * kC, (int)b, raw_full);
        tma_load_3d(base + L::kOffRaw + kC * DK * 2, &map_q, hk * g.dk, c * kC, (int)b, raw_full);
      }
    };
    if (staged && lw == 0) copy_kq(0);
    for (int c = 0; c < n_chunks; ++c) {
      const int ks = c % L::kKqStages;
      const int left = tokens(c);
      int* exps = reinterpret_cast<int*>(gbase + L::kOffExp) + (c & 1) * 2 * kC;
      if (staged) wait(raw_full, c);
      if (c >= L::kKqStages) wait(kq_empty + 8 * ks, c / L::kKqStages + 1);
      // K (rows 0-63) and Q (64-127), each row scaled to [2^13, 2^14)
      // kBatch rows' loads and reductions are in flight together
      constexpr int kBatch = F32 ? 4 : 8;
      static_assert(2 * kC % (kBatch * kStep) == 0, "whole batches");
#pragma unroll 1
      for (int r0 = lw * kRowsPer + sub; r0 < 2 * kC; r0 += kBatch * kStep) {
        float f[kBatch][8];
        int ex[kBatch];  // floor(log2) of the row's largest value
        if constexpr (!F32) {
          uint4 x[kBatch];
          if (staged) {
#pragma unroll
            for (int p = 0; p < kBatch; ++p) {
              x[p] = *reinterpret_cast<const uint4*>(gbase + L::kOffRaw + (r0 + p * kStep) * DK * 2 + col * 2);
              if (valid <= 0) x[p] = make_uint4(0, 0, 0, 0);  // columns past dk are another head's
            }
          } else {
#pragma unroll 1
            for (int p = 0; p < kBatch; ++p) {
              const int r = r0 + p * kStep, i = r & (kC - 1);
              const int64_t t = (int64_t)c * kC + i;
              const uint16_t* src = reinterpret_cast<const uint16_t*>(r < kC ? k_base + t * g.ld_k : q_base + t * g.ld_q) + col;
              uint32_t e[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) e[j] = i < left && j < valid ? src[j] : 0;
              // by way of the rows' place in the staging buffer (this thread's own granules)
              *reinterpret_cast<uint4*>(gbase + L::kOffRaw + r * DK * 2 + col * 2) =
                  make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
            }
#pragma unroll
            for (int p = 0; p < kBatch; ++p)
              x[p] = *reinterpret_cast<const uint4*>(gbase + L::kOffRaw + (r0 + p * kStep) * DK * 2 + col * 2);
          }
          // bit patterns of |x| order as the values do; two rows share a word
#pragma unroll
          for (int p = 0; p < kBatch; p += 2) {
            uint32_t m[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
              m[u] = __vmaxu2(__vmaxu2(x[p + u].x & 0x7fff7fffu, x[p + u].y & 0x7fff7fffu),
                              __vmaxu2(x[p + u].z & 0x7fff7fffu, x[p + u].w & 0x7fff7fffu));
            uint32_t both = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, o));
            ex[p] = (int)((both >> 7) & 255) - 127;
            ex[p + 1] = (int)(both >> 23) - 127;
          }
#pragma unroll
          for (int p = 0; p < kBatch; ++p) unpack8(f[p], x[p]);
        } else {
#pragma unroll
          for (int p = 0; p < kBatch; ++p) {
            const int r = r0 + p * kStep, i = r & (kC - 1);
            const bool in = i < left;
            const int64_t t = in ? (int64_t)c * kC + i : 0;
            const float* src = reinterpret_cast<const float*>(r < kC ? k_base + t * g.ld_k : q_base + t * g.ld_q) + col;
            if (vec_kq) {
              float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f), hi = lo;
              if (in && valid > 0) lo = *reinterpret_cast<const float4*>(src), hi = *reinterpret_cast<const float4*>(src + 4);
              f[p][0] = lo.x, f[p][1] = lo.y, f[p][2] = lo.z, f[p][3] = lo.w;
              f[p][4] = hi.x, f[p][5] = hi.y, f[p][6] = hi.z, f[p][7] = hi.w;
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) f[p][j] = in && j < valid ? src[j] : 0.0f;
            }
          }
          float mx[kBatch];
#pragma unroll
          for (int p = 0; p < kBatch; ++p) {
            mx[p] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) mx[p] = fmaxf(mx[p], fabsf(f[p][j]));
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
            for (int p = 0; p < kBatch; ++p) mx[p] = fmaxf(mx[p], __shfl_xor_sync(0xffffffffu, mx[p], o));
#pragma unroll
          for (int p = 0; p < kBatch; ++p) ex[p] = exponent_of(mx[p]);
        }
#pragma unroll
        for (int p = 0; p < kBatch; ++p) {
          const int r = r0 + p * kStep;
          const int e = ex[p] < -107 ? 120 : 13 - ex[p];
          const float cs = pow2(e);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = __fmul2_rn(make_float2(f[p][2 * j], f[p][2 * j + 1]), make_float2(cs, cs));
            if (F32) {
              split2(v.x, v.y, hi[j], lo[j]);
            } else {
              const __half2 t = __floats2half2_rn(v.x, v.y);
              hi[j] = *reinterpret_cast<const uint32_t*>(&t);
            }
          }
          if (col == 0) exps[r] = e;
          const uint32_t at =
              base + ks * L::kKq + (uint32_t)((col / 64) * 16384 + r * 128 + ((((col & 63) / 8) ^ (r & 7)) << 4));
          st_shared16(at, hi[0], hi[1], hi[2], hi[3]);
          if (F32) st_shared16(at + L::kKqTerm, lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      named_barrier(2, kLoadThreads + 32);  // every row's exponent is there, the raw rows are read
      if (staged && lw == 0 && c + 1 < n_chunks) copy_kq(c + 1);
      mbar_arrive(kq_full + 8 * ks);
      // V (bf16); rows past the sequence's end are zero, columns past the head's
      // are lanes that nothing reads
      if (!F32 && (!vec_v || lw == 0)) {
        if (c > 0) wait(v_empty, c - 1);
        if (vec_v) {
          if (lane == 0) {
            mbar_arrive_expect_tx(v_full, kC * kM * 2);
            tma_load_3d(base + L::kOffV, &map_v, h * g.dv + tile * kM, c * kC, (int)b, v_full);
          }
        } else {
          const int cols = g.dv - tile * kM < kM ? g.dv - tile * kM : kM;
          In* v_dst = reinterpret_cast<In*>(gbase + L::kOffV);
#pragma unroll 4
          for (int e = lt; e < kC * kM; e += kLoadThreads) {
            const int r = e / kM, q = e % kM;
            v_dst[e] = r < left && q < cols ? v_base[((int64_t)c * kC + r) * g.ld_v + q] : from_f32<In>(0.0f);
          }
          mbar_arrive(v_full);
        }
      }
    }
  } else if (warp == kGateWarp) {
    // -------------------------------------------------------------- gates ----
    // tokens lane and lane + 32 of a chunk: base-2 logarithms of alpha, summed and
    // kept as two floats each, so that differences between far-decayed tokens keep
    // 32-bit accuracy.  alpha below e^-200 is 0 in f32 all the same.
    const float neg_A = -expf(g.A_log[h]);
    const float dt_bias = g.dt_bias ? g.dt_bias[h] : 0.0f;
    const In* a_base = reinterpret_cast<const In*>(g.a) + b * g.T * g.ld_a + h;
    const In* b_base = reinterpret_cast<const In*>(g.b) + b * g.T * g.ld_b + h;
    float a_next[2], b_next[2];
    auto fetch = [&](int c) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t t = (int64_t)c * kC + lane + 32 * u;
        a_next[u] = t < g.T ? to_f32(a_base[t * g.ld_a]) : -INFINITY;  // past the end: alpha 1, beta 0
        b_next[u] = t < g.T ? to_f32(b_base[t * g.ld_b]) : -INFINITY;
      }
    };
    fetch(0);
    for (int c = 0; c < n_chunks; ++c) {
      Two G[2];
      float be[2];
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {
        const float a = u ? a_next[1] : a_next[0], bb = u ? b_next[1] : b_next[0];
        const float la = gdr_log_alpha(a, dt_bias, neg_A);
        Two x = two_log2(la < -200.0f ? -200.0f : la);
        const float y = gdr_beta(bb);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const Two t = two_shfl_up(x, o), sum = two_add(x, t);
          if (lane >= o) x = sum;
        }
        if (u)
          G[1] = x, be[1] = y;
        else
          G[0] = x, be[0] = y;
      }
      if (c + 1 < n_chunks) fetch(c + 1);
      const Two mid = two_shfl(G[0], 31);
      G[1] = two_add(G[1], mid);
      const Two last = two_shfl(G[1], 31);
      const int* exps = reinterpret_cast<const int*>(gbase + L::kOffExp) + (c & 1) * 2 * kC;
      Gates& gt = gates[c % kGateSlots];
      named_barrier(2, kLoadThreads + 32);  // the rows' exponents are there, this slot's last readers gone
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        const float ek = (float)exps[i], eq = (float)exps[kC + i];
        const float ik = pow2(-exps[i]), iq = pow2(-exps[kC + i]);
        const Two cj = two_add(G[u], Two{ek, 0.0f}), rk = two_add(G[u], Two{-ek, 0.0f}), rq = two_add(G[u], Two{-eq, 0.0f});
        const float eg = ex2_approx(G[u].h + G[u].l);
        gt.col_hi[i] = cj.h, gt.col_lo[i] = cj.l;
        gt.row_hi[i] = rk.h, gt.row_lo[i] = rk.l;
        gt.row_hi[kC + i] = rq.h, gt.row_lo[kC + i] = rq.l;
        gt.beta[i] = be[u];
        gt.fx[i] = eg * ik;
        gt.fd[i] = two_exp2(last, G[u]) * ik;
        gt.fq[i] = g.scale * eg * iq;
        if (u == 0) {
          gt.past[lane] = two_exp2(mid, G[0]) * ik;
        } else {
          const float e = two_exp2(G[1], mid);
          gt.since[0][lane] = -be[1] * e * ik;
          gt.since[1][lane] = e * iq;
        }
      }
      if (lane == 0) gt.total = ex2_approx(last.h + last.l);
      mbar_arrive(kq_full + 8 * (c % L::kKqStages));
    }
  } else {
    // --------------------------------------------------------------- MMAs ----
    if (lane == 0) {
      constexpr uint32_t id64 = idesc_f16(64, false), id3 = idesc_f16(DK, true);
      // [K; Q] K^T of chunk c, for the prepare warps
      auto issue_d0 = [&](int c) {
        const uint32_t kq = base + (c % L::kKqStages) * L::kKq;
        wait(kq_full + 8 * (c % L::kKqStages), c / L::kKqStages);
        if (c > 1) wait(d0_empty + 8 * (c & 1), c / 2 - 1);
        tcgen05_fence_after();
        uint32_t acc = 0;
#pragma unroll 1
        for (int term = 0; term < (F32 ? 3 : 1); ++term) {
          const uint32_t ka = kq + (term == 1 ? L::kKqTerm : 0), kb = kq + (term == 2 ? L::kKqTerm : 0);
#pragma unroll
          for (int k = 0; k < DK / 16; ++k) {
            mma_ss(tmem + kColD0 + 64 * (c & 1), smem_desc(ka + (k / 4) * 16384) + 2 * (k % 4),
                   smem_desc(kb + (k / 4) * 16384) + 2 * (k % 4), id64, acc);
            acc = 1;
          }
        }
        mma_commit(d0_full + 8 * (c & 1));
      };
      issue_d0(0);
      for (int c = 0; c < n_chunks; ++c) {
        const int ks = c % L::kKqStages;
        const uint32_t kq = base + ks * L::kKq, tp = base + L::kOffTp;
        wait(s_ready, c);
        tcgen05_fence_after();
        // D1: S_hi K_hi + S_lo K_hi (+ S_hi K_lo); keys first, the queries'
        // half runs under epilogue 1.  A's halves: 8 columns hi, 8 lo of every 16
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          uint32_t acc = 0;
#pragma unroll 1
          for (int term = 0; term < (F32 ? 3 : 2); ++term) {
            const uint32_t ad = tmem + kColS + (term == 1 ? 8 : 0);
            const uint32_t bd = kq + (term == 2 ? L::kKqTerm : 0) + part * 8192;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
              mma_ts(tmem + (part ? kColQ : kColX), ad + 16 * k, smem_desc(bd + (k / 4) * 16384) + 2 * (k % 4), id64, acc);
              acc = 1;
            }
          }
          if (part == 0) mma_commit(x_full);
        }
        // one chunk ahead; two accumulators, so the prepare warps need not be
        // done with this chunk's
        if (c + 1 < n_chunks) issue_d0(c + 1);
        wait(tp_full, c);
        wait(r_ready, c);
        tcgen05_fence_after();
        // D2: R_hi T_hi + R_hi T_lo + R_lo T_hi; T's half first, W's under epilogue 2
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          uint32_t acc = 0;
#pragma unroll 1
          for (int term = 0; term < 3; ++term) {
            const uint32_t ad = tmem + kColX + (term == 2 ? 8 : 0);
            const uint64_t bd = smem_desc(tp + (term == 1 ? 16384 : 0) + part * 8192);
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {
              mma_ts(tmem + (part ? kColO : kColU), ad + 16 * k, bd + 2 * k, id64, acc);
              acc = 1;
            }
          }
          mma_commit(part ? o_full : u_full);
        }
        mma_commit(tp_empty);
        wait(u_ready, c);
        tcgen05_fence_after();
        // D3: U_hi K_hi + U_lo K_hi (+ U_hi K_lo); K's rows are the contraction
        uint32_t acc = 0;
#pragma unroll 1
        for (int term = 0; term < (F32 ? 3 : 2); ++term) {
          const uint32_t ad = tmem + kColU + (term == 1 ? 8 : 0);
          const uint64_t bd = smem_desc(kq + (term == 2 ? L::kKqTerm : 0), 16384);
#pragma unroll
          for (int k = 0; k < kC / 16; ++k) {
            mma_ts(tmem + kColS, ad + 16 * k, bd + 128 * k, id3, acc);
            acc = 1;
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

// cuTensorMapEncodeTiled from the driver, looked up once
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !p) {
      cudaGetLastError();
      return nullptr;
    }
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// [B][T][cols] bf16, rows ld apart: boxes of 64 tokens of one sequence x `box`
// columns, starting at any multiple of 8 columns; outside it reads as zero.
// False if the layout has no such map (then the element-wise path loads it).
bool make_map(CUtensorMap* map, const void* p, int64_t B, int64_t T, int64_t cols, int64_t ld, int d, int box) {
  if (reinterpret_cast<uintptr_t>(p) % 16 || ld % 8 || d % 8 || T * ld * 2 >= (int64_t(1) << 40) || T > INT32_MAX - kC ||
      cols > INT32_MAX - box)
    return false;
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), (cuuint64_t)(T * ld * 2)};
  const cuuint32_t boxes[3] = {(cuuint32_t)box, (cuuint32_t)kC, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  CUtensorMap mk = {}, mq = {}, mv = {};
  int vec_kq, vec_v = 0;
  if (F32) {
    auto rows16 = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0; };
    vec_kq = rows16(a.k, a.ld_k) && rows16(a.q, a.ld_q) && a.dk % 8 == 0;
  } else {
    const int64_t kc = (int64_t)a.Hk * a.dk, vc = (int64_t)a.Hv * a.dv;
    vec_kq = make_map(&mk, a.k, a.B, a.T, kc, a.ld_k, a.dk, DK) && make_map(&mq, a.q, a.B, a.T, kc, a.ld_q, a.dk, DK);
    vec_v = make_map(&mv, a.v, a.B, a.T, vc, a.ld_v, a.dv, kM);
  }
  const int64_t ctas = a.B * a.Hv * ((a.dv + kM - 1) / kM);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  kern<<<(unsigned)ctas, kThreads, smem, stream>>>(a, mk, mq, mv, vec_kq, vec_v);
  return cudaGetLastError();
}

}  // namespace

// The chunks' output offsets inside a chunk are 32 bits.
bool gated_delta_takes_chunks(const GatedDeltaArgs& a) {
  return a.dk <= 128 && a.T > 16 && a.ld_y < (int64_t(1) << 23);
}

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
