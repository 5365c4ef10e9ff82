// gemm_w4.cu - projections with 4-bit weights and group scales, many rows, on the
// tensor cores (tcgen05):
//
//   C[m][n] = sum_g s[n][g] sum_{k in g} (q[n][k] - z[n][g]) a[m][k]  (+ R[m][n])
//
// A tile is 128 weight rows (the product's M: tensor memory's lanes) x BT
// activation rows (its N: columns).  The differences q - z are exact in bf16, so
// the tensor cores' sums over one group are those of the weights as they are; the
// scale of a group and weight row, one number per lane, meets the group's sum in
// f32 outside of tensor memory.  (Scales folded into bf16 weights would round
// every weight to 8 bits, and save only the epilogue's reads.)
//
// Roles of a CTA (persistent, one per SM):
//  * warp 0 brings activation tiles, BT x 64 bf16 with the 128-byte swizzle (TMA);
//  * warp 2 brings weights as they are stored, 128 rows x 64 bytes (128 k) a copy;
//  * a warpgroup (two for narrow tiles), a thread per weight row, makes bf16 of the
//    nibbles: two operations a pair (nibbles i and i + 4 of a word in the halves of
//    a register, 0x4300 above them: 128 + q; a packed subtraction of 128 + z), a
//    byte permutation that puts neighbours side by side, 16-byte stores into the
//    product's swizzled operand;
//  * warp 1 issues the products, one group of k into one of two accumulators;
//  * two warpgroups take the other accumulator meanwhile, each half of the columns:
//    total += scale * group's sum, BT / 2 totals a thread in registers, and store
//    the totals at the end of a tile (a warp stores 32 neighbours of a row of C).
// Few tiles: K is split over a cluster whose CTAs add their totals through
// distributed shared memory in rank order.
//
// Every wait is bounded (about a second); one that runs out sets
// MAMBA_FAULT_GEMM_WAIT and an abort flag that ends every role's loop, and the CTA
// still waits for its copies and products in flight and frees its tensor memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/mamba_ssm.h"
#include "async_copy.cuh"
#include "device_math.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace mamba {
namespace {

namespace cg = cooperative_groups;

constexpr int kBN = 128;    // weight rows per tile
constexpr int kBK = 64;     // k per operand stage: one 128-byte swizzle row
constexpr int kChunk = 128; // k per copy of weights
constexpr int kEpiWarps = 8;
constexpr int kSmemLimit = 232448;
constexpr long long kWaitLimit = 1ll << 31;  // SM cycles (about a second)

__device__ int g_gemm_w4_faults = 0;

template <int BT>
struct Cfg {
  static constexpr int kDqGroups = BT > 128 ? 1 : 2;  // warpgroups that make bf16 of nibbles
  static constexpr int kThreads = 128 * (1 + kDqGroups + 2);
  static constexpr int kEpiWarp = 4 * (1 + kDqGroups);
  // registers per thread of the roles; their sum over the warpgroups is within what
  // the CTA is launched with (128 x 4 and 96 x 5)
  static constexpr int kRegsLoad = 40;
  static constexpr int kRegsDq = kDqGroups == 1 ? 96 : 88;
  static constexpr int kRegsEpi = kDqGroups == 1 ? 184 : 128;
  static constexpr int kRegs = kRegsLoad + kDqGroups * kRegsDq + 2 * kRegsEpi;
  static_assert(kRegs <= (65536 / kThreads / 8 * 8) * (kThreads / 128), "more registers than a CTA has");
  static constexpr int kStageB = BT * kBK * 2;
  static constexpr int kStageA = kBN * kBK * 2;
  static constexpr int kStageQ = kBN * kChunk / 2;
  static constexpr int kSB = BT == 256 ? 4 : (BT == 128 ? 6 : 8);
  static constexpr int kSA = BT == 256 ? 3 : 4;
  static constexpr int kOffA = kSB * kStageB;
  static constexpr int kOffQ = kOffA + kSA * kStageA;
  static constexpr int kSQ0 = (kSmemLimit - 1024 - 512 - kOffQ) / kStageQ;
  static constexpr int kSQ = kSQ0 > 8 ? 8 : kSQ0;
  static constexpr int kOffBar = kOffQ + kSQ * kStageQ;
  static constexpr int kBars = 2 * (kSB + kSA + kSQ) + 5;
  static constexpr int kBytes = kOffBar + 8 * kBars + 16;
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base
  static constexpr int kTmemCols = 2 * BT;
  static constexpr int kPartPitch = kBN + 4;
  static_assert(kAlloc <= kSmemLimit && kSQ >= 2, "shared memory");
};

template <int BT>
__host__ __device__ constexpr uint32_t instr_desc() {
  // kind::f16, f32 accumulator, bf16 operands, both K-major, N = BT, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BT >> 3) << 17) | ((uint32_t)(kBN >> 4) << 24);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_bf16(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float4 dsmem_ld4(uint32_t local, int rank) {
  uint32_t addr;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// the 8 nibbles of w, less zc - 128, as 8 bf16 in their order
__device__ __forceinline__ uint4 unpack8(uint32_t w, __nv_bfloat162 zc) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), zc);
    p[i] = *reinterpret_cast<const uint32_t*>(&d);  // k = i and i + 4
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                    __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z) {
  const uint32_t v = (0x4300u | z) * 0x00010001u;
  return *reinterpret_cast<const __nv_bfloat162*>(&v);
}

__device__ __forceinline__ void fail_w4(volatile int* abort_flag) {
  atomicOr(&g_gemm_w4_faults, MAMBA_FAULT_GEMM_WAIT);
  *abort_flag = 1;
}

template <int BT, int GROUP, bool SPLIT>
__global__ void __launch_bounds__(Cfg<BT>::kThreads, 1)
    gemm_w4_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_q, void* c,
                   int64_t ld_c, int c_bf16, const void* __restrict__ scales, int64_t ld_s, int s_bf16,
                   const uint8_t* __restrict__ zeros, int64_t ld_z, const float* r, int64_t ld_r, int M, int N, int K,
                   int splits) {
  using L = Cfg<BT>;
  constexpr int SA = L::kSA, SB = L::kSB, SQ = L::kSQ;
  constexpr int kG = kChunk / GROUP;          // groups per chunk
  constexpr int kStepsPerGroup = GROUP / 16;  // products per group
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kOffBar;
  auto b_full = [&](int s) { return bars + 8 * s; };
  auto b_empty = [&](int s) { return bars + 8 * (SB + s); };
  auto a_full = [&](int s) { return bars + 8 * (2 * SB + s); };
  auto a_empty = [&](int s) { return bars + 8 * (2 * SB + SA + s); };
  auto q_full = [&](int s) { return bars + 8 * (2 * (SB + SA) + s); };
  auto q_empty = [&](int s) { return bars + 8 * (2 * (SB + SA) + SQ + s); };
  auto acc_full = [&](int a) { return bars + 8 * (2 * (SB + SA + SQ) + a); };
  auto acc_empty = [&](int a) { return bars + 8 * (2 * (SB + SA + SQ) + 2 + a); };
  const uint32_t drain = bars + 8 * (2 * (SB + SA + SQ) + 4);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(gbase + L::kOffBar + 8 * L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n_tiles = (N + kBN - 1) / kBN, m_tiles = (M + BT - 1) / BT;
  const int tiles = n_tiles * m_tiles;
  const int chunks = (K + kChunk - 1) / kChunk;
  int rank = 0, t_first = blockIdx.x, t_step = gridDim.x, cb = 0, ce = chunks;
  if constexpr (SPLIT) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    t_first = blockIdx.x / splits;
    t_step = gridDim.x / splits;
    cb = rank * chunks / splits;
    ce = (rank + 1) * chunks / splits;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < SB; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), 1);
    }
    for (int s = 0; s < SA; ++s) {
      mbar_init(a_full(s), 4);
      mbar_init(a_empty(s), 1);
    }
    for (int s = 0; s < SQ; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 4 * L::kDqGroups);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full(a), 1);
      mbar_init(acc_empty(a), kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_ptr)),
                 "r"(L::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = *tmem_ptr;
  // one CTA per SM: the next kernel may start its set-up
  grid_dependents_launch();
  grid_dependency_wait();

  if (warp < 4) {
    regs_dec<L::kRegsLoad>();
    if (warp == 0 && lane == 0) {
      // activations
      int g = 0;
      for (int t = t_first; t < tiles && !*abort_flag; t += t_step) {
        const int m0 = t / n_tiles * BT;
        for (int ks = 2 * cb; ks < 2 * ce; ++ks, ++g) {
          const int s = g % SB;
          if (g >= SB && !mbar_wait(b_empty(s), (g / SB + 1) & 1, kWaitLimit)) {
            fail_w4(abort_flag);
            break;
          }
          mbar_arrive_expect_tx(b_full(s), L::kStageB);
          tma_load_2d(base + s * L::kStageB, &map_a, ks * kBK, m0, b_full(s));
        }
      }
      for (int i = g > SB ? g - SB : 0; i < g; ++i)
        if (!mbar_wait(b_full(i % SB), (i / SB) & 1, kWaitLimit)) fail_w4(abort_flag);
    } else if (warp == 2 && lane == 0) {
      // weights
      int g = 0;
      for (int t = t_first; t < tiles && !*abort_flag; t += t_step) {
        const int n0 = t % n_tiles * kBN;
        for (int ch = cb; ch < ce; ++ch, ++g) {
          const int s = g % SQ;
          if (g >= SQ && !mbar_wait(q_empty(s), (g / SQ + 1) & 1, kWaitLimit)) {
            fail_w4(abort_flag);
            break;
          }
          mbar_arrive_expect_tx(q_full(s), L::kStageQ);
          tma_load_2d(base + L::kOffQ + s * L::kStageQ, &map_q, ch * (kChunk / 2), n0, q_full(s));
        }
      }
      for (int i = g > SQ ? g - SQ : 0; i < g; ++i)
        if (!mbar_wait(q_full(i % SQ), (i / SQ) & 1, kWaitLimit)) fail_w4(abort_flag);
    } else if (warp == 1 && lane == 0) {
      // products
      constexpr uint32_t idesc = instr_desc<BT>();
      int g = 0, acc = 0;
      bool ok = true;
      for (int t = t_first; t < tiles && ok && !*abort_flag; t += t_step) {
        for (int ch = cb; ch < ce && ok; ++ch) {
#pragma unroll
          for (int half = 0; half < 2; ++half, ++g) {
            if (!ok) break;
            const int sa = g % SA, sb = g % SB;
            if (!mbar_wait(a_full(sa), (g / SA) & 1, kWaitLimit) || !mbar_wait(b_full(sb), (g / SB) & 1, kWaitLimit)) {
              ok = false;
              break;
            }
            tcgen05_fence_after();
            const uint64_t da = smem_desc(base + L::kOffA + sa * L::kStageA), db = smem_desc(base + sb * L::kStageB);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              const int step = half * 4 + k;
              if (step % kStepsPerGroup == 0 && acc >= 2) {
                if (!mbar_wait(acc_empty(acc & 1), (acc / 2 + 1) & 1, kWaitLimit)) {
                  ok = false;
                  break;
                }
                tcgen05_fence_after();
              }
              mma_bf16(tmem + (uint32_t)((acc & 1) * BT), da + 2 * k, db + 2 * k, idesc, step % kStepsPerGroup != 0);
              if ((step + 1) % kStepsPerGroup == 0) {
                mma_commit(acc_full(acc & 1));
                ++acc;
              }
            }
            mma_commit(a_empty(sa));
            mma_commit(b_empty(sb));
          }
        }
      }
      if (!ok) fail_w4(abort_flag);
      mma_commit(drain);
      if (!mbar_wait(drain, 0, kWaitLimit)) fail_w4(abort_flag);
    }
  } else if (warp < L::kEpiWarp) {
    // nibbles to bf16: thread = weight row of the tile
    regs_dec<L::kRegsDq>();
    const int wg = warp / 4 - 1;
    const int row = threadIdx.x & 127;
    int g = 0;
    bool ok = true;
    for (int t = t_first; t < tiles && ok && !*abort_flag; t += t_step) {
      const int n = t % n_tiles * kBN + row;
      const uint8_t* zrow = zeros && n < N ? zeros + (int64_t)n * ld_z : nullptr;
      for (int ch = cb; ch < ce && ok; ++ch, ++g) {
        const int s = g % SQ;
        uint32_t zp[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) zp[b] = zrow && ch * kChunk + b * 32 < K ? zrow[ch * kG + b * 32 / GROUP] & 127u : 8u;
        if (!mbar_wait(q_full(s), (g / SQ) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        const uint4* src = reinterpret_cast<const uint4*>(gbase + L::kOffQ + s * L::kStageQ + row * 64);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (L::kDqGroups == 2 && half != wg) continue;
          const uint4 q[2] = {src[2 * half], src[2 * half + 1]};
          const int ks = 2 * g + half, sa = ks % SA;
          if (ks >= SA && !mbar_wait(a_empty(sa), (ks / SA + 1) & 1, kWaitLimit)) {
            ok = false;
            break;
          }
          unsigned char* dst = gbase + L::kOffA + sa * L::kStageA + row * 128;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const __nv_bfloat162 zc = zero_pair(zp[2 * half + b]);
            const uint32_t w[4] = {q[b].x, q[b].y, q[b].z, q[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(dst + (((b * 4 + i) ^ (row & 7)) << 4)) = unpack8(w[i], zc);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(a_full(sa));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty(s));
      }
    }
    if (!ok && lane == 0) fail_w4(abort_flag);
  } else {
    regs_inc<L::kRegsEpi>();
    constexpr int kCols = BT / 2;  // columns of a warp
    const int quad = warp & 3, h = (warp - L::kEpiWarp) / 4;
    const int row = quad * 32 + lane;
    int acc = 0;
    bool ok = true;
    for (int t = t_first; t < tiles && ok && !*abort_flag; t += t_step) {
      const int n = t % n_tiles * kBN + row, m0 = t / n_tiles * BT + h * kCols;
      const bool n_in = n < N;
      float2 total[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) total[j] = make_float2(0.0f, 0.0f);
      auto scale_of = [&](int gr) {
        if (!n_in || (int64_t)gr * GROUP >= K) return 0.0f;
        const int64_t i = (int64_t)n * ld_s + gr;
        return s_bf16 ? to_f32(static_cast<const __nv_bfloat16*>(scales)[i]) : static_cast<const float*>(scales)[i];
      };
      float next = scale_of(cb * kG);
      for (int gr = cb * kG; gr < ce * kG; ++gr, ++acc) {
        const float sc = next;
        if (gr + 1 < ce * kG) next = scale_of(gr + 1);
        if (!mbar_wait(acc_full(acc & 1), (acc / 2) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        tcgen05_fence_after();
        const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)((acc & 1) * BT + h * kCols);
        const float2 s2 = make_float2(sc, sc);
        uint32_t v[2][16];
        tmem_ld16(taddr, v[0]);
        tmem_wait(v[0]);
#pragma unroll
        for (int j = 0; j < kCols / 16; ++j) {
          if (j + 1 < kCols / 16) tmem_ld16(taddr + (uint32_t)(16 * (j + 1)), v[(j + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            total[8 * j + i] = __ffma2_rn(
                s2, make_float2(__uint_as_float(v[j & 1][2 * i]), __uint_as_float(v[j & 1][2 * i + 1])),
                total[8 * j + i]);
          if (j + 1 < kCols / 16) tmem_wait(v[(j + 1) & 1]);
        }
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(acc & 1));
      }
      if (!ok) break;
      if constexpr (SPLIT) {
        // over the idle operand ring: [column][row]
        float* part = reinterpret_cast<float*>(gbase) + (h * kCols) * L::kPartPitch + row;
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
          part[(2 * j) * L::kPartPitch] = total[j].x;
          part[(2 * j + 1) * L::kPartPitch] = total[j].y;
        }
      } else if (n_in) {
        const int cols = M - m0 < kCols ? M - m0 : kCols;
        const float* rp = r ? r + (int64_t)m0 * ld_r + n : nullptr;
        if (c_bf16) {
          __nv_bfloat16* cp = static_cast<__nv_bfloat16*>(c) + (int64_t)m0 * ld_c + n;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            float v = j & 1 ? total[j / 2].y : total[j / 2].x;
            if (j < cols) {
              if (rp) v += rp[(int64_t)j * ld_r];
              cp[(int64_t)j * ld_c] = __float2bfloat16_rn(v);
            }
          }
        } else {
          float* cp = static_cast<float*>(c) + (int64_t)m0 * ld_c + n;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            float v = j & 1 ? total[j / 2].y : total[j / 2].x;
            if (j < cols) {
              if (rp) v += rp[(int64_t)j * ld_r];
              cp[(int64_t)j * ld_c] = v;
            }
          }
        }
      }
    }
    if (!ok && lane == 0) fail_w4(abort_flag);
  }
  __syncwarp();
  if constexpr (SPLIT) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // the totals of every rank are in place
    if (warp >= L::kEpiWarp && !*abort_flag) {
      // rank q finishes columns [q BT / splits, (q + 1) BT / splits): each element the
      // ranks' totals in rank order, 4 weight rows a thread
      const int n0 = t_first % n_tiles * kBN, m0 = t_first / n_tiles * BT;
      const int e = threadIdx.x - 32 * L::kEpiWarp, n = n0 + (e & 31) * 4;
      for (int j = rank * BT / splits + e / 32; j < (rank + 1) * BT / splits; j += kEpiWarps) {
        if (m0 + j >= M) break;
        const uint32_t at = base + (uint32_t)((j * L::kPartPitch + (e & 31) * 4) * 4);
        float4 x = dsmem_ld4(at, 0);
        for (int q = 1; q < splits; ++q) {
          const float4 y = dsmem_ld4(at, q);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (n + i >= N) break;
          const float rv = r ? r[(int64_t)(m0 + j) * ld_r + n + i] : 0.0f;
          store_out(c, (int64_t)(m0 + j) * ld_c + n + i, c_bf16, r ? v[i] + rv : v[i]);
        }
      }
    }
    cluster.sync();  // every rank has read its peers' shared memory
  }
  tcgen05_fence_before();
  __syncthreads();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols) : "memory");
}

template <int BT, int GROUP, bool SPLIT>
cudaError_t launch_one(const LinearW4Args& g, const CUtensorMap& ma, const CUtensorMap& mq, int sms, int splits,
                       cudaStream_t stream) {
  auto kern = gemm_w4_kernel<BT, GROUP, SPLIT>;
  using L = Cfg<BT>;
  static int configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!__atomic_load_n(&configured[dev], __ATOMIC_RELAXED)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc)) != cudaSuccess)
      return e;
    // the roles' registers come out of what the CTA is launched with
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
    if (at.numRegs * (L::kThreads / 128) < L::kRegs) return cudaErrorInvalidConfiguration;
    __atomic_store_n(&configured[dev], 1, __ATOMIC_RELAXED);
  }
  const int64_t tiles = ((g.M + BT - 1) / BT) * ((g.N + kBN - 1) / kBN);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * splits : (tiles < sms ? tiles : sms)));
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, ma, mq, g.c, g.ld_c, g.c_bf16, g.scales, g.ld_s, g.s_bf16, g.zeros, g.ld_z,
                            g.r, g.ld_r, (int)g.M, (int)g.N, (int)g.K, SPLIT ? splits : 1);
}

template <int BT>
cudaError_t launch_bt(const LinearW4Args& g, int sms, cudaStream_t stream) {
  CUtensorMap ma, mq;
  const int64_t row_bytes = (g.K + 31) / 32 * 16;
  if (!tensor_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.a, g.M, g.K, (g.M > 1 ? g.ld_a : (g.K + 7) / 8 * 8) * 2,
                     BT, kBK, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tensor_map_2d(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.q, g.N, row_bytes, g.N > 1 ? g.ld_q : row_bytes, kBN,
                     kChunk / 2, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  // a cluster per tile where the tiles leave SMs idle: up to 8 CTAs, a chunk each at least
  const int64_t tiles = ((g.M + BT - 1) / BT) * ((g.N + kBN - 1) / kBN), chunks = (g.K + kChunk - 1) / kChunk;
  int64_t splits = tiles <= sms ? sms / tiles : 1;
  if (splits > 8) splits = 8;
  if (splits > chunks) splits = chunks;
  if constexpr (BT <= 128) {
    if (splits > 1) {
      if (g.group == 32) return launch_one<BT, 32, true>(g, ma, mq, sms, (int)splits, stream);
      if (g.group == 64) return launch_one<BT, 64, true>(g, ma, mq, sms, (int)splits, stream);
      return launch_one<BT, 128, true>(g, ma, mq, sms, (int)splits, stream);
    }
  }
  if (g.group == 32) return launch_one<BT, 32, false>(g, ma, mq, sms, 1, stream);
  if (g.group == 64) return launch_one<BT, 64, false>(g, ma, mq, sms, 1, stream);
  return launch_one<BT, 128, false>(g, ma, mq, sms, 1, stream);
}

}  // namespace

cudaError_t launch_gemm_w4(const LinearW4Args& g, const DeviceInfo& dev, cudaStream_t stream) {
  if (g.M <= 32) return launch_bt<32>(g, dev.sm_count, stream);
  if (g.M <= 64) return launch_bt<64>(g, dev.sm_count, stream);
  if (g.M <= 128) return launch_bt<128>(g, dev.sm_count, stream);
  return launch_bt<256>(g, dev.sm_count, stream);
}

int read_gemm_w4_faults(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemm_w4_faults, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_gemm_w4_faults, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace mamba
