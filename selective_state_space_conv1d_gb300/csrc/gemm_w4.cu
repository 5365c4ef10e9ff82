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
constexpr int kReduceChunks = 3;  // a cluster's reduction takes about as long as 3 chunks
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
  static constexpr int kRegsDq = 88;
  static constexpr int kRegsEpi = kDqGroups == 1 ? 192 : 128;
  static constexpr int kRegs = kRegsLoad + kDqGroups * kRegsDq + 2 * kRegsEpi;
  static_assert(kRegs <= (65536 / kThreads / 8 * 8) * (kThreads / 128), "more registers than a CTA has");
  static constexpr int kStageB = BT * kBK * 2;
  static constexpr int kStageA = kBN * kBK * 2;
  static constexpr int kStageQ = kBN * kChunk / 2;
  static constexpr int kStage = kStageB + kStageA;
  static constexpr int kS = BT == 256 ? 4 : (BT == 128 ? 5 : 6);  // operand stages
  static constexpr int kOffQ = kS * kStage;
  static constexpr int kSQ0 = (kSmemLimit - 1024 - 512 - kOffQ) / kStageQ;
  static constexpr int kSQ = kSQ0 > 8 ? 8 : kSQ0;                 // weights as they are stored
  static constexpr int kOffBar = kOffQ + kSQ * kStageQ;
  static constexpr int kBars = 2 * (kS + kSQ) + 5;
  static constexpr int kBytes = kOffBar + 8 * kBars + 16;
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base
  static constexpr int kTmemCols = 2 * BT;
  static constexpr int kPartPitch = kBN + 4;
  static_assert(kAlloc <= kSmemLimit && kSQ >= 2 && kS >= 4, "shared memory");
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

// a row's scale of group g, 0 past its groups
__device__ __forceinline__ float scale_at(const void* scales, int s_bf16, int64_t row, int g, int groups) {
  if (g >= groups) return 0.0f;
  return s_bf16 ? to_f32(static_cast<const __nv_bfloat16*>(scales)[row + g])
                : static_cast<const float*>(scales)[row + g];
}

// a row's zero point for the b-th 32 k
template <int GROUP>
__device__ __forceinline__ uint32_t zero_at(const uint8_t* row, int b, int K) {
  return row && b * 32 < K ? row[b * 32 / GROUP] & 127u : 8u;
}

// one weight row's totals down a column of C, the residual (or null) added: 16 at a
// time, a batch's residuals read together
template <typename T, int PAIRS>
__device__ __forceinline__ void store_totals(T* c, int64_t ld_c, const float* r, int64_t ld_r,
                                             const float2 (&total)[PAIRS], int cols) {
#pragma unroll
  for (int j0 = 0; j0 < 2 * PAIRS; j0 += 16) {
    if (j0 >= cols) return;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = j & 1 ? total[(j0 + j) / 2].y : total[(j0 + j) / 2].x;
    if (cols - j0 >= 16) {
      if (r) {
        float rv[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) rv[j] = r[j * ld_r];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += rv[j];
        r += 16 * ld_r;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        *c = from_f32<T>(v[j]);
        c += ld_c;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j0 + j < cols) c[j * ld_c] = from_f32<T>(r ? v[j] + r[j * ld_r] : v[j]);
    }
  }
}

// the stage that was written is handed to the tensor cores
__device__ __forceinline__ void hand_over(uint32_t bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
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
  constexpr int S = L::kS, SQ = L::kSQ;
  constexpr int kG = kChunk / GROUP;          // groups per chunk
  constexpr int kStepsPerGroup = GROUP / 16;  // products per group
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kOffBar;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (S + s); };
  auto q_full = [&](int s) { return bars + 8 * (2 * S + s); };
  auto q_empty = [&](int s) { return bars + 8 * (2 * S + SQ + s); };
  auto mid = [&](int a) { return bars + 8 * (2 * (S + SQ) + a); };
  auto acc_empty = [&](int a) { return bars + 8 * (2 * (S + SQ) + 2 + a); };
  const uint32_t drain = bars + 8 * (2 * (S + SQ) + 4);
  auto stage_b = [&](int s) { return base + (uint32_t)(s * L::kStage); };
  auto stage_a = [&](int s) { return base + (uint32_t)(s * L::kStage + L::kStageB); };
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
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 5);  // the copy of the activations and four warps' weights
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < SQ; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 4 * L::kDqGroups);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(mid(a), 1);
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
          const int s = g % S;
          if (g >= S && !mbar_wait(empty(s), (g / S + 1) & 1, kWaitLimit)) {
            fail_w4(abort_flag);
            break;
          }
          mbar_arrive_expect_tx(full(s), L::kStageB);
          tma_load_2d(stage_b(s), &map_a, ks * kBK, m0, full(s));
        }
      }
      // the copies issued land: their stages complete, unless the weights' side gave up
      for (int i = g > S ? g - S : 0; i < g; ++i)
        if (!mbar_wait(full(i % S), (i / S) & 1, kWaitLimit)) fail_w4(abort_flag);
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
            const int s = g % S;
            if (!mbar_wait(full(s), (g / S) & 1, kWaitLimit)) {
              ok = false;
              break;
            }
            tcgen05_fence_after();
            const uint64_t da = smem_desc(stage_a(s)), db = smem_desc(stage_b(s));
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              const int step = half * 4 + k;
              if (step % kStepsPerGroup == 0) {
                if (acc >= 2 && !mbar_wait(acc_empty(acc & 1), (acc / 2 + 1) & 1, kWaitLimit)) {
                  ok = false;
                  break;
                }
                tcgen05_fence_after();
              }
              mma_bf16(tmem + (uint32_t)((acc & 1) * BT), da + 2 * k, db + 2 * k, idesc, step % kStepsPerGroup != 0);
              if ((step + 1) % kStepsPerGroup == 0) ++acc;
              // a commit takes the issuing thread about 180 cycles: a stage's own says
              // too that the group which ends with it is complete
              if (GROUP == 32 && k == 1) mma_commit(mid(g & 1));
            }
            mma_commit(empty(s));
          }
        }
      }
      if (!ok) fail_w4(abort_flag);
      mma_commit(drain);
      if (!mbar_wait(drain, 0, kWaitLimit)) fail_w4(abort_flag);
    }
  } else if (warp < L::kEpiWarp) {
    // nibbles to bf16: thread = weight row of the tile.  A stage is handed over one
    // turn after it was written: its stores are done by then, and the fence that
    // makes them visible to the tensor cores waits for nothing.
    regs_dec<L::kRegsDq>();
    const int wg = warp / 4 - 1;
    const int row = threadIdx.x & 127;
    int g = 0, owed = -1;  // chunks taken; the stage not handed over yet
    bool ok = true;
    for (int t = t_first; t < tiles && ok && !*abort_flag; t += t_step) {
      const int n = t % n_tiles * kBN + row;
      const uint8_t* zrow = zeros && n < N ? zeros + (int64_t)n * ld_z : nullptr;
      uint32_t zp[4], zn[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) zn[b] = zero_at<GROUP>(zrow, cb * 4 + b, K);
      for (int ch = cb; ch < ce; ++ch, ++g) {
        const int s = g % SQ;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          zp[b] = zn[b];
          if (ch + 1 < ce) zn[b] = zero_at<GROUP>(zrow, ch * 4 + 4 + b, K);
        }
        if (!mbar_wait(q_full(s), (g / SQ) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        // the copy's 64-byte swizzle: piece b of row r at b ^ (r / 2 % 4)
        const unsigned char* src = gbase + L::kOffQ + s * L::kStageQ + row * 64;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (L::kDqGroups == 2 && half != wg) continue;
          uint4 q[2];
#pragma unroll
          for (int b = 0; b < 2; ++b)
            q[b] = *reinterpret_cast<const uint4*>(src + (((2 * half + b) ^ ((row >> 1) & 3)) << 4));
          const int ks = 2 * g + half, sa = ks % S;
          uint4 v[8];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const __nv_bfloat162 zc = zero_pair(zp[2 * half + b]);
            v[4 * b] = unpack8(q[b].x, zc);
            v[4 * b + 1] = unpack8(q[b].y, zc);
            v[4 * b + 2] = unpack8(q[b].z, zc);
            v[4 * b + 3] = unpack8(q[b].w, zc);
          }
          if (owed >= 0) hand_over(full(owed), lane);  // before a wait that may need it
          owed = -1;
          if (ks >= S && !mbar_wait(empty(sa), (ks / S + 1) & 1, kWaitLimit)) {
            ok = false;
            break;
          }
          unsigned char* dst = gbase + sa * L::kStage + L::kStageB + row * 128;
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + ((i ^ (row & 7)) << 4)) = v[i];
          owed = sa;
          // the copy of the next weights goes through another proxy than the reads of
          // these: it may start when they are done for certain, their results stored
          if (L::kDqGroups == 2 || half == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty(s));
          }
        }
        if (!ok) break;
      }
    }
    if (owed >= 0) hand_over(full(owed), lane);
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
      const int groups = n_in ? (K + GROUP - 1) / GROUP : 0;
      const int64_t s_row = (int64_t)n * ld_s;
      float next = scale_at(scales, s_bf16, s_row, cb * kG, groups);
      for (int gr = cb * kG; gr < ce * kG; ++gr, ++acc) {
        const float sc = next;
        next = scale_at(scales, s_bf16, s_row, gr + 1, groups);
        // the group is complete when its last stage is (or half of it): the products are
        // at most two groups ahead of this, so that barrier's next phase is not over
        const int ks = GROUP == 128 ? 2 * acc + 1 : (GROUP == 64 ? acc : acc / 2);
        const bool half = GROUP == 32 && !(acc & 1);
        if (!mbar_wait(half ? mid(ks & 1) : empty(ks % S), (half ? ks / 2 : ks / S) & 1, kWaitLimit)) {
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
        if (c_bf16)
          store_totals(static_cast<__nv_bfloat16*>(c) + (int64_t)m0 * ld_c + n, ld_c, rp, ld_r, total, cols);
        else
          store_totals(static_cast<float*>(c) + (int64_t)m0 * ld_c + n, ld_c, rp, ld_r, total, cols);
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

constexpr int kMaxSplits = 8;
constexpr int kMaxDevices = 64;

// Shared memory, the check of the registers, and how many clusters of each size the
// device holds at once (a GPC's SMs are no multiple of most sizes).
struct Resident {
  int configured;
  int clusters[kMaxSplits + 1];
};

template <int BT, int GROUP, bool SPLIT>
cudaError_t configure(const Resident** out) {
  auto kern = gemm_w4_kernel<BT, GROUP, SPLIT>;
  using L = Cfg<BT>;
  static Resident resident[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  Resident& r = resident[dev];
  if (!__atomic_load_n(&r.configured, __ATOMIC_ACQUIRE)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc)) != cudaSuccess)
      return e;
    // the roles' registers come out of what the CTA is launched with
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
    if (at.numRegs * (L::kThreads / 128) < L::kRegs) return cudaErrorInvalidConfiguration;
    if (SPLIT) {
      for (int size = 2; size <= kMaxSplits; ++size) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(L::kThreads);
        cfg.dynamicSmemBytes = L::kAlloc;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = size;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
        __atomic_store_n(&r.clusters[size], n, __ATOMIC_RELAXED);
      }
    }
    __atomic_store_n(&r.configured, 1, __ATOMIC_RELEASE);
  }
  *out = &r;
  return cudaSuccess;
}

// Chunks of K a CTA works through one after another, and the reduction's time in chunks
template <int BT, int GROUP>
cudaError_t choose_splits(const LinearW4Args& g, int sms, int* splits) {
  const Resident* r = nullptr;
  const cudaError_t e = configure<BT, GROUP, true>(&r);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((g.M + BT - 1) / BT) * ((g.N + kBN - 1) / kBN), chunks = (g.K + kChunk - 1) / kChunk;
  int64_t best = (tiles + sms - 1) / sms * chunks;
  *splits = 1;
  for (int size = 2; size <= kMaxSplits && size <= chunks; ++size) {
    const int64_t held = __atomic_load_n(&r->clusters[size], __ATOMIC_RELAXED);
    if (held < 1) continue;
    const int64_t cost = (tiles + held - 1) / held * ((chunks + size - 1) / size + kReduceChunks);
    if (cost < best) {
      best = cost;
      *splits = size;
    }
  }
  return cudaSuccess;
}

template <int BT, int GROUP, bool SPLIT>
cudaError_t launch_one(const LinearW4Args& g, const CUtensorMap& ma, const CUtensorMap& mq, int sms, int splits,
                       cudaStream_t stream) {
  auto kern = gemm_w4_kernel<BT, GROUP, SPLIT>;
  using L = Cfg<BT>;
  const Resident* held = nullptr;
  const cudaError_t e = configure<BT, GROUP, SPLIT>(&held);
  if (e != cudaSuccess) return e;
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
                     kChunk / 2, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  if constexpr (BT <= 128) {
    int splits = 1;
    const cudaError_t e = g.group == 32   ? choose_splits<BT, 32>(g, sms, &splits)
                          : g.group == 64 ? choose_splits<BT, 64>(g, sms, &splits)
                                          : choose_splits<BT, 128>(g, sms, &splits);
    if (e != cudaSuccess) return e;
    if (splits > 1) {
      if (g.group == 32) return launch_one<BT, 32, true>(g, ma, mq, sms, splits, stream);
      if (g.group == 64) return launch_one<BT, 64, true>(g, ma, mq, sms, splits, stream);
      return launch_one<BT, 128, true>(g, ma, mq, sms, splits, stream);
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
