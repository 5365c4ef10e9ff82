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
//  * warp 0 brings activations, BT x 64 bf16 with the 128-byte swizzle a copy (TMA);
//  * warp 2 brings weights as they are stored, 128 rows x 64 bytes (128 k) a copy;
//  * four warpgroups, a thread per weight row, make bf16 of the nibbles, 64 k of every
//    second chunk of 128 a warpgroup (two take the even chunks' halves, two the odd
//    ones'): two operations a pair (nibbles i and i + 4 of a word in the halves of a
//    register, 0x4300 above them: 128 + q; a packed subtraction of 128 + z), a byte
//    permutation that puts neighbours side by side, and a store into tensor memory,
//    where the product reads its weights (through shared memory they cost it 32 KB
//    written and 32 read per chunk, beside the activations' own: 343 us for 8192 x
//    10240 x 2560);
//  * warp 1 issues the products, a group of k into one of a few accumulators;
//  * two warpgroups take the finished accumulators meanwhile, each half of the columns:
//    total += scale * group's sum, BT / 2 totals a thread in registers, and store
//    the totals at the end of a tile (a warp stores 32 neighbours of a row of C).
// Few tiles: K is split over a cluster whose CTAs add their totals through
// distributed shared memory in rank order.
//
// 8192 x 10240 x 2560 in groups of 128 takes 330 us in a graph of four calls (1.30 PFLOP/s)
// and 349 call by call (long runs come under the power limit); in groups of 64 421 and of 32
// 629 in such a graph: a group costs its commit and a pass of the totals, whatever it holds.
// No unit is full (2048 rows: issue slots 65 %, the waiting roles' polls among them, tensor
// pipe 50, L2 29): the roles wait for one another, which for which is not measured.
// 128 rows in groups of 64: 18.7 us in a graph, 8 of them the start up to the first product
// and the end; 0.36 us a chunk.
// Against mamba_linear_bf16 (gemm.cu), us in a graph, groups of 128 here: 10240 x 2560, 16
// rows 13.4 and 22.3, 128 rows 15.6 and 15.3, 256 rows 27.3 and 18.0, 8192 rows 343 and 276;
// 2560 x 5120, 128 rows 11.2 and 16.3, 8192 rows 168 and 161.
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
constexpr int kBK = 64;     // k per operand block: one 128-byte swizzle row
constexpr int kChunk = 128; // k per copy of weights
constexpr int kEpiWarps = 8;
constexpr int kReduceChunks = 3;  // a cluster's reduction takes about as long as 3 chunks
constexpr int kSmemLimit = 232448;
constexpr long long kWaitLimit = 1ll << 31;  // SM cycles (about a second)

__device__ int g_gemm_w4_faults = 0;

constexpr int kDqGroups = 4;   // warpgroups that make bf16 of nibbles
constexpr int kThreads = 128 * (1 + kDqGroups + 2);
constexpr int kEpiWarp = 4 * (1 + kDqGroups);
// registers per thread of the roles; their sum over the warpgroups is what the CTA is
// launched with (72 x 7)
constexpr int kRegsLoad = 40, kRegsDq = 40, kRegsEpi = 152;
constexpr int kRegs = kRegsLoad + kDqGroups * kRegsDq + 2 * kRegsEpi;
static_assert(kRegs <= (65536 / kThreads / 8 * 8) * (kThreads / 128), "more registers than a CTA has");
constexpr int kSA = 4;         // stages of weights in tensor memory
constexpr int kDone = 8;       // barriers of finished stages
constexpr int kTmemCols = 512;

// Stages are of 128 k (a stage costs its waits and hand-overs, whatever it holds), of 64
// where tensor memory has no room for four such beside the accumulators.
template <int BT>
struct Cfg {
  static constexpr int kSub = BT > 128 ? 1 : 2;  // blocks of 64 k per stage
  static constexpr int kStageCols = 32 * kSub;   // of weights in tensor memory
  static constexpr int kOffA = kTmemCols - kSA * kStageCols;
  static constexpr int kAcc0 = kOffA / BT;       // accumulators
  static constexpr int kAcc = kAcc0 > 4 ? 4 : kAcc0;
  static constexpr int kBlockB = BT * kBK * 2;
  static constexpr int kStageB = kSub * kBlockB;
  static constexpr int kSB = BT == 128 ? 4 : 8;                   // stages of activations
  static constexpr int kStageQ = kBN * kChunk / 2;
  static constexpr int kOffQ = kSB * kStageB;
  static constexpr int kSQ0 = (kSmemLimit - 1024 - 512 - kOffQ) / kStageQ;
  static constexpr int kSQ = kSQ0 > 8 ? 8 : kSQ0;                 // chunks of weights as they are stored
  static constexpr int kOffBar = kOffQ + kSQ * kStageQ;
  static constexpr int kBars = kSA + kSB + 2 * kSQ + kDone + 3 * 4 + 1;
  static constexpr int kBytes = kOffBar + 8 * kBars + 16;
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base
  static constexpr int kPartPitch = kBN + 4;
  static_assert(kAlloc <= kSmemLimit && kSQ >= 4 && kAcc >= 2, "shared or tensor memory");
  // a stage's barrier is waited for by the copies (kSB stages later), the weights (kSA
  // later) and the totals (of up to kAcc groups of 128 k): none is a round behind
  static_assert(kSB <= kDone && kAcc * 2 / kSub < kDone, "a stage's barrier a round behind");
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

// A from tensor memory: lane = row, a 32-bit column = two values of K
__device__ __forceinline__ void mma_bf16(uint32_t tmem_d, uint32_t a, uint32_t b_hi, uint32_t b_lo, uint32_t idesc,
                                         uint32_t acc) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  .reg .b64 b;\n"
      "  mov.b64 b, {%3, %2};\n"
      "  setp.ne.b32 p, %5, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n"
      "}\n" ::"r"(tmem_d),
      "r"(a), "r"(b_hi), "r"(b_lo), "r"(idesc), "r"(acc)
      : "memory");
}

// one thread of a whole warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n  .reg .pred p;\n  elect.sync _|p, 0xffffffff;\n  selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
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

// The scales of a row's G groups in a chunk, as the bits that the loads bring (a value
// made of them would be waited for where it is made): mode 0 f32, 1 bf16 in a word each,
// 2 bf16 in pairs (aligned: a warp's rows are 32 lines of the cache, whatever it takes of
// them).  0 past the row's groups.
template <int G>
struct ChunkScales {
  uint32_t r[G];
  __device__ __forceinline__ void fetch(const void* scales, int mode, int64_t row, int g, int groups) {
    if (mode == 2 && G > 1) {
#pragma unroll
      for (int e = 0; e < G / 2; ++e) r[e] = 0;
      const uint16_t* p = static_cast<const uint16_t*>(scales) + row + g;
      if (g + G <= groups) {
        if constexpr (G == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          r[0] = v.x, r[1] = v.y;
        } else {
          r[0] = *reinterpret_cast<const uint32_t*>(p);
        }
      } else {
#pragma unroll
        for (int e = 0; e + 1 < G; ++e)
          if (g + e < groups) r[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
      }
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e)
        r[e] = g + e >= groups ? 0u
                               : (mode ? (uint32_t)static_cast<const uint16_t*>(scales)[row + g + e]
                                       : static_cast<const uint32_t*>(scales)[row + g + e]);
    }
  }
  __device__ __forceinline__ float get(int mode, int e) const {
    if (mode == 2 && G > 1) return __uint_as_float(e & 1 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16);
    return __uint_as_float(mode ? r[e] << 16 : r[e]);
  }
};

// a row's zero point for the b-th 32 k
template <int GROUP>
__device__ __forceinline__ uint32_t zero_at(const uint8_t* row, int b, int K) {
  return row && b * 32 < K ? row[b * 32 / GROUP] & 127u : 8u;
}

__device__ __forceinline__ void tmem_take(uint32_t taddr, uint32_t (&v)[8]) { tmem_ld8(taddr, v); }
__device__ __forceinline__ void tmem_take(uint32_t taddr, uint32_t (&v)[16]) { tmem_ld16(taddr, v); }

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

__device__ __forceinline__ void fail_w4(volatile int* abort_flag) {
  atomicOr(&g_gemm_w4_faults, MAMBA_FAULT_GEMM_WAIT);
  *abort_flag = 1;
}

template <int BT, int GROUP, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_w4_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_q, void* c,
                   int64_t ld_c, int c_bf16, const void* __restrict__ scales, int64_t ld_s, int s_mode,
                   const uint8_t* __restrict__ zeros, int64_t ld_z, const float* r, int64_t ld_r, int M, int N, int K,
                   int splits) {
  using L = Cfg<BT>;
  constexpr int SB = L::kSB, SQ = L::kSQ, kAcc = L::kAcc;
  constexpr int kG = kChunk / GROUP;          // groups per chunk
  constexpr int kStepsPerGroup = GROUP / 16;  // products per group
  constexpr int kStages = 2 / L::kSub;        // stages per chunk
  constexpr int kSteps = 4 * L::kSub;         // products per stage
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kOffBar;
  auto a_full = [&](int s) { return bars + 8 * s; };
  auto b_full = [&](int s) { return bars + 8 * (kSA + s); };
  auto q_full = [&](int s) { return bars + 8 * (kSA + SB + s); };
  auto q_empty = [&](int s) { return bars + 8 * (kSA + SB + SQ + s); };
  const uint32_t bars1 = bars + 8 * (kSA + SB + 2 * SQ);
  auto done = [&](int s) { return bars1 + 8 * s; };
  auto mid = [&](int a) { return bars1 + 8 * (kDone + a); };
  auto acc_empty = [&](int a) { return bars1 + 8 * (kDone + 4 + a); };
  const uint32_t drain = bars1 + 8 * (kDone + 8);
  auto stage_b = [&](int s) { return base + (uint32_t)(s * L::kStageB); };
  // the products of stage number st (and all before it) are complete
  auto stage_done = [&](int st) {
    return st < 0 || mbar_wait(done(st % kDone), (uint32_t)(st / kDone) & 1, kWaitLimit);
  };
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
    for (int s = 0; s < kSA; ++s) mbar_init(a_full(s), 4 * L::kSub);
    for (int s = 0; s < SB; ++s) mbar_init(b_full(s), 1);
    for (int s = 0; s < SQ; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 8);
    }
    for (int s = 0; s < kDone; ++s) mbar_init(done(s), 1);
    for (int a = 0; a < kAcc; ++a) {
      mbar_init(mid(a), 1);
      mbar_init(acc_empty(a), kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_ptr)),
                 "r"(kTmemCols)
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
    regs_dec<kRegsLoad>();
    if (warp == 0 && lane == 0) {
      // activations
      int g = 0;
      for (int t = t_first; t < tiles && !*abort_flag; t += t_step) {
        const int m0 = t / n_tiles * BT;
        for (int st = kStages * cb; st < kStages * ce; ++st, ++g) {
          const int s = g % SB;
          if (!stage_done(g - SB)) {
            fail_w4(abort_flag);
            break;
          }
          mbar_arrive_expect_tx(b_full(s), L::kStageB);
#pragma unroll
          for (int sub = 0; sub < L::kSub; ++sub)
            tma_load_2d(stage_b(s) + sub * L::kBlockB, &map_a, (st * L::kSub + sub) * kBK, m0, b_full(s));
        }
      }
      // every copy issued lands before this thread moves on
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
    } else if (warp == 1) {
      // products.  The whole warp goes through the loop and one thread of it issues: what
      // the instructions take from uniform registers (descriptors, addresses) stays there.
      // Counters wrap by masks: this warp's own instructions are what a stage takes least.
      constexpr uint32_t idesc = instr_desc<BT>();
      const uint64_t desc0 = smem_desc(base);
      const uint32_t desc_hi = (uint32_t)(desc0 >> 32), desc_lo = (uint32_t)desc0;
      const bool issuer = elect_one();
      int g = 0, acc = 0, inner = 0;
      bool ok = true;
      for (int t = t_first; t < tiles && ok && !*abort_flag; t += t_step) {
        for (int ch = cb; ch < ce && ok; ++ch) {
#pragma unroll
          for (int st = 0; st < kStages; ++st, ++g) {
            const int sa = g % kSA, sb = g % SB;
            ok = mbar_wait(a_full(sa), (g / kSA) & 1, kWaitLimit) && mbar_wait(b_full(sb), (g / SB) & 1, kWaitLimit);
            const uint32_t da = tmem + (uint32_t)(L::kOffA + sa * L::kStageCols);
            const uint32_t db = desc_lo + (uint32_t)(sb * (L::kStageB >> 4));
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const int step = st * kSteps + k;
              if (step % kStepsPerGroup == 0 && acc >= kAcc)
                ok = ok && mbar_wait(acc_empty(acc % kAcc), (uint32_t)(acc / kAcc + 1) & 1, kWaitLimit);
              if (!ok) break;
              if (k == 0 || step % kStepsPerGroup == 0) tcgen05_fence_after();
              const uint32_t d = tmem + (uint32_t)(acc % kAcc * BT);
              if (issuer)
                mma_bf16(d, da + 8 * k, desc_hi, db + (k / 4) * (L::kBlockB >> 4) + 2 * (k % 4), idesc,
                         step % kStepsPerGroup != 0);
              if ((step + 1) % kStepsPerGroup == 0) {
                ++acc;
                // a commit takes the issuing thread about 180 cycles: the stage's own
                // says too that the group which ends with it is complete
                if (k + 1 < kSteps) {
                  if (issuer) mma_commit(mid(inner % kAcc));
                  ++inner;
                }
              }
            }
            if (!ok) break;
            if (issuer) mma_commit(done(g % kDone));
          }
        }
      }
      if (!ok && issuer) fail_w4(abort_flag);
      if (issuer) mma_commit(drain);
      if (!mbar_wait(drain, 0, kWaitLimit) && issuer) fail_w4(abort_flag);
    }
  } else if (warp < kEpiWarp) {
    // nibbles to bf16: thread = weight row of the tile; warpgroups 0 and 1 take the halves
    // of one chunk, 2 and 3 those of the next
    regs_dec<kRegsDq>();
    const int wg = warp / 4 - 1, half = wg & 1;
    const int row = threadIdx.x & 127;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16) +
                               (uint32_t)(L::kOffA + (L::kSub == 2 ? half * 32 : 0));
    int g = 0;  // chunks so far
    bool ok = true;
    for (int t = t_first; t < tiles && ok && !*abort_flag; t += t_step) {
      const int n = t % n_tiles * kBN + row;
      const uint8_t* zrow = zeros && n < N ? zeros + (int64_t)n * ld_z : nullptr;
      for (int ch = cb; ch < ce; ++ch, ++g) {
        if ((g & 1) != wg / 2) continue;
        const int s = g % SQ;
        uint32_t zp[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) zp[b] = zero_at<GROUP>(zrow, ch * 4 + half * 2 + b, K);
        if (!mbar_wait(q_full(s), (g / SQ) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        const unsigned char* src = gbase + L::kOffQ + s * L::kStageQ + row * 64;
        const int st = g * kStages + (L::kSub == 2 ? 0 : half);
        const uint32_t at = lane_addr + (uint32_t)(st % kSA * L::kStageCols);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          // the copy's 64-byte swizzle: piece b of row r at b ^ (r / 2 % 4)
          const uint4 q = *reinterpret_cast<const uint4*>(src + (((half * 2 + b) ^ ((row >> 1) & 3)) << 4));
          const __nv_bfloat162 zc = zero_pair(zp[b]);
          const uint4 v[4] = {unpack8(q.x, zc), unpack8(q.y, zc), unpack8(q.z, zc), unpack8(q.w, zc)};
          if (b == 0) {
            if (!stage_done(st - kSA)) {
              ok = false;
              break;
            }
            tcgen05_fence_after();
          }
          const uint32_t lo[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
          const uint32_t hi[8] = {v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
          tmem_st8(at + 16 * b, lo);
          tmem_st8(at + 16 * b + 8, hi);
        }
        if (!ok) break;
        tmem_wait_st();
        tcgen05_fence_before();
        // the copy of the next weights goes through another proxy than the reads of these:
        // it may start when they are done for certain, their results stored
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(a_full(st % kSA));
          mbar_arrive(q_empty(s));
        }
      }
    }
    if (!ok && lane == 0) fail_w4(abort_flag);
  } else {
    regs_inc<kRegsEpi>();
    constexpr int kCols = BT / 2;  // columns of a warp
    const int quad = warp & 3, h = (warp - kEpiWarp) / 4;
    const int row = quad * 32 + lane;
    constexpr int kTake = BT > 128 ? 8 : 16;  // columns at a time
    int g = 0;  // chunks so far
    bool ok = true;
    for (int t = t_first; t < tiles && ok && !*abort_flag; t += t_step) {
      const int n = t % n_tiles * kBN + row, m0 = t / n_tiles * BT + h * kCols;
      const bool n_in = n < N;
      float2 total[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) total[j] = make_float2(0.0f, 0.0f);
      const int groups = n_in ? (K + GROUP - 1) / GROUP : 0;
      const int64_t s_row = (int64_t)n * ld_s;
      ChunkScales<kG> next;
      next.fetch(scales, s_mode, s_row, cb * kG, groups);
      for (int ch = cb; ch < ce && ok; ++ch, ++g) {
        const ChunkScales<kG> now = next;
        if (ch + 1 < ce) next.fetch(scales, s_mode, s_row, (ch + 1) * kG, groups);
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          // the group is complete when the stage that it ends with is, or at a barrier of its
          // own inside a stage: the products are at most kAcc groups ahead of this, so the
          // barrier's next phase is not over
          constexpr int kInner = kG > kStages ? kG - kStages : 0;  // such groups in a chunk
          const int last = (e + 1) * kStepsPerGroup - 1;           // its last product in the chunk
          uint32_t bar, parity;
          if ((last + 1) % kSteps == 0) {
            const int st = g * kStages + last / kSteps;
            bar = done(st % kDone), parity = (uint32_t)(st / kDone) & 1;
          } else {
            const int i = g * kInner + e - last / kSteps;
            bar = mid(i % kAcc), parity = (uint32_t)(i / kAcc) & 1;
          }
          if (!mbar_wait(bar, parity, kWaitLimit)) {
            ok = false;
            break;
          }
          tcgen05_fence_after();
          const int acc = (g * kG + e) % kAcc;
          const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * BT + h * kCols);
          const float sc = now.get(s_mode, e);
          const float2 s2 = make_float2(sc, sc);
          uint32_t v[2][kTake];
          tmem_take(taddr, v[0]);
          tmem_wait(v[0]);
#pragma unroll
          for (int j = 0; j < kCols / kTake; ++j) {
            if (j + 1 < kCols / kTake) tmem_take(taddr + (uint32_t)(kTake * (j + 1)), v[(j + 1) & 1]);
#pragma unroll
            for (int i = 0; i < kTake / 2; ++i)
              total[kTake / 2 * j + i] = __ffma2_rn(
                  s2, make_float2(__uint_as_float(v[j & 1][2 * i]), __uint_as_float(v[j & 1][2 * i + 1])),
                  total[kTake / 2 * j + i]);
            if (j + 1 < kCols / kTake) tmem_wait(v[(j + 1) & 1]);
          }
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(acc));
        }
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
    if (warp >= kEpiWarp && !*abort_flag) {
      // rank q finishes columns [q BT / splits, (q + 1) BT / splits): each element the
      // ranks' totals in rank order, 4 weight rows a thread
      const int n0 = t_first % n_tiles * kBN, m0 = t_first / n_tiles * BT;
      const int e = threadIdx.x - 32 * kEpiWarp, n = n0 + (e & 31) * 4;
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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
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
    if (at.numRegs * (kThreads / 128) < kRegs) return cudaErrorInvalidConfiguration;
    if (SPLIT) {
      for (int size = 2; size <= kMaxSplits; ++size) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(kThreads);
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
    // a second wave's start costs more than the smaller parts save (128 rows, weights 20480
    // x 2560, us: 160 tiles in two rounds 28, split over clusters in three waves 39)
    if (tiles > held) continue;
    const int64_t cost = (chunks + size - 1) / size + kReduceChunks;
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
  cfg.blockDim = dim3(kThreads);
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
  constexpr int kG = kChunk / GROUP;  // a chunk's scales in one load, where they are aligned
  const bool pairs = g.ld_s % kG == 0 && reinterpret_cast<uintptr_t>(g.scales) % (2 * kG) == 0;
  const int s_mode = !g.s_bf16 ? 0 : (pairs ? 2 : 1);
  return cudaLaunchKernelEx(&cfg, kern, ma, mq, g.c, g.ld_c, g.c_bf16, g.scales, g.ld_s, s_mode, g.zeros, g.ld_z,
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
  // rounds of tiles times a tile's width and fixed share (us, the weights 10240 x 2560: 192
  // rows in tiles of 192 17.8, of 128 27.3; 256 rows, two rounds of either, 31.4 and 27.5;
  // 8192 rows 331 and 415)
  auto cost = [&](int64_t bt) {
    const int64_t tiles = ((g.M + bt - 1) / bt) * ((g.N + kBN - 1) / kBN);
    return (tiles + dev.sm_count - 1) / dev.sm_count * (bt + 32);
  };
  return g.M <= 128 || cost(128) <= cost(192) ? launch_bt<128>(g, dev.sm_count, stream)
                                              : launch_bt<192>(g, dev.sm_count, stream);
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
