// linear_w4.cu - projections with 4-bit weights and group scales, few rows:
//
//   C[m][n] = sum_g s[n][g] sum_{k in g} (q[n][k] - z[n][g]) a[m][k]  (+ R[m][n])
//
// One warp-level tensor product (16 weight rows x 8 activation rows) per 16 k:
// the difference q - z, an integer of at most 4 bits and a sign, is exact in
// bf16, so the products are exact, the sums are f32, and the scale meets the
// sum of a group in f32: no weight is rounded.
//
// A nibble becomes a bf16 by two operations per pair: (w >> 4 i) & 0x000f000f
// puts nibbles i and i + 4 of a word into the low bits of the halves of a
// register, 0x4300 above them makes them 128 + q, and a packed subtraction
// takes 128 + z off.  The pairs (i, i + 4) are the product's k order; the
// activations are put into the same order.
//
// Bound: the weights' way from HBM, and close behind it the integer pipe that takes
// the nibbles apart.  A CTA takes 16 or 32 weight rows; bulk copies bring 1024 k
// (512 bytes a row) at a time, several such slabs in flight, and each of its 8 warps
// takes 128 k of a slab.  The warps' sums are added in warp order at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/mamba_ssm.h"
#include "async_copy.cuh"
#include "device_math.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace mamba {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 128;                // k of a warp's turn
constexpr int kSlab = kWarps * kChunk;     // k per stage
constexpr int kPitchW = kSlab / 2 + 16;    // bytes of a weight row in a stage: 8 rows' words meet 32 banks
constexpr int kPitchX = kSlab * 2 + 64;    // and of an activation row: two rows' 64 bytes meet 32 banks
constexpr int kSpan = 8 * kSlab;           // k whose scales are held at once
constexpr int kMaxStages = 4;
constexpr int kStageBudget = 72 * 1024;    // of a CTA's stages: three CTAs per SM
constexpr long long kWaitLimit = 1ll << 31;  // SM cycles (about a second)

__device__ int g_linear_w4_faults = 0;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// nibbles I and I + 4 of w as a pair of bf16, less the pair zc = 128 + z
template <int I>
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w, __nv_bfloat162 zc) {
  const uint32_t v = ((w >> (4 * I)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), zc);
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z) {
  const uint32_t v = (0x4300u | z) * 0x00010001u;
  return *reinterpret_cast<const __nv_bfloat162*>(&v);
}

struct RowsShape {
  int stages;       // slabs in flight
  int x_rows;       // activation rows of a stage
  int scale_pitch;  // floats per weight row of the scales held (odd)
};

// MT x 16 weight rows, NT x 8 activation rows
template <int MT, int NT, int GROUP>
__global__ void __launch_bounds__(kThreads, 3)
    linear_w4_rows_kernel(const LinearW4Args a, const RowsShape sh) {
  constexpr int kRows = 16 * MT, kCols = 8 * NT;
  constexpr int kG = kChunk / GROUP;  // groups per chunk
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint64_t bar_mem[2 * kMaxStages];
  __shared__ int abort_mem;
  volatile int* abort_flag = &abort_mem;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane >> 2, t = lane & 3;
  const int N = (int)a.N, K = (int)a.K;
  const int n0 = blockIdx.x * kRows, m0 = blockIdx.y * kCols;
  const int rows_m = a.M - m0 < kCols ? (int)(a.M - m0) : kCols;
  const int rows_n = N - n0 < kRows ? N - n0 : kRows;
  const int row_bytes = (K + 31) / 32 * 16;
  const int slabs = (K + kSlab - 1) / kSlab;
  const int groups = (K + GROUP - 1) / GROUP;
  const int stage_bytes = kRows * kPitchW + sh.x_rows * kPitchX;
  const uint32_t base = smem_u32(smem);
  float* scales = reinterpret_cast<float*>(smem + sh.stages * stage_bytes);
  unsigned char* zeros = reinterpret_cast<unsigned char*>(scales + kRows * sh.scale_pitch);
  auto full = [&](int s) { return smem_u32(bar_mem) + 8 * s; };
  auto empty = [&](int s) { return smem_u32(bar_mem) + 8 * (kMaxStages + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < sh.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kWarps);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();
  grid_dependency_begin();

  const __nv_bfloat16* x0 = static_cast<const __nv_bfloat16*>(a.a) + (int64_t)m0 * a.ld_a;
  auto fail = [&]() {
    atomicOr(&g_linear_w4_faults, MAMBA_FAULT_GEMM_WAIT);
    *abort_flag = 1;
  };
  // slab i by warp 0, a row per lane: whole 16 bytes inside K; the rest of a stage
  // keeps what it held (its nibbles meet activations that are made zero)
  auto issue = [&](int i) {
    const int s = i % sh.stages, off = i * (kSlab / 2), k0 = i * kSlab;
    const int wb = row_bytes - off < kSlab / 2 ? row_bytes - off : kSlab / 2;
    const int xb = (K - k0 < kSlab ? K - k0 : kSlab) / 8 * 16;
    const uint32_t w = base + s * stage_bytes, x = w + kRows * kPitchW;
    if (lane == 0) mbar_arrive_expect_tx(full(s), rows_n * wb + rows_m * xb);
    __syncwarp();
    if (lane < rows_n) bulk_g2s(w + lane * kPitchW, a.q + (int64_t)(n0 + lane) * a.ld_q + off, wb, full(s));
    if (lane < rows_m && xb > 0) bulk_g2s(x + lane * kPitchX, x0 + (int64_t)lane * a.ld_a + k0, xb, full(s));
  };
  int issued = 0;
  if (warp == 0)
    for (; issued < sh.stages && issued < slabs; ++issued) issue(issued);

  float total[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) total[i][j][0] = total[i][j][1] = total[i][j][2] = total[i][j][3] = 0.0f;

  bool ok = true;
  for (int i = 0; i < slabs && ok; ++i) {
    if (i % (kSpan / kSlab) == 0) {
      // the scales and zero points of the next kSpan k, 0 outside the matrix
      const int g0 = i * (kSlab / GROUP), left = groups - g0;
      const int held = left < kSpan / GROUP ? left : kSpan / GROUP;
      if (i > 0) __syncthreads();
      for (int e = threadIdx.x; e < kRows * sh.scale_pitch; e += kThreads) {
        const int row = e / sh.scale_pitch, gr = e % sh.scale_pitch;
        const bool in = row < rows_n && gr < held;
        const int64_t at = (int64_t)(n0 + row) * a.ld_s + g0 + gr;
        scales[e] = !in ? 0.0f
                        : (a.s_bf16 ? to_f32(static_cast<const __nv_bfloat16*>(a.scales)[at])
                                    : static_cast<const float*>(a.scales)[at]);
        if (a.zeros) zeros[e] = in ? a.zeros[(int64_t)(n0 + row) * a.ld_z + g0 + gr] & 127 : 0;
      }
      __syncthreads();
    }
    const int s = i % sh.stages, ch = i * kWarps + warp;
    if (!mbar_wait(full(s), (i / sh.stages) & 1, kWaitLimit)) {
      ok = false;
      break;
    }
    if (ch * kChunk < K) {
      const unsigned char* w = smem + s * stage_bytes + warp * (kChunk / 2) + g * kPitchW + t * 4;
      const unsigned char* x = smem + s * stage_bytes + kRows * kPitchW + warp * (kChunk * 2) + g * kPitchX + t * 16;
      const float* sc = scales + g * sh.scale_pitch + ch % (kSpan / kChunk) * kG;
      const unsigned char* zc = zeros + g * sh.scale_pitch + ch % (kSpan / kChunk) * kG;
      const bool tail = K - ch * kChunk < kChunk;
      float acc[MT][NT][4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b * 32 % GROUP == 0) {
#pragma unroll
          for (int mi = 0; mi < MT; ++mi)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[mi][j][0] = acc[mi][j][1] = acc[mi][j][2] = acc[mi][j][3] = 0.0f;
        }
        uint32_t xp[NT][4];  // the activations' pairs (k, k + 4)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint4 v = make_uint4(0, 0, 0, 0);
          const int m = j * 8 + g, k = ch * kChunk + b * 32 + t * 8;
          if (m < rows_m) {
            if (!tail || k + 8 <= K) {
              v = *reinterpret_cast<const uint4*>(x + j * 8 * kPitchX + b * 64);
            } else if (k < K) {  // a piece across K, from where it lies
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                h[e] = k + e < K ? reinterpret_cast<const uint16_t*>(x0)[(int64_t)m * a.ld_a + k + e] : 0u;
              v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
            }
          }
          xp[j][0] = __byte_perm(v.x, v.z, 0x5410);
          xp[j][1] = __byte_perm(v.x, v.z, 0x7632);
          xp[j][2] = __byte_perm(v.y, v.w, 0x5410);
          xp[j][3] = __byte_perm(v.y, v.w, 0x7632);
        }
        const int e = b * 32 / GROUP;
#pragma unroll
        for (int mi = 0; mi < MT; ++mi) {
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(w + (mi * 16) * kPitchW + b * 16);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(w + (mi * 16 + 8) * kPitchW + b * 16);
          const __nv_bfloat162 z0 = zero_pair(a.zeros ? zc[(mi * 16) * sh.scale_pitch + e] : 8u);
          const __nv_bfloat162 z1 = zero_pair(a.zeros ? zc[(mi * 16 + 8) * sh.scale_pitch + e] : 8u);
          const uint32_t p0[4] = {nibble_pair<0>(w0, z0), nibble_pair<1>(w0, z0), nibble_pair<2>(w0, z0),
                                  nibble_pair<3>(w0, z0)};
          const uint32_t p1[4] = {nibble_pair<0>(w1, z1), nibble_pair<1>(w1, z1), nibble_pair<2>(w1, z1),
                                  nibble_pair<3>(w1, z1)};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma16816(acc[mi][j], p0[0], p1[0], p0[1], p1[1], xp[j][0], xp[j][1]);
            mma16816(acc[mi][j], p0[2], p1[2], p0[3], p1[3], xp[j][2], xp[j][3]);
          }
          if ((b + 1) * 32 % GROUP == 0) {
            const float s0 = sc[(mi * 16) * sh.scale_pitch + e], s1 = sc[(mi * 16 + 8) * sh.scale_pitch + e];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              total[mi][j][0] = fmaf(s0, acc[mi][j][0], total[mi][j][0]);
              total[mi][j][1] = fmaf(s0, acc[mi][j][1], total[mi][j][1]);
              total[mi][j][2] = fmaf(s1, acc[mi][j][2], total[mi][j][2]);
              total[mi][j][3] = fmaf(s1, acc[mi][j][3], total[mi][j][3]);
            }
          }
        }
      }
    }
    if (i + sh.stages < slabs) {
      fence_proxy_async_smem();  // this warp's reads of the stage, before the next copy into it
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
      if (warp == 0) {  // the stage again, once every warp has read it
        if (!mbar_wait(empty(s), (i / sh.stages) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        issue(issued++);
      }
    }
  }
  if (!ok && lane == 0) fail();
  if (warp == 0)  // every copy has landed
    for (int i = issued > sh.stages ? issued - sh.stages : 0; i < issued; ++i)
      if (!mbar_wait(full(i % sh.stages), (i / sh.stages) & 1, kWaitLimit)) fail();
  __syncthreads();
  if (*abort_flag) return;
  // the warps' sums, [warp][m][row]
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int mi = 0; mi < MT; ++mi)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* p = part + (warp * kCols + j * 8 + 2 * t) * kRows + mi * 16 + g;
      p[0] = total[mi][j][0];
      p[kRows] = total[mi][j][1];
      p[8] = total[mi][j][2];
      p[kRows + 8] = total[mi][j][3];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < rows_m * kRows; e += kThreads) {
    const int n = n0 + e % kRows, m = m0 + e / kRows;
    if (n >= N) continue;
    float v = part[e];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += part[w * (kCols * kRows) + e];
    if (a.r) v += a.r[(int64_t)m * a.ld_r + n];
    store_out(a.c, (int64_t)m * a.ld_c + n, a.c_bf16, v);
  }
}

template <int MT, int NT, int GROUP>
cudaError_t launch_rows(const LinearW4Args& g, cudaStream_t stream) {
  auto kern = linear_w4_rows_kernel<MT, NT, GROUP>;
  constexpr int kRows = 16 * MT, kCols = 8 * NT;
  RowsShape sh;
  sh.x_rows = (int)(g.M < kCols ? g.M : kCols);
  const int stage = kRows * kPitchW + sh.x_rows * kPitchX;
  const int64_t slabs = (g.K + kSlab - 1) / kSlab;
  sh.stages = kStageBudget / stage;
  sh.stages = sh.stages < 2 ? 2 : (sh.stages > kMaxStages ? kMaxStages : sh.stages);
  if (sh.stages > slabs) sh.stages = (int)slabs;
  // the groups of whole chunks: a chunk across K reads (and ignores) those past the last
  const int64_t groups = (g.K + kChunk - 1) / kChunk * (kChunk / GROUP);
  sh.scale_pitch = (int)(groups < kSpan / GROUP ? groups : kSpan / GROUP) | 1;
  int smem = sh.stages * stage + kRows * sh.scale_pitch * (g.zeros ? 5 : 4);
  const int parts = kWarps * kCols * kRows * 4;  // the warps' sums, over the stages
  if (smem < parts) smem = parts;
  constexpr int kMost = 2 * (kRows * kPitchW + kCols * kPitchX) > kStageBudget ? 2 * (kRows * kPitchW + kCols * kPitchX)
                                                                               : kStageBudget;
  static_assert(kMost + kRows * (kSpan / GROUP + 1) * 5 + 1024 <= 232448, "shared memory over the opt-in limit");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMost + kRows * (kSpan / GROUP + 1) * 5);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((g.N + kRows - 1) / kRows), (unsigned)((g.M + kCols - 1) / kCols));
  return launch_pdl(true, kern, grid, dim3(kThreads), smem, stream, g, sh);
}

template <int MT, int NT>
cudaError_t launch_group(const LinearW4Args& g, cudaStream_t stream) {
  if (g.group == 32) return launch_rows<MT, NT, 32>(g, stream);
  if (g.group == 64) return launch_rows<MT, NT, 64>(g, stream);
  return launch_rows<MT, NT, 128>(g, stream);
}

}  // namespace

cudaError_t launch_linear_w4(const LinearW4Args& g, const DeviceInfo& dev, cudaStream_t stream) {
  if (g.M <= 0 || g.N <= 0) return cudaSuccess;
  if (g.M > 16) return launch_gemm_w4(g, dev, stream);
  const bool wide = g.N >= 64 * (int64_t)dev.sm_count;  // 32 rows a CTA, two CTAs per SM and more
  if (g.M > 8) return wide ? launch_group<2, 2>(g, stream) : launch_group<1, 2>(g, stream);
  return wide ? launch_group<2, 1>(g, stream) : launch_group<1, 1>(g, stream);
}

int read_linear_w4_faults(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_linear_w4_faults, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_linear_w4_faults, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace mamba
