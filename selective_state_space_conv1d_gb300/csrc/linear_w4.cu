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
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_math.cuh"
#include "async_copy.cuh"
#include "launch.h"

namespace mamba {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 128;  // k per step of a warp: 64 bytes of a row
constexpr int kStages = 4;   // chunks in flight per warp

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// A CTA takes 16 MT weight rows; its warps take the row's chunks of 128 k in
// turn (warp w chunks w, w + 8, ...: the CTA reads 512 neighbouring bytes of a
// row), each through a ring of kStages chunks of its own, and their sums are
// added in warp order at the end.
template <int MT, int GROUP, bool S_BF16, bool ZEROS>
__global__ void __launch_bounds__(kThreads)
    linear_w4_rows_kernel(void* __restrict__ c, int64_t ld_c, int c_bf16, const __nv_bfloat16* __restrict__ a,
                          int64_t ld_a, const uint8_t* __restrict__ q, int64_t ld_q, const void* __restrict__ scales,
                          int64_t ld_s, const uint8_t* __restrict__ zeros, int64_t ld_z, const float* r, int64_t ld_r,
                          int M, int N, int K) {
  constexpr int kRows = 16 * MT;
  constexpr int kStageW = kRows * 64;         // bytes of weights
  constexpr int kStageA = 8 * kChunk * 2;     // bytes of activations
  constexpr int kStage = kStageW + kStageA;
  constexpr int kG = kChunk / GROUP;          // groups per chunk
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows, m0 = blockIdx.y * 8;
  const int rows_m = M - m0 < 8 ? M - m0 : 8;
  const int blocks = (K + 31) / 32;           // 16-byte pieces of a row
  const int chunks = (K + kChunk - 1) / kChunk;
  const int groups = (K + GROUP - 1) / GROUP;
  unsigned char* ring = smem + warp * (kStages * kStage);
  const uint32_t ring_u = smem_u32(ring);
  grid_dependency_begin();

  // chunk `ch` into stage s: weight row i's piece b at granule b ^ (i / 2 % 4) of
  // its 64 bytes; the activations of row i at 256 i, piece p at p ^ i
  auto load = [&](int ch, int s) {
    if (ch < chunks) {
      const uint32_t w = ring_u + s * kStage, x = w + kStageW;
#pragma unroll
      for (int j = 0; j < kRows / 8; ++j) {
        const int row = j * 8 + g, b = ch * 4 + t, n = n0 + row;
        const bool in = n < N && b < blocks;
        cp_async16(w + row * 64 + ((t ^ ((row >> 1) & 3)) << 4), q + (in ? (int64_t)n * ld_q + b * 16 : 0), in);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = j * 32 + lane, row = p >> 4, piece = p & 15, k = ch * kChunk + piece * 8;
        if (row < rows_m) {
          const uint32_t dst = x + row * 256 + ((piece ^ row) << 4);
          // a piece across K ends in zeros: whole elements only
          const int bytes = K - k >= 8 ? 16 : (K > k ? (K - k) * 2 : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                       "l"(a + (bytes ? (int64_t)(m0 + row) * ld_a + k : 0)), "r"(bytes)
                       : "memory");
        }
      }
    }
    cp_async_commit();
  };

  float total[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i) total[i][0] = total[i][1] = total[i][2] = total[i][3] = 0.0f;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(warp + s * kWarps, s);

  int s = 0;
  for (int ch = warp; ch < chunks; ch += kWarps) {
    // this chunk's scales and zero points: rows g and g + 8 of each 16
    float sc[MT][2][kG];
    uint32_t zp[MT][2][kG];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          const int n = n0 + i * 16 + h * 8 + g, gr = ch * kG + e;
          const bool in = n < N && gr < groups;
          sc[i][h][e] = !in ? 0.0f
                            : (S_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(scales)[(int64_t)n * ld_s + gr])
                                      : static_cast<const float*>(scales)[(int64_t)n * ld_s + gr]);
          if (ZEROS) zp[i][h][e] = in ? zeros[(int64_t)n * ld_z + gr] & 127u : 0u;
        }
    load(ch + (kStages - 1) * kWarps, s == 0 ? kStages - 1 : s - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const unsigned char* w = ring + s * kStage;
    const unsigned char* x = w + kStageW;
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint4 xv = make_uint4(0, 0, 0, 0);
      if (g < rows_m) xv = *reinterpret_cast<const uint4*>(x + g * 256 + (((b * 4 + t) ^ g) << 4));
      const uint32_t x04 = __byte_perm(xv.x, xv.z, 0x5410), x15 = __byte_perm(xv.x, xv.z, 0x7632);
      const uint32_t x26 = __byte_perm(xv.y, xv.w, 0x5410), x37 = __byte_perm(xv.y, xv.w, 0x7632);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int r0 = i * 16 + g, off = ((b ^ ((g >> 1) & 3)) << 4) + t * 4;
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(w + r0 * 64 + off);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(w + (r0 + 8) * 64 + off);
        const int e = b * 32 / GROUP;
        const __nv_bfloat162 z0 = zero_pair(ZEROS ? zp[i][0][e] : 8u), z1 = zero_pair(ZEROS ? zp[i][1][e] : 8u);
        mma16816(acc[i], nibble_pair<0>(w0, z0), nibble_pair<0>(w1, z1), nibble_pair<1>(w0, z0),
                 nibble_pair<1>(w1, z1), x04, x15);
        mma16816(acc[i], nibble_pair<2>(w0, z0), nibble_pair<2>(w1, z1), nibble_pair<3>(w0, z0),
                 nibble_pair<3>(w1, z1), x26, x37);
        if ((b + 1) * 32 % GROUP == 0) {
          total[i][0] = fmaf(sc[i][0][e], acc[i][0], total[i][0]);
          total[i][1] = fmaf(sc[i][0][e], acc[i][1], total[i][1]);
          total[i][2] = fmaf(sc[i][1][e], acc[i][2], total[i][2]);
          total[i][3] = fmaf(sc[i][1][e], acc[i][3], total[i][3]);
          acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        }
      }
    }
    __syncwarp();
    s = s == kStages - 1 ? 0 : s + 1;
  }
  cp_async_wait<0>();
  __syncthreads();
  // the warps' sums, [warp][m][row]
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    float* p = part + warp * (8 * kRows) + i * 16 + g;
    p[2 * t * kRows] = total[i][0];
    p[(2 * t + 1) * kRows] = total[i][1];
    p[2 * t * kRows + 8] = total[i][2];
    p[(2 * t + 1) * kRows + 8] = total[i][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows_m * kRows; e += kThreads) {
    const int n = n0 + e % kRows, m = m0 + e / kRows;
    if (n >= N) continue;
    float v = part[e];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += part[w * (8 * kRows) + e];
    if (r) v += r[(int64_t)m * ld_r + n];
    store_out(c, (int64_t)m * ld_c + n, c_bf16, v);
  }
}

template <int MT, int GROUP, bool S_BF16, bool ZEROS>
cudaError_t launch_rows(const LinearW4Args& g, cudaStream_t stream) {
  constexpr int smem = kWarps * kStages * (16 * MT * 64 + 8 * kChunk * 2);
  static_assert(smem >= kWarps * 8 * 16 * MT * 4, "the warps' sums must fit in the rings");
  auto kern = linear_w4_rows_kernel<MT, GROUP, S_BF16, ZEROS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((g.N + 16 * MT - 1) / (16 * MT)), (unsigned)((g.M + 7) / 8));
  return launch_pdl(true, kern, grid, dim3(kThreads), smem, stream, g.c, g.ld_c, g.c_bf16,
                    static_cast<const __nv_bfloat16*>(g.a), g.ld_a, g.q, g.ld_q, g.scales, g.ld_s, g.zeros, g.ld_z,
                    g.r, g.ld_r, (int)g.M, (int)g.N, (int)g.K);
}

template <int GROUP>
cudaError_t launch_group(const LinearW4Args& g, cudaStream_t stream) {
  if (g.s_bf16) return g.zeros ? launch_rows<1, GROUP, true, true>(g, stream) : launch_rows<1, GROUP, true, false>(g, stream);
  return g.zeros ? launch_rows<1, GROUP, false, true>(g, stream) : launch_rows<1, GROUP, false, false>(g, stream);
}

}  // namespace

cudaError_t launch_linear_w4(const LinearW4Args& g, const DeviceInfo& dev, cudaStream_t stream) {
  if (g.M <= 0 || g.N <= 0) return cudaSuccess;
  if (g.M > 8) return launch_gemm_w4(g, dev, stream);
  if (g.group == 32) return launch_group<32>(g, stream);
  if (g.group == 64) return launch_group<64>(g, stream);
  return launch_group<128>(g, stream);
}

}  // namespace mamba
