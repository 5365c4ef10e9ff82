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
// Bound: the weights' way from HBM, and the warp-level product, which takes 32 cycles
// of a quarter of an SM (50000 x 2560: 11.7 us to read, 13.8 to multiply).  A CTA takes 16
// weight rows and its warps the rows' units of 128 k in turn.  Lane (g, t) reads 16 bytes
// of rows g and g + 8, straight into registers and some units ahead (tensor copies of 16
// x 64 bytes into shared memory took 33 us for those weights, bulk copies of 512 bytes
// 40).  Activations come from the L1 cache.  The warps' sums are added in warp order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_math.cuh"
#include "launch.h"

namespace mamba {
namespace {

constexpr int kUnit = 128;   // k of a warp's turn: 64 bytes of a weight row
constexpr int kSpan = 8192;  // k whose scales are held at once
constexpr int kRows = 16;

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

// 8 activations from k on, zeros past K (and past the rows: p null)
__device__ __forceinline__ uint4 load_x(const __nv_bfloat16* p, int k, int K) {
  if (!p || k >= K) return make_uint4(0, 0, 0, 0);
  if (k + 8 <= K) return *reinterpret_cast<const uint4*>(p + k);
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int j = 0; k + j < K; ++j) {
    const uint64_t v = reinterpret_cast<const uint16_t*>(p)[k + j];
    if (j < 4) lo |= v << (16 * j);
    else hi |= v << (16 * (j - 4));
  }
  return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}

// word t of the four lanes' w[0 .. 3] in the place of this lane's words: w[b] becomes
// word t of lane b's
__device__ __forceinline__ void transpose4(uint32_t (&w)[4], int t) {
  const bool odd = t & 1, high = t & 2;
  uint32_t s0 = odd ? w[0] : w[1], s1 = odd ? w[2] : w[3];
  s0 = __shfl_xor_sync(0xffffffffu, s0, 1);
  s1 = __shfl_xor_sync(0xffffffffu, s1, 1);
  if (odd) w[0] = s0, w[2] = s1;
  else w[1] = s0, w[3] = s1;
  s0 = high ? w[0] : w[2], s1 = high ? w[1] : w[3];
  s0 = __shfl_xor_sync(0xffffffffu, s0, 2);
  s1 = __shfl_xor_sync(0xffffffffu, s1, 2);
  if (high) w[0] = s0, w[1] = s1;
  else w[2] = s0, w[3] = s1;
}

// 16 weight rows, NT x 8 activation rows.  scale_pitch: floats per weight row of the
// scales held (odd: 8 rows in 8 banks), whole units of them.
//
// The k of one product have to be of one group.  With groups of 128 lane t multiplies
// word i of its own 16 bytes in product i (k = 32 t + 8 i ..); with smaller ones the four
// lanes of a row exchange words first, and product b takes word t of piece b (k = 32 b +
// 8 t ..).
template <int WARPS, int NT, int GROUP, int AHEAD>
__global__ void __launch_bounds__(32 * WARPS, NT == 1 ? 1024 / (32 * WARPS) : 768 / (32 * WARPS))
    linear_w4_rows_kernel(const LinearW4Args a, const int scale_pitch) {
  constexpr int kCols = 8 * NT;
  constexpr int kG = kUnit / GROUP;  // groups per unit
  constexpr bool kOwn = GROUP == kUnit;
  static_assert(kSpan / kUnit / WARPS % AHEAD == 0, "a span ends with the last of the registers ahead");
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane >> 2, t = lane & 3;
  const int N = (int)a.N, K = (int)a.K;
  const int n0 = blockIdx.x * kRows, m0 = blockIdx.y * kCols;
  const int rows_m = a.M - m0 < kCols ? (int)(a.M - m0) : kCols;
  const int rows_n = N - n0 < kRows ? N - n0 : kRows;
  const int pieces = (K + 31) / 32;  // 16 bytes of a weight row
  const int units = (K + kUnit - 1) / kUnit;
  const int groups = (K + GROUP - 1) / GROUP;
  float* part = reinterpret_cast<float*>(smem);
  float* scales = part + WARPS * kCols * kRows;
  unsigned char* zeros = reinterpret_cast<unsigned char*>(scales + kRows * scale_pitch);
  grid_dependency_begin();

  const uint8_t* q0 = g < rows_n ? a.q + (int64_t)(n0 + g) * a.ld_q + t * 16 : nullptr;
  const uint8_t* q1 = g + 8 < rows_n ? a.q + (int64_t)(n0 + g + 8) * a.ld_q + t * 16 : nullptr;
  uint4 ahead[AHEAD][2];
  auto fetch = [&](int u, uint4 (&w)[2]) {
    w[0] = w[1] = make_uint4(0, 0, 0, 0);
    if (u * 4 + t < pieces) {
      if (q0) w[0] = __ldcs(reinterpret_cast<const uint4*>(q0 + (int64_t)u * 64));
      if (q1) w[1] = __ldcs(reinterpret_cast<const uint4*>(q1 + (int64_t)u * 64));
    }
  };
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) fetch(warp + d * WARPS, ahead[d]);

  const __nv_bfloat16* xr[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    xr[j] = j * 8 + g < rows_m ? static_cast<const __nv_bfloat16*>(a.a) + (int64_t)(m0 + j * 8 + g) * a.ld_a : nullptr;

  float total[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) total[j][0] = total[j][1] = total[j][2] = total[j][3] = 0.0f;

  int u = warp;
  for (int span = 0; span < K; span += kSpan) {
    {
      // the scales and zero points of the next kSpan k, 0 outside the matrix
      const int g0 = span / GROUP, left = groups - g0;
      const int held = left < kSpan / GROUP ? left : kSpan / GROUP;
      if (span > 0) __syncthreads();
#pragma unroll
      for (int row = warp; row < kRows; row += WARPS) {
        const int n = n0 + row;
        const float* sf = static_cast<const float*>(a.scales) + (int64_t)n * a.ld_s + g0;
        const __nv_bfloat16* sb = static_cast<const __nv_bfloat16*>(a.scales) + (int64_t)n * a.ld_s + g0;
        const uint8_t* z = a.zeros + (int64_t)n * a.ld_z + g0;
        for (int gr = lane; gr < scale_pitch; gr += 32) {
          const bool in = row < rows_n && gr < held;
          const float v = !in ? 0.0f : (a.s_bf16 ? to_f32(__ldg(sb + gr)) : __ldg(sf + gr));
          const uint32_t zv = a.zeros && in ? __ldg(z + gr) & 127u : 0u;
          scales[row * scale_pitch + gr] = v;
          if (a.zeros) zeros[row * scale_pitch + gr] = (unsigned char)zv;
        }
      }
      __syncthreads();
    }
    const int u_end = units < (span + kSpan) / kUnit ? units : (span + kSpan) / kUnit;
    while (u < u_end) {
#pragma unroll
      for (int d = 0; d < AHEAD; ++d) {
        if (u >= u_end) break;
        uint4 xv[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            xv[j][i] = load_x(xr[j], u * kUnit + (kOwn ? t * 32 + i * 8 : i * 32 + t * 8), K);
        // (registers that stay where they are: a move would wait for the load)
        uint32_t w0[4] = {ahead[d][0].x, ahead[d][0].y, ahead[d][0].z, ahead[d][0].w};
        uint32_t w1[4] = {ahead[d][1].x, ahead[d][1].y, ahead[d][1].z, ahead[d][1].w};
        fetch(u + AHEAD * WARPS, ahead[d]);
        if (!kOwn) {
          transpose4(w0, t);
          transpose4(w1, t);
        }
        const float* sc = scales + g * scale_pitch + (u * kUnit - span) / GROUP;
        const unsigned char* zc = zeros + g * scale_pitch + (u * kUnit - span) / GROUP;
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i * 32 % GROUP == 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
          }
          const int e = i * 32 / GROUP;
          const __nv_bfloat162 z0 = zero_pair(a.zeros ? zc[e] : 8u);
          const __nv_bfloat162 z1 = zero_pair(a.zeros ? zc[8 * scale_pitch + e] : 8u);
          const uint32_t p0[4] = {nibble_pair<0>(w0[i], z0), nibble_pair<1>(w0[i], z0), nibble_pair<2>(w0[i], z0),
                                  nibble_pair<3>(w0[i], z0)};
          const uint32_t p1[4] = {nibble_pair<0>(w1[i], z1), nibble_pair<1>(w1[i], z1), nibble_pair<2>(w1[i], z1),
                                  nibble_pair<3>(w1[i], z1)};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            // the activations' pairs (k, k + 4)
            mma16816(acc[j], p0[0], p1[0], p0[1], p1[1], __byte_perm(xv[j][i].x, xv[j][i].z, 0x5410),
                     __byte_perm(xv[j][i].x, xv[j][i].z, 0x7632));
            mma16816(acc[j], p0[2], p1[2], p0[3], p1[3], __byte_perm(xv[j][i].y, xv[j][i].w, 0x5410),
                     __byte_perm(xv[j][i].y, xv[j][i].w, 0x7632));
          }
          if ((i + 1) * 32 % GROUP == 0) {
            const float s0 = sc[e], s1 = sc[8 * scale_pitch + e];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              total[j][0] = fmaf(s0, acc[j][0], total[j][0]);
              total[j][1] = fmaf(s0, acc[j][1], total[j][1]);
              total[j][2] = fmaf(s1, acc[j][2], total[j][2]);
              total[j][3] = fmaf(s1, acc[j][3], total[j][3]);
            }
          }
        }
        u += WARPS;
      }
    }
  }
  // the warps' sums, [warp][m][row]
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float* p = part + (warp * kCols + j * 8 + 2 * t) * kRows + g;
    p[0] = total[j][0];
    p[kRows] = total[j][1];
    p[8] = total[j][2];
    p[kRows + 8] = total[j][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows_m * kRows; e += 32 * WARPS) {
    const int n = n0 + e % kRows, m = m0 + e / kRows;
    if (n >= N) continue;
    float v = part[e];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) v += part[w * (kCols * kRows) + e];
    if (a.r) v += a.r[(int64_t)m * a.ld_r + n];
    store_out(a.c, (int64_t)m * a.ld_c + n, a.c_bf16, v);
  }
}

template <int WARPS, int NT, int GROUP, int AHEAD>
cudaError_t launch_rows(const LinearW4Args& g, cudaStream_t stream) {
  constexpr int kCols = 8 * NT;
  // the groups of whole units: a unit across K reads (and ignores) those past the last
  const int64_t groups = (g.K + kUnit - 1) / kUnit * (kUnit / GROUP);
  const int scale_pitch = (int)(groups < kSpan / GROUP ? groups : kSpan / GROUP) | 1;
  static_assert(WARPS * kCols * kRows * 4 + kRows * (kSpan / GROUP + 1) * 5 <= 48 * 1024, "static limit of shared memory");
  const int smem = WARPS * kCols * kRows * 4 + kRows * scale_pitch * (g.zeros ? 5 : 4);
  const dim3 grid((unsigned)((g.N + kRows - 1) / kRows), (unsigned)((g.M + kCols - 1) / kCols));
  return launch_pdl(true, linear_w4_rows_kernel<WARPS, NT, GROUP, AHEAD>, grid, dim3(32 * WARPS), smem, stream, g,
                    scale_pitch);
}

template <int WARPS, int NT, int AHEAD>
cudaError_t launch_group(const LinearW4Args& g, cudaStream_t stream) {
  if (g.group == 32) return launch_rows<WARPS, NT, 32, AHEAD>(g, stream);
  if (g.group == 64) return launch_rows<WARPS, NT, 64, AHEAD>(g, stream);
  return launch_rows<WARPS, NT, 128, AHEAD>(g, stream);
}

}  // namespace

cudaError_t launch_linear_w4(const LinearW4Args& g, const DeviceInfo& dev, cudaStream_t stream) {
  if (g.M <= 0 || g.N <= 0) return cudaSuccess;
  if (g.M > 16) return launch_gemm_w4(g, dev, stream);
  // two CTAs per SM or fewer: more warps to a row, so that all of it is on its way at once
  const bool few = (g.N + kRows - 1) / kRows <= 2 * (int64_t)dev.sm_count && g.K > 8 * kUnit;
  if (g.M > 8) return few ? launch_group<16, 2, 2>(g, stream) : launch_group<8, 2, 2>(g, stream);
  return few ? launch_group<16, 1, 2>(g, stream) : launch_group<8, 1, 2>(g, stream);
}

}  // namespace mamba
