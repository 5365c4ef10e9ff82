// linear_w4.cu - projections with 4-bit weights and group scales, few rows:
//
//   C[m][n] = sum_g s[n][g] sum_{k in g} (q[n][k] - z[n][g]) a[m][k]  (+ R[m][n])
//
// The difference q - z, an integer of few bits, is exact in bf16 and in f32, so the
// products are exact, the sums are f32, and the scale meets the sum of a group in f32:
// no weight is rounded.  Three kernels:
//
//   one row         f32 units (one_kernel), where the weights are not many
//   up to 8 rows    warp-level products of 16 weight rows x 8 activation rows (rows_kernel)
//   more            tensor memory and tcgen05 (gemm_w4.cu)
//
// The first two read a weight row's bytes once, gemm_w4.cu once for every tile of activation
// rows.  50000 x 2560, whose bytes take 10 us of HBM: one row 31 us on the f32 units and 26 in
// products; four rows 28, with neither the weights' nor the activations' loads in the loop
// 21.  No unit is full there (issue slots 39 %, ALU pipe 41, tensor pipe 10; 20 warps an
// SM): a warp waits for its loads in half of its time, and beside them stand the scales that
// start every CTA and the last of 1.7 waves.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_math.cuh"
#include "launch.h"

namespace mamba {
namespace {

constexpr int kUnit = 128;   // k of a warp's turn: 64 bytes of a weight row
constexpr int kSpan = 8192;  // k whose scales are held at once
constexpr int kRows = 16, kCols = 8;
constexpr int kAhead = 2;    // units on their way to a warp's registers

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

// 8 activations from k on, zeros past K
__device__ __forceinline__ uint4 load_x(const __nv_bfloat16* p, int k, int K) {
  if (k >= K) return make_uint4(0, 0, 0, 0);
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

constexpr int kOneWarps = 8;
constexpr int kOneRows = 4;  // weight rows of a warp
constexpr int kOneK = 512;   // k of a warp's turn, 16 a lane

// two nibbles' bytes of w as f32, by a byte permutation each
template <uint32_t SEL0, uint32_t SEL1>
__device__ __forceinline__ float2 nibbles_f32(uint32_t w, uint32_t magic, float2 zero) {
  const float2 v = make_float2(__uint_as_float(__byte_perm(w, magic, SEL0)), __uint_as_float(__byte_perm(w, magic, SEL1)));
  return __fadd2_rn(v, zero);
}

// One activation row.  A warp takes four weight rows, lane l k = 512 i + 16 l .. of
// them (256 neighbouring bytes a row); 2^kw_shift warps of a CTA share their rows and take
// the turns i in turn.  A nibble becomes f32 by one byte permutation: its byte moved to bits
// 8 .. 15 below 0x47 (even nibbles: 2^15 + q) or 0x45 (odd nibbles, left in the byte's high
// half: 2^11 + q), less 2^15 + z or 2^11 + z, all exact.  A lane's 16 products, of one
// group, are summed and meet their scale; the lanes' totals are added by a butterfly, the
// warps' in order.  Lanes and rows outside the matrix read inside it and multiply zeros, or
// are not stored: the loop has no branches (it is bound by its instructions).
template <bool ZEROS>
__global__ void __launch_bounds__(32 * kOneWarps, 3) linear_w4_one_kernel(const LinearW4Args a, int group_shift, int kw_shift) {
  constexpr int R = kOneRows;
  __shared__ float part[kOneWarps][R];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int kw_n = 1 << kw_shift, kw = warp & (kw_n - 1), rw = warp >> kw_shift;
  const int rows_cta = (kOneWarps >> kw_shift) * R;
  const int N = (int)a.N, K = (int)a.K;
  const int n0 = blockIdx.x * rows_cta + rw * R;
  const int k_last = (K + 31) / 32 * 32 - 16, g_last = (K - 1) >> group_shift;
  const int turns = (K + kOneK - 1) / kOneK;
  grid_dependency_begin();

  // rows past N: the last one's bytes
  const int n_first = n0 < N ? n0 : N - 1;
  const int last = N - 1 - n_first < R - 1 ? N - 1 - n_first : R - 1;
  const uint8_t* qp = a.q + (int64_t)n_first * a.ld_q;
  const uint16_t* sh = static_cast<const uint16_t*>(a.scales) + (int64_t)n_first * a.ld_s;
  const uint32_t* sw = static_cast<const uint32_t*>(a.scales) + (int64_t)n_first * a.ld_s;
  const uint8_t* zp = ZEROS ? a.zeros + (int64_t)n_first * a.ld_z : nullptr;
  int64_t dq[R], ds[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    dq[r] = (r < last ? r : last) * a.ld_q;
    ds[r] = (r < last ? r : last) * a.ld_s;
  }
  uint2 w_next[R];
  uint32_t s_next[R], z_next[R];
  auto fetch = [&](int i) {
    const int k0 = i * kOneK + lane * 16;
    const int k = k0 < k_last ? k0 : k_last, g0 = k0 >> group_shift, g = g0 < g_last ? g0 : g_last;
    const uint8_t* qk = qp + (k >> 1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w_next[r] = __ldcs(reinterpret_cast<const uint2*>(qk + dq[r]));
      s_next[r] = a.s_bf16 ? (uint32_t)__ldg(sh + ds[r] + g) : __ldg(sw + ds[r] + g);
      if (ZEROS) z_next[r] = __ldg(zp + (r < last ? r : last) * a.ld_z + g);
    }
  };
  float total[R];
#pragma unroll
  for (int r = 0; r < R; ++r) total[r] = 0.0f;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.a);
  if (kw < turns) fetch(kw);
#pragma unroll 1
  for (int i = kw; i < turns; i += kw_n) {
    const int k = i * kOneK + lane * 16;
    uint4 xv[2];
    if ((i + 1) * kOneK <= K) {
      xv[0] = reinterpret_cast<const uint4*>(x + k)[0];
      xv[1] = reinterpret_cast<const uint4*>(x + k)[1];
    } else {
      xv[0] = load_x(x, k, K);
      xv[1] = load_x(x, k + 8, K);
    }
    uint2 w[R];
    float sc[R];
    uint32_t z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[r] = w_next[r];
      sc[r] = k < K ? __uint_as_float(a.s_bf16 ? s_next[r] << 16 : s_next[r]) : 0.0f;
      z[r] = ZEROS ? z_next[r] & 127u : 8u;
    }
    if (i + kw_n < turns) fetch(i + kw_n);
    float2 acc[R];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // the activations in pairs (k, k + 2), even and odd
      float2 xe[2], xo[2];
      const uint32_t u[4] = {xv[h].x, xv[h].y, xv[h].z, xv[h].w};
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        xe[p] = make_float2(__uint_as_float(u[2 * p] << 16), __uint_as_float(u[2 * p + 1] << 16));
        xo[p] = make_float2(__uint_as_float(u[2 * p] & 0xffff0000u), __uint_as_float(u[2 * p + 1] & 0xffff0000u));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float e = __uint_as_float(0xc7000000u | z[r] << 8), o = __uint_as_float(0xc5000000u | z[r] << 12);
        const float2 ze = make_float2(e, e), zo = make_float2(o, o);
        const uint32_t word = h ? w[r].y : w[r].x;
        const uint32_t even = word & 0x0f0f0f0fu, odd = word & 0xf0f0f0f0u;
        const float2 e0 = nibbles_f32<0x7404, 0x7414>(even, 0x47000000u, ze);
        const float2 e1 = nibbles_f32<0x7424, 0x7434>(even, 0x47000000u, ze);
        const float2 o0 = nibbles_f32<0x7404, 0x7414>(odd, 0x45000000u, zo);
        const float2 o1 = nibbles_f32<0x7424, 0x7434>(odd, 0x45000000u, zo);
        acc[r] = h ? __ffma2_rn(e0, xe[0], acc[r]) : __fmul2_rn(e0, xe[0]);
        acc[r] = __ffma2_rn(e1, xe[1], acc[r]);
        acc[r] = __ffma2_rn(o0, xo[0], acc[r]);
        acc[r] = __ffma2_rn(o1, xo[1], acc[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) total[r] = fmaf(sc[r], acc[r].x + acc[r].y, total[r]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v = total[r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) part[warp][r] = v;
  }
  __syncthreads();
  if (threadIdx.x < rows_cta) {
    const int row = threadIdx.x, n = blockIdx.x * rows_cta + row;
    if (n >= N) return;
    const int first = (row / R) << kw_shift;
    float v = part[first][row % R];
    for (int j = 1; j < kw_n; ++j) v += part[first + j][row % R];
    if (a.r) v += a.r[n];
    store_out(a.c, n, a.c_bf16, v);
  }
}

// as many warps to a row as it takes to give every SM 24 warps
cudaError_t launch_one(const LinearW4Args& g, int sms, cudaStream_t stream) {
  const int64_t warps = (g.N + kOneRows - 1) / kOneRows, want = 24 * (int64_t)sms, turns = (g.K + kOneK - 1) / kOneK;
  int kw_shift = 0;
  while (kw_shift < 3 && (warps << kw_shift) < want && (1 << kw_shift) < turns) ++kw_shift;
  const int rows_cta = (kOneWarps >> kw_shift) * kOneRows;
  const int shift = g.group == 32 ? 5 : (g.group == 64 ? 6 : 7);
  const dim3 grid((unsigned)((g.N + rows_cta - 1) / rows_cta)), block(32 * kOneWarps);
  return g.zeros ? launch_pdl(true, linear_w4_one_kernel<true>, grid, block, 0, stream, g, shift, kw_shift)
                 : launch_pdl(true, linear_w4_one_kernel<false>, grid, block, 0, stream, g, shift, kw_shift);
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

// 16 weight rows, 8 activation rows.  scale_pitch: floats per weight row of the
// scales held (odd: 8 rows in 8 banks), whole units of them.
//
// The k of one product have to be of one group.  With groups of 128 lane t multiplies
// word i of its own 16 bytes in product i (k = 32 t + 8 i ..); with smaller ones the four
// lanes of a row exchange words first, and product b takes word t of piece b (k = 32 b +
// 8 t ..).
template <int WARPS, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 16 ? 2 : 768 / (32 * WARPS))
    linear_w4_rows_kernel(const LinearW4Args a, const int scale_pitch) {
  constexpr int kG = kUnit / GROUP;  // groups per unit
  constexpr bool kOwn = GROUP == kUnit;
  static_assert(kSpan / kUnit / WARPS % kAhead == 0, "a span ends with the last of the registers ahead");
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane >> 2, t = lane & 3;
  const int N = (int)a.N, K = (int)a.K;
  const int n0 = blockIdx.x * kRows, rows_m = (int)a.M;
  const int rows_n = N - n0 < kRows ? N - n0 : kRows;
  const int pieces = (K + 31) / 32;  // 16 bytes of a weight row
  const int units = (K + kUnit - 1) / kUnit;
  const int groups = (K + GROUP - 1) / GROUP;
  float* part = reinterpret_cast<float*>(smem);
  float* scales = part + WARPS * kCols * kRows;
  unsigned char* zeros = reinterpret_cast<unsigned char*>(scales + kRows * scale_pitch);
  grid_dependency_begin();

  // what lies outside the matrix is read inside it: rows past the last are not stored (and
  // their scales are 0), pieces past the last meet activations of 0
  const uint8_t* q0 = a.q + (int64_t)(n0 + (g < rows_n ? g : rows_n - 1)) * a.ld_q;
  const uint8_t* q1 = a.q + (int64_t)(n0 + (g + 8 < rows_n ? g + 8 : rows_n - 1)) * a.ld_q;
  const uint32_t q_last = (uint32_t)(pieces - 1) * 16;
  uint4 ahead[kAhead][2];
  auto fetch = [&](int u, uint4 (&w)[2]) {
    const uint32_t at = (uint32_t)(u * 4 + t) * 16, off = at < q_last ? at : q_last;
    w[0] = __ldcs(reinterpret_cast<const uint4*>(q0 + off));
    w[1] = __ldcs(reinterpret_cast<const uint4*>(q1 + off));
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) fetch(warp + d * WARPS, ahead[d]);

  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.a) + (g < rows_m ? g : rows_m - 1) * a.ld_a;
  float total[4] = {0.0f, 0.0f, 0.0f, 0.0f};

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
          const uint32_t zv = ZEROS && in ? __ldg(z + gr) & 127u : 0u;
          scales[row * scale_pitch + gr] = v;
          if (ZEROS) zeros[row * scale_pitch + gr] = (unsigned char)zv;
        }
      }
      __syncthreads();
    }
    const int u_end = units < (span + kSpan) / kUnit ? units : (span + kSpan) / kUnit;
    while (u < u_end) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        if (u >= u_end) break;
        uint4 xv[4];
        const int k = u * kUnit + (kOwn ? t * 32 : t * 8);  // and 8 or 32 further for the next
        if ((u + 1) * kUnit <= K) {
#pragma unroll
          for (int i = 0; i < 4; ++i) xv[i] = *reinterpret_cast<const uint4*>(x + k + i * (kOwn ? 8 : 32));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) xv[i] = load_x(x, k + i * (kOwn ? 8 : 32), K);
        }
        // (registers that stay where they are: a move would wait for the load)
        uint32_t w0[4] = {ahead[d][0].x, ahead[d][0].y, ahead[d][0].z, ahead[d][0].w};
        uint32_t w1[4] = {ahead[d][1].x, ahead[d][1].y, ahead[d][1].z, ahead[d][1].w};
        fetch(u + kAhead * WARPS, ahead[d]);
        if (!kOwn) {
          transpose4(w0, t);
          transpose4(w1, t);
        }
        const float* sc = scales + g * scale_pitch + (u * kUnit - span) / GROUP;
        const unsigned char* zc = zeros + g * scale_pitch + (u * kUnit - span) / GROUP;
        float acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i * 32 % GROUP == 0) acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
          const int e = i * 32 / GROUP;
          const __nv_bfloat162 z0 = zero_pair(ZEROS ? zc[e] : 8u), z1 = zero_pair(ZEROS ? zc[8 * scale_pitch + e] : 8u);
          const uint32_t p0[4] = {nibble_pair<0>(w0[i], z0), nibble_pair<1>(w0[i], z0), nibble_pair<2>(w0[i], z0),
                                  nibble_pair<3>(w0[i], z0)};
          const uint32_t p1[4] = {nibble_pair<0>(w1[i], z1), nibble_pair<1>(w1[i], z1), nibble_pair<2>(w1[i], z1),
                                  nibble_pair<3>(w1[i], z1)};
          // the activations' pairs (k, k + 4)
          mma16816(acc, p0[0], p1[0], p0[1], p1[1], __byte_perm(xv[i].x, xv[i].z, 0x5410),
                   __byte_perm(xv[i].x, xv[i].z, 0x7632));
          mma16816(acc, p0[2], p1[2], p0[3], p1[3], __byte_perm(xv[i].y, xv[i].w, 0x5410),
                   __byte_perm(xv[i].y, xv[i].w, 0x7632));
          if ((i + 1) * 32 % GROUP == 0) {
            const float s0 = sc[e], s1 = sc[8 * scale_pitch + e];
            total[0] = fmaf(s0, acc[0], total[0]);
            total[1] = fmaf(s0, acc[1], total[1]);
            total[2] = fmaf(s1, acc[2], total[2]);
            total[3] = fmaf(s1, acc[3], total[3]);
          }
        }
        u += WARPS;
      }
    }
  }
  // the warps' sums, [warp][m][row]
  float* p = part + (warp * kCols + 2 * t) * kRows + g;
  p[0] = total[0];
  p[kRows] = total[1];
  p[8] = total[2];
  p[kRows + 8] = total[3];
  __syncthreads();
  for (int e = threadIdx.x; e < rows_m * kRows; e += 32 * WARPS) {
    const int n = n0 + e % kRows, m = e / kRows;
    if (n >= N) continue;
    float v = part[e];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) v += part[w * (kCols * kRows) + e];
    if (a.r) v += a.r[(int64_t)m * a.ld_r + n];
    store_out(a.c, (int64_t)m * a.ld_c + n, a.c_bf16, v);
  }
}

template <int WARPS, int GROUP>
cudaError_t launch_rows(const LinearW4Args& g, cudaStream_t stream) {
  // the groups of whole units: a unit across K reads (and ignores) those past the last
  const int64_t groups = (g.K + kUnit - 1) / kUnit * (kUnit / GROUP);
  const int scale_pitch = (int)(groups < kSpan / GROUP ? groups : kSpan / GROUP) | 1;
  static_assert(WARPS * kCols * kRows * 4 + kRows * (kSpan / GROUP + 1) * 5 <= 48 * 1024, "shared memory without opt-in");
  const int smem = WARPS * kCols * kRows * 4 + kRows * scale_pitch * (g.zeros ? 5 : 4);
  const dim3 grid((unsigned)((g.N + kRows - 1) / kRows));
  return g.zeros ? launch_pdl(true, linear_w4_rows_kernel<WARPS, GROUP, true>, grid, dim3(32 * WARPS), smem, stream, g,
                              scale_pitch)
                 : launch_pdl(true, linear_w4_rows_kernel<WARPS, GROUP, false>, grid, dim3(32 * WARPS), smem, stream, g,
                              scale_pitch);
}

template <int WARPS>
cudaError_t launch_group(const LinearW4Args& g, cudaStream_t stream) {
  if (g.group == 32) return launch_rows<WARPS, 32>(g, stream);
  if (g.group == 64) return launch_rows<WARPS, 64>(g, stream);
  return launch_rows<WARPS, 128>(g, stream);
}

}  // namespace

cudaError_t launch_linear_w4(const LinearW4Args& g, const DeviceInfo& dev, cudaStream_t stream) {
  if (g.M <= 0 || g.N <= 0) return cudaSuccess;
  // (10240 x 2560, us: 8 rows 11.4, 9 rows on the tensor memory path 13.3)
  if (g.M > kCols) return launch_gemm_w4(g, dev, stream);
  // one row: on the f32 units, but for many long weight rows in groups of 128, where a unit of
  // products takes fewer instructions (us, products against f32 units: 20480 x 2560 13.2 and
  // 15.1, 50000 x 2560 26 and 31; 10240 x 2560 9.4 and 9.2, 2560 x 5120 7.4 and 6.2; groups of
  // 32, whose words change lanes first, 50000 x 2560 43 and 36)
  const bool much = g.N / kOneRows * ((g.K + kUnit - 1) / kUnit) >= 16 * 24 * (int64_t)dev.sm_count;
  if (g.M == 1 && !(much && g.group == kUnit)) return launch_one(g, dev.sm_count, stream);
  // as many warps to 16 weight rows as make 32 for every SM (24 of them resident at once, by
  // their registers): a warp's start and end cost it what three units do (50000 x 2560, 4
  // rows, us: eight warps 36, two 33, two with 80 registers a thread instead of 64, 28, and
  // one 30; 20480 x 2560: two 14, one 25)
  const int64_t ctas = (g.N + kRows - 1) / kRows, want = 32 * (int64_t)dev.sm_count, units = (g.K + kUnit - 1) / kUnit;
  if (ctas * 2 >= want || units <= 2) return launch_group<2>(g, stream);
  if (ctas * 4 >= want || units <= 4) return launch_group<4>(g, stream);
  if (ctas * 8 >= want || units <= 8) return launch_group<8>(g, stream);
  return launch_group<16>(g, stream);
}

}  // namespace mamba
