// token_logprobs.cu - what a row of logits l [V] says about tokens:
//
//   log p(t) = l_t - m - ln S1,   H = ln S1 - S2 / S1,
//   m = max l,  S1 = sum e^d,  S2 = sum d e^d,  d = l - m
//
// and the likeliest tokens with their log p, by value and then by index.
//
// Bound: HBM, one pass over the logits.  A row is cut over the CTAs of a cluster
// (one CTA if there are rows enough), a CTA's slice over its threads in vectors of
// 16 bytes, in turn: a slice's vector i to thread i % 256.  A thread keeps a running maximum (with
// the first vector that holds it) and the two sums below it, in units of log2: e^d is
// 2^(l L - r) with L = log2 e and r = L max l rounded once, one multiply-add and one
// exponential an element.  (Rounding r moves every term alike, and the same r is in the
// logarithm's other side.)  Elements below -2^100, -inf among them, are taken as -2^100, so
// that no product is 0 times infinity; a row whose maximum is 2^24 from 0 or further gets
// its sums again, from differences l - m.
//
// Alternatives cost no second pass: an element of the row's first n is at least as
// large as the n-th largest thread maximum, so it lies in the subset of a thread
// whose maximum reaches that bound, and only those subsets (n of 256, rarely
// more) are read again, out of the caches.  (128 rows of 128000 bf16: 11 us without
// alternatives, 16.6 with 20; 8192 rows of 50000 with one token each: 137 us, 6.0 TB/s;
// 2048 such rows keep 60 % of the issue slots busy, with the warps' longest wait the one for
// loads.)  Elements are compared as 64-bit keys,
// value above inverted index, so all keys differ and ties go to the lowest index.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/mamba_ssm.h"
#include "device_math.cuh"
#include "launch.h"

namespace mamba {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = MAMBA_MAX_TOP;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 2048;
constexpr float kLowest = -3.402823466e38f;
constexpr float kLeast = -0x1p100f;  // its product with log2 e is exact
constexpr float kNear = 0x1p24f;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// order of the values as unsigned integers: NaN above all, -0 equal to 0
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  if (o == 0xffffffffu) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
  return (uint64_t)order_of(v) << 32 | (uint32_t)~index;
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// A row from the 16-byte granule of its first element on: vector v holds the
// elements VEC v - skew ... of the row.
template <typename T>
struct Row {
  static constexpr int VEC = 16 / sizeof(T);
  static constexpr uint32_t kNothing = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
  const T* base;  // 16-byte aligned
  int skew, V;
  int full_lo, full_hi;  // the vectors that lie inside the row
  __device__ Row(const void* p, int64_t v) {
    const uintptr_t u = reinterpret_cast<uintptr_t>(p);
    base = reinterpret_cast<const T*>(u & ~(uintptr_t)15);
    skew = (int)((u & 15) / sizeof(T));
    V = (int)v;
    full_lo = skew ? 1 : 0;
    full_hi = (int)(((int64_t)skew + V) / VEC);
  }
  __device__ int vectors() const { return (int)(((int64_t)skew + V + VEC - 1) / VEC); }
  // the words of vector v, -inf outside the row (whose memory is not read)
  __device__ uint4 load(int v) const {
    if (v >= full_lo && v < full_hi) return reinterpret_cast<const uint4*>(base)[v];
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        const uint32_t lo = inside(element(v, 2 * i)) ? bits(v, 2 * i) : 0xff80u;
        const uint32_t hi = inside(element(v, 2 * i + 1)) ? bits(v, 2 * i + 1) : 0xff80u;
        w[i] = lo | hi << 16;
      } else {
        w[i] = inside(element(v, i)) ? bits(v, i) : 0xff800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ uint32_t bits(int v, int j) const {
    const int64_t at = (int64_t)v * VEC + j;
    if constexpr (sizeof(T) == 2) return reinterpret_cast<const uint16_t*>(base)[at];
    else return reinterpret_cast<const uint32_t*>(base)[at];
  }
  __device__ int64_t element(int v, int j) const { return (int64_t)v * VEC - skew + j; }
  __device__ bool inside(int64_t e) const { return e >= 0 && e < V; }
  static __device__ void unpack(const uint4& u, float (&x)[VEC]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
  // the largest value (NaN if there is one), and the values, none below kLeast
  static __device__ float largest(const uint4& u) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
      return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
      return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                     max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
  }
  static __device__ void bounded(const uint4& u, float (&x)[VEC]) {
    if constexpr (sizeof(T) == 2) {
      constexpr uint32_t kLow = 0xf180f180u;  // kLeast in bf16, twice
      unpack(make_uint4(max2(u.x, kLow), max2(u.y, kLow), max2(u.z, kLow), max2(u.w, kLow)), x);
    } else {
      unpack(u, x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = max_nan(x[i], kLeast);
    }
  }
  static __device__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

// Running maximum m and sums of one thread; ref is L times the largest bounded value, s1
// and s2 the sums of 2^d and d 2^d, d = l L - ref.
struct Stats {
  float m, ref, s1, s2;
};

__device__ __forceinline__ void rescale(Stats& s, float ref) {
  const float d = s.ref - ref;  // <= 0; NaN with a NaN, and so are the sums then
  const float c = ex2_approx(d);
  s.s2 = c == 0.0f ? 0.0f : c * fmaf(d, s.s1, s.s2);  // (sums below a far reference may be infinite)
  s.s1 = c == 0.0f ? 0.0f : s.s1 * c;
  s.ref = ref;
}

template <int VEC>
__device__ __forceinline__ void add_terms(Stats& s, const float (&x)[VEC]) {
  const float2 l2 = make_float2(kLog2e, kLog2e), r2 = make_float2(-s.ref, -s.ref);
  float2 a1 = make_float2(0.0f, 0.0f), a2 = a1;
#pragma unroll
  for (int j = 0; j < VEC; j += 2) {
    const float2 d = __ffma2_rn(make_float2(x[j], x[j + 1]), l2, r2);
    const float2 e = make_float2(ex2_approx(d.x), ex2_approx(d.y));
    a1 = __fadd2_rn(a1, e);
    a2 = __ffma2_rn(e, d, a2);
  }
  s.s1 += a1.x + a1.y;
  s.s2 += a2.x + a2.y;
}

struct SharedState {
  uint64_t keys[kCandidates];
  uint64_t top[kMaxTop];                  // this CTA's first n, in order
  uint64_t all[kMaxCluster * kMaxTop];    // the cluster's
  uint64_t bound[kWarps];
  int subset[kThreads];
  float stat[kWarps][4];
  float mine[4];                          // this CTA's maximum, reference, sums
  int n_subset, n_keys;
  uint64_t reach;                         // a bound that n of this CTA's elements reach
};

// BLOCKS: CTAs an SM holds, and with them a thread's registers and its reads ahead
template <typename T, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS) token_logprobs_kernel(const TokenLogprobsArgs a, int cluster) {
  constexpr int kAhead = BLOCKS > 2 ? 4 : 6;
  using R = Row<T>;
  constexpr int VEC = R::VEC;
  __shared__ SharedState sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t row = blockIdx.x / cluster;
  const int rank = (int)(blockIdx.x % cluster);
  grid_dependency_begin();
  const R r(static_cast<const T*>(a.logits) + row * a.ld, a.V);
  const int nv = r.vectors();
  const int v_lo = (int)((int64_t)nv * rank / cluster), v_hi = (int)((int64_t)nv * (rank + 1) / cluster);

  Stats st{-INFINITY, kLeast * kLog2e, 0.0f, 0.0f};
  int first = -1;  // the first vector that holds m
  auto take = [&](const uint4& u0, const uint4& u1, int v) {
    const float m0 = R::largest(u0), m1 = R::largest(u1);
    // NaN stands above all; the first of equal ones stays
    if (first < 0 || (!(m0 <= st.m) && st.m == st.m)) st.m = m0, first = v;
    if (!(m1 <= st.m) && st.m == st.m) st.m = m1, first = v + kThreads;
    const float ref = max_nan(st.ref, st.m * kLog2e);
    if (ref != st.ref) rescale(st, ref);
    float x[VEC];
    R::bounded(u0, x);
    add_terms(st, x);
    R::bounded(u1, x);
    add_terms(st, x);
  };
  const uint4 nothing = make_uint4(R::kNothing, R::kNothing, R::kNothing, R::kNothing);
  // vectors that lie inside the row, two at a time and kAhead on their way; the row's ends
  // are their threads' first and last
  const int hi = v_hi < r.full_hi ? v_hi : r.full_hi;
  auto full = [&](int v) { return v >= r.full_lo && v < hi ? __ldg(reinterpret_cast<const uint4*>(r.base) + v) : nothing; };
  int v = v_lo + (int)threadIdx.x;
  if (v == 0 && r.full_lo > 0) take(r.load(0), nothing, 0);
  if (v < hi) {
    uint4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = full(v + i * kThreads);
    while (v < hi) {
#pragma unroll
      for (int i = 0; i < kAhead; i += 2) {
        take(ahead[i], ahead[i + 1], v);
        ahead[i] = full(v + kAhead * kThreads);
        ahead[i + 1] = full(v + (kAhead + 1) * kThreads);
        if ((v += 2 * kThreads) >= hi) break;
      }
    }
  }
  if (r.full_hi < nv && v_hi == nv && nv - 1 >= r.full_lo && (nv - 1 - v_lo) % kThreads == (int)threadIdx.x)
    take(r.load(nv - 1), nothing, nv - 1);

  // sums over the CTA
  auto join = [&](Stats s) {
    float m = s.m, ref = s.ref;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      ref = max_nan(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    }
    rescale(s, ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s.s1 += __shfl_xor_sync(0xffffffffu, s.s1, o);
      s.s2 += __shfl_xor_sync(0xffffffffu, s.s2, o);
    }
    if (lane == 0) {
      sh.stat[warp][0] = m, sh.stat[warp][1] = ref;
      sh.stat[warp][2] = s.s1, sh.stat[warp][3] = s.s2;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      Stats t{sh.stat[0][0], sh.stat[0][1], 0.0f, 0.0f};
      for (int w = 1; w < kWarps; ++w) t.m = max_nan(t.m, sh.stat[w][0]), t.ref = max_nan(t.ref, sh.stat[w][1]);
      for (int w = 0; w < kWarps; ++w) {
        Stats q{0.0f, sh.stat[w][1], sh.stat[w][2], sh.stat[w][3]};
        rescale(q, t.ref);
        t.s1 += q.s1, t.s2 += q.s2;
      }
      sh.mine[0] = t.m, sh.mine[1] = t.ref, sh.mine[2] = t.s1, sh.mine[3] = t.s2;
    }
  };
  if (threadIdx.x == 0) sh.n_subset = sh.n_keys = 0;
  join(st);

  const int n = a.n_top;
  uint64_t key = 0, bound = 0;
  if (n > 0) {
    // the thread's largest key
    if (first >= 0) {
      float x[VEC];
      R::unpack(r.load(first), x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int64_t e = r.element(first, j);
        if (r.inside(e)) {
          const uint64_t k = key_of(x[j], (uint32_t)e);
          key = k > key ? k : key;
        }
      }
    }
    // a bound that n thread maxima reach: the n-th of the warps' first 2 ceil(n / 8) (of all
    // thread maxima, unless one warp holds more than twice its share of the first n).  Where
    // there is none, fewer than half of the threads have an element, and every one is taken.
    const int per_warp = (n + kWarps - 1) / kWarps * 2;
    uint64_t left = key;
    for (int i = 0; i < per_warp; ++i) {
      const uint64_t best = warp_max(left);
      if (left == best) left = 0;
      if (lane == 0) sh.keys[i * kWarps + warp] = best;
    }
    if (threadIdx.x == 0) sh.reach = 0;
    __syncthreads();
    if ((int)threadIdx.x < per_warp * kWarps) {
      const uint64_t k = sh.keys[threadIdx.x];
      int above = 0;
#pragma unroll 8
      for (int j = 0; j < per_warp * kWarps; ++j) above += sh.keys[j] > k;
      if (above == n - 1 && k != 0) sh.reach = k;
    }
  }
  // the row's sums, from the CTAs', and the best of their bounds: the CTA it comes from has n
  // elements that reach it
  Stats row_st;
  auto gather = [&]() {
    if (cluster > 1) {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
      row_st = Stats{-INFINITY, kLeast * kLog2e, 0.0f, 0.0f};
      for (int c = 0; c < cluster; ++c) {
        const float* p = cl.map_shared_rank(sh.mine, c);
        row_st.m = max_nan(row_st.m, p[0]);
        row_st.ref = max_nan(row_st.ref, p[1]);
        if (n > 0) {
          const uint64_t o = *cl.map_shared_rank(&sh.reach, c);
          bound = o > bound ? o : bound;
        }
      }
      for (int c = 0; c < cluster; ++c) {
        const float* p = cl.map_shared_rank(sh.mine, c);
        Stats o{0.0f, p[1], p[2], p[3]};
        rescale(o, row_st.ref);
        row_st.s1 += o.s1, row_st.s2 += o.s2;
      }
    } else {
      __syncthreads();
      row_st = Stats{sh.mine[0], sh.mine[1], sh.mine[2], sh.mine[3]};
      if (n > 0) bound = sh.reach;
    }
  };
  gather();
  // a maximum whose product with L is off by a part of 1 or more (a row of nothing but -inf
  // among them): the sums from differences, their reference 0
  const bool far = fabsf(row_st.m) >= kNear;
  const float top_l = max_nan(row_st.m, kLowest);
  if (far) {
    Stats f{row_st.m, 0.0f, 0.0f, 0.0f};
    for (int v = v_lo + (int)threadIdx.x; v < v_hi; v += kThreads) {
      float x[VEC];
      R::unpack(r.load(v), x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = max_nan(x[j] - top_l, kLeast) * kLog2e, e = ex2_approx(d);
        f.s1 += e;
        f.s2 = fmaf(e, d, f.s2);
      }
    }
    if (cluster > 1) cg::this_cluster().sync();
    else __syncthreads();
    join(f);
    gather();
  }

  // the elements that reach the bound, and the first n of them
  if (n > 0) {
    if (key >= bound && key != 0) sh.subset[atomicAdd(&sh.n_subset, 1)] = threadIdx.x;
    if (threadIdx.x < kMaxTop) sh.top[threadIdx.x] = 0;
    __syncthreads();
    // the elements of those subsets that reach the bound, a thread's reads together
    const int per = (v_hi - v_lo + kThreads - 1) / kThreads, items = sh.n_subset * per;
    for (int i0 = threadIdx.x; i0 < items; i0 += 4 * kThreads) {
      uint4 u[4];
      int at[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + q * kThreads;
        at[q] = i < items ? v_lo + sh.subset[i / per] + i % per * kThreads : v_hi;
        u[q] = at[q] < v_hi ? r.load(at[q]) : nothing;
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        if (order_of(R::largest(u[0])) >= (uint32_t)(bound >> 32) && at[0] < v_hi) {
          float x[VEC];
          R::unpack(u[0], x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int64_t e = r.element(at[0], j);
            if (!r.inside(e)) continue;
            const uint64_t k = key_of(x[j], (uint32_t)e);
            if (k >= bound) {
              const int i = atomicAdd(&sh.n_keys, 1);
              if (i < kCandidates) sh.keys[i] = k;
            }
          }
        }
        u[0] = u[1], u[1] = u[2], u[2] = u[3];
        at[0] = at[1], at[1] = at[2], at[2] = at[3];
      }
    }
    __syncthreads();
    const int count = sh.n_keys;
    if (count <= kCandidates) {
      for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t k = sh.keys[i];
        int above = 0;
        for (int j = 0; j < count; ++j) above += sh.keys[j] > k;
        if (above < n) sh.top[above] = k;
      }
    } else {
      // more than the list holds (values that repeat in the threads' pattern): one
      // pass over the slice per alternative, the first of them without a key to stay below: a NaN
      // at index 0 has the largest there is
      uint64_t last = 0;
      for (int i = 0; i < n; ++i) {
        uint64_t k_best = 0;
        for (int v = v_lo + (int)threadIdx.x; v < v_hi; v += kThreads) {
          float x[VEC];
          R::unpack(r.load(v), x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int64_t e = r.element(v, j);
            if (!r.inside(e)) continue;
            const uint64_t k = key_of(x[j], (uint32_t)e);
            if ((i == 0 || k < last) && k > k_best) k_best = k;
          }
        }
        k_best = warp_max(k_best);
        __syncthreads();
        if (lane == 0) sh.bound[warp] = k_best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) k_best = sh.bound[w] > k_best ? sh.bound[w] : k_best;
        if (threadIdx.x == 0) sh.top[i] = k_best;
        last = k_best;
      }
    }
  }
  if (n > 0 && cluster > 1) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int i = threadIdx.x; i < cluster * n; i += kThreads) sh.all[i] = cl.map_shared_rank(sh.top, i / n)[i % n];
  }
  __syncthreads();
  const float s1 = row_st.s1, s2 = row_st.s2;
  const float log_s1 = log2f(s1);  // -inf for a row of -inf
  // ln of the row's sum of e^(l - top_l): the reference is not quite L top_l
  const float log_sum = (log_s1 - (far ? 0.0f : fmaf(top_l, kLog2e, -row_st.ref))) * kLn2;
  // The row's largest element adds 2^(L top_l - r) to S1, which is 1 only before rounding, so the
  // logarithm of a certain token may come out 2^-24 above 0 and the entropy as much below: both
  // are cut at 0 (a NaN compares false and stays).
  auto logprob_of = [&](float l) {
    const float v = (l - top_l) - log_sum;
    return l == -INFINITY && s1 == s1 ? -INFINITY : (v > 0.0f ? 0.0f : v);
  };
  if (n > 0) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t k = sh.top[i];
      if (k == 0) continue;  // this slice holds fewer
      int place = i;
      if (cluster > 1) {
        place = 0;
        for (int j = 0; j < cluster * n; ++j) place += sh.all[j] > k;
      }
      if (place >= n) continue;
      a.top_logprob[row * n + place] = logprob_of(value_of((uint32_t)(k >> 32)));
      a.top_id[row * n + place] = index_of(k);
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    if (a.entropy) {
      const float h = (log_s1 - s2 / s1) * kLn2;
      a.entropy[row] = s1 == 0.0f || h < 0.0f ? 0.0f : h;
    }
    if (a.logprob) {
      const int64_t t = a.tokens[row];
      a.logprob[row] = t < 0 ? 0.0f
                             : (t < a.V ? logprob_of(to_f32(static_cast<const T*>(a.logits)[row * a.ld + t])) : NAN);
    }
  }
  if (cluster > 1) cg::this_cluster().sync();  // nobody's shared memory is read past here
}

template <typename T>
cudaError_t launch_typed(const TokenLogprobsArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  // few rows: a row over a cluster, up to two CTAs per SM and no slice under 4096 elements
  // (128 x 128000 bf16, 20 alternatives, us, all with three CTAs an SM: one CTA a row 34, two
  // 24, four 33, eight 49)
  int cluster = 1;
  while (cluster < kMaxCluster && a.M * cluster * 2 <= dev.sm_count * (int64_t)2 && a.V / (cluster * 2) >= 4096) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // no more CTAs than two an SM: the registers of both (128 x 128000 bf16, 20 alternatives, us:
  // 16.5 with two an SM, 19.7 with three, 22.7 with four; 4096 x 50000: 94, 77 and 71)
  return a.M * cluster <= dev.sm_count * (int64_t)2 ? cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, 2>, a, cluster)
                                                     : cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, 4>, a, cluster);
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobsArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.M <= 0) return cudaSuccess;
  return a.bf16 ? launch_typed<__nv_bfloat16>(a, dev, stream) : launch_typed<float>(a, dev, stream);
}

}  // namespace mamba
