// token_logprobs.cu - what a row of logits l [V] says about tokens:
//
//   log p(t) = l_t - m - ln S1,   H = ln S1 - S2 / S1,
//   m = max l,  S1 = sum e^d,  S2 = sum d e^d,  d = l - m
//
// and the likeliest tokens with their log p, by value and then by index.
//
// Bound: HBM, one pass over the logits.  A row is cut over the CTAs of a cluster
// (one CTA if there are rows enough), a CTA's slice over its threads in vectors of
// 16 bytes, vector v to thread v % 256.  A thread keeps a running maximum (with
// the first vector that holds it) and the two sums below it.
//
// Alternatives cost no second pass: an element of the row's first n is at least as
// large as the n-th largest thread maximum, so it lies in the subset of a thread
// whose maximum reaches that bound, and only those subsets (n of 256, and a few
// more) are read again, out of the caches.  Elements are compared as 64-bit keys,
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
  const T* base;  // 16-byte aligned
  int skew;
  int64_t V;
  __device__ Row(const void* p, int64_t v) {
    const uintptr_t u = reinterpret_cast<uintptr_t>(p);
    base = reinterpret_cast<const T*>(u & ~(uintptr_t)15);
    skew = (int)((u & 15) / sizeof(T));
    V = v;
  }
  __device__ int64_t vectors() const { return (skew + V + VEC - 1) / VEC; }
  // the values of vector v, -inf outside the row (whose memory is not read)
  __device__ void load(int64_t v, float (&x)[VEC]) const {
    const int64_t e0 = v * VEC - skew;
    if (e0 >= 0 && e0 + VEC <= V) {
      const uint4 u = *reinterpret_cast<const uint4*>(base + v * VEC);
      unpack(u, x);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        x[j] = e0 + j >= 0 && e0 + j < V ? to_f32(base[v * VEC + j]) : -INFINITY;
    }
  }
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
  __device__ bool inside(int64_t e) const { return e >= 0 && e < V; }
};

// running maximum and sums of one thread; ref is max(m, lowest finite), so a
// row of -inf has sums of nothing and no inf - inf
struct Stats {
  float m, ref, s1, s2;
};

__device__ __forceinline__ void rescale(Stats& s, float ref) {
  const float d = fmaxf(s.ref - ref, -1e30f);  // <= 0; NaN only when ref is NaN, and then s1 becomes NaN below
  const float c = ex2_approx(d * kLog2e);
  s.s2 = c * fmaf(d, s.s1, s.s2);
  s.s1 *= c;
  s.ref = ref;
}

struct SharedState {
  uint64_t keys[kCandidates];
  uint64_t top[kMaxTop];                  // this CTA's first n, in order
  uint64_t all[kMaxCluster * kMaxTop];    // the cluster's
  uint64_t bound[kWarps];
  int subset[kThreads];
  float stat[kWarps][3];
  float mine[3];                          // this CTA's reference, S1, S2
  int n_subset, n_keys;
  uint64_t best;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const TokenLogprobsArgs a, int cluster) {
  using R = Row<T>;
  constexpr int VEC = R::VEC;
  __shared__ SharedState sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t row = blockIdx.x / cluster;
  const int rank = (int)(blockIdx.x % cluster);
  grid_dependency_begin();
  const R r(static_cast<const T*>(a.logits) + row * a.ld, a.V);
  const int64_t nv = r.vectors();
  const int64_t v_lo = nv * rank / cluster, v_hi = nv * (rank + 1) / cluster;

  Stats st{-INFINITY, kLowest, 0.0f, 0.0f};
  int64_t first = -1;  // the first vector that holds m
  for (int64_t v = v_lo + threadIdx.x; v < v_hi; v += kThreads) {
    float x[VEC];
    r.load(v, x);
    float vm = x[0];
#pragma unroll
    for (int j = 1; j < VEC; ++j) vm = max_nan(vm, x[j]);
    if (first < 0 || (!(vm <= st.m) && st.m == st.m)) {
      st.m = vm;
      first = v;
    }
    const float ref = max_nan(st.ref, vm);
    if (ref != st.ref) rescale(st, ref);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float d = max_nan(x[j] - ref, -1e30f);
      const float e = ex2_approx(d * kLog2e);
      st.s1 += e;
      st.s2 = fmaf(e, d, st.s2);
    }
  }

  // the CTA's sums
  float ref = st.ref;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ref = max_nan(ref, __shfl_xor_sync(0xffffffffu, ref, o));
  if (lane == 0) sh.stat[warp][0] = ref;
  if (threadIdx.x == 0) sh.n_subset = sh.n_keys = 0;
  __syncthreads();
  ref = sh.stat[0][0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) ref = max_nan(ref, sh.stat[w][0]);
  rescale(st, ref);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    st.s1 += __shfl_xor_sync(0xffffffffu, st.s1, o);
    st.s2 += __shfl_xor_sync(0xffffffffu, st.s2, o);
  }
  if (lane == 0) {
    sh.stat[warp][1] = st.s1;
    sh.stat[warp][2] = st.s2;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float s1 = 0.0f, s2 = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      s1 += sh.stat[w][1];
      s2 += sh.stat[w][2];
    }
    sh.mine[0] = ref;
    sh.mine[1] = s1;
    sh.mine[2] = s2;
  }

  const int n = a.n_top;
  if (n > 0) {
    // the thread's largest key
    uint64_t key = 0;
    if (first >= 0) {
      float x[VEC];
      r.load(first, x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int64_t e = first * VEC - r.skew + j;
        if (r.inside(e)) {
          const uint64_t k = key_of(x[j], (uint32_t)e);
          key = k > key ? k : key;
        }
      }
    }
    // a bound that at least n thread maxima reach: the j-th largest of each warp,
    // j = ceil(n / 8), and of those the ceil(n / j)-th
    const int per_warp = (n + kWarps - 1) / kWarps;
    uint64_t left = key, best = 0;
    for (int i = 0; i < per_warp; ++i) {
      best = warp_max(left);
      if (left == best) left = 0;
    }
    if (lane == 0) sh.bound[warp] = best;
    __syncthreads();
    const int need = (n + per_warp - 1) / per_warp;
    uint64_t bound = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      int above = 0;
#pragma unroll
      for (int u = 0; u < kWarps; ++u) above += sh.bound[u] > sh.bound[w] || (sh.bound[u] == sh.bound[w] && u < w);
      if (above == need - 1) bound = sh.bound[w];
    }
    if (bound == 0) {  // fewer vectors than threads: the n-th largest of all thread maxima
      sh.keys[threadIdx.x] = key;
      if (threadIdx.x == 0) sh.best = 0;
      __syncthreads();
      int above = 0;
      for (int j = 0; j < kThreads; ++j) above += sh.keys[j] > key;
      if (above == n - 1 && key != 0) sh.best = key;
      __syncthreads();
      bound = sh.best;
    }
    if (key >= bound && key != 0) sh.subset[atomicAdd(&sh.n_subset, 1)] = threadIdx.x;
    if (threadIdx.x < kMaxTop) sh.top[threadIdx.x] = 0;
    __syncthreads();
    // the elements of those subsets that reach the bound
    for (int s = warp; s < sh.n_subset; s += kWarps) {
      for (int64_t v = v_lo + sh.subset[s] + (int64_t)lane * kThreads; v < v_hi; v += 32 * kThreads) {
        float x[VEC];
        r.load(v, x);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int64_t e = v * VEC - r.skew + j;
          if (!r.inside(e)) continue;
          const uint64_t k = key_of(x[j], (uint32_t)e);
          if (k >= bound) {
            const int i = atomicAdd(&sh.n_keys, 1);
            if (i < kCandidates) sh.keys[i] = k;
          }
        }
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
      // pass over the slice per alternative
      uint64_t last = ~0ull;
      for (int i = 0; i < n; ++i) {
        uint64_t k_best = 0;
        for (int64_t v = v_lo + threadIdx.x; v < v_hi; v += kThreads) {
          float x[VEC];
          r.load(v, x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int64_t e = v * VEC - r.skew + j;
            if (!r.inside(e)) continue;
            const uint64_t k = key_of(x[j], (uint32_t)e);
            if (k < last && k > k_best) k_best = k;
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
  __syncthreads();

  // the row's sums and first n, from the CTAs'
  float s1, s2;
  if (cluster > 1) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    ref = kLowest;
    for (int c = 0; c < cluster; ++c) ref = max_nan(ref, *cl.map_shared_rank(&sh.mine[0], c));
    s1 = s2 = 0.0f;
    for (int c = 0; c < cluster; ++c) {
      const float* p = cl.map_shared_rank(sh.mine, c);
      Stats o{0.0f, p[0], p[1], p[2]};
      rescale(o, ref);
      s1 += o.s1;
      s2 += o.s2;
    }
    if (n > 0) {
      for (int i = threadIdx.x; i < cluster * n; i += kThreads) sh.all[i] = cl.map_shared_rank(sh.top, i / n)[i % n];
    }
    cl.sync();  // nobody's shared memory is read past here
  } else {
    ref = sh.mine[0];
    s1 = sh.mine[1];
    s2 = sh.mine[2];
  }
  const float log_s1 = logf(s1);  // -inf for a row of -inf
  auto logprob_of = [&](float l) { return l == -INFINITY && s1 == s1 ? -INFINITY : (l - ref) - log_s1; };
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
    if (a.entropy) a.entropy[row] = s1 == 0.0f ? 0.0f : log_s1 - s2 / s1;
    if (a.logprob) {
      const int64_t t = a.tokens[row];
      a.logprob[row] = t < 0 ? 0.0f
                             : (t < a.V ? logprob_of(to_f32(static_cast<const T*>(a.logits)[row * a.ld + t])) : NAN);
    }
  }
}

template <typename T>
cudaError_t launch_typed(const TokenLogprobsArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  // few rows: a row over a cluster, until every SM has a CTA or a slice falls under 4096 elements
  int cluster = 1;
  while (cluster < kMaxCluster && a.M * cluster * 2 <= dev.sm_count * 2 && a.V / (cluster * 2) >= 4096) cluster *= 2;
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
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, a, cluster);
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobsArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.M <= 0) return cudaSuccess;
  return a.bf16 ? launch_typed<__nv_bfloat16>(a, dev, stream) : launch_typed<float>(a, dev, stream);
}

}  // namespace mamba
