// gated_delta_chunk.cu - the gated delta rule over long sequences, 64 tokens at
// a time on the tensor cores (formulas in gated_delta.cuh).
//
// With G_i the running sum of log alpha inside a chunk, K, Q, V its rows and S
// [dv][dk] the state before it, the chunk's corrections u_i = beta_i (v_i -
// alpha_i S_{i-1} k_i) solve a unit lower triangular system:
//
//   A_ij = beta_i e^{G_i - G_j} k_i.k_j (j < i),   T = (I + A)^-1 diag(beta)
//   P_ij = scale e^{G_i - G_j} q_i.k_j (j <= i)
//   R    = V - e^G K S^T                           [64][dv]
//   U    = T R,   Y = scale e^G Q S^T + P U
//   S'   = e^{G_63} S + (diag(e^{G_63 - G}) U)^T K
//
// T and P do not depend on the state: they are made while the previous chunk is
// still in flight.  X (I + A) = I is solved in blocks of 16 columns: the diagonal
// blocks of I + A are inverted by substitution (a lane a row, D_k), then
// Y_j = B_j - sum_{k > j} Y_k (D_k A_kj), X_k = Y_k D_k in warp-level tensor-core
// products.  (A thread a row for the whole substitution read A 64 times over from
// shared memory, 7-8 us a chunk; in f32 arithmetic by blocks it was 4.7.)  What
// remains on the path from state to state is three products and their epilogues,
// all held transposed, a tensor-memory lane per value component n:
//
//   D1 = S K^T    128 x 64 x dk      R^T = V^T - e^G D1                  (epilogue 1)
//   D2 = R^T T^T  128 x 64 x 64      U^T, and U^T decayed to the end     (epilogue 2)
//   D3 = U^T K    128 x dk x 64      S'  = e^G S + D3                    (epilogue 3)
//
// The output's two products, S Q^T and U^T P^T, run under epilogues 2 and 3.
//
// S, R^T and U^T go back to tensor memory as the A operands of the next product:
// nothing of the chain touches shared memory.  The f32 state stays in registers.
//
// Precision: f32 operands are the sum of three bf16 terms (24 bits, f32's range,
// so no scaling and no look at the data), bf16 keys and queries one.  Of the nine
// products of two such sums the six above 2^-24 are taken.  (Two f16 halves with
// power-of-two scales hold 22 bits for fewer products, but finding the scales,
// maxima over lanes and rows, took twice the instructions.)  A bf16 output of
// bf16 tensors with dk > 64, which feeds back into nothing, takes the products above
// 2^-16 alone (FULL): 4e-6 off in the mean before its own rounding of 2e-3.
//
// Bound: neither HBM (40 KB and 1.5 us of tensor-core time a chunk) nor the tensor
// cores but the instructions of the epilogues and of T, on a chain of dependent
// steps.  A further chunk of 128 x 128, bf16, takes 4.3 us with 12 CTAs, 4.5 with 76
// (one of each pair of SMs) and 4.8 with all 152: the loops of all roles are larger
// than the instruction cache, which is shared in pairs.  (64 x 64: 3.8, 3.9 and 4.4;
// f32 6.4, 6.4 and 6.7, of 128 x 128 14.1 throughout.)  So roles keep no more code than
// they need (one lookup per item, short waits, sums by a product with the identity)
// and few spills: each of these took 3 to 8 % off a chunk.
//
// An item is a (sequence, value head, 128 value components); its chunks follow one
// another.  How items and their chunks are laid over the SMs: see Plan.  A CTA's
// warps are specialised:
//   0-15  epilogues 1-3, output, the state in registers (lane = component; four
//         warps per lane quarter, each a quarter of the columns)
//   16-23 prepare: A and P from [K; Q] K^T and the gates, T and P to shared memory;
//         a chain of small dependent steps, longer than the path from state to
//         state, so two groups of four take the chunks in turn
//   24    the gates
//   25    issues the MMAs
//   26-27 load: tensor copies, or f32 / unaligned tensors by hand
#include <cuda.h>
#include <cudaTypedefs.h>

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
constexpr int kMainWarps = 16, kPrepWarps = 8, kLoadWarps = 2;
constexpr int kParts = kMainWarps / 4;  // warps that share a lane quarter of tensor memory
constexpr int kTok = kC / kParts;       // tokens of a chunk per such warp
constexpr int kGateWarp = kMainWarps + kPrepWarps, kMmaWarp = kGateWarp + 1, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr int kGroupWarps = kPrepWarps / 2, kGroupThreads = 32 * kGroupWarps, kLoadThreads = 32 * kLoadWarps;
constexpr int kGateSlots = 4;
constexpr int kLdA = kC + 4;      // row stride of A and P in shared memory, floats
constexpr long long kWaitLimit = 1ll << 31;  // SM cycles (about a second)
constexpr int kWaitTries = 1 << 18;          // of 4 us

__device__ int g_delta_faults = 0;

// per-chunk scalars and vectors, written by the gate warp
struct Gates {
  float hi[kC], lo[kC];  // G_i (base 2) as two floats
  float beta[kC];
  float eg[kC];     // e^{G_i}
  float egs[kC];    // scale e^{G_i}
  float fd[kC];     // e^{G_63 - G_i}
  float past[32];   // e^{G_31 - G_j}, j < 32
  float since[32];  // e^{G_i - G_31}, i = 32 ..
  float total;      // e^{G_63}
  // which chunk it is, for the warps that have no registers to keep track
  int at, begin, end;       // its number in the sequence, and those of the piece run here
  int tile, h, b, bh;       // the item
  int tokens;               // of the chunk inside the sequence
  int phi, pad[2];          // the schedule's
};

// FULL: the output takes all terms of its operands
template <int DK, bool F32, bool FULL>
struct Smem {
  static constexpr int kTerms = F32 ? 3 : 1;          // bf16 terms of K and Q
  static constexpr int kBlocks = DK / 64;
  static constexpr int kKqTerm = kBlocks * 16384;     // [K; Q]: 128 rows x 64 bf16 per block
  static constexpr int kKq = kTerms * kKqTerm;
  static constexpr int kKqStages = F32 ? (DK == 64 ? 2 : 1) : 3;
  static constexpr int kT = 3 * 8192;                 // T in three terms: 64 rows x 64 bf16
  static constexpr int kPTerms = FULL ? 3 : 2;
  static constexpr int kP = kPTerms * 8192;           // P
  static constexpr int kV = F32 ? 0 : kC * kM * 2;    // f32 values are read where they are used
  static constexpr int kOffT = kKqStages * kKq;
  static constexpr int kPBuffers = F32 || (FULL && DK > 64) ? 2 : 3;
  static constexpr int kAhead = F32 ? 1 : 2;          // chunks that are prepared ahead
  static constexpr int kOffP = kOffT + kT;
  static constexpr int kOffV = kOffP + kPBuffers * kP;
  static constexpr int kOffA = kOffV + kV;            // A, f32 [64][kLdA], of each group
  static constexpr int kOffGates = kOffA + 2 * kC * kLdA * 4;
  static constexpr int kOffBar = kOffGates + kGateSlots * (int)sizeof(Gates);
  static constexpr int kBars = 2 * kKqStages + 2 * kGateSlots + 2 + 3 + 2 * kPBuffers + 1 + 4 + 12 + 1;
  static constexpr int kBytes = kOffBar + 8 * kBars + 64;  // and tensor memory's address, the abort flag, the schedule
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(sizeof(Gates) % 16 == 0, "gate slots must keep 16-byte alignment");
  static_assert(kAlloc <= 232448, "shared memory over the opt-in limit");
};

// How the work is laid over CTAs (one an SM).
//  kWide: items in order, every CTA an equal run of their chunks, so that an item
//    may begin in one CTA and end in the next.  A CTA first runs the beginning of
//    its last item and leaves the state for the next CTA, then its whole items,
//    then the end of its first: by then the state it needs has long been there
//    (the CTA before started with it), and no two items wait in a circle.
//  Few items, long sequences: each is cut into `parts` of equal length, for which
//  three launches are made.
//  kAheadPass: the state at the end of every part but the last, the first part from
//    state_in, the others from zero; and, as one more item per head, the part's linear
//    map Phi of the state before it (the same recurrence with values of zero, from the
//    identity).  Nothing of the output is computed.
//  (join_kernel: state before part p + 1 = (state before part p) Phi_p + that.)
//  kPartsPass: all parts again, from their states, with their output.
enum { kWide = 0, kAheadPass = 1, kPartsPass = 2 };
struct Plan {
  int mode;
  int n_chunks;      // of a sequence
  int tiles, items;  // of 128 value components; B Hv tiles
  int parts, part_len;
  float* states;     // kWide: [CTA][128][dk]; else [parts - 1][B Hv][dv][dk], the state before parts 1 ..
  float* first;      // [B Hv][dv][dk], state_in: state_out, which may lie over it, is written before all have read it
  float* phi;        // [parts - 2][B Hv][dk][dk], of parts 1 ..
  int* flags;        // kWide: [CTA], the warps whose part of its state is there
};

// A CTA's chunks in the order in which it runs them: the beginning of an item
// (a_len chunks), b_count whole items, the end of an item (or a part of one).
struct Schedule {
  int a_item, a_len, b_first, b_count, t_item, t_begin, t_len, total;
  bool phi, quiet;  // a part's map instead of its values; no output
};
__device__ __forceinline__ Schedule make_schedule(const Plan& p, int heads) {
  Schedule s = {};
  const int n = p.n_chunks;
  if (p.mode == kWide) {
    const int64_t all = (int64_t)p.items * n;
    const int64_t lo = all * blockIdx.x / gridDim.x, hi = all * (blockIdx.x + 1) / gridDim.x;
    const int first = (int)(lo / n), last = (int)(hi / n);  // last: the item that hi lies in
    const int lo_c = (int)(lo % n), hi_c = (int)(hi % n);
    s.b_first = first + (lo_c > 0), s.b_count = last - s.b_first;  // no CTA has less than an item's chunks
    s.a_item = last, s.a_len = hi_c;
    if (lo_c > 0) s.t_item = first, s.t_begin = lo_c, s.t_len = n - lo_c;
  } else {
    s.quiet = p.mode == kAheadPass;
    const int values = p.items * (p.parts - s.quiet);  // CTAs that run values; the others run Phi
    int i = (int)blockIdx.x, part;
    if (i < values) {
      s.t_item = i % p.items, part = i / p.items;
    } else {
      i -= values;
      s.t_item = i % heads * p.tiles, part = 1 + i / heads;
      s.phi = true;
    }
    s.t_begin = part * p.part_len;
    s.t_len = n - s.t_begin < p.part_len ? n - s.t_begin : p.part_len;
  }
  s.total = s.a_len + s.b_count * n + s.t_len;
  return s;
}
struct Cursor {
  int item, c, begin, end, b_left;
  __device__ __forceinline__ void start(const Schedule& s, int n) {
    b_left = s.b_count + 1;  // as if before the whole items
    item = s.a_item, c = begin = 0, end = s.a_len;
    if (s.a_len == 0) piece(s, n);
  }
  __device__ __forceinline__ void piece(const Schedule& s, int n) {
    if (--b_left > 0) {
      item = s.b_first + s.b_count - b_left, begin = 0, end = n;
    } else {
      item = s.t_item, begin = s.t_begin, end = s.t_begin + s.t_len;
    }
    c = begin;
  }
  __device__ __forceinline__ void next(const Schedule& s, int n) {
    if (++c >= end) piece(s, n);
  }
};

// Tensor memory columns.  D1 is replaced by R's first two terms, later by those of
// the decayed U.  S's three terms take 1.5 dk columns from kColS, where D3 (dk
// columns) replaces them; R's third terms, then the decayed U's, and U's take the
// place of S's third, which only D1 reads.  (With FULL the queries' product reads those
// too: then R's third terms take the output's place if dk > 64; with dk <= 64 S's
// third terms lie before kColThird.)
constexpr uint32_t kColX = 0, kColQ = 64, kColU = 128, kColO = 192, kColS = 256, kColThird = 384, kColU3 = 416,
                   kColD0 = 448, kTmemCols = 512;

// kind::f16, bf16 A and B, f32 accumulator, M = 128; b_mn: B is MN-major; A's
// second terms, and B's where B is a sum too, are stored negated
constexpr uint32_t kNegA = 1u << 13, kNegB = 1u << 14;
__host__ __device__ constexpr uint32_t neg_bits(int ta, int tb) { return (ta == 1 ? kNegA : 0u) | (tb == 1 ? kNegB : 0u); }
__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kM >> 4) << 24);
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

// (a, b) as three bf16 pairs, each the rounding of what the ones before leave.  The
// remainder's instruction gives it negated, so the second pair comes out negated
// and the third not: the tensor products take the sign back (kNegA, kNegB).
__device__ __forceinline__ void split3n(float a, float b, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  float ra, rb;
  asm("{\n"
      "  .reg .b16 l, h;\n"
      "  cvt.rn.bf16x2.f32 %0, %4, %3;\n"
      "  mov.b32 {l, h}, %0;\n"
      "  sub.rn.f32.bf16 %1, l, %3;\n"
      "  sub.rn.f32.bf16 %2, h, %4;\n"
      "}\n"
      : "=&r"(t0), "=&f"(ra), "=&f"(rb)
      : "f"(a), "f"(b));
  asm("{\n"
      "  .reg .b16 l, h;\n"
      "  cvt.rn.bf16x2.f32 %0, %4, %3;\n"
      "  mov.b32 {l, h}, %0;\n"
      "  sub.rn.f32.bf16 %1, l, %3;\n"
      "  sub.rn.f32.bf16 %2, h, %4;\n"
      "}\n"
      : "=&r"(t1), "=&f"(a), "=&f"(b)
      : "f"(ra), "f"(rb));
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(t2) : "f"(a), "f"(b));
}
// with its sign, for the warp-level products
__device__ __forceinline__ void split3(float a, float b, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  split3n(a, b, t0, t1, t2);
  t1 ^= 0x80008000u;
}

// and as two
__device__ __forceinline__ void split2n(float a, float b, uint32_t& t0, uint32_t& t1) {
  float ra, rb;
  asm("{\n"
      "  .reg .b16 l, h;\n"
      "  cvt.rn.bf16x2.f32 %0, %4, %3;\n"
      "  mov.b32 {l, h}, %0;\n"
      "  sub.rn.f32.bf16 %1, l, %3;\n"
      "  sub.rn.f32.bf16 %2, h, %4;\n"
      "}\n"
      : "=&r"(t0), "=&f"(ra), "=&f"(rb)
      : "f"(a), "f"(b));
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(t1) : "f"(ra), "f"(rb));
}

// (a0, a1) += (b0 c0, b1 c1) in one instruction
__device__ __forceinline__ void fma2(float& a0, float& a1, float b0, float b1, float c0, float c1) {
  asm("{\n"
      "  .reg .b64 a, b, c;\n"
      "  mov.b64 a, {%0, %1};\n"
      "  mov.b64 b, {%2, %3};\n"
      "  mov.b64 c, {%4, %5};\n"
      "  fma.rn.f32x2 a, b, c, a;\n"
      "  mov.b64 {%0, %1}, a;\n"
      "}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// four 8 x 8 matrices of 16-bit values, lane l holding two of row l / 4 of each
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
// D[16][8] += A[16][16] B[16][8]
__device__ __forceinline__ void mma_sync(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  elect.sync _|p, 0xffffffff;\n"
      "  selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r));
  return r != 0;
}

// True once the phase of parity `parity` has completed, false after a while (4 us):
// until then the warp sleeps in the barrier's hardware.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "  selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
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

// boxes of four-dimensional tensor maps from and to shared memory
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(w), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(map), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}

// The products of two sums of terms, smallest first, as (term of a, term of b) in
// two bits each.  Three terms by one: 3, or the first 2; three by three: the 6
// above 2^-24, or the 3 above 2^-16.
template <bool THREE>
__device__ __forceinline__ constexpr void term_pair(int i, int& a, int& b) {
  if (THREE) {
    // (0,2) (2,0) (1,1) (0,1) (1,0) (0,0)
    a = (0x118 >> (2 * i)) & 3, b = (0x052 >> (2 * i)) & 3;
  } else {
    a = 2 - i, b = 0;
  }
}

// MAPS: q, k and v come through tensor maps (bf16, dk a multiple of 8) and the states
// are 16-byte aligned.  A kernel of its own, so that the loops of the other loads do
// not lie between its own.
template <int DK, bool F32, bool MAPS, bool FULL>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const GatedDeltaArgs g, const __grid_constant__ CUtensorMap map_k,
                                                            const __grid_constant__ CUtensorMap map_q,
                                                            const __grid_constant__ CUtensorMap map_v,
                                                            const __grid_constant__ CUtensorMap map_y, int vec_y,
                                                            const Plan plan) {
  using L = Smem<DK, F32, FULL>;
  static_assert(FULL || !F32, "f32 tensors take all terms");
  // The output of a chunk comes in the next one, under D2; with all its terms and dk >
  // 64 before epilogue 1, since S's third terms leave R's no columns but the output's.
  constexpr bool kEarly = F32 || (FULL && DK > 64);
  // U P^T of all terms is twice as long: in the next chunk, under epilogue 1, and not
  // before the product that it waits for (4.4 us a chunk against 4.8, 4.3 with half)
  constexpr bool kLate = FULL && !kEarly;
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
  const uint32_t gate_full = next_bars(kGateSlots), gate_empty = next_bars(kGateSlots);
  const uint32_t v_full = next_bars(1), v_empty = next_bars(1), t_full = next_bars(1);
  // of the chunk's parity: a group of prepare warps sees every other chunk
  const uint32_t t_empty = next_bars(2), d0_full = next_bars(2), d0_empty = next_bars(2);
  const uint32_t p_full = next_bars(L::kPBuffers), p_empty = next_bars(L::kPBuffers), o_empty = next_bars(1);
  // in halves (the warps of parts 0, 1 and of 2, 3): the products start on the first
  const uint32_t s_ready = next_bars(2), r_ready = next_bars(2), w_ready = next_bars(2), s_full = next_bars(2);
  const uint32_t x_full = next_bars(1), u_full = next_bars(1), u_ready = next_bars(1), o_full = next_bars(1), drained = next_bars(1);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(gbase + L::kOffBar + 8 * L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
  Schedule& sched = *reinterpret_cast<Schedule*>(tmem_ptr + 2);
  Gates* gates = reinterpret_cast<Gates*>(gbase + L::kOffGates);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n_all = plan.n_chunks;
  struct Item {
    int tile, h, hk;
    int64_t b;
  };
  auto item_of = [&](const Cursor& k) {
    const int bh = k.item / plan.tiles, h = bh % g.Hv;
    return Item{k.item % plan.tiles, h, h / (g.Hv / g.Hk), bh / g.Hv};
  };
  auto tokens_of = [&](const Cursor& k) { return (int)(g.T - (int64_t)k.c * kC < kC ? g.T - (int64_t)k.c * kC : kC); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kKqStages; ++s) mbar_init(kq_full + 8 * s, MAPS ? 1 : kLoadThreads), mbar_init(kq_empty + 8 * s, 1);
    for (int s = 0; s < kGateSlots; ++s) mbar_init(gate_full + 8 * s, 32), mbar_init(gate_empty + 8 * s, kMainWarps + kGroupWarps);
    mbar_init(v_full, MAPS ? 1 : kLoadThreads), mbar_init(v_empty, kMainWarps);
    mbar_init(t_full, kGroupWarps), mbar_init(o_empty, kMainWarps);
    for (int s = 0; s < 2; ++s) mbar_init(t_empty + 8 * s, 1), mbar_init(d0_full + 8 * s, 1), mbar_init(d0_empty + 8 * s, kGroupWarps);
    for (int s = 0; s < L::kPBuffers; ++s) mbar_init(p_full + 8 * s, kGroupWarps / 2), mbar_init(p_empty + 8 * s, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_ready + 8 * s, kMainWarps / 2), mbar_init(r_ready + 8 * s, kMainWarps / 2);
      mbar_init(w_ready + 8 * s, kMainWarps / 2), mbar_init(s_full + 8 * s, 1);
    }
    mbar_init(x_full, 1), mbar_init(u_full, 1), mbar_init(u_ready, kMainWarps), mbar_init(o_full, 1), mbar_init(drained, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (threadIdx.x == 32) sched = make_schedule(plan, (int)(g.B * g.Hv));
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
  const int n_chunks = sched.total;  // that this CTA runs

  // The gate, MMA and load warps' waits are counted; one that runs out sets the abort
  // flag, and every role then runs on through its loop without waiting, so that all
  // named barriers are met and the CTA ends.  The epilogue and prepare warps wait for
  // those warps alone (or for what they have started and wait for themselves), so
  // theirs only look at the flag: 12 instructions less at every wait are 3 % of a
  // chunk, the loops being larger than the instruction cache.
  auto wait_counted = [&](uint32_t bar, int phase) {
#pragma unroll 1
    for (int tries = 0; !mbar_sleep(bar, (uint32_t)(phase & 1)); ++tries) {
      if (tries > kWaitTries) *abort_flag = 1;
      if (*abort_flag) break;
    }
  };
  // for what is in flight at the end, whatever the flag says
  auto landed = [&](uint32_t bar, int phase) {
#pragma unroll 1
    for (int tries = 0; !mbar_sleep(bar, (uint32_t)(phase & 1)); ++tries) {
      if (tries > kWaitTries) {
        *abort_flag = 1;
        break;
      }
    }
  };
  auto wait = [&](uint32_t bar, int phase) {
    while (!mbar_sleep(bar, (uint32_t)(phase & 1))) {
      if (*abort_flag) break;
    }
  };

  if (warp < kMainWarps) {
    // ---------------------------------------------------------- epilogues ----
    constexpr int HK = DK / kParts;  // key components per thread
    const int quad = warp & 3, part = warp >> 2;
    const uint32_t half = 8 * (part >> 1);  // this warp's of two barriers
    const int lane_n = quad * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
    float s[HK] = {};
    // four of this lane's values of a [..][dk] state, `left` of them inside it
    auto load_state = [&](const float* src, bool vec) {
#pragma unroll
      for (int j = 0; j < HK; j += 4) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int left = g.dk - part * HK - j;
        if (src) {
          const float* p = src + part * HK + j;
          if (vec) {
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
    };
    auto store_state = [&](float* dst, bool vec) {
#pragma unroll
      for (int j = 0; j < HK; j += 4) {
        float* p = dst + part * HK + j;
        const int left = g.dk - part * HK - j;
        if (vec) {
          if (left > 0) *reinterpret_cast<float4*>(p) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        } else {
          if (left > 0) p[0] = s[j];
          if (left > 1) p[1] = s[j + 1];
          if (left > 2) p[2] = s[j + 2];
          if (left > 3) p[3] = s[j + 3];
        }
      }
    };
    // False once a wait has run out: what was read of the gates before may then be
    // unwritten, or of another chunk (their writer changes a slot that is in use only
    // after it has seen the flag), and no global address is made of it.  Warps decide
    // as one.
    auto live = [&]() {
      asm volatile("" ::: "memory");
      return __all_sync(0xffffffffu, *abort_flag == 0) != 0;
    };
    auto vec_state = [&](const float* p) { return MAPS || (g.dk % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0); };
    const int64_t all_states = g.B * g.Hv * (int64_t)g.dv * g.dk;
    // the state before the chunk's piece
    auto enter = [&](const Gates& k) {
      const int n = k.tile * kM + lane_n, begin = k.begin;
      const int64_t row = ((int64_t)k.bh * g.dv + n) * g.dk;
      if (!live()) return;
      if (k.phi) {
#pragma unroll
        for (int j = 0; j < HK; ++j) s[j] = part * HK + j == lane_n ? 1.0f : 0.0f;
        return;
      }
      const float* src = g.state_in ? g.state_in + row : nullptr;
      if (plan.mode == kWide && begin > 0) {  // the CTA before has run the item's beginning
        volatile int* flag = plan.flags + blockIdx.x - 1;
        const long long t0 = clock64();
        while (*flag < kMainWarps && !*abort_flag) {
          if (clock64() - t0 > kWaitLimit) {
            *abort_flag = 1;
          }
          __nanosleep(200);
        }
        __threadfence();
        src = plan.states + ((int64_t)(blockIdx.x - 1) * kM + lane_n) * g.dk;
      } else if (plan.mode == kAheadPass && begin > 0) {
        src = nullptr;
      } else if (plan.mode == kPartsPass) {
        if (begin > 0)
          src = plan.states + (begin / plan.part_len - 1) * all_states + row;
        else if (src)
          src = plan.first + row;
      }
      load_state(n < g.dv ? src : nullptr, vec_state(src));
      if (plan.mode == kAheadPass && src && n < g.dv) store_state(plan.first + row, vec_state(plan.first));
    };
    // and after it
    auto leave = [&](const Gates& k) {
      const int n = k.tile * kM + lane_n;
      const int64_t row = ((int64_t)k.bh * g.dv + n) * g.dk;
      const int p = plan.mode == kWide ? 0 : k.begin / plan.part_len, bh = k.bh;
      const bool inside = k.end < n_all, hand_over = inside && plan.mode == kWide, phi = k.phi;
      if (!live()) return;
      float* dst = n < g.dv ? g.state_out : nullptr;
      if (dst) dst += row;
      if (hand_over)
        dst = plan.states + ((int64_t)blockIdx.x * kM + lane_n) * g.dk;
      else if (phi)
        dst = lane_n < g.dk ? plan.phi + (((p - 1) * g.B * g.Hv + bh) * g.dk + lane_n) * g.dk : nullptr;
      else if (plan.mode == kAheadPass)
        dst = n < g.dv ? plan.states + p * all_states + row : nullptr;
      else if (inside)
        dst = nullptr;
      if (dst) store_state(dst, vec_state(dst));
      if (hand_over) {
        // counted warp by warp: a barrier here would depend on what the gates say, which
        // the warps need not agree on once a wait has run out
        __threadfence();
        __syncwarp();
        if (lane == 0) atomicAdd(plan.flags + blockIdx.x, 1);
      }
    };
    const int i0 = part * kTok;  // this thread's tokens of a chunk
    const uint32_t y_step = (uint32_t)g.ld_y * (g.y_bf16 ? 2 : 4);  // bytes; a chunk's rows fit 32 bits
    auto arrive = [&](uint32_t bar) {
      tmem_wait_st();
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // chunk c's output; it comes in the next chunk while D2 is in flight, so that
    // the path from state to state does not wait for it
    auto output = [&](int c) {
      const Gates& gt = gates[c % kGateSlots];
      const bool quiet = sched.quiet;
      const bool direct = kEarly || !vec_y;
      char* y_at = nullptr;
      int y_rows = 0;
      if (direct && !quiet) {
        const int n = gt.tile * kM + lane_n;
        y_at = reinterpret_cast<char*>(g.y) +
               ((gt.b * g.T + (int64_t)gt.at * kC + i0) * g.ld_y + (int64_t)gt.h * g.dv + n) * (g.y_bf16 ? 2 : 4);
        y_rows = n < g.dv ? gt.tokens - i0 : 0;
        if (!live()) y_rows = 0;
      }
      wait(o_full, c);
      tcgen05_fence_after();
      // staged over the chunk's values, which epilogue 1 of the next chunk has just
      // taken (the last chunk's own are long gone too), for a tensor store; or
      // stored from here
      __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(gbase + L::kOffV) + i0 * kM + lane_n;
#pragma unroll 1
      for (int i = quiet ? kTok : 0; i < kTok; i += 8) {
        uint32_t xq[8], xo[8];
        tmem_ld8(t_lane + kColQ + (uint32_t)(i0 + i), xq);
        tmem_ld8(t_lane + kColO + (uint32_t)(i0 + i), xo);
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; j += 4) *reinterpret_cast<float4*>(&o[j]) = *reinterpret_cast<const float4*>(&gt.egs[i0 + i + j]);
        tmem_wait(xq);
        tmem_wait(xo);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float lo = __uint_as_float(xo[j]), hi = __uint_as_float(xo[j + 1]);
          fma2(lo, hi, o[j], o[j + 1], __uint_as_float(xq[j]), __uint_as_float(xq[j + 1]));
          o[j] = lo, o[j + 1] = hi;
        }
        if (!direct) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const __nv_bfloat162 w = __floats2bfloat162_rn(o[j], o[j + 1]);
            stage[(i + j) * kM] = w.x, stage[(i + j + 1) * kM] = w.y;
          }
          continue;
        }
        uint32_t at = (uint32_t)i * y_step;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (i + j < y_rows) {
            if (g.y_bf16)
              *reinterpret_cast<__nv_bfloat16*>(y_at + at) = __float2bfloat16_rn(o[j]);
            else
              *reinterpret_cast<float*>(y_at + at) = o[j];
          }
          at += y_step;
        }
      }
      if (!kEarly) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_empty);
      }
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty), mbar_arrive(gate_empty + 8 * (c % kGateSlots));
    };
#pragma unroll 1
    for (int c = 0; c <= n_chunks; ++c) {
      const Gates& gt = gates[c % kGateSlots];
      if (kEarly && c > 0) {  // U's third terms are read, where S's third come next
        wait(o_full, c - 1);
        tcgen05_fence_after();
      }
      if (c < n_chunks) {
        wait(gate_full + 8 * (c % kGateSlots), c / kGateSlots);
        if (__any_sync(0xffffffffu, gt.at == gt.begin)) enter(gt);
        // S to tensor memory: of this warp's HK columns of D3's place the first
        // half the first terms, the rest the second; the third terms beyond D3
        const uint32_t at = t_lane + kColS + (uint32_t)(part * HK), at2 = t_lane + kColS + (uint32_t)(DK + part * HK / 2);
#pragma unroll
        for (int j0 = 0; j0 < HK; j0 += 16) {
          uint32_t t0[8], t1[8], t2[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) split3n(s[j0 + 2 * j], s[j0 + 2 * j + 1], t0[j], t1[j], t2[j]);
          tmem_st8(at + (uint32_t)(j0 / 2), t0);
          tmem_st8(at + (uint32_t)(HK / 2 + j0 / 2), t1);
          if (j0 == 0 && half == 0 && c > 0) {  // D3's second half reads the decayed U there
            wait(s_full + 8, c - 1);
            tcgen05_fence_after();
          }
          tmem_st8(at2 + (uint32_t)(j0 / 2), t2);
        }
        arrive(s_ready + half);
      }
      if (!kEarly && c == n_chunks) wait(v_full, c);  // the output before the last has left its place
      if (c > 0 && (kEarly || c == n_chunks)) output(c - 1);
      if (c == n_chunks) break;
      {  // epilogue 1: R^T = V^T - e^G D1
        static_assert(kTok == 16, "one tensor-memory load");
        float r[kTok];
        if (F32) {
          const int n = gt.tile * kM + lane_n;
          int rows = n < g.dv && !gt.phi ? gt.tokens - i0 : 0;
          const In* v = reinterpret_cast<const In*>(g.v) + (gt.b * g.T + (int64_t)gt.at * kC + i0) * g.ld_v + (int64_t)gt.h * g.dv + n;
          if (!live()) rows = 0;
#pragma unroll
          for (int j = 0; j < kTok; ++j) {
            r[j] = j < rows ? to_f32(*v) : 0.0f;
            v += g.ld_v;
          }
        } else {
          wait(v_full, c);
          const In* v = reinterpret_cast<const In*>(gbase + L::kOffV) + i0 * kM + lane_n;
#pragma unroll
          for (int j = 0; j < kTok; ++j) r[j] = to_f32(v[j * kM]);
          if (kEarly) {  // no output takes their place
            __syncwarp();
            if (lane == 0) mbar_arrive(v_empty);
          }
          if (gt.phi) {
#pragma unroll
            for (int j = 0; j < kTok; ++j) r[j] = 0.0f;
          }
        }
        wait(x_full, c);
        tcgen05_fence_after();
#pragma unroll
        for (int j0 = 0; j0 < kTok; j0 += 8) {  // all of it is read before the first is replaced
          uint32_t x[8];
          tmem_ld8(t_lane + kColX + (uint32_t)(i0 + j0), x);
          tmem_wait(x);
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 eg = *reinterpret_cast<const float4*>(&gt.eg[i0 + j0 + j]);
            fma2(r[j0 + j], r[j0 + j + 1], -eg.x, -eg.y, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
            fma2(r[j0 + j + 2], r[j0 + j + 3], -eg.z, -eg.w, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
          }
        }
        uint32_t t0[8], t1[8], t2[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split3n(r[2 * j], r[2 * j + 1], t0[j], t1[j], t2[j]);
        tmem_st8(t_lane + kColX + (uint32_t)i0, t0);
        tmem_st8(t_lane + kColX + (uint32_t)(i0 + 8), t1);
        tmem_st8(t_lane + (kEarly ? kColO + (uint32_t)i0 : kColThird + (uint32_t)(8 * part)), t2);
        arrive(r_ready + half);
      }
      if (!kEarly) {
        if (c > 0) {
          // every warp has its values before one writes its output there
          named_barrier(5, 32 * kMainWarps);
          output(c - 1);
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(v_empty);
        }
      }
      {  // epilogue 2: U^T for the output, and decayed to the chunk's end for S
        wait(u_full, c);
        tcgen05_fence_after();
        uint32_t x[16];
        tmem_ld16(t_lane + kColU + (uint32_t)i0, x);
        tmem_wait(x);
#pragma unroll
        for (int j0 = 0; j0 < 8; j0 += 4) {
          uint32_t t0[4], t1[4], t2[4];
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint32_t* u = x + 2 * (j0 + j);
            const float4 fd = *reinterpret_cast<const float4*>(&gt.fd[i0 + 2 * (j0 + j)]);
            split3n(fd.x * __uint_as_float(u[0]), fd.y * __uint_as_float(u[1]), t0[j], t1[j], t2[j]);
            split3n(fd.z * __uint_as_float(u[2]), fd.w * __uint_as_float(u[3]), t0[j + 1], t1[j + 1], t2[j + 1]);
          }
          tmem_st4(t_lane + kColX + (uint32_t)(i0 + j0), t0);
          tmem_st4(t_lane + kColX + (uint32_t)(i0 + 8 + j0), t1);
          tmem_st4(t_lane + kColThird + (uint32_t)(8 * part + j0), t2);
        }
        arrive(w_ready + half);
        if (!sched.quiet) {
          uint32_t t0[8], t1[8], t2[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (FULL)
              split3n(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]), t0[j], t1[j], t2[j]);
            else
              split2n(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]), t0[j], t1[j]);
          }
          tmem_st8(t_lane + kColU + (uint32_t)i0, t0);
          tmem_st8(t_lane + kColU + (uint32_t)(i0 + 8), t1);
          if (FULL) tmem_st8(t_lane + kColU3 + (uint32_t)(8 * part), t2);
        }
        arrive(u_ready);
      }
      {  // epilogue 3: S = e^G S + D3
        const float total = gt.total;
        wait(s_full + half, c);
        tcgen05_fence_after();
#pragma unroll
        for (int j0 = 0; j0 < HK; j0 += 16) {
          uint32_t x[16];
          tmem_ld16(t_lane + kColS + (uint32_t)(part * HK + j0), x);
          tmem_wait(x);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float lo = __uint_as_float(x[j]), hi = __uint_as_float(x[j + 1]);
            fma2(lo, hi, total, total, s[j0 + j], s[j0 + j + 1]);
            s[j0 + j] = lo, s[j0 + j + 1] = hi;
          }
        }
      }
      if (__any_sync(0xffffffffu, gt.at + 1 == gt.end)) leave(gt);
    }
  } else if (warp < kGateWarp) {
    // ------------------------------------------------------------ prepare ----
    const int quad = warp & 3;
    const int group = (warp - kMainWarps) >> 2;  // takes chunks group, group + 2, ..
    const int bar_id = 1 + group;
    const int row = quad * 32 + lane;       // row of [K; Q]
    const bool is_t = quad < 2;             // warp-uniform
    const bool upper = quad & 1;            // tokens 32-63: the rows with columns past 31
    const int i = row & (kC - 1);           // token
    float* a_s = reinterpret_cast<float*>(gbase + L::kOffA) + group * kC * kLdA;
    // The blocks (k, j) of D and N = -D A, in three terms of 16 rows of 32 bytes, take
    // A's place: the first two that of their block of A, the third one above the
    // diagonal.  Rows are 17 granules of 16 bytes apart, so no two of eight share banks.
    const uint32_t n_s = base + L::kOffA + (uint32_t)(group * kC * kLdA * 4);
    auto term_at = [&](int k, int j, int t) {
      int a = k, b = j, off = 32 * t;
      if (t == 2) {
        if (k == j)
          a = k < 3 ? 0 : 1, b = k < 3 ? k + 1 : 2, off = 32;
        else
          a = j, b = k, off = 0;
      }
      return n_s + (uint32_t)(a * 16 * kLdA * 4 + b * 64 + off);
    };
    const int rb = quad;  // T's block of 16 rows that this warp solves
    const int fr = lane / 4, fc = 2 * (lane % 4);  // accumulator fragment: rows fr, fr + 8, columns fc, fc + 1
    // this lane's row for ldmatrix: matrices (k 0-7, n 0-7), (k 8-15, n 0-7), (k 0-7, n 8-15), ..
    const uint32_t ld_at = (uint32_t)((lane & 15) * kLdA * 4 + (lane >> 4) * 16);
    // acc += x m over three terms each, the small and the large products in two
    // chains (one is 20 cycles long, 66 while tcgen05 products are in flight)
    auto product = [&](float (&acc)[2][4], const uint32_t (&x)[3][4], const uint32_t (&m)[3][4]) {
      float small[2][4];
#pragma unroll
      for (int nn = 0; nn < 2; ++nn)
#pragma unroll
        for (int e = 0; e < 4; ++e) small[nn][e] = 0.0f;
#pragma unroll
      for (int p = 0; p < 6; ++p) {
        int ta, tb;
        term_pair<true>(p, ta, tb);
#pragma unroll
        for (int nn = 0; nn < 2; ++nn) mma_sync(p < 3 ? small[nn] : acc[nn], x[ta], m[tb][2 * nn], m[tb][2 * nn + 1]);
      }
#pragma unroll
      for (int nn = 0; nn < 2; ++nn)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nn][e] += small[nn][e];
    };
    // the A operand of a 16 x 16 block held as two accumulators
    auto operand = [&](uint32_t (&x)[3][4], const float (&c)[2][4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) split3(c[e / 2][2 * (e & 1)], c[e / 2][2 * (e & 1) + 1], x[0][e], x[1][e], x[2][e]);
    };
#pragma unroll 1
    for (int c = group; c < n_chunks; c += 2) {
      const Gates& gt = gates[c % kGateSlots];
      const uint32_t t_d0 = tmem + ((uint32_t)(quad * 32) << 16) + kColD0;
      wait(gate_full + 8 * (c % kGateSlots), c / kGateSlots);
      wait(d0_full + 8 * group, c / 2);
      tcgen05_fence_after();
      named_barrier(bar_id, kGroupThreads);  // the previous chunk's blocks are read
      if (is_t || !sched.quiet) {
        // a row per thread: -A in f32, P in its terms (granule q of row r at
        // q ^ (r % 8))
        const int pb = c % L::kPBuffers;
        if (!is_t && c >= L::kPBuffers) wait(p_empty + 8 * pb, c / L::kPBuffers - 1);
        float* dst = a_s + i * kLdA;
        const uint32_t dst_p = base + L::kOffP + pb * L::kP + (uint32_t)(i * 128);
        auto put8 = [&](int j, const float (&o)[8]) {
          if (is_t) {
            *reinterpret_cast<float4*>(dst + j) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4*>(dst + j + 4) = make_float4(o[4], o[5], o[6], o[7]);
          } else {
            uint32_t t[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (FULL)
                split3n(o[2 * e], o[2 * e + 1], t[0][e], t[1][e], t[2][e]);
              else
                split2n(o[2 * e], o[2 * e + 1], t[0][e], t[1][e]);
            }
            const uint32_t at = dst_p + (uint32_t)(((j / 8) ^ (i & 7)) << 4);
#pragma unroll
            for (int e = 0; e < L::kPTerms; ++e)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + e * 8192), "r"(t[e][0]), "r"(t[e][1]),
                           "r"(t[e][2]), "r"(t[e][3])
                           : "memory");
          }
        };
        const float scale_row = is_t ? -gt.beta[i] : g.scale;
        if (upper) {
          // the 32 columns before these rows' own: the decay factors at token 31
          const float since = gt.since[lane] * scale_row;
#pragma unroll 1
          for (int j = 0; j < 32; j += 8) {
            uint32_t d[8];
            float o[8];
            tmem_ld8(t_d0 + (uint32_t)j, d);
#pragma unroll
            for (int e = 0; e < 8; e += 4) *reinterpret_cast<float4*>(&o[e]) = *reinterpret_cast<const float4*>(&gt.past[j + e]);
            tmem_wait(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= since * __uint_as_float(d[e]);
            put8(j, o);
          }
        }
        const float rh = gt.hi[i], rl = gt.lo[i];
        const int jd = upper ? 32 : 0;
#pragma unroll 1
        for (int j = jd; j < jd + 32; j += 8) {
          const int last = (is_t ? i - 1 : i) - j;  // A is strictly lower, P lower
          uint32_t d[8];
          tmem_ld8(t_d0 + (uint32_t)j, d);
          float o[8], cl[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            *reinterpret_cast<float4*>(&o[e]) = *reinterpret_cast<const float4*>(&gt.hi[j + e]);
            *reinterpret_cast<float4*>(&cl[e]) = *reinterpret_cast<const float4*>(&gt.lo[j + e]);
          }
          tmem_wait(d);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float w = ex2_approx((rh - o[e]) + (rl - cl[e])) * scale_row;
            o[e] = e <= last ? __uint_as_float(d[e]) * w : 0.0f;
          }
          put8(j, o);
        }
        if (!is_t) fence_proxy_async_smem();
      }
      tcgen05_fence_before();
      named_barrier(bar_id, kGroupThreads);
      if (lane == 0) {
        mbar_arrive(d0_empty + 8 * group);
        if (!is_t) mbar_arrive(p_full + 8 * (c % L::kPBuffers));
      }
      // the inverse of diagonal block `quad` of I + A over the block itself, a lane
      // a row (16-31 repeat 0-15): X (I + A) = I, columns from the last
      float* blk = a_s + 16 * quad * (kLdA + 1);
      {
        const int r = lane & 15;
        float x[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) x[q] = q == r ? 1.0f : 0.0f;
#pragma unroll
        for (int k = 15; k >= 1; --k) {
#pragma unroll
          for (int q = 0; q < k; q += 4) {
            const float4 a = *reinterpret_cast<const float4*>(blk + k * kLdA + q);
            fma2(x[q], x[q + 1], x[k], x[k], a.x, a.y);  // zero from column k on
            if (q + 2 < k) fma2(x[q + 2], x[q + 3], x[k], x[k], a.z, a.w);
          }
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t t[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split3(x[8 * q + 2 * e], x[8 * q + 2 * e + 1], t[0][e], t[1][e], t[2][e]);
#pragma unroll
            for (int e = 0; e < 3; ++e)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(term_at(quad, quad, e) + r * kLdA * 4 + 16 * q),
                           "r"(t[e][0]), "r"(t[e][1]), "r"(t[e][2]), "r"(t[e][3])
                           : "memory");
          }
        }
      }
      named_barrier(bar_id, kGroupThreads);
      // N_kj = D_k (-A_kj) below the diagonal, blocks (1,0) (2,0) (2,1) (3,0) (3,1)
      // (3,2) by warps 3 0 1 2 3 0
#pragma unroll 1
      for (int p = (quad + 1) % 4; p < 6; p += 4) {
        const int k = p < 1 ? 1 : p < 3 ? 2 : 3, j = p - k * (k - 1) / 2;
        const float* m = a_s + 16 * k * kLdA + 16 * j;
        uint32_t xt[3][4], mt[3][4];
#pragma unroll
        for (int nn = 0; nn < 2; ++nn)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            split3(m[(8 * kk + fc) * kLdA + 8 * nn + fr], m[(8 * kk + fc + 1) * kLdA + 8 * nn + fr], mt[0][2 * nn + kk],
                   mt[1][2 * nn + kk], mt[2][2 * nn + kk]);
#pragma unroll
        for (int e = 0; e < 3; ++e) ldmatrix4(xt[e], term_at(k, k, e) + ld_at);
        float x[2][4] = {};
        product(x, xt, mt);
        operand(xt, x);
        __syncwarp();  // the block of A is read
#pragma unroll
        for (int e = 0; e < 3; ++e) stmatrix4(term_at(k, j, e) + ld_at, xt[e]);
      }
      named_barrier(bar_id, kGroupThreads);  // D and N are there
      {
        // rows 16 rb .. of T = X diag(beta): the identity's first step takes N's blocks
        // and D's as they are (the sum of the terms: a product by the identity)
        float x[4][2][4];
        const uint32_t one = (fr == fc ? 0x3f80u : 0u) | (fr == fc + 1 ? 0x3f800000u : 0u);
        const uint32_t identity[4] = {one, 0, 0, one};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int nn = 0; nn < 2; ++nn)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k][nn][e] = 0.0f;
          if (k > rb) continue;
#pragma unroll
          for (int e = 2; e >= 0; --e) {
            uint32_t m[4];
            ldmatrix4_trans(m, term_at(rb, k, e) + ld_at);
            mma_sync(x[k][0], identity, m[0], m[1]);
            mma_sync(x[k][1], identity, m[2], m[3]);
          }
        }
#pragma unroll
        for (int k = 2; k >= 0; --k) {
          if (k >= rb) continue;  // warp-uniform
          uint32_t xt[3][4];
          operand(xt, x[k]);
#pragma unroll
          for (int nn = 0; nn < 2; ++nn)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k][nn][e] = 0.0f;  // replaced by Y_k D_k
#pragma unroll
          for (int u = 1; u <= k + 1; ++u) {  // the next block first, the diagonal's last
            const int j = u <= k ? k - u : k;
            uint32_t m[3][4];
#pragma unroll
            for (int e = 0; e < 3; ++e) ldmatrix4_trans(m[e], term_at(k, j, e) + ld_at);
            product(x[j], xt, m);
          }
        }
        // columns times beta, in three terms to shared memory
        const uint32_t at = base + L::kOffT + (uint32_t)(rb * 2048) +
                            (uint32_t)((((lane >> 3) & 1) * 8 + (lane & 7)) * 128 + ((((lane >> 4) & 1) ^ (lane & 7)) << 4));
        if (c > 0) wait(t_empty + 8 * ((c - 1) & 1), (c - 1) / 2);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k > rb) continue;
          uint32_t xt[3][4];
#pragma unroll
          for (int nn = 0; nn < 2; ++nn) {
            const float2 be = *reinterpret_cast<const float2*>(&gt.beta[16 * k + 8 * nn + fc]);
            x[k][nn][0] *= be.x, x[k][nn][1] *= be.y, x[k][nn][2] *= be.x, x[k][nn][3] *= be.y;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            split3n(x[k][e / 2][2 * (e & 1)], x[k][e / 2][2 * (e & 1) + 1], xt[0][e], xt[1][e], xt[2][e]);
#pragma unroll
          for (int e = 0; e < 3; ++e) stmatrix4((at ^ (uint32_t)(k << 5)) + e * 8192, xt[e]);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(t_full);
        mbar_arrive(gate_empty + 8 * (c % kGateSlots));
      }
    }
  } else if (warp == kGateWarp) {
    // -------------------------------------------------------------- gates ----
    // tokens lane and lane + 32 of a chunk: base-2 logarithms of alpha, summed and
    // kept as two floats each, so that differences between far-decayed tokens keep
    // 32-bit accuracy.  alpha below e^-200 is 0 in f32 all the same.
    float neg_A = 0.0f, dt_bias = 0.0f;
    Cursor at_chunk;
    at_chunk.start(sched, n_all);
    Item it = {};
    const In* a_base = nullptr;
    const In* b_base = nullptr;
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
      if (at_chunk.c == at_chunk.begin) {
        it = item_of(at_chunk);
        a_base = reinterpret_cast<const In*>(g.a) + it.b * g.T * g.ld_a + it.h;
        b_base = reinterpret_cast<const In*>(g.b) + it.b * g.T * g.ld_b + it.h;
        neg_A = -expf(g.A_log[it.h]);
        dt_bias = g.dt_bias ? g.dt_bias[it.h] : 0.0f;
      }
      Two G[2];
      float la[2], be[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t t = (int64_t)at_chunk.c * kC + lane + 32 * u;
        la[u] = t < g.T ? to_f32(a_base[t * g.ld_a]) : 0.0f;
        be[u] = t < g.T ? to_f32(b_base[t * g.ld_b]) : 0.0f;
      }
      const int left = tokens_of(at_chunk) - lane;
#pragma unroll 1
      for (int u = 0; u < 2; ++u) {  // once, then with the two tokens' places changed
        const float l = gdr_log_alpha(la[0], dt_bias, neg_A), beta = gdr_beta(be[0]);
        const bool inside = 32 * u < left;  // past the end alpha is 1 and beta 0, whatever the head's A and bias
        la[0] = la[1], be[0] = be[1];
        la[1] = inside ? l : 0.0f, be[1] = inside ? beta : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) G[u] = two_log2(la[u] < -200.0f ? -200.0f : la[u]);
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const Two sum = two_add(G[u], two_shfl_up(G[u], o));
          if (lane >= o) G[u] = sum;
        }
      }
      const Two mid = two_shfl(G[0], 31);
      G[1] = two_add(G[1], mid);
      const Two last = two_shfl(G[1], 31);
      Gates& gt = gates[c % kGateSlots];
      if (c >= kGateSlots) wait_counted(gate_empty + 8 * (c % kGateSlots), c / kGateSlots + 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        gt.hi[i] = G[u].h, gt.lo[i] = G[u].l;
        gt.beta[i] = be[u];
        const float eg = ex2_approx(G[u].h + G[u].l);
        gt.eg[i] = eg, gt.egs[i] = g.scale * eg;
        gt.fd[i] = two_exp2(last, G[u]);
      }
      gt.past[lane] = two_exp2(mid, G[0]);
      gt.since[lane] = two_exp2(G[1], mid);
      if (lane == 0) {
        gt.total = ex2_approx(last.h + last.l);
        gt.at = at_chunk.c, gt.begin = at_chunk.begin, gt.end = at_chunk.end, gt.tokens = tokens_of(at_chunk);
        gt.tile = it.tile, gt.h = it.h, gt.b = (int)it.b, gt.bh = (int)it.b * g.Hv + it.h;
        gt.phi = sched.phi;
      }
      at_chunk.next(sched, n_all);
      mbar_arrive(gate_full + 8 * (c % kGateSlots));
    }
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------------- MMAs ----
    // The whole warp runs the loop, so that descriptors stay uniform, and one
    // elected lane issues: by a lane of a branch of its own a product took 50
    // cycles to issue and 32 to run.
    const bool elected = elect_one(), quiet = sched.quiet;
    constexpr uint32_t id64 = idesc_bf16(64, false);
    // D3 in two halves of its columns, where each is a block of K
    constexpr int kHalves = DK / 64;
    constexpr uint32_t id3 = idesc_bf16(64, true);
    constexpr int HK = DK / kParts;
    // products with K or Q; the output's without the smallest for bf16 tensors
    constexpr int kPairs = F32 ? 6 : 3, kSkipQ = FULL ? 0 : 1, kSkipP = FULL ? 0 : 3;
    const uint64_t kq0 = smem_desc(base), kq0_mn = smem_desc(base, 16384), t0 = smem_desc(base + L::kOffT), p0 = smem_desc(base + L::kOffP);
    auto commit = [&](uint32_t bar) {
      if (elected) mma_commit(bar);
    };
    // [K; Q] K^T of chunk c, for the prepare warps
    auto issue_d0 = [&](int c) {
      const uint64_t kq = kq0 + (uint64_t)((c % L::kKqStages) * (L::kKq / 16));
      wait_counted(kq_full + 8 * (c % L::kKqStages), c / L::kKqStages);
      if (c > 0) wait_counted(d0_empty + 8 * ((c - 1) & 1), (c - 1) / 2);
      tcgen05_fence_after();
#pragma unroll
      for (int p = 0; p < (F32 ? 6 : 1); ++p) {
        int ta = 0, tb = 0;
        if (F32) term_pair<true>(p, ta, tb);
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
          const uint64_t at = kq + (k / 4) * 1024 + 2 * (k % 4);
          if (elected) mma_ss(tmem + kColD0, at + ta * (L::kKqTerm / 16), at + tb * (L::kKqTerm / 16), id64 | neg_bits(ta, tb), p > 0 || k > 0);
        }
      }
      commit(d0_full + 8 * (c & 1));
    };
    // S times the keys (0) or the queries (1)
    auto issue_d1 = [&](int c, int part, int k0, int k1) {
      const uint64_t kq = kq0 + (uint64_t)((c % L::kKqStages) * (L::kKq / 16) + part * 512);
      const uint32_t d = tmem + (part ? kColQ : kColX);
      const int first = part ? kSkipQ : 0;
#pragma unroll
      for (int p = first; p < kPairs; ++p) {
        int ta = 0, tb = 0;
        term_pair<F32>(p, ta, tb);
#pragma unroll
        for (int k = k0; k < k1; ++k) {
          const uint32_t w = (16 * k % HK) / 2, q = 16 * k / HK;
          const uint32_t ad = (ta < 2 ? ta * (HK / 2) : DK) + w + q * (ta < 2 ? HK : HK / 2);
          if (elected)
            mma_ts(d, tmem + kColS + ad, kq + tb * (L::kKqTerm / 16) + (k / 4) * 1024 + 2 * (k % 4), id64 | neg_bits(ta, tb),
                   p > first || k > 0);
        }
      }
    };
    // the output's U P^T
    auto issue_o = [&](int c) {
      wait_counted(p_full + 8 * (c % L::kPBuffers), c / L::kPBuffers);
      wait_counted(u_ready, c);
      tcgen05_fence_after();
      const uint64_t pd = p0 + (uint64_t)((c % L::kPBuffers) * (L::kP / 16));
      if (!quiet) {
#pragma unroll
        for (int p = kSkipP; p < 6; ++p) {
          int ta = 0, tb = 0;
          term_pair<true>(p, ta, tb);
#pragma unroll
          for (int k = 0; k < kC / 16; ++k) {
            const uint32_t ad = ta < 2 ? kColU + 8 * ta + 16 * k : kColU3 + 8 * k;
            if (elected)
              mma_ts(tmem + kColO + 16 * k, tmem + ad, pd + tb * 512 + 130 * k,
                     idesc_bf16(kC - 16 * k, false) | neg_bits(ta, tb), p > kSkipP || k > 0);
          }
        }
      }
      commit(o_full);
      commit(p_empty + 8 * (c % L::kPBuffers));
    };
    issue_d0(0);
    for (int c = 0; c < n_chunks; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wait_counted(s_ready + 8 * h, c);
        tcgen05_fence_after();
        issue_d1(c, 0, h * (DK / 32), (h + 1) * (DK / 32));
      }
      commit(x_full);
      if (kLate && c > 0) issue_o(c - 1);
      if (L::kAhead > 1 && c == 0 && n_chunks > 1) issue_d0(1);
      if (kEarly) {  // S's third terms make room for the decayed U's
        if (c > 0) wait_counted(o_empty, c - 1);
        tcgen05_fence_after();  // the output's loads come before the product over them
        if (!quiet) issue_d1(c, 1, 0, DK / 16);
      }
      wait_counted(t_full, c);
      // D2 = R T^T.  T is lower triangular: 16 tokens of the contraction reach the
      // columns from their own on
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wait_counted(r_ready + 8 * h, c);
        tcgen05_fence_after();
#pragma unroll
        for (int p = 0; p < 6; ++p) {
          int ta = 0, tb = 0;
          term_pair<true>(p, ta, tb);
#pragma unroll
          for (int k = 2 * h; k < 2 * h + 2; ++k) {
            const uint32_t ad = ta < 2 ? kColX + 8 * ta + 16 * k : kEarly ? kColO + 16 * k : kColThird + 8 * k;
            if (elected)
              mma_ts(tmem + kColU + 16 * k, tmem + ad, t0 + tb * 512 + 130 * k,
                     idesc_bf16(kC - 16 * k, false) | neg_bits(ta, tb), p > 0 || k > 0);
          }
        }
      }
      commit(u_full);
      commit(t_empty + 8 * (c & 1));
      if (!kEarly) {  // the queries' product, under epilogue 2
        if (c > 0) wait_counted(o_empty, c - 1);
        tcgen05_fence_after();
        if (!quiet) issue_d1(c, 1, 0, DK / 16);
      }
      // D3 = U K; K's rows are the contraction
      const uint64_t kq_mn = kq0_mn + (uint64_t)((c % L::kKqStages) * (L::kKq / 16));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wait_counted(w_ready + 8 * h, c);
        tcgen05_fence_after();
#pragma unroll
        for (int nh = 0; nh < kHalves; ++nh) {
#pragma unroll
          for (int p = 0; p < kPairs; ++p) {
            int ta = 0, tb = 0;
            term_pair<F32>(p, ta, tb);
#pragma unroll
            for (int k = 2 * h; k < 2 * h + 2; ++k) {
              const uint32_t ad = ta < 2 ? kColX + 8 * ta + 16 * k : kColThird + 8 * k;
              if (elected)
                mma_ts(tmem + kColS + 64 * nh, tmem + ad, kq_mn + tb * (L::kKqTerm / 16) + 1024 * nh + 128 * k,
                       id3 | neg_bits(ta, tb), p > 0 || k > 0);
            }
          }
          if (h == 1) commit(s_full + 8 * nh);
        }
      }
      if (kHalves == 1) commit(s_full + 8);
      commit(kq_empty + 8 * (c % L::kKqStages));
      if (!kLate) issue_o(c);
      if (c + L::kAhead < n_chunks) issue_d0(c + L::kAhead);
    }
    if (kLate) issue_o(n_chunks - 1);
    // every MMA and commit is done before tensor memory is freed and the barriers go
    // away, after a wait that ran out too
    commit(drained);
    landed(drained, 0);
  } else {
    // --------------------------------------------------------------- load ----
    const int lt = threadIdx.x - 32 * kLoadWarp;
    // A chunk's place in the tensors.  The cursor runs two chunks ahead of the values'
    // load: that chunk's rows are prefetched, the next one's keys and queries loaded,
    // this one's values, and the output of two before stored.
    struct At {
      int tile, h, hk, b, t;
    };
    Cursor ahead;
    ahead.start(sched, n_all);
    At next = {};  // the cursor's
    auto place = [&]() {
      if (ahead.c == ahead.begin) {
        const Item it = item_of(ahead);
        next = At{it.tile, it.h, it.hk, (int)it.b, ahead.c * kC};
      } else {
        next.t += kC;
      }
      ahead.next(sched, n_all);
    };
    // a chunk's output from its place over the values
    auto store_y = [&](const At& at) {
      if (lt == 0 && !sched.quiet) {
        tma_store_4d(&map_y, base + L::kOffV, at.tile * kM, at.h, at.t, at.b);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      }
      // the other path's element-wise loads write there next
      if (!MAPS) named_barrier(4, kLoadThreads);
    };
    // a row of four values that 16-byte accesses reach
    const bool wide_kq = g.dk % 4 == 0 && g.ld_k % 4 == 0 && g.ld_q % 4 == 0 &&
                         ((reinterpret_cast<uintptr_t>(g.k) | reinterpret_cast<uintptr_t>(g.q)) & 15) == 0;
    // A chunk's rows to the second-level cache, ahead of their load: f32 rows, which are
    // read element-wise, come in a third of the time (30.4 us a chunk without), and CTAs
    // at different chunks, whose rows share no pages, took 5.9 us a chunk
    // instead of 6.5.
    auto prefetch = [&](const At& at) {
      if (!F32) {
        if (lt == 0 && MAPS) {
#pragma unroll
          for (int kb = 0; kb < L::kBlocks; ++kb) {
            tma_prefetch_4d(&map_k, 64 * kb, at.hk, at.t, at.b);
            tma_prefetch_4d(&map_q, 64 * kb, at.hk, at.t, at.b);
          }
        }
        if (lt == 0 && MAPS) tma_prefetch_4d(&map_v, at.tile * kM, at.h, at.t, at.b);
        return;
      }
      const int rows = g.T - at.t < kC ? (int)(g.T - at.t) : kC, cols = g.dv - at.tile * kM < kM ? g.dv - at.tile * kM : kM;
      const int64_t row = at.b * g.T + at.t;
      auto lines = [&](const void* p, int64_t ld, int n) {
        const float* first = reinterpret_cast<const float*>(p) + row * ld;
        for (int e = lt; e < 4 * rows; e += kLoadThreads)
          if (32 * (e & 3) < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(first + (e / 4) * ld + 32 * (e & 3)));
      };
      lines(reinterpret_cast<const float*>(g.k) + (int64_t)at.hk * g.dk, g.ld_k, g.dk);
      lines(reinterpret_cast<const float*>(g.q) + (int64_t)at.hk * g.dk, g.ld_q, g.dk);
      lines(reinterpret_cast<const float*>(g.v) + (int64_t)at.h * g.dv + at.tile * kM, g.ld_v, cols);
    };
    // Copies that this thread has started.  Once a wait has run out it starts no more: the
    // places may be in use, and a barrier takes no second copy before the first has landed.
    int kq_started = 0, v_started = 0;
    // the keys and queries of chunk c
    auto load_kq = [&](int c, const At& at) {
      const int ks = c % L::kKqStages;
      const uint32_t kq = base + ks * L::kKq;
      if (c >= L::kKqStages) wait_counted(kq_empty + 8 * ks, c / L::kKqStages + 1);
      if (MAPS) {
        // tokens past the end and components past dk read as zero
        if (lt == 0 && !*abort_flag) {
          kq_started = c + 1;
          mbar_arrive_expect_tx(kq_full + 8 * ks, L::kKqTerm);
#pragma unroll
          for (int kb = 0; kb < L::kBlocks; ++kb) {
            tma_load_4d(kq + kb * 16384, &map_k, 64 * kb, at.hk, at.t, at.b, kq_full + 8 * ks);
            tma_load_4d(kq + kb * 16384 + 8192, &map_q, 64 * kb, at.hk, at.t, at.b, kq_full + 8 * ks);
          }
        }
      } else {
        // by hand, eight components of a row at a time, kBatch of these in flight per
        // thread: K rows 0-63, Q 64-127; granule q of row r at q ^ (r % 8)
        constexpr int kBatch = 4;
        const int left = g.T - at.t < kC ? (int)(g.T - at.t) : kC;
        const In* k_base = reinterpret_cast<const In*>(g.k) + (at.b * g.T + at.t) * g.ld_k + (int64_t)at.hk * g.dk;
        const In* q_base = reinterpret_cast<const In*>(g.q) + (at.b * g.T + at.t) * g.ld_q + (int64_t)at.hk * g.dk;
#pragma unroll 1
        for (int e0 = lt; e0 < 2 * kC * (DK / 8); e0 += kBatch * kLoadThreads) {
          float f[kBatch][8];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int e = e0 + u * kLoadThreads, r = e / (DK / 8), col = e % (DK / 8) * 8, i = r & (kC - 1);
            const int valid = i < left ? g.dk - col : 0;
            const In* src = (r < kC ? k_base + (int64_t)i * g.ld_k : q_base + (int64_t)i * g.ld_q) + col;
            if (F32 && wide_kq) {
              float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
              if (valid > 0) a = *reinterpret_cast<const float4*>(src);
              if (valid > 4) b = *reinterpret_cast<const float4*>(src + 4);
              f[u][0] = a.x, f[u][1] = a.y, f[u][2] = a.z, f[u][3] = a.w;
              f[u][4] = b.x, f[u][5] = b.y, f[u][6] = b.z, f[u][7] = b.w;
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) f[u][j] = j < valid ? to_f32(src[j]) : 0.0f;
            }
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int e = e0 + u * kLoadThreads, r = e / (DK / 8), col = e % (DK / 8) * 8;
            const uint32_t dst = kq + (uint32_t)((col / 64) * 16384 + r * 128 + ((((col & 63) / 8) ^ (r & 7)) << 4));
            uint32_t x[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split3n(f[u][2 * j], f[u][2 * j + 1], x[0][j], x[1][j], x[2][j]);
#pragma unroll
            for (int p = 0; p < L::kTerms; ++p)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + p * L::kKqTerm), "r"(x[p][0]), "r"(x[p][1]),
                           "r"(x[p][2]), "r"(x[p][3])
                           : "memory");
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(kq_full + 8 * ks);
      }
    };
    At here = {}, before = {}, two_before = {};
    place();
    prefetch(next);
#pragma unroll 1
    for (int c = -1; c < n_chunks; ++c) {
      // a chunk ahead of the values, whose place is free later
      const At after = next;
      if (c + 1 < n_chunks) load_kq(c + 1, after);
      if (c + 2 < n_chunks) {
        place();
        prefetch(next);
      }
      // V (bf16); tokens past the sequence's end and components past dv are zero
      if (!F32 && c >= 0) {
        if (c > 0) wait_counted(v_empty, c - 1);
        if (!kEarly && vec_y && c > 1) store_y(two_before);
        if (MAPS) {
          if (lt == 0 && !*abort_flag) {
            v_started = c + 1;
            mbar_arrive_expect_tx(v_full, kC * kM * 2);
            tma_load_4d(base + L::kOffV, &map_v, here.tile * kM, here.h, here.t, here.b, v_full);
          }
        } else {
          const int left = g.T - here.t < kC ? (int)(g.T - here.t) : kC;
          const int cols = g.dv - here.tile * kM < kM ? g.dv - here.tile * kM : kM;
          const In* v_base = reinterpret_cast<const In*>(g.v) + (here.b * g.T + here.t) * g.ld_v + (int64_t)here.h * g.dv + here.tile * kM;
          In* v_dst = reinterpret_cast<In*>(gbase + L::kOffV);
#pragma unroll 4
          for (int e = lt; e < kC * kM; e += kLoadThreads) {
            const int r = e / kM, q = e % kM;
            v_dst[e] = r < left && q < cols ? v_base[(int64_t)r * g.ld_v + q] : from_f32<In>(0.0f);
          }
          mbar_arrive(v_full);
        }
      }
      two_before = before, before = here, here = after;
    }
    if (MAPS && lt == 0 && *abort_flag) {  // nothing may land after the CTA has ended
#pragma unroll 1
      for (int c = kq_started > L::kKqStages ? kq_started - L::kKqStages : 0; c < kq_started; ++c)
        landed(kq_full + 8 * (c % L::kKqStages), c / L::kKqStages);
      if (v_started > 0) landed(v_full, v_started - 1);
    }
    if (!kEarly) {  // the last two chunks' outputs
      wait_counted(v_empty, n_chunks - 1);
      if (vec_y && n_chunks > 1) store_y(two_before);
      if (!MAPS || lt == 0) mbar_arrive(v_full);
      wait_counted(v_empty, n_chunks);
      if (vec_y) store_y(before);
      if (lt == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(&g_delta_faults, MAMBA_FAULT_DELTA_WAIT);
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

// Tensor maps over bf16 rows ld apart, of [B][T] tokens; outside them everything
// reads as zero.  False if the layout has no such map (then the element-wise path
// loads it).
bool mappable(const void* p, int64_t T, int64_t ld, int d) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && d % 8 == 0 && T * ld * 2 < (int64_t(1) << 40) &&
         T <= INT32_MAX - kC;
}
// [B][T][H][d] by boxes of 64 (swizzled) or 128 components of one head of 64 tokens
bool make_map_heads(CUtensorMap* map, const void* p, int64_t B, int64_t T, int H, int d, int64_t ld, int box = 64) {
  auto enc = encode_fn();
  if (!enc || !mappable(p, T, ld, d)) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)(d * 2), (cuuint64_t)(ld * 2), (cuuint64_t)(T * ld * 2)};
  const cuuint32_t boxes[4] = {(cuuint32_t)box, 1, (cuuint32_t)kC, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, box == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// states [parts - 1][heads][dv][dk], phi [parts - 2][heads][dk][dk]: states[p] +=
// states[p - 1] phi[p - 1] for p = 1 .. parts - 2, kJoinRows rows of a head per CTA.
// The rows stay in shared memory and the next map is on its way while this one is
// multiplied: a thread sums 8 rows x 4 columns over an eighth of the map's rows (two
// wide loads for 32 multiplies), and the eighths are added up over the used map.
constexpr int kJoinRows = 16, kJoinThreads = 512, kJoinSplit = 8, kJoinLd = 128;
constexpr int kJoinSmem = (2 * 128 * kJoinLd + 128 * kJoinRows) * 4;
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__global__ void __launch_bounds__(kJoinThreads) join_kernel(float* states, const float* phi, int heads, int dv, int dk, int parts) {
  extern __shared__ float join_smem[];
  float* maps = join_smem;                   // [2][dk][kJoinLd]
  float* x = join_smem + 2 * 128 * kJoinLd;  // [128][kJoinRows]: column j of the rows
  const int row_tiles = (dv + kJoinRows - 1) / kJoinRows;
  const int head = blockIdx.x / row_tiles, r0 = blockIdx.x % row_tiles * kJoinRows;
  const int64_t step = (int64_t)heads * dv * dk;
  float* s = states + ((int64_t)head * dv + r0) * dk;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c0 = lane * 4, q0 = warp % 2 * 8, split = warp / 2;  // columns, rows, eighth
  const int j0 = split * dk / kJoinSplit, j1 = (split + 1) * dk / kJoinSplit;
  auto fetch = [&](int p) {  // phi[p - 1], 16 bytes at a time where its rows allow
    const float* f = phi + ((int64_t)(p - 1) * heads + head) * dk * dk;
    float* to = maps + (p & 1) * 128 * kJoinLd;
    if (dk % 4 == 0) {
      if (c0 < dk)
        for (int j = warp; j < dk; j += kJoinThreads / 32) cp_async16(smem_u32(to + j * kJoinLd + c0), f + j * dk + c0);
    } else {
      for (int j = warp; j < dk; j += kJoinThreads / 32)
        for (int c = lane; c < dk; c += 32) to[j * kJoinLd + c] = f[j * dk + c];
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (parts > 2) fetch(1);
  for (int i = threadIdx.x; i < kJoinRows * dk; i += kJoinThreads)
    x[i % dk * kJoinRows + i / dk] = r0 + i / dk < dv ? s[(int64_t)(i / dk) * dk + i % dk] : 0.0f;
  // The sums that this thread joins and keeps: row `warp`, columns c0 .. c0 + 3.
  const bool mine = r0 + warp < dv;
  for (int p = 1; p <= parts - 2; ++p) {
    if (p + 1 <= parts - 2) fetch(p + 1);
    float* next = s + p * step + (int64_t)warp * dk + c0;
    float sum[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) sum[c] = mine && c0 + c < dk ? next[c] : 0.0f;
    if (p + 1 <= parts - 2)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* m = maps + (p & 1) * 128 * kJoinLd;
    float acc[8][4] = {};
#pragma unroll 4
    for (int j = j0; j < j1; ++j) {
      const float4 f = *reinterpret_cast<const float4*>(m + j * kJoinLd + c0);
      const float4 u = *reinterpret_cast<const float4*>(x + j * kJoinRows + q0);
      const float4 v = *reinterpret_cast<const float4*>(x + j * kJoinRows + q0 + 4);
      const float fs[4] = {f.x, f.y, f.z, f.w}, xs[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(xs[r], fs[c], acc[r][c]);
    }
    __syncthreads();  // the map and the rows are read
#pragma unroll
    for (int r = 0; r < 8; ++r)
      *reinterpret_cast<float4*>(m + (split * kJoinRows + q0 + r) * kJoinLd + c0) =
          make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kJoinSplit; ++e) {
      const float4 f = *reinterpret_cast<const float4*>(m + (e * kJoinRows + warp) * kJoinLd + c0);
      sum[0] += f.x, sum[1] += f.y, sum[2] += f.z, sum[3] += f.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c0 + c < dk) {
        x[(c0 + c) * kJoinRows + warp] = sum[c];
        if (mine) next[c] = sum[c];
      }
    __syncthreads();
  }
}

struct Maps {
  CUtensorMap k, q, v, y;
  bool inputs, y_too;  // which there are
};

template <int DK, bool F32, bool MAPS, bool FULL>
cudaError_t launch_chunk(const GatedDeltaArgs& a, const Maps& maps, const Plan& plan, int ctas, cudaStream_t stream) {
  auto kern = chunk_kernel<DK, F32, MAPS, FULL>;
  constexpr int smem = Smem<DK, F32, FULL>::kAlloc;
  static int configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!__atomic_load_n(&configured[dev], __ATOMIC_RELAXED)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSmem)) != cudaSuccess)
      return e;
    __atomic_store_n(&configured[dev], 1, __ATOMIC_RELAXED);
  }
  auto launch = [&](const Plan& plan, int ctas) {
    kern<<<(unsigned)ctas, kThreads, smem, stream>>>(a, maps.k, maps.q, maps.v, maps.y, maps.y_too, plan);
    return cudaGetLastError();
  };
  if (plan.mode == kWide) {
    if (plan.flags && (e = cudaMemsetAsync(plan.flags, 0, (size_t)ctas * sizeof(int), stream)) != cudaSuccess) return e;
    return launch(plan, ctas);
  }
  const int heads = (int)(a.B * a.Hv);
  if ((e = launch(plan, plan.items * (plan.parts - 1) + heads * (plan.parts - 2))) != cudaSuccess) return e;
  const int row_tiles = (a.dv + kJoinRows - 1) / kJoinRows;
  join_kernel<<<(unsigned)(heads * row_tiles), kJoinThreads, kJoinSmem, stream>>>(plan.states, plan.phi, heads, a.dv, a.dk, plan.parts);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  Plan second = plan;
  second.mode = kPartsPass;
  return launch(second, plan.items * plan.parts);
}

// The layout of a call over `sms` SMs, and the scratch that it wants; with less
// (ws_bytes) items are not cut.  Returns the CTAs of a kWide launch.
//
// Cutting few items into P parts makes n chunks in a row n / P in each of two launches
// and P - 2 join steps, if the parts' CTAs and the maps' fit the SMs.  By type and key
// size, fitted to 1 to 48 heads of 4 to 64 chunks, whole and in 3 to 32 parts (us
// between events around a call): whole 25 + chunk n, in parts parts + 1.87 chunk n / P +
// join (P - 2).
// The choice was within 8 % of the best of all at each, and the same but for 1 % in the
// mean.  12 heads of 64 x 64, 12 chunks, f32: 71 us in 6 parts, 102 whole; bf16 62 and
// 71; of 128 x 128 f32 106 and 175; 20 chunks bf16 in 7 parts 86 and 114.
constexpr double kStartUs = 25, kPassesUs = 1.87;
struct PlanCosts {
  double chunk, parts, join;
};
PlanCosts plan_costs(const GatedDeltaArgs& a) {
  if (a.dk <= 64) return PlanCosts{a.in_bf16 ? 3.8 : 6.4, 38, 2.2};
  return PlanCosts{a.in_bf16 ? 4.4 : 13.1, 47, 3.5};
}
int make_plan(const GatedDeltaArgs& a, int sms, int64_t ws_bytes, char* ws, Plan* p, int64_t* want) {
  *p = Plan{};
  p->n_chunks = (int)((a.T + kC - 1) / kC);
  p->tiles = (a.dv + kM - 1) / kM;
  const int64_t heads = a.B * a.Hv, items = heads * p->tiles;
  p->items = (int)items;
  *want = 0;
  auto round256 = [](int64_t b) { return (b + 255) / 256 * 256; };
  // Whole items leave the SMs of the last round idle; cut, they cost the states' way
  // from CTA to CTA and chunks that share no pages.  4096 tokens: 320 items 719 us cut,
  // 896 whole; 240 items 564 and 625, of 1024 tokens 175 and 177.
  const int64_t rounds = (items + sms - 1) / sms;
  if (items > sms && rounds * sms * 4 > items * 5) {
    const int64_t states = (int64_t)sms * kM * a.dk * 4;
    *want = round256(states) + round256(sms * (int64_t)sizeof(int));
    if (ws && ws_bytes >= *want) {
      p->states = reinterpret_cast<float*>(ws);
      p->flags = reinterpret_cast<int*>(ws + round256(states));
      return sms;
    }
    return p->items;
  }
  if (items > sms) return p->items;
  int best = 1;
  const PlanCosts cost = plan_costs(a);
  double best_us = 0.95 * (kStartUs + cost.chunk * p->n_chunks);  // worth three launches for a twentieth
  for (int parts = 3; parts <= p->n_chunks && items * parts <= sms && items * (parts - 1) + heads * (parts - 2) <= sms; ++parts) {
    const int len = (p->n_chunks + parts - 1) / parts;
    if ((parts - 1) * len >= p->n_chunks) continue;  // the last part would be empty
    const double us = cost.parts + kPassesUs * cost.chunk * len + cost.join * (parts - 2);
    if (us < best_us) best = parts, best_us = us;
  }
  if (best > 1) {
    const int64_t one = round256(heads * a.dv * a.dk * 4), states = heads * a.dv * a.dk * 4 * (best - 1);
    const int64_t phi = heads * a.dk * a.dk * 4 * (int64_t)(best - 2);
    *want = one + round256(states) + round256(phi);
    if (ws && ws_bytes >= *want) {
      p->mode = kAheadPass;
      p->parts = best, p->part_len = (p->n_chunks + best - 1) / best;
      p->first = reinterpret_cast<float*>(ws);
      p->states = reinterpret_cast<float*>(ws + one);
      p->phi = reinterpret_cast<float*>(ws + one + round256(states));
    }
  }
  return p->items;
}

}  // namespace

// Up to 16 tokens go token by token: 40 heads of 16 tokens 18.6 us against 18.6 for
// a chunk (8 tokens 10.5, 32 tokens 31.0 against 18.5); 8 heads 11.2 against 16.9 (32
// tokens 18.7 and 16.8); 1024 heads 121 against 107 (12 tokens 94).  Items and chunk
// numbers, and output offsets inside a chunk, are 32 bits.
bool gated_delta_takes_chunks(const GatedDeltaArgs& a) {
  return a.dk <= 128 && a.T > 16 && a.ld_y < (int64_t(1) << 23) && a.T < (int64_t(1) << 30) &&
         a.B * a.Hv * ((a.dv + kM - 1) / kM) < (int64_t(1) << 30);
}

int64_t gated_delta_chunk_workspace(const GatedDeltaArgs& a, const DeviceInfo& dev) {
  Plan plan;
  int64_t want = 0;
  make_plan(a, dev.sm_count, 0, nullptr, &plan, &want);
  return want;
}

cudaError_t launch_gated_delta_chunk(const GatedDeltaArgs& a, const DeviceInfo& dev, void* ws, int64_t ws_bytes,
                                     cudaStream_t stream) {
  if (a.B <= 0 || a.Hv <= 0 || a.dv <= 0) return cudaSuccess;
  Plan plan;
  int64_t want = 0;
  const int ctas = make_plan(a, dev.sm_count, ws_bytes, static_cast<char*>(ws), &plan, &want);
  Maps maps = {};
  if (!a.in_bf16) {
    return a.dk <= 64 ? launch_chunk<64, true, false, true>(a, maps, plan, ctas, stream)
                      : launch_chunk<128, true, false, true>(a, maps, plan, ctas, stream);
  }
  maps.inputs = make_map_heads(&maps.k, a.k, a.B, a.T, a.Hk, a.dk, a.ld_k) &&
                make_map_heads(&maps.q, a.q, a.B, a.T, a.Hk, a.dk, a.ld_q) &&
                make_map_heads(&maps.v, a.v, a.B, a.T, a.Hv, a.dv, a.ld_v, kM) &&
                ((reinterpret_cast<uintptr_t>(a.state_in) | reinterpret_cast<uintptr_t>(a.state_out)) & 15) == 0;
  maps.y_too = a.y_bf16 && make_map_heads(&maps.y, a.y, a.B, a.T, a.Hv, a.dv, a.ld_y, kM);
  // All terms wherever y keeps 32 bits, and with dk <= 64, where they cost little (152
  // heads of 4096 tokens 308 us against 303, 12 heads 269 and 260).  With dk > 64 they put
  // the output on the path from state to state (12 heads of 4096 tokens 325 us against
  // 300, 3 x 101 tokens 20.5 and 18.5), which a bf16 y, rounded to 2^-9, does not need.
  if (a.dk <= 64)
    return maps.inputs ? launch_chunk<64, false, true, true>(a, maps, plan, ctas, stream)
                       : launch_chunk<64, false, false, true>(a, maps, plan, ctas, stream);
  if (a.y_bf16)
    return maps.inputs ? launch_chunk<128, false, true, false>(a, maps, plan, ctas, stream)
                       : launch_chunk<128, false, false, false>(a, maps, plan, ctas, stream);
  return maps.inputs ? launch_chunk<128, false, true, true>(a, maps, plan, ctas, stream)
                     : launch_chunk<128, false, false, true>(a, maps, plan, ctas, stream);
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
