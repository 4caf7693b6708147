// What the kernels on whole rows of logits share: log probabilities
// (token_logprobs.cu), distillation losses (distill.cu) and the gradients of both
// (row_grad.cuh).
//
// A row belongs to one CTA, or to those of a cluster where rows are few or, for
// gradients, longer than three slices on an SM.  Losses and log probabilities read
// their part of it once through registers; gradients keep their slice in shared
// memory between the sums and the gradient (the log probabilities of 4093 rows of
// 152064 through shared memory: 594 us, 200 through registers).  The CTAs' sums
// meet in distributed shared memory; one cluster barrier per row.
//
// Mathematics: with m near the maximum and c = log2(e) / T,
//   Z = sum 2^((z - m) c),  S = sum 2^((z - m) c) (z - m),
//   ln p_j = (z_j - m) / T - ln Z,  H = ln Z - S / (T Z).
// Parts with references m_i join as Z = sum Z_i w_i, S = sum w_i (S_i + Z_i (m_i -
// m)), w_i = 2^((m_i - m) c): a warp takes its own maximum as its reference, a
// CTA joins its warps and every CTA the cluster's.
//
// Bound: HBM for binary32; in bf16 the instructions for two elements in four bytes
// come near it (two conversions, a maximum, a subtraction, a multiplication, an
// exponential at 32 per cycle and SM, a sum: half of the issue slots at full
// bandwidth), so that what follows a row's last byte shows.
#pragma once

#include <limits.h>

#include <algorithm>

#include "cache.cuh"
#include "launch.h"
#include "smp_scores.h"
#include "tma.cuh"

namespace smp {

constexpr int kRowBadToken = 128;
constexpr int kMaxIds = SMP_MAX_ROW_IDS;
constexpr int kMaxRanks = 16;
constexpr int kMaxParts = 8;   // CTAs of a row that is streamed

// The rows of a call, as every kernel here gets them.
struct RowsArgs {
  const void* logits;
  int64_t stride;
  int rows, vocab;
  int slice;          // elements per CTA, whole vectors
  float temperature;
  const float* temperatures;
  int32_t* status;
  uint64_t wait_limit;
  int first_round;    // CTAs that may stand before the kernel ahead has ended
};

// The statistics of some elements: a reference that none exceeds by more than 2^16
// of weight, sum 2^((z - m) c) and, where wanted, the same weighted by z - m.  No
// elements: -inf, 0, 0; +inf among them: m is +inf.
struct Stats {
  float m, z, s;
};

// ------------------------------------------------------------------ elements

constexpr float kLog2e = 0x1.715476p+0f;

template <typename T>
struct RowVec;
template <>
struct RowVec<uint16_t> {
  static constexpr int kPer = 8;
  static constexpr uint32_t kNegInf2 = 0xFF80FF80u;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {   // NaN only if both are
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t top(const uint4& x, uint32_t so_far) {
    return max2(so_far, max2(max2(x.x, x.y), max2(x.z, x.w)));
  }
  static __device__ __forceinline__ float finish(uint32_t m) {
    return fmaxf(__uint_as_float(m & 0xFFFF0000u), __uint_as_float(m << 16));
  }
  // The eight values, none below `floor` (both halves of a word), NaN as floor.
  static __device__ __forceinline__ void get(const uint4& x, uint32_t floor, float (&v)[8]) {
    const uint32_t w[4] = {max2(x.x, floor), max2(x.y, floor), max2(x.z, floor), max2(x.w, floor)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_low(w[i]), v[2 * i + 1] = bf16_high(w[i]);
  }
  static __device__ __forceinline__ void get(const uint4& x, uint32_t floor, uint64_t (&v)[4]) {
    const uint32_t w[4] = {max2(x.x, floor), max2(x.y, floor), max2(x.z, floor), max2(x.w, floor)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("mov.b64 %0, {%1, %2};" : "=l"(v[i]) : "f"(bf16_low(w[i])), "f"(bf16_high(w[i])));
  }
  // The eight values as they are.
  static __device__ __forceinline__ void raw(const uint4& x, uint64_t (&v)[4]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("mov.b64 %0, {%1, %2};" : "=l"(v[i]) : "f"(bf16_low(w[i])), "f"(bf16_high(w[i])));
  }
  // The values rounded, their signs turned by `sign` (of both halves of a word).
  static __device__ __forceinline__ uint4 put(const float (&v)[8], uint32_t sign) {
    return make_uint4(pack_bf16(v[0], v[1]) ^ sign, pack_bf16(v[2], v[3]) ^ sign, pack_bf16(v[4], v[5]) ^ sign,
                      pack_bf16(v[6], v[7]) ^ sign);
  }
  static constexpr uint32_t kSign = 0x80008000u;
  static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
  static __device__ __forceinline__ uint16_t minus_inf() { return 0xFF80u; }
  // The largest value <= x that both halves of a word can hold.
  static __device__ __forceinline__ uint32_t below(float x) {
    const uint32_t b = __float_as_uint(x);
    const uint32_t h = (b >> 16) + ((b & 0xFFFFu) && (b >> 31) ? 1u : 0u);
    return h | (h << 16);
  }
  static __device__ __forceinline__ float value(uint32_t w) { return bf16_low(w); }
};
template <>
struct RowVec<float> {
  static constexpr int kPer = 4;
  static constexpr uint32_t kNegInf2 = 0xFF800000u;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ uint32_t top(const uint4& x, uint32_t so_far) {
    return max2(so_far, max2(max2(x.x, x.y), max2(x.z, x.w)));
  }
  static __device__ __forceinline__ float finish(uint32_t m) { return __uint_as_float(m); }
  static __device__ __forceinline__ void get(const uint4& x, uint32_t floor, float (&v)[4]) {
    v[0] = __uint_as_float(max2(x.x, floor)), v[1] = __uint_as_float(max2(x.y, floor));
    v[2] = __uint_as_float(max2(x.z, floor)), v[3] = __uint_as_float(max2(x.w, floor));
  }
  static __device__ __forceinline__ void get(const uint4& x, uint32_t floor, uint64_t (&v)[2]) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v[0]) : "r"(max2(x.x, floor)), "r"(max2(x.y, floor)));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v[1]) : "r"(max2(x.z, floor)), "r"(max2(x.w, floor)));
  }
  static __device__ __forceinline__ void raw(const uint4& x, uint64_t (&v)[2]) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v[0]) : "r"(x.x), "r"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v[1]) : "r"(x.z), "r"(x.w));
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[4], uint32_t sign) {
    return make_uint4(__float_as_uint(v[0]) ^ sign, __float_as_uint(v[1]) ^ sign, __float_as_uint(v[2]) ^ sign,
                      __float_as_uint(v[3]) ^ sign);
  }
  static constexpr uint32_t kSign = 0x80000000u;
  static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  static __device__ __forceinline__ float minus_inf() { return __uint_as_float(0xFF800000u); }
  static __device__ __forceinline__ uint32_t below(float x) { return __float_as_uint(x); }
  static __device__ __forceinline__ float value(uint32_t w) { return __uint_as_float(w); }
};

// Words that elements far below the reference m are raised to before they enter
// sums, so that -inf, NaN and masks of the type's lowest value give a weight of
// exactly 0 and no 0 * inf: at least 175 T below m (2^-252 of it), or the next
// value below m where T is less than m's own spacing, and finite.  Below the
// type's lowest value there is only -inf: then every other element equals m, and
// sums weighted with z - m are 0 without looking.
template <typename T>
__device__ __forceinline__ bool is_lowest(float m) {
  return m <= (RowVec<T>::kPer == 8 ? -0x1.fep+127f : -0x1.fffffep+127f);
}
template <typename T>
__device__ __forceinline__ uint32_t floor_word(float m, float temperature) {
  using V = RowVec<T>;
  if (is_lowest<T>(m)) return V::kNegInf2;
  const float lowest = V::kPer == 8 ? -0x1.fep+127f : -0x1.fffffep+127f;
  uint32_t w = V::below(fmaxf(__fmaf_rn(-175.0f, temperature, m), lowest));
  if (V::value(w) >= m) {   // one step down: away from 0 for negative values, and across it
    uint32_t b = V::kPer == 8 ? w & 0xFFFFu : w;
    const uint32_t sign = V::kPer == 8 ? 0x8000u : 0x80000000u;
    b = b == 0u ? sign + 1u : b & sign ? b + 1u : b - 1u;
    w = V::kPer == 8 ? b | (b << 16) : b;
  }
  return w;
}

// A logit as the sampler reads it: NaN is -inf.
__device__ __forceinline__ float clean(float z) { return z == z ? z : __uint_as_float(0xFF800000u); }

// ------------------------------------------------------------------ sums

// Floats in the order of signed integers (no NaN); its own inverse.
__device__ __forceinline__ int float_order(int bits) { return bits ^ ((bits >> 31) & 0x7FFFFFFF); }
__device__ __forceinline__ float warp_max_f(float v) {
  return __int_as_float(float_order(__reduce_max_sync(~0u, float_order(__float_as_int(v)))));
}
__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Two binary32 numbers in one register pair, and operations on both.
typedef uint64_t pair_t;
__device__ __forceinline__ pair_t pair(float a, float b) {
  pair_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ pair_t both(float x) { return pair(x, x); }
__device__ __forceinline__ void parts(pair_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) {
  pair_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
  pair_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
  pair_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float sum_of(pair_t v) {
  float a, b;
  parts(v, a, b);
  return a + b;
}
__device__ __forceinline__ pair_t ex2_both(pair_t y) {
  float a, b;
  parts(y, a, b);
  return pair(ex2_approx(a), ex2_approx(b));
}

// The running statistics of one thread's elements: a group of vectors is taken
// in at a time, relative to an element m that none exceeds by more than 2^16 of
// weight (a reference that follows every new maximum changed in some lane of the
// warp at almost every group: 1.2 of 7.6 instructions per element).
template <typename T, bool kWeighted>
struct Running {
  using V = RowVec<T>;
  float m = -INFINITY;
  pair_t z = 0, s = 0, minus_m = 0;
  uint32_t floor = 0;

  // The largest of the elements that come next.
  __device__ __forceinline__ void raise(float top, float temperature, float c) {
    if (__fmul_rn(__fsub_rn(top, m), c) > 16.0f) {
      if (m > -INFINITY) {
        const float d = __fsub_rn(m, top), w = ex2_approx(__fmul_rn(d, c));
        if (kWeighted) s = w == 0.0f ? 0 : mul2(fma2(z, both(d), s), both(w));
        z = mul2(z, both(w));
      }
      m = top;
      minus_m = both(-m);
      floor = floor_word<T>(m, temperature);
    }
  }
  // Vectors that m is fit for; m is not -inf.  Their weights are summed before they
  // enter the thread's sums, which so take a rounding per call and not one per
  // element.
  template <int kN>
  __device__ __forceinline__ void add(const uint4 (&y)[kN], float c) {
    pair_t sum = 0, weighted = 0;
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      pair_t v[V::kPer / 2];
      V::get(y[u], floor, v);
#pragma unroll
      for (int i = 0; i < V::kPer / 2; ++i) {
        const pair_t d = add2(v[i], minus_m), e = ex2_both(mul2(d, both(c)));
        sum = u + i == 0 ? e : add2(sum, e);
        if (kWeighted) weighted = u + i == 0 ? mul2(e, d) : fma2(e, d, weighted);
      }
    }
    z = add2(z, sum);
    if (kWeighted) s = add2(s, weighted);
  }
  // Any vectors.
  template <int kN>
  __device__ __forceinline__ void take(const uint4 (&y)[kN], float temperature, float c) {
    uint32_t w = V::kNegInf2;
#pragma unroll
    for (int u = 0; u < kN; ++u) w = V::top(y[u], w);
    raise(V::finish(w), temperature, c);
    if (m > -INFINITY) add(y, c);
  }
  __device__ __forceinline__ void add_one(float v, float temperature, float c) {   // clean
    if (v > -INFINITY) {
      raise(v, temperature, c);
      const float d = __fsub_rn(v, m), e = ex2_approx(__fmul_rn(d, c));
      z = add2(z, pair(e, 0.0f));
      if (kWeighted && e > 0.0f) s = add2(s, pair(__fmul_rn(e, d), 0.0f));
    }
  }
  __device__ __forceinline__ Stats stats() const {
    return Stats{m, sum_of(z), kWeighted && !is_lowest<T>(m) ? sum_of(s) : 0.0f};
  }
};

// The statistics of the lanes' parts together, in every lane.
template <bool kWeighted>
__device__ __forceinline__ Stats warp_join(const Stats& part, float c) {
  Stats out;
  out.m = warp_max_f(part.m);
  float z = 0.0f, s = 0.0f;
  if (part.z != 0.0f) {
    const float d = __fsub_rn(part.m, out.m), w = ex2_approx(__fmul_rn(d, c));
    z = part.z * w;
    if (kWeighted) s = w == 0.0f ? 0.0f : w * __fmaf_rn(part.z, d, part.s);
  }
  out.z = warp_sum_f(z);
  out.s = kWeighted ? warp_sum_f(s) : 0.0f;
  return out;
}

// ------------------------------------------------------------------ a part of a row, read once from memory

// Elements [lo, hi) of a row, whole vectors [full0, full1) of 16 bytes counted
// from element `first`; thread t of kThr takes vectors full0 + t, full0 + t + kThr,
// ... and the edge threads one element each outside them.
template <typename T>
struct Part {
  static constexpr int kPer = RowVec<T>::kPer;
  const T* row;
  int first, lo, hi, full0, full1;

  __device__ __forceinline__ Part(const T* r, int vocab, int slice, int rank) : row(r) {
    first = rank * slice - int((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
    lo = max(first, 0), hi = max(lo, min(first + slice, vocab));
    full0 = first < 0 ? 1 : 0;
    full1 = hi > lo ? max(full0, (hi - first) / kPer) : full0;
  }
  __device__ __forceinline__ bool holds(int id) const { return id >= lo && id < hi; }
  __device__ __forceinline__ const uint4* vec() const { return reinterpret_cast<const uint4*>(row + first); }
  // The id of this thread's edge element, or -1.
  __device__ __forceinline__ int edge() const {
    const int t = int(threadIdx.x), id = t < kPer ? first + t : first + full1 * kPer + t - kPer;
    return t < 2 * kPer && (t >= kPer || full0 == 1) && holds(id) ? id : -1;
  }
};

// Before a CTA waits for the kernel ahead: L2, where both see the same bytes, is asked
// for the first `most` vectors of its part.  160 losses of 32000 in bf16 6.6 us and
// not 6.9 with 32 KB, 37 gradients of 50021 in binary32 7.8 and not 8.5 with 64 KB; 256
// log probabilities of 128256 20.4 and not 20.8 with 32 KB, 21.2 with 64 KB.
__device__ __forceinline__ void ask_early(const RowsArgs& r, const uint4* from, int vectors, int most) {
  constexpr int kPiece = 512;
  const int at = int(threadIdx.x) * kPiece, n = min(vectors, most);
  if (int(blockIdx.x) < r.first_round && threadIdx.x < 32 && at < n)
    prefetch_l2(reinterpret_cast<uintptr_t>(from + at), uint32_t(min(kPiece, n - at)) * 16u);
}

// A vector past the L1 cache, of memory that the kernel does not write.
__device__ __forceinline__ uint4 load_vector(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

constexpr int kUnit = 4;     // vectors of a thread that are loaded and taken in together

// Takes the part's whole vectors into `run`, a unit per thread at a time: while
// one unit is taken in, the next is on its way.  change(y, k) may alter vector k
// (from the first whole one) first; seen(top) gets the largest element of each
// unit, in order.
template <int kThr, typename T, bool kWeighted, typename Change, typename Seen>
__device__ __forceinline__ void stream(const Part<T>& s, Running<T, kWeighted>& run, float temperature,
                                       float c, Change&& change, Seen&& seen) {
  using V = RowVec<T>;
  constexpr int kStep = kUnit * kThr;
  const int vecs = s.full1 - s.full0, pairs = vecs / (2 * kStep);
  uint4 x[2][kUnit];
  const uint4* p = s.vec() + s.full0 + threadIdx.x;
  auto load = [&](uint4 (&y)[kUnit], const uint4* from) {
#pragma unroll
    for (int u = 0; u < kUnit; ++u) y[u] = load_vector(from + u * kThr);
  };
  auto load_some = [&](uint4 (&y)[kUnit], int unit) {
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      y[u] = make_uint4(V::kNegInf2, V::kNegInf2, V::kNegInf2, V::kNegInf2);
      if (int(threadIdx.x) + unit * kStep + u * kThr < vecs) y[u] = load_vector(p + unit * kStep + u * kThr);
    }
  };
  auto take = [&](uint4 (&y)[kUnit], int unit) {
    uint32_t w = V::kNegInf2;
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      change(y[u], int(threadIdx.x) + (unit * kUnit + u) * kThr);
      w = V::top(y[u], w);
    }
    const float top = V::finish(w);
    run.raise(top, temperature, c);
    if (run.m > -INFINITY) run.add(y, c);
    seen(top);
  };
  if (pairs > 0) {
    load(x[0], p), load(x[1], p + kStep);
    for (int q = 0;; ++q) {
      take(x[0], 2 * q);
      if (q + 1 == pairs) break;
      load(x[0], p + (2 * q + 2) * kStep);
      take(x[1], 2 * q + 1);
      load(x[1], p + (2 * q + 3) * kStep);
    }
    load_some(x[0], 2 * pairs);
    take(x[1], 2 * pairs - 1);
  } else {
    load_some(x[0], 0);
  }
  if (2 * pairs * kStep < vecs) {   // what two whole units leave
    load_some(x[1], 2 * pairs + 1);
    take(x[0], 2 * pairs);
    if ((2 * pairs + 1) * kStep < vecs) take(x[1], 2 * pairs + 1);
  }
}

// Barrier of a CTA's first kThr threads, the ones that work on whole rows.
template <int kThr>
__device__ __forceinline__ void workers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThr) : "memory");
}

// The same, and whether the predicate holds for one of them.
template <int kThr>
__device__ __forceinline__ bool workers_any(bool pred) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(int(pred)), "n"(kThr)
      : "memory");
  return r != 0;
}

// What the CTAs of a cluster tell one another, and the room their warps meet in.
struct Meeting {
  Stats warp[kWarps];
  alignas(16) float mail[kMaxRanks][4];
};

// A CTA's four numbers to every CTA of the cluster (lane r of the calling warp
// writes to rank r).
__device__ __forceinline__ void post(Meeting& meet, int rank, int ranks, float a, float b, float c, float d) {
  const int lane = int(threadIdx.x) & 31;
  if (ranks == 1) {
    if (lane == 0) *reinterpret_cast<float4*>(meet.mail[0]) = make_float4(a, b, c, d);
  } else if (lane < ranks) {
    const uint32_t to = map_rank(smem_addr(meet.mail[rank]), uint32_t(lane));
    st_cluster_u64(to, uint64_t(__float_as_uint(b)) << 32 | __float_as_uint(a));
    st_cluster_u64(to + 8, uint64_t(__float_as_uint(d)) << 32 | __float_as_uint(c));
  }
}
__device__ __forceinline__ float4 posted(const Meeting& meet, int ranks) {
  const int lane = int(threadIdx.x) & 31;
  return lane < ranks ? *reinterpret_cast<const float4*>(meet.mail[lane]) : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
}

// "This CTA runs": arrive early, wait before the first write to another CTA.
__device__ __forceinline__ void cluster_arrive_early(int ranks) {
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");
}
__device__ __forceinline__ void cluster_all_run(int ranks) {
  if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// Everything posted before is there after.
__device__ __forceinline__ void cluster_meet(int ranks) {
  if (ranks > 1) hw_cluster_sync();
  else __syncthreads();
}

__device__ __forceinline__ float row_temperature(const RowsArgs& a, int row) {
  return a.temperatures ? a.temperatures[row] : a.temperature;
}
__device__ __forceinline__ bool temperature_fits(float t) { return t >= SMP_MIN_TEMPERATURE && t <= SMP_MAX_TEMPERATURE; }

// Vector x without the elements whose bits are set.
__device__ __forceinline__ void erase(uint4& x, uint32_t bits, uint16_t) {
  uint32_t* w[4] = {&x.x, &x.y, &x.z, &x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bits >> (2 * i) & 1u) *w[i] = (*w[i] & 0xFFFF0000u) | 0xFF80u;
    if (bits >> (2 * i + 1) & 1u) *w[i] = (*w[i] & 0xFFFFu) | 0xFF800000u;
  }
}
__device__ __forceinline__ void erase(uint4& x, uint32_t bits, float) {
  uint32_t* w[4] = {&x.x, &x.y, &x.z, &x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (bits >> i & 1u) *w[i] = RowVec<float>::kNegInf2;
}

// Both statistics together: m, Z and the factors 2^((m_i - m) c).
struct Whole {
  float m, zsum, reach, ids_reach;
  __device__ __forceinline__ Whole(const Stats& r, const Stats& k, float c) {
    m = fmaxf(r.m, k.m);
    reach = r.z > 0.0f ? ex2_approx(__fmul_rn(__fsub_rn(r.m, m), c)) : 0.0f;
    ids_reach = k.z > 0.0f ? ex2_approx(__fmul_rn(__fsub_rn(k.m, m), c)) : 0.0f;
    zsum = __fadd_rn(r.z > 0.0f ? __fmul_rn(r.z, reach) : 0.0f, k.z > 0.0f ? __fmul_rn(k.z, ids_reach) : 0.0f);
  }
};

// The row's loss, in one warp, from the statistics outside the teacher's ids (r)
// and of the whole row (m, zsum): the places' ids (-1: none), their t and the
// student's logits there, sum t ln t, and the teacher's mass outside them.
__device__ __forceinline__ float row_loss(const int* ids, const float* t, const float* student, int room, float t_log_t,
                                          const Stats& r, float m, float zsum, float rest, float temperature) {
  const int lane = int(threadIdx.x) & 31;
  const float log_z = logf(zsum);
  float loss = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxIds / 32; ++i) {
    const int n = lane + 32 * i;
    if (n < room && ids[n] >= 0 && t[n] > 0.0f) {   // -t ln s, with t times a far logit before the division, which it might overflow
      const float far = __fdiv_rn(__fmul_rn(t[n], __fsub_rn(student[n], m)), temperature);
      loss = __fadd_rn(loss, __fsub_rn(__fmul_rn(t[n], log_z), far));
    }
  }
  loss = __fadd_rn(warp_sum_f(loss), t_log_t);
  if (rest > 0.0f) {
    const float far = __fdiv_rn(__fmul_rn(rest, __fsub_rn(r.m, m)), temperature);
    loss = __fadd_rn(loss, __fsub_rn(__fmul_rn(rest, __fadd_rn(logf(rest), __fsub_rn(log_z, logf(r.z)))), far));
  }
  return loss;
}

// ------------------------------------------------------------------ host

// Checks that the calls on rows share.
inline smp_status check_rows(const void* logits, int32_t rows, int32_t vocab, int64_t stride, smp_dtype dtype,
                             float temperature, const float* temperatures, const int32_t* status) {
  if (dtype != SMP_F32 && dtype != SMP_BF16) return SMP_ERR_DTYPE;
  if (rows < 0 || rows > (1 << 24) || vocab <= 0 || stride < vocab || stride > (int64_t(1) << 40)) return SMP_ERR_INVALID_ARG;
  if (vocab > SMP_MAX_VOCAB) return SMP_ERR_UNSUPPORTED;
  if (!temperatures && !(temperature >= SMP_MIN_TEMPERATURE && temperature <= SMP_MAX_TEMPERATURE)) return SMP_ERR_INVALID_ARG;
  if ((rows > 0 && !logits) || misaligned(logits, dtype == SMP_F32 ? 4 : 2) || misaligned(temperatures, 4) ||
      misaligned(status, 4))
    return SMP_ERR_INVALID_ARG;
  return SMP_OK;
}

// A gradient's rows: in the logits' place, or where they share no element with them
// (as two halves of wider rows, of one stride, do not).
inline bool grad_fits(const void* logits, int32_t rows, int32_t vocab, int64_t stride, smp_dtype dtype, const void* grad,
                      int64_t grad_stride) {
  if (grad_stride < vocab || grad_stride > (int64_t(1) << 40)) return false;
  if (rows <= 0) return true;
  if (grad == logits) return rows == 1 || grad_stride == stride;
  const int64_t elem = dtype == SMP_F32 ? 4 : 2;
  const uintptr_t z = reinterpret_cast<uintptr_t>(logits), g = reinterpret_cast<uintptr_t>(grad);
  const uintptr_t z_bytes = uintptr_t(((rows - 1) * stride + vocab) * elem), g_bytes = uintptr_t(((rows - 1) * grad_stride + vocab) * elem);
  if (g >= z + z_bytes || z >= g + g_bytes) return true;
  if (rows == 1 || grad_stride != stride) return false;
  const int64_t apart = int64_t(g > z ? g - z : z - g) % (stride * elem);   // of a row and the other's last before it
  return apart >= vocab * elem && apart <= (stride - vocab) * elem;
}

// The launch of a kernel whose CTAs read their parts of a row from memory once: a
// row per CTA, or parts of it while all of them fit on the SMs together, three on
// each, and are of 30 KB at least, or of `least` while each has an SM of its own.
// Losses of 150 rows of 32000 in bf16: 6.5 us with two CTAs a row, 7.2 with one,
// 8.1 with four (a second wave); of 8192 in binary32: 4.6, 4.6 and 6.7; of 8 rows of
// 32000 in bf16 4.2 with four and 4.6 with two.  Log probabilities of a row of
// 128256 with eight: 7.0, with one 11.4; of 8192 in bf16 with one 5.5, with two 6.1.
inline smp_status shape_parts(RowsArgs& r, int elem, int least, LaunchShape& ls) {
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  const int64_t bytes = int64_t(r.vocab) * elem, sms = device_sms(dev);
  int c = 1;
  auto may = [&](int64_t room, int64_t part) { return c < kMaxParts && int64_t(r.rows) * c * 2 <= room && bytes >= 2 * c * part; };
  while (may(3 * sms, 30 * 1024) || may(sms, least)) c *= 2;
  ls.cluster = forced_cluster() ? std::min(forced_cluster(), kMaxParts) : c;
  const int per = 16 / elem;
  r.slice = ((r.vocab + per - 1 + ls.cluster - 1) / ls.cluster + per - 1) / per * per;
  return SMP_OK;
}

// Whether four CTAs of 256 threads on an SM, with fewer registers each, take fewer
// rounds than three: 4093 losses of 152064 in bf16 then take 191 us and not 203, 500
// log probabilities of 128256 with one alternative 30 and not 36; but 700, two rounds
// either way, 47 and not 40, and 400, one round, 29 and not 24.
inline bool four_on_sm(const RowsArgs& r, const LaunchShape& ls) {
  const int64_t before_last = int64_t(r.rows) * ls.cluster - 1, sms = device_sms(current_device());
  return before_last / (4 * sms) < before_last / (3 * sms);
}

// Launches `kernel` on every row; `a` is its argument, whose member `rows` is a
// RowsArgs.  Without a cluster where one CTA has a row: as clusters of one, no more
// than 16 small CTAs came to stand on an SM (8192 rows of 8191, CTAs of 32 threads:
// 68 us, 39 this way).
template <typename Args>
smp_status launch_rows(const void* kernel, Args a, LaunchShape ls, cudaStream_t st, int threads) {
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  ls.pdl = true;
  a.rows.wait_limit = wait_limit_ns();
  a.rows.first_round = 4 * device_sms(dev);
  cudaError_t err = prepare_kernel(kernel, dev, ls);
  if (err != cudaSuccess) return fail_cuda(err);
  const dim3 grid(unsigned(a.rows.rows) * unsigned(ls.cluster)), block{unsigned(threads)};
  if (ls.cluster > 1) {
    err = launch_cluster(kernel, grid, block, ls, st, &a);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = ls.smem, cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr, cfg.numAttrs = 1;
    void* params[1] = {&a};
    err = cudaLaunchKernelExC(&cfg, kernel, params);
  }
  return err == cudaSuccess ? SMP_OK : fail_cuda(err);
}

}  // namespace smp
