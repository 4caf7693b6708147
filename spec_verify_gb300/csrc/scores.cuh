// What the kernels on whole rows of logits share: log probabilities and their
// gradient (token_logprobs.cu), distillation (distill.cu).
//
// A row belongs to the CTAs of one cluster.  Each copies its slice of the row
// into shared memory with bulk copies and keeps it there, so that the maximum,
// the sums, the likeliest tokens and the gradient all come from one read of the
// row, and the gradient replaces the logits in place before one bulk copy takes
// it out.  The CTAs' sums meet in distributed shared memory; one cluster
// barrier per row.
//
// Mathematics: with m the maximum and c = log2(e) / T,
//   Z = sum 2^((z - m) c),  S = sum 2^((z - m) c) (z - m),
//   ln p_j = (z_j - m) / T - ln Z,  H = ln Z - S / (T Z).
// Parts with maxima m_i join as Z = sum Z_i w_i, S = sum w_i (S_i + Z_i (m_i -
// m)), w_i = 2^((m_i - m) c): a warp takes its own maximum as its reference, a
// CTA joins its warps and every CTA the cluster's.
#pragma once

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
};

// The statistics of some elements: their maximum, sum 2^((z - m) c) and, where
// wanted, the same weighted by z - m.  No elements: -inf, 0, 0.
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

// ------------------------------------------------------------------ the slice of a row

// Elements [lo, hi) of a row in `buf`, element `id` at buf[id - first]; the row
// is laid out as in memory modulo 16 bytes, so that its whole vectors [full0,
// full1) go by bulk copies.  The edge vectors hold -inf outside the row.
template <typename T>
struct Slice {
  static constexpr int kPer = RowVec<T>::kPer;
  T* buf;
  int first, lo, hi, vecs, full0, full1;

  __device__ __forceinline__ Slice(T* b, const T* row, int vocab, int slice, int rank) : buf(b) {
    first = rank * slice - int((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    lo = max(first, 0), hi = max(lo, min(first + slice, vocab));
    vecs = hi > lo ? (hi - first + kPer - 1) / kPer : 0;
    full0 = first < 0 && vecs ? 1 : 0;
    full1 = vecs ? max(full0, (hi - first) / kPer) : 0;
  }
  __device__ __forceinline__ bool holds(int id) const { return id >= lo && id < hi; }
  __device__ __forceinline__ float at(int id) const { return clean(load1(buf + (id - first))); }
  __device__ __forceinline__ uint4* vec() const { return reinterpret_cast<uint4*>(buf); }

  // Starts the copy of the slice (thread 0), and fills the edges (every thread).
  __device__ __forceinline__ void load(const T* row, int vocab, uint64_t* bar) const {
    if (threadIdx.x == 0) {
      const uint32_t bytes = uint32_t(full1 - full0) * 16u;
      const uint64_t policy = evict_first_policy();
      asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                   : "memory");
      const char* src = reinterpret_cast<const char*>(row + first + full0 * kPer);
      char* dst = reinterpret_cast<char*>(buf) + full0 * 16;
      for (uint32_t at = 0; at < bytes; at += kPiece)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
            "%4;" ::"r"(smem_addr(dst + at)),
            "l"(src + at), "r"(min(kPiece, bytes - at)), "r"(smem_addr(bar)), "l"(policy)
            : "memory");
    }
    if (threadIdx.x < 2 * kPer) {
      const int i = int(threadIdx.x) % kPer;
      const bool head = int(threadIdx.x) < kPer;
      if (head ? full0 > 0 : full1 < vecs) {
        const int id = first + (head ? 0 : full1 * kPer) + i;
        buf[id - first] = id >= 0 && id < vocab ? row[id] : RowVec<T>::minus_inf();
      }
    }
  }

  // Writes the slice to a row of the output, whole vectors by a bulk copy where
  // the output row is aligned as the slice is.  Called by all threads after the
  // last change of `buf`; returns once `buf` has been read.
  __device__ __forceinline__ void store(T* row) const {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    const bool bulk = (reinterpret_cast<uintptr_t>(row + first) & 15u) == 0;
    if (bulk) {
      if (threadIdx.x == 0) {
        const uint32_t bytes = uint32_t(full1 - full0) * 16u;
        char* dst = reinterpret_cast<char*>(row + first + full0 * kPer);
        const char* src = reinterpret_cast<const char*>(buf) + full0 * 16;
        for (uint32_t at = 0; at < bytes; at += kPiece)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + at),
                       "r"(smem_addr(src + at)), "r"(min(kPiece, bytes - at))
                       : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      if (threadIdx.x < 2 * kPer) {
        const int i = int(threadIdx.x) % kPer;
        const bool head = int(threadIdx.x) < kPer;
        const int id = first + (head ? 0 : full1 * kPer) + i;
        if ((head ? full0 > 0 : full1 < vecs) && id >= lo && id < hi) row[id] = buf[id - first];
      }
      if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    } else {
      for (int id = lo + int(threadIdx.x); id < hi; id += kThreads) row[id] = buf[id - first];
    }
  }

  // The same value everywhere (a row that was not read, or an error row).
  __device__ __forceinline__ void fill(float x) const {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = x;
    const uint4 w = RowVec<T>::put(v);
    for (int j = int(threadIdx.x); j < vecs; j += kThreads) vec()[j] = w;
  }

  static constexpr uint32_t kPiece = 16384;
};

// ------------------------------------------------------------------ sums

__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Two binary32 numbers at a time.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return reinterpret_cast<const float2&>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return reinterpret_cast<const float2&>(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return reinterpret_cast<const float2&>(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The running statistics of one thread's elements: a group of vectors is taken
// in at a time, relative to the largest element so far.
template <typename T, bool kWeighted>
struct Running {
  using V = RowVec<T>;
  float m = -INFINITY;
  float2 z = make_float2(0.0f, 0.0f), s = make_float2(0.0f, 0.0f);
  uint32_t floor = 0;

  // A maximum of the elements that come next.
  __device__ __forceinline__ void raise(float top, float temperature, float c) {
    if (top > m) {
      if (m > -INFINITY) {
        const float d = __fsub_rn(m, top), w = ex2_approx(__fmul_rn(d, c));
        if (kWeighted) s = w == 0.0f ? both(0.0f) : mul2(fma2(z, both(d), s), both(w));
        z = mul2(z, both(w));
      }
      m = top;
      floor = floor_word<T>(m, temperature);
    }
  }
  // A vector none of whose elements is above m; m is not -inf.
  __device__ __forceinline__ void add(const uint4& x, float c) {
    float v[V::kPer];
    V::get(x, floor, v);
#pragma unroll
    for (int i = 0; i < V::kPer; i += 2) {
      const float2 d = add2(make_float2(v[i], v[i + 1]), both(-m)), y = mul2(d, both(c));
      const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
      z = add2(z, e);
      if (kWeighted) s = fma2(e, d, s);
    }
  }
  __device__ __forceinline__ void add_one(float v, float temperature, float c) {   // clean
    if (v > -INFINITY) {
      raise(v, temperature, c);
      const float d = __fsub_rn(v, m), e = ex2_approx(__fmul_rn(d, c));
      z.x += e;
      if (kWeighted && e > 0.0f) s.x = __fmaf_rn(e, d, s.x);
    }
  }
  __device__ __forceinline__ Stats stats() const {
    return Stats{m, z.x + z.y, kWeighted && !is_lowest<T>(m) ? s.x + s.y : 0.0f};
  }
};

// The largest of this thread's elements (vectors tid, tid + kThreads, ...).
template <typename T>
__device__ __forceinline__ float thread_top(const Slice<T>& s) {
  uint32_t m = RowVec<T>::kNegInf2;
  for (int j = int(threadIdx.x); j < s.vecs; j += kThreads) m = RowVec<T>::top(s.vec()[j], m);
  return RowVec<T>::finish(m);
}

// The statistics of the lanes' parts together, in every lane.
__device__ __forceinline__ Stats warp_join(const Stats& part, float c) {
  Stats out;
  out.m = warp_max_f(part.m);
  float z = 0.0f, s = 0.0f;
  if (part.z != 0.0f) {
    const float d = __fsub_rn(part.m, out.m), w = ex2_approx(__fmul_rn(d, c));
    z = part.z * w;
    s = w == 0.0f ? 0.0f : w * __fmaf_rn(part.z, d, part.s);
  }
  out.z = warp_sum_f(z), out.s = warp_sum_f(s);
  return out;
}

// The statistics of this warp's elements, given its threads' maxima.
template <typename T, bool kWeighted>
__device__ __forceinline__ Stats warp_stats(const Slice<T>& s, float mine, float temperature, float c) {
  Running<T, kWeighted> run;
  run.raise(mine, temperature, c);
  if (run.m > -INFINITY)
    for (int j = int(threadIdx.x); j < s.vecs; j += kThreads) run.add(s.vec()[j], c);
  return warp_join(run.stats(), c);
}

// ------------------------------------------------------------------ a part of a row, read once from memory

// Elements [lo, hi) of a row, whole vectors [full0, full1) of 16 bytes counted
// from element `first`; thread t takes vectors full0 + t, full0 + t + kThreads,
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

// A vector that is not wanted again soon, past the L1 cache.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

constexpr int kUnit = 4;     // vectors of a thread that are loaded and taken in together

// Takes the part's whole vectors into `run`, a unit per thread at a time: while
// one unit is taken in, the next is on its way, in x[0] and x[1], which hold all
// of the thread's vectors where there are two units at most.  change(y, k) may
// alter vector k (from the first whole one) first; seen(top) gets the largest
// element of each unit, in order.
template <typename T, bool kWeighted, typename Change, typename Seen>
__device__ __forceinline__ void stream(const Part<T>& s, Running<T, kWeighted>& run, uint4 (&x)[2][kUnit],
                                       const float& temperature, const float& c, Change&& change, Seen&& seen) {
  using V = RowVec<T>;
  constexpr int kStep = kUnit * kThreads;
  const int vecs = s.full1 - s.full0, pairs = vecs / (2 * kStep);
  const uint4* p = s.vec() + s.full0 + threadIdx.x;
  auto load = [&](uint4 (&y)[kUnit], const uint4* from) {
#pragma unroll
    for (int u = 0; u < kUnit; ++u) y[u] = load_once(from + u * kThreads);
  };
  auto load_some = [&](uint4 (&y)[kUnit], int unit) {
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      y[u] = make_uint4(V::kNegInf2, V::kNegInf2, V::kNegInf2, V::kNegInf2);
      if (int(threadIdx.x) + unit * kStep + u * kThreads < vecs) y[u] = load_once(p + unit * kStep + u * kThreads);
    }
  };
  auto take = [&](uint4 (&y)[kUnit], int unit) {
    uint32_t w = V::kNegInf2;
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      change(y[u], int(threadIdx.x) + (unit * kUnit + u) * kThreads);
      w = V::top(y[u], w);
    }
    const float top = V::finish(w);
    run.raise(top, temperature, c);
    if (run.m > -INFINITY) {
#pragma unroll
      for (int u = 0; u < kUnit; ++u) run.add(y[u], c);
    }
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

// Waits for the slice (every thread); true when some thread's wait ran out.
__device__ __forceinline__ bool slice_is_late(uint64_t* bar, uint64_t limit) {
  const bool late = !wait_full(bar, 0, limit);
  if (late) wait_full(bar, 0, kWaitLimitNs);   // the copy lands in this CTA's memory: not before that is over
  return __syncthreads_or(late);
}

__device__ __forceinline__ float row_temperature(const RowsArgs& a, int row) {
  return a.temperatures ? a.temperatures[row] : a.temperature;
}
__device__ __forceinline__ bool temperature_fits(float t) { return t >= SMP_MIN_TEMPERATURE && t <= SMP_MAX_TEMPERATURE; }

// First occurrence of each id in `ids` and the sum of `add` over its places:
// what thread k < count gets for id k.
__device__ __forceinline__ bool first_of_id(const int* ids, const float* add, int count, int k, float& sum) {
  bool first = true;
  sum = 0.0f;
  for (int i = 0; i < count; ++i)
    if (ids[i] == ids[k]) {
      first &= i >= k;
      sum += add[i];
    }
  return first;
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

// A gradient's rows: beside the logits, or in their place.
inline bool grad_fits(const void* logits, int32_t rows, int32_t vocab, int64_t stride, const void* grad, int64_t grad_stride) {
  if (grad_stride < vocab || grad_stride > (int64_t(1) << 40)) return false;
  return grad != logits || rows <= 1 || grad_stride == stride;
}

// The launch of a kernel whose CTAs read their parts of a row from memory once:
// one row per CTA where there are many rows, parts of it where they would leave
// SMs without work.
inline smp_status shape_parts(RowsArgs& r, int elem, LaunchShape& ls) {
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  const int64_t bytes = int64_t(r.vocab) * elem;
  int c = 1;
  while (c < kMaxParts && int64_t(r.rows) * c * 2 <= int64_t(device_sms(dev)) * 4 && bytes >= int64_t(c) * 16 * 1024) c *= 2;
  ls.cluster = forced_cluster() ? std::min(forced_cluster(), kMaxParts) : c;
  const int per = 16 / elem;
  r.slice = ((r.vocab + per - 1 + ls.cluster - 1) / ls.cluster + per - 1) / per * per;
  return SMP_OK;
}

// The launch of a kernel whose CTAs keep their slices in shared memory.
inline smp_status shape_slices(RowsArgs& r, int elem, LaunchShape& ls) {
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  const int64_t bytes = int64_t(r.vocab) * elem;
  int c = 1;
  while (c < 16 && bytes > int64_t(c) * 68 * 1024) c *= 2;
  while (c < 8 && int64_t(r.rows) * c * 2 <= int64_t(device_sms(dev)) * 3 && bytes >= int64_t(c) * 16 * 1024) c *= 2;
  const int forced = forced_cluster();
  ls.cluster = forced && bytes <= int64_t(forced) * 160 * 1024 ? forced : c;
  const int per = 16 / elem;
  r.slice = ((r.vocab + per - 1 + ls.cluster - 1) / ls.cluster + per - 1) / per * per;
  ls.smem = size_t(r.slice) * elem;
  return SMP_OK;
}

// Launches `kernel` on every row; `a` is its argument, whose member `rows` is a
// RowsArgs.
template <typename Args>
smp_status launch_rows(const void* kernel, Args a, LaunchShape ls, cudaStream_t st) {
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  ls.pdl = true;
  a.rows.wait_limit = wait_limit_ns();
  cudaError_t err = prepare_kernel(kernel, dev, ls);
  if (err != cudaSuccess) return fail_cuda(err);
  err = launch_cluster(kernel, dim3(unsigned(a.rows.rows) * unsigned(ls.cluster)), dim3(kThreads), ls, st, &a);
  return err == cudaSuccess ? SMP_OK : fail_cuda(err);
}

}  // namespace smp
