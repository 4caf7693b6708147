// The gradient of a row's loss in its logits, for distillation and for log
// probabilities with entropies: every logit read once, every gradient written
// once.
//
// A row belongs to the CTAs of one cluster, which each keep a slice of it in shared
// memory: fetched by bulk copies, summed, turned into gradients in place once the
// cluster's sums are known, and sent off by bulk copies.  Three CTAs stand on an
// SM (five where slices are small), so that one loads or stores while the others
// compute.  What the teacher's row gives (or the gradients of the log probabilities)
// is worked up by a warp beside the workers while the slice arrives and is summed.
//
// Bound: HBM, every logit read once and every gradient written once, where slices
// hide one another's phases: 4096 rows of 128256 in bf16 with 64 ids 341 us (91 % of
// a plain copy), 8192 of 32000, a quarter of them padding, 137 (99 %).  With
// entropies 354 for 4096 of 128256, a quarter padding (77 %), and 422 without padding
// where ids alone take 363: a unit that a slice's end cuts short is filled with -inf,
// which weighted sums take for a masked element, so that 12 of a row's 32 warps sum
// their share twice and turn it with care (all 32 of 152064 tokens: 170 and 136).
// Slices of whole units go without: 4096 rows of 32768 in 85, with ids alone 84.
// Tried, against 358 us for the first case as it then stood: the row read again from
// L2 for its gradient (490); persistent CTAs with two slices and a barrier between
// them (630), sums sent warp by warp (582), and sixteen workers with warps of their
// own for copies and joins (522).
//
// Mathematics (scores.cuh for the sums).  Distillation, with R the statistics
// outside the teacher's ids (whose places hold -inf while the rest is summed, so
// that the student's mass outside them is a sum of its own and not a difference)
// and m, Z those of the whole row:
//   ln s_j = (z_j - m) / T - ln Z,   ln s_rest = (m_R - m) / T + ln Z_R - ln Z,
//   dz_j = 2^((z_j - m_R) c) (w / T) ((sum t + r) 2^((m_R - m) c) / Z - r / Z_R)
// outside the ids, (w / T) (s_j (sum t + r) - t) on them.  Log probabilities:
//   dz_j = 2^((z_j - m) c) (A + B (z_j - m)) + (1 / T) (the id's own g),
//   B = -h / (T^2 Z),  A = -(G - h S / (T Z)) / (T Z).
#pragma once

#include "scores.cuh"

namespace smp {

struct RowGradArgs {
  RowsArgs rows;
  const int32_t* ids;
  const float* values;       // the teacher's log probabilities, or the gradients of the log probabilities
  int count, tail;
  const float* weights;      // distillation: of the rows; else: the gradients of the entropies
  float* loss;               // distillation alone
  void* grad;
  int64_t grad_stride;
  int ahead;                 // rows between a CTA's and that of the CTA that takes its place on the SM
};

// ------------------------------------------------------------------ the slice of a row

// Elements [lo, hi) of a row in shared memory at `buf`, element `id` at
// buf[id - first]; the row is laid out as in memory modulo 16 bytes, so that its
// whole vectors [full0, full1) go by bulk copies.  The edge vectors hold -inf
// outside the row.
template <typename T, int kThr>
struct Slice {
  static constexpr int kPer = RowVec<T>::kPer;
  static constexpr uint32_t kPiece = 16384;
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
  // The id of this lane's edge element, or -1.
  __device__ __forceinline__ int edge() const {
    const int lane = int(threadIdx.x) & 31, id = lane < kPer ? first + lane : first + full1 * kPer + lane - kPer;
    return lane < 2 * kPer && (lane < kPer ? full0 > 0 : full1 < vecs) ? id : INT_MIN;
  }

  // One warp: starts the copy of the slice, whose bytes `bar` is told to expect,
  // and fills the edges.
  __device__ __forceinline__ void fetch(const T* row, int vocab, uint64_t* bar) const {
    if ((threadIdx.x & 31) == 0) {
      const uint32_t bytes = uint32_t(full1 - full0) * 16u;
      const uint64_t policy = evict_first_policy();
      asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
      const char* src = reinterpret_cast<const char*>(row + first + full0 * kPer);
      char* dst = reinterpret_cast<char*>(buf) + full0 * 16;
      for (uint32_t at = 0; at < bytes; at += kPiece)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
            "%4;" ::"r"(smem_addr(dst + at)),
            "l"(src + at), "r"(min(kPiece, bytes - at)), "r"(smem_addr(bar)), "l"(policy)
            : "memory");
    }
    const int id = edge();
    if (id != INT_MIN) buf[id - first] = id >= 0 && id < vocab ? row[id] : RowVec<T>::minus_inf();
  }

  // All workers: writes the slice to a row of the output, by bulk copies where
  // that is aligned as the slice is and element by element where it is not (4096
  // rows of 50021 in bf16 193 us and not 141); returns once `buf` has been read.
  __device__ __forceinline__ void leave(T* row) const {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    workers_sync<kThr>();
    if ((reinterpret_cast<uintptr_t>(row + first) & 15u) != 0) {
      for (int id = lo + int(threadIdx.x); id < hi; id += kThr) row[id] = buf[id - first];
    } else if (threadIdx.x < 32) {
      if (threadIdx.x == 0) {
        const uint32_t bytes = uint32_t(full1 - full0) * 16u;
        char* dst = reinterpret_cast<char*>(row + first + full0 * kPer);
        const char* src = reinterpret_cast<const char*>(buf) + full0 * 16;
        for (uint32_t at = 0; at < bytes; at += kPiece)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + at), "r"(smem_addr(src + at)),
                       "r"(min(kPiece, bytes - at))
                       : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      const int id = edge();
      if (holds(id)) row[id] = buf[id - first];
      if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
  }
  // All workers: the same value everywhere.
  __device__ __forceinline__ void fill(float x) const {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = x;
    const uint4 w = RowVec<T>::put(v);
    for (int j = int(threadIdx.x); j < vecs; j += kThr) vec()[j] = w;
  }
};

// ------------------------------------------------------------------ what is known of a row before it is read

struct RowFacts {
  int flags;                  // found among the values
  float scale, given, rest, t_log_t;   // distillation: w / T, sum t, r, sum t ln t
  float sum;                  // else: G
  Stats on_ids;               // distillation: of the ids' logits
  alignas(16) int ids[kMaxIds];   // of the places that are the first of their id, -1 elsewhere
  float add[kMaxIds];         // the sum of t (or of g) over all places of the id
  float logit[kMaxIds];       // the student's
};

// A row's small inputs in one warp: places lane, lane + 32, ...
template <typename T, int kEach>
struct Inputs {
  int id[kEach];
  float value[kEach];
  T logit[kEach];
  __device__ __forceinline__ void ask(const RowGradArgs& a, int row, const T* z) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = (int(threadIdx.x) & 31) + 32 * i;
      id[i] = k < a.count ? a.ids[int64_t(row) * a.count + k] : -1;
      value[i] = k < a.count ? a.values[int64_t(row) * a.count + k] : 0.0f;
    }
    // every CTA has all of the ids' logits: what they add to Z needs no exchange
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      logit[i] = RowVec<T>::minus_inf();
      if (id[i] >= 0 && id[i] < a.rows.vocab) logit[i] = z[id[i]];
    }
  }
};

// Fills `f`, of a row whose ids are good (one warp).
template <bool kDistill, typename T, int kEach>
__device__ __forceinline__ void learn_row(const Inputs<T, kEach>& in, int count, bool tail, float temperature, float weight,
                                          RowFacts& f) {
  const int lane = int(threadIdx.x) & 31;
  float v[kEach], logit[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    v[i] = in.id[i] >= 0 ? in.value[i] : kDistill ? -INFINITY : 0.0f;
    logit[i] = clean(load1(&in.logit[i]));
    f.ids[lane + 32 * i] = in.id[i], f.logit[lane + 32 * i] = logit[i];
  }
  if (kDistill) {
    float top = -INFINITY, given = 1.0f, rest = 0.0f, log_sum = 0.0f, t_log_t = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kEach; ++i) bad |= !(v[i] < INFINITY), top = fmaxf(top, v[i]);
    if (tail) {   // r = 1 - sum t is a small difference: from fixed-point exponentials, exact to 2^-45 each
      const RowScale unit = make_row_scale_unit(0.0f);
      uint64_t mass = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) mass += mass_fixed(fminf(v[i], 1.0f), unit, kExp2Table);   // 0 for -inf
      mass = warp_sum<uint64_t>(mass);
      bad |= mass > kFixedOne + (kFixedOne >> 6);
      given = float(mass) * 0x1p-44f;
      rest = mass < kFixedOne ? float(kFixedOne - mass) * 0x1p-44f : 0.0f;
    } else {
      top = warp_max_f(top);
      bad |= !(top > -INFINITY);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum += expf(__fsub_rn(v[i], top));
      log_sum = __fadd_rn(top, logf(warp_sum_f(sum)));
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float log_t = __fsub_rn(v[i], log_sum);
      v[i] = in.id[i] >= 0 ? expf(log_t) : 0.0f;
      if (v[i] > 0.0f) t_log_t = __fmaf_rn(v[i], log_t, t_log_t);
    }
    t_log_t = warp_sum_f(t_log_t);
    bad = __any_sync(~0u, bad);
    if (lane == 0) {
      f.flags = bad ? kRowBadParams : 0;
      f.scale = __fdiv_rn(weight, temperature), f.given = given, f.rest = rest, f.t_log_t = t_log_t;
    }
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += v[i];
    sum = warp_sum_f(sum);
    if (lane == 0) f.sum = sum, f.flags = 0;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) f.add[lane + 32 * i] = v[i];
  __syncwarp();
  // Only the first place of an id stays, with the sum over all of them.
  bool first[kEach], again = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const unsigned same = __match_any_sync(~0u, in.id[i]);   // all lanes together, whatever their ids
    first[i] = in.id[i] >= 0 && (same & ((1u << lane) - 1u)) == 0;
#pragma unroll
    for (int n = 0; n < 32 * i; n += 4) {
      const int4 w = *reinterpret_cast<const int4*>(f.ids + n);
      first[i] &= w.x != in.id[i] && w.y != in.id[i] && w.z != in.id[i] && w.w != in.id[i];
    }
    again |= in.id[i] >= 0 && !first[i];
  }
  Stats k{-INFINITY, 0.0f, 0.0f};
  if (kDistill) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) k.m = fmaxf(k.m, logit[i]);
    k.m = warp_max_f(k.m);
    const float c = __fdiv_rn(kLog2e, temperature);
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (first[i] && logit[i] > -INFINITY) k.z += ex2_approx(__fmul_rn(__fsub_rn(logit[i], k.m), c));
    k.z = warp_sum_f(k.z);
    if (lane == 0) f.on_ids = k;
  }
  if (__any_sync(~0u, again)) {
    float sum[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      sum[i] = 0.0f;
      if (first[i])
        for (int n = 0; n < count; ++n) sum[i] += f.ids[n] == in.id[i] ? f.add[n] : 0.0f;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      f.add[lane + 32 * i] = sum[i];
      if (!first[i]) f.ids[lane + 32 * i] = -1;
    }
  }
}

// ------------------------------------------------------------------ the sweeps

// Calls take(vectors, first) for this thread's vectors of the slice, kUnit at a
// time, -inf in the places of those that are not there.
template <typename T, int kThr, typename Take>
__device__ __forceinline__ void each_unit(const Slice<T, kThr>& s, Take&& take) {
  using V = RowVec<T>;
  const uint4* p = s.vec();
#pragma unroll 1
  for (int j = int(threadIdx.x); j < s.vecs; j += kUnit * kThr) {
    uint4 y[kUnit];
    if (j + (kUnit - 1) * kThr < s.vecs) {
#pragma unroll
      for (int u = 0; u < kUnit; ++u) y[u] = p[j + u * kThr];
    } else {
#pragma unroll
      for (int u = 0; u < kUnit; ++u) {
        y[u] = make_uint4(V::kNegInf2, V::kNegInf2, V::kNegInf2, V::kNegInf2);
        if (j + u * kThr < s.vecs) y[u] = p[j + u * kThr];
      }
    }
    take(y, j == int(threadIdx.x));
  }
}

// The statistics of this warp's share of the slice.  Where no element is NaN, +inf
// or further above the thread's first ones than binary32 reaches (2^127 of
// weight), and with weights none is -inf, nothing has to be looked at before it
// enters the sums: y = z c - m c in one fused multiply-add, m the largest of the
// first unit.  The sums say whether that held (they are finite); otherwise the
// share is summed again with care, and `plain` is false: so for weighted sums of a
// unit that the slice's end cuts short, too, filled with -inf as it is.  A sum of 2^16 or more is
// brought below that by a higher reference, so that sums of many threads, warps
// and CTAs stay far from binary32's ends, and so do what they are divided into
// (weighted ones too: where sum_y is finite, sum is below 2^122).
template <bool kWeighted, typename T, int kThr>
__device__ __forceinline__ Stats slice_stats(const Slice<T, kThr>& s, float temperature, float c, bool& plain) {
  using V = RowVec<T>;
  float m = 0.0f;
  pair_t z = 0, zy = 0, shift = 0;
  const pair_t c2 = both(c);
  each_unit(s, [&](const uint4 (&y)[kUnit], bool first) {
    if (first) {
      uint32_t w = V::kNegInf2;
#pragma unroll
      for (int u = 0; u < kUnit; ++u) w = V::top(y[u], w);
      m = V::finish(w);
      shift = both(-__fmul_rn(m, c));
    }
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      pair_t v[V::kPer / 2];
      V::raw(y[u], v);
#pragma unroll
      for (int i = 0; i < V::kPer / 2; ++i) {
        const pair_t x = fma2(v[i], c2, shift), e = ex2_both(x);
        z = add2(z, e);
        if (kWeighted) zy = fma2(e, x, zy);
      }
    }
  });
  const float sum = sum_of(z), sum_y = kWeighted ? sum_of(zy) : 0.0f, at_m = __fmul_rn(m, c);
  const bool none = int(threadIdx.x) >= s.vecs;
  plain = __all_sync(~0u, none || (sum < INFINITY && fabsf(sum_y) < INFINITY && fabsf(at_m) < 0x1p20f));
  if (plain) {   // the sums are relative to the rounded m c: y = (z - ref) c + off
    float ref = m;
    if (sum >= 0x1p16f) ref = __fadd_rn(m, __fdiv_rn(float((__float_as_int(sum) >> 23) - 127 - 15), c));
    const float off = __fmaf_rn(ref, c, -at_m), back = ex2_approx(-off);
    Stats part{-INFINITY, 0.0f, 0.0f};
    if (!none) part = Stats{ref, sum * back, kWeighted ? __fdiv_rn(__fmaf_rn(-off, sum, sum_y) * back, c) : 0.0f};
    return warp_join<kWeighted>(part, c);
  }
  Running<T, kWeighted> run;
  each_unit(s, [&](const uint4 (&y)[kUnit], bool) { run.take(y, temperature, c); });
  return warp_join<kWeighted>(run.stats(), c);
}

// Replaces the slice's elements z by 2^((z - m) c) (A + B (z - m)); plain: as
// slice_stats found them.
template <bool kWeighted, typename T, int kThr>
__device__ __forceinline__ void slice_grad(const Slice<T, kThr>& s, float m, float temperature, float c, float ca, float cb, bool plain) {
  using V = RowVec<T>;
  uint4* p = s.vec();
  const pair_t c2 = both(c);
  auto turn_all = [&](auto&& turn) {
    int j = int(threadIdx.x);
#pragma unroll 1
    for (; j + (kUnit - 1) * kThr < s.vecs; j += kUnit * kThr) {
      uint4 y[kUnit];
#pragma unroll
      for (int u = 0; u < kUnit; ++u) y[u] = p[j + u * kThr];
#pragma unroll
      for (int u = 0; u < kUnit; ++u) p[j + u * kThr] = turn(y[u]);
    }
#pragma unroll 1
    for (; j < s.vecs; j += kThr) p[j] = turn(p[j]);
  };
  // With weights, 2^y (A + b y) with b = B / c and y = z c - m c has to be 0 wherever 2^y is, at a mask of -1e38 say:
  // b y is finite for any finite y while |b| is below 1/2, so a larger b gives n of its powers of two to the other
  // factor, as 2^(y + n) (2^-n (A - b n) + 2^-n b (y + n)).  It is larger where h is above 0.7 T Z: sums of entropies of
  // sharp rows, which the careful sweep would slow down (4096 rows of 128256: 430 us, 421 this way).
  const float b = kWeighted ? __fdiv_rn(cb, c) : 0.0f;
  const int n = max(0, int(__float_as_uint(b) >> 23 & 255u) - 125);
  if (plain && fabsf(__fmul_rn(m, c)) < 128.0f && n <= 16) {
    if (kWeighted) {
      const float lift = float(n), down = __int_as_float((127 - n) << 23);
      const pair_t shift = both(__fmaf_rn(-m, c, lift)), ca2 = both(__fmaf_rn(-lift, b * down, ca * down)), cb2 = both(b * down);
      turn_all([&](const uint4& x) {
        pair_t v[V::kPer / 2];
        float r[V::kPer];
        V::raw(x, v);
#pragma unroll
        for (int i = 0; i < V::kPer / 2; ++i) {
          const pair_t y = fma2(v[i], c2, shift);
          parts(mul2(ex2_both(y), fma2(y, cb2, ca2)), r[2 * i], r[2 * i + 1]);
        }
        return V::put(r);
      });
    } else {   // 2^(z c - m c + log2 |A|), with A's sign; the constant is below 128 + 150, its rounding at most 2^-16
      const pair_t shift = both(__fmaf_rn(-m, c, log2f(fabsf(ca))));
      const uint32_t sign = ca < 0.0f ? V::kSign : 0u;
      turn_all([&](const uint4& x) {
        pair_t v[V::kPer / 2];
        float r[V::kPer];
        V::raw(x, v);
#pragma unroll
        for (int i = 0; i < V::kPer / 2; ++i) parts(ex2_both(fma2(v[i], c2, shift)), r[2 * i], r[2 * i + 1]);
        return V::put(r, sign);
      });
    }
    return;
  }
  const uint32_t floor = floor_word<T>(m, temperature);
  const pair_t minus_m = both(-m), ca2 = both(ca), cb2 = both(cb);
  turn_all([&](const uint4& x) {
    pair_t v[V::kPer / 2];
    float r[V::kPer];
    V::get(x, floor, v);
#pragma unroll
    for (int i = 0; i < V::kPer / 2; ++i) {
      const pair_t d = add2(v[i], minus_m), e = ex2_both(mul2(d, c2)), even = mul2(e, ca2);
      parts(kWeighted ? fma2(mul2(e, d), cb2, even) : even, r[2 * i], r[2 * i + 1]);   // B d may overflow, e d not
    }
    return V::put(r);
  });
}

// ------------------------------------------------------------------ the kernel

// What the CTA will want that comes when this one has gone, asked of L2: its slice,
// if the row is read, and the values of its ids.  HBM is then busy while the CTAs
// of an SM happen to compute, and a slice arrives sooner (4096 rows of 128256: 367
// us, 415 without).  In two steps of one warp, so that nothing waits in between.
template <typename T, bool kDistill, int kEach, int kThr>
struct LookAhead {
  int row, ids[kEach];
  float weight;
  __device__ __forceinline__ void ask(const RowGradArgs& a, int now) {
    row = now < a.rows.rows - a.ahead ? now + a.ahead : -1;
    weight = !kDistill && a.weights && row >= 0 ? a.weights[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = (int(threadIdx.x) & 31) + 32 * i;
      ids[i] = row >= 0 && k < a.count ? a.ids[int64_t(row) * a.count + k] : -1;
    }
  }
  __device__ __forceinline__ void fetch(const RowGradArgs& a, int rank) const {
    bool some = weight != 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) some |= ids[i] >= 0;
    if (!__any_sync(~0u, some)) return;
    const int lane = int(threadIdx.x) & 31;
    const T* z = static_cast<const T*>(a.rows.logits) + int64_t(row) * a.rows.stride;
    const Slice<T, kThr> s(nullptr, z, a.rows.vocab, a.rows.slice, rank);
    const uintptr_t from = reinterpret_cast<uintptr_t>(z + s.first + s.full0 * Slice<T, kThr>::kPer);
    const uint32_t bytes = uint32_t(s.full1 - s.full0) * 16u, at = uint32_t(lane) * Slice<T, kThr>::kPiece;
    if (at < bytes) prefetch_l2(from + at, min(Slice<T, kThr>::kPiece, bytes - at));
    for (int k = lane; k < a.count; k += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.values + int64_t(row) * a.count + k));
  }
};

// kEach: places per lane, count rounded up to whole warps.  kThr: threads that work
// on the slice, before the warp that works up the row's small inputs.
template <typename T, bool kDistill, int kEach, int kThr, int kOnSm>
__global__ void __launch_bounds__(kThr + 32, kOnSm) row_grad_kernel(const __grid_constant__ RowGradArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];   // the slice
  __shared__ Meeting meet;
  __shared__ RowFacts f;
  __shared__ uint64_t bar;
  const int ranks = int(cluster_size()), rank = int(cluster_rank()), row = int(blockIdx.x) / ranks;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  const T* z = static_cast<const T*>(a.rows.logits) + int64_t(row) * a.rows.stride;
  T* out = static_cast<T*>(a.grad) + int64_t(row) * a.grad_stride;
  constexpr int kLearner = kThr / 32;
  const Slice<T, kThr> s(reinterpret_cast<T*>(dynamic), z, a.rows.vocab, a.rows.slice, rank);
  if (tid == 0) {
    mbar_init(&bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  ask_early(a.rows, reinterpret_cast<const uint4*>(z + s.first + s.full0 * Slice<T, kThr>::kPer), s.full1 - s.full0, 4096);
  grid_dependency_wait();
  cluster_arrive_early(ranks);
  const float temperature = row_temperature(a.rows, row);
  const float weight = a.weights ? a.weights[row] : kDistill ? 1.0f : 0.0f;
  int id = tid < a.count ? a.ids[int64_t(row) * a.count + tid] : -1;
  Inputs<T, kEach> in;
  if (warp == kLearner) in.ask(a, row, z);
  const bool some = __syncthreads_or(id >= 0) || (!kDistill && weight != 0.0f), past = __syncthreads_or(id >= a.rows.vocab);
  int flags = !some ? 0 : (past ? kRowBadToken : 0) | (temperature_fits(temperature) ? 0 : kRowBadParams);
  const bool read = some && !flags;
  if (read && warp == 0) {
    s.fetch(z, a.rows.vocab, &bar);
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&bar)) : "memory");
  }
  const float nan = __uint_as_float(0x7FC00000u), c = __fdiv_rn(kLog2e, temperature);
  LookAhead<T, kDistill, kEach, kThr> next;
  if (warp == kLearner) next.ask(a, row);
  if (!read) {
    cluster_all_run(ranks);
    if (warp == kLearner) {
      if (rank == 0 && lane == 0) {
        if (kDistill) a.loss[row] = flags ? nan : 0.0f;
        if (flags && a.rows.status) atomicOr(a.rows.status, flags);
      }
      next.fetch(a, rank);
      return;
    }
    s.fill(flags ? nan : 0.0f);
    s.leave(out);
    return;
  }
  bool late = false, plain = false;
  if (warp == kLearner) {
    learn_row<kDistill>(in, a.count, a.tail != 0, temperature, weight, f);
    next.fetch(a, rank);
    cluster_all_run(ranks);
  } else {
    late = !wait_full(&bar, 0, a.rows.wait_limit);
    if (late) wait_full(&bar, 0, kWaitLimitNs);   // the copy lands in this CTA's memory: not before that is over
    if (kDistill && s.holds(id)) s.buf[id - s.first] = RowVec<T>::minus_inf();
    late = workers_any<kThr>(late);
    const bool weighted = !kDistill && weight != 0.0f;
    const Stats part = weighted ? slice_stats<!kDistill>(s, temperature, c, plain) : slice_stats<false>(s, temperature, c, plain);
    if (lane == 0) meet.warp[warp] = part;
    cluster_all_run(ranks);
    workers_sync<kThr>();
    if (warp == 0) {
      const Stats none{-INFINITY, 0.0f, 0.0f}, mine = lane < kThr / 32 ? meet.warp[lane] : none;
      const Stats cta = weighted ? warp_join<true>(mine, c) : warp_join<false>(mine, c);
      post(meet, rank, ranks, cta.m, cta.z, cta.s, late ? 1.0f : 0.0f);
    }
  }
  cluster_meet(ranks);
  const float4 p = posted(meet, ranks);
  if (__any_sync(~0u, lane < ranks && p.w != 0.0f)) flags = kRowTimeout;
  float m, ca = 0.0f, cb = 0.0f, share = 0.0f;   // share: of this thread's id, by itself
  id = tid < 32 * kEach ? f.ids[tid] : -1;
  const bool here = s.holds(id);
  if (kDistill) {
    const Stats all = warp_join<false>(Stats{p.x, p.y, 0.0f}, c);
    const Whole whole(all, f.on_ids, c);
    if (!flags) flags = f.flags ? f.flags : fabsf(whole.m) < INFINITY ? 0 : kRowNonFinite;
    const float rest = all.z > 0.0f ? f.rest : 0.0f, total = rest > 0.0f ? 1.0f : f.given, inv_z = __frcp_rn(whole.zsum);
    if (warp == kLearner) {
      if (rank == 0) {
        const float loss = row_loss(f.ids, f.add, f.logit, 32 * kEach, f.t_log_t, all, whole.m, whole.zsum, rest, temperature);
        if (lane == 0) a.loss[row] = flags ? nan : loss;
      }
    }
    m = all.z > 0.0f ? all.m : 0.0f;   // nothing outside the ids: any finite reference
    if (all.z > 0.0f) ca = f.scale * (total * whole.reach * inv_z - __fmul_rn(rest, __frcp_rn(all.z)));
    if (here) {
      const float value = f.logit[tid];
      const float p_id = value > -INFINITY ? __fmul_rn(ex2_approx(__fmul_rn(__fsub_rn(value, whole.m), c)), inv_z) : 0.0f;
      share = __fmul_rn(f.scale, __fmaf_rn(p_id, total, -f.add[tid]));
    }
  } else {
    const Stats all = weight != 0.0f ? warp_join<true>(Stats{p.x, p.y, p.z}, c) : warp_join<false>(Stats{p.x, p.y, 0.0f}, c);
    if (!flags && !(fabsf(all.m) < INFINITY)) flags = kRowNonFinite;
    const float inv_t = __frcp_rn(temperature), inv_z = __frcp_rn(all.z), ht = __fmul_rn(weight, inv_t);
    m = all.m;
    ca = -__fmul_rn(__fmul_rn(__fmaf_rn(-ht, __fmul_rn(all.s, inv_z), f.sum), inv_t), inv_z);
    cb = -__fmul_rn(__fmul_rn(ht, inv_t), inv_z);
    if (here) {
      const float d = __fsub_rn(f.logit[tid], m), e = ex2_approx(__fmul_rn(d, c));
      share = __fmaf_rn(f.add[tid], inv_t, e == 0.0f ? 0.0f : __fmaf_rn(cb, __fmul_rn(e, d), __fmul_rn(e, ca)));
    }
  }
  if (warp == kLearner) {
    if (flags && rank == 0 && lane == 0 && a.rows.status) atomicOr(a.rows.status, flags);
    return;
  }
  if (flags) s.fill(nan);
  else if (!kDistill && weight != 0.0f && !is_lowest<T>(m)) slice_grad<!kDistill>(s, m, temperature, c, ca, cb, plain);
  else slice_grad<false>(s, m, temperature, c, ca, 0.0f, plain);
  workers_sync<kThr>();
  if (here && !flags) store1(s.buf + (id - s.first), share);
  s.leave(out);
}

template <typename T, bool kDistill, int kThr, int kOnSm>
smp_status launch_row_grad_of(const RowGradArgs& a, const LaunchShape& ls, cudaStream_t st) {
  const void* kernel = a.count <= 32   ? reinterpret_cast<const void*>(&row_grad_kernel<T, kDistill, 1, kThr, kOnSm>)
                       : a.count <= 64 ? reinterpret_cast<const void*>(&row_grad_kernel<T, kDistill, 2, kThr, kOnSm>)
                                       : reinterpret_cast<const void*>(&row_grad_kernel<T, kDistill, 4, kThr, kOnSm>);
  return launch_rows(kernel, a, ls, st, kThr + 32);
}

template <typename T, bool kDistill>
smp_status launch_row_grad(RowGradArgs a, cudaStream_t st) {
  LaunchShape ls;
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  // As few CTAs per row as let three of them stand on an SM.  More where rows are few and longer than 32 KB, while each
  // CTA has an SM of its own (two of a pair may share one, and two with 60 KB each) and 15 KB: 37 rows of 32000 in bf16
  // 5.3 us with four CTAs a row, 6.0 with two, 5.7 with eight; of 128256 9.5 with eight and 10.0 with four; of 8192 4.0
  // with one and 4.8 with two; 76 rows of 32000 in binary32 7.6 with two and 8.7 with four; 150 in bf16 9.4 with one and
  // 8.6 with two.
  const int elem = int(sizeof(T)), per = 16 / elem;
  auto slice = [&](int c) { return ((a.rows.vocab + per - 1 + c - 1) / c + per - 1) / per * per; };
  int c = 1;
  while (c < 16 && slice(c) * elem > 72 * 1024) c *= 2;
  auto may = [&](int64_t room, int64_t least) { return int64_t(a.rows.rows) * c * 2 <= room && slice(c) * elem > least; };
  const int64_t sms = device_sms(dev);
  while (c < 8 && (c == 1 ? may(2 * sms, 32 * 1024) : may(sms, 15 * 1024) || may(2 * sms, 60 * 1024))) c *= 2;
  // Twice the CTAs, of 128 threads then (below), for distillation in pairs and fours with long slices and up to 64 ids,
  // which every CTA of a cluster works up: 4096 rows of 128256 in bf16 with 64 ids 341 us and not 358, of 50021 in
  // binary32 273 and not 284, of 32000 159 and not 163; but with 100 ids 408 and not 397, of 50021 in bf16 (a pair, 50
  // KB) 139 and not 133, of 128256 in binary32 (eight) 228 and not 213 for 1200; log probabilities with entropies 377
  // and not 355, with most of their warps in the careful sums (above).  Clusters of 16, binary32 from 147454 tokens on:
  // 1200 rows of 152064 277, ids alone 279 (78 and 77 % of a plain copy).
  if (kDistill && a.count <= 64 && int64_t(a.rows.rows) * c > 3 * sms &&
      (c == 4 ? slice(c) * elem > 42 * 1024 : c == 2 && slice(c) * elem > 60 * 1024))
    c *= 2;
  if (forced_cluster() && slice(forced_cluster()) * elem <= 200 * 1024) c = forced_cluster();
  ls.cluster = c;
  a.rows.slice = slice(c);
  ls.smem = size_t(a.rows.slice) * elem;
  // Five CTAs of 128 threads on an SM instead of three of 256 where slices are small enough for that and more than
  // stand at once: 1200 rows of 152064 in bf16 132 us and not 143, 4096 of 8192 28 and not 39; but 300 of 8192 6.1 and
  // not 5.2, and with 128 threads on slices of 64 KB 4096 rows of 32000 86 and not 84 (117 and not 100 with entropies).
  const bool small = ls.smem <= 42 * 1024 && int64_t(a.rows.rows) * c > 3 * sms;
  const int on_sm = small ? 5 : std::max<int>(1, std::min<int>(3, int(227 * 1024 / (ls.smem + 3 * 1024))));
  a.ahead = std::max(1, int(sms) * on_sm / c);
  return small ? launch_row_grad_of<T, kDistill, 128, 5>(a, ls, st) : launch_row_grad_of<T, kDistill, kThreads, 3>(a, ls, st);
}

}  // namespace smp
