// Log probabilities of given tokens, entropies and likeliest tokens of rows of
// logits, and the gradient of log probabilities and entropies.
//
// Bound: the forward call reads every logit once from HBM.  4093 rows of 152064 in
// bf16 with entropies: 178 us (the copy rate) without alternatives, 200 with one,
// 208 with twenty; 2046 in binary32 with eight 193.  The difference is what follows
// a row's stream: a bound, the runs that reach it read again, most of them from HBM
// (608 rows in flight are more than L2 holds).  Vectors kept in shared memory as they
// pass, against a bound that follows the stream, spare that but cost the stream more
// (2048 rows of 128256 with 64 alternatives: 157 us, 105 this way).
//
// Likeliest tokens: each CTA finds the `top` largest of its slice before the
// cluster's barrier, so that the lists travel with the sums.  The n-th largest
// of its threads' maxima (32 to 256, at least 2 n) is at most the slice's n-th
// largest element, since n threads each hold an element that large: everything at
// or above it (a few more than n) is collected and ranked by comparing packed
// (value, id) words.  Where more reach the bound than the list holds, the slice is
// gone through once for every alternative: equal logits, and rows masked with a
// finite value that leave fewer tokens than are wanted.  256 rows of 128256 in bf16
// with ten tokens left and the others at -1e4, twenty wanted: 786 us; with the others
// at -inf 18.
// The first CTA of the cluster puts the CTAs' candidates in order, by counting for
// each the larger ones, or by bisection in lists that the CTAs have ordered where
// many alternatives are wanted.
#include <cuda_runtime.h>

#include <algorithm>

#include "row_grad.cuh"

namespace smp {

constexpr int kCandidates = 512;   // collected before the slow exact way takes over
// Of the successor's part.  16 KB: 8192 rows of 32000 with twenty alternatives 109 us, with 64 KB 120; 4093 of 152064 208
// and 206; 2048 of 128256 with five 94 and 94, with 8 KB 96.
constexpr int kAheadVectors = 1024;
constexpr int kShortLists = 32;    // most alternatives whose candidates are only put in order at the end

struct ScoreArgs {
  RowsArgs rows;
  const int32_t* ids;
  int count, top;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int run_room;   // most runs of any CTA
  int list_room;  // words of a CTA's list
  int ahead;      // rows between a CTA's and that of the CTA that takes its place on the SM
};

// A thread's units of kUnit vectors come in up to kRuns runs whose maxima are kept.
static_assert(kUnit == 4, "runs are counted in shifts");
constexpr int kRuns = 16;

// What slice_top works with, in shared memory.
template <int kThr>
struct TopRoom {
  static constexpr int kCandidates = kThr == kThreads ? smp::kCandidates : smp::kCandidates / 2;
  alignas(16) uint16_t keys[kThr];
  uint16_t hits[kCandidates];      // thread | run << 8
  uint64_t cand[kCandidates];
  uint64_t scratch[kThr / 32];
  uint32_t bound;
  int hit_count, found;
};

// The largest value that `top` of the keys reach, in one warp: bisection between
// the smallest and the largest key, which are a few hundred apart in ordinary rows
// (256 threads that count keys bit by bit behind a barrier each took 1.1 to 2.4 us,
// this 0.3).
template <int kThr>
__device__ __forceinline__ uint32_t nth_key(const uint16_t* keys, int top) {
  constexpr int kEach = kThr / 32;
  uint32_t k[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) k[i] = keys[(int(threadIdx.x) & 31) + 32 * i];
  uint32_t lo = k[0], hi = k[0];
#pragma unroll
  for (int i = 1; i < kEach; ++i) lo = min(lo, k[i]), hi = max(hi, k[i]);
  lo = __reduce_min_sync(~0u, top <= 32 ? hi : lo), hi = __reduce_max_sync(~0u, hi);   // 32 keys reach the lanes' least maximum
  if (top == 1) return hi;
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) n += kEach == 1 ? __popc(__ballot_sync(~0u, k[i] >= mid)) : int(k[i] >= mid);
    if ((kEach == 1 ? n : __reduce_add_sync(~0u, n)) >= top) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The candidates for a part's `top` largest elements, as packed words in
// room.cand; returns how many, at least the `top` largest (or all that are
// finite) among them.  `mine` is the largest of this thread's elements,
// run_top[run][thread] of each run of 2^run_bits units, `edge` its edge element's
// id.
template <int kThr, typename T>
__device__ __forceinline__ int slice_top(const Part<T>& s, float mine, const float* run_top, int runs, int run_bits, int edge,
                                         int top, TopRoom<kThr>& room) {
  constexpr int kCandidates = TopRoom<kThr>::kCandidates;
  using V = RowVec<T>;
  constexpr int kPer = V::kPer;
  const int tid = int(threadIdx.x);
  const uint32_t key = key_of_bits(__float_as_uint(mine)) >> 16;
  room.keys[tid] = uint16_t(key);
  if (tid == 0) room.hit_count = room.found = 0;
  __syncthreads();
  if (tid < 32) {
    const uint32_t b = nth_key<kThr>(room.keys, top);
    if (tid == 0) room.bound = b;
  }
  __syncthreads();
  const uint32_t bound = room.bound, least = max(bound << 16, kKeyNegInf + 1u);
  const float limit = value_of_key(least);
  auto keep = [&](int place, float v, int id) {
    if (place < kCandidates) room.cand[place] = pack_key_id(key_of_bits(__float_as_uint(v)), uint32_t(id));
  };
  // The elements of kUnit vectors (of the ids at[u], or none: -1) that reach the
  // limit; one atomic for all of a thread's.
  auto take = [&](const uint4 (&y)[kUnit], const int (&at)[kUnit]) {
    uint32_t mask = 0;
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      if (at[u] < 0 || !(V::finish(V::top(y[u], V::kNegInf2)) >= limit)) continue;
      float v[kPer];
      V::get(y[u], V::kNegInf2, v);
#pragma unroll
      for (int q = 0; q < kPer; ++q) mask |= (v[q] >= limit ? 1u : 0u) << (u * kPer + q);
    }
    if (mask) {
      int place = atomicAdd(&room.found, __popc(mask));
#pragma unroll
      for (int u = 0; u < kUnit; ++u) {
        if (!(mask >> (u * kPer) & ((1u << kPer) - 1u))) continue;
        float v[kPer];
        V::get(y[u], V::kNegInf2, v);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (mask >> (u * kPer + q) & 1u) keep(place++, v[q], at[u] + q);
      }
    }
  };
  const int vecs = s.full1 - s.full0;
  if (mine >= limit) {
    if (edge >= 0) {
      const float v = Elem<T>::widen(s.row[edge]);
      if (v >= limit) keep(atomicAdd(&room.found, 1), v, edge);
    }
    uint32_t mask = 0;
#pragma unroll 4
    for (int run = 0; run < runs; ++run) mask |= (run_top[run * kThr + tid] >= limit ? 1u : 0u) << run;
    int place = mask ? atomicAdd(&room.hit_count, __popc(mask)) : 0;
    for (; mask; mask &= mask - 1, ++place)
      if (place < kCandidates) room.hits[place] = uint16_t(tid | (__ffs(mask) - 1) << 8);
  }
  __syncthreads();
  // The vectors of the runs that reach the limit again, from L2, spread over the
  // threads (each thread its own runs: 3.0 us where this takes 1.9).
  const int vectors = min(room.hit_count, kCandidates) << (run_bits + 2);
  for (int i0 = tid; i0 < vectors; i0 += kUnit * kThr) {
    uint4 y[kUnit];
    int at[kUnit];
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      const int i = i0 + u * kThr;
      at[u] = -1;
      if (i < vectors) {
        const int hit = room.hits[i >> (run_bits + 2)], of = i & ((kUnit << run_bits) - 1);
        const int k = (hit & 255) + (((hit >> 8) << (run_bits + 2)) + of) * kThr;
        if (k < vecs) at[u] = s.first + (s.full0 + k) * kPer, y[u] = s.vec()[s.full0 + k];
      }
    }
    take(y, at);
  }
  __syncthreads();
  int have = room.found;
  if (have > kCandidates || room.hit_count > kCandidates) {   // many equal values: one maximum after another, each below the last (slow: above)
    uint64_t last = ~0ull;
    for (have = 0; have < top; ++have) {
      uint64_t best = 0;
      for (int id = s.lo + tid; id < s.hi; id += kThr) {
        const uint32_t k = key_of_bits(Elem<T>::bits(s.row[id]));
        const uint64_t v = k > kKeyNegInf ? pack_key_id(k, uint32_t(id)) : 0;
        if (v < last && v > best) best = v;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) best = max(best, shfl_xor_u64(best, o));
      __syncthreads();
      if ((tid & 31) == 0) room.scratch[tid >> 5] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThr / 32; ++w) best = max(best, room.scratch[w]);
      if (best == 0) break;
      if (tid == 0) room.cand[have] = best;
      last = best;
    }
    __syncthreads();
  }
  return have;
}

// How many of the `count` words of `list` are above v; four neighbouring lanes
// count together, and all of them get it.
__device__ __forceinline__ int count_above(const uint64_t* list, int count, uint64_t v) {
  int n = 0;
#pragma unroll 8
  for (int j = int(threadIdx.x) & 3; j < count; j += 4) n += list[j] > v;
  n += __shfl_xor_sync(~0u, n, 1);
  return n + __shfl_xor_sync(~0u, n, 2);
}

// kOnSm: CTAs on an SM.
// kThr: threads of a CTA, 256 for parts of rows.  Where rows are many, smaller CTAs,
// of which more stand on an SM, overlap more of what follows a row's stream; kThr
// is at least twice the alternatives wanted, so that the threads' maxima bound them.
template <typename T, bool kEntropy, bool kTop, int kThr, int kOnSm>
__global__ void __launch_bounds__(kThr, kOnSm) token_logprobs_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];   // with kTop: TopRoom, the runs' maxima, the lists
  __shared__ Meeting meet;
  const int ranks = int(cluster_size()), rank = int(cluster_rank()), row = int(blockIdx.x) / ranks;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  const T* z = static_cast<const T*>(a.rows.logits) + int64_t(row) * a.rows.stride;
  const Part<T> s(z, a.rows.vocab, a.rows.slice, rank);
  ask_early(a.rows, s.vec() + s.full0, s.full1 - s.full0, 2048);
  grid_dependency_wait();
  cluster_arrive_early(ranks);

  const float temperature = row_temperature(a.rows, row), c = __fdiv_rn(kLog2e, temperature);
  const int id = tid < a.count ? a.ids[int64_t(row) * a.count + tid] : -1;
  float* logprobs = a.logprobs + int64_t(row) * a.count;
  if (!kEntropy && !kTop && !__syncthreads_or(id >= 0)) {   // every id is padding
    cluster_all_run(ranks);
    if (rank == 0 && tid < a.count) logprobs[tid] = 0.0f;
    return;
  }
  TopRoom<kThr>& room = *reinterpret_cast<TopRoom<kThr>*>(dynamic);
  float* run_top = reinterpret_cast<float*>(dynamic + sizeof(TopRoom<kThr>));
  const int units_all = (s.full1 - s.full0 + kThr * kUnit - 1) / (kThr * kUnit);   // of a thread
  const int run_bits = units_all <= kRuns ? 0 : 32 - __clz((units_all - 1) / kRuns);   // 2^run_bits units in a run
  const int runs = (units_all + (1 << run_bits) - 1) >> run_bits;
  uint64_t* lists = reinterpret_cast<uint64_t*>(run_top + a.run_room * kThr);
  int flags = temperature_fits(temperature) ? 0 : kRowBadParams;
  Stats all{-INFINITY, 0.0f, 0.0f};
  int have = 0, theirs = 0;   // candidates of this CTA, of the CTA of this lane's number
  const float value = flags == 0 && s.holds(id) ? clean(load1(z + id)) : 0.0f;
  if (flags == 0) {
    Running<T, kEntropy> run;
    const int edge = s.edge();
    const float at_edge = edge >= 0 ? clean(load1(z + edge)) : -INFINITY;
    float best = -INFINITY, mine = at_edge;   // the largest of the run, of the thread
    int in_run = 0, r = 0;
    stream<kThr>(s, run, temperature, c, [](uint4&, int) {}, [&](float top) {
      if (kTop) {
        best = fmaxf(best, top), mine = fmaxf(mine, top);
        if (++in_run == 1 << run_bits) {
          run_top[r * kThr + tid] = best;
          best = -INFINITY, in_run = 0, ++r;
        }
      }
    });
    if (tid == 0 && (kTop || kEntropy) && row < a.rows.rows - a.ahead) {   // L2 is asked for the start of the successor's part
      const Part<T> next(z + a.ahead * a.rows.stride, a.rows.vocab, a.rows.slice, rank);
      prefetch_l2(reinterpret_cast<uintptr_t>(next.vec() + next.full0), uint32_t(min(next.full1 - next.full0, kAheadVectors)) * 16u);
    }
    run.add_one(at_edge, temperature, c);
    if (kTop) {
      for (; r < runs; ++r, best = -INFINITY) run_top[r * kThr + tid] = best;
    }
    const Stats part = warp_join<kEntropy>(run.stats(), c);
    if (lane == 0) meet.warp[warp] = part;
    cluster_all_run(ranks);
    if (kTop) {
      have = slice_top<kThr>(s, mine, run_top, runs, run_bits, edge, a.top, room);
      if (ranks > 1) {
        const uint32_t to = map_rank(smem_addr(lists + rank * a.list_room), 0);
        if (have <= a.list_room && a.top <= kShortLists) {   // as they are: the first CTA puts them in order
          for (int i = tid; i < have; i += kThr) st_cluster_u64(to + uint32_t(i) * 8u, room.cand[i]);
        } else {
          for (int i0 = 0; i0 < have; i0 += kThr / 4) {
            const int i = i0 + (tid >> 2);
            const uint64_t v = i < have ? room.cand[i] : ~0ull;
            const int place = count_above(room.cand, have, v);
            if ((tid & 3) == 0 && i < have && place < a.top) st_cluster_u64(to + uint32_t(place) * 8u, v);
          }
          have = min(have, a.top);
          for (int i = have + tid; i < a.top; i += kThr) st_cluster_u64(to + uint32_t(i) * 8u, 0);
        }
      }
    }
    __syncthreads();
    if (warp == 0) {
      const Stats cta = warp_join<kEntropy>(lane < kThr / 32 ? meet.warp[lane] : Stats{-INFINITY, 0.0f, 0.0f}, c);
      post(meet, rank, ranks, cta.m, cta.z, cta.s, float(have));
    }
    cluster_meet(ranks);
    const float4 p = posted(meet, ranks);
    all = warp_join<kEntropy>(Stats{p.x, p.y, p.z}, c);
    theirs = lane < ranks ? int(p.w) : 0;
    if (!(fabsf(all.m) < INFINITY)) flags = kRowNonFinite;
  } else {
    cluster_all_run(ranks);
  }
  const float nan = __uint_as_float(0x7FC00000u), log_z = logf(all.z);
  auto logprob = [&](float v) { return __fsub_rn(__fdiv_rn(__fsub_rn(v, all.m), temperature), log_z); };
  if (tid < a.count) {
    const bool past = id >= a.rows.vocab;
    if (flags == 0 && s.holds(id)) logprobs[tid] = logprob(value);
    else if (rank == 0 && (id < 0 || past || flags)) logprobs[tid] = id < 0 ? 0.0f : nan;
    if (rank == 0 && past && a.rows.status) atomicOr(a.rows.status, kRowBadToken);
  }
  if (rank != 0) return;
  if (tid == 0) {
    if (flags && a.rows.status) atomicOr(a.rows.status, flags);
    if (kEntropy) a.entropy[row] = flags ? nan : __fsub_rn(log_z, __fdiv_rn(all.s, __fmul_rn(temperature, all.z)));
  }
  if (kTop) {
    int32_t* top_ids = a.top_ids + int64_t(row) * a.top;
    float* top_logprobs = a.top_logprobs + int64_t(row) * a.top;
    if (flags) {
      for (int i = tid; i < a.top; i += kThr) top_ids[i] = -1, top_logprobs[i] = nan;
      return;
    }
    auto emit = [&](int place, uint64_t v) {   // 0: no token
      if (place < a.top) {
        top_ids[place] = v ? int32_t(~uint32_t(v)) : -1;
        top_logprobs[place] = v ? logprob(value_of_key(uint32_t(v >> 32))) : -INFINITY;
      }
    };
    if (ranks == 1 || a.top <= kShortLists) {   // a token's place is the number of larger ones
      int total = have;
      if (ranks > 1) {   // the lists one after the other in room.cand
        const int upto = int(warp_inclusive_scan<uint32_t>(uint32_t(theirs)));
        total = __shfl_sync(~0u, upto, 31);
        for (int e = tid; e < ranks * a.list_room; e += kThr) {   // a warp's words are of one list
          const int from = e / (2 * kShortLists), i = e % (2 * kShortLists), n = __shfl_sync(~0u, theirs, from);
          const int at = __shfl_sync(~0u, upto, from) - n + i;
          if (i < n) room.cand[at] = lists[e];
        }
        __syncthreads();
      }
      for (int e = tid; e < total; e += kThr) {
        const uint64_t v = room.cand[e];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < total; ++j) place += room.cand[j] > v;
        emit(place, v);
      }
      for (int i = total + tid; i < a.top; i += kThr) emit(i, 0);
      return;
    }
    // A token's place is the number of larger ones in all lists, by bisection in
    // all of them at once.  An entry that is none finds all tokens larger: those of
    // list 0 fill the places that are left.
    for (int e = tid; e < ranks * a.top; e += kThr) {
      const uint64_t v = lists[e];
      int lo[kMaxParts], hi[kMaxParts];
#pragma unroll
      for (int r = 0; r < kMaxParts; ++r) lo[r] = 0, hi[r] = r < ranks ? a.top : 0;
      for (int left = a.top; left > 0; left >>= 1) {
#pragma unroll
        for (int r = 0; r < kMaxParts; ++r) {
          const int mid = (lo[r] + hi[r]) >> 1;
          if (lo[r] < hi[r]) {
            if (lists[r * a.top + mid] > v) lo[r] = mid + 1;
            else hi[r] = mid;
          }
        }
      }
      int place = v ? 0 : e < a.top ? e - lo[0] : a.top;
#pragma unroll
      for (int r = 0; r < kMaxParts; ++r) place += lo[r];
      emit(place, v);
    }
  }
}

template <typename T, int kThr, int kOnSm>
static smp_status launch_scores_of(ScoreArgs a, LaunchShape ls, cudaStream_t st) {
  const void* kernel =
      a.entropy ? (a.top ? reinterpret_cast<const void*>(&token_logprobs_kernel<T, true, true, kThr, kOnSm>)
                         : reinterpret_cast<const void*>(&token_logprobs_kernel<T, true, false, kThr, kOnSm>))
                : (a.top ? reinterpret_cast<const void*>(&token_logprobs_kernel<T, false, true, kThr, kOnSm>)
                         : reinterpret_cast<const void*>(&token_logprobs_kernel<T, false, false, kThr, kOnSm>));
  a.ahead = std::max(1, device_sms(current_device()) * kOnSm / ls.cluster);
  if (a.top) {
    a.list_room = a.top <= kShortLists ? 2 * kShortLists : a.top;
    const int unit = kThr * kUnit * RowVec<T>::kPer;
    a.run_room = std::min(kRuns, (a.rows.slice + unit - 1) / unit);
    ls.smem = sizeof(TopRoom<kThr>) + size_t(a.run_room) * kThr * 4 + (ls.cluster > 1 ? size_t(ls.cluster) * a.list_room * 8 : 0);
  }
  return launch_rows(kernel, a, ls, st, kThr);
}

template <typename T>
static smp_status launch_scores(ScoreArgs a, cudaStream_t st) {
  LaunchShape ls;
  const smp_status ok = shape_parts(a.rows, int(sizeof(T)), 30 * 1024, ls);
  if (ok != SMP_OK) return ok;
  const int sms = device_sms(current_device());
  // Small CTAs for rows that are many and not long, as many threads as leave no SM without work: 8192 rows of 32000 in
  // bf16 with one alternative 99 us with 32 threads, 106 with 64, 114 with 128, 143 with 256; 1200 rows with eight 29,
  // 22, 19, 24; 2048 rows of 128256 with twenty: 108 with 64, 101 with 128 and 256.
  if (ls.cluster == 1 && !forced_cluster() && int64_t(a.rows.vocab) * int(sizeof(T)) < 200 * 1024) {
    const int least = std::max(2 * a.top, a.count);
    auto fills = [&](int threads) { return threads >= least && int64_t(a.rows.rows) * threads >= int64_t(sms) * 768; };
    if (fills(32)) return launch_scores_of<T, 32, 32>(a, ls, st);
    if (fills(64)) return launch_scores_of<T, 64, 16>(a, ls, st);
    if (fills(128)) return launch_scores_of<T, 128, 8>(a, ls, st);
  }
  // Halves of long rows where four on an SM hold them: 256 rows of 128256 in bf16 20.9 us, whole ones with three on an
  // SM 22.8; 300 rows of 32000 in binary32 12.2 and 11.9.
  if (ls.cluster == 1 && !forced_cluster() && a.rows.rows <= 2 * sms && int64_t(a.rows.vocab) * int(sizeof(T)) >= 200 * 1024) {
    constexpr int kPer = RowVec<T>::kPer;
    ls.cluster = 2;
    a.rows.slice = ((a.rows.vocab + kPer - 1 + 1) / 2 + kPer - 1) / kPer * kPer;
  }
  return four_on_sm(a.rows, ls) ? launch_scores_of<T, kThreads, 4>(a, ls, st) : launch_scores_of<T, kThreads, 3>(a, ls, st);
}

}  // namespace smp

extern "C" smp_status smp_token_logprobs(const void* logits, int32_t rows, int32_t vocab, int64_t stride, smp_dtype dtype,
                                         float temperature, const float* temperatures, const int32_t* ids, int32_t count,
                                         int32_t top, float* out_logprobs, float* out_entropy, int32_t* out_top_ids,
                                         float* out_top_logprobs, int32_t* status, void* stream) {
  using namespace smp;
  const smp_status ok = check_rows(logits, rows, vocab, stride, dtype, temperature, temperatures, status);
  if (ok != SMP_OK) return ok;
  if (count < 0 || count > SMP_MAX_ROW_IDS || top < 0 || top > SMP_MAX_ROW_IDS) return SMP_ERR_INVALID_ARG;
  if (count == 0 && top == 0 && !out_entropy) return SMP_ERR_INVALID_ARG;
  if (rows > 0 && ((count > 0 && (!ids || !out_logprobs)) || (top > 0 && (!out_top_ids || !out_top_logprobs))))
    return SMP_ERR_INVALID_ARG;
  if (misaligned(ids, 4) || misaligned(out_logprobs, 4) || misaligned(out_entropy, 4) || misaligned(out_top_ids, 4) ||
      misaligned(out_top_logprobs, 4))
    return SMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    const smp_status rc = clear_status(status, st);
    if (rc != SMP_OK) return rc;
  }
  if (rows == 0) return SMP_OK;
  ScoreArgs a{};
  a.rows.logits = logits, a.rows.stride = stride, a.rows.rows = rows, a.rows.vocab = vocab;
  a.rows.temperature = temperature, a.rows.temperatures = temperatures, a.rows.status = status;
  a.ids = ids, a.count = count, a.top = top;
  a.logprobs = out_logprobs, a.entropy = out_entropy, a.top_ids = out_top_ids, a.top_logprobs = out_top_logprobs;
  return dtype == SMP_F32 ? launch_scores<float>(a, st) : launch_scores<uint16_t>(a, st);
}

extern "C" smp_status smp_token_logprobs_grad(const void* logits, int32_t rows, int32_t vocab, int64_t stride,
                                              smp_dtype dtype, float temperature, const float* temperatures,
                                              const int32_t* ids, int32_t count, const float* grad_logprobs,
                                              const float* grad_entropy, void* out_grad, int64_t grad_stride,
                                              int32_t* status, void* stream) {
  using namespace smp;
  const smp_status ok = check_rows(logits, rows, vocab, stride, dtype, temperature, temperatures, status);
  if (ok != SMP_OK) return ok;
  if (count < 0 || count > SMP_MAX_ROW_IDS) return SMP_ERR_INVALID_ARG;
  if (count == 0 && !grad_entropy) return SMP_ERR_INVALID_ARG;
  if (!grad_fits(logits, rows, vocab, stride, dtype, out_grad, grad_stride)) return SMP_ERR_INVALID_ARG;
  if (rows > 0 && (!out_grad || (count > 0 && (!ids || !grad_logprobs)))) return SMP_ERR_INVALID_ARG;
  if (misaligned(ids, 4) || misaligned(grad_logprobs, 4) || misaligned(grad_entropy, 4) ||
      misaligned(out_grad, dtype == SMP_F32 ? 4 : 2))
    return SMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    const smp_status rc = clear_status(status, st);
    if (rc != SMP_OK) return rc;
  }
  if (rows == 0) return SMP_OK;
  RowGradArgs a{};
  a.rows.logits = logits, a.rows.stride = stride, a.rows.rows = rows, a.rows.vocab = vocab;
  a.rows.temperature = temperature, a.rows.temperatures = temperatures, a.rows.status = status;
  a.ids = ids, a.count = count, a.values = grad_logprobs, a.weights = grad_entropy;
  a.grad = out_grad, a.grad_stride = grad_stride;
  return dtype == SMP_F32 ? launch_row_grad<float, false>(a, st) : launch_row_grad<uint16_t, false>(a, st);
}
