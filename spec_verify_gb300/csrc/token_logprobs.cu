// Log probabilities of given tokens, entropies and likeliest tokens of rows of
// logits, and the gradient of log probabilities and entropies.
//
// Bound: the forward call reads every logit once from HBM, the gradient reads
// and writes them once (scores.cuh says how a row stays on chip).
//
// Likeliest tokens: each CTA finds the `top` largest of its slice before the
// cluster's barrier, so that the lists travel with the sums.  The n-th largest
// of its 256 threads' maxima is at most the slice's n-th largest element, since
// n threads each hold an element that large: everything at or above it (a few
// more than n) is collected and ranked by comparing packed (value, id) words.
// The first CTA of the cluster merges the sorted lists by binary search.
#include <cuda_runtime.h>

#include <algorithm>

#include "row_grad.cuh"

namespace smp {

constexpr int kCandidates = 512;   // collected before the slow exact way takes over

struct ScoreArgs {
  RowsArgs rows;
  const int32_t* ids;
  int count, top;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int run_room;   // most runs of any CTA
};

// A thread's units of kUnit vectors come in up to kRuns runs whose maxima are
// kept, `units` in each.
constexpr int kRuns = 16;

// What slice_top works with, in shared memory.
struct TopRoom {
  alignas(16) uint16_t keys[kThreads];
  int hits[kCandidates];           // thread | run << 8
  uint64_t cand[kCandidates];
  uint64_t scratch[kWarps];
  uint32_t bound;
  int hit_count, found;
};

// The largest value that `top` of the 256 keys reach, in one warp: bisection
// between the smallest and the largest key, which are a few hundred apart in
// ordinary rows (256 threads that count keys bit by bit behind a barrier each
// took 1.1 to 2.4 us, this 0.3).
__device__ __forceinline__ uint32_t nth_key(const uint16_t* keys, int top) {
  const uint4 w = reinterpret_cast<const uint4*>(keys)[int(threadIdx.x) & 31];
  const uint32_t k[8] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16, w.z & 0xFFFFu, w.z >> 16, w.w & 0xFFFFu, w.w >> 16};
  uint32_t lo = k[0], hi = k[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = min(lo, k[i]), hi = max(hi, k[i]);
  lo = __reduce_min_sync(~0u, lo), hi = __reduce_max_sync(~0u, hi);
  if (top == 1) return hi;
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) >> 1;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) n += k[i] >= mid;
    if (int(__reduce_add_sync(~0u, n)) >= top) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The `top` largest elements of the part, in order, as packed words (0: none)
// to `list` of the cluster's first CTA.  `mine` is the largest of this thread's
// elements, run_top[run][thread] of each run, `edge` its edge element's id; `x`
// are the thread's vectors where it has two units of them at most.
template <typename T>
__device__ __forceinline__ void slice_top(const Part<T>& s, float mine, const float* run_top, int runs, int units, int edge,
                                          const uint4 (&x)[2][kUnit], int top, TopRoom& room, uint64_t* list, int ranks) {
  using V = RowVec<T>;
  constexpr int kPer = V::kPer;
  const int tid = int(threadIdx.x);
  const uint32_t key = key_of_bits(__float_as_uint(mine)) >> 16;
  room.keys[tid] = uint16_t(key);
  if (tid == 0) room.hit_count = room.found = 0;
  __syncthreads();
  if (tid < 32) {
    const uint32_t b = nth_key(room.keys, top);
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
  const bool at_hand = vecs < 2 * kUnit * kThreads;
  if (mine >= limit) {
    if (edge >= 0) {
      const float v = Elem<T>::widen(s.row[edge]);
      if (v >= limit) keep(atomicAdd(&room.found, 1), v, edge);
    }
    if (at_hand) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int at[kUnit];
#pragma unroll
        for (int u = 0; u < kUnit; ++u) {
          const int k = tid + (h * kUnit + u) * kThreads;
          at[u] = k < vecs ? s.first + (s.full0 + k) * kPer : -1;
        }
        take(x[h], at);
      }
    } else {
      uint32_t mask = 0;
#pragma unroll 4
      for (int run = 0; run < runs; ++run) mask |= (run_top[run * kThreads + tid] >= limit ? 1u : 0u) << run;
      int place = mask ? atomicAdd(&room.hit_count, __popc(mask)) : 0;
      for (; mask; mask &= mask - 1, ++place)
        if (place < kCandidates) room.hits[place] = tid | (__ffs(mask) - 1) << 8;
    }
  }
  __syncthreads();
  const int hits = room.hit_count, run_vecs = units * kUnit;
  bool listed = hits <= kCandidates;
  if (listed && hits) {   // the runs' vectors again (from L2), every thread some at a time
    for (int i0 = tid; i0 < hits * run_vecs; i0 += kUnit * kThreads) {
      uint4 y[kUnit];
      int at[kUnit];
#pragma unroll
      for (int u = 0; u < kUnit; ++u) {
        const int i = i0 + u * kThreads;
        at[u] = -1;
        if (i < hits * run_vecs) {
          const int hit = room.hits[i / run_vecs], k = (hit & 255) + ((hit >> 8) * run_vecs + i % run_vecs) * kThreads;
          if (k < vecs) at[u] = s.first + (s.full0 + k) * kPer, y[u] = s.vec()[s.full0 + k];
        }
      }
      take(y, at);
    }
    __syncthreads();
  }
  listed = listed && room.found <= kCandidates;
  const uint32_t to = ranks > 1 ? map_rank(smem_addr(list), 0) : 0;
  auto put = [&](int place, uint64_t v) {
    if (ranks > 1) st_cluster_u64(to + uint32_t(place) * 8u, v);
    else list[place] = v;
  };
  if (listed) {   // a candidate's place is the number of larger ones: four lanes count for each
    const int have = room.found;
    for (int i0 = 0; i0 < have; i0 += kThreads / 4) {
      const int i = i0 + (tid >> 2);
      const uint64_t v = i < have ? room.cand[i] : ~0ull;
      int place = 0;
#pragma unroll 8
      for (int j = tid & 3; j < have; j += 4) place += room.cand[j] > v;
      place += __shfl_xor_sync(~0u, place, 1);
      place += __shfl_xor_sync(~0u, place, 2);
      if ((tid & 3) == 0 && i < have && place < top) put(place, v);
    }
    for (int i = have + tid; i < top; i += kThreads) put(i, 0);
  } else {   // many equal values: one maximum after another, each below the last
    uint64_t last = ~0ull;
    for (int n = 0; n < top; ++n) {
      uint64_t best = 0;
      for (int id = s.lo + tid; id < s.hi; id += kThreads) {
        const uint32_t k = key_of_bits(Elem<T>::bits(s.row[id]));
        const uint64_t v = k > kKeyNegInf ? pack_key_id(k, uint32_t(id)) : 0;
        if (v < last && v > best) best = v;
      }
      best = block_max_u64(best, room.scratch);
      if (tid == 0) put(n, best);
      if (best == 0) {
        for (int i = n + 1 + tid; i < top; i += kThreads) put(i, 0);
        break;
      }
      last = best;
    }
  }
}

template <typename T, bool kEntropy, bool kTop>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(const __grid_constant__ ScoreArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];   // with kTop: TopRoom, the runs' maxima, the lists
  __shared__ Meeting meet;
  const int ranks = int(cluster_size()), rank = int(cluster_rank()), row = int(blockIdx.x) / ranks;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  grid_dependency_wait();
  cluster_arrive_early(ranks);

  const T* z = static_cast<const T*>(a.rows.logits) + int64_t(row) * a.rows.stride;
  const Part<T> s(z, a.rows.vocab, a.rows.slice, rank);
  const float temperature = row_temperature(a.rows, row), c = __fdiv_rn(kLog2e, temperature);
  const int id = tid < a.count ? a.ids[int64_t(row) * a.count + tid] : -1;
  float* logprobs = a.logprobs + int64_t(row) * a.count;
  if (!kEntropy && !kTop && !__syncthreads_or(id >= 0)) {   // every id is padding
    cluster_all_run(ranks);
    if (rank == 0 && tid < a.count) logprobs[tid] = 0.0f;
    return;
  }
  TopRoom& room = *reinterpret_cast<TopRoom*>(dynamic);
  float* run_top = reinterpret_cast<float*>(dynamic + sizeof(TopRoom));
  const int units_all = (s.full1 - s.full0 + kThreads * kUnit - 1) / (kThreads * kUnit);   // of a thread
  const int units = (units_all + kRuns - 1) / kRuns, runs = units ? (units_all + units - 1) / units : 0;
  uint64_t* lists = reinterpret_cast<uint64_t*>(run_top + a.run_room * kThreads);
  int flags = temperature_fits(temperature) ? 0 : kRowBadParams;
  Stats all{-INFINITY, 0.0f, 0.0f};
  const float value = flags == 0 && s.holds(id) ? clean(load1(z + id)) : 0.0f;
  if (flags == 0) {
    Running<T, kEntropy> run;
    const int edge = s.edge();
    const float at_edge = edge >= 0 ? clean(load1(z + edge)) : -INFINITY;
    float best = -INFINITY, mine = at_edge;   // the largest of the run, of the thread
    int in_run = 0, r = 0;
    uint4 x[2][kUnit];
    stream<true>(s, run, x, temperature, c, [](uint4&, int) {}, [&](float top) {
      if (kTop) {
        best = fmaxf(best, top), mine = fmaxf(mine, top);
        if (++in_run == units) {
          run_top[r * kThreads + tid] = best;
          best = -INFINITY, in_run = 0, ++r;
        }
      }
    });
    run.add_one(at_edge, temperature, c);
    if (kTop) {
      for (; r < runs; ++r, best = -INFINITY) run_top[r * kThreads + tid] = best;
    }
    const Stats part = warp_join<kEntropy>(run.stats(), c);
    if (lane == 0) meet.warp[warp] = part;
    cluster_all_run(ranks);
    if (kTop) slice_top(s, mine, run_top, runs, units, edge, x, a.top, room, lists + rank * a.top, ranks);
    __syncthreads();
    if (warp == 0) {
      const Stats cta = warp_join<kEntropy>(lane < kWarps ? meet.warp[lane] : Stats{-INFINITY, 0.0f, 0.0f}, c);
      post(meet, rank, ranks, cta.m, cta.z, cta.s, 0.0f);
    }
    cluster_meet(ranks);
    const float4 p = posted(meet, ranks);
    all = warp_join<kEntropy>(Stats{p.x, p.y, p.z}, c);
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
      for (int i = tid; i < a.top; i += kThreads) top_ids[i] = -1, top_logprobs[i] = nan;
      return;
    }
    if (ranks == 1) {   // one list, in order
      for (int i = tid; i < a.top; i += kThreads) {
        const uint64_t v = lists[i];
        top_ids[i] = v ? int32_t(~uint32_t(v)) : -1;
        top_logprobs[i] = v ? logprob(value_of_key(uint32_t(v >> 32))) : -INFINITY;
      }
      return;
    }
    // A token's place is the number of larger ones in all lists, by bisection in
    // all of them at once.  An entry that is none finds all tokens larger: those of
    // list 0 fill the places that are left.
    for (int e = tid; e < ranks * a.top; e += kThreads) {
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
      if (place < a.top) {
        top_ids[place] = v ? int32_t(~uint32_t(v)) : -1;
        top_logprobs[place] = v ? logprob(value_of_key(uint32_t(v >> 32))) : -INFINITY;
      }
    }
  }
}

template <typename T>
static smp_status launch_scores(ScoreArgs a, cudaStream_t st) {
  const void* kernel =
      a.entropy ? (a.top ? reinterpret_cast<const void*>(&token_logprobs_kernel<T, true, true>)
                         : reinterpret_cast<const void*>(&token_logprobs_kernel<T, true, false>))
                : (a.top ? reinterpret_cast<const void*>(&token_logprobs_kernel<T, false, true>)
                         : reinterpret_cast<const void*>(&token_logprobs_kernel<T, false, false>));
  LaunchShape ls;
  const smp_status ok = shape_parts(a.rows, int(sizeof(T)), ls);
  if (ok != SMP_OK) return ok;
  if (a.top) {
    const int unit = kThreads * kUnit * RowVec<T>::kPer;
    a.run_room = std::min(kRuns, (a.rows.slice + unit - 1) / unit);
    ls.smem = sizeof(TopRoom) + size_t(a.run_room) * kThreads * 4 + size_t(ls.cluster) * a.top * 8;
  }
  return launch_rows(kernel, a, ls, st);
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
  if (!grad_fits(logits, rows, vocab, stride, out_grad, grad_stride)) return SMP_ERR_INVALID_ARG;
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
