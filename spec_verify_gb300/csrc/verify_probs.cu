// Verification of drafted tokens against the target's probabilities, from
// random numbers that the caller supplies ("Decoding & Speculative Sampling",
// section 39.4, eqs. 39.3 and 39.4).
//
// Mathematics: with E_i independent exponential variables, P(argmax_i w_i /
// E_i = i) = w_i / sum w (the minimum of exponentials of rates w_i), so the
// replacement needs neither the residual's mass nor a cumulative sum, and a
// maximum, unlike a sum, does not depend on the order in which CTAs meet.
//
// Bound: one row each of p, q and the noise per request from HBM (the accept
// tests touch 2k elements).  A request's row is split over the CTAs of one
// cluster; every warp repeats the accept tests itself (k <= 16 lanes), so the
// stream starts without a barrier, and the CTAs' maxima meet in distributed
// shared memory.
#include <cuda_runtime.h>

#include "cache.cuh"
#include "launch.h"
#include "smp.h"

namespace smp {

struct ProbsArgs {
  const void* p;
  const void* q;
  const int32_t* ids;
  const int32_t* lens;
  const float* uniforms;
  const float* noise;
  int batch, k, vocab;
  int slice;   // elements per CTA, a multiple of 8
  int32_t* out_len;
  int32_t* out_ids;
  int32_t* status;
};

// The best candidate so far of one thread, whose ids ascend: a larger quotient
// replaces it, an equal one does not.
struct Best {
  float score = 0.0f;   // 0 is no candidate
  int id = 0;
};

// The exact quotient is only formed where w / e can reach the best score:
// best * e is off by at most 2^-24, so a w below it by 2^-20 cannot (products
// too small for that bound are not trusted).
__device__ __forceinline__ void race(Best& best, float p, float q, float e, int id) {
  const float w = __fsub_rn(p, q), reach = best.score * e;
  if (w > 0.0f && !(w < reach * (1.0f - 0x1p-20f) && reach > 1e-30f)) {
    const float score = __fdiv_rn(w, e);
    if (score > best.score) best.score = score, best.id = id;
  }
}

// 16 bytes of elements.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int kN = 4;
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ float at(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Piece<uint16_t> {
  static constexpr int kN = 8;
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? bf16_high(w) : bf16_low(w);
  }
};

// The noise of one batch of a thread's pieces.
template <typename T>
struct NoiseBatch {
  static constexpr int kN = Piece<T>::kN, kBatch = kN == 4 ? 2 : 1;
  Piece<float> v[kBatch][kN / 4];
  __device__ __forceinline__ void load(const float* e, int i0, int hi) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (i0 + u * kThreads * kN < hi) {
#pragma unroll
        for (int h = 0; h < kN / 4; ++h) v[u][h].load(e + i0 + u * kThreads * kN + 4 * h);
      }
  }
};

// The best candidate of elements [lo, hi) of one row; q may be nullptr, and
// `certain` is the id where it then counts as 1 (or -1).  16-byte loads, all of
// a batch issued before the first is used, where every row's address allows
// them (vector: lo and hi are then multiples of a piece); else one element per
// load, as many in flight.
// The first batch of noise, which does not depend on the row chosen, comes in
// `ev` when `have_noise`.
template <typename T, bool kQ>
__device__ __forceinline__ Best race_slice(const T* p, const T* q, const float* e, int lo, int hi, int certain,
                                           bool vector, NoiseBatch<T>& ev, bool have_noise) {
  Best best;
  constexpr int kN = Piece<T>::kN, kBatch = NoiseBatch<T>::kBatch;
  if (vector) {
    for (int i0 = lo + int(threadIdx.x) * kN; i0 < hi; i0 += kBatch * kThreads * kN) {
      Piece<T> pv[kBatch], qv[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kThreads * kN;
        if (i < hi) {
          pv[u].load(p + i);
          if (kQ) qv[u].load(q + i);
        }
      }
      if (!have_noise) ev.load(e, i0, hi);
      have_noise = false;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kThreads * kN;
        if (i < hi) {
#pragma unroll
          for (int j = 0; j < kN; ++j)
            race(best, pv[u].at(j), kQ ? qv[u].at(j) : (i + j == certain ? 1.0f : 0.0f), ev.v[u][j / 4].at(j % 4), i + j);
        }
      }
    }
  } else {
    constexpr int kSingles = 4;
    for (int i0 = lo + int(threadIdx.x); i0 < hi; i0 += kSingles * kThreads) {
      float pv[kSingles], qv[kSingles], ev[kSingles];
#pragma unroll
      for (int u = 0; u < kSingles; ++u) {
        const int i = i0 + u * kThreads;
        if (i < hi) {
          pv[u] = load1(p + i);
          qv[u] = kQ ? load1(q + i) : (i == certain ? 1.0f : 0.0f);
          ev[u] = e[i];
        }
      }
#pragma unroll
      for (int u = 0; u < kSingles; ++u)
        if (i0 + u * kThreads < hi) race(best, pv[u], qv[u], ev[u], i0 + u * kThreads);
    }
  }
  return best;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) verify_probs_kernel(const ProbsArgs a) {
  __shared__ uint64_t scratch[kWarps];
  __shared__ uint64_t mail[2][16];
  allow_dependent_launch();
  grid_dependency_wait();
  const int ranks = int(cluster_size()), rank = int(cluster_rank());
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // "this CTA runs": waited for before the mail
  const int b = int(blockIdx.x) / ranks, lane = int(threadIdx.x) & 31;
  const int64_t v = a.vocab;
  const T* p = static_cast<const T*>(a.p) + int64_t(b) * (a.k + 1) * v;
  const T* q = a.q ? static_cast<const T*>(a.q) + int64_t(b) * a.k * v : nullptr;
  const float* e = a.noise + int64_t(b) * v;

  const int lo = min(rank * a.slice, a.vocab), hi = min(lo + a.slice, a.vocab);
  const bool noise_fits = reinterpret_cast<uintptr_t>(e) % 16 == 0 && a.vocab % Piece<T>::kN == 0;
  NoiseBatch<T> noise;
  if (noise_fits) noise.load(e, lo + int(threadIdx.x) * Piece<T>::kN, hi);

  const int drafts = a.lens ? a.lens[b] : a.k;
  bool bad = drafts < 0 || drafts > a.k, reject = false;
  int id = 0;
  if (!bad && lane < drafts) {
    id = a.ids[b * a.k + lane];
    bad = id < 0 || id >= a.vocab;
    if (!bad) {
      const float qx = q ? load1(q + lane * v + id) : 1.0f;
      reject = !(__fmul_rn(a.uniforms[b * a.k + lane], qx) < load1(p + lane * v + id));
    }
  }
  bad = __any_sync(~0u, bad);
  const unsigned rejects = __ballot_sync(~0u, reject);
  const int stop = bad ? 0 : (rejects ? __ffs(rejects) - 1 : drafts);
  const bool replace = stop < drafts;
  uint64_t best = 0;
  if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (!bad) {
    const T* row = p + stop * v;
    const T* draft = replace && q ? q + stop * v : nullptr;
    const int certain = replace && !q ? __shfl_sync(~0u, id, stop) : -1;
    for (int pass = 0; pass < 2; ++pass) {
      // pass 1 is reached when the difference is zero everywhere: the draw is from p itself
      const bool vector =
          noise_fits && (reinterpret_cast<uintptr_t>(row) | reinterpret_cast<uintptr_t>(draft)) % 16 == 0;
      const Best mine =
          pass == 0 && draft
              ? race_slice<T, true>(row, draft, e, lo, hi, -1, vector, noise, noise_fits)
              : race_slice<T, false>(row, nullptr, e, lo, hi, pass == 0 ? certain : -1, vector, noise, noise_fits && pass == 0);
      best = block_max_u64(mine.score > 0.0f ? pack_key_id(__float_as_uint(mine.score), uint32_t(mine.id)) : 0, scratch);
      if (ranks > 1) {
        if (int(threadIdx.x) < ranks) st_cluster_u64(map_rank(smem_addr(&mail[pass][rank]), threadIdx.x), best);
        hw_cluster_sync();
        for (int r = 0; r < ranks; ++r) best = mail[pass][r] > best ? mail[pass][r] : best;
      }
      if (best || !replace) break;
    }
  }
  if (rank == 0 && threadIdx.x < 32) {
    const bool error = bad || best == 0;
    const int token = int(~uint32_t(best));
    if (lane <= a.k) {
      const int out = error ? -1 : lane < stop ? id : lane == stop ? token : -1;
      a.out_ids[int64_t(b) * (a.k + 1) + lane] = out;
    }
    if (lane == 0) {
      a.out_len[b] = error ? -1 : stop;
      if (error && a.status) atomicOr(a.status, bad ? kRowBadDraft : kRowNonFinite);
    }
  }
}

// CTAs per request: as many as fit beside each other in one wave (four CTAs
// per SM), while a CTA keeps 2000 elements.  256 rows of 128256: 61 us with 2
// CTAs a row, 66 with 4 (a second, partial wave), 87 with 1; 32 rows of 32000:
// 7.6 us with 8, 10.1 with 4, 8.3 with 16 (of 128256: 17.3, 26.2 and 19.0), so
// 16 are left to batches of few rows: 16 rows of 32000 6.9 us with 8 and 6.0
// with 16, 1 row 6.6 and 5.2.  The limit is on the low side: 24 rows still take
// 6.2 us with 16 and 7.2 with 8.
static int probs_cluster(int batch, int vocab, int sms) {
  int c = 1;
  while (c < 16 && int64_t(batch) * c * 2 <= int64_t(sms) * 4 && vocab / (2 * c) >= 2000) c *= 2;
  return c == 16 && int64_t(batch) * 8 >= sms ? 8 : c;
}

template <typename T>
static smp_status launch_probs(ProbsArgs a, cudaStream_t st) {
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  const void* kernel = reinterpret_cast<const void*>(&verify_probs_kernel<T>);
  LaunchShape ls;
  ls.pdl = true;
  ls.cluster = forced_cluster() ? forced_cluster() : probs_cluster(a.batch, a.vocab, device_sms(dev));
  cudaError_t err = prepare_kernel(kernel, dev, ls);
  if (err != cudaSuccess) return fail_cuda(err);
  a.slice = ((a.vocab + ls.cluster - 1) / ls.cluster + 7) / 8 * 8;
  err = launch_cluster(kernel, dim3(unsigned(a.batch) * unsigned(ls.cluster)), dim3(kThreads), ls, st, &a);
  if (err != cudaSuccess) return fail_cuda(err);
  return SMP_OK;
}

}  // namespace smp

extern "C" smp_status smp_spec_verify_probs(const void* p, const void* q, const int32_t* draft_ids,
                                            const int32_t* draft_lens, int32_t batch, int32_t k, int32_t vocab,
                                            smp_dtype dtype, const float* uniforms, const float* noise,
                                            int32_t* out_accepted_len, int32_t* out_ids, int32_t* status,
                                            void* stream) {
  using namespace smp;
  if (dtype != SMP_F32 && dtype != SMP_BF16) return SMP_ERR_DTYPE;
  if (batch < 0 || batch > (1 << 20) || k < 0 || k > SMP_MAX_DRAFT || vocab <= 0) return SMP_ERR_INVALID_ARG;
  if (vocab > SMP_MAX_VOCAB) return SMP_ERR_UNSUPPORTED;
  if (batch > 0 && (!p || !noise || !out_accepted_len || !out_ids || (k > 0 && (!draft_ids || !uniforms))))
    return SMP_ERR_INVALID_ARG;
  const size_t elem = dtype == SMP_F32 ? 4 : 2;
  if (misaligned(p, elem) || misaligned(q, elem) || misaligned(draft_ids, 4) || misaligned(draft_lens, 4) ||
      misaligned(uniforms, 4) || misaligned(noise, 4) || misaligned(out_accepted_len, 4) || misaligned(out_ids, 4) ||
      misaligned(status, 4))
    return SMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    const smp_status rc = clear_status(status, st);
    if (rc != SMP_OK) return rc;
  }
  if (batch == 0) return SMP_OK;
  ProbsArgs a{};
  a.p = p;
  a.q = q;
  a.ids = draft_ids;
  a.lens = draft_lens;
  a.uniforms = uniforms;
  a.noise = noise;
  a.batch = batch;
  a.k = k;
  a.vocab = vocab;
  a.out_len = out_accepted_len;
  a.out_ids = out_ids;
  a.status = status;
  return dtype == SMP_F32 ? launch_probs<float>(a, st) : launch_probs<uint16_t>(a, st);
}
