// Distillation from a teacher of whom each row's likeliest tokens are known:
// the divergence of the student's rows (its gradient: row_grad.cuh).
//
// Mathematics: the teacher's ids are taken out of what is summed (as -inf), so that
// the student's mass outside them is a sum of its own, with its own reference, and
// not a difference of two sums.  With R the rest's statistics, K the ids' and both
// together m, Z:
//   ln s_j = (z_j - m) / T - ln Z,   ln s_rest = (m_R - m) / T + ln Z_R - ln Z.
//
// Bound: the loss reads every logit once from HBM: 2039 rows of 152064 in binary32
// 187 us (the copy rate), 4093 in bf16 191.  Short rows take longer, with one
// id as with twenty, most likely for what stands before a row's first load (its ids,
// the cleared bits, two votes): 4096 of 32000 in bf16 57, their log probabilities 42.
#include <cuda_runtime.h>

#include "row_grad.cuh"

namespace smp {

// The loss alone: nothing has to stay on chip, so a row streams through one CTA
// (or the CTAs of a cluster, where rows are few), and a bit per element says
// which are the teacher's.  A warp beside the workers of the first CTA works up the
// teacher's row meanwhile.
template <typename T, int kEach, int kThr, int kOnSm>
__global__ void __launch_bounds__(kThr + 32, kOnSm) distill_loss_kernel(const __grid_constant__ RowGradArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];   // a bit per element of the part
  __shared__ Meeting meet;
  __shared__ RowFacts f;
  const int ranks = int(cluster_size()), rank = int(cluster_rank()), row = int(blockIdx.x) / ranks;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  const T* z = static_cast<const T*>(a.rows.logits) + int64_t(row) * a.rows.stride;
  const Part<T> s(z, a.rows.vocab, a.rows.slice, rank);
  ask_early(a.rows, s.vec() + s.full0, s.full1 - s.full0, 2048);
  grid_dependency_wait();
  cluster_arrive_early(ranks);

  const float temperature = row_temperature(a.rows, row), c = __fdiv_rn(kLog2e, temperature);
  constexpr int kIds = (kMaxIds + kThr - 1) / kThr;   // of a thread
  int id[kIds];
  bool some = false, beyond = false;
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    const int k = tid + i * kThr;
    id[i] = k < a.count ? a.ids[int64_t(row) * a.count + k] : -1;
    some |= id[i] >= 0, beyond |= id[i] >= a.rows.vocab;
  }
  Inputs<T, kEach> in;
  if (warp == kThr / 32 && rank == 0) in.ask(a, row, z);
  uint32_t* bits = reinterpret_cast<uint32_t*>(dynamic);
  for (int i = tid; i < (a.rows.slice + 31) / 32; i += kThr + 32) bits[i] = 0;
  const bool live = __syncthreads_or(some), past = __syncthreads_or(beyond);
  int flags = (past ? kRowBadToken : 0) | (temperature_fits(temperature) ? 0 : kRowBadParams);
  if (!live || flags) {
    cluster_all_run(ranks);
    if (rank == 0 && tid == 0) {
      a.loss[row] = live ? __uint_as_float(0x7FC00000u) : 0.0f;
      if (live && a.rows.status) atomicOr(a.rows.status, flags);
    }
    return;
  }
  if (warp == kThr / 32) {
    if (rank == 0) learn_row<true>(in, a.count, a.tail != 0, temperature, 1.0f, f);
    cluster_all_run(ranks);
  } else {
#pragma unroll
    for (int i = 0; i < kIds; ++i)
      if (s.holds(id[i])) atomicOr(&bits[(id[i] - s.first) >> 5], 1u << ((id[i] - s.first) & 31));
    const int edge = s.edge();
    const float at_edge = edge >= 0 ? clean(load1(z + edge)) : -INFINITY;
    workers_sync<kThr>();
    Running<T, false> run;
    const unsigned char* bytes = dynamic;
    stream<kThr>(
        s, run, temperature, c,
        [&](uint4& y, int k) {
          const int j = s.full0 + k;
          if (j < s.full1) {
            const uint32_t b = Part<T>::kPer == 8 ? bytes[j] : bytes[j >> 1] >> (4 * (j & 1)) & 15u;
            if (b) erase(y, b, T{});
          }
        },
        [](float) {});
    if (edge >= 0 && !(bits[(edge - s.first) >> 5] >> ((edge - s.first) & 31) & 1u)) run.add_one(at_edge, temperature, c);
    const Stats part = warp_join<false>(run.stats(), c);
    if (lane == 0) meet.warp[warp] = part;
    cluster_all_run(ranks);
    workers_sync<kThr>();
    if (warp == 0) {
      const Stats cta = warp_join<false>(lane < kThr / 32 ? meet.warp[lane] : Stats{-INFINITY, 0.0f, 0.0f}, c);
      post(meet, rank, ranks, cta.m, cta.z, 0.0f, 0.0f);
    }
  }
  cluster_meet(ranks);
  if (rank != 0 || warp != kThr / 32) return;
  const float4 p = posted(meet, ranks);
  const Stats r = warp_join<false>(Stats{p.x, p.y, 0.0f}, c);
  const Whole all(r, f.on_ids, c);
  flags = f.flags;
  if (!flags && !(fabsf(all.m) < INFINITY)) flags = kRowNonFinite;
  const float loss = row_loss(f.ids, f.add, f.logit, 32 * kEach, f.t_log_t, r, all.m, all.zsum, r.z > 0.0f ? f.rest : 0.0f,
                              temperature);
  if (lane == 0) {
    a.loss[row] = flags ? __uint_as_float(0x7FC00000u) : loss;
    if (flags && a.rows.status) atomicOr(a.rows.status, flags);
  }
}

template <typename T, int kThr, int kOnSm>
static smp_status launch_distill_loss_of(const RowGradArgs& a, const LaunchShape& ls, cudaStream_t st) {
  const void* kernel = a.count <= 32   ? reinterpret_cast<const void*>(&distill_loss_kernel<T, 1, kThr, kOnSm>)
                       : a.count <= 64 ? reinterpret_cast<const void*>(&distill_loss_kernel<T, 2, kThr, kOnSm>)
                                       : reinterpret_cast<const void*>(&distill_loss_kernel<T, 4, kThr, kOnSm>);
  return launch_rows(kernel, a, ls, st, kThr + 32);
}

template <typename T>
static smp_status launch_distill_loss(RowGradArgs a, cudaStream_t st) {
  LaunchShape ls;
  const smp_status ok = shape_parts(a.rows, int(sizeof(T)), 8 * 1024, ls);
  if (ok != SMP_OK) return ok;
  ls.smem = size_t(a.rows.slice + 127) / 128 * 16;
  // Small CTAs for rows that are many and not long (more rows in flight): 4096 rows of 32000 in bf16 63 us with 64
  // threads, 69 with 128, 74 with 256; 1200 of 8192 9.7, 12.9 and 15.3; but 300 of 32000 18.5, 12.3 and 9.6, and 4096 of
  // 128256 212, 215 and 202.
  if (ls.cluster == 1 && !forced_cluster() && int64_t(a.rows.vocab) * int(sizeof(T)) < 200 * 1024 &&
      a.rows.rows >= 6 * device_sms(current_device()))
    return launch_distill_loss_of<T, 64, 9>(a, ls, st);
  return four_on_sm(a.rows, ls) ? launch_distill_loss_of<T, kThreads, 4>(a, ls, st)
                                : launch_distill_loss_of<T, kThreads, 3>(a, ls, st);
}

}  // namespace smp

extern "C" smp_status smp_distill(const void* logits, int32_t rows, int32_t vocab, int64_t stride, smp_dtype dtype,
                                  float temperature, const float* temperatures, const int32_t* teacher_ids,
                                  const float* teacher_logprobs, int32_t count, int32_t tail, const float* weights,
                                  float* out_loss, void* out_grad, int64_t grad_stride, int32_t* status, void* stream) {
  using namespace smp;
  const smp_status ok = check_rows(logits, rows, vocab, stride, dtype, temperature, temperatures, status);
  if (ok != SMP_OK) return ok;
  if (count < 1 || count > SMP_MAX_ROW_IDS) return SMP_ERR_INVALID_ARG;
  if (out_grad && !grad_fits(logits, rows, vocab, stride, dtype, out_grad, grad_stride)) return SMP_ERR_INVALID_ARG;
  if (rows > 0 && (!teacher_ids || !teacher_logprobs || !out_loss)) return SMP_ERR_INVALID_ARG;
  if (misaligned(teacher_ids, 4) || misaligned(teacher_logprobs, 4) || misaligned(weights, 4) || misaligned(out_loss, 4) ||
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
  a.ids = teacher_ids, a.values = teacher_logprobs, a.count = count, a.tail = tail;
  a.weights = weights, a.loss = out_loss, a.grad = out_grad, a.grad_stride = grad_stride;
  if (!out_grad) return dtype == SMP_F32 ? launch_distill_loss<float>(a, st) : launch_distill_loss<uint16_t>(a, st);
  return dtype == SMP_F32 ? launch_row_grad<float, true>(a, st) : launch_row_grad<uint16_t, true>(a, st);
}
