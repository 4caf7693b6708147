// Distillation from a teacher of whom each row's likeliest tokens are known:
// the divergence of the student's rows, and its gradient in the same pass.
//
// Mathematics: the teacher's ids are taken out of the slice (their places hold
// -inf while the rest is summed), so that the student's mass outside them is a
// sum of its own, with its own maximum, and not a difference of two sums.  With
// R the rest's statistics, K the ids' and both together m, Z:
//   ln s_j = (z_j - m) / T - ln Z,   ln s_rest = (m_R - m) / T + ln Z_R - ln Z,
//   dz_j = 2^((z_j - m_R) c) (w / T) ((sum t + r) 2^((m_R - m) c) / Z - r / Z_R)
// outside the ids, and (w / T) (s_j (sum t + r) - t) on them.
//
// Bound: the loss reads every logit once from HBM, the gradient reads and
// writes them once (scores.cuh says how a row stays on chip).
#include <cuda_runtime.h>

#include "scores.cuh"

namespace smp {

struct DistillArgs {
  RowsArgs rows;
  const int32_t* ids;
  const float* values;
  int count, tail;
  const float* weights;
  float* loss;
  void* grad;
  int64_t grad_stride;
};

// The teacher's row: t and ln t of each place, sum t, r.
struct Teacher {
  int ids[kMaxIds];
  float t[kMaxIds], log_t[kMaxIds];
  float given, rest;
  int flags;
  bool live;
};

// Fills `teach` (one warp).  r = 1 - sum t is a small difference: it is taken
// from fixed-point exponentials, which are exact to 2^-45 each.
__device__ __forceinline__ void read_teacher(const DistillArgs& a, int row, Teacher& teach) {
  const int lane = int(threadIdx.x) & 31;
  constexpr int kEach = kMaxIds / 32;
  float l[kEach];
  bool live[kEach], any = false, past = false, bad = false;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int k = lane + 32 * i;
    const int id = k < a.count ? a.ids[int64_t(row) * a.count + k] : -1;
    live[i] = id >= 0;
    l[i] = live[i] ? a.values[int64_t(row) * a.count + k] : -INFINITY;
    teach.ids[k] = id;
    any |= live[i];
    past |= id >= a.rows.vocab;
    bad |= !(l[i] < INFINITY);
    top = fmaxf(top, l[i]);
  }
  float log_sum = 0.0f, given = 0.0f, rest = 0.0f;
  if (a.tail) {
    uint64_t mass = 0;
    const RowScale unit = make_row_scale_unit(0.0f);
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (live[i]) mass += mass_fixed(fminf(l[i], 1.0f), unit, kExp2Table);
    mass = warp_sum<uint64_t>(mass);
    bad |= mass > kFixedOne + (kFixedOne >> 6);
    given = float(mass) * 0x1p-44f;
    rest = mass < kFixedOne ? float(kFixedOne - mass) * 0x1p-44f : 0.0f;
  } else {
    top = warp_max_f(top);
    bad |= !(top > -INFINITY);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += expf(__fsub_rn(l[i], top));
    log_sum = __fadd_rn(top, logf(warp_sum_f(sum)));
    given = 1.0f;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int k = lane + 32 * i;
    teach.log_t[k] = __fsub_rn(l[i], log_sum);
    teach.t[k] = live[i] ? expf(teach.log_t[k]) : 0.0f;
  }
  any = __any_sync(~0u, any), past = __any_sync(~0u, past), bad = __any_sync(~0u, bad);
  if (lane == 0) {
    teach.given = given, teach.rest = rest, teach.live = any;
    teach.flags = (past ? kRowBadToken : 0) | (bad ? kRowBadParams : 0);
  }
}

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

// The row's loss, in one warp, from the joined statistics outside the ids (r)
// and on them (k); m and zsum: of the whole row.
__device__ __forceinline__ float row_loss(const Teacher& teach, const float* student, const Stats& r, float m, float zsum,
                                          float rest, float temperature) {
  const int lane = int(threadIdx.x) & 31;
  const float log_z = logf(zsum);
  float loss = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxIds / 32; ++i) {
    const int n = lane + 32 * i;
    const float t = teach.t[n];
    if (t > 0.0f) {   // t (ln t - ln s), with t times a far logit before the division, which it might overflow
      const float far = __fdiv_rn(__fmul_rn(t, __fsub_rn(student[n], m)), temperature);
      loss = __fadd_rn(loss, __fsub_rn(__fmul_rn(t, __fadd_rn(teach.log_t[n], log_z)), far));
    }
  }
  loss = warp_sum_f(loss);
  if (rest > 0.0f) {
    const float far = __fdiv_rn(__fmul_rn(rest, __fsub_rn(r.m, m)), temperature);
    loss = __fadd_rn(loss, __fsub_rn(__fmul_rn(rest, __fadd_rn(logf(rest), __fsub_rn(log_z, logf(r.z)))), far));
  }
  return loss;
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

// The loss alone: nothing has to stay on chip, so a row streams through one CTA
// (or the CTAs of a cluster, where rows are few), and a bit per element says
// which are the teacher's.  The cluster's first CTA holds the teacher's row.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) distill_loss_kernel(const __grid_constant__ DistillArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];   // a bit per element of the part
  __shared__ Meeting meet;
  __shared__ Stats ids_warp[kMaxIds / 32];
  __shared__ Teacher teach;
  __shared__ float student[kMaxIds];
  const int ranks = int(cluster_size()), rank = int(cluster_rank()), row = int(blockIdx.x) / ranks;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  grid_dependency_wait();
  cluster_arrive_early(ranks);

  const T* z = static_cast<const T*>(a.rows.logits) + int64_t(row) * a.rows.stride;
  const Part<T> s(z, a.rows.vocab, a.rows.slice, rank);
  const float temperature = row_temperature(a.rows, row), c = __fdiv_rn(kLog2e, temperature);
  const int id = tid < a.count ? a.ids[int64_t(row) * a.count + tid] : -1;
  uint32_t* bits = reinterpret_cast<uint32_t*>(dynamic);
  for (int i = tid; i < (a.rows.slice + 31) / 32; i += kThreads) bits[i] = 0;
  const bool live = __syncthreads_or(id >= 0), past = __syncthreads_or(id >= a.rows.vocab);
  int flags = (past ? kRowBadToken : 0) | (temperature_fits(temperature) ? 0 : kRowBadParams);
  if (!live || flags) {
    cluster_all_run(ranks);
    if (rank == 0 && tid == 0) {
      a.loss[row] = live ? __uint_as_float(0x7FC00000u) : 0.0f;
      if (live && a.rows.status) atomicOr(a.rows.status, flags);
    }
    return;
  }
  if (s.holds(id)) atomicOr(&bits[(id - s.first) >> 5], 1u << ((id - s.first) & 31));
  const float value = rank == 0 && id >= 0 ? clean(load1(z + id)) : -INFINITY;
  if (rank == 0 && warp == 0) read_teacher(a, row, teach);
  __syncthreads();
  Running<T, false> run;
  const int edge = s.edge();
  const bool apart = edge >= 0 && (bits[(edge - s.first) >> 5] >> ((edge - s.first) & 31) & 1u);
  const float at_edge = edge >= 0 && !apart ? clean(load1(z + edge)) : -INFINITY;
  const unsigned char* bytes = dynamic;
  uint4 x[2][kUnit];
  stream(
      s, run, x, temperature, c,
      [&](uint4& y, int k) {
        const int j = s.full0 + k;
        if (j < s.full1) {
          const uint32_t b = Part<T>::kPer == 8 ? bytes[j] : bytes[j >> 1] >> (4 * (j & 1)) & 15u;
          if (b) erase(y, b, T{});
        }
      },
      [](float) {});
  run.add_one(at_edge, temperature, c);
  const Stats part = warp_join(run.stats(), c);
  if (lane == 0) meet.warp[warp] = part;
  if (rank == 0 && warp < kMaxIds / 32) {
    float sum;
    const bool counts = id >= 0 && value > -INFINITY && first_of_id(teach.ids, teach.t, a.count, tid, sum);
    const Stats on_ids = warp_join(counts ? Stats{value, 1.0f, 0.0f} : Stats{-INFINITY, 0.0f, 0.0f}, c);
    if (lane == 0) ids_warp[warp] = on_ids;
    student[tid] = value;
  }
  cluster_all_run(ranks);
  __syncthreads();
  const Stats none{-INFINITY, 0.0f, 0.0f};
  if (warp == 0) {
    const Stats cta = warp_join(lane < kWarps ? meet.warp[lane] : none, c);
    post(meet, rank, ranks, cta.m, cta.z, 0.0f, 0.0f);
  }
  cluster_meet(ranks);
  if (rank != 0 || warp != 0) return;
  const float4 p = posted(meet, ranks);
  const Stats r = warp_join(Stats{p.x, p.y, 0.0f}, c);
  const Stats k = warp_join(lane < kMaxIds / 32 ? ids_warp[lane] : none, c);
  const Whole all(r, k, c);
  flags = teach.flags;
  if (!flags && !(fabsf(all.m) < INFINITY)) flags = kRowNonFinite;
  const float loss = row_loss(teach, student, r, all.m, all.zsum, r.z > 0.0f ? teach.rest : 0.0f, temperature);
  if (lane == 0) {
    a.loss[row] = flags ? __uint_as_float(0x7FC00000u) : loss;
    if (flags && a.rows.status) atomicOr(a.rows.status, flags);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) distill_grad_kernel(const __grid_constant__ DistillArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ Meeting meet;
  __shared__ Stats ids_warp[kMaxIds / 32];
  __shared__ Teacher teach;
  __shared__ uint64_t bar;
  __shared__ float student[kMaxIds];   // the cluster's first CTA: the student's logits of the ids
  constexpr int kPer = RowVec<T>::kPer;
  const int ranks = int(cluster_size()), rank = int(cluster_rank()), row = int(blockIdx.x) / ranks;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  if (tid == 0) {
    mbar_init(&bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  grid_dependency_wait();
  cluster_arrive_early(ranks);

  const T* z = static_cast<const T*>(a.rows.logits) + int64_t(row) * a.rows.stride;
  T* out = static_cast<T*>(a.grad) + int64_t(row) * a.grad_stride;
  const float temperature = row_temperature(a.rows, row), c = __fdiv_rn(kLog2e, temperature);
  const Slice<T> s(reinterpret_cast<T*>(dynamic), z, a.rows.vocab, a.rows.slice, rank);
  const float nan = __uint_as_float(0x7FC00000u);
  if (warp == 0) read_teacher(a, row, teach);
  __syncthreads();
  int flags = teach.flags | (temperature_fits(temperature) ? 0 : kRowBadParams);
  if (!teach.live || flags) {
    cluster_all_run(ranks);
    if (rank == 0 && tid == 0) {
      a.loss[row] = teach.live ? nan : 0.0f;
      if (teach.live && a.rows.status) atomicOr(a.rows.status, flags);
    }
    s.fill(teach.live ? nan : 0.0f);
    s.store(out);
    return;
  }
  s.load(z, a.rows.vocab, &bar);
  const float weight = a.weights ? a.weights[row] : 1.0f;
  const int id = tid < kMaxIds ? teach.ids[tid] : -1;
  const bool here = s.holds(id);
  float t_here = 0.0f;   // the id's t, over all its places
  const bool first = here && first_of_id(teach.ids, teach.t, a.count, tid, t_here);
  const bool late = slice_is_late(&bar, a.rows.wait_limit);
  const float value = here ? s.at(id) : -INFINITY;
  __syncthreads();
  if (first) s.buf[id - s.first] = RowVec<T>::minus_inf();
  __syncthreads();
  const Stats part = warp_stats<T, false>(s, thread_top(s), temperature, c);
  const Stats on_ids = warp_join(first && value > -INFINITY ? Stats{value, 1.0f, 0.0f} : Stats{-INFINITY, 0.0f, 0.0f}, c);
  if (lane == 0) {
    meet.warp[warp] = part;
    if (warp < kMaxIds / 32) ids_warp[warp] = on_ids;
  }
  cluster_all_run(ranks);
  if (here) {
    if (ranks == 1) student[tid] = value;
    else asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_rank(smem_addr(&student[tid]), 0)), "f"(value) : "memory");
  }
  __syncthreads();
  if (warp == 0) {
    const Stats none{-INFINITY, 0.0f, 0.0f};
    const Stats r = warp_join(lane < kWarps ? meet.warp[lane] : none, c);
    const Stats k = warp_join(lane < kMaxIds / 32 ? ids_warp[lane] : none, c);
    post(meet, rank, ranks, r.m, r.z, k.m, late ? -1.0f : k.z);
  }
  cluster_meet(ranks);
  const float4 p = posted(meet, ranks);
  const Stats r = warp_join(Stats{p.x, p.y, 0.0f}, c), k = warp_join(Stats{p.z, fmaxf(p.w, 0.0f), 0.0f}, c);
  const Whole all(r, k, c);
  if (!(fabsf(all.m) < INFINITY)) flags = kRowNonFinite;
  if (__any_sync(~0u, lane < ranks && p.w < 0.0f)) flags = kRowTimeout;
  if (flags) {
    if (rank == 0 && tid == 0) {
      a.loss[row] = nan;
      if (a.rows.status) atomicOr(a.rows.status, flags);
    }
    s.fill(nan);
    s.store(out);
    return;
  }
  const float rest = r.z > 0.0f ? teach.rest : 0.0f;
  if (rank == 0 && warp == 0) {
    const float loss = row_loss(teach, student, r, all.m, all.zsum, rest, temperature);
    if (lane == 0) a.loss[row] = loss;
  }
  const float scale = __fdiv_rn(weight, temperature), inv_z = __fdiv_rn(1.0f, all.zsum);
  const float total = rest > 0.0f ? 1.0f : teach.given;
  const float outside = r.z > 0.0f ? scale * (total * all.reach * inv_z - __fdiv_rn(rest, r.z)) : 0.0f;
  const float top = r.z > 0.0f ? r.m : 0.0f;   // nothing outside the ids: any finite reference
  const uint32_t floor = floor_word<T>(top, temperature);
  for (int j = tid; j < s.vecs; j += kThreads) {
    float v[kPer];
    RowVec<T>::get(s.vec()[j], floor, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = __fmul_rn(ex2_approx(__fmul_rn(__fsub_rn(v[i], top), c)), outside);
    s.vec()[j] = RowVec<T>::put(v);
  }
  __syncthreads();
  if (first) {
    const float share = value > -INFINITY ? __fmul_rn(ex2_approx(__fmul_rn(__fsub_rn(value, all.m), c)), inv_z) : 0.0f;
    store1(s.buf + (id - s.first), __fmul_rn(scale, __fmaf_rn(share, total, -t_here)));
  }
  s.store(out);
}

template <typename T>
static smp_status launch_distill(DistillArgs a, cudaStream_t st) {
  LaunchShape ls;
  const smp_status ok = a.grad ? shape_slices(a.rows, int(sizeof(T)), ls) : shape_parts(a.rows, int(sizeof(T)), ls);
  if (ok != SMP_OK) return ok;
  if (!a.grad) ls.smem = size_t(a.rows.slice + 127) / 128 * 16;
  return launch_rows(a.grad ? reinterpret_cast<const void*>(&distill_grad_kernel<T>)
                            : reinterpret_cast<const void*>(&distill_loss_kernel<T>),
                     a, ls, st);
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
  if (out_grad && !grad_fits(logits, rows, vocab, stride, out_grad, grad_stride)) return SMP_ERR_INVALID_ARG;
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
  DistillArgs a{};
  a.rows.logits = logits, a.rows.stride = stride, a.rows.rows = rows, a.rows.vocab = vocab;
  a.rows.temperature = temperature, a.rows.temperatures = temperatures, a.rows.status = status;
  a.ids = teacher_ids, a.values = teacher_logprobs, a.count = count, a.tail = tail, a.weights = weights;
  a.loss = out_loss, a.grad = out_grad, a.grad_stride = grad_stride;
  return dtype == SMP_F32 ? launch_distill<float>(a, st) : launch_distill<uint16_t>(a, st);
}
