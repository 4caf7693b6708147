// Block tables and slot maps of one step, from request lengths.
//
// Mathematics: with n_b the blocks that request b lacks, its first new block
// is entry head + sum_{c<b} n_c of the free list and its first token is
// sum_{c<b} add_c: two exclusive prefix sums, after which every token's
// place follows from its own request alone.
//
// Bound: 16 bytes written per token (position, request, slot) and the latency
// of one launch for small steps.  32 requests of 5 tokens: 3.5 us; 509 prompts
// into a million places: 10.9 us, 1.6 TB/s, about half of it the prefix sums.  Tokens, not requests, are split over the
// CTAs, since one prompt can be longer than all other requests together.
// Every CTA repeats the prefix sums over all requests (12 bytes each, from
// L2) instead of waiting for another kernel or CTA, keeps those that meet its
// own tokens in shared memory, and finds each token's request by a running
// maximum over the marks that the requests' first tokens leave.
#include <cuda_runtime.h>

#include "cache.cuh"
#include "launch.h"
#include "smp.h"

namespace smp {

constexpr uint32_t kPlanMost = 0x7FFFFFFF;    // where the prefix sums stop: beyond any max_tokens and free_count

struct PlanArgs {
  const int32_t* lens;
  const int32_t* add;
  const int32_t* held;
  int batch;
  const int32_t* free_blocks;
  int free_count;
  const int32_t* free_head;
  int32_t* table;
  int stride;
  int shift;        // log2(block_size)
  int num_blocks;
  int max_tokens;
  int32_t* out_lens;
  int32_t* out_held;
  int32_t* out_head;
  int32_t* out_start;
  int32_t* out_position;
  int32_t* out_request;
  int64_t* out_slot;
  bool vector;      // the per-token outputs take 16-byte stores
  int32_t* status;
};

// What a token needs to know of its request.
struct PlanRequest {
  int request;
  int first;      // the request's first token in the step
  int len;        // tokens held before the step
  int held;       // blocks held before the step
  int fresh;      // index into free_blocks of the request's first new block
};

// Sums that stop at kPlanMost, which no request fits behind: 32 bits do for
// any lengths, at half the instructions of exact sums in 64.
__device__ __forceinline__ uint32_t plan_add(uint32_t x, uint32_t y) { return min(x + y, kPlanMost); }

// Sums of x and y over the threads before this one; x_all and y_all get the
// sums over all threads.
__device__ __forceinline__ void block_exclusive2(uint32_t& x, uint32_t& y, uint32_t (*scratch)[2], uint32_t& x_all,
                                                 uint32_t& y_all) {
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t xo = __shfl_up_sync(~0u, x, d), yo = __shfl_up_sync(~0u, y, d);
    if (lane >= d) x = plan_add(x, xo), y = plan_add(y, yo);
  }
  __syncthreads();
  if (lane == 31) scratch[warp][0] = x, scratch[warp][1] = y;
  x = __shfl_up_sync(~0u, x, 1), y = __shfl_up_sync(~0u, y, 1);
  if (lane == 0) x = y = 0;
  __syncthreads();
  x_all = y_all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) x = plan_add(x, x_all), y = plan_add(y, y_all);
    x_all = plan_add(x_all, scratch[w][0]), y_all = plan_add(y_all, scratch[w][1]);
  }
}

template <int kPlanTokensPerThread>
__global__ void __launch_bounds__(kThreads) block_plan_kernel(const PlanArgs a) {
  constexpr int kPlanTokens = kThreads * kPlanTokensPerThread;
  __shared__ PlanRequest req[kPlanTokens];   // at the local index of the request's first token here
  __shared__ int16_t mark[kPlanTokens];      // that index, or -1
  __shared__ uint32_t scratch[kWarps][2];
  __shared__ int warp_last[kWarps];
  allow_dependent_launch();
  grid_dependency_wait();
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = int64_t(blockIdx.x) * kPlanTokens, t1 = t0 + kPlanTokens;
  const int64_t head = *a.free_head;
  const uint32_t avail = head >= 0 && head <= a.free_count ? uint32_t(a.free_count - head) : 0;
  const uint32_t round = (1u << a.shift) - 1;
  int flags = head >= 0 && head <= a.free_count ? 0 : kRowBadLength;
#pragma unroll
  for (int i = 0; i < kPlanTokensPerThread; ++i) mark[i * kThreads + tid] = -1;

  // Prefix sums over the requests.  Sums wanted so far decide who is served;
  // both kinds grow with b, so the served requests that add anything are the
  // first ones.
  uint32_t tokens = 0, blocks = 0;               // wanted by the requests before this chunk
  uint32_t served_tokens = 0, served_blocks = 0; // of the served ones before this chunk
  int next_len = 0, next_add = 0, next_held = 0; // of the next chunk, loaded a chunk early
  if (tid < a.batch) next_len = a.lens[tid], next_add = a.add[tid], next_held = a.held[tid];
  for (int base = 0; base < a.batch; base += kThreads) {
    const int b = base + tid, len = next_len, add = next_add, held = next_held;
    if (b + kThreads < a.batch)
      next_len = a.lens[b + kThreads], next_add = a.add[b + kThreads], next_held = a.held[b + kThreads];
    uint32_t want = 0, need = 0;
    if (b < a.batch) {
      // lengths >= 0 whose sum passes 2^31 - 1 are negative as int32
      const uint32_t after = uint32_t(len) + uint32_t(add), blocks_after = (after + round) >> a.shift;
      const bool valid = len >= 0 && add >= 0 && int(after) >= 0 && held <= a.stride && int(blocks_after) <= a.stride &&
                         int((uint32_t(len) + round) >> a.shift) <= held;
      if (!valid) flags |= kRowBadLength;
      want = valid ? add : 0;
      need = want && int(blocks_after) > held ? blocks_after - held : 0;
    }
    uint32_t chunk_tokens, chunk_blocks, before_t = want, before_b = need;
    block_exclusive2(before_t, before_b, scratch, chunk_tokens, chunk_blocks);
    before_t = plan_add(before_t, tokens), before_b = plan_add(before_b, blocks);
    tokens = plan_add(tokens, chunk_tokens);
    blocks = plan_add(blocks, chunk_blocks);
    const bool fits = before_t + want <= uint32_t(a.max_tokens) && before_b + need <= avail;
    const bool served = want > 0 && fits;
    if (want > 0 && !fits) flags |= kRowNoCapacity;
    uint32_t start = before_t;
    if (tokens <= uint32_t(a.max_tokens) && blocks <= avail) {           // all of them so far
      served_tokens = tokens, served_blocks = blocks;
    } else {
      uint32_t got_tokens, got_blocks, t_served = served ? want : 0, b_served = served ? need : 0;
      block_exclusive2(t_served, b_served, scratch, got_tokens, got_blocks);
      start = served_tokens + t_served;
      served_tokens += got_tokens;
      served_blocks += got_blocks;
    }
    if (b < a.batch) {
      if ((base / kThreads) % int(gridDim.x) == int(blockIdx.x)) {
        a.out_lens[b] = served ? len + add : len;
        a.out_held[b] = served ? held + int(need) : held;
        a.out_start[b] = int(start);
      }
      if (served && start < t1 && start + want > t0) {
        const int at = start > t0 ? int(start - t0) : 0;
        mark[at] = int16_t(at);
        req[at] = {b, int(start), len, held, int(head + before_b)};
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.out_start[a.batch] = int(served_tokens);
    *a.out_head = int(head + served_blocks);
  }
  __syncthreads();

  // The running maximum of the marks is each token's request.
  int owner[kPlanTokensPerThread], run = -1;
#pragma unroll
  for (int i = 0; i < kPlanTokensPerThread; ++i) {
    run = max(run, int(mark[tid * kPlanTokensPerThread + i]));
    owner[i] = run;
  }
  int before = run;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before = max(before, o);
  }
  if (lane == 31) warp_last[warp] = before;
  before = __shfl_up_sync(~0u, before, 1);
  if (lane == 0) before = -1;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = max(before, warp_last[w]);

  int position[kPlanTokensPerThread], request[kPlanTokensPerThread];
  int64_t slot[kPlanTokensPerThread];
  const int64_t first = t0 + tid * kPlanTokensPerThread;
#pragma unroll
  for (int i = 0; i < kPlanTokensPerThread; ++i) {
    const int64_t t = first + i;
    position[i] = request[i] = -1;
    slot[i] = -1;
    if (t < served_tokens) {
      const PlanRequest& r = req[max(owner[i], before)];
      position[i] = r.len + int(t - r.first);
      request[i] = r.request;
      const int block = position[i] >> a.shift;
      const int64_t entry = int64_t(request[i]) * a.stride + block;
      const int id = block < r.held ? a.table[entry] : a.free_blocks[r.fresh + block - r.held];
      if (id >= 0 && id < a.num_blocks) slot[i] = (int64_t(id) << a.shift) + (position[i] & int(round));
      else flags |= kRowBadBlock;
      if (block >= r.held && (position[i] & int(round)) == 0) a.table[entry] = id;
    }
  }
  if (a.vector && first + kPlanTokensPerThread <= a.max_tokens) {
#pragma unroll
    for (int i = 0; i < kPlanTokensPerThread; i += 4) {
      *reinterpret_cast<int4*>(a.out_position + first + i) = make_int4(position[i], position[i + 1], position[i + 2], position[i + 3]);
      *reinterpret_cast<int4*>(a.out_request + first + i) = make_int4(request[i], request[i + 1], request[i + 2], request[i + 3]);
      reinterpret_cast<longlong2*>(a.out_slot + first + i)[0] = make_longlong2(slot[i], slot[i + 1]);
      reinterpret_cast<longlong2*>(a.out_slot + first + i)[1] = make_longlong2(slot[i + 2], slot[i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPlanTokensPerThread; ++i) {
      if (first + i >= a.max_tokens) break;
      a.out_position[first + i] = position[i];
      a.out_request[first + i] = request[i];
      a.out_slot[first + i] = slot[i];
    }
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

}  // namespace smp

extern "C" smp_status smp_block_plan(const int32_t* lens, const int32_t* add, const int32_t* held, int32_t batch,
                                     const int32_t* free_blocks, int32_t free_count, const int32_t* free_head,
                                     int32_t* block_table, int32_t table_stride, int32_t block_size,
                                     int32_t num_blocks, int32_t max_tokens, int32_t* out_lens, int32_t* out_held,
                                     int32_t* out_free_head, int32_t* out_start, int32_t* out_position,
                                     int32_t* out_request, int64_t* out_slot, int32_t* status, void* stream) {
  using namespace smp;
  if (batch < 0 || batch > (1 << 24) || free_count < 0 || table_stride < 0 || num_blocks <= 0 || max_tokens < 0)
    return SMP_ERR_INVALID_ARG;
  if (uint32_t(max_tokens) >= kPlanMost || uint32_t(free_count) >= kPlanMost) return SMP_ERR_INVALID_ARG;
  if (block_size < 16 || block_size > 256 || (block_size & (block_size - 1))) return SMP_ERR_INVALID_ARG;
  if (!free_head || !out_free_head || !out_start) return SMP_ERR_INVALID_ARG;
  if (batch > 0 && (!lens || !add || !held || !out_lens || !out_held || (table_stride > 0 && !block_table)))
    return SMP_ERR_INVALID_ARG;
  if (free_count > 0 && !free_blocks) return SMP_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!out_position || !out_request || !out_slot)) return SMP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(lens), static_cast<const void*>(add), static_cast<const void*>(held),
                        static_cast<const void*>(free_blocks), static_cast<const void*>(free_head),
                        static_cast<const void*>(block_table), static_cast<const void*>(out_lens),
                        static_cast<const void*>(out_held), static_cast<const void*>(out_free_head),
                        static_cast<const void*>(out_start), static_cast<const void*>(out_position),
                        static_cast<const void*>(out_request), static_cast<const void*>(status)})
    if (misaligned(p, 4)) return SMP_ERR_INVALID_ARG;
  if (misaligned(out_slot, 8)) return SMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    const smp_status rc = clear_status(status, st);
    if (rc != SMP_OK) return rc;
  }
  PlanArgs a{};
  a.lens = lens, a.add = add, a.held = held, a.batch = batch;
  a.free_blocks = free_blocks, a.free_count = free_count, a.free_head = free_head;
  a.table = block_table, a.stride = table_stride, a.num_blocks = num_blocks;
  for (a.shift = 0; (1 << a.shift) < block_size;) ++a.shift;
  a.max_tokens = max_tokens;
  a.out_lens = out_lens, a.out_held = out_held, a.out_head = out_free_head, a.out_start = out_start;
  a.out_position = out_position, a.out_request = out_request, a.out_slot = out_slot;
  a.vector = !misaligned(out_position, 16) && !misaligned(out_request, 16) && !misaligned(out_slot, 16);
  a.status = status;
  LaunchShape ls;
  ls.pdl = true;
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  // eight tokens per thread once four fill the GPU twice: half the repeated sums (a million tokens: 10.9 us, 12.2
  // with four; 160 tokens take 3.5 us with four)
  const bool many = max_tokens > device_sms(dev) * 2 * 4 * kThreads;
  const int per_cta = (many ? 8 : 4) * kThreads;
  const int64_t ctas = (int64_t(max_tokens) + per_cta - 1) / per_cta;
  const cudaError_t err =
      launch_cluster(many ? reinterpret_cast<const void*>(&block_plan_kernel<8>) : reinterpret_cast<const void*>(&block_plan_kernel<4>),
                     dim3(unsigned(ctas > 0 ? ctas : 1)), dim3(kThreads), ls, st, &a);
  if (err != cudaSuccess) return fail_cuda(err);
  return SMP_OK;
}
