// The norm of every query and key head and the position rotation, in one pass.
//
// Mathematics: y_i = x_i w_i / sqrt(mean x^2 + eps); a rotated pair (a, b)
// becomes (a cos - b sin, b cos + a sin).  A head is held in the registers of
// one group of lanes from its only read to its only write: the sum of squares
// is a butterfly over the group, and a pair's other half, when it lies in
// another lane, comes by shuffle.
//
// Bound: HBM, one read and one write of every element (the table row, 4 bytes
// per rotated element, is shared by a token's heads).  Eight elements per
// lane keep loads at 16 bytes, so a group has head_dim / 8 lanes rounded up
// to a power of two.
#include <cuda_runtime.h>

#include "cache.cuh"
#include "launch.h"
#include "smp.h"

namespace smp {

struct NormRopeArgs {
  const void* x[2];          // q, k
  void* out[2];
  const float* weight[2];
  int64_t stride[2], out_stride[2];
  int heads[2];
  int chunks[2];             // head chunks per token
  int tokens, dim, rotary, table_rows;
  bool interleaved;
  float eps;
  const float* table;
  const int32_t* positions;
  int32_t* status;
};

// Vector form: kLanes lanes per head, each with 8 elements; kHeads heads of one
// token per group, all loaded before the first is used.  CTAs of four warps
// let an SM start new loads in smaller turns: 16 K tokens of 40 heads of 128,
// bf16, in 60 us (5.7 TB/s, 85 % of a plain copy), 62 with eight warps, 72
// with two.
constexpr int kRopeThreads = 128;

template <typename T, int kLanes, int kHeads>
__global__ void __launch_bounds__(kRopeThreads, 6) norm_rope_kernel(const NormRopeArgs a) {
  allow_dependent_launch();
  grid_dependency_wait();
  const int per_token = a.chunks[0] + a.chunks[1];
  const uint32_t item = blockIdx.x * uint32_t(kRopeThreads / kLanes) + threadIdx.x / kLanes;
  const int l = int(threadIdx.x) % kLanes;
  const int token = int(item / uint32_t(per_token));
  if (token >= a.tokens) return;      // whole groups leave together
  const unsigned group = kLanes == 32 ? ~0u : ((1u << kLanes) - 1) << ((threadIdx.x & 31) / kLanes * kLanes);
  int chunk = int(item - uint32_t(token) * uint32_t(per_token));
  const int which = chunk >= a.chunks[0];
  if (which) chunk -= a.chunks[0];
  const int position = a.positions[token];
  if (position < 0) return;
  const bool live = l * 8 < a.dim;
  const int h0 = chunk * kHeads, heads = min(kHeads, a.heads[which] - h0);
  const T* x = static_cast<const T*>(a.x[which]) + token * a.stride[which] + int64_t(h0) * a.dim + l * 8;
  T* out = static_cast<T*>(a.out[which]) + token * a.out_stride[which] + int64_t(h0) * a.dim + l * 8;
  Eight<T> raw[kHeads];                // as loaded: all heads are in flight before the first is used
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    raw[h].clear();
    if (live && h < heads) raw[h].load(x + h * a.dim);
  }
  float w[8], c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.0f, c[i] = 1.0f, s[i] = 0.0f;
  if (a.weight[which] && live) load8(a.weight[which] + l * 8, w);
  // Per element: y' = y c + partner s, with the sign of its side in s.
  const int half = a.rotary / 2;
  int partner = l;
  bool bad = position >= a.table_rows && a.rotary > 0;
  if (!bad && l * 8 < a.rotary) {
    const float* row = a.table + int64_t(position) * a.rotary;
    if (a.interleaved) {               // half is a multiple of 4: a lane rotates or not
      const float4 cs = reinterpret_cast<const float4*>(row)[l], sn = reinterpret_cast<const float4*>(row + half)[l];
      const float c4[4] = {cs.x, cs.y, cs.z, cs.w}, s4[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = c4[i / 2];
        s[i] = i % 2 ? s4[i / 2] : -s4[i / 2];
      }
    } else {                           // half is a multiple of 8: a lane is on one side
      const bool upper = l * 8 >= half;
      const int j = l * 8 - (upper ? half : 0);
      partner = upper ? l - half / 8 : l + half / 8;
      load8(row + j, c);
      load8(row + half + j, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = upper ? s[i] : -s[i];
    }
  }
  const float per_element = 1.0f / float(a.dim);
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float y[8], z[8], sum = 0.0f;
    raw[h].get(y);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(group, sum, o, kLanes);
    const float r = bad ? __int_as_float(0x7FC00000) : rsqrtf(fmaf(sum, per_element, a.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * r * w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = a.interleaved ? y[i ^ 1] : __shfl_sync(group, y[i], partner, kLanes);
      z[i] = l * 8 < a.rotary ? fmaf(y[i], c[i], other * s[i]) : y[i];
    }
    if (live && h < heads) store8(out + h * a.dim, z);
  }
  if (bad && l == 0 && a.status) atomicOr(a.status, kRowBadLength);
}

// General form, for sizes, strides or addresses that 16-byte accesses do not
// fit: one warp per head, element i in lane i % 32, pairs exchanged through
// shared memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const NormRopeArgs a) {
  __shared__ float buf[kWarps][SMP_MAX_HEAD_DIM];
  allow_dependent_launch();
  grid_dependency_wait();
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int64_t item = int64_t(blockIdx.x) * kWarps + warp;
  const int per_token = a.heads[0] + a.heads[1];
  const int token = int(item / per_token);
  if (token >= a.tokens) return;
  int h = int(item - int64_t(token) * per_token);
  const int which = h >= a.heads[0];
  if (which) h -= a.heads[0];
  const int position = a.positions[token];
  if (position < 0) return;
  const T* x = static_cast<const T*>(a.x[which]) + token * a.stride[which] + int64_t(h) * a.dim;
  T* out = static_cast<T*>(a.out[which]) + token * a.out_stride[which] + int64_t(h) * a.dim;
  float* y = buf[warp];
  float sum = 0.0f;
  for (int i = lane; i < a.dim; i += 32) {
    y[i] = load1(x + i);
    sum = fmaf(y[i], y[i], sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  const bool bad = position >= a.table_rows && a.rotary > 0;
  const float r = bad ? __int_as_float(0x7FC00000) : rsqrtf(sum / float(a.dim) + a.eps);
  for (int i = lane; i < a.dim; i += 32) y[i] = y[i] * r * (a.weight[which] ? a.weight[which][i] : 1.0f);
  __syncwarp();
  const int half = a.rotary / 2;
  const float* row = a.table + int64_t(position) * a.rotary;
  for (int i = lane; i < a.dim; i += 32) {
    float z = y[i];
    if (!bad && i < a.rotary) {
      const int j = a.interleaved ? i / 2 : (i < half ? i : i - half);
      const bool upper = a.interleaved ? i % 2 : i >= half;
      const float other = y[a.interleaved ? i ^ 1 : (upper ? i - half : i + half)];
      z = fmaf(z, row[j], upper ? other * row[half + j] : -(other * row[half + j]));
    }
    store1(out + i, z);
  }
  if (bad && lane == 0 && a.status) atomicOr(a.status, kRowBadLength);
}

template <typename T, int kLanes, int kHeads>
static cudaError_t launch_vector(NormRopeArgs a, cudaStream_t st) {
  LaunchShape ls;
  ls.pdl = true;
  for (int w = 0; w < 2; ++w) a.chunks[w] = (a.heads[w] + kHeads - 1) / kHeads;
  const int64_t items = int64_t(a.tokens) * (a.chunks[0] + a.chunks[1]);
  const int64_t grid = (items * kLanes + kRopeThreads - 1) / kRopeThreads;
  if (items > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_cluster(reinterpret_cast<const void*>(&norm_rope_kernel<T, kLanes, kHeads>), dim3(unsigned(grid)),
                        dim3(kRopeThreads), ls, st, &a);
}

template <typename T, int kHeads>
static cudaError_t launch_lanes(const NormRopeArgs& a, cudaStream_t st) {
  if (a.dim <= 64) return launch_vector<T, 8, kHeads>(a, st);
  if (a.dim <= 128) return launch_vector<T, 16, kHeads>(a, st);
  return launch_vector<T, 32, kHeads>(a, st);
}

template <typename T>
static smp_status launch_norm_rope(const NormRopeArgs& a, cudaStream_t st) {
  bool vector = a.dim % 8 == 0 && a.rotary % (a.interleaved ? 8 : 16) == 0 && !misaligned(a.table, 16) &&
                !misaligned(a.weight[0], 16) && !misaligned(a.weight[1], 16);
  for (int w = 0; w < 2 && vector; ++w) {
    if (a.heads[w] == 0) continue;
    vector = !misaligned(a.x[w], 16) && !misaligned(a.out[w], 16) && a.stride[w] * int64_t(sizeof(T)) % 16 == 0 &&
             a.out_stride[w] * int64_t(sizeof(T)) % 16 == 0;
  }
  cudaError_t err;
  if (vector) {
    // several heads per group share the table row and the weights and keep 128 bytes per lane in flight; one head
    // per group while that would leave SMs short of warps (40 heads of 128: 160 tokens in 3.5 us with one and 4.5 with
    // eight, 16 K tokens in 142 and 60)
    const int dev = current_device();
    if (dev < 0) return fail_cuda(cudaGetLastError());
    const int64_t warps = int64_t(a.tokens) * (a.heads[0] + a.heads[1]) * (a.dim <= 64 ? 8 : a.dim <= 128 ? 16 : 32) / 32;
    err = warps >= int64_t(device_sms(dev)) * 128 ? launch_lanes<T, Eight<T>::kInFlight>(a, st) : launch_lanes<T, 1>(a, st);
  } else {
    LaunchShape ls;
    ls.pdl = true;
    NormRopeArgs b = a;
    const int64_t grid = (int64_t(a.tokens) * (a.heads[0] + a.heads[1]) + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return SMP_ERR_INVALID_ARG;
    err = launch_cluster(reinterpret_cast<const void*>(&norm_rope_any_kernel<T>), dim3(unsigned(grid)),
                         dim3(kThreads), ls, st, &b);
  }
  return err == cudaSuccess ? SMP_OK : err == cudaErrorInvalidConfiguration ? SMP_ERR_INVALID_ARG : fail_cuda(err);
}

}  // namespace smp

extern "C" smp_status smp_qk_norm_rope(const void* q, const void* k, int32_t tokens, int32_t q_heads,
                                       int32_t k_heads, int32_t head_dim, int64_t q_stride, int64_t k_stride,
                                       smp_dtype dtype, const float* q_weight, const float* k_weight, float eps,
                                       const float* table, int32_t table_rows, int32_t rotary_dim,
                                       int32_t interleaved, const int32_t* positions, void* out_q, void* out_k,
                                       int64_t out_q_stride, int64_t out_k_stride, int32_t* status, void* stream) {
  using namespace smp;
  if (dtype != SMP_F32 && dtype != SMP_BF16) return SMP_ERR_DTYPE;
  if (tokens < 0 || q_heads <= 0 || q_heads > 65535 || k_heads < 0 || k_heads > 65535) return SMP_ERR_INVALID_ARG;
  if (head_dim <= 0 || head_dim > SMP_MAX_HEAD_DIM || rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 2)
    return SMP_ERR_INVALID_ARG;
  if (table_rows < 0 || (rotary_dim > 0 && tokens > 0 && !table) || !(eps >= 0.0f)) return SMP_ERR_INVALID_ARG;
  if (tokens > 0 && (!q || !out_q || !positions || (k_heads > 0 && (!k || !out_k)))) return SMP_ERR_INVALID_ARG;
  const int64_t q_row = int64_t(q_heads) * head_dim, k_row = int64_t(k_heads) * head_dim;
  if (q_stride < q_row || out_q_stride < q_row || (k_heads > 0 && (k_stride < k_row || out_k_stride < k_row)))
    return SMP_ERR_INVALID_ARG;
  const size_t elem = dtype == SMP_F32 ? 4 : 2;
  if (misaligned(q, elem) || misaligned(k, elem) || misaligned(out_q, elem) || misaligned(out_k, elem) ||
      misaligned(q_weight, 4) || misaligned(k_weight, 4) || misaligned(table, 4) || misaligned(positions, 4) ||
      misaligned(status, 4))
    return SMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    const smp_status rc = clear_status(status, st);
    if (rc != SMP_OK) return rc;
  }
  if (tokens == 0) return SMP_OK;
  NormRopeArgs a{};
  a.x[0] = q, a.x[1] = k;
  a.out[0] = out_q, a.out[1] = out_k;
  a.weight[0] = q_weight, a.weight[1] = k_weight;
  a.stride[0] = q_stride, a.stride[1] = k_stride;
  a.out_stride[0] = out_q_stride, a.out_stride[1] = out_k_stride;
  a.heads[0] = q_heads, a.heads[1] = k_heads;
  a.tokens = tokens, a.dim = head_dim, a.rotary = rotary_dim, a.table_rows = table_rows;
  a.interleaved = interleaved != 0;
  a.eps = eps;
  a.table = table;
  a.positions = positions;
  a.status = status;
  return dtype == SMP_F32 ? launch_norm_rope<float>(a, st) : launch_norm_rope<uint16_t>(a, st);
}
