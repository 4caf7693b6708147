// Causal attention over the paged 8-bit cache: the simplest form.  One CTA per
// request and query head; each warp takes every fourth key with an online
// softmax, the warps' states are merged at the end.
#include <cuda_runtime.h>

#include <math.h>

#include "cache.cuh"
#include "launch.h"
#include "smp.h"

namespace smp {

struct AttentionArgs {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int num_blocks, kv_heads, shift, dim;
  const void* q;
  int64_t q_stride;
  int tokens, q_heads;
  const int32_t* start;
  const int32_t* lens;
  const int32_t* table;
  int stride;
  float scale;
  int window;
  void* out;
  int64_t out_stride;
  float* lse;
  int32_t* status;
};

template <int kType>
__device__ __forceinline__ float code_value(uint8_t c) {
  if (kType == SMP_CACHE_I8) return float(int8_t(c));
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(uint16_t(c)));
  float f;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(h2));
  return f;
}

constexpr int kAttnWarps = 4;
constexpr int kPerLane = SMP_MAX_HEAD_DIM / 32;

template <typename T, int kType>
__global__ void __launch_bounds__(kAttnWarps * 32) attention_simple_kernel(const AttentionArgs a) {
  __shared__ float acc_s[kAttnWarps][SMP_MAX_HEAD_DIM];
  __shared__ float m_s[kAttnWarps], l_s[kAttnWarps];
  allow_dependent_launch();
  grid_dependency_wait();
  const int b = int(blockIdx.y), h = int(blockIdx.x), warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int g = h / (a.q_heads / a.kv_heads);
  int first = a.start[b], last = a.start[b + 1], len = a.lens[b], flags = 0;
  if (first < 0 || last < first || last > a.tokens) first = last = 0, flags |= kRowBadLength;
  const int64_t room = int64_t(a.stride) << a.shift;
  if (len < 0 || len > room) len = len < 0 ? 0 : int(room), flags |= kRowBadLength;
  for (int t = first; t < last; ++t) {
    const int position = len - (last - t);
    const int begin = a.window > 0 ? max(0, position - a.window + 1) : 0;
    float q[kPerLane], acc[kPerLane], m = -INFINITY, l = 0.0f;
    const T* qp = static_cast<const T*>(a.q) + t * a.q_stride + int64_t(h) * a.dim;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      q[i] = i * 32 + lane < a.dim ? load1(qp + i * 32 + lane) : 0.0f;
      acc[i] = 0.0f;
    }
    for (int j = begin + warp; j <= position; j += kAttnWarps) {
      const int id = a.table[int64_t(b) * a.stride + (j >> a.shift)];
      if (id < 0 || id >= a.num_blocks) {
        flags |= kRowBadBlock;
        continue;
      }
      const int64_t bh = int64_t(id) * a.kv_heads + g;
      const int64_t at = ((bh << a.shift) + (j & ((1 << a.shift) - 1))) * a.dim;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (i * 32 + lane < a.dim) s = fmaf(q[i], code_value<kType>(a.k[at + i * 32 + lane]), s);
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
      s *= a.k_scale[bh] * a.scale;
      const float top = fmaxf(m, s), old = expf(m - top), w = expf(s - top);
      m = top;
      l = fmaf(l, old, w);
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (i * 32 + lane < a.dim)
          acc[i] = fmaf(acc[i], old, w * a.v_scale[bh] * code_value<kType>(a.v[at + i * 32 + lane]));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) acc_s[warp][i * 32 + lane] = acc[i];
    if (lane == 0) m_s[warp] = m, l_s[warp] = l;
    __syncthreads();
    float top = m_s[0], total = 0.0f;
    for (int w = 1; w < kAttnWarps; ++w) top = fmaxf(top, m_s[w]);
    for (int w = 0; w < kAttnWarps; ++w)
      if (l_s[w] != 0.0f) total += l_s[w] * expf(m_s[w] - top);
    for (int i = int(threadIdx.x); i < a.dim; i += kAttnWarps * 32) {
      float o = 0.0f;
      for (int w = 0; w < kAttnWarps; ++w)
        if (l_s[w] != 0.0f) o += acc_s[w][i] * expf(m_s[w] - top);
      store1(static_cast<T*>(a.out) + t * a.out_stride + int64_t(h) * a.dim + i, total == 0.0f ? 0.0f : o / total);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[int64_t(t) * a.q_heads + h] = total == 0.0f ? -INFINITY : top + logf(total);
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

static bool attention_sizes_ok(int32_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t batch) {
  return tokens >= 0 && q_heads > 0 && q_heads <= 65535 && kv_heads > 0 && q_heads % kv_heads == 0 && head_dim >= 16 &&
         head_dim <= SMP_MAX_HEAD_DIM && head_dim % 16 == 0 && batch >= 0 && batch <= (1 << 20);
}

}  // namespace smp

extern "C" size_t smp_cache_attention_workspace_bytes(int32_t tokens, int32_t q_heads, int32_t kv_heads,
                                                      int32_t head_dim, int32_t batch) {
  if (!smp::attention_sizes_ok(tokens, q_heads, kv_heads, head_dim, batch)) return 0;
  return 16;
}

extern "C" smp_status smp_cache_attention(const smp_cache* cache, const void* q, int32_t tokens, int32_t q_heads,
                                          int64_t q_stride, smp_dtype dtype, const int32_t* start,
                                          const int32_t* lens, int32_t batch, const int32_t* block_table,
                                          int32_t table_stride, float scale, int32_t window, void* out,
                                          int64_t out_stride, float* out_lse, int32_t* status, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  using namespace smp;
  if (dtype != SMP_F32 && dtype != SMP_BF16) return SMP_ERR_DTYPE;
  const smp_status bad = check_cache(cache);
  if (bad != SMP_OK) return bad;
  if (!attention_sizes_ok(tokens, q_heads, cache->kv_heads, cache->head_dim, batch)) return SMP_ERR_INVALID_ARG;
  if (table_stride < 0 || window < 0 || !isfinite(scale)) return SMP_ERR_INVALID_ARG;
  const int64_t row = int64_t(q_heads) * cache->head_dim;
  if (q_stride < row || out_stride < row) return SMP_ERR_INVALID_ARG;
  if (tokens > 0 && batch > 0 && (!q || !out || !start || !lens || (table_stride > 0 && !block_table)))
    return SMP_ERR_INVALID_ARG;
  const size_t elem = dtype == SMP_F32 ? 4 : 2;
  if (misaligned(q, elem) || misaligned(out, elem) || misaligned(start, 4) || misaligned(lens, 4) ||
      misaligned(block_table, 4) || misaligned(out_lse, 4) || misaligned(status, 4))
    return SMP_ERR_INVALID_ARG;
  const size_t need = smp_cache_attention_workspace_bytes(tokens, q_heads, cache->kv_heads, cache->head_dim, batch);
  if (tokens > 0 && batch > 0 && (!workspace || workspace_bytes < need || misaligned(workspace, 16)))
    return SMP_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    const smp_status rc = clear_status(status, st);
    if (rc != SMP_OK) return rc;
  }
  if (tokens == 0 || batch == 0) return SMP_OK;
  AttentionArgs a{};
  a.k = static_cast<const uint8_t*>(cache->k), a.v = static_cast<const uint8_t*>(cache->v);
  a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks, a.kv_heads = cache->kv_heads, a.dim = cache->head_dim;
  for (a.shift = 0; (1 << a.shift) < cache->block_size;) ++a.shift;
  a.q = q, a.q_stride = q_stride, a.tokens = tokens, a.q_heads = q_heads;
  a.start = start, a.lens = lens, a.table = block_table, a.stride = table_stride;
  a.scale = scale, a.window = window;
  a.out = out, a.out_stride = out_stride, a.lse = out_lse, a.status = status;
  LaunchShape ls;
  ls.pdl = true;
  const bool e4m3 = cache->type == SMP_CACHE_E4M3;
  const void* kernel;
  if (dtype == SMP_F32)
    kernel = e4m3 ? (const void*)&attention_simple_kernel<float, SMP_CACHE_E4M3>
                  : (const void*)&attention_simple_kernel<float, SMP_CACHE_I8>;
  else
    kernel = e4m3 ? (const void*)&attention_simple_kernel<uint16_t, SMP_CACHE_E4M3>
                  : (const void*)&attention_simple_kernel<uint16_t, SMP_CACHE_I8>;
  const cudaError_t err = launch_cluster(kernel, dim3(unsigned(q_heads), unsigned(batch)), dim3(kAttnWarps * 32), ls, st, &a);
  return err == cudaSuccess ? SMP_OK : fail_cuda(err);
}
