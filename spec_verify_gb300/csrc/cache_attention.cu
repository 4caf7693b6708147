// Causal attention over the paged 8-bit cache: checks, workspace and launch
// (the kernels are in cache_attention.cuh).
#include "cache_attention.cuh"

#include "attention_rows.h"
#include "smp.h"

namespace smp {

static bool attention_sizes_ok(int32_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t batch) {
  return tokens >= 0 && q_heads > 0 && q_heads <= 65535 && kv_heads > 0 && q_heads % kv_heads == 0 && head_dim >= 16 &&
         head_dim <= SMP_MAX_HEAD_DIM && head_dim % 16 == 0 && batch >= 0 && batch <= (1 << 20);
}

}  // namespace smp

extern "C" size_t smp_cache_attention_workspace_bytes(int32_t tokens, int32_t q_heads, int32_t kv_heads,
                                                      int32_t head_dim, int32_t batch) {
  if (!smp::attention_sizes_ok(tokens, q_heads, kv_heads, head_dim, batch)) return 0;
  const int dev = smp::current_device();
  const size_t ctas = size_t(dev < 0 ? 160 : smp::device_sms(dev)) * smp::kAttnMaxCtas;
  // per main CTA: one join record and two parts, each the most rows of a unit with their sums and (m, l)
  const size_t padded = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  const size_t rows = padded == 256 ? 32 : 40;
  return ctas * (sizeof(smp::AttnJoin) + 2 * rows * (padded + 2) * 4);
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
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  AttnArgs a{};
  a.k = static_cast<const uint8_t*>(cache->k), a.v = static_cast<const uint8_t*>(cache->v);
  a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  a.num_blocks = cache->num_blocks, a.kv_heads = cache->kv_heads, a.dim = cache->head_dim;
  for (a.shift = 0; (1 << a.shift) < cache->block_size;) ++a.shift;
  a.q = q, a.q_stride = q_stride, a.tokens = tokens, a.q_heads = q_heads, a.group = q_heads / cache->kv_heads;
  a.start = start, a.lens = lens, a.batch = batch, a.table = block_table, a.stride = table_stride;
  a.scale = scale * 1.4426950408889634f, a.window = window;
  a.out = out, a.out_stride = out_stride, a.lse = out_lse, a.status = status;
  a.joins = static_cast<AttnJoin*>(workspace);
  a.partial = reinterpret_cast<float*>(a.joins + device_sms(dev) * kAttnMaxCtas);
  a.q_vector = !misaligned(q, 16) && q_stride * int64_t(elem) % 16 == 0;
  a.out_vector = !misaligned(out, 4 * elem) && out_stride % 4 == 0;
  const int64_t rows = attention_rows(tokens, batch, a.group);
  const bool e4m3 = cache->type == SMP_CACHE_E4M3, split = dtype == SMP_F32;
  const cudaError_t err = e4m3 ? split ? attn_launch<SMP_CACHE_E4M3, true>(a, rows, dev, st)
                                       : attn_launch<SMP_CACHE_E4M3, false>(a, rows, dev, st)
                               : split ? attn_launch<SMP_CACHE_I8, true>(a, rows, dev, st)
                                       : attn_launch<SMP_CACHE_I8, false>(a, rows, dev, st);
  return err == cudaSuccess ? SMP_OK : fail_cuda(err);
}
