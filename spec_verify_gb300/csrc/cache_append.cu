// Keys and values of a step's tokens into the paged 8-bit cache.
//
// Mathematics: a block and head share one scale s = 2^e, the smallest power of
// two with amax <= top * s, so x / s is exact and a code is one rounding of x.
// A block that already holds tokens keeps the larger of its scale and the one
// the new tokens need; when it grows by 2^d, the older codes are encoded again
// (e4m3: exact down to the subnormals; i8: one rounding at the new scale).
//
// Bound: HBM, two bytes read (bf16) and one written per element.  The work
// item is a run (the step's tokens inside one block) of one head, of k or of
// v: one CTA holds it in registers between the maximum and the encoding.
// Runs are found from the slots themselves: a CTA looks at kSpan consecutive
// tokens and handles the runs that begin there.
#include <cuda_runtime.h>

#include "cache.cuh"
#include "launch.h"
#include "smp.h"

namespace smp {

constexpr int kAppendThreads = 128;
constexpr int kMinScaleExp = -100;

struct AppendArgs {
  uint8_t* codes[2];
  float* scale[2];
  const void* x[2];
  int64_t stride[2];
  int tokens, heads, dim, shift;
  int64_t slots_end;             // num_blocks << shift
  const int64_t* slots;
  int32_t* status;
};

// The smallest power of two s >= 2^-100 with amax <= top * s; amax finite, >= 0.
template <int kType>
__device__ __forceinline__ float needed_scale(float amax) {
  // top = m 2^b with 1 <= m < 2: the exponent of amax less b, one more where
  // amax's significand is above m.  Subnormal amax ends at the lower limit.
  const uint32_t bits = __float_as_uint(amax), top = __float_as_uint(kTopCode<kType>);
  int e = int(bits >> 23) - int(top >> 23) + ((bits & 0x7FFFFFu) > (top & 0x7FFFFFu));
  e = max(e, kMinScaleExp);
  return __uint_as_float(uint32_t(e + 127) << 23);
}

// Codes of four numbers already divided by the scale, the first in the low byte.
template <int kType>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if (kType == SMP_CACHE_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return uint32_t(lo) | uint32_t(hi) << 16;
  }
  const float v[4] = {a, b, c, d};
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = v[i] != v[i] ? 0 : __float2int_rn(fminf(fmaxf(v[i], -127.0f), 127.0f));
    w |= uint32_t(q & 0xFF) << (8 * i);
  }
  return w;
}

template <int kType>
__device__ __forceinline__ float decode1(uint8_t c) {
  if (kType == SMP_CACHE_I8) return float(int8_t(c));
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(uint16_t(c)));
  float f;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(h2));
  return f;
}

// A binary32 result r of an operation with the rounding error `error` (exact
// value less r), moved to the neighbour with an odd last bit on the exact
// value's side unless it is exact or odd already: rounding that to the few
// bits of a code gives what rounding the exact value gives.
__device__ __forceinline__ float to_odd(float r, float error) {
  const uint32_t bits = __float_as_uint(r);
  if (error != 0.0f && error == error && !(bits & 1u) && r != 0.0f)
    return __uint_as_float((error > 0.0f) == (r > 0.0f) ? bits + 1 : bits - 1);
  return r;
}

__device__ __forceinline__ float quotient(float x, float s) {
  const float q = __fdiv_rn(x, s);
  return fabsf(q) <= 448.0f ? to_odd(q, __fmaf_rn(-q, s, x)) : q;
}

__device__ __forceinline__ float product(float x, float y) {
  const float p = __fmul_rn(x, y);
  return to_odd(p, __fmaf_rn(x, y, -p));
}

// Eight codes of x / s.  The quotient is a product with the exact inverse of a
// power of two; a block's scale that the caller set to something else divides.
template <int kType>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s, float inverse) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = inverse != 0.0f ? __fmul_rn(x[i], inverse) : quotient(x[i], s);
  return make_uint2(encode4<kType>(y[0], y[1], y[2], y[3]), encode4<kType>(y[4], y[5], y[6], y[7]));
}

template <typename T>
__device__ __forceinline__ void load_eight(const T* p, bool vector, float (&x)[8]) {
  if (vector) {
    load8(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = load1(p + i);
  }
}

// Vectors of eight elements that a thread keeps between the two sweeps of a
// run; longer runs are read again.
constexpr int kKept = 4;

template <typename T, int kType>
__device__ __forceinline__ void append_run(const AppendArgs& a, int which, int head, int token, int count,
                                           int64_t slot, bool vector, float* scratch, int& flags) {
  const int tid = int(threadIdx.x), per_row = a.dim / 8, vectors = count * per_row;
  const int64_t block = slot >> a.shift;
  const int offset = int(slot & ((1 << a.shift) - 1));
  const T* x = static_cast<const T*>(a.x[which]) + int64_t(head) * a.dim;
  const int64_t stride = a.stride[which];
  uint8_t* codes = a.codes[which] + ((block * a.heads + head) << a.shift) * a.dim;
  float* scale = a.scale[which] + block * a.heads + head;
  const float old = offset ? *scale : 0.0f;

  float kept[kKept][8];
  float amax = 0.0f;
  bool odd = false;
  auto row_of = [&](int v) { return x + (token + v / per_row) * stride + v % per_row * 8; };
  auto look = [&](const float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(y[i]);
      if (m <= 3.402823466e38f) amax = fmaxf(amax, m);
      else odd = true;
    }
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int v = tid + i * kAppendThreads;
    if (v < vectors) load_eight(row_of(v), vector, kept[i]);
  }
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (tid + i * kAppendThreads < vectors) look(kept[i]);
  for (int v = tid + kKept * kAppendThreads; v < vectors; v += kAppendThreads) {
    float y[8];
    load_eight(row_of(v), vector, y);
    look(y);
  }
  if (odd) flags |= kRowNonFinite;
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  __syncthreads();                       // also orders the load of `old` before the store below
  if ((tid & 31) == 0) scratch[tid >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, scratch[w]);

  const float s = fmaxf(needed_scale<kType>(amax), old);
  const float inverse = (__float_as_uint(s) & 0x7FFFFFu) == 0 ? __fdiv_rn(1.0f, s) : 0.0f;
  if (tid == 0) *scale = s;
  if (offset && s != old) {
    const float ratio = __fdiv_rn(old, s);
    for (int i = tid; i < offset * a.dim / 4; i += kAppendThreads) {
      uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
      const uint32_t w = *p;
      *p = encode4<kType>(product(decode1<kType>(uint8_t(w)), ratio), product(decode1<kType>(uint8_t(w >> 8)), ratio),
                          product(decode1<kType>(uint8_t(w >> 16)), ratio),
                          product(decode1<kType>(uint8_t(w >> 24)), ratio));
    }
  }
  uint2* out = reinterpret_cast<uint2*>(codes + offset * a.dim);   // rows of a run are contiguous
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int v = tid + i * kAppendThreads;
    if (v < vectors) out[v] = encode8<kType>(kept[i], s, inverse);
  }
  for (int v = tid + kKept * kAppendThreads; v < vectors; v += kAppendThreads) {
    float y[8];
    load_eight(row_of(v), vector, y);
    out[v] = encode8<kType>(y, s, inverse);
  }
}

// Grid: (spans of kSpan tokens, heads, k or v).
template <typename T, int kType, int kSpan>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a, const bool vector_k,
                                                                      const bool vector_v) {
  __shared__ float scratch[kAppendThreads / 32];
  allow_dependent_launch();
  grid_dependency_wait();
  const int which = int(blockIdx.z), head = int(blockIdx.y);
  const int64_t first = int64_t(blockIdx.x) * kSpan;
  const int last = int(first + kSpan < a.tokens ? first + kSpan : a.tokens);
  int flags = 0;
  auto usable = [&](int64_t s) { return s >= 0 && s < a.slots_end; };
  const int64_t inside = (1 << a.shift) - 1;
  for (int t = int(first); t < last; ++t) {
    const int64_t slot = a.slots[t];
    if (!usable(slot)) {
      if (slot >= 0) flags |= kRowBadLength;
      continue;
    }
    // a run goes on while the slots follow one another and the block does not end
    if (t > 0 && (slot & inside) != 0 && a.slots[t - 1] == slot - 1) continue;
    const int most = int(inside + 1 - (slot & inside));
    int count = 1;
    for (bool more = true; more && count < most;) {     // 32 slots at a time, the same in every warp
      const int i = count + (int(threadIdx.x) & 31);
      const bool follows = i < most && t + int64_t(i) < a.tokens && a.slots[t + int64_t(i)] == slot + i;
      const unsigned broken = ~__ballot_sync(~0u, follows);
      more = broken == 0;
      count += more ? 32 : __ffs(broken) - 1;
    }
    append_run<T, kType>(a, which, head, t, count, slot, which ? vector_v : vector_k, scratch, flags);
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

template <typename T, int kType>
static smp_status launch_append(const AppendArgs& a, cudaStream_t st) {
  bool vector[2];
  for (int w = 0; w < 2; ++w)
    vector[w] = !misaligned(a.x[w], 16) && a.stride[w] * int64_t(sizeof(T)) % 16 == 0;
  constexpr int kSpan = 4;
  const int64_t spans = (int64_t(a.tokens) + kSpan - 1) / kSpan;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(spans), unsigned(a.heads), 2);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, cache_append_kernel<T, kType, kSpan>, a, vector[0], vector[1]);
  return err == cudaSuccess ? SMP_OK : fail_cuda(err);
}

}  // namespace smp

extern "C" smp_status smp_cache_append(const smp_cache* cache, const void* k, const void* v, int32_t tokens,
                                       int64_t k_stride, int64_t v_stride, smp_dtype dtype, const int64_t* slots,
                                       int32_t* status, void* stream) {
  using namespace smp;
  if (dtype != SMP_F32 && dtype != SMP_BF16) return SMP_ERR_DTYPE;
  const smp_status bad = check_cache(cache);
  if (bad != SMP_OK) return bad;
  if (tokens < 0 || (tokens > 0 && (!k || !v || !slots))) return SMP_ERR_INVALID_ARG;
  const int64_t row = int64_t(cache->kv_heads) * cache->head_dim;
  if (k_stride < row || v_stride < row) return SMP_ERR_INVALID_ARG;
  const size_t elem = dtype == SMP_F32 ? 4 : 2;
  if (misaligned(k, elem) || misaligned(v, elem) || misaligned(slots, 8) || misaligned(status, 4))
    return SMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (status) {
    const smp_status rc = clear_status(status, st);
    if (rc != SMP_OK) return rc;
  }
  if (tokens == 0) return SMP_OK;
  AppendArgs a{};
  a.codes[0] = static_cast<uint8_t*>(cache->k), a.codes[1] = static_cast<uint8_t*>(cache->v);
  a.scale[0] = cache->k_scale, a.scale[1] = cache->v_scale;
  a.x[0] = k, a.x[1] = v;
  a.stride[0] = k_stride, a.stride[1] = v_stride;
  a.tokens = tokens, a.heads = cache->kv_heads, a.dim = cache->head_dim;
  for (a.shift = 0; (1 << a.shift) < cache->block_size;) ++a.shift;
  a.slots_end = int64_t(cache->num_blocks) << a.shift;
  a.slots = slots;
  a.status = status;
  const bool e4m3 = cache->type == SMP_CACHE_E4M3;
  if (dtype == SMP_F32)
    return e4m3 ? launch_append<float, SMP_CACHE_E4M3>(a, st) : launch_append<float, SMP_CACHE_I8>(a, st);
  return e4m3 ? launch_append<uint16_t, SMP_CACHE_E4M3>(a, st) : launch_append<uint16_t, SMP_CACHE_I8>(a, st);
}
