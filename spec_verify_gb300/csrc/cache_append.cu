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
// Runs are found from the slots themselves: a CTA looks at a span of up to 32
// consecutive tokens, one per lane, and handles the runs that begin there.
#include <cuda_runtime.h>

#include "cache.cuh"
#include "launch.h"
#include "smp.h"

namespace smp {

constexpr int kAppendThreads = 256;
constexpr int kMinScaleExp = -100;

struct AppendArgs {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  const void *new_k, *new_v;
  int64_t k_stride, v_stride;
  bool k_vector, v_vector;       // rows of k / v take 16-byte loads
  int span;                      // tokens a CTA looks at, 1 .. 32
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
  // adding 1.5 * 2^23 rounds to an integer whose low byte is the code
  const float v[4] = {a, b, c, d};
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = v[i] != v[i] ? 0.0f : fminf(fmaxf(v[i], -127.0f), 127.0f);
    q[i] = __float_as_uint(__fadd_rn(x, 12582912.0f));
  }
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
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

// One tensor's side of the call: k or v.
template <typename T>
struct AppendSide {
  uint8_t* codes;
  float* scale;
  const T* x;
  int64_t stride;
  bool vector;
};

template <typename T, int kType>
__device__ __forceinline__ void append_run(const AppendArgs& a, const AppendSide<T>& side, int head, int64_t token,
                                           int count, int64_t slot, float* scratch, int& flags) {
  const int tid = int(threadIdx.x), per_row = a.dim / 8, vectors = count * per_row;
  const int64_t block = slot >> a.shift;
  const int offset = int(slot & ((1 << a.shift) - 1));
  uint8_t* codes = side.codes + ((block * a.heads + head) << a.shift) * a.dim;
  float* scale = side.scale + block * a.heads + head;
  const float old = offset ? *scale : 0.0f;

  // vector v = tid + i * kAppendThreads is piece v % per_row of row v / per_row
  const int row0 = tid / per_row, piece0 = tid - row0 * per_row;
  const int step_row = kAppendThreads / per_row, step_piece = kAppendThreads - step_row * per_row;
  const T* x = side.x + token * side.stride + int64_t(head) * a.dim;
  float kept[kKept][8];
  float amax = 0.0f;
  bool odd = false;
  auto look = [&](const float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(y[i]);
      if (m <= 3.402823466e38f) amax = fmaxf(amax, m);
      else odd = true;
    }
  };
  int row = row0, piece = piece0;
  auto advance = [&] {
    row += step_row;
    piece += step_piece;
    if (piece >= per_row) piece -= per_row, ++row;
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    if (tid + i * kAppendThreads < vectors) load_eight(x + row * side.stride + piece * 8, side.vector, kept[i]);
    advance();
  }
  const int more_row = row, more_piece = piece;
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (tid + i * kAppendThreads < vectors) look(kept[i]);
  for (int v = tid + kKept * kAppendThreads; v < vectors; v += kAppendThreads) {
    float y[8];
    load_eight(x + row * side.stride + piece * 8, side.vector, y);
    advance();
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
  row = more_row, piece = more_piece;
  for (int v = tid + kKept * kAppendThreads; v < vectors; v += kAppendThreads) {
    float y[8];
    load_eight(x + row * side.stride + piece * 8, side.vector, y);
    advance();
    out[v] = encode8<kType>(y, s, inverse);
  }
}

// Grid: (spans of tokens, heads, k or v).
template <typename T, int kType>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a) {
  __shared__ float scratch[kAppendThreads / 32];
  allow_dependent_launch();
  grid_dependency_wait();
  const int head = int(blockIdx.y), lane = int(threadIdx.x) & 31;
  const AppendSide<T> side =
      blockIdx.z ? AppendSide<T>{a.v, a.v_scale, static_cast<const T*>(a.new_v), a.v_stride, a.v_vector}
                 : AppendSide<T>{a.k, a.k_scale, static_cast<const T*>(a.new_k), a.k_stride, a.k_vector};
  const int64_t first = int64_t(blockIdx.x) * a.span, mine = first + lane;
  const int64_t inside = (1 << a.shift) - 1;
  int flags = 0;
  // every warp looks at the whole span, a token per lane; a run goes on while
  // the slots follow one another and the block does not end
  int64_t slot = -1;
  if (lane < a.span && mine < a.tokens) slot = a.slots[mine];
  if (slot >= a.slots_end) slot = -1, flags |= kRowBadLength;
  const bool follows = slot >= 0 && mine > 0 && (slot & inside) != 0 && a.slots[mine - 1] == slot - 1;
  unsigned starts = __ballot_sync(~0u, slot >= 0 && !follows);
  while (starts) {
    const int at = __ffs(starts) - 1;
    starts &= starts - 1;
    const int64_t run = __shfl_sync(~0u, slot, at);
    const int most = int(inside + 1 - (run & inside));
    int count = 1;
    for (bool more = true; more && count < most;) {
      const int64_t i = first + at + count + lane;
      const bool on = count + lane < most && i < a.tokens && a.slots[i] == run + count + lane;
      const unsigned broken = ~__ballot_sync(~0u, on);
      more = broken == 0;
      count += more ? 32 : __ffs(broken) - 1;
    }
    append_run<T, kType>(a, side, head, first + at, count, run, scratch, flags);
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

template <typename T, int kType>
static smp_status launch_append(const AppendArgs& a, cudaStream_t st) {
  const int64_t spans = (int64_t(a.tokens) + a.span - 1) / a.span;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(spans), unsigned(a.heads), 2);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, cache_append_kernel<T, kType>, a);
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
  a.k = static_cast<uint8_t*>(cache->k), a.v = static_cast<uint8_t*>(cache->v);
  a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  a.new_k = k, a.new_v = v;
  a.k_stride = k_stride, a.v_stride = v_stride;
  a.k_vector = !misaligned(k, 16) && k_stride * int64_t(elem) % 16 == 0;
  a.v_vector = !misaligned(v, 16) && v_stride * int64_t(elem) % 16 == 0;
  a.tokens = tokens, a.heads = cache->kv_heads, a.dim = cache->head_dim;
  for (a.shift = 0; (1 << a.shift) < cache->block_size;) ++a.shift;
  a.slots_end = int64_t(cache->num_blocks) << a.shift;
  a.slots = slots;
  a.status = status;
  // spans as long as leaves every SM some 16 CTAs: a CTA without a run start only costs its launch
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  const int64_t fill = int64_t(tokens) * a.heads * 2 / (int64_t(device_sms(dev)) * 16);
  a.span = int(fill < 1 ? 1 : fill > 32 ? 32 : fill);
  const bool e4m3 = cache->type == SMP_CACHE_E4M3;
  if (dtype == SMP_F32)
    return e4m3 ? launch_append<float, SMP_CACHE_E4M3>(a, st) : launch_append<float, SMP_CACHE_I8>(a, st);
  return e4m3 ? launch_append<uint16_t, SMP_CACHE_E4M3>(a, st) : launch_append<uint16_t, SMP_CACHE_I8>(a, st);
}
