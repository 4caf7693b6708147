// Keys and values of a step's tokens into the paged 8-bit cache.
//
// Mathematics: a block and head share one scale s = 2^e, the smallest power of
// two with amax <= top * s, so x / s is exact and a code is one rounding of x.
// A block that already holds tokens keeps the larger of its scale and the one
// the new tokens need; when it grows by 2^d, the older codes are encoded again
// (e4m3: exact down to the subnormals; i8: one rounding at the new scale).
//
// Bound: HBM, two bytes read (bf16) and one written per element.  The work
// item is a run (the step's tokens inside one block) of one head, k and v: one
// CTA holds it in registers between the maximum and the encoding.
// Runs are found from the slots themselves: a CTA looks at a span of up to 32
// consecutive tokens, one per lane, and handles the runs that begin there.
#include <cuda_runtime.h>

#include "cache.cuh"
#include "launch.h"
#include "smp.h"

namespace smp {

constexpr int kAppendThreads = 256;       // 128 where the call is short of runs
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

// Four codes of x * inverse for finite x with |x * inverse| <= top, the first
// in the low byte; the product is exact, so each code is rounded once.
template <int kType>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inverse) {
  if (kType == SMP_CACHE_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inverse), "f"(a * inverse));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inverse), "f"(c * inverse));
    return uint32_t(lo) | uint32_t(hi) << 16;
  }
  // adding 1.5 * 2^23 rounds to an integer whose low byte is the code
  const float v[4] = {a, b, c, d};
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(__fmaf_rn(v[i], inverse, 12582912.0f));
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// One code of any x: infinities take the largest code, NaN e4m3's NaN or 0.
template <int kType>
__device__ __forceinline__ uint32_t encode1(float x) {
  if (kType == SMP_CACHE_E4M3) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.0f), "f"(x));
    return c & 0xFFu;
  }
  return x != x ? 0u : uint32_t(__float2int_rn(fminf(fmaxf(x, -127.0f), 127.0f))) & 0xFFu;
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

// Eight codes of x / s for finite x and a power of two s.
template <int kType>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inverse) {
  return make_uint2(encode4<kType>(x[0], x[1], x[2], x[3], inverse), encode4<kType>(x[4], x[5], x[6], x[7], inverse));
}

// The rare forms are out of line and rolled: inlined, they made the kernel
// miss its instruction cache (16 K tokens of prompts: 56 us, 27 out of line).

// Eight codes of any x and any s.
template <int kType>
__device__ __noinline__ uint2 encode8_any(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                          float s) {
  uint64_t out = 0;
  for (int i = 0; i < 8; ++i) {
    out |= uint64_t(encode1<kType>(quotient(x0, s))) << (8 * i);
    x0 = x1, x1 = x2, x2 = x3, x3 = x4, x4 = x5, x5 = x6, x6 = x7;
  }
  return make_uint2(uint32_t(out), uint32_t(out >> 32));
}

// The `count` codes before a run, encoded again after the scale grew.
template <int kThreads, int kType>
__device__ __noinline__ void encode_again(uint8_t* codes, int count, float old, float s) {
  const float ratio = __fdiv_rn(old, s);
  for (int i = int(threadIdx.x); i < count / 4; i += kThreads) {
    uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
    const uint32_t c = *p;
    uint32_t out = 0;
    for (int j = 0; j < 32; j += 8) out |= encode1<kType>(product(decode1<kType>(uint8_t(c >> j)), ratio)) << j;
    *p = out;
  }
}

// The largest finite |x| of eight.
template <typename T>
__device__ __noinline__ float finite_top(Eight<T> e) {
  float y[8], top = 0.0f;
  e.get(y);
  for (int i = 0; i < 8; ++i)
    if (fabsf(y[i]) <= 3.402823466e38f) top = fmaxf(top, fabsf(y[i]));
  return top;
}

// One tensor's side of the call: k or v.
template <typename T>
struct AppendSide {
  uint8_t* codes;
  float* scale;
  const T* x;
  int64_t stride;
  bool vector;
};

// A run of one head, k and v together: their loads are all in flight before
// the first is used, and one pair of barriers finds both maxima.
template <int kThreads, typename T, int kType>
__device__ __forceinline__ void append_run(const AppendArgs& a, const AppendSide<T> (&side)[2], int head,
                                           int64_t token, int count, int64_t slot, float (*scratch)[2], int& flags) {
  // vectors of eight elements that a thread keeps of each side between the two
  // sweeps of a run; longer runs are read again
  constexpr int kKept = Eight<T>::kInFlight / 2;
  const int tid = int(threadIdx.x), per_row = a.dim / 8, vectors = count * per_row;
  const int64_t block = slot >> a.shift;
  const int offset = int(slot & ((1 << a.shift) - 1));
  uint8_t* codes[2];
  float* scale[2];
  const T* x[2];
  float old[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    codes[w] = side[w].codes + ((block * a.heads + head) << a.shift) * a.dim;
    scale[w] = side[w].scale + block * a.heads + head;
    x[w] = side[w].x + token * side[w].stride + int64_t(head) * a.dim;
    old[w] = offset ? *scale[w] : 0.0f;
  }

  // vector v = tid + i * kThreads is piece v % per_row of row v / per_row
  const int row0 = tid / per_row, piece0 = tid - row0 * per_row;
  const int step_row = kThreads / per_row, step_piece = kThreads - step_row * per_row;
  Eight<T> kept[2][kKept];
  float amax[2] = {0.0f, 0.0f};
  bool odd = false;
  auto load = [&](int w, int row, int piece, Eight<T>& e) {
    const T* p = x[w] + row * side[w].stride + piece * 8;
    if (side[w].vector) e.load(p);
    else e.load_any(p);
  };
  // binary32 bits order like the magnitudes, and those at or above infinity's show what is not finite
  auto look = [&](const Eight<T>& e, float& top) {
    const uint32_t bits = e.top();
    if (bits >= 0x7F800000u) {
      odd = true;
      top = fmaxf(top, finite_top<T>(e));
    } else {
      top = fmaxf(top, __uint_as_float(bits));
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
    if (tid + i * kThreads < vectors) load(0, row, piece, kept[0][i]), load(1, row, piece, kept[1][i]);
    advance();
  }
  const int more_row = row, more_piece = piece;
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (tid + i * kThreads < vectors) look(kept[0][i], amax[0]), look(kept[1][i], amax[1]);
  for (int v = tid + kKept * kThreads; v < vectors; v += kThreads) {
    Eight<T> e[2];
    load(0, row, piece, e[0]), load(1, row, piece, e[1]);
    advance();
    look(e[0], amax[0]), look(e[1], amax[1]);
  }
  if (odd) flags |= kRowNonFinite;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    amax[0] = fmaxf(amax[0], __shfl_xor_sync(~0u, amax[0], o));
    amax[1] = fmaxf(amax[1], __shfl_xor_sync(~0u, amax[1], o));
  }
  __syncthreads();                       // also orders the loads of `old` before the stores below
  if ((tid & 31) == 0) scratch[tid >> 5][0] = amax[0], scratch[tid >> 5][1] = amax[1];
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
    amax[0] = fmaxf(amax[0], scratch[w][0]), amax[1] = fmaxf(amax[1], scratch[w][1]);

#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float s = fmaxf(needed_scale<kType>(amax[w]), old[w]);
    const float inverse = (__float_as_uint(s) & 0x7FFFFFu) == 0 ? __fdiv_rn(1.0f, s) : 0.0f;
    if (tid == 0) *scale[w] = s;
    if (offset && s != old[w]) encode_again<kThreads, kType>(codes[w], offset * a.dim, old[w], s);
    uint2* out = reinterpret_cast<uint2*>(codes[w] + offset * a.dim);   // rows of a run are contiguous
    const bool plain = inverse != 0.0f && !odd;
    auto encode = [&](const Eight<T>& e) {
      float y[8];
      e.get(y);
      return plain ? encode8<kType>(y, inverse) : encode8_any<kType>(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7], s);
    };
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int v = tid + i * kThreads;
      if (v < vectors) out[v] = encode(kept[w][i]);
    }
    row = more_row, piece = more_piece;
    for (int v = tid + kKept * kThreads; v < vectors; v += kThreads) {
      Eight<T> e;
      load(w, row, piece, e);
      advance();
      out[v] = encode(e);
    }
  }
}

// Grid: (spans of tokens, heads).  Prompts of 16 K tokens, 8 heads of 128, bf16
// to i8: 26 us, 3.9 TB/s of elements and codes (the codes mostly stay in L2;
// from binary32 35 us, 4.9 TB/s),
// in seven waves of CTAs that each wait for their loads once; the prefetch of
// the span's rows takes 1 us off.  160 tokens of 32 requests: 4.0 us, the
// latency of slots, elements, maximum and stores one after the other.
template <int kThreads, typename T, int kType>
__global__ void __launch_bounds__(kThreads, kThreads == kAppendThreads ? 4 : 6) cache_append_kernel(const AppendArgs a) {
  __shared__ float scratch[kThreads / 32][2];
  allow_dependent_launch();
  const int head = int(blockIdx.y), lane = int(threadIdx.x) & 31;
  if (a.span > 1) {
    // the span's rows into L2 while the slots are looked up (a hint, which changes no memory)
    const int lines = (a.dim * int(sizeof(T)) + 127) / 128;
    const int rows = int(min(int64_t(a.span), int64_t(a.tokens) - int64_t(blockIdx.x) * a.span));
    for (int i = int(threadIdx.x); i < 2 * rows * lines; i += kThreads) {
      const int w = i >= rows * lines, r = i / lines - w * rows, l = i % lines;
      const T* x = static_cast<const T*>(w ? a.new_v : a.new_k) +
                   (int64_t(blockIdx.x) * a.span + r) * (w ? a.v_stride : a.k_stride) + int64_t(head) * a.dim;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(x) + l * 128));
    }
  }
  grid_dependency_wait();
  const AppendSide<T> side[2] = {{a.k, a.k_scale, static_cast<const T*>(a.new_k), a.k_stride, a.k_vector},
                                 {a.v, a.v_scale, static_cast<const T*>(a.new_v), a.v_stride, a.v_vector}};
  const int64_t first = int64_t(blockIdx.x) * a.span;
  const int64_t inside = (1 << a.shift) - 1;
  int flags = 0;
  // Every warp looks at 64 tokens, two per lane: bit i of `on` says that token
  // first + i goes on with the run of the one before it (the slots follow one
  // another and the block has not ended).
  int64_t slot[2];
  unsigned goes_on[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t t = first + 32 * h + lane;
    slot[h] = t < a.tokens ? a.slots[t] : -1;
    const int64_t before = t > 0 && t < a.tokens ? a.slots[t - 1] : -1;
    goes_on[h] = __ballot_sync(~0u, slot[h] > 0 && slot[h] < a.slots_end && (slot[h] & inside) != 0 && before == slot[h] - 1);
  }
  const uint64_t on = goes_on[0] | uint64_t(goes_on[1]) << 32;
  if (lane < a.span && slot[0] >= a.slots_end) flags |= kRowBadLength;
  unsigned starts = __ballot_sync(~0u, lane < a.span && slot[0] >= 0 && slot[0] < a.slots_end) & ~goes_on[0];
  while (starts) {
    const int at = __ffs(starts) - 1;
    starts &= starts - 1;
    const int64_t run = __shfl_sync(~0u, slot[0], at);
    const uint64_t after = ~(at == 63 ? 0 : on >> (at + 1));
    int count = after ? __ffsll(int64_t(after)) : 64;            // 1 + the tokens that go on
    if (at + count >= 64) {                                      // the run may leave the 64 tokens
      count = 64 - at;
      const int most = int(inside + 1 - (run & inside));
      for (bool more = true; more && count < most;) {
        const int64_t i = first + at + count + lane;
        const bool next = count + lane < most && i < a.tokens && a.slots[i] == run + count + lane;
        const unsigned broken = ~__ballot_sync(~0u, next);
        more = broken == 0;
        count += more ? 32 : __ffs(broken) - 1;
      }
    }
    append_run<kThreads, T, kType>(a, side, head, first + at, count, run, scratch, flags);
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

template <int kThreads, typename T, int kType>
static smp_status launch_append_with(const AppendArgs& a, cudaStream_t st) {
  const int64_t spans = (int64_t(a.tokens) + a.span - 1) / a.span;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(spans), unsigned(a.heads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, cache_append_kernel<kThreads, T, kType>, a);
  return err == cudaSuccess ? SMP_OK : fail_cuda(err);
}

// Where a CTA looks at one token (fewer than 16 tokens and heads per SM), runs
// are short and few: half the threads start and meet sooner (32 requests' 5
// tokens, 8 heads of 128: 4.0 us, 5.4 with 256; 16 K tokens of prompts: 28 us
// with 128, 26 with 256).
template <typename T, int kType>
static smp_status launch_append(const AppendArgs& a, cudaStream_t st) {
  return a.span == 1 ? launch_append_with<kAppendThreads / 2, T, kType>(a, st)
                     : launch_append_with<kAppendThreads, T, kType>(a, st);
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
  // spans as long as leaves every SM some 8 CTAs: a CTA without a run start only costs its launch
  const int dev = current_device();
  if (dev < 0) return fail_cuda(cudaGetLastError());
  const int64_t fill = int64_t(tokens) * a.heads / (int64_t(device_sms(dev)) * 8);
  a.span = int(fill < 1 ? 1 : fill > 32 ? 32 : fill);
  const bool e4m3 = cache->type == SMP_CACHE_E4M3;
  if (dtype == SMP_F32)
    return e4m3 ? launch_append<float, SMP_CACHE_E4M3>(a, st) : launch_append<float, SMP_CACHE_I8>(a, st);
  return e4m3 ? launch_append<uint16_t, SMP_CACHE_E4M3>(a, st) : launch_append<uint16_t, SMP_CACHE_I8>(a, st);
}
