// What the kernels of the cached speculative step share: elements of eight at
// a time, the 8-bit codes, and warp reductions.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "smp_cache.h"

namespace smp {

constexpr int kRowBadLength = 16;
constexpr int kRowNoCapacity = 32;
constexpr int kRowBadBlock = 64;

template <int kType>
constexpr float kTopCode = kType == SMP_CACHE_E4M3 ? 448.0f : 127.0f;

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two binary32 numbers rounded to bf16 (nearest, ties to even), `a` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  return w;
}

// Eight consecutive elements as binary32, by 16-byte loads (T* 16-byte aligned).
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  x[0] = bf16_low(w.x), x[1] = bf16_high(w.x), x[2] = bf16_low(w.y), x[3] = bf16_high(w.y);
  x[4] = bf16_low(w.z), x[5] = bf16_high(w.z), x[6] = bf16_low(w.w), x[7] = bf16_high(w.w);
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Eight consecutive elements as loaded.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  static constexpr int kInFlight = 8;   // of them per lane: 128 bytes
  uint4 v;
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_any(const uint16_t* p) {   // any address
    v = make_uint4(p[0] | uint32_t(p[1]) << 16, p[2] | uint32_t(p[3]) << 16, p[4] | uint32_t(p[5]) << 16,
                   p[6] | uint32_t(p[7]) << 16);
  }
  // the largest |x| as binary32 bits, above those of infinity for a NaN
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = bf16_low(v.x), x[1] = bf16_high(v.x), x[2] = bf16_low(v.y), x[3] = bf16_high(v.y);
    x[4] = bf16_low(v.z), x[5] = bf16_high(v.z), x[6] = bf16_low(v.w), x[7] = bf16_high(v.w);
  }
};
template <>
struct Eight<float> {
  static constexpr int kInFlight = 4;
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void load_any(const float* p) {
    a = make_float4(p[0], p[1], p[2], p[3]), b = make_float4(p[4], p[5], p[6], p[7]);
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = uint16_t(pack_bf16(x, 0.0f)); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// Host checks shared by the calls that take a cache.
inline smp_status check_cache(const smp_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return SMP_ERR_INVALID_ARG;
  if (c->type != SMP_CACHE_E4M3 && c->type != SMP_CACHE_I8) return SMP_ERR_DTYPE;
  if (c->num_blocks <= 0 || c->kv_heads <= 0 || c->kv_heads > 65535) return SMP_ERR_INVALID_ARG;
  if (c->block_size < 16 || c->block_size > 256 || (c->block_size & (c->block_size - 1))) return SMP_ERR_INVALID_ARG;
  if (c->head_dim < 16 || c->head_dim > SMP_MAX_HEAD_DIM || c->head_dim % 16) return SMP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) % 16) return SMP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) % 4)
    return SMP_ERR_INVALID_ARG;
  return SMP_OK;
}

inline bool misaligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace smp
