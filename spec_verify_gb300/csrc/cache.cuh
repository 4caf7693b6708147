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
