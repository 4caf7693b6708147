// Causal attention over the paged 8-bit cache: the kernels, included by one
// translation unit per pair of cache type and query type.
//
// Mathematics.  For the rows of one key head (its queries times the query
// heads that share it) and tiles of keys:
//   S^T = K Q^T,  P = 2^(S k f - m),  l += sum P,  O^T += V^T (P v)
// with k and v the scales of a key's block, f a row's factor (scale * log2(e)
// over the power of two that Q was scaled by) and one reference m per row,
// which moves only when a weight P v passes 2^15, the range of 16-bit floats;
// it then puts the row's largest weight at 2^8, and l and O are multiplied by
// 2^(m_old - m_new).  Small weights keep all 11 bits down to 2^-22 of the
// largest (value scales below 2^-92: kLeastScale); l is summed from binary32 P.
//
// Both products run on the tensor cores with the cache as the 16-row operand
// (tokens, then head elements) and the query rows as the 8-wide one, so one
// to eight rows waste nothing.  8-bit codes become 16-bit floats exactly in
// registers.  A query row enters as 16-bit floats scaled by a power of two to
// a largest element near 2^9: a bf16 element's 8 bits are exact down to 2^-26
// of the row's largest, smaller ones round to 2^-33 of it; binary32 queries and their weights enter as a
// sum of two 16-bit floats (22 bits).
//
// Split.  The keys of all (request, row tile, key head) units form one line of
// work that is cut into equal shares, one per resident CTA, whatever the
// lengths; a unit cut by a share's end leaves its parts (m, l, O) in the
// workspace, and a second kernel joins them in order.  Nothing waits on
// another CTA.  A CTA is two warps.  Each takes half of a tile's keys for
// S and P and half of the head for O, over all rows: every code is converted
// once, and O, the largest thing in registers, is halved, so that a warp can
// hold 40 rows.  P passes through shared memory, one barrier per tile.
// K and V stream through rings in shared memory by 16-byte asynchronous
// copies, a tile ahead.
//
// Bound: HBM (one byte per code) for up to 8 rows per key head and long
// contexts; then latency: two warps per scheduler run one tile's chain of
// products, softmax, barrier and products with little beside it (40 rows: a
// third of the issue slots and two fifths of the tensor pipe are busy; the
// warps wait on fixed latencies and on instruction fetch).  Measured on heads
// of 128 in e4m3, with requests from a quarter of the longest up: 4 requests
// of up to 128 K keys, int8, 8 rows: 127 us, 5.7 TB/s (83 % of a plain copy);
// 32 requests of up to 4 K, 4 or 8 rows: 40 us, 4.0 TB/s; the same of up to 20
// rows: 59.5 us, 2.9 TB/s; 8 requests of up to 64 K, 40 rows: 211 us, 3.2 TB/s
// and 205 TFLOP/s.  Prompts read and convert the keys again for every 40 rows:
// 37 chunks of about 443 tokens, four query heads to a key head, over contexts
// of up to 1.2 K: 1667 us, 73 TFLOP/s.
#pragma once

#include <cuda_runtime.h>

#include <math.h>

#include <type_traits>

#include "cache.cuh"
#include "launch.h"

namespace smp {

constexpr int kAttnThreads = 64;
constexpr int kAttnUnitCost = 3;        // a unit's fixed cost, in tiles
// A CTA's smallest share, in tiles, for calls that do not fill the GPU.  More parts to join against fewer tiles in a
// row: 8 requests of 300 keys take 13.3, 14.6 and 16.1 us with shares of 1, 2 and 4; one of 1 K 15.2, 13.8 and 14.7;
// of 4 K 26.1, 21.1 and 18.3; of 8 K 28.8, 28.8 and 22.7.
constexpr int kAttnMinShare = 2;
constexpr float kTopWeight = 8.0f;      // a new reference puts a row's largest weight at 2^8
constexpr float kMostWeight = 15.0f;    // and is replaced once one passes 2^15
constexpr uint32_t kWeightLimit = 0x7800u;   // that as a 16-bit float
// The smallest value scale that a reference follows: P stays below 2^107, and the sum of two million such weights
// finite.  Of smaller scales, the largest weight is as much below 2^8 (2^-100: at 2^0, with 11 bits down to 2^-14 of it).
constexpr float kLeastScale = 0x1p-92f;

// A unit that is cut: where its rows are, and how many CTAs have parts of it.
struct alignas(16) AttnJoin {
  int parts;                 // 0: none
  int first;                 // the request's first token
  int live_rows, head;
  int64_t r0;                // of the row tile, among the request's rows
};

struct AttnArgs {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int num_blocks, kv_heads, shift, dim;
  const void* q;
  int64_t q_stride;
  int tokens, q_heads, group;
  const int32_t* start;
  const int32_t* lens;
  int batch;
  const int32_t* table;
  int stride;
  float scale;              // scale * log2(e)
  int window;
  void* out;
  int64_t out_stride;
  float* lse;
  int32_t* status;
  float* partial;           // [CTA][2][rows][dim_padded + 2]
  AttnJoin* joins;          // [CTA]: the unit that begins there and is cut
  bool q_vector, out_vector;   // queries and results take 16-byte (results: 4-element) accesses
};

// A request as the kernels see it, lengths cut to what the tables hold.
struct AttnRequest {
  int first, n, len;
  bool bad;
};

__device__ __forceinline__ AttnRequest attn_request(const AttnArgs& a, int b) {
  AttnRequest r;
  r.first = a.start[b];
  const int last = a.start[b + 1];
  r.n = last - r.first;
  r.len = a.lens[b];
  r.bad = false;
  if (r.first < 0 || last < r.first || last > a.tokens) r.first = 0, r.n = 0, r.bad = true;
  const int64_t room = int64_t(a.stride) << a.shift;
  if (r.len < 0) r.len = 0, r.bad = true;
  if (r.len > room) r.len = int(room), r.bad = true;
  return r;
}

// ---------------------------------------------------------------- the line of work

// A CTA's stay in one unit: tiles [tile_lo, tile_hi) of its keys for rows r0 ..
// r0 + live_rows - 1 of the request's n * group rows of one key head.
struct AttnSegment {
  bool whole, first;          // the whole unit; from its beginning
  int64_t r0;
  int live_rows, p_first, p_last, tile_lo, tile_hi;
};

// The smallest row tile of the kernel whose largest is `most`, in eights.  The
// more sizes one kernel has, the slower each came out (20 rows of 32 requests
// of up to 4 K keys: 68 us with one to five eights in one kernel, 59 us alone).
__host__ __device__ constexpr int attn_least_eights(int most) { return most == 2 ? 1 : most == 4 ? 2 : most == 5 ? 4 : most; }

// The units (request, row tile, key head) in order, each as long as its tiles
// of kTile keys plus kAttnUnitCost, and this CTA's place in them.  Equal
// shares, whatever the lengths: share j is [j share, (j + 1) share).  The row
// tile is one size for the call, from the longest request as the device sees
// it: the fewest tiles of up to kMaxNT eights, and then the smallest that are
// as few.
template <int kThreads, int kTile, int kMaxNT>
struct AttnLine {
  static constexpr int kLineWarps = kThreads / 32;
  struct Shared {
    int64_t scan[kLineWarps];
    int64_t found[2];
  };
  int64_t at, end, share, cost, pos;   // places on the line; the unit's length and the place in it
  int nt;                              // rows of a row tile, in eights
  int b, rt, head;
  AttnRequest req;

  static __device__ __forceinline__ int tile_base(const AttnArgs& a, const AttnRequest& r) {
    return a.window > 0 ? int(max(int64_t(r.len) - r.n - a.window + 1, int64_t(0)) / kTile) : 0;
  }
  // Row tiles of a request.
  __device__ __forceinline__ int row_tiles(const AttnArgs& a, const AttnRequest& r) const {
    const int64_t rows = int64_t(r.n) * a.group;
    return rows <= 8 * nt ? rows > 0 : int((rows + 8 * nt - 1) / (8 * nt));
  }
  static __device__ __forceinline__ int64_t unit_cost(const AttnArgs& a, const AttnRequest& r) {
    return max(0, int((int64_t(r.len) + kTile - 1) / kTile) - tile_base(a, r)) + kAttnUnitCost;
  }

  // Finds the share; every thread of the CTA calls it.  False: there is none.
  __device__ __forceinline__ bool begin(const AttnArgs& a, Shared& sh, int& flags) {
    const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    // the first kThreads requests stay in registers between the passes
    AttnRequest own{0, 0, 0, false};
    if (tid < a.batch) own = attn_request(a, tid);
    int64_t most = 0;
    for (int r = tid; r < a.batch; r += kThreads) {
      const AttnRequest q = r == tid ? own : attn_request(a, r);
      if (q.bad) flags |= kRowBadLength;
      most = max(most, int64_t(q.n) * a.group);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(~0u, most, o));
    if (lane == 0) sh.scan[warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLineWarps; ++w) most = max(most, sh.scan[w]);
    __syncthreads();
    const int64_t tiles = max((most + 8 * kMaxNT - 1) / (8 * kMaxNT), int64_t(1));
    nt = max(int(((most + tiles - 1) / tiles + 7) / 8), attn_least_eights(kMaxNT));
    auto cost_at = [&](const AttnRequest& r) { return int64_t(row_tiles(a, r)) * a.kv_heads * unit_cost(a, r); };
    auto cost_of = [&](int request) { return cost_at(attn_request(a, request)); };
    const int64_t first_cost = cost_at(own);
    int64_t sum = first_cost;
    for (int r = tid + kThreads; r < a.batch; r += kThreads) sum += cost_of(r);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) sh.scan[warp] = sum;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kLineWarps; ++w) total += sh.scan[w];
    share = max(int64_t(kAttnMinShare), (total + gridDim.x - 1) / gridDim.x);
    at = share * blockIdx.x;
    end = min(total, at + share);
    if (tid == 0) a.joins[blockIdx.x].parts = 0;
    if (at >= end) return false;
    for (int64_t base = 0, chunk = 0;; chunk += kThreads) {
      const int64_t request = chunk + tid;
      const int64_t c = chunk == 0 ? first_cost : request < a.batch ? cost_of(int(request)) : 0;
      int64_t inc = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, inc, d);
        if (lane >= d) inc += o;
      }
      __syncthreads();
      if (lane == 31) sh.scan[warp] = inc;
      __syncthreads();
      int64_t before = base;
#pragma unroll
      for (int w = 0; w < kLineWarps; ++w) {
        if (w < warp) before += sh.scan[w];
        base += sh.scan[w];
      }
      if (before + inc - c <= at && at < before + inc) sh.found[0] = request, sh.found[1] = before + inc - c;
      if (base > at) break;                // the same in every thread
    }
    __syncthreads();
    b = int(sh.found[0]);
    req = attn_request(a, b);
    cost = unit_cost(a, req);
    const int64_t unit = (at - sh.found[1]) / cost;
    pos = at - sh.found[1] - unit * cost;
    rt = int(unit / a.kv_heads);
    head = int(unit - int64_t(rt) * a.kv_heads);
    return true;
  }

  __device__ __forceinline__ AttnSegment segment(const AttnArgs& a) const {
    AttnSegment s;
    const int64_t take = min(cost - pos, end - at);
    s.first = pos == 0;
    s.whole = s.first && take == cost;
    s.r0 = int64_t(rt) * 8 * nt;
    s.live_rows = int(min(int64_t(8 * nt), int64_t(req.n) * a.group - s.r0));
    s.p_first = req.len - req.n + int(s.r0 / a.group);
    s.p_last = req.len - req.n + int((s.r0 + s.live_rows - 1) / a.group);
    const int see_first = a.window > 0 ? int(max(int64_t(0), int64_t(s.p_first) - a.window + 1)) : 0;
    const int base = tile_base(a, req);
    s.tile_lo = max(base + int(max(pos - kAttnUnitCost, int64_t(0))), see_first / kTile);
    s.tile_hi = min(base + int(max(pos + take - kAttnUnitCost, int64_t(0))), s.p_last >= 0 ? s.p_last / kTile + 1 : 0);
    return s;
  }

  // The parts of the unit at hand, from this CTA on.
  __device__ __forceinline__ int parts() const { return int((at - pos + cost - 1) / share) - int(blockIdx.x) + 1; }

  // To the next unit; false at the share's end.
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    at += min(cost - pos, end - at);
    if (at >= end) return false;
    pos = 0;
    if (++head == a.kv_heads) {
      head = 0;
      if (++rt == row_tiles(a, req)) {
        rt = 0;
        do req = attn_request(a, ++b);
        while (req.n == 0);
        cost = unit_cost(a, req);
      }
    }
    return true;
  }
};

// ---------------------------------------------------------------- small pieces

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8x8 tile of 16-bit values whose row lane / 4 this warp holds in pairs, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two binary32 numbers as 16-bit floats, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

__device__ __forceinline__ void store4(uint16_t* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// What pack_f16 left out, as 16-bit floats.
__device__ __forceinline__ uint32_t rest_f16(uint32_t packed, float lo, float hi) {
  float a, b;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(a), "=f"(b) : "r"(packed));
  return pack_f16(lo - a, hi - b);
}

// Four codes to four 16-bit floats, exactly.
template <int kType>
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kType == SMP_CACHE_E4M3) {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // 0x6400 + u is the 16-bit float 1024 + u; u = code + 128
    const uint32_t u = w ^ 0x80808080u;
    lo = __byte_perm(u, 0x64646464u, 0x4140);
    hi = __byte_perm(u, 0x64646464u, 0x4342);
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0xE480E480u));   // - 1152
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0xE480E480u));
  }
}

__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Pairs of binary32 numbers in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
  return y;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t y;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t y;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// 16 bytes global to shared, or zeros where !live (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// ---------------------------------------------------------------- shapes

template <int kDP, int kNT, bool kSplit>
struct AttnShape {
  static constexpr int kMT = kDP == 256 ? 1 : 2;                 // 16-token row tiles of S per warp
  static constexpr int kTile = 2 * kMT * 16;                     // tokens per tile
  static constexpr int kChunks = kDP / 16;                       // 16-byte chunks of a row
  static constexpr int kSteps = kDP / 16;                        // products of depth 16 over the head
  static constexpr int kDT = kDP / 32;                           // 16-row tiles of a warp's half of V^T
  static constexpr int kRows = 8 * kNT;                          // rows of a unit's row tile
  static constexpr int kParts = kSplit ? 2 : 1;
  static constexpr bool kQReg = kNT * kSteps * 2 * kParts <= 16; // query fragments in registers
  static constexpr int kDepth = kDP == 64 ? 4 : 2;               // stages of each ring
  static constexpr int kWarpK = kMT * 16 * kDP;                  // bytes of a warp's keys of a tile
  static constexpr int kVStage = kTile * kDP;
  static constexpr int kQ4 = kSteps * kParts / 2;                // 16-byte pieces of 8 rows' fragments per lane
  // shared memory: keys [warp][stage], values [stage], queries, weights [2][row tile of 16 tokens][8 rows][lane]
  static constexpr int kVAt = 2 * kDepth * kWarpK;
  static constexpr int kQAt = kVAt + kDepth * kVStage;
  static constexpr int kPAt = kQAt + (kQReg ? 0 : kNT * kQ4 * 512);
  static constexpr int kPStage = 2 * kMT * kNT * kParts * 256;
  static constexpr int kSmem = kPAt + 2 * kPStage;
};
constexpr int kAttnMaxCtas = 5;

// What a kernel with row tiles of up to kMaxNT eights needs: as many CTAs per
// SM as 228 KB (1 KB reserved and about 1.5 KB static per CTA) hold, but 5 at
// most, or 4 above two eights: the registers of five do not hold three (heads of
// 64, 32 requests of up to 8 K keys: 76 us with five, 67 us with four).
template <int kDP, int kMaxNT, bool kSplit>
struct AttnKernel {
  static constexpr int kSmem = AttnShape<kDP, kMaxNT, kSplit>::kSmem;
  static constexpr int kFit = 228 * 1024 / (kSmem + 2560);
  static constexpr int kMost = kMaxNT > 2 ? kAttnMaxCtas - 1 : kAttnMaxCtas;
  static constexpr int kCtas = kFit > kMost ? kMost : kFit;
  static constexpr int kRows = 8 * kMaxNT;
};
constexpr int kMetaStages = 8;      // tiles whose scales are kept: copies run up to three ahead of a warp one tile behind

// ---------------------------------------------------------------- main kernel

// Scales and exchanges of a CTA, beside its rings.
template <int kMT, int kRows>
struct AttnShared {
  float scales[2][kMetaStages][2][kMT];      // [warp][tile][k, v][16 tokens]
  int valid[2][kMetaStages][kMT];            // the tokens' block id is one
  float row_factor[kRows];
  float row_part[2][kRows];                  // of each warp: largest weights, sums
};

// One segment: its keys, values and queries to its result, or its part of one.
template <int kDP, int kNT, int kMaxNT, int kType, bool kSplit>
__device__ __forceinline__ void attention_segment(const AttnArgs& a, const AttnSegment& seg, const AttnRequest& req,
                                                  const int b, const int head, uint8_t* smem,
                                                  AttnShared<AttnShape<kDP, 1, kSplit>::kMT, 8 * kMaxNT>& sh, int& flags) {
  using S = AttnShape<kDP, kNT, kSplit>;
  using T = typename std::conditional<kSplit, float, uint16_t>::type;
  auto& scales = sh.scales;
  auto& valid = sh.valid;
  auto& row_factor = sh.row_factor;
  auto& row_part = sh.row_part;
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t base = smem_addr(smem), keys = base + uint32_t(warp * S::kDepth * S::kWarpK);

  // A warp copies the keys and the values of its own tokens of a tile; one instruction covers kRowsPerCopy rows.
  // Chunk c of row r lies at chunk c ^ swizzle(r): reads of keys (8 rows, 4 chunks) and of values (rows two apart)
  // then meet the banks evenly.
  constexpr int kRowsPerCopy = 32 / S::kChunks, kCopies = S::kMT * 16 / kRowsPerCopy, kPerMT = 16 / kRowsPerCopy;
  constexpr int kSwizzles = 8 / kRowsPerCopy;
  const int my_chunk = lane % S::kChunks, my_row = lane / S::kChunks;
  auto swizzle = [](int r) { return kDP == 64 ? (r >> 1) & 3 : (r & 6) ^ ((r & 1) << 2); };
  uint32_t lane_dst[kSwizzles];
#pragma unroll
  for (int i = 0; i < kSwizzles; ++i)
    lane_dst[i] = uint32_t(my_row * kDP + ((my_chunk ^ swizzle(i * kRowsPerCopy + my_row)) * 16));
  const int lane_src = my_row * kDP + my_chunk * 16;
  const int64_t block_bytes = (int64_t(a.kv_heads) << a.shift) * a.dim;
  const int n = req.n, len = req.len, live_rows = seg.live_rows, p_first = seg.p_first, p_last = seg.p_last,
            tile_lo = seg.tile_lo, iters = seg.tile_hi - seg.tile_lo;
  const int64_t r0 = seg.r0;

  // ---- the rings.  off, ok: where this warp's tokens of the tile last looked up are
  constexpr int kPer = 32 / S::kMT;                           // tiles whose block ids the lanes hold
  auto load_ids = [&](int k0) {
    const int k = k0 + lane / S::kMT, token = (tile_lo + k) * S::kTile + (warp * S::kMT + lane % S::kMT) * 16;
    int id = -1;
    // tokens that have left every row's window are not looked up: their pages may be gone
    if (k < iters && token < len && (a.window == 0 || int64_t(token) + 15 + a.window > p_first)) {
      id = a.table[int64_t(b) * a.stride + (token >> a.shift)];
      if (id < 0 || id >= a.num_blocks) id = -1, flags |= kRowBadBlock;
    }
    return id;
  };
  int ids = load_ids(0), ids_next = load_ids(kPer);
  const int64_t head_at = (int64_t(head) << a.shift) * a.dim;
  int64_t off[S::kMT];
  bool ok[S::kMT], full = false;
  // keys (and scales) of tile k, then its values; both leave one group of copies
  auto copy_tile = [&](const uint8_t* codes, uint32_t dst, int token0) {
    if (full) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        copy16(dst + uint32_t(i * kRowsPerCopy * kDP) + lane_dst[i % kSwizzles],
               codes + off[i / kPerMT] + (i % kPerMT) * kRowsPerCopy * kDP + lane_src);
    } else {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int row = i * kRowsPerCopy + my_row;
        if (my_chunk * 16 < a.dim)
          copy16(dst + uint32_t(row * kDP + ((my_chunk ^ swizzle(row)) * 16)),
                 codes + off[i / kPerMT] + (row % 16) * a.dim + my_chunk * 16, ok[i / kPerMT] && token0 + row < len);
      }
    }
  };
  auto issue_keys = [&](int k) {
    if (k < iters) {
      const int at = k % kPer * S::kMT, token0 = (tile_lo + k) * S::kTile + warp * S::kMT * 16;
      if (at == 0 && k > 0) {
        ids = ids_next;
        ids_next = load_ids(k + kPer);
      }
      full = token0 + S::kMT * 16 <= len && a.dim == kDP;
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt) {
        const int id = __shfl_sync(~0u, ids, at + mt);
        ok[mt] = id >= 0;
        full &= ok[mt];
        off[mt] = int64_t(max(id, 0)) * block_bytes + head_at + ((token0 + 16 * mt) & ((1 << a.shift) - 1)) * a.dim;
      }
      const int id = __shfl_sync(~0u, ids, at + lane % S::kMT);
      if (lane < 2 * S::kMT) {
        copy4(smem_addr(&scales[warp][k % kMetaStages][lane / S::kMT][lane % S::kMT]),
              (lane < S::kMT ? a.k_scale : a.v_scale) + int64_t(max(id, 0)) * a.kv_heads + head, id >= 0);
        if (lane < S::kMT) valid[warp][k % kMetaStages][lane] = id >= 0;
      }
      copy_tile(a.k, keys + uint32_t(k % S::kDepth * S::kWarpK), token0);
    }
    copies_commit();
  };
  auto issue_values = [&](int k) {
    if (k < iters)
      copy_tile(a.v, base + uint32_t(S::kVAt + k % S::kDepth * S::kVStage + warp * S::kWarpK),
                (tile_lo + k) * S::kTile + warp * S::kMT * 16);
    copies_commit();
  };
  for (int k = 0; k < S::kDepth - 1; ++k) {
    issue_keys(k);
    issue_values(k);
  }

  // ---- query fragments: lane (g, t) holds the 16-element chunks t + 4 h of row g of each 8 rows
  uint32_t qreg[S::kQReg ? kNT : 1][S::kQReg ? S::kSteps * S::kParts * 2 : 1];
  int see[kNT][2];                     // last visible position of columns 2t, 2t + 1
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    if (S::kQReg || nt % 2 == warp) {
      const int row = nt * 8 + g;
      const bool live = row < live_rows;
      const int64_t gr = r0 + row;
      const int64_t token = req.first + gr / a.group, qh = int64_t(head) * a.group + gr % a.group;
      const T* q = static_cast<const T*>(a.q) + (live ? token * a.q_stride + qh * a.dim : 0);
      float x[S::kSteps][4];
#pragma unroll
      for (int h = 0; h < kDP / 64; ++h) {
        const int d = (t + 4 * h) * 16;
        Eight<T> e[2];
        e[0].clear(), e[1].clear();
        if (live && d < a.dim) {
          if (a.q_vector) e[0].load(q + d), e[1].load(q + d + 8);
          else e[0].load_any(q + d), e[1].load_any(q + d + 8);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float y[8];
          e[i].get(y);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[h * 4 + i * 2 + j / 4][j % 4] = y[j];
        }
      }
      float top = 0.0f;
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[s][e]));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      // up: the power of two that takes the largest element to [2^9, 2^10); its inverse goes into the row's factor
      const int up_exp = min(max(263 - int(__float_as_uint(top) >> 23), 1), 253);
      const float up = __uint_as_float(uint32_t(up_exp) << 23);
      if (t == 0) row_factor[row] = __uint_as_float(uint32_t(254 - up_exp) << 23) * a.scale;
      uint32_t f[S::kSteps * S::kParts * 2];                 // per step: two words, with kSplit the two rests
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[s][e] *= up;
        uint32_t* const fs = f + s * S::kParts * 2;
        fs[0] = pack_f16(x[s][0], x[s][1]);
        fs[1] = pack_f16(x[s][2], x[s][3]);
        if (kSplit) {
          fs[S::kParts * 2 - 2] = rest_f16(fs[0], x[s][0], x[s][1]);
          fs[S::kParts * 2 - 1] = rest_f16(fs[1], x[s][2], x[s][3]);
        }
      }
      if (S::kQReg) {
#pragma unroll
        for (int i = 0; i < S::kSteps * S::kParts * 2; ++i) qreg[S::kQReg ? nt : 0][S::kQReg ? i : 0] = f[i];
      } else {
#pragma unroll
        for (int i = 0; i < S::kQ4; ++i)
          *reinterpret_cast<uint4*>(smem + S::kQAt + ((nt * S::kQ4 + i) * 32 + lane) * 16) =
              make_uint4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = nt * 8 + 2 * t + c;
      see[nt][c] = r < live_rows ? len - n + int((r0 + r) / a.group) : len;     // unused rows: everything, unread
    }
  }
  __syncthreads();
  const uint32_t q_at = base + uint32_t(S::kQAt + lane * 16);
  float factor[kNT][2];
  float o[kNT][S::kDT][4];
  float l[kNT][2], m[kNT][2];
  uint32_t has_ref = 0;                        // rows (2 nt + c) whose reference is set; m = 0 before
  constexpr uint32_t kAll = (1u << (2 * kNT)) - 1;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      factor[nt][c] = row_factor[nt * 8 + 2 * t + c];
      m[nt][c] = 0.0f, l[nt][c] = 0.0f;
      if (nt * 8 + 2 * t + c >= live_rows) has_ref |= 1u << (2 * nt + c);       // unused: never awaited
    }
#pragma unroll
    for (int d = 0; d < S::kDT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][d][e] = 0.0f;
  }

  for (int k = 0; k < iters; ++k) {
    const int token0 = (tile_lo + k) * S::kTile, meta = k % kMetaStages;
    copies_wait<2 * (S::kDepth - 1) - 1>();    // this warp's keys of the tile
    __syncwarp();
    issue_keys(k + S::kDepth - 1);
    const uint32_t kst = keys + uint32_t(k % S::kDepth * S::kWarpK), vst = base + uint32_t(S::kVAt + k % S::kDepth * S::kVStage);

    // ---- S^T = K Q^T for this warp's keys
    float s[S::kMT][kNT][4];
#pragma unroll
    for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.0f;
#pragma unroll
    for (int h = 0; h < kDP / 64; ++h) {
      uint4 w[S::kMT][2], q_two[kNT];
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
        for (int up = 0; up < 2; ++up)
          w[mt][up] = lds128(kst + uint32_t((mt * 16 + up * 8 + g) * kDP + (((t + 4 * h) ^ swizzle(g)) * 16)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t f[S::kMT][4];
#pragma unroll
        for (int mt = 0; mt < S::kMT; ++mt) {
          unpack4<kType>(reinterpret_cast<const uint32_t*>(&w[mt][0])[i], f[mt][0], f[mt][2]);
          unpack4<kType>(reinterpret_cast<const uint32_t*>(&w[mt][1])[i], f[mt][1], f[mt][3]);
        }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          uint32_t q[S::kParts * 2];
          if (S::kQReg) {
#pragma unroll
            for (int p = 0; p < S::kParts * 2; ++p)
              q[p] = qreg[S::kQReg ? nt : 0][S::kQReg ? (h * 4 + i) * S::kParts * 2 + p : 0];
          } else if (kSplit) {
            const uint4 x = lds128(q_at + uint32_t(nt * S::kQ4 + h * 4 + i) * 512);
            q[0] = x.x, q[1] = x.y, q[S::kParts * 2 - 2] = x.z, q[S::kParts * 2 - 1] = x.w;
          } else {
            if (i % 2 == 0) q_two[nt] = lds128(q_at + uint32_t(nt * S::kQ4 + (h * 4 + i) / 2) * 512);
            q[0] = i % 2 ? q_two[nt].z : q_two[nt].x, q[1] = i % 2 ? q_two[nt].w : q_two[nt].y;
          }
#pragma unroll
          for (int p = 0; p < S::kParts; ++p)
#pragma unroll
            for (int mt = 0; mt < S::kMT; ++mt) mma_f16(s[mt][nt], f[mt], q[2 * p], q[2 * p + 1]);
        }
      }
    }

    // ---- exponents: s = S k f - m, hidden ones -inf
    bool edge = token0 + S::kTile - 1 > p_first || (a.window > 0 && token0 <= p_last - a.window);
    float v_scale[S::kMT];
#pragma unroll
    for (int mt = 0; mt < S::kMT; ++mt) {
      float ks = scales[warp][meta][0][mt];
      v_scale[mt] = scales[warp][meta][1][mt];
      // a hidden weight is 0 times its value scale: one that is no number counts as 0, and the rows that do see its
      // tokens get NaN from their scores
      if (!(fabsf(v_scale[mt]) < INFINITY)) v_scale[mt] = 0.0f, ks = __int_as_float(0x7FC00000);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const uint64_t c = mul2(pair(ks, ks), pair(factor[nt][0], factor[nt][1]));
        const uint64_t less = pair(-m[nt][0], -m[nt][1]);
        unpair(fma2(pair(s[mt][nt][0], s[mt][nt][1]), c, less), s[mt][nt][0], s[mt][nt][1]);
        unpair(fma2(pair(s[mt][nt][2], s[mt][nt][3]), c, less), s[mt][nt][2], s[mt][nt][3]);
      }
    }
    // whether a row sees token `of` of the tile's row tile mt (of both warps'), element e
    auto visible = [&](int mt, int nt, int e) {
      const int j = token0 + mt * 16 + g + (e / 2) * 8, p = see[nt][e % 2];
      return j <= p && (a.window == 0 || j > p - a.window) && valid[mt / S::kMT][meta][mt % S::kMT];
    };
    bool mine = edge;
#pragma unroll
    for (int mt = 0; mt < S::kMT; ++mt) mine |= !valid[warp][meta][mt];
    if (mine) {
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!visible(warp * S::kMT + mt, nt, e)) s[mt][nt][e] = -INFINITY;
    }

    // ---- weights P v as 16-bit floats, transposed into the right operand of V^T P^T, for both warps
    uint32_t packed_max = 0;
    float sum[kNT][2];
    const uint32_t p_at = base + uint32_t(S::kPAt + (k & 1) * S::kPStage + lane * 8 * S::kParts);
    auto weigh = [&] {
      packed_max = 0;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        uint64_t all = pair(0.0f, 0.0f);
#pragma unroll
        for (int mt = 0; mt < S::kMT; ++mt) {
          const uint64_t vv = pair(v_scale[mt], v_scale[mt]);
          uint32_t f[S::kParts][2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint64_t p = pair(exp2_approx(s[mt][nt][half * 2]), exp2_approx(s[mt][nt][half * 2 + 1]));
            all = add2(all, p);
            float w0, w1;
            unpair(mul2(p, vv), w0, w1);
            const uint32_t hi = pack_f16(w0, w1);
            packed_max = max_f16x2(packed_max, hi);
            f[0][half] = transpose8(hi);
            if (kSplit) f[S::kParts - 1][half] = transpose8(rest_f16(hi, w0, w1));
          }
          const uint32_t at = p_at + uint32_t(((warp * S::kMT + mt) * kNT + nt) * S::kParts * 256);
          if (kSplit)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(f[0][0]), "r"(f[0][1]),
                         "r"(f[S::kParts - 1][0]), "r"(f[S::kParts - 1][1])
                         : "memory");
          else
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(f[0][0]), "r"(f[0][1]) : "memory");
        }
        unpair(all, sum[nt][0], sum[nt][1]);
      }
    };
    weigh();
    copies_wait<2 * (S::kDepth - 1) - 1>();    // this warp's values of the tile
    bool past = (packed_max & 0xFFFFu) > kWeightLimit || (packed_max >> 16) > kWeightLimit || has_ref != kAll;
#pragma unroll
    for (int mt = 0; mt < S::kMT; ++mt)        // P can pass its bound there while P v does not (0 is the scale of no block)
      past |= __float_as_uint(v_scale[mt]) - 1u < __float_as_uint(kLeastScale) - 1u;
    if (__syncthreads_or(past)) {
      // rare: the rows' largest weights over both warps' keys, and new references where they pass the limit
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float y = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < S::kMT; ++mt)
            y = fmaxf(y, fmaxf(s[mt][nt][c], s[mt][nt][c + 2]) + __log2f(fmaxf(v_scale[mt], kLeastScale)));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(~0u, y, d));
          if (g == 0) row_part[warp][nt * 8 + 2 * t + c] = y;
        }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float alpha[2] = {1.0f, 1.0f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float y = fmaxf(row_part[0][nt * 8 + 2 * t + c], row_part[1][nt * 8 + 2 * t + c]);
          const uint32_t bit = 1u << (2 * nt + c);
          if ((has_ref & bit) ? y > kMostWeight : y > -INFINITY) {
            const float up = y - kTopWeight;
            // in two steps: after blocks of the smallest scales, l has to take more than one factor of binary32 can
            const float half = has_ref & bit ? exp2_approx(-0.5f * up) : 1.0f;
            alpha[c] = half * half;
            has_ref |= bit;
            m[nt][c] += up;
            l[nt][c] = l[nt][c] * half * half;
#pragma unroll
            for (int mt = 0; mt < S::kMT; ++mt) s[mt][nt][c] -= up, s[mt][nt][c + 2] -= up;
          }
        }
#pragma unroll
        for (int d = 0; d < S::kDT; ++d) {
          o[nt][d][0] *= alpha[0], o[nt][d][1] *= alpha[1], o[nt][d][2] *= alpha[0], o[nt][d][3] *= alpha[1];
        }
      }
      weigh();
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) l[nt][0] += sum[nt][0], l[nt][1] += sum[nt][1];
    issue_values(k + S::kDepth - 1);

    // ---- O^T += V^T P^T for this warp's half of the head: lane (g, t) reads tokens 2t, 2t+1, 2t+8, 2t+9 of 16; row g
    // of row tile d is element kDP / 16 g + 2 d of the half, row g + 8 the next one
    constexpr int kWords = kDP / 64;           // 4-byte words of a lane's elements
    auto values = [&](int mt, uint32_t (&w)[4][4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1) + (i / 2) * 8;
        const uint32_t row = vst + uint32_t((mt * 16 + r) * kDP);
        if (kDP == 64) {
          w[i][0] = lds32(row + uint32_t((((warp * 2 + (g >> 2)) ^ swizzle(r)) * 16) + (g & 3) * 4));
        } else if (kDP == 128) {
          const uint2 x = lds64(row + uint32_t((((warp * 4 + (g >> 1)) ^ swizzle(r)) * 16) + (g & 1) * 8));
          w[i][0] = x.x, w[i][1] = x.y;
        } else {
          const uint4 x = lds128(row + uint32_t(((warp * 8 + g) ^ swizzle(r)) * 16));
          w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
        }
      }
    };
    bool nan = false;
    if (kType == SMP_CACHE_E4M3) {
#pragma unroll
      for (int mt = 0; mt < 2 * S::kMT; ++mt) edge |= !valid[mt / S::kMT][meta][mt % S::kMT];
      if (edge) {
        // a NaN code times a weight of 0 would reach rows that do not see its token
#pragma unroll
        for (int mt = 0; mt < 2 * S::kMT; ++mt) {
          uint32_t w[4][4];
          values(mt, w);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kWords; ++j) nan |= __vcmpeq4(w[i][j] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
        }
        nan = __any_sync(~0u, nan);
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2 * S::kMT; ++mt) {
      uint32_t w[4][4], pf[kNT][S::kParts][2];
      values(mt, w);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const uint32_t at = p_at + uint32_t((mt * kNT + nt) * S::kParts * 256);
        if (kSplit) {
          const uint4 x = lds128(at);
          pf[nt][0][0] = x.x, pf[nt][0][1] = x.y, pf[nt][S::kParts - 1][0] = x.z, pf[nt][S::kParts - 1][1] = x.w;
        } else {
          const uint2 x = lds64(at);
          pf[nt][0][0] = x.x, pf[nt][0][1] = x.y;
        }
      }
      if (kType == SMP_CACHE_E4M3 && nan) {
        // NaN codes become 0 for the product; a row that sees one gets NaN from a count of them
        uint32_t seen[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            seen[nt][half] = transpose8(
                pack_f16(visible(mt, nt, half * 2) ? 1.0f : 0.0f, visible(mt, nt, half * 2 + 1) ? 1.0f : 0.0f));
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          uint32_t z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = __vcmpeq4(w[i][j] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            w[i][j] &= ~z[i];
            z[i] &= 0x38383838u;                               // the code of 1
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t f[4];
            unpack4<kType>(__byte_perm(z[0], z[1], half ? 0x7362 : 0x5140), f[0], f[1]);
            unpack4<kType>(__byte_perm(z[2], z[3], half ? 0x7362 : 0x5140), f[2], f[3]);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_f16(count, f, seen[nt][0], seen[nt][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (count[e] > 0.0f) o[nt][2 * j + half][e] = __int_as_float(0x7FC00000);
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kWords; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t f[4];
          unpack4<kType>(__byte_perm(w[0][j], w[1][j], half ? 0x7362 : 0x5140), f[0], f[1]);
          unpack4<kType>(__byte_perm(w[2][j], w[3][j], half ? 0x7362 : 0x5140), f[2], f[3]);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int p = 0; p < S::kParts; ++p) mma_f16(o[nt][2 * j + half], f, pf[nt][p][0], pf[nt][p][1]);
        }
    }
  }
  copies_wait<0>();

  // ---- l over all keys; O needs no joining: a warp has its half of the head
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], d);
      if (g == 0) row_part[warp][nt * 8 + 2 * t + c] = l[nt][c];
    }
  __syncthreads();                             // and both warps are done with the rings
  float* const part = a.partial + (int64_t(blockIdx.x) * 2 + (seg.first ? 1 : 0)) * (8 * kMaxNT) * (kDP + 2);
  constexpr int kMine = kDP / 16;              // a lane's consecutive elements of a row
  const int d0 = warp * (kDP / 2) + g * kMine;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = nt * 8 + 2 * t + c;
      if (r >= live_rows) continue;
      const float all = row_part[0][r] + row_part[1][r];
      const float ref = has_ref >> (2 * nt + c) & 1 ? m[nt][c] : -INFINITY;     // -inf: nothing was seen (or only NaN)
      const int64_t gr = r0 + r, token = req.first + gr / a.group, qh = int64_t(head) * a.group + gr % a.group;
      const float inv = !seg.whole ? 1.0f : all == 0.0f ? 0.0f : 1.0f / all;
      float y[kMine];
#pragma unroll
      for (int d = 0; d < S::kDT; ++d) y[2 * d] = o[nt][d][c] * inv, y[2 * d + 1] = o[nt][d][c + 2] * inv;
      if (!seg.whole) {
#pragma unroll
        for (int i = 0; i < kMine; i += 4)
          *reinterpret_cast<float4*>(part + r * kDP + d0 + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
      } else if (d0 < a.dim) {
        T* const out = static_cast<T*>(a.out) + token * a.out_stride + qh * a.dim + d0;
#pragma unroll
        for (int i = 0; i < kMine; i += 4) {
          const float z[4] = {y[i], y[i + 1], y[i + 2], y[i + 3]};
          if (a.out_vector) {
            store4(out + i, z);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) store1(out + i + e, z[e]);
          }
        }
      }
      if (warp == 0 && g == 0) {
        if (!seg.whole) {
          part[8 * kMaxNT * kDP + r] = ref;
          part[8 * kMaxNT * (kDP + 1) + r] = all;
        } else if (a.lse) {
          a.lse[token * a.q_heads + qh] = all == 0.0f ? -INFINITY : (ref + log2f(all)) * 0.6931471805599453f;
        }
      }
    }
}

template <int kDP, int kMaxNT, int kType, bool kSplit>
__global__ void __launch_bounds__(kAttnThreads, (AttnKernel<kDP, kMaxNT, kSplit>::kCtas)) attention_kernel(const AttnArgs a) {
  using S = AttnShape<kDP, kMaxNT, kSplit>;
  using Line = AttnLine<kAttnThreads, S::kTile, kMaxNT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ typename Line::Shared line_shared;
  __shared__ AttnShared<S::kMT, S::kRows> sh;
  __shared__ Line line_at;
  const int tid = int(threadIdx.x);
  allow_dependent_launch();
  grid_dependency_wait();

  int flags = 0;
  {
    Line line;
    const bool work = line.begin(a, line_shared, flags);
    if (blockIdx.x != 0) flags = 0;            // one CTA reports the lengths
    if (!work) {
      if (flags && a.status) atomicOr(a.status, flags);
      return;
    }
    if (tid == 0) line_at = line;              // kept in shared memory: the segments need the registers
  }
  // chunks past the head's end are never written: they stay zero
  if (a.dim < kDP)
    for (int i = tid; i < S::kQAt / 16; i += kAttnThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const int nt = line_at.nt;
  for (bool more = true; more;) {
    {
      const AttnSegment seg = line_at.segment(a);
      const AttnRequest req = line_at.req;
      const int b = line_at.b, head = line_at.head;
      auto run = [&](auto size) {
        attention_segment<kDP, decltype(size)::value, kMaxNT, kType, kSplit>(a, seg, req, b, head, smem, sh, flags);
      };
      using std::integral_constant;
      constexpr int kMin = attn_least_eights(kMaxNT);
      if (kMin == kMaxNT || nt == kMaxNT) run(integral_constant<int, kMaxNT>());
      else if (kMin == kMaxNT - 1 || nt == kMaxNT - 1) run(integral_constant<int, kMin < kMaxNT ? kMaxNT - 1 : kMin>());
      else run(integral_constant<int, kMin>());
    }
    Line line = line_at;
    if (line.pos == 0 && line.end - line.at < line.cost && tid == 0) {     // begun here, and cut

      const AttnSegment seg = line.segment(a);
      AttnJoin j{};
      j.parts = line.parts(), j.first = line.req.first, j.r0 = seg.r0, j.live_rows = seg.live_rows, j.head = line.head;
      a.joins[blockIdx.x] = j;
    }
    more = line.next(a);
    __syncthreads();                           // everyone has read the line and the shared exchanges
    if (tid == 0) line_at = line;
    __syncthreads();
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

// ---------------------------------------------------------------- joining cut units
//
// Grid: (CTAs of the main kernel, row tiles of 8).  The unit that began in main
// CTA j and was cut there has its parts in slot 1 of j and slots 0 of the next
// CTAs; one warp joins one row.
constexpr int kJoinThreads = 256;

template <int kDP, bool kSplit>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnArgs a, const int rows) {
  using T = typename std::conditional<kSplit, float, uint16_t>::type;
  allow_dependent_launch();
  grid_dependency_wait();
  const AttnJoin u = a.joins[blockIdx.x];
  const int r = int(blockIdx.y) * (kJoinThreads / 32) + (int(threadIdx.x) >> 5), lane = int(threadIdx.x) & 31;
  if (u.parts < 2 || r >= u.live_rows) return;
  const int64_t slot = int64_t(rows) * (kDP + 2);
  auto part = [&](int i) { return a.partial + (int64_t(blockIdx.x + i) * 2 + (i == 0)) * slot; };
  constexpr int kPer = kDP / 32;
  float top = -INFINITY, all = 0.0f, x[kPer] = {};
  for (int i = lane; i < u.parts; i += 32) top = fmaxf(top, part(i)[rows * kDP + r]);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  for (int i0 = 0; i0 < u.parts; i0 += 32) {
    float f = 0.0f;
    if (i0 + lane < u.parts) {
      const float m = part(i0 + lane)[rows * kDP + r], l = part(i0 + lane)[rows * (kDP + 1) + r];
      // a part that saw only NaN has no reference, but a sum; factors in two steps, as in the main kernel
      const float half = m == -INFINITY ? 1.0f : exp2_approx(0.5f * (m - top));
      f = l == 0.0f ? 0.0f : half * half;
      if (l != 0.0f) all += l * half * half;
    }
    const int count = min(32, u.parts - i0);
#pragma unroll 8
    for (int i = 0; i < count; ++i) {
      const float w = __shfl_sync(~0u, f, i);
      const float* p = part(i0 + i) + r * kDP + lane * kPer;
      float y[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) y[e] = p[e];
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] = w != 0.0f ? fmaf(y[e], w, x[e]) : x[e];
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(~0u, all, d);
  const float inv = all == 0.0f ? 0.0f : 1.0f / all;
  const int64_t gr = u.r0 + r, token = u.first + gr / a.group, qh = int64_t(u.head) * a.group + gr % a.group;
  T* out = static_cast<T*>(a.out) + token * a.out_stride + qh * a.dim + lane * kPer;
  if (lane * kPer < a.dim) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) store1(out + e, x[e] * inv);
  }
  if (lane == 0 && a.lse)
    a.lse[token * a.q_heads + qh] = all == 0.0f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------- launch

template <int kDP, int kMaxNT, int kType, bool kSplit>
cudaError_t attn_launch_shape(const AttnArgs& a, int dev, cudaStream_t st) {
  using K = AttnKernel<kDP, kMaxNT, kSplit>;
  LaunchShape ls;
  ls.smem = size_t(K::kSmem);
  const int grid = device_sms(dev) * K::kCtas;         // one wave
  cudaError_t err = prepare_kernel(reinterpret_cast<const void*>(&attention_kernel<kDP, kMaxNT, kType, kSplit>), dev, ls);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = ls.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, attention_kernel<kDP, kMaxNT, kType, kSplit>, a);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3(unsigned(grid), unsigned(kMaxNT));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attention_join_kernel<kDP, kSplit>, a, K::kRows);
}

// Kernels per head size: row tiles of up to 16 rows, whose smaller state leaves
// room for five CTAs per SM, of 24, and of up to 40 (32 for heads of 256 and
// binary32 queries), beyond which the registers spill.  8 rows of 32 requests of
// up to 4 K keys: 40 us with the first and 49 with the second; 20 rows: 60 us
// with the second and 82 to 88 with the third.  `rows` is what the host
// expects of most requests; the kernel sees the longest itself, and takes
// several row tiles, which read the keys again, where its largest is too small.
template <int kType, bool kSplit, int kDP>
cudaError_t attn_launch_dim(const AttnArgs& a, int64_t rows, int dev, cudaStream_t st) {
  if (rows <= 16) return attn_launch_shape<kDP, 2, kType, kSplit>(a, dev, st);
  if constexpr (!kSplit && kDP != 256)
    if (rows <= 24) return attn_launch_shape<kDP, 3, kType, kSplit>(a, dev, st);
  return attn_launch_shape<kDP, kSplit || kDP == 256 ? 4 : 5, kType, kSplit>(a, dev, st);
}

// One translation unit per cache and query type defines its own.
template <int kType, bool kSplit>
cudaError_t attn_launch(const AttnArgs& a, int64_t rows, int dev, cudaStream_t st);

#define SMP_ATTENTION_INSTANCE(TYPE, SPLIT)                                                          \
  template <>                                                                                        \
  cudaError_t attn_launch<TYPE, SPLIT>(const AttnArgs& a, int64_t rows, int dev, cudaStream_t st) {  \
    if (a.dim <= 64) return attn_launch_dim<TYPE, SPLIT, 64>(a, rows, dev, st);                      \
    if (a.dim <= 128) return attn_launch_dim<TYPE, SPLIT, 128>(a, rows, dev, st);                    \
    return attn_launch_dim<TYPE, SPLIT, 256>(a, rows, dev, st);                                      \
  }

template <>
cudaError_t attn_launch<SMP_CACHE_E4M3, false>(const AttnArgs&, int64_t, int, cudaStream_t);
template <>
cudaError_t attn_launch<SMP_CACHE_E4M3, true>(const AttnArgs&, int64_t, int, cudaStream_t);
template <>
cudaError_t attn_launch<SMP_CACHE_I8, false>(const AttnArgs&, int64_t, int, cudaStream_t);
template <>
cudaError_t attn_launch<SMP_CACHE_I8, true>(const AttnArgs&, int64_t, int, cudaStream_t);

}  // namespace smp
