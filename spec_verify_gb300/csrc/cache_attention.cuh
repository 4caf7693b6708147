// Causal attention over the paged 8-bit cache: the kernels, included by one
// translation unit per pair of cache type and query type.
//
// Mathematics.  For the rows of one key head (its queries times the query
// heads that share it) and tiles of keys:
//   S^T = K Q^T,  P = 2^(S c - m),  l += sum P,  O^T += V^T (P v u)
// with c = scale * log2(e) * (the block's key scale), v the block's value
// scale, and two references per row that move only when they must: m, raised
// when a score passes it by more than 2^11 (then O and l are multiplied by
// 2^(m_old - m_new)), and u, a power of two, lowered when a weight P v u would
// pass 2^15, the range of 16-bit floats.  Both leave the largest weights far
// above the smallest normal 16-bit float, so the weights that matter keep all
// 11 bits whatever the scales of the blocks; l is summed from binary32 P.
//
// Both products run on the tensor cores with the cache as the 16-row operand
// (tokens, then head elements) and the query rows as the 8-wide one, so one
// to eight rows waste nothing.  8-bit codes become 16-bit floats exactly in
// registers.  A query row enters as 16-bit floats scaled by a power of two to
// a largest element near 2^9: for bf16 queries that is exact down to 2^-33 of
// the row's largest element; binary32 queries and their weights enter as a
// sum of two 16-bit floats (22 bits).
//
// Split.  The keys of all (request, row tile, key head) units form one line of
// work that is cut into equal shares, one per resident CTA, whatever the
// lengths; a unit cut by a share's end leaves its parts (m, l, O) in the
// workspace, and a second kernel joins them in order.  Inside a CTA the warps
// form teams: a team streams its own tiles through a ring in shared memory by
// 16-byte asynchronous copies, its warps taking 8 kNT rows each; teams are
// joined at the unit's end.  Nothing waits on another CTA.
//
// Bound: HBM (one byte per code) up to about 32 rows per key head, then the
// conversions and tensor cores.
#pragma once

#include <cuda_runtime.h>

#include <math.h>

#include "cache.cuh"
#include "launch.h"

namespace smp {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kAttnUnitCost = 3;        // a unit's fixed cost, in tiles
constexpr float kShift = 3.0f;          // a new reference m puts the row's largest score at 2^3
constexpr float kRaise = 11.0f;         // and is replaced once a score passes 2^11
constexpr uint32_t kWeightLimit = 0x7800u;       // 2^15 as a 16-bit float: u is lowered past it
constexpr int kWeightExp = 8;                    // a new u puts the largest weight in [2^8, 2^9)
constexpr int kMaxUExp = 60;                     // u <= 2^60 and v <= 2^66, so that v u is finite

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
  int4* joins;              // [CTA]: request, row tile, key head, parts of the unit that begins there (0: none)
  bool q_vector, out_vector;   // queries and results take 16-byte (results: 4-element) accesses
  int min_share;            // smallest share of a CTA, in tiles
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

// The larger of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
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

template <int kDP, int kNT, int kRG, bool kSplit>
struct AttnShape {
  static constexpr int kTile = kDP == 256 ? 16 : 32;             // tokens per tile
  static constexpr int kMT = kTile / 16;                         // 16-token row tiles of a tile
  static constexpr int kChunks = kDP / 16;                       // 16-byte chunks of a row
  static constexpr int kSteps = kDP / 16;                        // products of depth 16 over the head
  static constexpr int kDT = kDP / 16;                           // 16-row tiles of V^T
  static constexpr int kStage = 2 * kTile * kDP;                 // bytes of one ring stage (keys, then values)
  static constexpr int kTeams = kAttnWarps / kRG;
  static constexpr int kWarpRows = 8 * kNT;
  static constexpr int kRows = kWarpRows * kRG;                  // rows of a unit's row tile
  static constexpr int kParts = kSplit ? 2 : 1;
  static constexpr bool kQReg = kNT * kSteps * 2 * kParts <= 32; // query fragments in registers
  static constexpr int kOPitch = kDP + 4;                        // floats of a row when teams are joined
  // stages of a team's ring: 96, 80 or 64 KB per CTA for teams of 1, 2 or 4 warps, whose queries take up to 8, 16
  // or 32 KB
  static constexpr int kDepth = (kDP == 64 ? 2 : 1) * (kRG == 4 ? 8 : kRG == 2 ? 5 : 3);
  static constexpr int kRing = kTeams * kDepth * kStage;
  static constexpr int kJoin = kAttnWarps * kWarpRows * kOPitch * 4;
  static constexpr int kRingBytes = kRing > kJoin ? kRing : kJoin;
  static constexpr int kQueryBytes = kQReg ? 0 : kRows / 8 * kSteps * kParts * 32 * 8;
  // per stage: kMT key scales, kMT value scales, kMT flags; then (m, l, weight) of every warp's rows
  static constexpr int kScaleBytes = kTeams * kDepth * kMT * 12;
  static constexpr int kSmem = kRingBytes + kQueryBytes + kScaleBytes + 3 * kAttnWarps * kWarpRows * 4;
};

// ---------------------------------------------------------------- main kernel

template <int kDP, int kNT, int kRG, int kType, bool kSplit>
__global__ void __launch_bounds__(kAttnThreads, 2) attention_kernel(const AttnArgs a) {
  using S = AttnShape<kDP, kNT, kRG, kSplit>;
  using T = typename std::conditional<kSplit, float, uint16_t>::type;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[kAttnWarps + 1];
  __shared__ int64_t found[2];

  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  constexpr int teams = S::kTeams, rows = S::kRows, depth = S::kDepth, ring_bytes = S::kRingBytes;
  const int team = warp / kRG, rg = warp % kRG;
  const uint32_t ring = smem_addr(smem) + uint32_t(team * depth) * S::kStage;
  uint8_t* const meta = smem + ring_bytes + S::kQueryBytes;
  float* const meta_scale = reinterpret_cast<float*>(meta) + team * depth * S::kMT * 3;
  float* const row_m = reinterpret_cast<float*>(meta + S::kScaleBytes);       // [warp][row]
  float* const row_l = row_m + kAttnWarps * S::kWarpRows;
  float* const row_w = row_l + kAttnWarps * S::kWarpRows;

  allow_dependent_launch();
  grid_dependency_wait();

  // ---- this CTA's share of the line of work
  const int cta = int(blockIdx.x);
  auto unit_tiles = [&](const AttnRequest& r) {
    const int64_t lo = a.window > 0 ? max(int64_t(r.len) - r.n - a.window + 1, int64_t(0)) : 0;
    return max(0, (r.len + S::kTile - 1) / S::kTile - int(lo / S::kTile));
  };
  auto row_tiles = [&](const AttnRequest& r) {
    return int((int64_t(r.n) * a.group + rows - 1) / rows);
  };
  auto cost_of = [&](int b, int& flags) -> int64_t {
    const AttnRequest r = attn_request(a, b);
    if (r.bad) flags |= kRowBadLength;
    return int64_t(row_tiles(r)) * a.kv_heads * (unit_tiles(r) + kAttnUnitCost);
  };
  int flags = 0;
  int64_t sum = 0;
  const int64_t first_cost = tid < a.batch ? cost_of(tid, flags) : 0;
  sum = first_cost;
  for (int b = tid + kAttnThreads; b < a.batch; b += kAttnThreads) sum += cost_of(b, flags);
  if (cta != 0) flags = 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) scan[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kAttnWarps; ++w) total += scan[w];
  const int64_t share = max(int64_t(a.min_share), (total + gridDim.x - 1) / gridDim.x);
  const int64_t mine = share * cta, end = min(total, mine + share);
  if (tid == 0) a.joins[cta] = make_int4(0, 0, 0, 0);
  if (mine >= end) {
    if (flags && a.status) atomicOr(a.status, flags);
    return;
  }
  for (int64_t base = 0, chunk = 0;; chunk += kAttnThreads) {
    const int b = int(chunk) + tid;
    int ignored = 0;
    const int64_t c = chunk == 0 ? first_cost : b < a.batch ? cost_of(b, ignored) : 0;
    int64_t inc = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int64_t before = base;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      if (w < warp) before += scan[w];
      base += scan[w];
    }
    if (before + inc - c <= mine && mine < before + inc) found[0] = b, found[1] = before + inc - c;
    if (base > mine) break;              // the same in every thread
  }
  __syncthreads();

  // ---- unused chunks of padded heads stay zero
  if (a.dim < kDP) {
    for (int i = tid; i < ring_bytes / 16; i += kAttnThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }

  int b = int(found[0]);
  AttnRequest req = attn_request(a, b);
  int64_t cost = unit_tiles(req) + kAttnUnitCost;
  int64_t unit = (mine - found[1]) / cost, at = mine;
  int64_t pos = mine - found[1] - unit * cost;
  int rt = int(unit / a.kv_heads), head = int(unit - int64_t(rt) * a.kv_heads);

  // A stage's copies: one instruction covers kRowsPerCopy rows, keys first; the warps of a team take turns.
  constexpr int kRowsPerCopy = 32 / S::kChunks, kCopies = 2 * S::kTile / kRowsPerCopy, kHalf = kCopies / 2;
  constexpr int kPerMT = kHalf / S::kMT;                     // copies of 16 tokens' keys
  constexpr int kSwizzles = 8 / kRowsPerCopy / kRG > 1 ? 8 / kRowsPerCopy / kRG : 1;
  const int my_chunk = lane % S::kChunks, my_row = lane / S::kChunks;
  // chunk c of row r lies at chunk c ^ swizzle(r): 16-byte reads of keys (8 rows, 4 chunks) and of values (8 rows two
  // apart, 2 chunks) then meet every bank once
  auto swizzle = [](int r) { return kDP == 64 ? (r >> 1) & 3 : (r & 6) ^ ((r & 1) << 2); };
  uint32_t lane_dst[kSwizzles];
#pragma unroll
  for (int i = 0; i < kSwizzles; ++i)
    lane_dst[i] = uint32_t((rg * kRowsPerCopy + my_row) * kDP +
                           ((my_chunk ^ swizzle((i * kRG + rg) * kRowsPerCopy + my_row)) * 16));
  const int lane_src = ((rg % kPerMT) * kRowsPerCopy + my_row) * kDP + my_chunk * 16;

  while (at < end) {
    const int64_t take = min(cost - pos, end - at);
    const bool whole = pos == 0 && take == cost;
    const int n = req.n, len = req.len;
    // rows of this tile: r0 .. r0 + live - 1 of the request's n * group
    const int64_t r0 = int64_t(rt) * rows;
    const int live_rows = int(min(int64_t(rows), int64_t(n) * a.group - r0));
    const int p_first = len - n + int(r0 / a.group), p_last = len - n + int((r0 + live_rows - 1) / a.group);
    const int see_first = a.window > 0 ? int(max(int64_t(0), int64_t(p_first) - a.window + 1)) : 0;
    const int tile0 = int((a.window > 0 ? max(int64_t(len) - n - a.window + 1, int64_t(0)) : 0) / S::kTile);
    const int tile_lo = max(tile0 + int(max(pos - kAttnUnitCost, int64_t(0))), see_first / S::kTile);
    const int tile_hi = min(tile0 + int(max(pos + take - kAttnUnitCost, int64_t(0))),
                            p_last >= 0 ? p_last / S::kTile + 1 : 0);
    const int tiles = max(0, tile_hi - tile_lo);
    const int iters = (tiles - team + teams - 1) / teams;       // of this team (<= 0: none)

    // ---- the ring: copies run depth - 1 stages ahead
    constexpr int kPer = 32 / S::kMT;                           // iterations whose block ids the lanes hold
    auto load_ids = [&](int k0) {
      const int k = k0 + lane / S::kMT, token = (tile_lo + team + k * teams) * S::kTile + (lane % S::kMT) * 16;
      int id = -1;
      if (k < iters && token < len) {
        id = a.table[int64_t(b) * a.stride + (token >> a.shift)];
        if (id < 0 || id >= a.num_blocks) id = -1, flags |= kRowBadBlock;
      }
      return id;
    };
    int ids = load_ids(0), ids_next = load_ids(kPer);
    int in_k = 0, in_slot = 0, in_id = 0, in_token = (tile_lo + team) * S::kTile;
    const int64_t head_at = (int64_t(head) << a.shift) * a.dim, block_size_all = (int64_t(a.kv_heads) << a.shift) * a.dim;
    auto issue = [&]() {
      if (in_k < iters) {
        if (in_id == 32) {
          in_id = 0;
          ids = ids_next;
          ids_next = load_ids(in_k + kPer);
        }
        const uint32_t dst = ring + uint32_t(in_slot) * S::kStage;
        int64_t off[S::kMT];
        bool ok[S::kMT], full = in_token + S::kTile <= len && a.dim == kDP;
#pragma unroll
        for (int mt = 0; mt < S::kMT; ++mt) {
          const int id = __shfl_sync(~0u, ids, in_id + mt);
          ok[mt] = id >= 0;
          full &= ok[mt];
          off[mt] = int64_t(max(id, 0)) * block_size_all + head_at + ((in_token + 16 * mt) & ((1 << a.shift) - 1)) * a.dim;
        }
        if (rg == 0) {
          const int id = __shfl_sync(~0u, ids, in_id + lane % S::kMT);
          if (lane < 2 * S::kMT) {
            float* m = meta_scale + in_slot * S::kMT * 3 + lane;
            copy4(smem_addr(m), (lane < S::kMT ? a.k_scale : a.v_scale) + int64_t(max(id, 0)) * a.kv_heads + head, id >= 0);
            if (lane < S::kMT) reinterpret_cast<int*>(m)[2 * S::kMT] = id >= 0;
          }
        }
        if (full) {
          // every chunk of every row: a lane's offsets are constants but for kSwizzles of them
#pragma unroll
          for (int j = 0; j < kCopies / kRG; ++j) {
            const int jj = j * kRG % kHalf;                            // + rg: the copy's place in its half
            const bool second = kRG > kPerMT ? rg >= kPerMT : jj >= kPerMT;
            copy16(dst + uint32_t((j * kRG / kHalf) * S::kTile * kDP + jj * kRowsPerCopy * kDP) +
                       lane_dst[jj / kRG % kSwizzles],
                   (j * kRG / kHalf ? a.v : a.k) + (second ? off[S::kMT - 1] : off[0]) + lane_src +
                       (jj % kPerMT) * kRowsPerCopy * kDP);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kCopies / kRG; ++j) {
            const int jj = j * kRG % kHalf + rg, row = jj * kRowsPerCopy + my_row;
            const bool second = jj >= kPerMT;
            if (my_chunk * 16 < a.dim)
              copy16(dst + uint32_t((j * kRG / kHalf) * S::kTile * kDP + row * kDP + ((my_chunk ^ swizzle(row)) * 16)),
                     (j * kRG / kHalf ? a.v : a.k) + (second ? off[S::kMT - 1] : off[0]) + (row % 16) * a.dim +
                         my_chunk * 16,
                     (second ? ok[S::kMT - 1] : ok[0]) && in_token + row < len);
          }
        }
        ++in_k;
        in_id += S::kMT;
        in_token += teams * S::kTile;
        in_slot = in_slot + 1 == depth ? 0 : in_slot + 1;
      }
      copies_commit();
    };
    for (int k = 0; k < depth - 1; ++k) issue();

    // ---- query fragments: lane (g, t) holds the 16-element chunks t + 4 h of row g of each row tile
    constexpr int kQ4 = S::kSteps * S::kParts / 2;             // 16-byte pieces of a row tile's fragments per lane
    uint32_t qreg[S::kQReg ? kNT : 1][S::kQReg ? S::kSteps * S::kParts * 2 : 1];
    float factor[kNT][2];
    int see[kNT][2];                     // last visible position of columns 2t, 2t + 1
    {
      uint4* const qs = reinterpret_cast<uint4*>(smem + ring_bytes) + rg * kNT * kQ4 * 32;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const int row = rg * S::kWarpRows + nt * 8 + g;
        const bool ok = row < live_rows;
        const int64_t gr = r0 + row;
        const int token = req.first + int(gr / a.group), qh = head * a.group + int(gr % a.group);
        const T* q = static_cast<const T*>(a.q) + (ok ? token * a.q_stride + int64_t(qh) * a.dim : 0);
        float x[S::kSteps][4];
#pragma unroll
        for (int h = 0; h < kDP / 64; ++h) {
          const int d = (t + 4 * h) * 16;
          if (ok && d < a.dim && a.q_vector) {
            float y[8];
            load8(q + d, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[h * 4 + e / 4][e % 4] = y[e];
            load8(q + d + 8, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[h * 4 + 2 + e / 4][e % 4] = y[e];
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[h * 4 + e / 4][e % 4] = ok && d < a.dim ? load1(q + d + e) : 0.0f;
          }
        }
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[s][e]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        // up: the power of two that takes the largest element to [2^9, 2^10); down: its inverse
        const int up_exp = min(max(263 - int(__float_as_uint(top) >> 23), 1), 253);
        const float up = __uint_as_float(uint32_t(up_exp) << 23);
        const float down = __uint_as_float(uint32_t(254 - up_exp) << 23) * a.scale;
        factor[nt][0] = __shfl_sync(~0u, down, 8 * t);
        factor[nt][1] = __shfl_sync(~0u, down, 8 * t + 4);
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
        } else if (team == 0) {
#pragma unroll
          for (int i = 0; i < kQ4; ++i)
            qs[(nt * kQ4 + i) * 32 + lane] = make_uint4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int64_t r = r0 + rg * S::kWarpRows + nt * 8 + 2 * t + c;
          see[nt][c] = r - r0 < live_rows ? len - n + int(r / a.group) : len;     // unused rows: everything, unread
        }
      }
    }
    if (!S::kQReg) __syncthreads();
    const uint32_t q_at = smem_addr(smem + ring_bytes) + uint32_t(rg * kNT * kQ4 * 32 + lane) * 16;

    float o[kNT][S::kDT][4];
    float l[kNT][2], m[kNT][2], u[kNT][2];
    uint32_t set_m = 0;                          // rows (2 nt + c) whose reference is set; m = 0, u = 1 before
    constexpr uint32_t kAllSet = (1u << (2 * kNT)) - 1;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = 0.0f, u[nt][c] = 1.0f, l[nt][c] = 0.0f;
        if (rg * S::kWarpRows + nt * 8 + 2 * t + c >= live_rows) set_m |= 1u << (2 * nt + c);   // unused: never awaited
      }
#pragma unroll
      for (int d = 0; d < S::kDT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][d][e] = 0.0f;
    }

    uint32_t set_u = set_m;
    int slot = 0, token0 = (tile_lo + team) * S::kTile;
    for (int k = 0; k < iters; ++k) {
      copies_wait<depth - 2>();
      if (kRG == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kRG * 32) : "memory");
      issue();
      const uint32_t kst = ring + uint32_t(slot) * S::kStage, vst = kst + S::kTile * kDP;
      const float* sc = meta_scale + slot * S::kMT * 3;

      // ---- S^T = K Q^T
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
              const uint4 x = lds128(q_at + uint32_t(nt * kQ4 + h * 4 + i) * 512);
              q[0] = x.x, q[1] = x.y, q[S::kParts * 2 - 2] = x.z, q[S::kParts * 2 - 1] = x.w;
            } else {
              if (i % 2 == 0) q_two[nt] = lds128(q_at + uint32_t(nt * kQ4 + (h * 4 + i) / 2) * 512);
              q[0] = i % 2 ? q_two[nt].z : q_two[nt].x, q[1] = i % 2 ? q_two[nt].w : q_two[nt].y;
            }
#pragma unroll
            for (int p = 0; p < S::kParts; ++p)
#pragma unroll
              for (int mt = 0; mt < S::kMT; ++mt) mma_f16(s[mt][nt], f[mt], q[2 * p], q[2 * p + 1]);
          }
        }
      }

      // ---- exponents: s = S c - m, masked; m raised where one passes the limit
      bool edge = token0 + S::kTile - 1 > p_first || (a.window > 0 && token0 <= p_last - a.window);
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt) {
        edge |= !reinterpret_cast<const int*>(sc)[2 * S::kMT + mt];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const uint64_t c = mul2(pair(sc[mt], sc[mt]), pair(factor[nt][0], factor[nt][1]));
          const uint64_t less = pair(-m[nt][0], -m[nt][1]);
          unpair(fma2(pair(s[mt][nt][0], s[mt][nt][1]), c, less), s[mt][nt][0], s[mt][nt][1]);
          unpair(fma2(pair(s[mt][nt][2], s[mt][nt][3]), c, less), s[mt][nt][2], s[mt][nt][3]);
        }
      }
      auto visible = [&](int mt, int nt, int e) {
        const int j = token0 + mt * 16 + g + (e / 2) * 8, p = see[nt][e % 2];
        return j <= p && (a.window == 0 || j > p - a.window) && reinterpret_cast<const int*>(sc)[2 * S::kMT + mt];
      };
      if (edge) {
#pragma unroll
        for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!visible(mt, nt, e)) s[mt][nt][e] = -INFINITY;
      }
      float largest = s[0][0][0];
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) largest = max3(largest, s[mt][nt][c], s[mt][nt][c + 2]);
      if (__any_sync(~0u, largest > kRaise || set_m != kAllSet)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float alpha[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
            for (int mt = 1; mt < S::kMT; ++mt) x = fmaxf(x, fmaxf(s[mt][nt][c], s[mt][nt][c + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
            const uint32_t bit = 1u << (2 * nt + c);
            alpha[c] = 1.0f;
            if ((set_m & bit) ? x > kShift : x > -INFINITY) {
              const float up = x - kShift;
              if (set_m & bit) alpha[c] = exp2_approx(-up);
              set_m |= bit;
              m[nt][c] += up;
              l[nt][c] *= alpha[c];
#pragma unroll
              for (int mt = 0; mt < S::kMT; ++mt) s[mt][nt][c] -= up, s[mt][nt][c + 2] -= up;
            }
          }
#pragma unroll
          for (int d = 0; d < S::kDT; ++d) {
            o[nt][d][0] *= alpha[0], o[nt][d][1] *= alpha[1], o[nt][d][2] *= alpha[0], o[nt][d][3] *= alpha[1];
          }
        }
      }

      // ---- weights P v u as 16-bit floats; u lowered where one passes the limit
      float v_scale[S::kMT];
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt) v_scale[mt] = fminf(sc[S::kMT + mt], 0x1p66f);
      uint32_t pf[S::kMT][kNT][S::kParts][2];
      uint32_t packed_max = 0;
      auto weigh = [&]() {
#pragma unroll
        for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            const uint64_t vu = mul2(pair(v_scale[mt], v_scale[mt]), pair(u[nt][0], u[nt][1]));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float p0, p1;
              unpair(mul2(pair(s[mt][nt][half * 2], s[mt][nt][half * 2 + 1]), vu), p0, p1);
              pf[mt][nt][0][half] = pack_f16(p0, p1);
              if (kSplit) pf[mt][nt][S::kParts - 1][half] = rest_f16(pf[mt][nt][0][half], p0, p1);
              packed_max = max_f16x2(packed_max, pf[mt][nt][0][half]);
            }
          }
      };
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        uint64_t sum = pair(l[nt][0], l[nt][1]);
#pragma unroll
        for (int mt = 0; mt < S::kMT; ++mt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = exp2_approx(s[mt][nt][e]);
          sum = add2(sum, add2(pair(s[mt][nt][0], s[mt][nt][1]), pair(s[mt][nt][2], s[mt][nt][3])));
        }
        unpair(sum, l[nt][0], l[nt][1]);
      }
      weigh();
      if (__any_sync(~0u, (packed_max & 0xFFFFu) > kWeightLimit || (packed_max >> 16) > kWeightLimit || set_u != kAllSet)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float beta[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = 0.0f;
#pragma unroll
            for (int mt = 0; mt < S::kMT; ++mt) x = fmaxf(x, fmaxf(s[mt][nt][c], s[mt][nt][c + 2]) * v_scale[mt]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
            const uint32_t bit = 1u << (2 * nt + c);
            beta[c] = 1.0f;
            const int exp = min(kWeightExp + 127 - int(__float_as_uint(x) >> 23), kMaxUExp);
            const float lower = __uint_as_float(uint32_t(max(exp, -126) + 127) << 23);
            if (x > 0.0f && (!(set_u & bit) || lower < u[nt][c])) {
              if (set_u & bit) beta[c] = lower / u[nt][c];
              u[nt][c] = lower;
              set_u |= bit;
            }
          }
#pragma unroll
          for (int d = 0; d < S::kDT; ++d) {
            o[nt][d][0] *= beta[0], o[nt][d][1] *= beta[1], o[nt][d][2] *= beta[0], o[nt][d][3] *= beta[1];
          }
        }
        weigh();
      }
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int p = 0; p < S::kParts; ++p)
#pragma unroll
            for (int half = 0; half < 2; ++half) pf[mt][nt][p][half] = transpose8(pf[mt][nt][p][half]);

      // ---- O^T += V^T P^T: lane (g, t) reads elements of tokens 2t, 2t+1, 2t+8, 2t+9; row g of tile d is element
      // 16 g + 2 d (8 g + 2 d of 64), row g + 8 the next one
      auto values = [&](int mt, int part, uint32_t (&w)[4][4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * t + (i & 1) + (i / 2) * 8;
          const uint32_t row = vst + uint32_t((mt * 16 + r) * kDP);
          if (kDP == 64) {
            const uint2 x = lds64(row + uint32_t((((g >> 1) ^ swizzle(r)) * 16) + (g & 1) * 8));
            w[i][0] = x.x, w[i][1] = x.y;
          } else {
            const uint4 x = lds128(row + uint32_t(((g + 8 * part) ^ swizzle(r)) * 16));
            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
          }
        }
      };
      constexpr int kPartsV = kDP == 256 ? 2 : 1, kWords = kDP == 64 ? 2 : 4;
      bool nan = false;
      if (kType == SMP_CACHE_E4M3 && edge) {
        // a NaN code times a weight of 0 would reach rows that do not see its token
#pragma unroll
        for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
          for (int part = 0; part < kPartsV; ++part) {
            uint32_t w[4][4];
            values(mt, part, w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < kWords; ++j) nan |= __vcmpeq4(w[i][j] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
          }
        nan = __any_sync(~0u, nan);
      }
#pragma unroll
      for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
        for (int part = 0; part < kPartsV; ++part) {
          uint32_t w[4][4];
          values(mt, part, w);
          if (kType == SMP_CACHE_E4M3 && nan) {
            // NaN codes become 0 for the product; a row that sees one gets NaN from a count of them
            uint32_t seen[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int half = 0; half < 2; ++half)
                seen[nt][half] = transpose8(pack_f16(visible(mt, nt, half * 2) ? 1.0f : 0.0f,
                                                     visible(mt, nt, half * 2 + 1) ? 1.0f : 0.0f));
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
                const int d = part * 8 + 2 * j + half;
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                  float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma_f16(count, f, seen[nt][0], seen[nt][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (count[e] > 0.0f) o[nt][d][e] = __int_as_float(0x7FC00000);
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
              const int d = part * 8 + 2 * j + half;
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int p = 0; p < S::kParts; ++p) mma_f16(o[nt][d], f, pf[mt][nt][p][0], pf[mt][nt][p][1]);
            }
        }
      slot = slot + 1 == depth ? 0 : slot + 1;
      token0 += teams * S::kTile;
    }
    copies_wait<0>();

    // ---- join the teams: (m, l) of every row, then O through the ring's memory
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], d);
        if (g == 0) {
          row_m[warp * S::kWarpRows + nt * 8 + 2 * t + c] = set_m >> (2 * nt + c) & 1 ? m[nt][c] : -INFINITY;
          row_l[warp * S::kWarpRows + nt * 8 + 2 * t + c] = l[nt][c];
        }
      }
    __syncthreads();                              // every team is done with the ring
    float* const join = reinterpret_cast<float*>(smem) + warp * S::kWarpRows * S::kOPitch;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const float back[2] = {1.0f / u[nt][0], 1.0f / u[nt][1]};
#pragma unroll
      for (int d = 0; d < S::kDT; ++d)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int e = kDP == 64 ? 8 * g + 2 * d : (d / 8) * 128 + 16 * g + 2 * (d % 8);
          *reinterpret_cast<float2*>(join + (nt * 8 + 2 * t + c) * S::kOPitch + e) =
              make_float2(o[nt][d][c] * back[c], o[nt][d][c + 2] * back[c]);
        }
    }
    // each warp's weight in its row, and the rows' joined (m, l) in the first team's place
    for (int r = tid; r < rows; r += kAttnThreads) {
      float top = -INFINITY, all = 0.0f;
      for (int w = 0; w < teams; ++w) top = fmaxf(top, row_m[w * rows + r]);
      for (int w = 0; w < teams; ++w) {
        const float mw = row_m[w * rows + r], f = mw == -INFINITY ? 0.0f : exp2_approx(mw - top);
        // a NaN score leaves its row's reference alone: its sum, not the weight, is NaN
        row_w[w * rows + r] = row_l[w * rows + r] != 0.0f ? (mw == -INFINITY ? 1.0f : f) : 0.0f;
        if (row_l[w * rows + r] != 0.0f) all += row_l[w * rows + r] * row_w[w * rows + r];
      }
      row_m[r] = top;
      row_l[r] = all;
    }
    __syncthreads();
    constexpr int kVecs = kDP / 4;
    float* const part = a.partial + (int64_t(cta) * 2 + (pos > 0 ? 0 : 1)) * rows * (kDP + 2);
    for (int i = tid; i < rows * kVecs; i += kAttnThreads) {
      const int r = i / kVecs, d = i % kVecs * 4;
      if (r >= live_rows) break;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int w = 0; w < teams; ++w) {
        const float f = row_w[w * rows + r];
        if (f != 0.0f) {
          const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * rows + r) * S::kOPitch + d);
          x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
        }
      }
      if (whole) {
        const float inv = row_l[r] == 0.0f ? 0.0f : 1.0f / row_l[r];
        const int64_t gr = r0 + r;
        T* out = static_cast<T*>(a.out) + (req.first + gr / a.group) * a.out_stride +
                 (int64_t(head) * a.group + gr % a.group) * a.dim;
        const float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
        if (d < a.dim) {
          if (a.out_vector) {
            store4(out + d, y);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) store1(out + d + e, y[e]);
          }
        }
      } else {
        *reinterpret_cast<float4*>(part + r * kDP + d) = x;
      }
    }
    for (int r = tid; r < live_rows; r += kAttnThreads) {
      if (!whole) {
        part[rows * kDP + r] = row_m[r];
        part[rows * kDP + rows + r] = row_l[r];
      } else if (a.lse) {
        const int64_t gr = r0 + r;
        a.lse[(req.first + gr / a.group) * a.q_heads + int64_t(head) * a.group + gr % a.group] =
            row_l[r] == 0.0f ? -INFINITY : (row_m[r] + log2f(row_l[r])) * 0.6931471805599453f;
      }
    }
    if (!whole && pos == 0 && tid == 0)
      a.joins[cta] = make_int4(b, rt, head, int((at + cost - 1) / share) - cta + 1);
    __syncthreads();

    // ---- the next unit
    at += take;
    pos = 0;
    if (++head == a.kv_heads) {
      head = 0;
      if (++rt == row_tiles(req)) {
        rt = 0;
        if (at < end) {
          do req = attn_request(a, ++b);
          while (req.n == 0);
          cost = unit_tiles(req) + kAttnUnitCost;
        }
      }
    }
    // unused chunks of padded heads were overwritten by the join
    if (a.dim < kDP && at < end) {
      for (int i = tid; i < ring_bytes / 16; i += kAttnThreads)
        reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
  }
  if (flags && a.status) atomicOr(a.status, flags);
}

// ---------------------------------------------------------------- joining cut units
//
// Grid: (CTAs of the main kernel, row tiles of 8).  The unit that began in
// main CTA j and was cut there has its parts in slot 1 of j and slots 0 of the
// next CTAs; one warp joins one row.
template <int kDP, bool kSplit>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttnArgs a, const int rows) {
  using T = typename std::conditional<kSplit, float, uint16_t>::type;
  allow_dependent_launch();
  grid_dependency_wait();
  const int4 u = a.joins[blockIdx.x];
  if (u.w < 2) return;
  const AttnRequest req = attn_request(a, u.x);
  const int r = int(blockIdx.y) * 8 + (int(threadIdx.x) >> 5), lane = int(threadIdx.x) & 31;
  const int64_t gr = int64_t(u.y) * rows + r;
  if (r >= rows || gr >= int64_t(req.n) * a.group) return;
  const int64_t slot = int64_t(rows) * (kDP + 2);
  auto part = [&](int i) { return a.partial + (int64_t(blockIdx.x + i) * 2 + (i == 0)) * slot; };
  float top = -INFINITY, all = 0.0f;
  for (int i = lane; i < u.w; i += 32) top = fmaxf(top, part(i)[rows * kDP + r]);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  constexpr int kPer = kDP / 32;
  float x[kPer] = {};
  for (int i0 = 0; i0 < u.w; i0 += 32) {
    float f = 0.0f;
    if (i0 + lane < u.w) {
      const float m = part(i0 + lane)[rows * kDP + r], l = part(i0 + lane)[rows * kDP + rows + r];
      f = l == 0.0f ? 0.0f : m == -INFINITY ? 1.0f : exp2_approx(m - top);
      if (l != 0.0f) all += l * f;
    }
    const int count = min(32, u.w - i0);
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const float w = __shfl_sync(~0u, f, i);
      if (w != 0.0f) {
        const float* p = part(i0 + i) + r * kDP + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = fmaf(p[e], w, x[e]);
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(~0u, all, d);
  const float inv = all == 0.0f ? 0.0f : 1.0f / all;
  const int64_t token = req.first + gr / a.group, qh = int64_t(u.z) * a.group + gr % a.group;
  T* out = static_cast<T*>(a.out) + token * a.out_stride + qh * a.dim + lane * kPer;
  if (lane * kPer < a.dim) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) store1(out + e, x[e] * inv);
  }
  if (lane == 0 && a.lse)
    a.lse[token * a.q_heads + qh] = all == 0.0f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------- launch

constexpr int kAttnCtasPerSm = 2;

template <int kDP, int kNT, int kRG, int kType, bool kSplit>
cudaError_t attn_launch_shape(const AttnArgs& a, int dev, cudaStream_t st) {
  using S = AttnShape<kDP, kNT, kRG, kSplit>;
  LaunchShape ls;
  ls.smem = size_t(S::kSmem);
  // one wave: as many CTAs as fit at once (228 KB of shared memory per SM, 1 KB of it reserved per CTA)
  const int grid = device_sms(dev) * (2 * (S::kSmem + 1280) <= 228 * 1024 ? kAttnCtasPerSm : 1);
  cudaError_t err = prepare_kernel(reinterpret_cast<const void*>(&attention_kernel<kDP, kNT, kRG, kType, kSplit>), dev, ls);
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
  err = cudaLaunchKernelEx(&cfg, attention_kernel<kDP, kNT, kRG, kType, kSplit>, a);
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3(unsigned(grid), unsigned(S::kRows / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attention_join_kernel<kDP, kSplit>, a, S::kRows);
}

// The smallest row tile that holds `rows` rows of a key head: more row tiles
// of 8 per warp while the registers hold their sums (they share the codes'
// conversion), then more warps per team.
template <int kType, bool kSplit, int kDP>
cudaError_t attn_launch_dim(const AttnArgs& a, int64_t rows, int dev, cudaStream_t st) {
  if (rows <= 8) return attn_launch_shape<kDP, 1, 1, kType, kSplit>(a, dev, st);
  if (rows <= 16) return attn_launch_shape<kDP, 2, 1, kType, kSplit>(a, dev, st);
  if constexpr (kSplit || kDP == 256) {
    if (rows <= 32) return attn_launch_shape<kDP, 2, 2, kType, kSplit>(a, dev, st);
    return attn_launch_shape<kDP, 2, 4, kType, kSplit>(a, dev, st);
  } else {
    if (rows <= 24) return attn_launch_shape<kDP, 3, 1, kType, kSplit>(a, dev, st);
    if (rows <= 32) return attn_launch_shape<kDP, 4, 1, kType, kSplit>(a, dev, st);
    if (rows <= 48) return attn_launch_shape<kDP, 3, 2, kType, kSplit>(a, dev, st);
    if (rows <= 64) return attn_launch_shape<kDP, 4, 2, kType, kSplit>(a, dev, st);
    if (rows <= 96) return attn_launch_shape<kDP, 3, 4, kType, kSplit>(a, dev, st);
    return attn_launch_shape<kDP, 4, 4, kType, kSplit>(a, dev, st);
  }
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
