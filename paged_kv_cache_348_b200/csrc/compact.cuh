// compact.cuh -- the kept tokens of a sequence moved to the front of its pages.
//
// Row i of the new sequence is row keep[i] of the old one (keep ascending), for every kv
// head of every layer's K and V pool.  Old rows are read through the source table, new ones
// written through the destination table; the two may name the same blocks (in place).
//
// What bounds it: every kept row is read and written once, nothing is computed, so HBM.  A
// row is 64 to 256 bytes at an arbitrary place, so the loads are 16 bytes a lane with a
// row's lanes side by side (whole 32-byte sectors) and what hides their latency is bytes in
// flight: kU = 8 loads a thread and 4 CTAs an SM.  16 sequences x 8 heads x 4 layers, 1024
// rows of 256 bytes each: 89 us, 6.0 TB/s; one sequence and layer, 513 rows: 7.1 us.
//
// In place, writing new rows [i0, i1) overwrites old rows that only new rows j <= keep[j] <
// i1 take.  So one CTA walks a (sequence, kv head, pool) list front to back in chunks and
// the one condition is that all loads of a chunk are done before its first store: one
// barrier a chunk.  Lists of different sequences, heads, layers and pools share no byte that
// is written, so they need no order.
#pragma once
#include <cstdint>

#include "decode.cuh"
#include "kv_ops.cuh"

namespace pkv {

constexpr int DEV_BAD_KEEP = 0x20;
constexpr int kCompactThreads = 256;
constexpr int kScaledLayersPerLaunch = 64;        // pointers of this many layers a launch

struct CompactArgs {
  const int32_t* src_tables;      // [num_seqs][src_width]
  const int32_t* dst_tables;      // [num_seqs][dst_width]
  const int32_t* context_lens;    // [num_seqs]
  const int32_t* keep;            // [layer][seq][head][max_keep] by the strides below
  const int32_t* keep_lens;       // [num_seqs]
  int32_t* status;                // nullable
  int src_width, dst_width, num_kv_heads, block_size, num_blocks, max_keep;
  int bs_log;                                     // block_size is a power of two
  long long keep_layer, keep_seq, keep_head;      // strides in elements (0: shared)
};

struct ScaledLayerPtrs {
  uint4* k[kScaledLayersPerLaunch];
  uint4* v[kScaledLayersPerLaunch];
  float* ks[kScaledLayersPerLaunch];
  float* vs[kScaledLayersPerLaunch];
};

// Kept rows of sequence s, and its old length, both clamped to what the tables hold.
__device__ __forceinline__ int compact_rows(const CompactArgs& a, int s, int& ctx, bool report) {
  ctx = clamp_ctx(a.context_lens[s], a.src_width * a.block_size, report ? a.status : nullptr);
  int n = a.keep_lens[s];
  const int cap = min(a.max_keep, a.dst_width * a.block_size);
  if (n < 0 || n > cap) {
    if (report && a.status) atomicOr(a.status, DEV_BAD_KEEP);
    n = n < 0 ? 0 : cap;
  }
  return n;
}

// Old and new row (block, kv head, offset) of kept row i; false (and a status bit) when the
// position or a block id is out of range.
__device__ __forceinline__ bool compact_row(const CompactArgs& a, const int32_t* keep, int s,
                                            int h, int ctx, int i, int& src, int& dst) {
  const int t = __ldg(keep + i);
  if (t < 0 || t >= ctx) {
    if (a.status) atomicOr(a.status, DEV_BAD_KEEP);
    return false;
  }
  const int lg = a.bs_log, in = a.block_size - 1;
  const int sb = __ldg(a.src_tables + (long long)s * a.src_width + (t >> lg));
  const int db = __ldg(a.dst_tables + (long long)s * a.dst_width + (i >> lg));
  if ((unsigned)sb >= (unsigned)a.num_blocks || (unsigned)db >= (unsigned)a.num_blocks) {
    if (a.status) atomicOr(a.status, DEV_BAD_BLOCK_ID);
    return false;
  }
  // (a pool has fewer than 2^31 rows)
  src = ((sb * a.num_kv_heads + h) << lg) + (t & in);
  dst = ((db * a.num_kv_heads + h) << lg) + (i & in);
  return true;
}

// Rows moved byte for byte (16-bit pools, 8-bit pools with one scale per pool).  CPR: 16-byte
// pieces per row.  grid = (sequences * kv heads, layers * 2 pools).
template <int CPR>
__global__ void __launch_bounds__(kCompactThreads, 4)
    pa_compact_kernel(const __grid_constant__ LayerPtrs P, const CompactArgs a, int layer0) {
  constexpr int kU = 8;                                   // 16-byte loads a thread and chunk
  constexpr int kRows = kCompactThreads * kU / CPR;       // rows of a chunk
  constexpr int kPer = (kRows + kCompactThreads - 1) / kCompactThreads;
  // places of three chunks (-1: nothing to move): chunk c + 1's are found while the slowest
  // warp may still be storing chunk c - 1
  __shared__ int src_s[3][kRows], dst_s[3][kRows];
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
  const int layer = blockIdx.y >> 1, pool = blockIdx.y & 1;
  const int tid = threadIdx.x;
  int ctx;
  const int n = compact_rows(a, s, ctx, h == 0 && blockIdx.y == 0 && tid == 0);
  const int32_t* keep = a.keep + (layer0 + layer) * a.keep_layer + s * a.keep_seq + h * a.keep_head;
  uint4* base = pool ? P.v[layer] : P.k[layer];
  auto places = [&](int c) {                              // rows of chunk c -> src_s, dst_s
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int r = tid + k * kCompactThreads, i = c * kRows + r;
      if (r >= kRows) break;
      int src = -1, dst = -1;
      if (i < n && (!compact_row(a, keep, s, h, ctx, i, src, dst) || src == dst)) src = dst = -1;
      src_s[c % 3][r] = src;
      dst_s[c % 3][r] = dst;
    }
  };
  const int nc = (n + kRows - 1) / kRows;
  if (nc) places(0);
  __syncthreads();
  for (int c = 0; c < nc; ++c) {
    uint4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int e = u * kCompactThreads + tid;
      const int src = src_s[c % 3][e / CPR];
      if (src >= 0) x[u] = *(base + (long long)src * CPR + e % CPR);
    }
    if (c + 1 < nc) places(c + 1);
    __syncthreads();                                      // every load of the chunk is done
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int e = u * kCompactThreads + tid;
      const int dst = dst_s[c % 3][e / CPR];
      if (dst >= 0) *(base + (long long)dst * CPR + e % CPR) = x[u];
    }
  }
}

// 8-bit (E4M3) pools with per-(block, kv head) scales: a kept row's values are scale * code of
// its old block; a new block's scale is the one that its first moved row fixes (e4m3_block_scale
// of that row's largest magnitude, the rule of the append; the row at offset 0 unless that one
// has to be left out), and every row of the block is quantised with it.  The powers of two make value / scale exact, so a code changes only
// where the scale grew past its low bits or shrank below its magnitude.
//
// Half the bytes of a 16-bit row and a conversion both ways: what bounds it is the latency of
// a chunk (place, row, block scale, barrier, store): 5.4 of a warp's 12.4 cycles an instruction
// are the barrier's.  So a thread has few rows at a time (kU = 2: 64 registers, 4 CTAs an SM), the next chunk's rows are loaded before this one's are
// stored (reading ahead is always safe: rows still to be stored over lie below every position
// that is still to be read), block and offset come by shift and mask, and only the rows that
// fix a scale search their maximum.  16 sequences x 8 heads x 2 layers of 700 rows: 31.3 us,
// 2.8 TB/s (57.0 with kU = 4 and neither of these; the bytes alone take 13.6).  Taking the rows
// that fix a scale from what is moved, not from the offset, is 0.9 us of it.
template <int CPR>
__global__ void __launch_bounds__(kCompactThreads, 4)
    pa_compact_e4m3_bs_kernel(const __grid_constant__ ScaledLayerPtrs P, const CompactArgs a,
                              int layer0) {
  constexpr int kU = 2;
  constexpr int kRows = kCompactThreads * kU / CPR;       // a multiple of every block size
  static_assert(kRows % 32 == 0 && kRows <= kCompactThreads, "whole blocks, one place a thread");
  // places of four chunks: chunk c + 2's are found while the slowest warp may still be storing
  // chunk c - 1.  src_s: twice the old row, plus one where the row fixes its block's scale (a pool
  // has fewer than 2^31 rows)
  __shared__ uint32_t src_s[4][kRows];
  __shared__ int dst_s[4][kRows];
  constexpr uint32_t kNone = 0xffffffffu;                 // src_s: nothing to move
  __shared__ float new_s[2][kRows];                       // a chunk's new block scales
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
  const int layer = blockIdx.y >> 1, pool = blockIdx.y & 1;
  const int tid = threadIdx.x, lg = a.bs_log, in = a.block_size - 1;
  int ctx;
  const int n = compact_rows(a, s, ctx, h == 0 && blockIdx.y == 0 && tid == 0);
  const int32_t* keep = a.keep + (layer0 + layer) * a.keep_layer + s * a.keep_seq + h * a.keep_head;
  uint4* base = pool ? P.v[layer] : P.k[layer];
  float* scales = pool ? P.vs[layer] : P.ks[layer];
  const int nc = (n + kRows - 1) / kRows;
  auto places = [&](int c) {
    if (c < nc && tid < kRows) {
      const int i = c * kRows + tid;
      int src = -1, dst = -1;
      if (i < n && !compact_row(a, keep, s, h, ctx, i, src, dst)) src = dst = -1;
      // the first row of each block that is moved at all: no moved row between its block's
      // start and it (whole warps: kRows is a multiple of 32, and so is no block wider)
      const int r = tid & 31;
      const uint32_t moved = __ballot_sync(0xffffffffu, src >= 0);
      const uint32_t before = ((1u << r) - 1u) & ~((1u << (r & ~in)) - 1u);
      src_s[c & 3][tid] = src < 0 ? kNone : 2u * (uint32_t)src + !(moved & before);
      dst_s[c & 3][tid] = dst;
    }
  };
  struct Piece {
    uint4 x;
    float sc;
    bool lead;
  };
  auto load = [&](int c, Piece (&p)[kU]) {
    if (c >= nc) return;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int e = u * kCompactThreads + tid;
      const uint32_t src2 = src_s[c & 3][e / CPR], src = src2 >> 1;
      p[u].x = make_uint4(0u, 0u, 0u, 0u);
      p[u].sc = 1.f;
      p[u].lead = src2 != kNone && (src2 & 1u);
      if (src2 != kNone) {
        p[u].x = *(base + (long long)src * CPR + e % CPR);
        p[u].sc = scales[src >> lg];                      // = block * heads + head
      }
    }
  };
  places(0);
  places(1);
  __syncthreads();
  Piece now[kU], nxt[kU];
  load(0, now);
  for (int c = 0; c < nc; ++c) {
    load(c + 1, nxt);
    places(c + 2);
    // the first moved row of each new block fixes its scale
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = (u * kCompactThreads + tid) / CPR;
      const bool first = now[u].lead;
      if (!__any_sync(0xffffffffu, first)) continue;
      const uint32_t w[4] = {now[u].x.x, now[u].x.y, now[u].x.z, now[u].x.w};
      float am = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2x2(w[k], lo, hi);
        const float2 f0 = unpack2<__half>(lo), f1 = unpack2<__half>(hi);
        am = fmaxf(am, fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))));
      }
#pragma unroll
      for (int o = 1; o < CPR; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      if (first && tid % CPR == 0) new_s[c & 1][r >> lg] = e4m3_block_scale(am * now[u].sc);
    }
    __syncthreads();                                      // loads done, new scales known
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int e = u * kCompactThreads + tid;
      const int r = e / CPR;
      const int dst = dst_s[c & 3][r];
      if (dst >= 0) {
        const float ns = new_s[c & 1][r >> lg];
        const float inv = 1.f / ns;                       // a power of two: exact
        const uint32_t w[4] = {now[u].x.x, now[u].x.y, now[u].x.z, now[u].x.w};
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t lo, hi;
          e4m3x4_to_f16x2x2(w[k], lo, hi);
          const float2 f0 = unpack2<__half>(lo), f1 = unpack2<__half>(hi);
          const float sc = now[u].sc;
          q[k] = f32x2_to_e4m3x2(f0.x * sc * inv, f0.y * sc * inv) |
                 (f32x2_to_e4m3x2(f1.x * sc * inv, f1.y * sc * inv) << 16);
        }
        *(base + (long long)dst * CPR + e % CPR) = make_uint4(q[0], q[1], q[2], q[3]);
        if (now[u].lead && e % CPR == 0) scales[dst >> lg] = ns;
      }
      now[u] = nxt[u];
    }
  }
}

}  // namespace pkv
