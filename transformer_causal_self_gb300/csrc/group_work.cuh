// How the grouped attention kernels (group_attn.cu, group_tc.cu) share out a batch.
//
// A segment is one KV head of one sequence and one block of its query rows; its work is its
// cache rows in tiles of `unit` rows.  The tiles of all segments, in order, are one line that is
// cut into equal ranges, one per CTA, whatever the sequences' lengths; a CTA's part of a
// segment is a piece.  Pieces are numbered CTA + segment: both only grow along the line, so a
// number occurs once and a segment's pieces are neighbours; partial results are stored by it.
// The line depends on the lengths, which only the device knows: every CTA sums them up itself
// (one load per sequence and a scan), and the first leaves the sums for the merge.
#pragma once

#include "common.cuh"

namespace csattn {

struct GroupLine {
  const int32_t* lens;
  long long* prefix;  // [B + 1]: tiles before sequence b, and of all
  int B, drafts, min_len, max_len;  // a length outside [min_len, max_len] has no work
  int unit, heads;                  // heads: segments per sequence (KV heads * row blocks)
  int tiles_per_cta;                // 0: such that the grid takes all
  __host__ __device__ __forceinline__ int tiles(int L) const {
    return L < min_len || L > max_len ? 0 : (L + drafts + unit - 1) / unit;
  }
};

// A CTA's position on the line.
struct GroupPiece {
  int b, head, t0, n;   // sequence, segment of it, first tile, tiles (0: no more)
  int L;                // its length
  long long left;       // tiles of the CTA's range after this piece

  __device__ __forceinline__ int segment(const GroupLine& g) const { return b * g.heads + head; }
  // enter the segment at tile t0
  __device__ __forceinline__ void take(const GroupLine& g) {
    L = g.lens[b];
    const int have = g.tiles(L) - t0;
    n = left < have ? static_cast<int>(left) : have;
    left -= n;
  }
  __device__ __forceinline__ void next(const GroupLine& g) {
    n = 0;
    if (left <= 0) return;
    t0 = 0;
    if (++head == g.heads) {
      head = 0;
      do ++b;
      while (b < g.B && g.tiles(g.lens[b]) == 0);
      if (b >= g.B) return;  // (the range ends with the line)
    }
    take(g);
  }
};

constexpr int kLineSmem = 8 * 33 + 32;  // bytes of shared memory that group_start needs

// The CTA's first piece (n = 0: none).  All threads call it with the same arguments; a length
// that is not valid raises kStatusDeviceArg unless it is `reported`.
__device__ __forceinline__ GroupPiece group_start(const GroupLine& g, uint8_t* smem,
                                                  uint32_t* status, int reported) {
  long long* s_sum = reinterpret_cast<long long*>(smem);  // [33]
  long long* s_left = s_sum + 33;
  int* s_at = reinterpret_cast<int*>(s_left + 1);         // b, head, t0
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int per = (g.B + nt - 1) / nt, b0 = min(g.B, tid * per), b1 = min(g.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = g.lens[b], t = g.tiles(L);
    if (blockIdx.x == 0 && (L < g.min_len || L > g.max_len) && L != reported)
      atomicOr(status, kStatusDeviceArg);
    mine += t;
  }
  long long sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) s_sum[warp] = sum;
  if (tid == 0) *s_left = 0;
  __syncthreads();
  long long before = sum - mine, all = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += s_sum[w];
    all += s_sum[w];
  }
  const long long line = all * g.heads;
  const long long per_cta =
      g.tiles_per_cta > 0 ? g.tiles_per_cta : (line + gridDim.x - 1) / gridDim.x;
  const long long w0 = per_cta * blockIdx.x;
  if (blockIdx.x == 0) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      g.prefix[b] = at;
      at += g.tiles(g.lens[b]);
    }
    if (tid == 0) g.prefix[g.B] = all;
  }
  if (w0 < line && before * g.heads <= w0 && w0 < (before + mine) * g.heads) {
    long long at = before;
    int b = b0, t = 0;
    for (;; ++b) {
      t = g.tiles(g.lens[b]);
      if (w0 < (at + t) * g.heads) break;
      at += t;
    }
    const long long in = w0 - at * g.heads;
    s_at[0] = b;
    s_at[1] = static_cast<int>(in / t);
    s_at[2] = static_cast<int>(in % t);
    *s_left = per_cta;
  }
  __syncthreads();
  GroupPiece p{};
  p.left = *s_left;
  if (p.left > 0) {
    p.b = s_at[0];
    p.head = s_at[1];
    p.t0 = s_at[2];
    p.take(g);
  }
  return p;
}

}  // namespace csattn
