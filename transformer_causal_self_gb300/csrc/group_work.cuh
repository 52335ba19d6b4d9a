// How the grouped attention kernels (group_attn.cu, group_tc.cu) share out a batch.
//
// A segment is one KV head of one sequence and one block of its query rows; its work is its
// cache rows in tiles of `unit` rows.  The tiles of all segments, in order, are one line that is
// cut into equal ranges, one per CTA, whatever the sequences' lengths; a CTA's part of a
// segment is a piece.  Pieces are numbered CTA + segment: both only grow along the line, so a
// number occurs once and a segment's pieces are neighbours; partial results are stored by it.
// The line depends on the lengths, which only the device knows: every warp sums them up itself
// (a load per 32 sequences and a scan).  What the merge has to know of a segment is left by the
// CTA that begins it.  (32 bits: the host checks that the line is shorter than 2^31 tiles.)
#pragma once

#include "common.cuh"

namespace csattn {

// tma_load_3d for data that is not read again soon: its lines leave L2 first
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void tma_load_3d_once(void* smem_dst, const CUtensorMap* m,
                                                 uint64_t* bar, int x, int y, int z,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// a bulk copy of `bytes` (addresses and bytes multiples of 16)
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1], %2, [%3];" ::"r"(smem_u32(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Partial results over an e4m3 cache hold values of the output's size times 2^-kPartLog2: 4096 of
// them, as large as bf16 goes, add up within fp32, and bf16's least (2^-133) keeps four bits.
constexpr float kPartLog2 = 12.f, kPartScale = 4096.f;
// e with l in [2^(e-1), 2^e), at most 100 (also of infinities and NaN): 2^-e is a normal number
__device__ __forceinline__ int log2_above(float l) {
  return min(static_cast<int>((__float_as_uint(l) >> 23) & 0xffu) - 126, 100);
}

struct GroupLine {
  const int32_t* lens;
  int2* seg;            // [B * heads] of a segment: its first piece and their number
  int B, drafts, min_len, max_len;  // a length outside [min_len, max_len] has no work
  int unit, heads;                  // heads: segments per sequence (KV heads * row blocks)
  int tiles_per_cta;                // 0: such that the grid takes all, but
  int least_tiles;                  // no fewer than this
  __host__ __device__ __forceinline__ int tiles(int L) const {
    return L < min_len || L > max_len ? 0 : (L + drafts + unit - 1) / unit;
  }
};

// A CTA's position on the line.
struct GroupPiece {
  int b, head, t0, n;  // sequence, segment of it, first tile, tiles (0: no more)
  int L;               // its length
  int left, per;       // tiles of the CTA's range after this piece, and of every CTA's

  __device__ __forceinline__ int segment(const GroupLine& g) const { return b * g.heads + head; }
  // enter the segment at tile t0
  __device__ __forceinline__ void take(const GroupLine& g) {
    L = g.lens[b];
    n = min(left, g.tiles(L) - t0);
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
  // by one thread of the CTA, for each of its pieces
  __device__ __forceinline__ void leave_for_merge(const GroupLine& g) const {
    if (t0 != 0) return;
    const int s = segment(g);
    g.seg[s] = make_int2(static_cast<int>(blockIdx.x) + s, 1 + (g.tiles(L) - n + per - 1) / per);
  }
};

// The CTA's first piece (n = 0: none); every warp calls it by itself.  The first warp of the
// first CTA raises kStatusDeviceArg for a length that is not valid, unless that is `reported`.
__device__ __forceinline__ GroupPiece group_start(const GroupLine& g, uint32_t* status,
                                                  bool reported) {
  const int lane = threadIdx.x & 31;
  const bool tell = blockIdx.x == 0 && threadIdx.x < 32;
  unsigned sum = 0, first = 0;  // first: the tiles of sequence `lane`
  for (int b = lane; b < g.B; b += 32) {
    const int L = g.lens[b], t = g.tiles(L);
    sum += t;
    if (b == lane) first = t;
    if (tell && t == 0) {
      if ((L < g.min_len || L > g.max_len) && !reported) atomicOr(status, kStatusDeviceArg);
      for (int h = 0; h < g.heads; ++h) g.seg[b * g.heads + h] = make_int2(0, 0);
    }
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  const unsigned line = sum * g.heads;
  GroupPiece p{};
  p.per = g.tiles_per_cta > 0 ? g.tiles_per_cta
                              : max(g.least_tiles, (line + gridDim.x - 1) / gridDim.x);
  const unsigned w0 = static_cast<unsigned>(p.per) * blockIdx.x;
  if (line == 0 || w0 / p.per != blockIdx.x || w0 >= line) return p;  // (w0 may have wrapped)
  unsigned before = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    const unsigned t = b0 == 0 ? first : (b < g.B ? g.tiles(g.lens[b]) : 0);
    unsigned upto = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, (before + upto) * g.heads > w0);
    if (hit != 0u) {
      const int src = __ffs(hit) - 1;
      const unsigned tb = __shfl_sync(0xffffffffu, t, src);
      const unsigned in = w0 - (before + __shfl_sync(0xffffffffu, upto, src) - tb) * g.heads;
      p.b = b0 + src;
      p.head = in / tb;
      p.t0 = in - p.head * tb;
      p.left = p.per;
      p.take(g);
      return p;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}

}  // namespace csattn
