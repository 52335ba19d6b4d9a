// Decode over a 4-bit cache (fp4.cuh): one new query per sequence and head.
//
// out = softmax(q K^T scale) V with K and V in e2m1 times a scale per 16 channels.  All Hq / Hkv
// query rows of a KV head read the same cache rows, so they are one side of a matrix product and
// a row is read from HBM and taken to f16 once for 8 * NT of them.  A CTA:
//   warp 4      producer: tiles of 64, 128 or 192 K and V rows and their scale bytes into a ring by
//               TMA, and a piece's queries, as f16, behind its first tile
//   warps 0..3  RG groups of 16 cache rows each per tile, by mma.sync m16n8k16 with the cache rows
//               (then the channels) on the side of 16 and the query rows on the side of 8:
//               S^T = K Q^T, then O^T += V^T P^T, softmax statistics in fp32 between the two;
//               each leaves a partial result of its own per piece.
// CTAs, a wave of them, take equal ranges of all the tiles (group_work.cuh); the partial results
// are merged by group_merge_kernel.
//
// The operands: K and V enter as x4 * s, which f16 holds exactly (one conversion and one product
// for two of them); q is taken to f16 by a power of two per row (query_to_f16: exact but for
// channels below 2^-31 of the largest, which are off by 2^-39 of it); the weights are 2^(x - m)
// with m = the running maximum - 7, rounded to f16: to 11 bits, and below 2^-21 of the largest,
// where f16's subnormals begin, to steps of 2^-31 of it, because bf16's 8 bits would cost every
// output 2^-9, and the rest of a weight in a second product half as many mma again.  Their sum is
// taken ahead of that rounding.  Sums are fp32.  The maximum is raised only when a score exceeds it
// by 2^8, and only then do the lanes exchange theirs.
//
// The index of a product's sum may run over the channels (the rows) in any order that both sides
// share, and its rows may be any 16 cache rows.  So a lane takes a row's channels as whole words
// of the cache: for S^T lane (g, j) the j-th quarter of row perm(g), for O^T the g-th eighth of
// rows perm(2j), perm(2j + 1); there two rows' nibbles are paired in the words before they are
// taken apart, four instructions for 16 values.  perm keeps both kinds of loads free of bank
// conflicts.
//
// What bounds it (128 channels, 4 query heads per KV head): latency.  A group of 16 rows of K and V
// is 284 instructions, 64 of them conversions, 64 products with scales and 16 mma; in a loop of
// their own these three kinds take 260 cycles of a scheduler (the conversions alone 200, the mma
// 187), and with all else a group takes 450.  No unit is near its rate (issue slots 54 %, ALU
// 46 %, tensor pipe 25 %, HBM 58 %): what is left is the chain copy, conversion, scale, mma,
// maximum, exponentials, turn, conversion, scale, mma, of which three warps per scheduler do not
// cover all.
// 64 sequences of 512 to 8192 rows take 64.8 us for 322 MB (5.0 TB/s; the 8-bit cache 93 us), 4
// of 30000 to 32768 32.1 us for 145 MB, of which 5 us are two launches, the first tile and the
// merge.  With the copies alone these take 57.1 and 27.0 us, with the products alone 60.6 and
// 31.9.  16-row pages take longer, 16 sequences of 4000 to 8000 rows 33.0 us (64-row pages 27.4,
// contiguous 25.7); their copies alone take 25.6 against 21.4, which is 4.2 of those 7.3 us, and
// where the rest goes was not found.  Without gain: more warps with
// fewer registers (four CTAs), two sums per score, the next tile's scores before this one's
// values, K and V in stages of their own, tile rows of 128 bytes, all copies by the lanes (the
// 16-row pages 37.4 us), rarer polling.
#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "group_work.cuh"
#include "internal.h"

namespace csattn {
namespace {

constexpr int NW = 4;  // compute warps, RG groups of 16 rows of a tile each
constexpr int kThreads = 32 * (NW + 1);
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 100000000ull;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kWeightLog2 = 7.0f;  // weights are at most 2^(8 + 7) < 65504

template <int D, int NT, int RG>
struct Cfg {
  static constexpr int KT = 16 * NW * RG;  // cache rows per tile
  static constexpr int ROW = D / 2;
  static constexpr int SROW = D / 16;  // scale bytes of a row
  static constexpr int TILE = KT * ROW;
  static constexpr int STAGE = 2 * TILE;
  static constexpr int CODES = 2 * KT * SROW;       // keys' scales, values' scales
  static constexpr int ROWS = 8 * NT;               // query rows of a CTA
  static constexpr int QS = 2 * D + 16;             // bytes between query rows
  static constexpr int CTAS = decode_fp4_ctas(D, ROWS);
  static constexpr int Q_BYTES = ROWS * QS;         // twice: the next piece's go to the other
  static constexpr int BARS = 192;
  static constexpr int REST = 1024 + 2 * Q_BYTES + BARS + 2 * ROWS * 4;
  // the ring: what the resident CTAs have room for (1 KB of an SM's 228 goes with each)
  static constexpr int ROOM = (228 * 1024 / CTAS - 1024 - REST) / (STAGE + CODES);
  static constexpr int NS = ROOM < 6 ? ROOM : 6;
  static constexpr int RING = NS * STAGE;
  static constexpr int SMEM = REST + RING + NS * CODES;
  static_assert(NS >= 2 && 8 * (2 * NS + 4) + 4 <= BARS, "barriers");
};

struct Params {
  const __nv_bfloat16* q;
  GroupLine line;
  CacheRows rows;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int lost;          // arrivals that the queries' barrier waits for and nothing makes (selftest)
  int box_rows;
  int nbox, batch;   // boxes of a tile; tiles whose boxes' pages a warp's lanes read at once
  int lanes_tile;    // lane * lanes_tile >> 16 is lane / nbox
  int box_shift;     // box_rows in the copies by lanes is 2^box_shift (or one box: all its bits)
  bool code_copies;  // scale bytes come by bulk copies, a box's at a time; else by the lanes'
  float* part_o;
  float* part_ml;
  uint32_t* status;
  int rep, rblocks, part_rows;
  float scale_log2;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// max over the eight lanes that hold one query row's column
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}

// N bytes to shared memory without a register between; zeros where `there` is false
template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src),
               "n"(N), "r"(there ? N : 0)
               : "memory");
}

// The cache row (of eight) that fragment row m stands for.  128 channels: rows of 64 bytes, whose
// four chunks TMA's 64-byte swizzle permutes by (row / 2) % 4.  The quarters of rows perm(2p) and
// perm(2p + 1), loaded together, cover all banks as one row is even and one odd; the eighths 0..3
// of rows perm(0), perm(2), .. = 0 3 4 7 do, as their chunks are {0,1} ^ row / 2.
// 64 channels: rows of 32 bytes, not swizzled; loaded together are rows that differ modulo 4.
template <int D>
__device__ __forceinline__ int perm(int m) {
  if constexpr (D == 128) return m ^ ((m >> 1) & 1);
  // 0 2 1 3 6 4 7 5
  return (0x57463120u >> (4 * m)) & 7u;
}

template <int D, int NT, int RG, int H>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT, RG>::CTAS)
    decode_fp4_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D, NT, RG>;
  constexpr int KT = C::KT;
  using Scales = std::conditional_t<D == 128, uint2, uint32_t>;  // a row's scale bytes
  constexpr int NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* s_codes = smem + C::RING;
  uint8_t* s_q = s_codes + NS * C::CODES;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_q + 2 * C::Q_BYTES);
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;   // [2]: a piece's queries in buffer piece % 2
  uint64_t* q_empty = q_full + 2;  // [2]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(q_empty + 2);
  float* s_qf = reinterpret_cast<float*>(s_q + 2 * C::Q_BYTES + C::BARS);  // [2][ROWS]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // let the merge be scheduled once every CTA has started; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], p.code_copies ? 1 : 33);
      mbar_init(&empty[s], NW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1 + p.lost);
      mbar_init(&q_empty[i], NW);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  GroupPiece pc = group_start(p.line, p.status, false);
  if (pc.n == 0) return;
  __syncthreads();

  if (warp == NW) {
    // ------------------------------------------------------------ producer
    // lane i copies box i of a tile (paged: boxes of box_rows rows never cross a page; a
    // box past the sequence, or a page index outside the pool, which is reported, reads
    // zeros: its plane is past the tensor map).  Lane 0 waits and arms the stage first.
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    // (the kernel before may have written the cache's rows by plain stores)
    asm volatile("fence.proxy.async.global;" ::: "memory");
    const uint64_t once = evict_first_policy();
    const CacheRows& R = p.rows;
    const int nbox = p.nbox, r0 = lane * p.box_rows;
    int issued = 0, s = 0, phase = 1;  // (a stage's first use waits for nothing: phase 1 is over)
    // The pages of `batch` tiles' boxes from tile t on, one per lane (-1: past the sequence), and
    // the rows in them: a batch of the piece is read while the one before it is used.  (Each tile's
    // one tile ahead: 64 sequences of 512 to 8192 rows 66.5 against 63.8 us.)
    const int lane_tile = lane * p.lanes_tile >> 16;
    auto pages_of = [&](const GroupPiece& pc, int t, int& prow) {
      const int row = (pc.t0 + t) * KT + lane_tile * KT + (lane - lane_tile * nbox) * p.box_rows;
      prow = 0;
      if (lane_tile >= min(p.batch, pc.n - t) || row >= pc.L) return -1;
      const int at = row / R.page_size;
      prow = row - at * R.page_size;
      return R.block_table[static_cast<size_t>(pc.b) * R.max_pages + at];
    };
    // The queries of a piece: D/16 lanes per row, 16 channels each, read ahead of the piece's
    // first tile and staged behind it.
    constexpr int G = D / 16, PASSES = C::ROWS * G / 32;
    const int qc = lane % G;
    uint4 q_lo[PASSES], q_hi[PASSES];
    auto load_queries = [&](const GroupPiece& pc) {
      const int kvh = pc.head / p.rblocks;
      const int first = (pc.head - kvh * p.rblocks) * C::ROWS;
      const size_t at = (static_cast<size_t>(pc.b) * R.Hkv + kvh) * p.rep;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int col = 32 / G * i + lane / G, row = first + (H == 2 ? col : col / 2);
        q_lo[i] = q_hi[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < p.rep && (H == 2 || col % 2 == 0)) {
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (at + row) * D + 16 * qc);
          q_lo[i] = src[0];
          q_hi[i] = src[1];
        }
      }
    };
    auto stage_queries = [&](int piece) {
      const int buf = piece & 1;
      bool room = true;
      if (piece >= 2 && lane == 0)
        room = ctl_wait(&q_empty[buf], ((piece >> 1) - 1) & 1, abort_flag, p.status, kWaitNs);
      if (!__all_sync(0xffffffffu, room)) return false;
      const float none[8] = {};
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = 32 / G * i + lane / G;
        uint8_t* dst = s_q + buf * C::Q_BYTES + r * C::QS + 32 * qc;
        const float factor = query_to_f16<G>(q_lo[i], q_hi[i], 0, none, none);
        if (qc == 0) s_qf[buf * C::ROWS + r] = factor * p.scale_log2;
        *reinterpret_cast<uint4*>(dst) = q_lo[i];
        *reinterpret_cast<uint4*>(dst + 16) = q_hi[i];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[buf]);
      return true;
    };
    bool ok = true;
    for (int piece = 0; pc.n > 0 && ok; pc.next(p.line), ++piece) {
      const int b = pc.b, kvh = pc.head / p.rblocks, total = pc.L;
      load_queries(pc);
      int rows_now = 0, rows_next = 0, pages_next = -1, batch0 = 0;
      int pages_now = R.block_table != nullptr ? pages_of(pc, 0, rows_now) : -1;
      for (int t = 0; t < pc.n; ++t) {
        const int row0 = (pc.t0 + t) * KT;
        uint8_t* codes = s_codes + s * C::CODES;
        int plane = b * R.Hkv + kvh, prow = row0;
        int code_rows = min(KT, R.Lmax - row0);  // rows of the lane's box whose scales are copied
        bool lost = false;                       // its page is outside the pool
        if (R.block_table != nullptr) {
          const bool in = lane < nbox && row0 + r0 < total;
          if (t - batch0 == p.batch) {
            batch0 = t;
            pages_now = pages_next;
            rows_now = rows_next;
          }
          const int from = (t - batch0) * nbox + lane;
          const int page = __shfl_sync(0xffffffffu, pages_now, from);
          prow = __shfl_sync(0xffffffffu, rows_now, from);
          lost = in && (page < 0 || page >= R.num_pages);
          plane = in && !lost ? page * R.Hkv + kvh : R.num_pages * R.Hkv;
          code_rows = in && !lost ? p.box_rows : 0;
          if (lost) atomicOr(p.status, kStatusDeviceArg);
        }
        if (lane >= nbox) code_rows = 0;
        uint32_t bytes = C::STAGE;
        if (p.code_copies)
          bytes += 2 * C::SROW * __reduce_add_sync(0xffffffffu, static_cast<unsigned>(code_rows));
        bool room = true;
        if (lane == 0) room = ctl_wait(&empty[s], phase, abort_flag, p.status, kWaitNs);
        if (!__all_sync(0xffffffffu, room)) {
          ok = false;
          break;
        }
        if (lost && p.code_copies) {  // the rows read as zeros: their scales have to be numbers
          for (int i = 0; i < p.box_rows * C::SROW; i += 16) {
            *reinterpret_cast<uint4*>(codes + r0 * C::SROW + i) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(codes + (KT + r0) * C::SROW + i) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
        __syncwarp();
        if (lane < nbox) {
          uint8_t* kd = smem + s * C::STAGE + r0 * C::ROW;
          tma_load_3d_once(kd, &tm_k, &full[s], 0, prow, plane, once);
          tma_load_3d_once(kd + C::TILE, &tm_v, &full[s], 0, prow, plane, once);
          if (p.code_copies && code_rows > 0) {
            const size_t at =
                static_cast<size_t>(plane) * (R.block_table != nullptr ? R.page_size : R.Lmax) +
                prow;
            bulk_load(codes + r0 * C::SROW, p.k_scale + at * C::SROW, code_rows * C::SROW,
                      &full[s]);
            bulk_load(codes + (KT + r0) * C::SROW, p.v_scale + at * C::SROW, code_rows * C::SROW,
                      &full[s]);
          }
        }
        if (!p.code_copies) {
          const bool paged = R.block_table != nullptr;
          const int per = paged ? 16 / C::SROW : 1;  // rows of a copy
          for (int i = 0; i * 32 * per < KT; ++i) {
            const int r = per * (lane + 32 * i), box = min(r, KT - 1) >> p.box_shift;
            const int in_box = r - box * p.box_rows;
            const bool there = __shfl_sync(0xffffffffu, code_rows, box) > in_box;
            const long long at =
                static_cast<long long>(__shfl_sync(0xffffffffu, plane, box)) *
                    (paged ? R.page_size : R.Lmax) +
                __shfl_sync(0xffffffffu, prow, box) + in_box;
            const size_t from = there ? at * C::SROW : 0;
            if (r >= KT) continue;
            if (paged) {
              copy_async<16>(codes + r * C::SROW, p.k_scale + from, there);
              copy_async<16>(codes + (KT + r) * C::SROW, p.v_scale + from, there);
            } else {
              copy_async<C::SROW>(codes + r * C::SROW, p.k_scale + from, there);
              copy_async<C::SROW>(codes + (KT + r) * C::SROW, p.v_scale + from, there);
            }
          }
          // arrives when this lane's copies are there
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_u32(&full[s]))
                       : "memory");
        }
        __syncwarp();
        ++issued;
        // Behind the first tile: the queries are there by the time that it has been asked for.
        // (Behind as many as find room they came late: 1 x 1000 rows 7.8 against 7.3 us, 1 x 16000
        // 14.8 against 13.9, and the batches above the same.)
        if (t == 0) ok = stage_queries(piece);
        if (t == batch0 && R.block_table != nullptr)
          pages_next = pages_of(pc, t + p.batch, rows_next);
        if (++s == NS) s = 0, phase ^= 1;
        if (!ok) break;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0 && *abort_flag) {
      const int first = issued > NS ? issued - NS : 0;
      for (int t = first; t < issued; ++t)
        mbar_wait(&full[t % NS], (t / NS) & 1, nullptr, p.status, kDrainNs);
    }
    return;
  }

  // ---------------------------------------------------------------- compute warps
  constexpr int KW = D / 32;  // words of a row that a lane has for S^T (a quarter)
  constexpr int VW = D / 64;  // for O^T (an eighth)
  const int g = lane >> 2, j = lane & 3;
  const int cq = 2 * j;  // fragment columns cq and cq + 1, of which H have query rows
  const uint32_t smem_base = smem_u32(smem), codes_base = smem_u32(s_codes);
  const int wrow = 16 * RG * warp;  // first row of the warp in a tile
  // a lane's byte offsets within a tile, for the first 16 rows
  const int kr = wrow + perm<D>(g);
  const int va = wrow + perm<D>(2 * j), vb = wrow + perm<D>(2 * j + 1);
  auto chunk = [](int row, int byte) {
    return D == 128 ? row * 64 + (byte ^ (((row >> 1) & 3) << 4)) : row * 32 + byte;
  };
  const uint32_t k_off = chunk(kr, 4 * KW * j);
  const uint32_t va_off = chunk(va, 4 * VW * g), vb_off = chunk(vb, 4 * VW * g);
  const uint32_t ks_off = kr * C::SROW + (D / 64) * j;
  const uint32_t vs_a = (KT + va) * C::SROW + (D == 128 ? g : g >> 1);
  const uint32_t vs_b = (KT + vb) * C::SROW + (D == 128 ? g : g >> 1);
  bool ok = true;
  int s = 0, phase = 0;  // the ring's next stage, and which of its uses
  for (int piece = 0; pc.n > 0; pc.next(p.line), ++piece) {
    const int kvh = pc.head / p.rblocks;
    const int row_base = (pc.head - kvh * p.rblocks) * C::ROWS;  // first query row
    const int k_begin = pc.t0 * KT, ntiles = pc.n;
    const int k_end = min(pc.L, k_begin + ntiles * KT);

    ok = __all_sync(0xffffffffu, ctl_wait(&q_full[piece & 1], (piece >> 1) & 1, abort_flag,
                                          p.status, kWaitNs));
    if (!ok) break;
    // the lane's quarter of its query row, in pairs of channels
    uint32_t qb[NT][D / 8];
    float qf[NT][H];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t q_addr =
          smem_u32(s_q) + (piece & 1) * C::Q_BYTES + (8 * n + g) * C::QS + (D / 2) * j;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t w[4];
        lds<4>(q_addr + 16 * i, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) qb[n][4 * i + e] = w[e];
      }
#pragma unroll
      for (int h = 0; h < H; ++h)  // (not 0: a masked score times it stays -inf)
        qf[n][h] = fmaxf(s_qf[(piece & 1) * C::ROWS + 8 * n + cq + h], 0x1p-120f);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_empty[piece & 1]);

    float o[D / 16][NT][4];
    float m_ref[NT][H], l_part[NT][H];  // m_ref: the maximum - kWeightLog2
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[c][n][0] = o[c][n][1] = o[c][n][2] = o[c][n][3] = 0.f;
#pragma unroll
      for (int h = 0; h < H; ++h) m_ref[n][h] = -INFINITY, l_part[n][h] = 0.f;
    }

    bool unset = true;  // some query row has no maximum yet
    for (int t = 0; t < ntiles && ok; ++t) {
      if (!__all_sync(0xffffffffu, ctl_wait(&full[s], phase, abort_flag, p.status, kWaitNs))) {
        ok = false;
        break;
      }
      const uint32_t kbase = smem_base + s * C::STAGE, vbase = kbase + C::TILE;
      const uint32_t cbase = codes_base + s * C::CODES;
      const int key0 = k_begin + t * KT + wrow;  // first cache row of the warp
      // S^T: rows perm(g) and perm(g) + 8 of each group of 16
      float sc[RG][NT][4];
#pragma unroll
      for (int rg = 0; rg < RG; ++rg) {
        uint32_t ka[KW], kb[KW];
        lds<KW>(kbase + k_off + (16 * rg) * C::ROW, ka);
        lds<KW>(kbase + k_off + (16 * rg + 8) * C::ROW, kb);
        uint32_t sa[D / 64], sb[D / 64];
        if constexpr (D == 128) {
          const uint32_t x = lds_u16(cbase + ks_off + (16 * rg) * C::SROW);
          const uint32_t y = lds_u16(cbase + ks_off + (16 * rg + 8) * C::SROW);
          sa[0] = (x & 0xffu) * 0x00800080u;
          sa[1] = (x >> 8) * 0x00800080u;
          sb[0] = (y & 0xffu) * 0x00800080u;
          sb[1] = (y >> 8) * 0x00800080u;
        } else {
          sa[0] = lds_u8(cbase + ks_off + (16 * rg) * C::SROW) * 0x00800080u;
          sb[0] = lds_u8(cbase + ks_off + (16 * rg + 8) * C::SROW) * 0x00800080u;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
          sc[rg][n][0] = sc[rg][n][1] = sc[rg][n][2] = sc[rg][n][3] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {  // a word: eight channels, two steps of the sum
          const uint32_t fa = sa[w / 2], fb = sb[w / 2];
          const uint32_t a0 = mul_f16x2(e2m1x2_to_f16x2<0>(ka[w]), fa);
          const uint32_t a1 = mul_f16x2(e2m1x2_to_f16x2<0>(kb[w]), fb);
          const uint32_t a2 = mul_f16x2(e2m1x2_to_f16x2<1>(ka[w]), fa);
          const uint32_t a3 = mul_f16x2(e2m1x2_to_f16x2<1>(kb[w]), fb);
          const uint32_t c0 = mul_f16x2(e2m1x2_to_f16x2<2>(ka[w]), fa);
          const uint32_t c1 = mul_f16x2(e2m1x2_to_f16x2<2>(kb[w]), fb);
          const uint32_t c2 = mul_f16x2(e2m1x2_to_f16x2<3>(ka[w]), fa);
          const uint32_t c3 = mul_f16x2(e2m1x2_to_f16x2<3>(kb[w]), fb);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma(sc[rg][n], a0, a1, a2, a3, qb[n][4 * w], qb[n][4 * w + 1]);
            mma(sc[rg][n], c0, c1, c2, c3, qb[n][4 * w + 2], qb[n][4 * w + 3]);
          }
        }
      }
      // rows past the sequence: their scores become -inf, and their values' scales, which may be
      // NaN, 0 (a branch that few tiles take)
      const bool edge = key0 + 16 * RG > k_end;
      if (edge) {
#pragma unroll
        for (int rg = 0; rg < RG; ++rg)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (key0 + 16 * rg + 8 * i + perm<D>(g) >= k_end) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < H; ++h) sc[rg][n][2 * i + h] = -INFINITY;
            }
        for (int r = lane; r < 16 * RG; r += 32)
          if (key0 + r >= k_end)
            *reinterpret_cast<Scales*>(s_codes + s * C::CODES + (KT + wrow + r) * C::SROW) =
                Scales{};
        __syncwarp();
      }
      // The largest scores; where one exceeds the maximum by the threshold (or there is none yet)
      // the maxima are raised first.
      float top[NT][H];
      bool over = unset;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          top[n][h] = fmaxf(sc[0][n][h], sc[0][n][2 + h]);
#pragma unroll
          for (int rg = 1; rg < RG; ++rg)
            top[n][h] = fmax3(top[n][h], sc[rg][n][h], sc[rg][n][2 + h]);
          top[n][h] = __fmul_rn(top[n][h], qf[n][h]);
          over |= top[n][h] - m_ref[n][h] > kRescaleThreshold + kWeightLog2;
        }
      if (__any_sync(0xffffffffu, over)) {
        unset = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float f[2] = {1.f, 1.f};  // what the sums so far are scaled by
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const float most = column_max(top[n][h]), mx = most - kWeightLog2;
            if (most - m_ref[n][h] > kRescaleThreshold + kWeightLog2) {
              f[h] = ex2_approx(m_ref[n][h] - mx);  // 0 when m_ref was -inf
              l_part[n][h] *= f[h];
              m_ref[n][h] = mx;
            }
            unset |= m_ref[n][h] == -INFINITY;
          }
          if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              o[c][n][0] *= f[0];
              o[c][n][2] *= f[0];
              if (H == 2) {
                o[c][n][1] *= f[1];
                o[c][n][3] *= f[1];
              }
            }
          }
        }
        unset = __any_sync(0xffffffffu, unset);
      }
      // Weights, turned to the layout of the second product.  A score is rounded by itself, as in the
      // maximum, and the difference is exact where it counts: scores past 2^24, between which
      // fp32 has no numbers, then have weights of at most 2^15 all the same (with an FMA, whose
      // product is not rounded, they are off by a score's last bit: infinities, or no weight at all).
      uint32_t pb[RG][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float ref[H];  // (a row that has seen nothing yet: 2^-inf = 0, and a NaN score stays NaN)
#pragma unroll
        for (int h = 0; h < H; ++h) ref[h] = m_ref[n][h] == -INFINITY ? 0.f : m_ref[n][h];
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
          float w[4] = {};
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < H; ++h) {
              w[2 * i + h] = ex2_approx(__fmul_rn(sc[rg][n][2 * i + h], qf[n][h]) - ref[h]);
              l_part[n][h] += w[2 * i + h];
            }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            pb[rg][n][i] = transpose8x8(pack_f16x2(w[2 * i], w[2 * i + 1]));
        }
      }
      // O^T: rows perm(2j), perm(2j + 1) and eight further
#pragma unroll
      for (int rg = 0; rg < RG; ++rg) {
        uint32_t x[2][2][VW];  // [+8][row of the pair]
        uint32_t sv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lds<VW>(vbase + va_off + (16 * rg + 8 * i) * C::ROW, x[i][0]);
          lds<VW>(vbase + vb_off + (16 * rg + 8 * i) * C::ROW, x[i][1]);
          const uint32_t ua = lds_u8(cbase + vs_a + (16 * rg + 8 * i) * C::SROW);
          const uint32_t ub = lds_u8(cbase + vs_b + (16 * rg + 8 * i) * C::SROW);
          sv[i] = ua * 0x80u + ub * 0x800000u;
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          // the rows' even channels, then their odd ones: byte b is channel 8w + 2b (+ 1)
          uint32_t ev[2], od[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t u = x[i][0][w], v = x[i][1][w];
            ev[i] = (u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u);
            od[i] = ((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u);
          }
          auto step = [&](int c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            a0 = mul_f16x2(a0, sv[0]);
            a1 = mul_f16x2(a1, sv[0]);
            a2 = mul_f16x2(a2, sv[1]);
            a3 = mul_f16x2(a3, sv[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma(o[c][n], a0, a1, a2, a3, pb[rg][n][0], pb[rg][n][1]);
          };
          step(4 * w, e2m1x2_to_f16x2<0>(ev[0]), e2m1x2_to_f16x2<0>(od[0]),
               e2m1x2_to_f16x2<0>(ev[1]), e2m1x2_to_f16x2<0>(od[1]));
          step(4 * w + 1, e2m1x2_to_f16x2<1>(ev[0]), e2m1x2_to_f16x2<1>(od[0]),
               e2m1x2_to_f16x2<1>(ev[1]), e2m1x2_to_f16x2<1>(od[1]));
          step(4 * w + 2, e2m1x2_to_f16x2<2>(ev[0]), e2m1x2_to_f16x2<2>(od[0]),
               e2m1x2_to_f16x2<2>(ev[1]), e2m1x2_to_f16x2<2>(od[1]));
          step(4 * w + 3, e2m1x2_to_f16x2<3>(ev[0]), e2m1x2_to_f16x2<3>(od[0]),
               e2m1x2_to_f16x2<3>(ev[1]), e2m1x2_to_f16x2<3>(od[1]));
        }
      }
      if (edge) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (++s == NS) s = 0, phase ^= 1;
    }

#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        l_part[n][h] += __shfl_xor_sync(0xffffffffu, l_part[n][h], 4);
        l_part[n][h] += __shfl_xor_sync(0xffffffffu, l_part[n][h], 8);
        l_part[n][h] += __shfl_xor_sync(0xffffffffu, l_part[n][h], 16);
      }
    if (!ok) break;
    if (threadIdx.x == 0) pc.leave_for_merge(p.line);
    // The warp's partial result, relative to m_ref.
    const size_t slot = (static_cast<size_t>(blockIdx.x) + pc.segment(p.line)) * NW + warp;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int r = H == 2 ? 8 * n + cq + h : j;
        if (row_base + r >= p.rep) continue;
        const size_t at = slot * p.part_rows + r;
        if (g == 0)
          *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m_ref[n][h], l_part[n][h]);
        float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + (D / 8) * g);
#pragma unroll
        for (int c = 0; c < D / 16; c += 2)
          dst[c / 2] = make_float4(o[c][n][h], o[c][n][2 + h], o[c + 1][n][h], o[c + 1][n][2 + h]);
      }
  }
  // After a wait that ran out (otherwise n = 0): the merge, which follows whatever happened here,
  // reads where a segment's results are, those of the segments that were not reached too.
  if (threadIdx.x == 0)
    for (; pc.n > 0; pc.next(p.line)) pc.leave_for_merge(p.line);
}

template <int D, int NT, int RG, int H>
cudaError_t launch_t(const GroupArgs& a, cudaStream_t stream) {
  using C = Cfg<D, NT, RG>;
  constexpr int KT = C::KT;
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.line = group_line(a);
  p.rows = CacheRows{a.cache.block_table, a.Hkv, a.cache.Lmax, a.cache.page_size,
                     a.cache.num_pages, a.cache.max_pages};
  p.k_scale = static_cast<const uint8_t*>(a.cache.k_scale);
  p.v_scale = static_cast<const uint8_t*>(a.cache.v_scale);
  p.lost = a.lost;
  const bool paged = a.cache.block_table != nullptr;
  p.box_rows = KT;
  if (paged && a.cache.page_size % KT != 0) p.box_rows = std::min(a.cache.page_size, 64);
  p.nbox = KT / p.box_rows;
  p.batch = 32 / p.nbox;
  p.lanes_tile = 65536 / p.nbox + 1;
  // (the scales' base is 16-byte aligned, and so is every page's and tile's.  By lanes where a box
  // is small: 16 sequences of 4000 to 8000 rows in 16-row pages 33.7 against 36.9 us, with 64
  // channels 32.4 against 36.9, in 32-row pages the same and 27.8 against 29.3; in 64-row pages, 64
  // sequences of 512 to 8192 rows, 71.0 against 66.5.)
  p.code_copies = paged ? p.box_rows >= 64 : a.cache.Lmax % (16 / C::SROW) == 0;
  p.box_shift = !paged ? 31 : (p.box_rows == 16 ? 4 : 5);
  p.part_o = a.part_o;
  p.part_ml = a.part_ml;
  p.status = a.status;
  p.rep = a.Hq / a.Hkv;
  p.rblocks = a.plan.rblocks;
  p.part_rows = a.plan.part_rows;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);

  alignas(64) CUtensorMap tk, tv;
  const int rows = paged ? a.cache.page_size : a.cache.Lmax;
  const int planes = paged ? a.cache.num_pages * a.Hkv : a.B * a.Hkv;
  if (!make_tmap_u8_3d(&tk, a.cache.k, C::ROW, rows, planes, p.box_rows, D == 128) ||
      !make_tmap_u8_3d(&tv, a.cache.v, C::ROW, rows, planes, p.box_rows, D == 128))
    return cudaErrorInvalidValue;
  static SmemLimitOnce smem_limit;
  cudaError_t e = smem_limit.set(decode_fp4_kernel<D, NT, RG, H>, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.plan.grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp4_kernel<D, NT, RG, H>, p, tk, tv);
}

template <int D, int NT, int H>
cudaError_t launch_unit(const GroupArgs& a, cudaStream_t stream) {
  return a.plan.unit == kFp4ShortTile ? launch_t<D, NT, kFp4ShortTile / (16 * NW), H>(a, stream)
                                      : launch_t<D, NT, fp4_long_tile(D) / (16 * NW), H>(a, stream);
}
template <int D>
cudaError_t launch_rows(const GroupArgs& a, cudaStream_t stream) {
  // Up to four query rows take every other column of a product, so that a lane has weights of one
  // column to work out and not of two (64 sequences of 512 to 8192 rows: 64.0 against 65.1 us; 32
  // of 4000 to 8000 with 64 channels 32.0 against 32.9).
  if (a.Hq / a.Hkv <= 4) return launch_unit<D, 1, 1>(a, stream);
  return a.plan.block_rows <= 8 ? launch_unit<D, 1, 2>(a, stream) : launch_unit<D, 2, 2>(a, stream);
}

}  // namespace

cudaError_t launch_decode_fp4(const GroupArgs& a, cudaStream_t stream) {
  return a.d == 64 ? launch_rows<64>(a, stream) : launch_rows<128>(a, stream);
}

}  // namespace csattn
