// Attention of a few query rows per KV head over a cache, bf16 or e4m3: the decode of an
// 8-bit cache (one query per head) and the drafts of a token tree (T queries per head).
//
// All T * Hq/Hkv query rows of a KV head read the same cache rows, so they are one side of a
// matrix product and every cache row is read from HBM once per 8 * NT of them.  A CTA:
//   warp 4      producer: 64-row K and V tiles (and their scale bytes) into a ring by TMA, and a
//               piece's queries, rotated, ahead of its other tiles
//   warps 0..3  16 cache rows each per tile, by mma.sync m16n8k16 with the cache rows (then the
//               channels) on the side of 16 and the query rows on the side of 8:
//               S^T = K Q^T, then O^T += V^T P^T; softmax statistics in fp32 between the two;
//               each leaves a partial result of its own per piece.
// CTAs, a wave of them, take equal ranges of all the tiles (group_work.cuh).
// With one query per head a KV head has 4 or 8 query rows: on the side of 8 nothing or little
// is padding, which halves products, exponentials and accumulators against the other way
// round, and an e4m3 row is taken to f16 once for all query rows.  The partial results are
// merged by group_merge_kernel.
//
// e4m3 rows k8 * 2^ek, v8 * 2^ev enter the products as f16 (exact), never scaled:
//   S column j:  x_j = (q16 . k8_j) * 2^ek_j * row factor  (q is taken to f16 with its largest
//                channel in [2^14, 2^15.5): 11 bits, and channels below 2^-38 of the largest
//                vanish)
//   denominator: sum_j 2^(x_j - m)      with m the running maximum of x
//   numerator:   sum_j w_j v8_j, w_j = 2^((x_j - m) + ev_j - n), n that of (x - m) + ev
// Two maxima keep w_j in f16's range whatever the values' scales: a row with small values and
// a large weight (a first token that takes up attention) counts in full.  n is relative to m, so
// that no exponent is lost beside a large score.  w is rounded to f16 (11 bits) scaled by 2^7,
// so what is below 2^-32 of the largest vanishes; the bf16 cache's P is rounded to bf16 (8
// bits: the values on the other side of the product are bf16, and f16 would not hold them), as in
// the other bf16 kernels; sums are fp32 throughout.
// A maximum is raised only when a score exceeds it by 2^8, and only then do the lanes exchange
// theirs: the usual tile costs one vote.
//
// What bounds it (128 channels, 4 query heads per KV head, e4m3): HBM for long sequences, 88.6 us
// for 561 MB of 8 sequences (6.3 TB/s; the issue slots are 42 % busy, most of it e4m3 to f16);
// 64 sequences of 512 to 8192 rows take 93.3 us for 576 MB (their ends add pieces: a piece's
// queries and scale bytes are taken off the compute warps, which cost 114 us), and one of 1000
// rows 8.7 us, the latencies of two launches, the lengths, a tile and the merge.
#include "fp8.cuh"
#include "group_work.cuh"
#include "internal.h"

namespace csattn {
namespace {

constexpr int KT = 64;  // cache rows per tile
constexpr int NW = 4;   // compute warps, 16 rows of a tile each
constexpr int kThreads = 32 * (NW + 1);
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 100000000ull;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kWeightLog2 = 7.0f;  // e4m3: w is held times 2^7 (w <= 2^(8 + 7) < 65504)

template <int D, bool F8, int NT>
struct Cfg {
  static constexpr int ROW = F8 ? D : 2 * D;
  static constexpr int TILE = KT * ROW;
  static constexpr int STAGE = 2 * TILE;
  static constexpr int ROWS = 8 * NT;               // query rows of a CTA
  static constexpr int QS = 2 * D + 16;             // bytes between query rows (no bank twice)
  // resident CTAs (group_attn_ctas) and ring: 160-190 KB in flight per SM
  static constexpr int CTAS = group_attn_ctas(D, F8, ROWS);
  static constexpr int NS = STAGE == 32768 ? 3 : (STAGE == 16384 ? (F8 && CTAS == 2 ? 5 : 4) : 6);
  static constexpr int RING = NS * STAGE;
  static constexpr int Q_BYTES = ROWS * QS;         // twice: the next piece's go to the other
  static constexpr int BARS = 192;
  static constexpr int CODES = F8 ? 2 * KT : 0;     // scale bytes of a tile: keys', values'
  static constexpr int SMEM = 1024 + RING + 2 * Q_BYTES + BARS + 2 * ROWS * 4 + NS * CODES;
  static_assert(8 * (2 * NS + 4) + 4 <= BARS, "barriers");
};

struct GParams {
  const __nv_bfloat16* q;
  const float* q_factor;
  const uint32_t* anc;
  GroupLine line;
  CacheRows rows;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int words, rope;
  int lost;          // arrivals that the queries' barrier waits for and nothing makes (selftest)
  int box_rows;
  bool code_copies;  // scale bytes lie so that bulk copies can take them
  float* part_o;
  float* part_ml;
  uint32_t* status;
  int Hq, Hkv, T, rep, rblocks, part_rows;
  float scale_log2;
  RopeTable theta;
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F8) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// byte offset of the 16-byte chunk cc of row r of a TMA tile: bf16 tiles are 64-channel
// blocks of 128-byte rows, e4m3 tiles rows of D bytes; the swizzle is as wide as the row
template <int D, bool F8>
__device__ __forceinline__ uint32_t tile_off(int r, int cc) {
  if constexpr (!F8) return (cc >> 3) * (KT * 128) + r * 128 + (((cc & 7) ^ (r & 7)) << 4);
  if constexpr (D == 128) return r * 128 + ((cc ^ (r & 7)) << 4);
  return r * 64 + ((cc ^ ((r >> 1) & 3)) << 4);
}

// the 16 mask bits of drafts j0.. (j0 > -16) of a query with mask words `anc`; the rows
// before the drafts (j < 0) are seen by every query
__device__ __forceinline__ uint32_t draft_bits(const uint32_t* anc, int words, int j0) {
  if (words == 0) return j0 >= 0 ? 0u : (1u << -j0) - 1u;
  if (j0 < 0) return ((anc[0] << -j0) | ((1u << -j0) - 1u)) & 0xffffu;
  const int w = j0 >> 5;
  if (w >= words) return 0u;
  return __funnelshift_r(anc[w], w + 1 < words ? anc[w + 1] : 0u, j0 & 31) & 0xffffu;
}

// zero the halves (bf16) or bytes (e4m3) of a word that hold an infinity or NaN
template <bool F8>
__device__ __forceinline__ uint32_t finite_word(uint32_t w) {
  if constexpr (F8) return finite_e4m3x4(w);
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

// max over the eight lanes that hold one query row's column
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

template <int D, bool F8, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, F8, NT>::CTAS)
    group_attn_kernel(const __grid_constant__ GParams p, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D, F8, NT>;
  constexpr int NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* s_q = smem + C::RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::RING + 2 * C::Q_BYTES);
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;   // [2]: a piece's queries in buffer piece % 2
  uint64_t* q_empty = q_full + 2;  // [2]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(q_empty + 2);
  float* s_qf = reinterpret_cast<float*>(smem + C::RING + 2 * C::Q_BYTES + C::BARS);  // [2][ROWS]
  uint8_t* s_codes = reinterpret_cast<uint8_t*>(s_qf + 2 * C::ROWS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // what launch_tree_prep wrote is visible from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // let the merge be scheduled once every CTA has started; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], F8 && !p.code_copies ? 2 : 1);
      mbar_init(&empty[s], NW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1 + p.lost);
      mbar_init(&q_empty[i], NW);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // (a tree's lengths have been checked by launch_tree_prep)
  GroupPiece pc = group_start(p.line, p.status, p.line.drafts > 0);
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
    // (the kernel before wrote the drafts' rows by plain stores)
    asm volatile("fence.proxy.async.global;" ::: "memory");
    // (64 sequences of 512-8192 rows: 99.3 -> 93.6 us; the partial results, the lengths and the
    // code stay in L2)
    const uint64_t once = evict_first_policy();
    const CacheRows& R = p.rows;
    const int M = p.T * p.rep;
    const int nbox = KT / p.box_rows, r0 = lane * p.box_rows;
    int issued = 0;
    // The queries of a piece: D/16 lanes per row, 16 channels each.  Rotated here for one query
    // per head (then all rows are at one position); a tree's come rotated.  They are read ahead
    // of a piece's first tile and staged behind it.
    constexpr int G = D / 16, PASSES = C::ROWS * G / 32;
    const int qc = lane % G;
    int e0, e1;
    rope_piece(p.rope, D / 2, qc, &e0, &e1);
    uint4 q_lo[PASSES], q_hi[PASSES];
    float factor[PASSES];
    auto load_queries = [&](const GroupPiece& pc) {
      const int kvh = pc.head / p.rblocks;
      const int row0 = (pc.head - kvh * p.rblocks) * C::ROWS + lane / G;
      const size_t at = (static_cast<size_t>(pc.b) * p.Hkv + kvh) * M + row0;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        q_lo[i] = q_hi[i] = make_uint4(0u, 0u, 0u, 0u);
        factor[i] = 1.f;
        if (row0 + 32 / G * i < M) {
          const __nv_bfloat16* src = p.q + (at + 32 / G * i) * D;
          q_lo[i] = *reinterpret_cast<const uint4*>(src + e0);
          q_hi[i] = *reinterpret_cast<const uint4*>(src + e1);
          if (F8 && p.q_factor != nullptr) factor[i] = p.q_factor[at + 32 / G * i];
        }
      }
    };
    auto stage_queries = [&](int pos, int piece) {
      const int buf = piece & 1;
      bool room = true;
      if (piece >= 2 && lane == 0)
        room = ctl_wait(&q_empty[buf], ((piece >> 1) - 1) & 1, abort_flag, p.status, kWaitNs);
      if (!__all_sync(0xffffffffu, room)) return false;
      float cs[8], sn[8];
      if constexpr (F8) {
        // lane i has angles N (i / G).. of chunk i % G, and hands them to the lanes of the chunk
        constexpr int N = G / 4;
        float c1[N], s1[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int at = 8 * qc + N * (lane / G) + j;
          c1[j] = 1.f;
          s1[j] = 0.f;
          if (p.rope != 0)
            angle_cos_sin(pos, p.theta.hi[at], p.theta.lo[at], c1[j], s1[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          cs[j] = __shfl_sync(0xffffffffu, c1[j % N], G * (j / N) + qc);
          sn[j] = __shfl_sync(0xffffffffu, s1[j % N], G * (j / N) + qc);
        }
      }
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = 32 / G * i + lane / G;
        uint8_t* dst = s_q + buf * C::Q_BYTES + r * C::QS;
        if constexpr (F8) {
          if (p.q_factor == nullptr)
            factor[i] = query_to_f16<G>(q_lo[i], q_hi[i], p.rope, cs, sn);
          if (qc == 0) s_qf[buf * C::ROWS + r] = factor[i] * p.scale_log2;
          // a lane's four bytes of a K row are channels 4(lane%4).. of 16, so the product's
          // index runs over the 16 channels as 0 1, 4 5, 8 9, 12 13, then 2 3, 6 7, ...
          const uint32_t wl[4] = {q_lo[i].x, q_lo[i].y, q_lo[i].z, q_lo[i].w};
          const uint32_t wh[4] = {q_hi[i].x, q_hi[i].y, q_hi[i].z, q_hi[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int off = 2 * ((j >> 1) * 2 + (j & 1) * 8);  // bytes within a half chunk
            const int b0 = (e0 & 15) ? 8 : 0, b1 = (e1 & 15) ? 8 : 0;
            *reinterpret_cast<uint32_t*>(dst + 2 * (e0 & ~15) + off + b0) = wl[j];
            *reinterpret_cast<uint32_t*>(dst + 2 * (e1 & ~15) + off + b1) = wh[j];
          }
        } else {
          *reinterpret_cast<uint4*>(dst + 2 * e0) = q_lo[i];
          *reinterpret_cast<uint4*>(dst + 2 * e1) = q_hi[i];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[buf]);
      return true;
    };
    bool ok = true;
    for (int piece = 0; pc.n > 0 && ok; pc.next(p.line), ++piece) {
      const int b = pc.b, kvh = pc.head / p.rblocks, total = pc.L + p.line.drafts;
      // the queries behind as many tiles as find room at once: the ring, or (it is full of the
      // last piece's) one
      const int q_at = min(pc.n, piece == 0 && (!F8 || p.code_copies) ? NS : 1) - 1;
      load_queries(pc);
      // without bulk copies: the bytes of two rows per lane, a tile ahead
      auto load_codes = [&](int t, uint8_t (&byte)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = (pc.t0 + t) * KT + lane + 32 * i;
          const long long at = t < pc.n && r < total ? R.at(b, kvh, r) : -1;
          byte[i] = at >= 0 ? p.k_scale[at] : 0;
          byte[2 + i] = at >= 0 ? p.v_scale[at] : 0;
        }
      };
      uint8_t byte[4];
      if (F8 && !p.code_copies) load_codes(0, byte);
      for (int t = 0; t < pc.n; ++t) {
        const int s = issued % NS, use = issued / NS, row0 = (pc.t0 + t) * KT;
        uint8_t* codes = s_codes + s * C::CODES;
        int plane = b * p.Hkv + kvh, prow = row0;
        int code_rows = min(KT, R.Lmax - row0);  // scale bytes of the lane's box to copy
        bool lost = false;                       // its page is outside the pool
        if (R.block_table != nullptr) {
          const int tr = row0 + r0;
          plane = R.num_pages * p.Hkv;
          prow = 0;
          code_rows = 0;
          if (lane < nbox && tr < total) {
            const int page =
                R.block_table[static_cast<size_t>(b) * R.max_pages + tr / R.page_size];
            lost = page < 0 || page >= R.num_pages;
            if (!lost) {
              plane = page * p.Hkv + kvh;
              code_rows = p.box_rows;
            } else {
              atomicOr(p.status, kStatusDeviceArg);
            }
            prow = tr % R.page_size;
          }
        }
        if (lane >= nbox) code_rows = 0;
        bool room = true;
        if (lane == 0 && use > 0)
          room = ctl_wait(&empty[s], (use - 1) & 1, abort_flag, p.status, kWaitNs);
        if (!__all_sync(0xffffffffu, room)) {
          ok = false;
          break;
        }
        uint32_t bytes = C::STAGE;
        if constexpr (F8) {
          if (lost && p.code_copies) {  // the rows read as zeros: their scale has to be a number
            for (int i = 0; i < p.box_rows; i += 16) {
              *reinterpret_cast<uint4*>(codes + r0 + i) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(codes + KT + r0 + i) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          if (p.code_copies)
            bytes += 2 * __reduce_add_sync(0xffffffffu, static_cast<unsigned>(code_rows));
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
        __syncwarp();
        if (lane < nbox) {
          uint8_t* kd = smem + s * C::STAGE + r0 * (F8 ? D : 128);
          uint8_t* vd = kd + C::TILE;
          constexpr int kBlocks = F8 ? 1 : D / 64;
          for (int kb = 0; kb < kBlocks; ++kb)
            tma_load_3d_once(kd + kb * (KT * 128), &tm_k, &full[s], kb * 64, prow, plane, once);
          for (int kb = 0; kb < kBlocks; ++kb)
            tma_load_3d_once(vd + kb * (KT * 128), &tm_v, &full[s], kb * 64, prow, plane, once);
          if (F8 && p.code_copies && code_rows > 0) {
            const size_t at =
                static_cast<size_t>(plane) * (R.block_table != nullptr ? R.page_size : R.Lmax) +
                prow;
            bulk_load(codes + r0, p.k_scale + at, code_rows, &full[s]);
            bulk_load(codes + KT + r0, p.v_scale + at, code_rows, &full[s]);
          }
        }
        __syncwarp();
        ++issued;
        if (t == q_at) ok = stage_queries(pc.L - 1, piece);
        if (F8 && !p.code_copies) {
          uint8_t next[4];
          load_codes(t + 1, next);
          codes[lane] = byte[0];
          codes[lane + 32] = byte[1];
          codes[KT + lane] = byte[2];
          codes[KT + lane + 32] = byte[3];
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
#pragma unroll
          for (int i = 0; i < 4; ++i) byte[i] = next[i];
        }
        if (!ok) break;
      }
    }
    if (lane == 0 && *abort_flag) {
      const int first = issued > NS ? issued - NS : 0;
      for (int t = first; t < issued; ++t)
        mbar_wait(&full[t % NS], (t / NS) & 1, nullptr, p.status, kDrainNs);
    }
    return;
  }

  // ---------------------------------------------------------------- compute warps
  const int M = p.T * p.rep;      // query rows of the KV head: row = t * rep + head
  const int r0 = lane >> 2;       // fragment rows r0 and r0 + 8 (cache rows)
  const int cq = 2 * (lane & 3);  // fragment columns cq and cq + 1 (query rows)
  const int mi = lane >> 3;       // which 8x8 matrix this lane addresses
  const uint32_t smem_base = smem_u32(smem);
  // addresses of the lane's matrix rows within a tile
  const int kr = 16 * warp + (lane & 7) + 8 * (mi & 1);
  const int vr = 16 * warp + (lane & 7) + 8 * (F8 ? (mi & 1) : (mi >> 1));
  bool ok = true;
  int used = 0;  // tiles of the CTA so far
  for (int piece = 0; pc.n > 0; pc.next(p.line), ++piece) {
    const int b = pc.b, kvh = pc.head / p.rblocks, L = pc.L, total = L + p.line.drafts;
    const int row_base = (pc.head - kvh * p.rblocks) * C::ROWS;  // first query row
    const int k_begin = pc.t0 * KT, ntiles = pc.n;
    const int k_end = min(total, k_begin + ntiles * KT);

    ok = __all_sync(0xffffffffu, mbar_wait(&q_full[piece & 1], (piece >> 1) & 1, abort_flag,
                                           p.status, kWaitNs));
    if (!ok) break;
    const uint32_t q_addr = smem_u32(s_q + (piece & 1) * C::Q_BYTES) + (lane & 7) * C::QS + mi * 16;
    uint32_t qb[NT][D / 16][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += 2) {
        uint32_t w[4];
        ldsm_x4(q_addr + j * 8 * C::QS + kk * 32, w);
        qb[j][kk][0] = w[0];
        qb[j][kk][1] = w[1];
        qb[j][kk + 1][0] = w[2];
        qb[j][kk + 1][1] = w[3];
      }
    float qf[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        qf[j][h] = F8 ? s_qf[(piece & 1) * C::ROWS + 8 * j + cq + h] : p.scale_log2;
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_empty[piece & 1]);

    float o[D / 16][NT][4];
    float m_used[NT][2], n_used[NT][2], l_part[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[c][j][0] = o[c][j][1] = o[c][j][2] = o[c][j][3] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) m_used[j][h] = n_used[j][h] = -INFINITY, l_part[j][h] = 0.f;
    }

    bool unset = true;  // some query row has no maximum yet
    for (int t = 0; t < ntiles && ok; ++t, ++used) {
      const int s = used % NS;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (used / NS) & 1, abort_flag, p.status,
                                             kWaitNs))) {
        ok = false;
        break;
      }
      const uint32_t kbase = smem_base + s * C::STAGE;
      const uint32_t vbase = kbase + C::TILE;
      const int key0 = k_begin + t * KT + 16 * warp;  // first cache row of the warp
      float sc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += 2) {
        uint32_t a[2][4];
        if constexpr (F8) {
          uint32_t w[4];
          ldsm_x4(kbase + tile_off<D, F8>(kr, kk + (mi >> 1)), w);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[i][0] = e4m3x2_to_f16x2(w[2 * i]);
            a[i][1] = e4m3x2_to_f16x2(w[2 * i + 1]);
            a[i][2] = e4m3x2_hi_to_f16x2(w[2 * i]);
            a[i][3] = e4m3x2_hi_to_f16x2(w[2 * i + 1]);
          }
        } else {
          ldsm_x4(kbase + tile_off<D, F8>(kr, 2 * kk + (mi >> 1)), a[0]);
          ldsm_x4(kbase + tile_off<D, F8>(kr, 2 * kk + 2 + (mi >> 1)), a[1]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma<F8>(sc[j], a[0], qb[j][kk][0], qb[j][kk][1]);
          mma<F8>(sc[j], a[1], qb[j][kk + 1][0], qb[j][kk + 1][1]);
        }
      }
      // factors of the thread's two cache rows
      float kf[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f};
      if constexpr (F8) {  // (of rows past the sequence: any value, their scores are -inf below)
        const uint8_t* codes = s_codes + s * C::CODES + 16 * warp + r0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          kf[i] = __uint_as_float(static_cast<uint32_t>(codes[8 * i]) << 23);
          ev[i] = static_cast<float>(static_cast<int>(codes[KT + 8 * i]) - 127);
        }
      }
      // cache rows that a query row does not see: their scores become -inf
      const bool edge = key0 + 16 > min(L, k_end);
      uint32_t hide = 0u;  // bit 4j + 2i + h
      if (edge) {
        const uint32_t in = key0 + 16 <= k_end ? 0xffffu
                            : key0 >= k_end    ? 0u
                                               : (1u << (k_end - key0)) - 1u;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int tq = min((row_base + 8 * j + cq + h) / p.rep, p.T - 1);
            const uint32_t* anc = p.anc + (static_cast<size_t>(b) * p.T + tq) * p.words;
            const uint32_t see =
                in & (key0 + 16 <= L ? 0xffffu : draft_bits(anc, p.words, key0 - L));
#pragma unroll
            for (int i = 0; i < 2; ++i)
              hide |= (1u ^ ((see >> (r0 + 8 * i)) & 1u)) << (4 * j + 2 * i + h);
          }
      }
      // x - m for every score (x rounded by itself, as in m: the largest gives 0); where one
      // exceeds its maximum by the threshold (or there is none yet) the maxima are raised first
      float d[NT][4];
      bool over = false;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e >> 1, h = e & 1;
          d[j][e] = __fmul_rn(sc[j][e], F8 ? kf[i] * qf[j][h] : qf[j][h]) - m_used[j][h];
          if (edge && ((hide >> (4 * j + e)) & 1u)) d[j][e] = -INFINITY;
          over |= d[j][e] > kRescaleThreshold;
          if constexpr (F8) over |= d[j][e] + ev[i] > n_used[j][h] + kRescaleThreshold;
        }
      if (__any_sync(0xffffffffu, over || unset)) {
        unset = false;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float f[2] = {1.f, 1.f};  // what the sums so far are scaled by
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              x[i] = __fmul_rn(sc[j][2 * i + h], F8 ? kf[i] * qf[j][h] : qf[j][h]);
              if (edge && ((hide >> (4 * j + 2 * i + h)) & 1u)) x[i] = -INFINITY;
            }
            const float mx = column_max(fmaxf(x[0], x[1]));
            if (mx > m_used[j][h] + kRescaleThreshold) {
              const float r = m_used[j][h] - mx;
              l_part[j][h] *= ex2_approx(r);  // 0 when m_used was -inf
              if constexpr (F8)
                n_used[j][h] += r;  // the numerator's reference m + n stays where it was
              else
                f[h] = ex2_approx(r);
              m_used[j][h] = mx;
            }
            // (a row that has seen nothing yet: 2^-inf = 0, and a NaN score stays NaN)
            const float m_ref = m_used[j][h] == -INFINITY ? 0.f : m_used[j][h];
            unset |= m_used[j][h] == -INFINITY;
#pragma unroll
            for (int i = 0; i < 2; ++i) d[j][2 * i + h] = x[i] - m_ref;
            if constexpr (F8) {
              const float my = column_max(fmaxf(d[j][h] + ev[0], d[j][2 + h] + ev[1]));
              if (my > n_used[j][h] + kRescaleThreshold) {
                f[h] = ex2_approx(n_used[j][h] - my);
                n_used[j][h] = my;
              }
            }
          }
          if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              o[c][j][0] *= f[0];
              o[c][j][1] *= f[1];
              o[c][j][2] *= f[0];
              o[c][j][3] *= f[1];
            }
          }
        }
        unset = __any_sync(0xffffffffu, unset);
      }
      // weights, turned to the layout of the second product
      uint32_t pb[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = ex2_approx(d[j][e]);
          l_part[j][e & 1] += v;
          w[e] = v;
          if constexpr (F8) {
            const float n_ref = n_used[j][e & 1] == -INFINITY ? 0.f : n_used[j][e & 1];
            w[e] = ex2_approx(d[j][e] + (ev[e >> 1] + (kWeightLog2 - n_ref)));
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          pb[j][i] = transpose8x8(F8 ? pack_f16x2(w[2 * i], w[2 * i + 1])
                                     : pack_bf16x2(w[2 * i], w[2 * i + 1]));
      }
      // Values of rows that not every query sees must not reach a product (0 * inf is NaN):
      // rows past the sequence are zeroed, and in the drafts' rows what is not finite (the
      // merge puts it where it belongs).
      if (edge) {
        uint8_t* vt = smem + s * C::STAGE + C::TILE;
        for (int e = lane; e < 16 * (C::ROW / 16); e += 32) {
          const int rr = e / (C::ROW / 16), cc = e % (C::ROW / 16);
          uint4* at = reinterpret_cast<uint4*>(vt + tile_off<D, F8>(16 * warp + rr, cc));
          if (key0 + rr >= k_end) {
            *at = make_uint4(0u, 0u, 0u, 0u);
          } else if (key0 + rr >= L) {
            const uint4 v = *at;
            *at = make_uint4(finite_word<F8>(v.x), finite_word<F8>(v.y), finite_word<F8>(v.z),
                             finite_word<F8>(v.w));
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int c = 0; c < D / 16; c += 2) {
        uint32_t a[2][4];
        if constexpr (F8) {
          // a transposed load hands a lane channels (2n, 2n + 1) of two cache rows: regrouped by
          // channel they are rows n (even channels) and n + 8 (odd) of the operand
          uint32_t r[4];
          ldsm_x4_t(vbase + tile_off<D, F8>(vr, c + (mi >> 1)), r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t u = __byte_perm(r[2 * i], 0u, 0x3120);
            const uint32_t v = __byte_perm(r[2 * i + 1], 0u, 0x3120);
            a[i][0] = e4m3x2_to_f16x2(u);
            a[i][1] = e4m3x2_hi_to_f16x2(u);
            a[i][2] = e4m3x2_to_f16x2(v);
            a[i][3] = e4m3x2_hi_to_f16x2(v);
          }
        } else {
          ldsm_x4_t(vbase + tile_off<D, F8>(vr, 2 * c + (mi & 1)), a[0]);
          ldsm_x4_t(vbase + tile_off<D, F8>(vr, 2 * c + 2 + (mi & 1)), a[1]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma<F8>(o[c][j], a[0], pb[j][0], pb[j][1]);
          mma<F8>(o[c + 1][j], a[1], pb[j][0], pb[j][1]);
        }
      }
      if (edge) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l_part[j][h] += __shfl_xor_sync(0xffffffffu, l_part[j][h], 4);
        l_part[j][h] += __shfl_xor_sync(0xffffffffu, l_part[j][h], 8);
        l_part[j][h] += __shfl_xor_sync(0xffffffffu, l_part[j][h], 16);
      }
    if (!ok) break;
    if (threadIdx.x == 0) pc.leave_for_merge(p.line);
    // The warp's partial result.  bf16: relative to the maximum of x.  e4m3: to the power of two
    // that leaves l in [0.5, 1), and its values times 2^-kPartLog2, so that they are of the
    // output's size whatever the values' scales; the factor of o is taken in two halves, 2^n
    // alone leaving fp32's range at the ends of the codes'.
    const size_t slot =
        (static_cast<size_t>(blockIdx.x) + pc.segment(p.line)) * NW + warp;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * j + cq + h;
        if (row_base + r >= M) continue;
        // (a row that saw nothing holds zeros, or NaN if its scores were NaN)
        float m = m_used[j][h], l = l_part[j][h], f = 1.f;
        if (F8 && n_used[j][h] != -INFINITY) {
          // (beside a maximum past 2^23 it would be lost)
          const int up = fabsf(m) < 8388608.f ? log2_above(l) : 0;
          m += static_cast<float>(up);
          l *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
          f = ex2_approx(0.5f * (n_used[j][h] -
                                 (kWeightLog2 + kPartLog2 + static_cast<float>(up))));
        }
        const size_t at = slot * p.part_rows + r;
        float* dst = p.part_o + at * D;
        if (r0 == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          if constexpr (F8) {
            *reinterpret_cast<float2*>(dst + 16 * c + 2 * r0) =
                make_float2(o[c][j][h] * f * f, o[c][j][2 + h] * f * f);
          } else {
            dst[16 * c + r0] = o[c][j][h];
            dst[16 * c + r0 + 8] = o[c][j][2 + h];
          }
        }
      }
  }
  // After a wait that ran out (otherwise n = 0): the merge, which follows whatever happened here,
  // reads where a segment's results are, those of the segments that were not reached too.
  if (threadIdx.x == 0)
    for (; pc.n > 0; pc.next(p.line)) pc.leave_for_merge(p.line);
}

// out[b, h, t, :] = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s over the partial results of a
// query row: `subs` for each piece of its segment, times 2^kPartLog2 for an e4m3 cache.  W warps
// per row (W > 1 for few rows with many partials), four (d = 128) or two channels per lane.
template <int D, int W>
__global__ void __launch_bounds__(32 * (W > 4 ? W : 4)) group_merge_kernel(
    const float* __restrict__ part_o, const float* __restrict__ part_ml, const int2* seg, int heads,
    int subs, int part_rows, int block_rows, int rblocks, const uint32_t* __restrict__ anc,
    const uint8_t* __restrict__ vflag, const __nv_bfloat16* __restrict__ v_new, bool f8,
    __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int rows, int Hq, int Hkv, int T,
    int words) {
  constexpr int V = D / 32;
  constexpr int U = W > 1 ? 8 : 4;  // partial results whose loads are in flight together
  __shared__ float s_part[W > 4 ? W : (W > 1 ? 4 : 1)][V * 32 + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int at_row = static_cast<int>(blockIdx.x) * (W < 4 ? 4 / W : 1) + warp / W;
  // (a warp past the last row works on that row, too, where there is a barrier to come)
  const bool live = at_row < rows;
  const int row = live ? at_row : rows - 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (W == 1 && !live) return;
  const int rep = Hq / Hkv;
  const int t = row % T, bh = row / T, b = bh / Hq, h = bh - b * Hq, g = h / rep;
  const uint32_t* mine = anc + (static_cast<size_t>(b) * T + t) * words;
  const int qrow = t * rep + h - g * rep, rb = qrow / block_rows;
  const int2 at_seg = seg[b * heads + g * rblocks + rb];
  int ns = at_seg.y * subs;
  if (words > 0 && ((mine[t >> 5] >> (t & 31)) & 1u) == 0u) ns = 0;  // padding
  // partial i of the row is row qrow - rb * block_rows of slot at_seg.x * subs + i
  const size_t at0 =
      static_cast<size_t>(at_seg.x) * subs * part_rows + qrow - rb * block_rows;
  float m = -INFINITY, acc[V], l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int s0 = warp % W; s0 < ns; s0 += U * W) {
    float2 ml[U];
    float o[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * W;
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < V; ++i) o[u][i] = 0.f;
      if (s >= ns) continue;
      const size_t at = at0 + static_cast<size_t>(s) * part_rows;
      ml[u] = *reinterpret_cast<const float2*>(part_ml + 2 * at);
      const float* po = part_o + at * D + V * lane;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(o[u]) = *reinterpret_cast<const float4*>(po);
      else
        *reinterpret_cast<float2*>(o[u]) = *reinterpret_cast<const float2*>(po);
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mx = fmaxf(mx, ml[u].x);
    // (one that saw nothing holds zeros, or NaN)
    const float f = m == -INFINITY ? 1.f : ex2_approx(m - mx);
    l *= f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= f;
    m = mx;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float e = ml[u].x == -INFINITY ? 1.f : ex2_approx(ml[u].x - m);
      l += e * ml[u].y;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += e * o[u][i];
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) s_part[warp][V * lane + i] = acc[i];
    if (lane == 0) {
      s_part[warp][V * 32] = l;
      s_part[warp][V * 32 + 1] = m;
    }
    __syncthreads();
    if (!live || warp % W != 0) return;
    float mx = m;
#pragma unroll
    for (int w = 1; w < W; ++w) mx = fmaxf(mx, s_part[warp + w][V * 32 + 1]);
    l = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float mw = s_part[warp + w][V * 32 + 1];
      const float e = mw == -INFINITY ? 1.f : ex2_approx(mw - mx);
      l += e * s_part[warp + w][V * 32];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += e * s_part[warp + w][V * lane + i];
    }
    m = mx;
  }
  const bool any = !(l <= 0.f);  // NaN stays
  const float inv = any ? (f8 ? kPartScale : 1.f) / l : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = any ? acc[i] * inv : 0.f;
  if (vflag != nullptr && ns > 0) {
    for (int w = 0; w < words; ++w) {
      const int j = 32 * w + lane;
      const bool hit = j < T && ((mine[w] >> lane) & 1u) &&
                       vflag[(static_cast<size_t>(b) * Hkv + g) * T + j] != 0;
      for (uint32_t left = __ballot_sync(0xffffffffu, hit); left != 0u; left &= left - 1u) {
        const __nv_bfloat16* v =
            v_new + ((static_cast<size_t>(b) * Hkv + g) * T + 32 * w + __ffs(left) - 1) * D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float x = __bfloat162float(v[V * lane + i]);
          // (an e4m3 cache holds NaN for an infinity)
          if (!isfinite(x)) acc[i] += f8 ? __int_as_float(0x7fffffff) : x;
        }
      }
    }
  }
  __nv_bfloat16* o = out + static_cast<size_t>(row) * D + V * lane;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(o + i) = pack_bf16x2(acc[i], acc[i + 1]);
  if (lse != nullptr && lane == 0)
    lse[row] = any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, bool F8, int NT>
cudaError_t launch_t(const GroupArgs& a, cudaStream_t stream) {
  using C = Cfg<D, F8, NT>;
  GParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_factor = a.q_factor;
  p.anc = a.anc;
  p.line = group_line(a);
  p.rows = CacheRows{a.cache.block_table, a.Hkv, a.cache.Lmax, a.cache.page_size,
                     a.cache.num_pages, a.cache.max_pages};
  p.k_scale = static_cast<const uint8_t*>(a.cache.k_scale);
  p.v_scale = static_cast<const uint8_t*>(a.cache.v_scale);
  p.words = a.words;
  p.rope = a.rope;
  p.lost = a.lost;
  const bool paged = a.cache.block_table != nullptr;
  p.box_rows = paged && a.cache.page_size < KT ? a.cache.page_size : KT;
  const uintptr_t scales =
      reinterpret_cast<uintptr_t>(p.k_scale) | reinterpret_cast<uintptr_t>(p.v_scale);
  p.code_copies = scales % 16 == 0 && (paged || a.cache.Lmax % 16 == 0);
  p.part_o = a.part_o;
  p.part_ml = a.part_ml;
  p.status = a.status;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.T = a.T;
  p.rep = a.Hq / a.Hkv;
  p.rblocks = a.plan.rblocks;
  p.part_rows = a.plan.part_rows;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.theta = a.theta;

  alignas(64) CUtensorMap tk, tv;
  const int rows = paged ? a.cache.page_size : a.cache.Lmax;
  const int planes = paged ? a.cache.num_pages * a.Hkv : a.B * a.Hkv;
  const bool made = F8 ? make_tmap_u8_3d(&tk, a.cache.k, D, rows, planes, p.box_rows, true) &&
                             make_tmap_u8_3d(&tv, a.cache.v, D, rows, planes, p.box_rows, true)
                       : make_tmap_bf16_3d(&tk, a.cache.k, D, rows, planes, p.box_rows) &&
                             make_tmap_bf16_3d(&tv, a.cache.v, D, rows, planes, p.box_rows);
  if (!made) return cudaErrorInvalidValue;
  static SmemLimitOnce smem_limit;
  cudaError_t e = smem_limit.set(group_attn_kernel<D, F8, NT>, C::SMEM);
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
  return cudaLaunchKernelEx(&cfg, group_attn_kernel<D, F8, NT>, p, tk, tv);
}

template <int D, bool F8>
cudaError_t launch_rows(const GroupArgs& a, cudaStream_t stream) {
  return a.plan.block_rows <= 8 ? launch_t<D, F8, 1>(a, stream) : launch_t<D, F8, 2>(a, stream);
}

template <int D, int W>
cudaError_t launch_merge(const GroupArgs& a, const uint8_t* vflag, const void* v_new, void* out,
                         float* lse, cudaStream_t stream) {
  const int rows = a.B * a.Hq * a.T;
  cudaLaunchConfig_t cfg = {};
  constexpr int kRowsPerCta = W < 4 ? 4 / W : 1;
  cfg.gridDim = dim3((static_cast<unsigned>(rows) + kRowsPerCta - 1) / kRowsPerCta, 1, 1);
  cfg.blockDim = dim3(32 * (W > 4 ? W : 4), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(
      &cfg, group_merge_kernel<D, W>, static_cast<const float*>(a.part_o),
      static_cast<const float*>(a.part_ml), a.seg, a.Hkv * a.plan.rblocks, a.plan.subs,
      a.plan.part_rows, a.plan.block_rows, a.plan.rblocks, a.anc, vflag,
      static_cast<const __nv_bfloat16*>(v_new), a.cache.k_scale != nullptr,
      static_cast<__nv_bfloat16*>(out), lse, rows, a.Hq, a.Hkv, a.T, a.words);
}

}  // namespace

cudaError_t launch_group_attn(const GroupArgs& a, cudaStream_t stream) {
  const bool f8 = a.cache.k_scale != nullptr;
  if (a.d == 64) return f8 ? launch_rows<64, true>(a, stream) : launch_rows<64, false>(a, stream);
  return f8 ? launch_rows<128, true>(a, stream) : launch_rows<128, false>(a, stream);
}

cudaError_t launch_group_merge(const GroupArgs& a, const uint8_t* vflag, const void* v_new,
                               void* out, float* lse, cudaStream_t stream) {
  // Warps per row, by the partials that a row has on average.  The whole decode in us with 1, 2,
  // 4, 8, 16 warps: 8192 rows of 5: 59.4, 63.0; 2048 rows of 8: 113.2, 111.5, 115.1; 1024 of 11:
  // -, 48.3, 49.0, 51.4; 512 of 18: -, 30.2, 29.7, 30.5; 128 of 60: -, -, 47.7, 46.3, 46.5; 32 of
  // 230: -, -, 25.9, 22.0, 20.5.
  const int rows = a.B * a.Hq * a.T, segments = a.B * a.Hkv * a.plan.rblocks;
  const int partials = static_cast<int>(
      a.plan.subs * (static_cast<long long>(a.plan.grid) + segments) / segments);
  if (partials > 120)
    return a.d == 128 ? launch_merge<128, 16>(a, vflag, v_new, out, lse, stream)
                      : launch_merge<64, 16>(a, vflag, v_new, out, lse, stream);
  if (partials > 40)
    return a.d == 128 ? launch_merge<128, 8>(a, vflag, v_new, out, lse, stream)
                      : launch_merge<64, 8>(a, vflag, v_new, out, lse, stream);
  if (partials > 12)
    return a.d == 128 ? launch_merge<128, 4>(a, vflag, v_new, out, lse, stream)
                      : launch_merge<64, 4>(a, vflag, v_new, out, lse, stream);
  if (rows <= 4096)
    return a.d == 128 ? launch_merge<128, 2>(a, vflag, v_new, out, lse, stream)
                      : launch_merge<64, 2>(a, vflag, v_new, out, lse, stream);
  return a.d == 128 ? launch_merge<128, 1>(a, vflag, v_new, out, lse, stream)
                    : launch_merge<64, 1>(a, vflag, v_new, out, lse, stream);
}

}  // namespace csattn
