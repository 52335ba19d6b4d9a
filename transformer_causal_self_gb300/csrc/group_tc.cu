// Grouped attention over a cache on the 5th-generation tensor cores: the form of group_attn.cu
// for many query rows per KV head (wide token trees), with the same arguments and the same
// partial results.
//
// The T * Hq/Hkv query rows of a KV head are the 128 rows (TMEM lanes) of one or two tiles;
// the cache comes in tiles of 128 rows.  Two streams, each with a warpgroup of softmax, keep
// the tensor core busy while the other turns scores into weights:
//   more than 128 query rows: stream x is query tile x, both see every cache tile;
//   up to 128: stream x takes every second cache tile, with sums of its own that meet at
//              the end.
// Grid (split * row block, KV head, sequence), one CTA per SM:
//   warps 0-3, 4-7  softmax of stream 0 and 1, a query row per thread; before that they
//                   write the queries to shared memory, at the end the partial results
//   warp 8          TMA producer          warp 9   TMEM owner and MMA issuer (one thread)
//   warps 10-11     bf16: clean the values of tiles that not every query sees
//   warps 12-15     e4m3: take the tiles to f16
// TMEM columns: S_0 [0,128) S_1 [128,256) O_0 [256,256+D) O_1 [256+D,256+2D); P overwrites the
// first half of its S and is read by the second product from there.
//
// An e4m3 tile becomes f16 with one scale for all its rows: row j is multiplied by 2^(7 - (E -
// e_j)), E the largest exponent of the tile (at least -100 for values).  That is exact while
// e_j is within about 15 of E; below, a row's error is an absolute 2^-32 of the tile's largest
// value, which fp32 sums would not resolve either.  So the scales reach the softmax as two
// numbers per tile, and one exponential serves denominator and numerator:
//   w = 2^(x + E_v - R), O += w V16, l += 2^(-E_v) * sum w, R the running maximum of x + E_v.
// R is raised only by more than 2^8, as elsewhere; w is then at most 2^8 (bf16), or 2^15 with
// the 2^7 that the e4m3 path adds for f16's range.
#include "fp8.cuh"
#include "internal.h"

namespace csattn {
namespace {

constexpr int BN = 128;  // cache rows per tile
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 100000000ull;
constexpr float kRescaleThreshold = 8.0f;
constexpr int kMinValueCode = 27;  // E_v >= -100
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpClean = 10, kWarpConvert = 12;

template <int D, bool F8>
struct Cfg {
  static constexpr int kThreads = F8 ? 512 : 384;
  static constexpr int TILE = BN * D * 2;  // a Q, K or V tile of 16-bit values
  static constexpr int RAW = BN * D;       // an e4m3 tile
  static constexpr int NRAW = F8 ? 4 : 0;
  static constexpr int RAW_DEPTH = F8 ? 4 : 1;
  // ring tiles that fit beside one or two query tiles
  static constexpr int NS1 = F8 ? 4 : (D == 128 ? 6 : 8);
  static constexpr int NS2 = F8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);
  static constexpr int TILES = (NS1 + 1 > NS2 + 2 ? NS1 + 1 : NS2 + 2) * TILE + NRAW * RAW;
  static constexpr int SMEM = 1024 + TILES + 320 + 128 * 8 + (F8 ? 8 * 8 + 2 * 256 + 32 : 0);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

struct TParams {
  const uint16_t* q;
  const float* q_factor;
  const int32_t* lens;
  const uint32_t* anc;
  CacheRows rows;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int drafts, words;
  int box_rows;
  float* part_o;
  float* part_ml;
  uint32_t* status;
  int Hq, Hkv, T, rep, max_seq_len, min_len, chunk, n_splits, rblocks, pair;
  float scale_log2;
};

// f16 or bf16 operands, fp32 accumulators, M = 128
constexpr uint32_t idesc(bool f16, int N, int b_mn) {
  return idesc_bf16_f32(128, N, 0, b_mn) & (f16 ? ~((7u << 7) | (7u << 10)) : ~0u);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, kWaitNs)) != 0;
}

// 32 mask bits of drafts j0.. (j0 > -32) of a query with mask words `anc`; rows before the
// drafts (j < 0) are seen by every query
__device__ __forceinline__ uint32_t draft_bits32(const uint32_t* anc, int words, int j0) {
  if (j0 <= -32) return 0xffffffffu;
  if (words == 0) return j0 >= 0 ? 0u : (1u << -j0) - 1u;
  if (j0 < 0) return (anc[0] << -j0) | ((1u << -j0) - 1u);
  const int w = j0 >> 5;
  if (w >= words) return 0u;
  return __funnelshift_r(anc[w], w + 1 < words ? anc[w + 1] : 0u, j0 & 31);
}

__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b));
}

// zero the halves of a word of bf16 that hold an infinity or NaN
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 2^(7 - below) in f16 (0 where that is less than f16's least)
__device__ __forceinline__ uint16_t row_scale(int below) {
  return __half_as_ushort(
      __float2half_rn(below > 60 ? 0.f : __uint_as_float((127u + 7u - below) << 23)));
}

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, 1)
    group_tc_kernel(const __grid_constant__ TParams p, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D, F8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int pair = p.pair;
  const int NS = pair ? C::NS2 : C::NS1;
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + (1 + pair) * C::TILE;
  uint8_t* sRaw = smem + C::TILES - C::NRAW * C::RAW;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::TILES);
  uint64_t* q_ready = bars + 0;    // [2]
  uint64_t* s_full = bars + 2;     // [2]
  uint64_t* p_full = bars + 4;     // [2]
  uint64_t* o_full = bars + 6;     // [2]
  uint64_t* teardown = bars + 8;
  uint64_t* kv_full = bars + 9;    // [8]
  uint64_t* kv_empty = bars + 17;  // [8]
  uint64_t* raw_full = bars + 25;  // [4]
  uint64_t* raw_empty = bars + 29; // [4]
  uint64_t* edge_full = bars + 33; // [4] bf16: values to be cleaned, one per edge tile (256
                                   // drafts that begin inside a tile touch three)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 37);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::TILES + 320);  // [128]
  float2* s_tile = s_ml + 128;                           // e4m3 [8]: 2^(E_k - 7), E_v of a tile
  uint16_t* s_mul = reinterpret_cast<uint16_t*>(s_tile + 8);  // e4m3 [2][128] row factors
  int* s_max = reinterpret_cast<int*>(s_mul + 256);           // e4m3 [2][4]

  const int split = blockIdx.x / p.rblocks, rb = blockIdx.x - split * p.rblocks;
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int L = p.lens[b];
  if (L < p.min_len || L > p.max_seq_len - p.drafts) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0 && (p.drafts == 0 || L != -1))
      atomicOr(p.status, kStatusDeviceArg);
    return;
  }
  const int total = L + p.drafts;
  const int k_begin = split * p.chunk;
  const int k_end = min(total, k_begin + p.chunk);
  if (k_begin >= k_end) return;
  const int n = (k_end - k_begin + BN - 1) / BN;  // tiles
  const int step = pair ? 1 : 2;                  // between a stream's tiles
  // first tile with rows that not every query sees
  const int first_edge = max(0, min(n, (min(L, k_end) - k_begin) / BN));

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_ready[x], 4);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(teardown, 1);
    for (int s = 0; s < 8; ++s) {
      mbar_init(&kv_full[s], F8 ? 4 : 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
      mbar_init(&edge_full[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kWarpProducer) {
    // ------------------------------------------------------------ TMA producer
    // fills K_0, V_0, K_1, V_1, ...; lane i copies box i of a tile (see group_attn.cu)
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const CacheRows& R = p.rows;
    const int nbox = BN / p.box_rows, r0 = lane * p.box_rows;
    const uint32_t depth = F8 ? C::NRAW : NS;
    uint64_t* full = F8 ? raw_full : kv_full;
    uint64_t* empty = F8 ? raw_empty : kv_empty;
    // the barrier of fill f: bf16 values of edge tiles go by way of the cleaning warps
    auto landed = [&](uint32_t f) {
      const int i = static_cast<int>(f >> 1) - first_edge;
      return !F8 && (f & 1u) && i >= 0 ? &edge_full[i] : &full[f % depth];
    };
    uint32_t f = 0;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      int plane = b * p.Hkv + kvh, prow = k_begin + j * BN;
      if (lane < nbox && R.block_table != nullptr) {
        const int tr = prow + r0;
        plane = R.num_pages * p.Hkv;
        prow = 0;
        if (tr < total) {
          const int page = R.block_table[static_cast<size_t>(b) * R.max_pages + tr / R.page_size];
          if (page >= 0 && page < R.num_pages)
            plane = page * p.Hkv + kvh;
          else
            atomicOr(p.status, kStatusDeviceArg);
          prow = tr % R.page_size;
        }
      }
      for (int v = 0; v < 2; ++v, ++f) {
        const uint32_t s = f % depth, use = f / depth;
        int okw = 1;
        if (lane == 0) {
          if (use > 0 && !ctl_wait(&empty[s], (use - 1) & 1, abort_flag, p.status, kWaitNs))
            okw = 0;
          else
            mbar_arrive_expect_tx(landed(f), F8 ? C::RAW : C::TILE);
        }
        okw = __shfl_sync(0xffffffffu, okw, 0);
        if (!okw) {
          ok = false;
          break;
        }
        const CUtensorMap* tm = v == 0 ? &tm_k : &tm_v;
        if (lane < nbox) {
          if constexpr (F8) {
            tma_load_3d(sRaw + s * C::RAW + r0 * D, tm, landed(f), 0, prow, plane);
          } else {
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_3d(sKV + s * C::TILE + kb * (BN * 128) + r0 * 128, tm, landed(f), kb * 64,
                          prow, plane);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0 && *abort_flag) {
      // every copy still in flight lands before the CTA's shared memory is released
      const uint32_t first = f > depth ? f - depth : 0u;
      for (uint32_t i = first; i < f; ++i)
        mbar_wait(landed(i), landed(i) == &full[i % depth] ? (i / depth) & 1 : 0, nullptr,
                  p.status, kDrainNs);
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t kv0 = smem_u32(sKV);
      constexpr uint32_t kIdS = idesc(F8, BN, 0), kIdO = idesc(F8, D, 1);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!ok) return false;
        ok = ctl_wait(bar, parity, abort_flag, p.status, kWaitNs);
        tc_fence_after();
        return ok;
      };
      auto full = [&](uint32_t f) { return wait(&kv_full[f % NS], (f / NS) & 1); };
      auto qk = [&](int x, int j) {
        const uint32_t q = smem_u32(sQ) + (pair ? x : 0) * C::TILE;
        const uint32_t k = kv0 + (2u * j % NS) * C::TILE;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = static_cast<uint32_t>((kk >> 2) * (BN * 128) + (kk & 3) * 32);
          umma_ss(tmem + 128u * x, smem_desc_sw128(q + off, 16, 1024),
                  smem_desc_sw128(k + off, 16, 1024), kIdS, kk > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[x]);
      };
      auto pv = [&](int x, int j) {
        const uint32_t v = kv0 + ((2u * j + 1u) % NS) * C::TILE;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          umma_ts(tmem + 256u + D * x, tmem + 128u * x + 8u * kk,
                  smem_desc_sw128(v + 2048u * kk, BN * 128, 1024), kIdO,
                  (j >= step || kk > 0) ? 1u : 0u);
      };
      wait(&q_ready[0], 0);
      if (pair) wait(&q_ready[1], 0);
      // first tiles of both streams
      for (int j = 0; j < step && j < n; ++j) {
        if (!full(2 * j)) break;
        for (int x = pair ? 0 : j; x <= (pair ? 1 : j); ++x) qk(x, j);
        tc_commit(&kv_empty[2u * j % NS]);
      }
      uint32_t np[2] = {0, 0};
      for (int j = 0; j < n && ok; ++j) {
        const int x0 = pair ? 0 : (j & 1), x1 = pair ? 1 : x0, jn = j + step;
        for (int x = x0; x <= x1 && ok; ++x) {
          if (!wait(&p_full[x], np[x] & 1)) break;
          ++np[x];
          if (x == x0 && !full(2 * j + 1)) break;
          pv(x, j);
          if (x == x1) tc_commit(&kv_empty[(2u * j + 1u) % NS]);
          if (jn >= n) {
            tc_commit(&o_full[x]);
          } else {
            if (x == x0 && !full(2 * jn)) break;
            qk(x, jn);
            if (x == x1) tc_commit(&kv_empty[2u * jn % NS]);
          }
        }
      }
      // every MMA issued above has completed once this barrier flips
      tc_commit(teardown);
      mbar_wait(teardown, 0, nullptr, p.status, kDrainNs);
    }
    __syncwarp();
  } else if (!F8 && warp >= kWarpClean) {
    // ------------------------------------------------------------ clean values (bf16)
    // Values of rows that not every query sees must not reach a product (0 * inf is NaN):
    // rows past the sequence are zeroed, and in the drafts' rows what is not finite (the
    // merge puts it where it belongs).
    bool ok = true;
    for (int j = first_edge; j < n; ++j) {  // (to the end: the two warps' barriers go together)
      const uint32_t s = (2 * j + 1) % NS;
      ok = ok && warp_wait(&edge_full[j - first_edge], 0, abort_flag, p.status);
      const int key0 = k_begin + j * BN;
      uint8_t* tile = sKV + s * C::TILE;
      for (int e = threadIdx.x - 32 * kWarpClean; ok && e < BN * (D / 8); e += 64) {
        // (chunks of a row in any order: all are treated alike)
        const int kb = e / (BN * 8), r = e / 8 % BN, c = e % 8;
        if (key0 + r < L) continue;
        uint4* at = reinterpret_cast<uint4*>(tile + kb * (BN * 128) + r * 128 + c * 16);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (key0 + r < k_end) {
          v = *at;
          v = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z),
                         finite_bf16x2(v.w));
        }
        *at = v;
      }
      fence_proxy_async_smem();
      asm volatile("bar.sync 3, 64;" ::: "memory");
      if (ok && threadIdx.x == 32 * kWarpClean) mbar_arrive(&kv_full[s]);
    }
  } else if (F8 && warp >= kWarpConvert) {
    // ------------------------------------------------------------ e4m3 tiles to f16
    const int tid = threadIdx.x - 32 * kWarpConvert;  // the row whose scale bytes it loads
    constexpr int G = D / 16;                         // 16-channel pieces of a row
    auto load_code = [&](int j) -> uint32_t {         // both bytes; 0 where there is no row
      const int r = k_begin + j * BN + tid;
      if (j >= n || r >= k_end) return 0u;
      const long long at = p.rows.at(b, kvh, r);
      if (at < 0) return 0u;
      return p.k_scale[at] | (static_cast<uint32_t>(p.v_scale[at]) << 8);
    };
    uint32_t code = load_code(0);
    bool ok = true;
    for (int j = 0; j < n; ++j) {  // (to the end: the four warps' barriers go together)
      const int key0 = k_begin + j * BN;
      const uint32_t next = load_code(j + 1);
      // the tile's largest codes, then every row's factor
      const int ck = code & 0xff, cv = max(static_cast<int>(code >> 8), kMinValueCode);
      const int mk = __reduce_max_sync(0xffffffffu, ck), mv = __reduce_max_sync(0xffffffffu, cv);
      if (lane == 0) {
        s_max[warp - kWarpConvert] = mk;
        s_max[4 + warp - kWarpConvert] = mv;
      }
      asm volatile("bar.sync 3, 128;" ::: "memory");
      const int Ek = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
      const int Ev = max(max(s_max[4], s_max[5]), max(s_max[6], s_max[7]));
      s_mul[tid] = row_scale(Ek - ck);
      s_mul[128 + tid] = row_scale(Ev - static_cast<int>(code >> 8));
      if (tid == 0)
        s_tile[j & 7] = make_float2(__uint_as_float(static_cast<uint32_t>(max(Ek - 7, 1)) << 23),
                                    static_cast<float>(Ev - 127));
      asm volatile("bar.sync 3, 128;" ::: "memory");
      code = next;
      for (int v = 0; v < 2 && ok; ++v) {
        const uint32_t f = 2 * j + v, rs = f % C::RAW_DEPTH, s = f % NS;
        if (!warp_wait(&raw_full[rs], (f / C::RAW_DEPTH) & 1, abort_flag, p.status) ||
            (f >= static_cast<uint32_t>(NS) &&
             !warp_wait(&kv_empty[s], (f / NS - 1) & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        const uint8_t* src = sRaw + rs * C::RAW;
        uint8_t* dst = sKV + s * C::TILE;
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int e = i * 128 + tid, r = e / G, c = e % G;
          uint4 x = *reinterpret_cast<const uint4*>(src + 16 * e);
          const uint32_t m1 = s_mul[128 * v + r], m = m1 | (m1 << 16);
          if (key0 + r >= L) {  // rows past the end: zeros; drafts' values: the finite ones
            if (key0 + r >= k_end) x = make_uint4(0u, 0u, 0u, 0u);
            if (v == 1) {
              x.x = finite_e4m3x4(x.x);
              x.y = finite_e4m3x4(x.y);
              x.z = finite_e4m3x4(x.z);
              x.w = finite_e4m3x4(x.w);
            }
          }
          const uint4 lo = make_uint4(hmul2(e4m3x2_to_f16x2(x.x), m),
                                      hmul2(e4m3x2_hi_to_f16x2(x.x), m),
                                      hmul2(e4m3x2_to_f16x2(x.y), m),
                                      hmul2(e4m3x2_hi_to_f16x2(x.y), m));
          const uint4 hi = make_uint4(hmul2(e4m3x2_to_f16x2(x.z), m),
                                      hmul2(e4m3x2_hi_to_f16x2(x.z), m),
                                      hmul2(e4m3x2_to_f16x2(x.w), m),
                                      hmul2(e4m3x2_hi_to_f16x2(x.w), m));
          // chunks 2c and 2c + 1 of the row; rows' second halves store them the other way
          // round, so that eight lanes write eight different banks
          uint8_t* at = dst + (c >> 2) * (BN * 128) + r * 128;
          const int c0 = 2 * (c & 3), flip = (c >> 2) & 1;
          *reinterpret_cast<uint4*>(at + (((c0 + flip) ^ (r & 7)) << 4)) = flip ? hi : lo;
          *reinterpret_cast<uint4*>(at + (((c0 + 1 - flip) ^ (r & 7)) << 4)) = flip ? lo : hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&kv_full[s]);
          mbar_arrive(&raw_empty[rs]);
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;  // of the query tile
    const int M = p.T * p.rep;
    const int qrow = rb * (pair ? 256 : 128) + (pair ? x * 128 : 0) + row;
    const bool live = qrow < M;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const int t = live ? qrow / p.rep : 0;
    const int h = kvh * p.rep + (live ? qrow - t * p.rep : 0);
    const size_t qi = (static_cast<size_t>(b) * p.Hq + h) * p.T + t;
    if (pair || x == 0) {
      // the row's query, 16-byte chunks in the swizzled layout of a K-major operand
      uint8_t* dst = sQ + (pair ? x : 0) * C::TILE + row * 128;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + qi * D);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = live ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(dst + (c >> 3) * (BN * 128) + (((c & 7) ^ (row & 7)) << 4)) = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_ready[pair ? x : 0]);
    }
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128u * x;
    const uint32_t tO = tmem + lane_off + 256u + static_cast<uint32_t>(D) * x;
    float row_factor = p.scale_log2;
    if (F8) row_factor *= p.q_factor[qi];
    const uint32_t* anc = p.anc + (static_cast<size_t>(b) * p.T + t) * p.words;

    float R = -INFINITY, l = 0.f;
    uint32_t ns = 0;
    bool ok = true;
    for (int j = pair ? 0 : x; j < n; j += step) {
      if (!warp_wait(&s_full[x], ns & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      ++ns;
      tc_fence_after();
      if (warp_live) {
        float c = row_factor, ev = 0.f;
        if constexpr (F8) {
          const float2 ts = s_tile[j & 7];
          c *= ts.x;
          ev = ts.y;
        }
        c = fmaxf(c, 1.17549435e-38f);  // (a hidden score's -inf times 0 would be NaN)
        const int key0 = k_begin + j * BN;
        const bool edge = j >= first_edge;
        // the rows that this query does not see
        uint32_t hide[4] = {0u, 0u, 0u, 0u};
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k0 = key0 + 32 * i;
            uint32_t see = k0 + 32 <= k_end ? 0xffffffffu
                           : k0 >= k_end    ? 0u
                                            : (1u << (k_end - k0)) - 1u;
            hide[i] = ~(see & draft_bits32(anc, p.words, k0 - L));
          }
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t r[64];
          tmem_ld64_sync(tS + 64u * i, r);
          if (edge) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if ((hide[2 * i + (e >> 5)] >> (e & 31)) & 1u) r[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 64; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mq[k] = fmax3(mq[k], __uint_as_float(r[e + k]), __uint_as_float(r[e + 4 + k]));
        }
        const float top = __fmul_rn(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])), c) + ev;
        const bool mine = top > R + kRescaleThreshold;
        if (__any_sync(0xffffffffu, mine)) {
          const float f = mine ? ex2_approx(R - top) : 1.f;
          l *= f;
          if (ns > 1) {
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              uint32_t r[32];
              tmem_ld32_sync(tO + 32u * i, r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tmem_st32(tO + 32u * i, r);
            }
            tmem_st_wait();
          }
          if (mine) R = top;
        }
        // (nothing seen yet: 2^-inf = 0, and a NaN score stays NaN)
        const float off = (F8 ? ev + 7.f : 0.f) - (R == -INFINITY ? 0.f : R);
        float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t r[32], pk[16];
          tmem_ld32_sync(tS + 32u * i, r);
          if (edge) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((hide[i] >> e) & 1u) r[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float y0, y1;
            // (two roundings, as in `top`: the largest gives 2^0)
            fmul2(y0, y1, __uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]), c);
            fadd2(y0, y1, y0, y1, off, off);
            const float w0 = ex2_approx(y0), w1 = ex2_approx(y1);
            if (e & 1)
              fadd2(sb0, sb1, sb0, sb1, w0, w1);
            else
              fadd2(sa0, sa1, sa0, sa1, w0, w1);
            pk[e] = F8 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1);
          }
          tmem_st16(tS + 16u * i, pk);
        }
        const float sum = (sa0 + sa1) + (sb0 + sb1);
        l += F8 ? sum * ex2_approx(-ev - 7.f) : sum;
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[x]);
    }
    // partial result: R, l and O, relative to 2^R
    const float o_scale = F8 ? 1.f / 16384.f : 1.f;  // 2^-7 of w, 2^-7 of V16
    if (!pair) {
      if (x == 1) s_ml[row] = make_float2(R, l);
      asm volatile("bar.sync 2, 256;" ::: "memory");  // (every softmax warp gets here)
    }
    if (ok && (pair || x == 0) && warp_live &&
        warp_wait(&o_full[x], 0, abort_flag, p.status) &&
        (pair || n < 2 || warp_wait(&o_full[1], 0, abort_flag, p.status))) {
      tc_fence_after();
      float f0 = o_scale, f1 = 0.f;
      if (!pair && n > 1) {
        const float2 other = s_ml[row];
        const float m = fmaxf(R, other.x);
        // (a stream that saw nothing holds zeros, or NaN)
        const float e0 = R == -INFINITY ? 1.f : ex2_approx(R - m);
        const float e1 = other.x == -INFINITY ? 1.f : ex2_approx(other.x - m);
        l = l * e0 + other.y * e1;
        R = m;
        f0 = o_scale * e0;
        f1 = o_scale * e1;
      }
      const size_t at = qi * static_cast<size_t>(p.n_splits) + split;
      float* dst = p.part_o + at * D;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t r[32];
        tmem_ld32_sync(tO + 32u * i, r);
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(r[e]) * f0;
        if (!pair && n > 1) {
          tmem_ld32_sync(tO + D + 32u * i, r);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(r[e]), f1, o[e]);
        }
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(dst + 32 * i + e) =
                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (live) {
        p.part_ml[2 * at] = R;
        p.part_ml[2 * at + 1] = l;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool F8>
cudaError_t launch_t(const GroupArgs& a, cudaStream_t stream) {
  using C = Cfg<D, F8>;
  TParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_factor = a.q_factor;
  p.lens = a.lens;
  p.anc = a.anc;
  p.rows = CacheRows{a.cache.block_table, a.Hkv, a.cache.Lmax, a.cache.page_size,
                     a.cache.num_pages, a.cache.max_pages};
  p.k_scale = static_cast<const uint8_t*>(a.cache.k_scale);
  p.v_scale = static_cast<const uint8_t*>(a.cache.v_scale);
  p.drafts = a.drafts;
  p.words = a.words;
  const bool paged = a.cache.block_table != nullptr;
  const int ps = a.cache.page_size;
  p.box_rows = !paged || ps % BN == 0 ? BN : (ps < 64 ? ps : 64);
  p.part_o = a.part_o;
  p.part_ml = a.part_ml;
  p.status = a.status;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.T = a.T;
  p.rep = a.Hq / a.Hkv;
  p.max_seq_len = a.max_seq_len;
  p.min_len = a.min_len;
  p.chunk = a.chunk;
  p.n_splits = a.n_splits;
  const int rows = a.T * p.rep;
  p.pair = rows > 128 ? 1 : 0;
  p.rblocks = (rows + 255) / 256;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);

  alignas(64) CUtensorMap tk, tv;
  const int trows = paged ? ps : a.cache.Lmax;
  const int planes = paged ? a.cache.num_pages * a.Hkv : a.B * a.Hkv;
  const bool made = F8 ? make_tmap_u8_3d(&tk, a.cache.k, D, trows, planes, p.box_rows, false) &&
                             make_tmap_u8_3d(&tv, a.cache.v, D, trows, planes, p.box_rows, false)
                       : make_tmap_bf16_3d(&tk, a.cache.k, D, trows, planes, p.box_rows) &&
                             make_tmap_bf16_3d(&tv, a.cache.v, D, trows, planes, p.box_rows);
  if (!made) return cudaErrorInvalidValue;
  static SmemLimitOnce smem_limit;
  cudaError_t e = smem_limit.set(group_tc_kernel<D, F8>, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_splits) * p.rblocks, a.Hkv, a.B);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.after_prep ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, group_tc_kernel<D, F8>, p, tk, tv);
}

}  // namespace

cudaError_t launch_group_tc(const GroupArgs& a, cudaStream_t stream) {
  const bool f8 = a.cache.k_scale != nullptr;
  if (a.d == 64) return f8 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
  return f8 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
}

}  // namespace csattn
