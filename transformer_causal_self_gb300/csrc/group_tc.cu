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
// One CTA per SM; the CTAs take equal ranges of all the tiles (group_work.cuh), and the rings
// and barriers run on from one piece to the next:
//   warps 0-3, 4-7  softmax of stream 0 and 1, a query row per thread, and the partial results
//                   at a piece's end
//   warp 8          TMA producer          warp 9   TMEM owner and MMA issuer
//   warps 10-11     bf16: clean the values of tiles that not every query sees
//                   e4m3: scale bytes of every second tile
//   warps 12-15     e4m3: take the keys' tiles to f16;  warps 16-19  the values'
// TMEM columns: S_0 [0,128) S_1 [128,256) O_0 [256,256+D) O_1 [256+D,256+2D); P overwrites the
// first half of its S and is read by the second product from there.
//
// An e4m3 tile becomes f16 with one scale for all its rows: row j is multiplied by 2^(7 - (E -
// e_j)), E the largest exponent of the tile (at least -102 for values).  That is exact while
// e_j is within 22 of E.  So the scales reach the softmax as two numbers per tile, and one
// exponential serves denominator and numerator:
//   w = 2^(x + E_v - R), O += w V16, l += 2^(-E_v) * sum w, R the running maximum of x + E_v.
// R is raised only by more than 2^8, as elsewhere; w is then at most 2^8 (bf16), or 2^15 with
// the 2^7 that the e4m3 path adds for f16's range.  Where x + E_v is so far below R that w would
// leave fp32's range (small values beside large ones), a tile's weights are taken relative to its
// own maximum: its values vanish beside the others, its share of l need not.
// A tile whose rows are further apart (values: by more than 2^12, where R, which counts E_v
// whether a query sees the largest row or not, would cost the others' weights bits of f16) keeps
// its rows as they are, times 2^7, and the softmax takes every column's exponents from the scale
// bytes: x_j = S_j 2^(e_j - 7), w_j = 2^(x_j + ev_j - R), R over the columns that the query sees,
// and a second exponential for l.  So a draft that a query does not see, or padding, has no part
// in its output however large it is.  Rows of the least code (zeros) do not count as far apart.
//
// A 128-row tile of 128 channels takes an SM (slope from 8000 to 24000 rows) 1.38 us with up to 128
// query rows over bf16 (HBM) and 1.85 with 256 (1380 TFLOP/s: 32 products of N = 128, which at one
// in 118 cycles take 1.82 us; one rounding less in the softmax changed nothing); over e4m3 1.29
// (half the bytes; the tiles' way through shared memory, raw and as f16, is 0.87, the rest is the
// chain copy, conversion, S, softmax, O) and 2.00.  64 channels: 0.78, 1.22, 0.97, 1.59 us.  A
// piece adds 3 to 6 us: partial results, next scores.
#include "fp8.cuh"
#include "internal.h"

namespace csattn {
namespace {

constexpr int BN = 128;  // cache rows per tile
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 100000000ull;
constexpr float kRescaleThreshold = 8.0f;
// e4m3: below R by kLowTile (2^(7 - 96 - 30) is still a normal number) the largest weight of a tile
// is put at 2^-kLowWeight, which is 0 in f16
constexpr float kLowTile = 96.0f, kLowWeight = 60.0f;
constexpr int kMinValueCode = 25;  // E_v >= -102 (the least code is within 22 of it)
constexpr int kWideKeys = 22, kWideValues = 12;  // exponents further apart: a column each;
constexpr float kOwnScales = 1000.f;              // such a tile's E_v
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpClean = 10, kWarpConvert = 12;

template <int D, bool F8>
struct Cfg {
  // e4m3: 640 threads have 96 registers each; some of the others' go to the softmax
  // (2*136 + 64 + 2*72 = 5*96; a tile took 1.57 us, 1.58-1.69 with 112..144 there, 2.0 with none
  // moved, when this was chosen)
  static constexpr int kThreads = F8 ? 640 : 384;
  static constexpr int TILE = BN * D * 2;  // a Q, K or V tile of 16-bit values
  static constexpr int RAW = BN * D;       // an e4m3 tile
  // raw tiles: as much as four of 128 channels (with eight of 64 the warps that read the scale
  // bytes are far enough ahead: 8 x 32 drafts over 8000 rows, 64-row pages, 48.9 -> 45.0 us)
  static constexpr int NRAW = F8 ? 512 / D : 0;
  // ring tiles that fit beside one or two query tiles
  static constexpr int NS1 = F8 ? 4 : (D == 128 ? 6 : 8);
  static constexpr int NS2 = F8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);
  static constexpr int TILES = (NS1 + 1 > NS2 + 2 ? NS1 + 1 : NS2 + 2) * TILE + NRAW * RAW;
  static constexpr int BARS = NRAW > 4 ? 384 : 336;
  static constexpr int SMEM = 1024 + TILES + BARS + 128 * 8 + (F8 ? 8 * 8 + NRAW * BN : 0);
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

struct TParams {
  const float* q_factor;
  const uint32_t* anc;
  GroupLine line;
  CacheRows rows;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int words, scale_words;  // scale_words: four rows' scale bytes can be read as a word
  int box_rows;
  float* part_o;
  float* part_ml;
  uint32_t* status;
  int Hq, Hkv, T, rep, rblocks, part_rows, pair;
  int lost;  // arrivals that the queries' barrier waits for and nothing makes (selftest)
  float scale_log2;
};

// What a piece is to every role.
struct View {
  int b, kvh, rb;            // sequence, KV head, block of query rows
  int L, total;              // rows every query sees, and with the drafts
  int k_begin, k_end, n;     // cache rows and tiles of the piece
  int first_edge;            // first tile with rows that not every query sees
  __device__ __forceinline__ View(const GroupPiece& pc, const TParams& p)
      : b(pc.b), kvh(pc.head / p.rblocks), rb(pc.head - kvh * p.rblocks), L(pc.L),
        total(pc.L + p.line.drafts), k_begin(pc.t0 * BN),
        k_end(min(total, k_begin + pc.n * BN)), n(pc.n),
        first_edge(max(0, min(n, (min(L, k_end) - k_begin) / BN))) {}
};

// f16 or bf16 operands, fp32 accumulators, M = 128
constexpr uint32_t idesc(bool f16, int N, int b_mn) {
  return idesc_bf16_f32(128, N, 0, b_mn) & (f16 ? ~((7u << 7) | (7u << 10)) : ~0u);
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
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

// A TMEM load of 32 columns in two halves: issue, and the wait after which the registers hold
// the columns (named in the wait, so that no use can be scheduled before it).
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// -inf into the scores of 32 columns whose bit in `hide` is set
__device__ __forceinline__ void mask_scores(uint32_t taddr, uint32_t hide) {
  uint32_t r[32];
  tmem_ld32_sync(taddr, r);
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if ((hide >> e) & 1u) r[e] = 0xff800000u;
  tmem_st32(taddr, r);
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

// Scale bytes of a tile, four rows in each lane of a warp (0 where there is no row): the largest
// (at least `least`), and whether one of the lane's rows is more than `limit` below it.
struct TileScale {
  int E;
  bool far;
  __device__ __forceinline__ TileScale(uint32_t four, int least, int limit) {
    const uint32_t a = four & 0xff00ffu, b = (four >> 8) & 0xff00ffu;
    const uint32_t hi = __vmaxu2(a, b);
    E = max(static_cast<int>(__reduce_max_sync(0xffffffffu, max(hi & 0xffffu, hi >> 16))), least);
    // 4 is taken off each half, so that codes up to kScaleMin wrap round to the top.  (The upper
    // half loses 5 where the lower one does not carry: code 4 may go with them, and others are
    // far one octave earlier.)
    static_assert(kScaleMin == 3, "codes that do not count");
    const uint32_t lo = __vminu2(a + 0xfffbfffcu, b + 0xfffbfffcu);
    far = E - 4 - static_cast<int>(min(lo & 0xffffu, lo >> 16)) > limit;
  }
};

__device__ __forceinline__ void tmem_ld4_sync(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st2(uint32_t taddr, const uint32_t (&r)[2]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1])
               : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// The softmax of a tile whose columns keep scales of their own (see the file's head), for the
// thread's row: S in TMEM becomes the weights, R and l (and O, if there is one) are brought up to
// date; returns R and l.  Out of line: these tiles are rare, and inline the softmax loop no longer
// fits the instruction cache as well (16 x 32 drafts over 512..8192 rows: 76.8 us with it inline,
// 73.8 like this, when this was chosen).  A row far away in every tile costs 25 % of such a step,
// every second row far away 80 %.
template <int D>
__device__ __noinline__ float2 own_scales(const TParams& p, int b, int kvh, int row0, int k_end,
                                          uint32_t tS, uint32_t tO, bool has_o, float row_factor,
                                          float R, float l) {
  const int lane = threadIdx.x & 31, r = row0 + 4 * lane;
  uint32_t own_k = 0u, own_v = 0u;  // four rows' codes (no page ends inside them)
  const long long at = r < k_end ? p.rows.at(b, kvh, r) : -1;
  for (int i = 0; at >= 0 && i < 4 && r + i < k_end; ++i) {
    own_k |= static_cast<uint32_t>(p.k_scale[at + i]) << (8 * i);
    own_v |= static_cast<uint32_t>(p.v_scale[at + i]) << (8 * i);
  }
  __syncwarp();
  const TileScale sk(own_k, 0, kWideKeys), sv(own_v, kMinValueCode, kWideValues);
  if (!__any_sync(0xffffffffu, sk.far)) own_k = 0x01010101u * sk.E;
  own_v = __any_sync(0xffffffffu, sv.far) ? __vmaxu4(own_v, 0x01010101u * kMinValueCode)
                                          : 0x01010101u * sv.E;
  __syncwarp();
  float top = -INFINITY;
  for (int i = 0; i < BN; i += 4) {  // y_j = x_j + ev_j
    const uint32_t ek = __shfl_sync(0xffffffffu, own_k, i >> 2);
    const uint32_t ev = __shfl_sync(0xffffffffu, own_v, i >> 2);
    uint32_t s4[4];
    tmem_ld4_sync(tS + i, s4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f = __uint_as_float(((ek >> (8 * e)) & 0xffu) << 23);
      // (neither 0 nor infinity: a hidden score is -inf, another may be 0)
      const float g = fminf(fmaxf(row_factor * f * 0.0078125f, 1.17549435e-38f), 3e38f);
      const float y = __fmul_rn(__uint_as_float(s4[e]), g) +
                      (static_cast<float>((ev >> (8 * e)) & 0xffu) - 127.f);
      top = fmaxf(top, y);
      s4[e] = __float_as_uint(y);
    }
    tmem_st4(tS + i, s4);
  }
  tmem_st_wait();
  const bool mine = top > R + kRescaleThreshold;
  if (__any_sync(0xffffffffu, mine)) {
    const float f = mine ? ex2_approx(0.5f * (R - top)) : 1.f;
    l = l * f * f;
    if (mine) R = top;
    __syncwarp();
    for (int i = 0; has_o && i < D; i += 4) {
      uint32_t o4[4];
      tmem_ld4_sync(tO + i, o4);
#pragma unroll
      for (int e = 0; e < 4; ++e) o4[e] = __float_as_uint(__uint_as_float(o4[e]) * f * f);
      tmem_st4(tO + i, o4);
    }
  }
  // w_j = 2^(y_j - R), and 2^x_j by way of y_j - top, then - ev_j (-120 <= -ev_j <= 102, so times
  // 2^18): beside a large score ev_j is lost in y_j
  const float Rn = R == -INFINITY ? 0.f : R, at0 = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  __syncwarp();
  for (int i = 0; i < BN; i += 4) {
    const uint32_t ev = __shfl_sync(0xffffffffu, own_v, i >> 2);
    uint32_t s4[4];
    float w[4];
    tmem_ld4_sync(tS + i, s4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y = __uint_as_float(s4[e]);
      sum += ex2_approx((y - at0) + (145.f - static_cast<float>((ev >> (8 * e)) & 0xffu)));
      w[e] = ex2_approx((y - Rn) + 7.f);
    }
    const uint32_t pk[2] = {pack_f16x2(w[0], w[1]), pack_f16x2(w[2], w[3])};
    tmem_st2(tS + i / 2, pk);
  }
  tmem_st_wait();
  const float g = top == -INFINITY ? 1.f : ex2_approx(0.5f * (top - R));
  return make_float2(R, l + sum * (1.f / 262144.f) * g * g);
}

// 2^(7 - below) in f16 (0 where that is less than f16's least)
__device__ __forceinline__ uint16_t row_scale(int below) {
  return __half_as_ushort(
      __float2half_rn(below > 60 ? 0.f : __uint_as_float((127u + 7u - below) << 23)));
}

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, 1)
    group_tc_kernel(const __grid_constant__ TParams p, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
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
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* s_full = bars + 2;     // [2]
  uint64_t* p_full = bars + 4;     // [2]
  uint64_t* o_full = bars + 6;     // [2]
  uint64_t* o_empty = bars + 8;    // [2]
  uint64_t* teardown = bars + 10;
  uint64_t* kv_full = bars + 11;   // [8]
  uint64_t* kv_empty = bars + 19;  // [8]
  constexpr int kRaw = C::NRAW > 4 ? C::NRAW : 4;
  uint64_t* raw_full = bars + 27;            // [kRaw]
  uint64_t* raw_empty = raw_full + kRaw;     // [kRaw]
  uint64_t* edge_full = raw_empty + kRaw;    // [4] bf16: values to be cleaned, edge by edge tile
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(edge_full + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::TILES + C::BARS);  // [128]
  float2* s_tile = s_ml + 128;  // e4m3 [8]: 2^E_k, E_v (or kOwnScales) of a tile
  uint8_t* s_below = reinterpret_cast<uint8_t*>(s_tile + 8);  // [NRAW][BN]: rows of raw tiles
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_empty[x], pair ? 4 : 8);
    }
    mbar_init(teardown, 1);
    mbar_init(q_full, 1 + p.lost);
    mbar_init(q_empty, 1);
    for (int s = 0; s < 8; ++s) {
      mbar_init(&kv_full[s], F8 ? 4 : 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&raw_full[s], F8 ? 2 : 1);
      mbar_init(&raw_empty[s], 4);
      mbar_init(&edge_full[s], 1);
    }
    for (int s = 4; s < C::NRAW; ++s) {
      mbar_init(&raw_full[s], 2);
      mbar_init(&raw_empty[s], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  GroupPiece pc = group_start(p.line, p.status, true);  // (n = 0: every loop below ends at once)
  const int step = pair ? 1 : 2;  // between a stream's tiles

  if (warp >= 8 && warp < 12) {
    if constexpr (F8) regs_dec<64>();
    if (warp == kWarpProducer) {
      // ------------------------------------------------------------ TMA producer
      // fills K_0, V_0, K_1, V_1, ...; lane i copies box i of a tile (see group_attn.cu)
      // (8 sequences of 8192-16384 rows, 256 query rows: 109.8 -> 106.8 us; two row blocks that read
      // the same tiles are no slower)
      const uint64_t once = evict_first_policy();
      const CacheRows& R = p.rows;
      const int nbox = BN / p.box_rows, r0 = lane * p.box_rows;
      const uint32_t depth = F8 ? C::NRAW : NS;
      uint64_t* full = F8 ? raw_full : kv_full;
      uint64_t* empty = F8 ? raw_empty : kv_empty;
      uint32_t f = 0, edges = 0, piece = 0, queries = 0;
      uint64_t recent = 0;  // a byte per fill, the latest lowest: 8 + (edge % 8), or 0
      bool ok = true;
      // The piece's queries, once the products with the last piece's are done: behind its first
      // tile, so that this wait does not hold that up.
      auto load_queries = [&](const View& w) {
        bool done = true;
        if (lane == 0 && queries > 0)
          done = ctl_wait(q_empty, (queries - 1) & 1, abort_flag, p.status, kWaitNs);
        if (!__all_sync(0xffffffffu, done)) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, (1 + pair) * C::TILE);
          for (int x = 0; x <= pair; ++x)
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_3d(sQ + x * C::TILE + kb * (BN * 128), &tm_q, q_full, kb * 64,
                          (w.rb * (1 + pair) + x) * BN, w.b * p.Hkv + w.kvh);
        }
        ++queries;
        __syncwarp();
        return true;
      };
      // (the kernel before wrote queries and the drafts' rows by plain stores)
      asm volatile("fence.proxy.async.global;" ::: "memory");
      if (pc.n > 0) load_queries(View(pc, p));
      for (; pc.n > 0 && ok; pc.next(p.line), ++piece) {
        const View w(pc, p);
        for (int j = 0; j < w.n && ok; ++j) {
          if (j == 1 && piece > 0 && !(ok = load_queries(w))) break;
          int plane = w.b * p.Hkv + w.kvh, prow = w.k_begin + j * BN;
          if (lane < nbox && R.block_table != nullptr) {
            const int tr = prow + r0;
            plane = R.num_pages * p.Hkv;
            prow = 0;
            if (tr < w.total) {
              const int page =
                  R.block_table[static_cast<size_t>(w.b) * R.max_pages + tr / R.page_size];
              if (page >= 0 && page < R.num_pages)
                plane = page * p.Hkv + w.kvh;
              else
                atomicOr(p.status, kStatusDeviceArg);
              prow = tr % R.page_size;
            }
          }
          for (int v = 0; v < 2; ++v, ++f) {
            const uint32_t s = f % depth, use = f / depth;
            // bf16 values of edge tiles go by way of the cleaning warps
            const bool edge = !F8 && v == 1 && j >= w.first_edge;
            uint64_t* landed = edge ? &edge_full[edges & 3] : &full[s];
            int okw = 1;
            if (lane == 0) {
              if (use > 0 && !ctl_wait(&empty[s], (use - 1) & 1, abort_flag, p.status, kWaitNs))
                okw = 0;
              else
                mbar_arrive_expect_tx(landed, F8 ? C::RAW : C::TILE);
            }
            if (!__shfl_sync(0xffffffffu, okw, 0)) {
              ok = false;
              break;
            }
            const CUtensorMap* tm = v == 0 ? &tm_k : &tm_v;
            if (lane < nbox) {
              if constexpr (F8) {
                tma_load_3d_once(sRaw + s * C::RAW + r0 * D, tm, landed, 0, prow, plane, once);
              } else {
                for (int kb = 0; kb < D / 64; ++kb)
                  tma_load_3d_once(sKV + s * C::TILE + kb * (BN * 128) + r0 * 128, tm, landed,
                                   kb * 64, prow, plane, once);
              }
            }
            recent = (recent << 8) | (edge ? 8u + (edges & 7u) : 0u);
            edges += edge;
            __syncwarp();
          }
        }
        if (ok && w.n == 1 && piece > 0) ok = load_queries(w);
      }
      if (lane == 0 && *abort_flag) {
        // every copy still in flight lands before the CTA's shared memory is released
        for (uint32_t i = 1; i <= depth && i <= f; ++i, recent >>= 8) {
          const uint32_t e = recent & 15u;
          mbar_wait(e ? &edge_full[e & 3u] : &full[(f - i) % depth],
                    e ? (e >> 2) & 1u : ((f - i) / depth) & 1u, nullptr, p.status, kDrainNs);
        }
        if (queries > 0) mbar_wait(q_full, (queries - 1) & 1, nullptr, p.status, kDrainNs);
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp keeps the books, so that addresses stay in uniform registers; one lane
      // issues.  Descriptors differ in their low words alone, by constants within a product, and
      // all waits of a step come ahead of its products: the tensor core's queue is short.
      const bool leader = elect_one();
      const uint64_t hi = smem_desc_sw128(0, 16, 1024), hi_v = smem_desc_sw128(0, BN * 128, 1024);
      const uint32_t q_lo = smem_u32(sQ) >> 4, kv_lo = smem_u32(sKV) >> 4;
      constexpr uint32_t kIdS = idesc(F8, BN, 0), kIdO = idesc(F8, D, 1);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = warp_wait(bar, parity, abort_flag, p.status);
        return ok;
      };
      auto full = [&](uint32_t f) { return wait(&kv_full[f % NS], (f / NS) & 1); };
      // S_x = Q K^T with the keys of fill f
      auto qk = [&](int x, uint32_t f) {
        const uint64_t q = hi + q_lo + (pair ? x : 0) * (C::TILE >> 4);
        const uint64_t k = hi + kv_lo + (f % NS) * (C::TILE >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = static_cast<uint32_t>((kk >> 2) * (BN * 8) + (kk & 3) * 2);
            umma_ss(tmem + 128u * x, q + off, k + off, kIdS, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[x]);
        }
        __syncwarp();
      };
      auto pv = [&](int x, uint32_t f, bool accumulate) {
        const uint64_t v = hi_v + kv_lo + (f % NS) * (C::TILE >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            umma_ts(tmem + 256u + D * x, tmem + 128u * x + 8u * kk, v + 128u * kk, kIdO,
                    (accumulate || kk > 0) ? 1u : 0u);
        }
        __syncwarp();
      };
      auto release = [&](uint64_t* bar) {  // when what has been issued is done
        if (leader) tc_commit(bar);
        __syncwarp();
      };
      uint32_t F = 0, np[2] = {0, 0}, used[2] = {0, 0}, piece = 0;
      for (; pc.n > 0 && ok; pc.next(p.line), ++piece) {
        const int n = pc.n;
        wait(q_full, piece & 1);
        // first tiles of both streams
        for (int j = 0; j < step && j < n; ++j) {
          if (!full(F + 2 * j)) break;
          tc_fence_after();
          for (int x = pair ? 0 : j; x <= (pair ? 1 : j); ++x) qk(x, F + 2 * j);
          release(&kv_empty[(F + 2 * j) % NS]);
          if (j == n - 1) release(q_empty);
        }
        for (int j = 0; j < n && ok; ++j) {
          const int x0 = pair ? 0 : (j & 1), x1 = pair ? 1 : x0, jn = j + step;
          if (!full(F + 2 * j + 1) || (jn < n && !full(F + 2 * jn))) break;
          for (int x = x0; x <= x1 && ok; ++x) {
            // the stream's first tile of a piece: its O has been read
            if (j < step) {
              if (used[x] > 0 && !wait(&o_empty[x], (used[x] - 1) & 1)) break;
              ++used[x];
            }
            if (!wait(&p_full[x], np[x] & 1)) break;
            ++np[x];
            tc_fence_after();
            pv(x, F + 2 * j + 1, j >= step);
            if (x == x1) release(&kv_empty[(F + 2 * j + 1) % NS]);
            if (jn >= n) {
              release(&o_full[x]);
            } else {
              qk(x, F + 2 * jn);
              if (x == x1) {
                release(&kv_empty[(F + 2 * jn) % NS]);
                if (jn == n - 1) release(q_empty);
              }
            }
          }
        }
        F += 2 * n;
      }
      // every MMA issued above has completed once this barrier flips
      release(teardown);
      if (leader) mbar_wait(teardown, 0, nullptr, p.status, kDrainNs);
      __syncwarp();
    } else if (F8) {
      if constexpr (F8) {
        // ---------------------------------------------------------- scale bytes (e4m3)
        // Of every tile: the exponents that the softmax needs (s_tile), and how far every row is
        // below its tile's largest (s_below: a byte per row and raw tile), with the raw tiles'
        // barriers as the copies.  The two warps take every second tile (8 sequences of 8000 rows,
        // 64 channels, 20 query rows: 50.1 us, 54.3 with one warp for all).
        const int ps = p.rows.block_table != nullptr ? p.rows.page_size : 0;
        bool ok = true;
        uint32_t tile0 = 0;
        for (; pc.n > 0 && ok; tile0 += pc.n, pc.next(p.line)) {
          const View w(pc, p);
          const int first = (warp - kWarpClean + tile0) & 1;  // of the warp's tiles
          // Four rows per lane (no page ends inside them), packed.  The page number comes first, so
          // each of the two loads is issued a tile ahead of its use, and taken over at the tile's
          // end (a register move waits for a load).
          const int row0 = w.k_begin + first * BN + 4 * lane;
          int pg = ps > 0 ? row0 / ps : 0, ofs = row0 - pg * ps;  // of the next page lookup
          const int32_t* const table =
              p.rows.block_table + static_cast<size_t>(w.b) * p.rows.max_pages;
          auto load_page = [&](int i) -> int {  // of the warp's i-th tile
            const int page = ps > 0 && row0 + 2 * i * BN < w.k_end ? table[pg] : 0;
            if (ps >= BN) {
              ofs += 2 * BN;
              while (ofs >= ps) ++pg, ofs -= ps;
            } else if (ps > 0) {
              pg += 2 * BN / ps;
            }
            return page;
          };
          // four rows' bytes of an array; 0 where there is no row
          auto load_codes = [&](const uint8_t* scale, int i, int page, int at_ofs) -> uint32_t {
            const int r = row0 + 2 * i * BN, left = w.k_end - r;
            if (left <= 0) return 0u;
            size_t at;
            if (ps == 0) {
              at = (static_cast<size_t>(w.b) * p.Hkv + w.kvh) * p.rows.Lmax + r;
            } else {
              if (page < 0 || page >= p.rows.num_pages) return 0u;
              at = (static_cast<size_t>(page) * p.Hkv + w.kvh) * ps + at_ofs;
            }
            if (p.scale_words) return *reinterpret_cast<const uint32_t*>(scale + at);
            uint32_t x = 0u;
            for (int e = 0; e < min(left, 4); ++e)
              x |= static_cast<uint32_t>(scale[at + e]) << (8 * e);
            return x;
          };
          auto valid = [&](int i) -> uint32_t {  // bytes of rows there are
            const int left = w.k_end - (row0 + 2 * i * BN);
            return left >= 4 ? ~0u : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
          };
          int ofs1 = ofs;
          int page = load_page(0);
          uint32_t ck = load_codes(p.k_scale, 0, page, ofs1);
          uint32_t cv = load_codes(p.v_scale, 0, page, ofs1);
          ofs1 = ofs;
          page = load_page(1);
          for (int i = 0; first + 2 * i < w.n; ++i) {
            const uint32_t tile = tile0 + first + 2 * i;
            const uint32_t nk = load_codes(p.k_scale, i + 1, page, ofs1);
            const uint32_t nv = load_codes(p.v_scale, i + 1, page, ofs1);
            const uint32_t there = valid(i);
            ck &= there;
            cv &= there;
            const int ofs2 = ofs;
            const int page_next = load_page(i + 2);
            const TileScale sk(ck, 0, kWideKeys), sv(cv, kMinValueCode, kWideValues);
            const bool wide_k = __any_sync(0xffffffffu, sk.far);
            const bool wide_v = __any_sync(0xffffffffu, sv.far);
            // (no byte borrows: E is the largest; rows of their own scale: 2^7, or the floor's)
            const uint32_t below[2] = {
                wide_k ? 0u : 0x01010101u * sk.E - ck,
                (wide_v ? __vmaxu4(cv, 0x01010101u * kMinValueCode) : 0x01010101u * sv.E) - cv};
            for (int v = 0; v < 2; ++v) {
              const uint32_t f = 2 * tile + v, rs = f % C::NRAW;
              if (f >= C::NRAW)
                ok = warp_wait(&raw_empty[rs], (f / C::NRAW - 1) & 1, abort_flag, p.status);
              if (!ok) break;
              reinterpret_cast<uint32_t*>(s_below)[BN / 4 * rs + lane] = below[v];
              if (v == 0 && lane == 0)
                s_tile[tile & 7] =
                    make_float2(__uint_as_float(static_cast<uint32_t>(sk.E) << 23),
                                wide_k || wide_v ? kOwnScales : static_cast<float>(sv.E - 127));
              __syncwarp();
              if (lane == 0) mbar_arrive(&raw_full[rs]);
            }
            if (!ok) break;
            ck = nk;
            cv = nv;
            page = page_next;
            ofs1 = ofs2;
          }
        }
      }
    } else {
      // ------------------------------------------------------------ clean values (bf16)
      // Values of rows that not every query sees must not reach a product (0 * inf is NaN):
      // rows past the sequence are zeroed, and in the drafts' rows what is not finite (the
      // merge puts it where it belongs).
      bool ok = true;
      uint32_t F = 0, edges = 0;
      for (; pc.n > 0; pc.next(p.line)) {  // (to the end: the two warps' barriers go together)
        const View w(pc, p);
        for (int j = w.first_edge; j < w.n; ++j, ++edges) {
          const uint32_t s = (F + 2 * j + 1) % NS;
          ok = ok && warp_wait(&edge_full[edges & 3], (edges >> 2) & 1, abort_flag, p.status);
          const int key0 = w.k_begin + j * BN;
          uint8_t* tile = sKV + s * C::TILE;
          for (int e = threadIdx.x - 32 * kWarpClean; ok && e < BN * (D / 8); e += 64) {
            // (chunks of a row in any order: all are treated alike)
            const int kb = e / (BN * 8), r = e / 8 % BN, c = e % 8;
            if (key0 + r < w.L) continue;
            uint4* at = reinterpret_cast<uint4*>(tile + kb * (BN * 128) + r * 128 + c * 16);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (key0 + r < w.k_end) {
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
        F += 2 * w.n;
      }
    }
  } else if (warp >= kWarpConvert) {
    // ------------------------------------------------------------ e4m3 tiles to f16
    if constexpr (F8) {
      regs_dec<72>();
      const int v = (warp - kWarpConvert) >> 2;  // 0: keys, 1: values
      const int tid = (threadIdx.x - 32 * kWarpConvert) & 127;
      constexpr int G = D / 16;                  // 16-channel pieces of a row
      const uint32_t raw0 = smem_u32(sRaw), kv0 = smem_u32(sKV);
      // The thread's piece: column c of row r0.  Eight lanes share a wavefront, and a row's pieces
      // c and c + 4 go to the same banks (to the tile's two halves); so at 128 channels two rows
      // change places in their upper four pieces, and odd rows' chunks lie between even ones'.
      const int c = tid % G;
      const int r0 = D == 128 ? 2 * (tid >> 4) + (((tid >> 2) ^ (tid >> 3)) & 1) : tid / G;
      uint32_t to0, to1;                         // where the thread's two chunks go in a tile
      {
        const uint32_t at = (c >> 2) * (BN * 128) + r0 * 128;
        to0 = at + (((2 * (c & 3)) ^ (r0 & 7)) << 4);
        to1 = at + (((2 * (c & 3) + 1) ^ (r0 & 7)) << 4);
      }
      bool ok = true;
      uint32_t f = v;                            // its next fill
      for (; pc.n > 0 && ok; pc.next(p.line)) {
        const View w(pc, p);
        for (int j = 0; j < w.n; ++j, f += 2) {
          const int key0 = w.k_begin + j * BN;
          const uint32_t rs = f % C::NRAW, s = f % NS;
          ok = warp_wait(&raw_full[rs], (f / C::NRAW) & 1, abort_flag, p.status) &&
               (f < static_cast<uint32_t>(NS) ||
                warp_wait(&kv_empty[s], (f / NS - 1) & 1, abort_flag, p.status));
          if (!ok) break;
          // the factors of the warp's 32 rows, one per lane: row i * (128 / G) + (32 / G) * warp + q
          // of the tile in lane (32 / G) * i + q
          uint32_t factor;
          {
            constexpr int Q = 32 / G;
            const int r = (lane / Q) * (128 / G) + Q * (warp & 3) + lane % Q;
            factor = row_scale(s_below[BN * (f % C::NRAW) + r]);
            factor |= factor << 16;
          }
          const bool edge = key0 + BN > min(w.L, w.k_end);
          // piece i of the thread is row i * (128 / G) + r0
          constexpr int kRowStep = 128 / G;  // (a multiple of 8: the swizzle stays)
          const uint32_t src = raw0 + rs * C::RAW + r0 * D + 16 * c;
          const uint32_t dst0 = kv0 + s * C::TILE + to0, dst1 = kv0 + s * C::TILE + to1;
#pragma unroll 1
          for (int i0 = 0; i0 < G; i0 += 4) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = lds128(src + (i0 + i) * 2048);
            if (edge) {  // rows past the end: zeros; the drafts' values: if finite
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = key0 + (i0 + i) * kRowStep + r0;
                if (r >= w.k_end) x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (v == 1 && r >= w.L)
                  x[i] = make_uint4(finite_e4m3x4(x[i].x), finite_e4m3x4(x[i].y),
                                    finite_e4m3x4(x[i].z), finite_e4m3x4(x[i].w));
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t mm =
                  __shfl_sync(0xffffffffu, factor, (32 / G) * (i0 + i) + r0 % (32 / G));
              const uint4 lo = make_uint4(hmul2(e4m3x2_to_f16x2(x[i].x), mm),
                                          hmul2(e4m3x2_hi_to_f16x2(x[i].x), mm),
                                          hmul2(e4m3x2_to_f16x2(x[i].y), mm),
                                          hmul2(e4m3x2_hi_to_f16x2(x[i].y), mm));
              const uint4 hi = make_uint4(hmul2(e4m3x2_to_f16x2(x[i].z), mm),
                                          hmul2(e4m3x2_hi_to_f16x2(x[i].z), mm),
                                          hmul2(e4m3x2_to_f16x2(x[i].w), mm),
                                          hmul2(e4m3x2_hi_to_f16x2(x[i].w), mm));
              sts128(dst0 + (i0 + i) * (kRowStep * 128), lo);
              sts128(dst1 + (i0 + i) * (kRowStep * 128), hi);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&kv_full[s]);
            mbar_arrive(&raw_empty[rs]);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (F8) regs_inc<136>();
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;  // of the query tile
    const int M = p.T * p.rep;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128u * x;
    const uint32_t tO = tmem + lane_off + 256u + static_cast<uint32_t>(D) * x;
    uint32_t ns = 0, tile0 = 0, done[2] = {0, 0};  // done: pieces in which stream 0, 1 had tiles
    bool ok = true;
    // the thread's query row of a piece, of the KV head's (at or past M: none), and its factor
    auto row_of = [&](const View& w) {
      return (w.rb * (1 + pair) + (pair ? x : 0)) * BN + row;
    };
    auto factor_of = [&](const GroupPiece& q) -> float {
      if (!F8 || q.n == 0) return 1.f;
      const View w(q, p);
      const int r = row_of(w);
      return r < M ? p.q_factor[(static_cast<size_t>(w.b) * p.Hkv + w.kvh) * M + r] : 1.f;
    };
    float factor = factor_of(pc);
    while (pc.n > 0) {  // (to the end: the warps' barriers go together)
      const View w(pc, p);
      const int r = row_of(w);
      const bool live = r < M;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int t = live ? r / p.rep : 0;
      const float row_factor = p.scale_log2 * factor;
      const uint32_t* anc = p.anc + (static_cast<size_t>(w.b) * p.T + t) * p.words;
      const size_t slot = static_cast<size_t>(blockIdx.x) + pc.segment(p.line);
      if (threadIdx.x == 0) pc.leave_for_merge(p.line);

      float R = -INFINITY, l = 0.f;
      for (int j = pair ? 0 : x; j < w.n && ok; j += step) {
        if (!warp_wait(&s_full[x], ns & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        if (warp_live) {
          float c = row_factor, ev = 0.f;
          if constexpr (F8) {
            const float2 ts = s_tile[(tile0 + j) & 7];
            c *= ts.x;
            c *= 0.0078125f;  // (by itself: 2^(E_k - 7) may be too small)
            ev = ts.y;
          }
          c = fmaxf(c, 1.17549435e-38f);  // (a hidden score's -inf times 0 would be NaN)
          if (j >= w.first_edge) {  // rows that this query does not see
            const int key0 = w.k_begin + j * BN;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int k0 = key0 + 32 * i;
              const uint32_t in = k0 + 32 <= w.k_end ? 0xffffffffu
                                  : k0 >= w.k_end    ? 0u
                                                     : (1u << (w.k_end - k0)) - 1u;
              mask_scores(tS + 32u * i, ~(in & draft_bits32(anc, p.words, k0 - w.L)));
            }
            tmem_st_wait();
          }
          if constexpr (F8) {
            if (__builtin_expect(ev == kOwnScales, 0)) {
              const float2 t = own_scales<D>(p, w.b, w.kvh, w.k_begin + j * BN, w.k_end, tS, tO,
                                             j >= step, row_factor, R, l);
              R = t.x;
              l = t.y;
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[x]);
              continue;
            }
          }
          // (the next columns' load runs beside the arithmetic on these)
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t ra[32], rb[32];
          auto max32 = [&](const uint32_t (&r)[32]) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mq[k] = fmax3(mq[k], __uint_as_float(r[e + k]), __uint_as_float(r[e + 4 + k]));
          };
          if constexpr (F8) {
            // (20 warps leave 96 registers: the loads in flight would spill)
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              tmem_ld32_issue(tS + 32u * i, ra);
              tmem_ld32_wait(ra);
              max32(ra);
            }
          } else {
            tmem_ld32_issue(tS, ra);
            tmem_ld32_wait(ra);
            tmem_ld32_issue(tS + 32u, rb);
            max32(ra);
            tmem_ld32_wait(rb);
            tmem_ld32_issue(tS + 64u, ra);
            max32(rb);
            tmem_ld32_wait(ra);
            tmem_ld32_issue(tS + 96u, rb);
            max32(ra);
            tmem_ld32_wait(rb);
            tmem_ld32_issue(tS, ra);
            max32(rb);
          }
          const float top = __fmul_rn(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])), c) + ev;
          const bool mine = top > R + kRescaleThreshold;
          if (__any_sync(0xffffffffu, mine)) {
            float f = mine ? ex2_approx(F8 ? 0.5f * (R - top) : R - top) : 1.f;
            l *= f;
            if constexpr (F8) {  // (O may vanish beside the tile to come, l need not)
              l *= f;
              f *= f;
            }
            if (j >= step) {
              if constexpr (!F8) tmem_ld32_wait(ra);
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
          // what the tile's weights are relative to
          const bool low = F8 && top < R - kLowTile && top != -INFINITY;
          const float Rt = low ? top + (7.f + kLowWeight) : R;
          // (nothing seen yet: 2^-inf = 0, and a NaN score stays NaN)
          const float off = (F8 ? ev + 7.f : 0.f) - (Rt == -INFINITY ? 0.f : Rt);
          float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
          auto weights32 = [&](const uint32_t (&r)[32], uint32_t at) {
            uint32_t pk[16];
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
            tmem_st16(at, pk);
          };
          if constexpr (F8) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              tmem_ld32_issue(tS + 32u * i, ra);
              tmem_ld32_wait(ra);
              weights32(ra, tS + 16u * i);
            }
          } else {
            tmem_ld32_wait(ra);
            tmem_ld32_issue(tS + 32u, rb);
            weights32(ra, tS);
            tmem_ld32_wait(rb);
            tmem_ld32_issue(tS + 64u, ra);
            weights32(rb, tS + 16u);
            tmem_ld32_wait(ra);
            tmem_ld32_issue(tS + 96u, rb);
            weights32(ra, tS + 32u);
            tmem_ld32_wait(rb);
            weights32(rb, tS + 48u);
          }
          // (the weights are handed over ahead of the arithmetic on their sum)
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x]);
          const float sum = (sa0 + sa1) + (sb0 + sb1);
          if constexpr (F8) {  // (a factor at a time: their product may leave fp32's range)
            const float g = low ? ex2_approx(0.5f * (Rt - R)) : 1.f;
            l += sum * 0.0078125f * ex2_approx(-ev) * g * g;
          } else {
            l += sum;
          }
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x]);
        }
      }
      tile0 += w.n;
      // (what the next piece begins with is read beside the end of this one)
      pc.next(p.line);
      factor = factor_of(pc);
      // Partial result: R, l and O, relative to 2^R; four channels of all rows together, so that
      // a warp's lanes, which hold a row each, store 512 bytes in a row.  With one query tile
      // stream 0 adds stream 1's sums to its own and hands back the factors of the two outputs;
      // then each stream's warps write half of the channels.
      const bool two = !pair && w.n > 1;  // both streams had tiles of this row
      // e4m3: relative to the power of two that leaves l in [0.5, 1), R counting the values' scales;
      // returned is what O is multiplied by (2^-7 of w, 2^-7 of V16, kPartLog2)
      auto relative = [](float& R, float& l) -> float {
        if constexpr (!F8) return 1.f;
        const int up = log2_above(l);
        const float f = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        R += static_cast<float>(up);
        l *= f;
        return f * (1.f / (16384.f * kPartScale));
      };
      float f0 = 1.f, f1 = 0.f;
      if (pair) {
        f0 = relative(R, l);
      } else {
        if (x == 1) s_ml[row] = make_float2(R, l);
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (x == 0) {
          f0 = relative(R, l);
          if (two) {
            float2 other = s_ml[row];
            f1 = relative(other.x, other.y);
            const float m = fmaxf(R, other.x);
            // (a stream that saw nothing holds zeros, or NaN)
            const float e0 = R == -INFINITY ? 1.f : ex2_approx(R - m);
            const float e1 = other.x == -INFINITY ? 1.f : ex2_approx(other.x - m);
            l = l * e0 + other.y * e1;
            R = m;
            f0 *= e0;
            f1 *= e1;
          }
          s_ml[row] = make_float2(f0, f1);
        }
        asm volatile("bar.sync 5, 256;" ::: "memory");
        if (x == 1) {
          const float2 f = s_ml[row];
          f0 = f.x;
          f1 = f.y;
        }
      }
      const int own = pair ? x : 0;  // the (first) stream whose output this is
      ok = ok && warp_wait(&o_full[own], done[0] & 1, abort_flag, p.status) &&
           (!two || warp_wait(&o_full[1], done[1] & 1, abort_flag, p.status));
      if (ok) {
        tc_fence_after();
        if (warp_live) {
          const size_t at = slot * p.part_rows + 128 * own + row;
          float4* dst = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * p.part_rows +
                        128 * own + row;
          const uint32_t t0 = tmem + lane_off + 256u + static_cast<uint32_t>(D * own);
          const int i1 = pair || x == 1 ? D / 32 : D / 64;
#pragma unroll 1
          for (int i = pair || x == 0 ? 0 : D / 64; i < i1; ++i) {
            uint32_t r[32];
            tmem_ld32_sync(t0 + 32u * i, r);
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(r[e]) * f0;
            if (two) {
              tmem_ld32_sync(t0 + D + 32u * i, r);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(r[e]), f1, o[e]);
            }
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                dst[static_cast<size_t>(8 * i + e / 4) * p.part_rows] =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          if (live && (pair || x == 0))
            *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(R, l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&o_empty[own]);
          if (two) mbar_arrive(&o_empty[1]);
        }
      }
      ++done[0];
      done[1] += two || pair;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// group_merge_kernel (group_attn.cu) for this kernel's layout: a warp takes eight query rows and
// 4 V quads of channels, so that its loads are 128 bytes in a row each and its output fills whole
// sectors.  For many rows the instructions per row and the registers count (all CTAs resident at
// once hide the three loads that follow one another), so V is 2 with three partial results in
// flight; for few rows the latency, so V is 1 with eight.  The whole step with 16384 rows of two
// to four: 74.3 us (V = 2, 3 in flight), 75-76 (2 or 4 in flight; V = 4), 91 (V = 1); with 256
// rows of eight: 13.4 us with V = 1, 14 with V = 2.
template <int D, int V>
struct MergeShape {
  static constexpr int WARPS = D / 16 / V;  // of the same rows
  static constexpr int GROUPS = WARPS < 4 ? 4 / WARPS : 1;
  static constexpr int ROWS = 8 * GROUPS, THREADS = 32 * WARPS * GROUPS;
};

template <int D, int V>
__global__ void __launch_bounds__(MergeShape<D, V>::THREADS) group_tc_merge_kernel(
    const float4* __restrict__ part_o, const float* __restrict__ part_ml, const int2* seg,
    int blocks, int part_rows, int block_rows, int rblocks, const uint32_t* __restrict__ anc,
    const uint8_t* __restrict__ vflag, const __nv_bfloat16* __restrict__ v_new, bool f8,
    __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int Hkv, int rep, int T, int words) {
  using S = MergeShape<D, V>;
  constexpr int U = V == 1 ? 8 : 3;  // partial results whose loads are in flight together
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at_block = static_cast<int>(blockIdx.x) / blocks;  // (sequence, KV head, row block)
  const int in_block = (static_cast<int>(blockIdx.x) - at_block * blocks) * S::ROWS +
                       8 * (warp / S::WARPS) + (lane & 7);
  const int quad = (warp % S::WARPS) * 4 * V + (lane >> 3);  // and quad + 4, ...
  const int plane = at_block / rblocks, rb = at_block - plane * rblocks;
  const int b = plane / Hkv, g = plane - b * Hkv;
  const int r = rb * block_rows + in_block;
  const bool live = r < T * rep && in_block < part_rows;
  const int t = live ? r / rep : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 at_seg = seg[at_block];
  const uint32_t* mine = anc + (static_cast<size_t>(b) * T + t) * words;
  const uint32_t own = mine[t >> 5];
  bool odd = false;  // does any draft have values that are not finite?
  for (int j = lane; j < T; j += 32) odd |= vflag[static_cast<size_t>(plane) * T + j] != 0;
  const int ns = live && ((own >> (t & 31)) & 1u) ? at_seg.y : 0;  // 0: padding
  float m = -INFINITY, l = 0.f;
  float4 acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < ns; s0 += U) {
    float2 ml[U];
    float4 o[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      if (s0 + u >= ns) continue;
      const size_t slot = static_cast<size_t>(at_seg.x) + s0 + u;
      ml[u] = *reinterpret_cast<const float2*>(part_ml + 2 * (slot * part_rows + in_block));
#pragma unroll
      for (int v = 0; v < V; ++v)
        o[u][v] = part_o[(slot * (D / 4) + quad + 4 * v) * part_rows + in_block];
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mx = fmaxf(mx, ml[u].x);
    // (one that saw nothing holds zeros, or NaN)
    const float f = m == -INFINITY ? 1.f : ex2_approx(m - mx);
    l *= f;
    m = mx;
#pragma unroll
    for (int v = 0; v < V; ++v)
      acc[v] = make_float4(acc[v].x * f, acc[v].y * f, acc[v].z * f, acc[v].w * f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u >= ns) break;
      const float e = ml[u].x == -INFINITY ? 1.f : ex2_approx(ml[u].x - m);
      l += e * ml[u].y;
#pragma unroll
      for (int v = 0; v < V; ++v)
        acc[v] = make_float4(acc[v].x + e * o[u][v].x, acc[v].y + e * o[u][v].y,
                             acc[v].z + e * o[u][v].z, acc[v].w + e * o[u][v].w);
    }
  }
  const bool any = !(l <= 0.f);  // NaN stays
  const float inv = any ? (f8 ? kPartScale : 1.f) / l : 0.f;
  float x[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    x[v][0] = any ? acc[v].x * inv : 0.f;
    x[v][1] = any ? acc[v].y * inv : 0.f;
    x[v][2] = any ? acc[v].z * inv : 0.f;
    x[v][3] = any ? acc[v].w * inv : 0.f;
  }
  if (__any_sync(0xffffffffu, odd)) {
    for (int w = 0; w < words; ++w) {
      const int j = 32 * w + lane;
      const uint32_t flags = __ballot_sync(
          0xffffffffu, j < T && vflag[static_cast<size_t>(plane) * T + j] != 0);
      for (uint32_t left = ns > 0 ? flags & mine[w] : 0u; left != 0u; left &= left - 1u) {
        const __nv_bfloat16* vn =
            v_new + (static_cast<size_t>(plane) * T + 32 * w + __ffs(left) - 1) * D + 4 * quad;
#pragma unroll
        for (int e = 0; e < 4 * V; ++e) {
          const float y = __bfloat162float(vn[16 * (e / 4) + e % 4]);
          // (an e4m3 cache holds NaN for an infinity)
          if (!isfinite(y)) x[e / 4][e % 4] += f8 ? __int_as_float(0x7fffffff) : y;
        }
      }
    }
  }
  if (!live) return;
  const size_t row = (static_cast<size_t>(plane) * rep + r - t * rep) * T + t;  // [B, Hq, T]
#pragma unroll
  for (int v = 0; v < V; ++v)
    *reinterpret_cast<uint2*>(out + row * D + 4 * quad + 16 * v) =
        make_uint2(pack_bf16x2(x[v][0], x[v][1]), pack_bf16x2(x[v][2], x[v][3]));
  if (lse != nullptr && quad == 0)
    lse[row] = any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, int V>
cudaError_t launch_merge(const GroupArgs& a, const uint8_t* vflag, const void* v_new, void* out,
                         float* lse, cudaStream_t stream) {
  using S = MergeShape<D, V>;
  const int blocks = (a.plan.part_rows + S::ROWS - 1) / S::ROWS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.Hkv * a.plan.rblocks * blocks), 1, 1);
  cfg.blockDim = dim3(S::THREADS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(
      &cfg, group_tc_merge_kernel<D, V>, reinterpret_cast<const float4*>(a.part_o),
      static_cast<const float*>(a.part_ml), static_cast<const int2*>(a.seg), blocks,
      a.plan.part_rows, a.plan.block_rows, a.plan.rblocks, a.anc, vflag,
      static_cast<const __nv_bfloat16*>(v_new), a.cache.k_scale != nullptr,
      static_cast<__nv_bfloat16*>(out), lse, a.Hkv, a.Hq / a.Hkv, a.T, a.words);
}

template <int D, bool F8>
cudaError_t launch_t(const GroupArgs& a, cudaStream_t stream) {
  using C = Cfg<D, F8>;
  TParams p{};
  p.q_factor = a.q_factor;
  p.anc = a.anc;
  p.line = group_line(a);
  p.rows = CacheRows{a.cache.block_table, a.Hkv, a.cache.Lmax, a.cache.page_size,
                     a.cache.num_pages, a.cache.max_pages};
  p.k_scale = static_cast<const uint8_t*>(a.cache.k_scale);
  p.v_scale = static_cast<const uint8_t*>(a.cache.v_scale);
  p.words = a.words;
  const uintptr_t scales =
      reinterpret_cast<uintptr_t>(p.k_scale) | reinterpret_cast<uintptr_t>(p.v_scale);
  p.scale_words = scales % 4 == 0 && (a.cache.block_table != nullptr || a.cache.Lmax % 4 == 0);
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
  p.rblocks = a.plan.rblocks;
  p.part_rows = a.plan.part_rows;
  const int rows = a.T * p.rep;
  p.pair = a.plan.block_rows == 256 ? 1 : 0;
  p.lost = a.lost;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);

  alignas(64) CUtensorMap tq, tk, tv;
  const int trows = paged ? ps : a.cache.Lmax;
  const int planes = paged ? a.cache.num_pages * a.Hkv : a.B * a.Hkv;
  const bool made = F8 ? make_tmap_u8_3d(&tk, a.cache.k, D, trows, planes, p.box_rows, false) &&
                             make_tmap_u8_3d(&tv, a.cache.v, D, trows, planes, p.box_rows, false)
                       : make_tmap_bf16_3d(&tk, a.cache.k, D, trows, planes, p.box_rows) &&
                             make_tmap_bf16_3d(&tv, a.cache.v, D, trows, planes, p.box_rows);
  // (16-bit values, whichever: f16 for an 8-bit cache)
  if (!made || !make_tmap_bf16_3d(&tq, a.q, D, rows, a.B * a.Hkv, BN)) return cudaErrorInvalidValue;
  static SmemLimitOnce smem_limit;
  cudaError_t e = smem_limit.set(group_tc_kernel<D, F8>, C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.plan.grid), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, group_tc_kernel<D, F8>, p, tq, tk, tv);
}

}  // namespace

cudaError_t launch_group_tc(const GroupArgs& a, cudaStream_t stream) {
  const bool f8 = a.cache.k_scale != nullptr;
  if (a.d == 64) return f8 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
  return f8 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
}

cudaError_t launch_group_tc_merge(const GroupArgs& a, const uint8_t* vflag, const void* v_new,
                                  void* out, float* lse, cudaStream_t stream) {
  if (a.B * a.Hq * a.T <= 4096)
    return a.d == 64 ? launch_merge<64, 1>(a, vflag, v_new, out, lse, stream)
                     : launch_merge<128, 1>(a, vflag, v_new, out, lse, stream);
  return a.d == 64 ? launch_merge<64, 2>(a, vflag, v_new, out, lse, stream)
                   : launch_merge<128, 2>(a, vflag, v_new, out, lse, stream);
}

}  // namespace csattn
