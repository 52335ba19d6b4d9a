// The 4-bit KV cache as it is written and read back (format: fp4.cuh).
//
// Append: a token's keys and values, as given (rotated already), to the row that the lengths, the
// block table or a slot map name.  Read: rows 0..seq_lens[b]-1 back to bf16, exactly.  A thread
// has eight channels of a key and of the value beside it: 16 bytes of bf16 and four of e2m1, so
// that a warp's loads and stores are contiguous on both sides and a row is found once; two lanes
// share a block of 16 and its scale byte.  Both move each byte once.  128 channels, 8 KV heads: the
// append of 4 x 4096 tokens takes 15.5 us (86 MB, 5.5 TB/s; three quarters of the issue slots are
// busy, most of them rounding; 16.7 with each scale worked out by both lanes), of 64 tokens 1.7;
// the read of 32768 rows in 128-row pages 28.3 us (172 MB, 6.1 TB/s), of 64 x 64..256 rows 11.9,
// whose blocks have little to do between the length, the table and the row.
// (16 channels per thread, which leaves half sectors to each store: 36.9 us for the 32768 rows;
// keys and values in threads of their own: 40.5.)
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"

namespace csattn {
namespace {

constexpr int kThreads = 128;

struct AppendParams {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  long long k_token, k_head, k_seq;  // strides in elements
  long long v_token, v_head, v_seq;
  uint8_t* k_cache;
  uint8_t* v_cache;
  uint8_t* k_scale;
  uint8_t* v_scale;
  const int32_t* cache_lens;  // null: slots
  const int64_t* slots;
  CacheRows rows;
  int Tn;
  unsigned per_head;  // 0: blockIdx.y is the head; else it is blockIdx.x modulo Hkv
  uint32_t* status;
};

// the largest magnitude's bits in a lane's eight channels
__device__ __forceinline__ uint32_t top8(const uint4& x) {
  const uint32_t m = absmax_bf16x2(absmax_bf16x2(x.x, x.y), absmax_bf16x2(x.z, x.w)) & 0x7fff7fffu;
  return max(m & 0xffffu, m >> 16);
}
// 1 / s of a scale byte; 0 of a scale of 0, which leaves zeros, and negative of a NaN, which goes
// with them
__device__ __forceinline__ float inverse_of(uint32_t code) {
  const float s = fp4_scale(code);
  return code == kFp4Nan ? -1.f : (s > 0.f ? fp4_inverse(s) : 0.f);
}
__device__ __forceinline__ uint32_t quantise8(const uint4& x, float inv) {
  return inv < 0.f ? 0u : pack_e2m1x8(x, inv);
}

// Thread item (b, g, t, c), U tokens a block's rows apart: consecutive threads write consecutive
// rows of a KV head.
template <int D, int U>
__global__ void __launch_bounds__(kThreads)
    append_fp4_kernel(const __grid_constant__ AppendParams p) {
  constexpr int G = D / 8, R = kThreads / G;  // lanes of a row, a block's rows
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = static_cast<int>(threadIdx.x) % G;
  const int Hkv = p.rows.Hkv;
  int blk = static_cast<int>(blockIdx.x), g = static_cast<int>(blockIdx.y);
  if (p.per_head != 0) {
    blk = static_cast<int>(__umulhi(blockIdx.x, p.per_head));
    g = static_cast<int>(blockIdx.x) - blk * Hkv;
  }
  const int t0 = blk * (R * U) + static_cast<int>(threadIdx.x) / G;
  const int b = static_cast<int>(blockIdx.z);
  const __nv_bfloat16* k_src = p.k_new + b * p.k_seq + g * p.k_head + 8 * c;
  const __nv_bfloat16* v_src = p.v_new + b * p.v_seq + g * p.v_head + 8 * c;
  uint4 k[U], v[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int t = t0 + i * R;
    k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t < p.Tn) {
      k[i] = *reinterpret_cast<const uint4*>(k_src + t * p.k_token);
      v[i] = *reinterpret_cast<const uint4*>(v_src + t * p.v_token);
    }
  }
  long long row[U];
  bool wrong = false;
  const int L = p.slots == nullptr ? p.cache_lens[b] : 0;
  const bool fits = L >= 0 && L <= p.rows.Lmax - p.Tn;  // (no overflow: Lmax, Tn < 2^30)
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int t = t0 + i * R;
    row[i] = -1;
    if (t >= p.Tn) continue;
    if (p.slots != nullptr) {
      const long long slot = p.slots[t];
      if (slot >= 0) {  // (a negative one: no token)
        // (a pool of 2^32 rows does not fit the card)
        const unsigned ps = p.rows.page_size, at32 = static_cast<unsigned>(slot), page = at32 / ps;
        if ((slot >> 32) == 0 && page < static_cast<unsigned>(p.rows.num_pages))
          row[i] = (static_cast<long long>(page) * Hkv + g) * ps + (at32 - page * ps);
        else
          wrong = true;
      }
    } else {
      if (fits) row[i] = p.rows.at(b, g, L + t);
      wrong |= row[i] < 0;
    }
  }
  if (wrong && c == 0 && g == 0) atomicOr(p.status, kStatusDeviceArg);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    // Two lanes share a block of the key and one of the value: the even one finds the key's scale,
    // the odd one the value's.
    const bool odd = (c & 1) != 0;
    const uint32_t kt = top8(k[i]), vt = top8(v[i]);
    const uint32_t code = fp4_scale_code(
        max(odd ? vt : kt, __shfl_xor_sync(0xffffffffu, odd ? kt : vt, 1)));
    const float mine = inverse_of(code), other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const uint32_t k4 = quantise8(k[i], odd ? other : mine);
    const uint32_t v4 = quantise8(v[i], odd ? mine : other);
    if (row[i] < 0) continue;
    *reinterpret_cast<uint32_t*>(p.k_cache + row[i] * (D / 2) + 4 * c) = k4;
    *reinterpret_cast<uint32_t*>(p.v_cache + row[i] * (D / 2) + 4 * c) = v4;
    (odd ? p.v_scale : p.k_scale)[row[i] * (D / 16) + c / 2] = static_cast<uint8_t>(code);
  }
}

// e2m1 times s as bf16: both steps are exact
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t h, float s) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x * s, f.y * s);
}

// Eight channels of a key and of the value beside it per thread item (b, g, r, c), kRows rows a
// block's rows apart: a row is found once for both.
constexpr int kRows = 2;
template <int D>
__global__ void __launch_bounds__(kThreads) read_fp4_kernel(
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
    const int32_t* __restrict__ seq_lens, CacheRows rows, __nv_bfloat16* __restrict__ k_out,
    __nv_bfloat16* __restrict__ v_out, int Lout, uint32_t* status, int blocks, int shift) {
  constexpr int G = D / 8, R = kThreads / G;
  const int bg = static_cast<int>(blockIdx.x) / blocks;
  const int blk = static_cast<int>(blockIdx.x) - bg * blocks;
  const int b = bg / rows.Hkv, g = bg - b * rows.Hkv;
  const int c = static_cast<int>(threadIdx.x) % G;
  const int r0 = blk * (R * kRows) + static_cast<int>(threadIdx.x) / G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (the table is read beside the length; its entries of no row are any)
  int at[kRows], page[kRows];
  if (rows.block_table != nullptr) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      // (shift: of a page size that is a power of two, or negative)
      const int r = min(r0 + k * R, rows.Lmax - 1);
      at[k] = shift >= 0 ? r >> shift : r / rows.page_size;
      page[k] = rows.block_table[static_cast<size_t>(b) * rows.max_pages + at[k]];
    }
  }
  const int n = seq_lens[b];
  if (n < 0 || n > Lout || n > rows.Lmax) {
    if (blk == 0 && g == 0 && threadIdx.x == 0) atomicOr(status, kStatusDeviceArg);
    return;  // the sequence is left as it was
  }
  uint32_t x[kRows][2], code[kRows][2];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = r0 + k * R;
    x[k][0] = x[k][1] = code[k][0] = code[k][1] = 0u;
    if (r < n) {
      long long row = (static_cast<long long>(b) * rows.Hkv + g) * rows.Lmax + r;
      if (rows.block_table != nullptr)
        row = page[k] < 0 || page[k] >= rows.num_pages
                  ? -1
                  : (static_cast<long long>(page[k]) * rows.Hkv + g) * rows.page_size + r -
                        at[k] * rows.page_size;
      if (row >= 0) {
        x[k][0] = *reinterpret_cast<const uint32_t*>(k_cache + row * (D / 2) + 4 * c);
        x[k][1] = *reinterpret_cast<const uint32_t*>(v_cache + row * (D / 2) + 4 * c);
        code[k][0] = k_scale[row * (D / 16) + c / 2];
        code[k][1] = v_scale[row * (D / 16) + c / 2];
      } else if (c == 0) {
        atomicOr(status, kStatusDeviceArg);  // the row reads as zeros
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = r0 + k * R;
    if (r >= n) break;
    const size_t to = (static_cast<size_t>(bg) * Lout + r) * D + 8 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s = fp4_scale(code[k][i]);
      const uint32_t y = x[k][i];
      *reinterpret_cast<uint4*>((i == 0 ? k_out : v_out) + to) =
          make_uint4(to_bf16x2(e2m1x2_to_f16x2<0>(y), s), to_bf16x2(e2m1x2_to_f16x2<1>(y), s),
                     to_bf16x2(e2m1x2_to_f16x2<2>(y), s), to_bf16x2(e2m1x2_to_f16x2<3>(y), s));
    }
  }
}

CacheRows rows_of(const KvCache& c, int Hkv) {
  return CacheRows{c.block_table, Hkv, c.Lmax, c.page_size, c.num_pages, c.max_pages};
}

}  // namespace

cudaError_t launch_cache_append_fp4(const Fp4AppendArgs& a, cudaStream_t stream) {
  AppendParams p{};
  p.k_new = static_cast<const __nv_bfloat16*>(a.k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(a.v_new);
  p.k_token = a.k_strides[0];
  p.k_head = a.k_strides[1];
  p.k_seq = a.k_strides[2];
  p.v_token = a.v_strides[0];
  p.v_head = a.v_strides[1];
  p.v_seq = a.v_strides[2];
  p.k_cache = static_cast<uint8_t*>(a.cache.k);
  p.v_cache = static_cast<uint8_t*>(a.cache.v);
  p.k_scale = static_cast<uint8_t*>(a.cache.k_scale);
  p.v_scale = static_cast<uint8_t*>(a.cache.v_scale);
  p.cache_lens = a.cache_lens;
  p.slots = a.slots;
  p.rows = rows_of(a.cache, a.Hkv);
  p.Tn = a.Tn;
  p.status = a.status;
  // two tokens per thread where that still fills the GPU
  const long long threads = static_cast<long long>(a.B) * a.Hkv * a.Tn * (a.d / 8);
  const int U = threads >= 2LL * 12 * kSms * kThreads ? 2 : 1;
  const unsigned rows = kThreads / (a.d / 8) * U;
  auto* kernel = a.d == 128 ? (U == 2 ? append_fp4_kernel<128, 2> : append_fp4_kernel<128, 1>)
                            : (U == 2 ? append_fp4_kernel<64, 2> : append_fp4_kernel<64, 1>);
  const unsigned blocks = (static_cast<unsigned>(a.Tn) + rows - 1) / rows;
  // Blocks that run together read what lies together: the heads of a token first where they are
  // beside one another (16384 tokens by slots: 17.9 us, tokens first 19.7).  x / Hkv is then the
  // upper half of x * ceil(2^32 / Hkv), exact while x * Hkv < 2^32.
  const unsigned heads = static_cast<unsigned>(a.Hkv);  // (Hkv, B <= 65535)
  const bool heads_first = heads > 1 && a.k_strides[1] < a.k_strides[0] &&
                           1ull * blocks * heads < (1u << 31) &&
                           1ull * blocks * heads * heads < (1ull << 32);
  if (heads_first) p.per_head = static_cast<unsigned>(((1ull << 32) + heads - 1) / heads);
  const dim3 grid(heads_first ? blocks * heads : blocks, heads_first ? 1u : heads,
                  static_cast<unsigned>(a.B));
  return launch_behind(kernel, grid, kThreads, stream, p);
}

cudaError_t launch_cache_read_fp4(const KvCache& cache, const int32_t* seq_lens, void* k_out,
                                  void* v_out, int B, int Hkv, int Lout, int d, uint32_t* status,
                                  cudaStream_t stream) {
  const long long per = kThreads / (d / 8) * kRows;
  const long long blocks = (std::min(Lout, cache.Lmax) + per - 1) / per;
  int shift = -1;
  if (cache.page_size > 0 && (cache.page_size & (cache.page_size - 1)) == 0)
    for (shift = 0; (1 << shift) < cache.page_size;) ++shift;
  // (a grid below 2^31: B * Hkv < 2^30, and B * Hkv * Lout < 2^33 where there are more blocks)
  auto* kernel = d == 128 ? read_fp4_kernel<128> : read_fp4_kernel<64>;
  return launch_behind(kernel, dim3(static_cast<unsigned>(blocks * B * Hkv)), kThreads, stream,
                       static_cast<const uint8_t*>(cache.k), static_cast<const uint8_t*>(cache.v),
                       static_cast<const uint8_t*>(cache.k_scale),
                       static_cast<const uint8_t*>(cache.v_scale), seq_lens, rows_of(cache, Hkv),
                       static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), Lout,
                       status, static_cast<int>(blocks), shift);
}

}  // namespace csattn
