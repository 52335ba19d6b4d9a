// The 4-bit KV cache as it is written and read back (format: fp4.cuh).
//
// Append: a token's keys and values, as given (rotated already), to the row that the lengths, the
// block table or a slot map name.  Read: rows 0..seq_lens[b]-1 back to bf16, exactly.  A thread
// has eight channels of a key and of the value beside it: 16 bytes of bf16 and four of e2m1, so
// that a warp's loads and stores are contiguous on both sides; two lanes share a block of 16 and
// its scale byte.  Both move each byte once.
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
  unsigned items;  // B * Hkv * Tn * (D / 8) < 2^30
  uint32_t* status;
};

// the byte and the e2m1 of a lane's eight channels; the lane beside it has the block's others
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint32_t* code) {
  const uint32_t m = absmax_bf16x2(absmax_bf16x2(x.x, x.y), absmax_bf16x2(x.z, x.w)) & 0x7fff7fffu;
  uint32_t top = max(m & 0xffffu, m >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  *code = fp4_scale_code(top);
  const float s = fp4_scale(*code);
  // (the reciprocal of 0 would meet zeros; that of a NaN goes with zeros for the values)
  return *code == kFp4Nan ? 0u : pack_e2m1x8(x, s > 0.f ? __frcp_rn(s) : 0.f);
}

// Thread item (b, g, t, c): consecutive threads write consecutive rows of a KV head.
template <int D>
__global__ void __launch_bounds__(kThreads) append_fp4_kernel(const __grid_constant__ AppendParams p) {
  constexpr int G = D / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  unsigned at = blockIdx.x * kThreads + threadIdx.x;
  const bool live = at < p.items;
  if (!live) at = 0;
  const int c = static_cast<int>(at % G);
  at /= G;
  const int t = static_cast<int>(at % p.Tn);
  at /= p.Tn;
  const int Hkv = p.rows.Hkv;
  const int g = static_cast<int>(at % Hkv), b = static_cast<int>(at / Hkv);
  const uint4 k = *reinterpret_cast<const uint4*>(p.k_new + b * p.k_seq + g * p.k_head +
                                                  t * p.k_token + 8 * c);
  const uint4 v = *reinterpret_cast<const uint4*>(p.v_new + b * p.v_seq + g * p.v_head +
                                                  t * p.v_token + 8 * c);
  long long row = -1;
  bool wrong = false;
  if (p.slots != nullptr) {
    const long long slot = p.slots[t];
    if (slot >= 0) {  // (a negative one: no token)
      // (a pool of 2^32 rows does not fit the card)
      const unsigned ps = p.rows.page_size, at32 = static_cast<unsigned>(slot), page = at32 / ps;
      wrong = (slot >> 32) != 0 || page >= static_cast<unsigned>(p.rows.num_pages);
      if (!wrong) row = (static_cast<long long>(page) * Hkv + g) * ps + (at32 - page * ps);
    }
  } else {
    const int L = p.cache_lens[b];
    wrong = L < 0 || L > p.rows.Lmax - p.Tn;  // (no overflow: Lmax, Tn < 2^30)
    if (!wrong) {
      row = p.rows.at(b, g, L + t);
      wrong = row < 0;
    }
  }
  if (live && wrong && c == 0 && g == 0) atomicOr(p.status, kStatusDeviceArg);
  uint32_t kc, vc;
  const uint32_t k4 = quantise8(k, &kc), v4 = quantise8(v, &vc);
  if (!live || row < 0) return;
  *reinterpret_cast<uint32_t*>(p.k_cache + row * (D / 2) + 4 * c) = k4;
  *reinterpret_cast<uint32_t*>(p.v_cache + row * (D / 2) + 4 * c) = v4;
  if ((c & 1) == 0) {
    p.k_scale[row * (D / 16) + c / 2] = static_cast<uint8_t>(kc);
    p.v_scale[row * (D / 16) + c / 2] = static_cast<uint8_t>(vc);
  }
}

// e2m1 times s as bf16: both steps are exact
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t h, float s) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x * s, f.y * s);
}

// Eight channels per thread item (b, g, r, c); kRows rows, a block's threads apart.
constexpr int kRows = 4;
template <int D>
__global__ void __launch_bounds__(kThreads) read_fp4_kernel(
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
    const int32_t* __restrict__ seq_lens, CacheRows rows, __nv_bfloat16* __restrict__ k_out,
    __nv_bfloat16* __restrict__ v_out, int Lout, uint32_t* status, int k_blocks) {
  constexpr int G = D / 8;
  const int bg = static_cast<int>(blockIdx.x) / (2 * k_blocks);
  int blk = static_cast<int>(blockIdx.x) - bg * (2 * k_blocks);
  const bool is_k = blk < k_blocks;
  if (!is_k) blk -= k_blocks;
  const int b = bg / rows.Hkv, g = bg - b * rows.Hkv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = seq_lens[b];
  if (n < 0 || n > Lout || n > rows.Lmax) {
    if (is_k && blk == 0 && g == 0 && threadIdx.x == 0) atomicOr(status, kStatusDeviceArg);
    return;  // the sequence is left as it was
  }
  const uint8_t* src = is_k ? k_cache : v_cache;
  const uint8_t* scale = is_k ? k_scale : v_scale;
  __nv_bfloat16* dst = (is_k ? k_out : v_out) + static_cast<size_t>(bg) * Lout * D;
  const int i0 = blk * (kThreads * kRows) + static_cast<int>(threadIdx.x);
  uint32_t x[kRows], code[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = i0 + k * kThreads, r = i / G, c = i % G;
    x[k] = code[k] = 0u;
    if (r < n) {
      const long long row = rows.at(b, g, r);
      if (row >= 0) {
        x[k] = *reinterpret_cast<const uint32_t*>(src + row * (D / 2) + 4 * c);
        code[k] = scale[row * (D / 16) + c / 2];
      } else if (c == 0) {
        atomicOr(status, kStatusDeviceArg);  // the row reads as zeros
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = i0 + k * kThreads, r = i / G, c = i % G;
    if (r >= n) break;
    const float s = fp4_scale(code[k]);
    *reinterpret_cast<uint4*>(dst + static_cast<size_t>(r) * D + 8 * c) =
        make_uint4(to_bf16x2(e2m1x2_to_f16x2<0>(x[k]), s), to_bf16x2(e2m1x2_to_f16x2<1>(x[k]), s),
                   to_bf16x2(e2m1x2_to_f16x2<2>(x[k]), s), to_bf16x2(e2m1x2_to_f16x2<3>(x[k]), s));
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
  p.items = static_cast<unsigned>(static_cast<long long>(a.B) * a.Hkv * a.Tn * (a.d / 8));
  p.status = a.status;
  auto* kernel = a.d == 128 ? append_fp4_kernel<128> : append_fp4_kernel<64>;
  return launch_behind(kernel, dim3(static_cast<unsigned>((p.items + kThreads - 1) / kThreads)),
                       kThreads, stream, p);
}

cudaError_t launch_cache_read_fp4(const KvCache& cache, const int32_t* seq_lens, void* k_out,
                                  void* v_out, int B, int Hkv, int Lout, int d, uint32_t* status,
                                  cudaStream_t stream) {
  const long long pieces = static_cast<long long>(std::min(Lout, cache.Lmax)) * (d / 8);
  const long long blocks = (pieces + kThreads * kRows - 1) / (kThreads * kRows);
  // (a grid below 2^31: B * Hkv < 2^30, and B * Hkv * Lout < 2^33 where there are more blocks)
  auto* kernel = d == 128 ? read_fp4_kernel<128> : read_fp4_kernel<64>;
  return launch_behind(kernel, dim3(static_cast<unsigned>(2 * blocks * B * Hkv)), kThreads, stream,
                       static_cast<const uint8_t*>(cache.k), static_cast<const uint8_t*>(cache.v),
                       static_cast<const uint8_t*>(cache.k_scale),
                       static_cast<const uint8_t*>(cache.v_scale), seq_lens, rows_of(cache, Hkv),
                       static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), Lout,
                       status, static_cast<int>(blocks));
}

}  // namespace csattn
