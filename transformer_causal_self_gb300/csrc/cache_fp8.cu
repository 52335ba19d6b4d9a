// The 8-bit KV cache as it is written and read back (format: fp8.cuh).
//
// Append: token t of sequence b goes to row r = cache_lens[b] + t, its key rotated at r
// in fp32 and rounded once, to e4m3; the value is rounded as given.  Read: rows
// 0..seq_lens[b]-1 back to bf16, exactly.  Both move each byte once and are bound by
// HBM (4 bytes in, 2 + 1/64 out per channel pair; the reverse for the read), by latency where
// they are short.  128 channels, 8 KV heads: the append of 4 x 4096 tokens takes 20.9 us (101 MB,
// 4.8 TB/s: less than two waves, whose loads, angles and stores follow one another), of 64 tokens
// 2.8 us; the read of 32768 rows 33.0 us (202 MB, 6.1 TB/s), of 8 x 17..1024 rows 4.9 us.
#include <algorithm>

#include "fp8.cuh"
#include "internal.h"

namespace csattn {
namespace {

constexpr int kThreads = 128;  // (256: 0.2 to 0.6 us more, a block's ends being further apart)
constexpr int kHeads = 2;  // KV heads whose loads (two each) a thread has in flight

// Thread item (b, head group, t, c): 16 channels of a token in `span` KV heads, kHeads at a time;
// the G = d/16 threads of a row are neighbouring lanes.  The first k_blocks blocks take the
// keys (whose angles serve all of the thread's heads), the others the values.
// (Seven blocks per SM: eight leave 64 registers and spill, 22.3 us for the prompts above against
// 20.9; six take 24.2.)
template <int D>
__global__ void __launch_bounds__(kThreads, 7) append_fp8_kernel(
    const __nv_bfloat16* __restrict__ k_new, const __nv_bfloat16* __restrict__ v_new,
    uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, uint8_t* __restrict__ k_scale,
    uint8_t* __restrict__ v_scale, const int32_t* __restrict__ cache_lens, CacheRows rows, int B,
    int Tn, int span, int rope, RopeTable theta, uint32_t* status, int k_blocks) {
  constexpr int G = D / 16;
  __shared__ float th_hi[64], th_lo[64];
  const int tid = static_cast<int>(threadIdx.x);
  const bool is_k = static_cast<int>(blockIdx.x) < k_blocks;
  const int layout = is_k ? rope : 0;
  if (layout != 0 && tid < D / 2) {
    th_hi[tid] = theta.hi[tid];
    th_lo[tid] = theta.lo[tid];
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int Hkv = rows.Hkv;
  const int groups = (Hkv + span - 1) / span;
  // (32-bit indices: B * Hkv * Tn * d < 2^33, so there are no more than 2^29 items)
  int i = (static_cast<int>(blockIdx.x) - (is_k ? 0 : k_blocks)) * kThreads + tid;
  bool live = i < B * groups * Tn * G;
  if (!live) i = 0;
  const int c = i % G;
  i /= G;
  const int t = i % Tn;
  i /= Tn;
  const int g0 = (i % groups) * span;
  const int b = i / groups;
  const int g1 = min(Hkv, g0 + span);
  int e0, e1;
  // (16 channels in a row where the rotation does not pair channel p with p + d/2: one store)
  const bool whole = layout != 1;
  rope_piece(whole ? 2 : 1, D / 2, c, &e0, &e1);
  const __nv_bfloat16* src =
      (is_k ? k_new : v_new) + (static_cast<size_t>(b) * Hkv * Tn + t) * D;
  const size_t head_step = static_cast<size_t>(Tn) * D;
  uint4 lo[kHeads], hi[kHeads];
  auto load = [&](int g) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      lo[k] = hi[k] = make_uint4(0u, 0u, 0u, 0u);
      if (g + k < g1) {
        lo[k] = *reinterpret_cast<const uint4*>(src + (g + k) * head_step + e0);
        hi[k] = *reinterpret_cast<const uint4*>(src + (g + k) * head_step + e1);
      }
    }
  };
  load(g0);
  const int L = cache_lens[b];
  if (L < 0 || L > rows.Lmax - Tn) {  // (no overflow: Lmax, Tn < 2^30)
    if (live && is_k && t == 0 && c == 0 && g0 == 0) atomicOr(status, kStatusDeviceArg);
    live = false;
  }
  // the row of KV head 0, and rows from a head to the next
  const long long row0 = live ? rows.at(b, 0, L + t) : 0;
  const long long row_step = rows.block_table == nullptr ? rows.Lmax : rows.page_size;
  if (row0 < 0) {
    if (c == 0) atomicOr(status, kStatusDeviceArg);
    live = false;
  }
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (layout != 0)
      angle_cos_sin(L + t, th_hi[8 * c + j], th_lo[8 * c + j], cs[j], sn[j]);
  }
  uint8_t* const out = is_k ? k_cache : v_cache;
  uint8_t* const scale = is_k ? k_scale : v_scale;
  // (a block's threads have the same number of rounds but for the last head group's: `span` is
  // a multiple of kHeads or all heads, and the bound below does not depend on the group)
  for (int s0 = 0; s0 < span; s0 += kHeads) {
    if (s0 > 0) load(g0 + s0);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      bool bad;
      const uint32_t top = row_absmax<G>(lo[k], hi[k], &bad);
      if (!live || g0 + s0 + k >= g1) continue;  // (no shuffle below)
      const long long row = row0 + (g0 + s0 + k) * row_step;
      const int code = scale_code(top, layout != 0);
      float y[16];
      rope16(scale_row(lo[k], code), scale_row(hi[k], code), layout, cs, sn, y);
      uint8_t* dst = out + row * D;
      const uint4 x = make_uint4(pack_e4m3x4(y[0], y[1], y[2], y[3], code, bad),
                                 pack_e4m3x4(y[4], y[5], y[6], y[7], code, bad),
                                 pack_e4m3x4(y[8], y[9], y[10], y[11], code, bad),
                                 pack_e4m3x4(y[12], y[13], y[14], y[15], code, bad));
      if (whole) {
        *reinterpret_cast<uint4*>(dst + e0) = x;
      } else {
        *reinterpret_cast<uint2*>(dst + e0) = make_uint2(x.x, x.y);
        *reinterpret_cast<uint2*>(dst + e1) = make_uint2(x.z, x.w);
      }
      if (c == 0) scale[row] = static_cast<uint8_t>(code);
    }
  }
}

// two e4m3 times 2^(code - 127) as bf16x2: both steps are exact for the codes a write makes
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two, float s) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x * s, f.y * s);
}

// 16 channels per thread item (b, g, r, c); consecutive items are consecutive rows of a
// sequence's KV head.  Blocks of a (b, g): k_blocks for the keys, then as many for the values.
constexpr int kRows = 2;  // row pieces per thread, kThreads apart: as many loads in flight
template <int D>
__global__ void __launch_bounds__(kThreads) read_fp8_kernel(
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale,
    const int32_t* __restrict__ seq_lens, CacheRows rows, __nv_bfloat16* __restrict__ k_out,
    __nv_bfloat16* __restrict__ v_out, int Lout, uint32_t* status, int k_blocks) {
  constexpr int G = D / 16;
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
  uint4 x[kRows];
  uint32_t code[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = i0 + k * kThreads, r = i / G, c = i % G;
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    code[k] = 0u;
    if (r < n) {
      const long long row = rows.at(b, g, r);
      if (row >= 0) {
        x[k] = *reinterpret_cast<const uint4*>(src + row * D + 16 * c);
        code[k] = scale[row];
      } else if (c == 0) {
        atomicOr(status, kStatusDeviceArg);  // the row reads as zeros
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = i0 + k * kThreads, r = i / G, c = i % G;
    if (r >= n) break;
    const float s = __uint_as_float(code[k] << 23);
    uint4* o = reinterpret_cast<uint4*>(dst + static_cast<size_t>(r) * D + 16 * c);
    o[0] = make_uint4(e4m3x2_to_bf16x2(x[k].x, s), e4m3x2_to_bf16x2(x[k].x >> 16, s),
                      e4m3x2_to_bf16x2(x[k].y, s), e4m3x2_to_bf16x2(x[k].y >> 16, s));
    o[1] = make_uint4(e4m3x2_to_bf16x2(x[k].z, s), e4m3x2_to_bf16x2(x[k].z >> 16, s),
                      e4m3x2_to_bf16x2(x[k].w, s), e4m3x2_to_bf16x2(x[k].w >> 16, s));
  }
}

CacheRows rows_of(const KvCache& c, int Hkv) {
  return CacheRows{c.block_table, Hkv, c.Lmax, c.page_size, c.num_pages, c.max_pages};
}

}  // namespace

cudaError_t launch_cache_append_fp8(const void* k_new, const void* v_new, const KvCache& cache,
                                    const int32_t* cache_lens, int B, int Hkv, int Tn, int d,
                                    int rope, const RopeTable& theta, uint32_t* status,
                                    cudaStream_t stream) {
  // All heads of a token in one thread while that still fills the GPU (one set of angles serves
  // them all): six blocks per SM; otherwise kHeads of them.
  const long long tokens = static_cast<long long>(B) * Tn * (d / 16);
  const int span = 2 * tokens >= 6LL * kSms * kThreads ? Hkv : std::min(Hkv, kHeads);
  const long long items = tokens * ((Hkv + span - 1) / span);
  const int blocks = static_cast<int>((items + kThreads - 1) / kThreads);
  auto* kernel = d == 128 ? append_fp8_kernel<128> : append_fp8_kernel<64>;
  return launch_behind(kernel, dim3(2 * blocks), kThreads, stream,
                       static_cast<const __nv_bfloat16*>(k_new),
                       static_cast<const __nv_bfloat16*>(v_new), static_cast<uint8_t*>(cache.k),
                       static_cast<uint8_t*>(cache.v), static_cast<uint8_t*>(cache.k_scale),
                       static_cast<uint8_t*>(cache.v_scale), cache_lens, rows_of(cache, Hkv), B, Tn,
                       span, rope, theta, status, blocks);
}

cudaError_t launch_cache_read_fp8(const KvCache& cache, const int32_t* seq_lens, void* k_out,
                                  void* v_out, int B, int Hkv, int Lout, int d, uint32_t* status,
                                  cudaStream_t stream) {
  const long long pieces = static_cast<long long>(std::min(Lout, cache.Lmax)) * (d / 16);
  const long long blocks = (pieces + kThreads * kRows - 1) / (kThreads * kRows);
  // (a grid below 2^31: B * Hkv < 2^30, and B * Hkv * Lout < 2^33 where there are more blocks)
  auto* kernel = d == 128 ? read_fp8_kernel<128> : read_fp8_kernel<64>;
  return launch_behind(kernel, dim3(static_cast<unsigned>(2 * blocks * B * Hkv)), kThreads, stream,
                       static_cast<const uint8_t*>(cache.k), static_cast<const uint8_t*>(cache.v),
                       static_cast<const uint8_t*>(cache.k_scale),
                       static_cast<const uint8_t*>(cache.v_scale), seq_lens, rows_of(cache, Hkv),
                       static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), Lout,
                       status, static_cast<int>(blocks));
}

}  // namespace csattn
