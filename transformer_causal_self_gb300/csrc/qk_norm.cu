// RMS norm of every head's queries and keys, its gain and the rotation, in one pass; and the
// gradients of that pass.
//
//   forward:  y = R_pos (n o w),  n = x r,  r = 1 / sqrt(mean(x^2) + eps)   over a head's d channels
//   backward: g = R_pos^T dy,  dx = r (g o w - n mean(g o w o n)),  dw = sum over rows of g o n
//             (r is worked out again from x: that costs no traffic, x is read for n anyway)
//
// A thread has 16 channels of a token, in two pieces of eight that hold whole pairs of the
// rotation, so the d/16 lanes of a row exchange nothing but the sums.  Its pieces' eight angles
// serve all heads that it takes of its token.  Everything between the load and the store is fp32,
// and each value is rounded once.  Both directions move each value once and are bound by HBM,
// by latency where there are few tokens.
#include <algorithm>

#include "fp8.cuh"
#include "internal.h"
#include "rope_turns.cuh"

namespace csattn {
namespace {

constexpr int kThreads = 128;
constexpr int kSumThreads = 512;

template <typename T>
struct Piece;  // eight channels as loaded
template <>
struct Piece<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float* y) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = bf16lo_to_f32(w[i]);
      y[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* y) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                   pack_bf16x2(y[6], y[7]));
  }
};
template <>
struct Piece<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* y) const {
    y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w;
    y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* y) {
    reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
};

// The pairs of 16 channels (u 0..7, v 8..15): split-half (u_i, v_i) with angle i, adjacent
// (u_2i, u_2i+1) with angle i and (v_2i, v_2i+1) with angle 4 + i.  sign -1: turned back.
__device__ __forceinline__ void turn16(float (&y)[16], int layout, const float (&cs)[8],
                                       const float (&sn)[8], float sign) {
  auto turn = [&](int p, int q, int i) {
    const float u = y[p], v = y[q], s = sign * sn[i];
    y[p] = fmaf(u, cs[i], -v * s);
    y[q] = fmaf(u, s, v * cs[i]);
  };
  if (layout == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(i, 8 + i, i);
  } else if (layout == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(2 * i, 2 * i + 1, i);
  }
}

template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What one thread does: 16 channels of a token in `span` heads from g0.
struct Item {
  int b, t, g0, c, e0, e1;
};
template <int D>
__device__ __forceinline__ Item item_of(unsigned i, int T, int groups, int span, int layout) {
  constexpr int G = D / 16;
  Item it;
  it.c = i % G;
  i /= G;
  it.t = i % T;
  i /= T;
  it.g0 = (i % groups) * span;
  it.b = i / groups;
  rope_piece(layout == 1 ? 1 : 2, D / 2, it.c, &it.e0, &it.e1);
  return it;
}

// cos and sin of the thread's eight angles at the token's position
__device__ __forceinline__ void angles(const QkNormArgs& a, const Item& it, bool live, bool tell,
                                       const float* th_hi, const float* th_lo, float (&cs)[8],
                                       float (&sn)[8]) {
  if (a.rope == 0) return;
  int pos = a.pos0 + it.t;
  if (a.positions != nullptr) {
    pos = a.positions[static_cast<size_t>(it.b) * a.T + it.t];
    if (pos < 0 || pos >= (1 << 24)) {  // (the token's outputs are then not meaningful)
      if (live && tell) atomicOr(a.status, kStatusDeviceArg);
      pos = 0;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    turn_cos_sin(pos, th_hi[8 * it.c + j], th_lo[8 * it.c + j], cs[j], sn[j]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const __grid_constant__ QkNormArgs a) {
  constexpr int G = D / 16;
  constexpr int U = sizeof(T) == 2 ? 2 : 1;  // heads whose loads are in flight together
  __shared__ float th_hi[64], th_lo[64];
  const int tid = static_cast<int>(threadIdx.x);
  if (a.rope != 0 && tid < D / 2) {
    th_hi[tid] = a.turns.hi[tid];
    th_lo[tid] = a.turns.lo[tid];
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool is_q = static_cast<int>(blockIdx.x) < a.q_blocks;
  const QkNormSide& s = is_q ? a.q : a.k;
  unsigned i = (blockIdx.x - (is_q ? 0 : a.q_blocks)) * kThreads + tid;
  const bool live = i < s.items;
  if (!live) i = 0;
  const Item it = item_of<D>(i, a.T, s.groups, s.span, a.rope);
  const T* src = static_cast<const T*>(s.x) + it.b * s.batch + it.t * s.token;
  T* dst = static_cast<T*>(s.y) + (static_cast<size_t>(it.b) * s.H * a.T + it.t) * D;
  Piece<T> lo[U], hi[U];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      lo[u].clear();
      hi[u].clear();
      if (h0 + u < s.H) {
        lo[u].load(src + (h0 + u) * s.head + it.e0);
        hi[u].load(src + (h0 + u) * s.head + it.e1);
      }
    }
  };
  load(it.g0);
  float w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = 1.f;
  if (s.w != nullptr) {
    Piece<T> p;
    p.load(static_cast<const T*>(s.w) + it.e0);
    p.get(w);
    p.load(static_cast<const T*>(s.w) + it.e1);
    p.get(w + 8);
  }
  float cs[8], sn[8];
  angles(a, it, live, is_q && it.g0 == 0 && it.c == 0, th_hi, th_lo, cs, sn);
  // (the same number of rounds for all lanes of a warp, whatever their heads)
  for (int r = 0; r < s.span; r += U) {
    if (r > 0) load(it.g0 + r);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[16];
      lo[u].get(y);
      hi[u].get(y + 8);
      if (a.norm) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum = fmaf(y[j], y[j], sum);
        const float rs = rsqrtf(fmaf(row_sum<G>(sum), 1.f / D, a.eps));
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] *= rs * w[j];
      }
      turn16(y, a.rope, cs, sn, 1.f);
      const int h = it.g0 + r + u;
      if (live && r + u < s.span && h < s.H) {
        T* out = dst + static_cast<size_t>(h) * a.T * D;
        Piece<T>::store(out + it.e0, y);
        Piece<T>::store(out + it.e1, y + 8);
      }
    }
  }
}

// Blocks take items kThreads * (blocks of the side) apart; what a block has of dw is added up in
// it and left for sum_kernel, so that the order of all sums depends on the sizes alone.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const __grid_constant__ QkNormArgs a) {
  constexpr int G = D / 16;
  constexpr int kWarps = kThreads / 32;
  __shared__ float th_hi[64], th_lo[64];
  __shared__ float s_dw[kWarps][D];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  if (a.rope != 0 && tid < D / 2) {
    th_hi[tid] = a.turns.hi[tid];
    th_lo[tid] = a.turns.lo[tid];
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool is_q = static_cast<int>(blockIdx.x) < a.q_blocks;
  const QkNormSide& s = is_q ? a.q : a.k;
  const unsigned blk = blockIdx.x - (is_q ? 0 : a.q_blocks);
  const unsigned step = (is_q ? a.q_blocks : gridDim.x - a.q_blocks) * kThreads;
  const int c = tid % G;  // (the same in every round: kThreads is a multiple of G)
  int e0, e1;
  rope_piece(a.rope == 1 ? 1 : 2, D / 2, c, &e0, &e1);
  float w[16], dw[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = 1.f, dw[j] = 0.f;
  if (s.w != nullptr) {
    Piece<T> p;
    p.load(static_cast<const T*>(s.w) + e0);
    p.get(w);
    p.load(static_cast<const T*>(s.w) + e1);
    p.get(w + 8);
  }
  for (unsigned i0 = blk * kThreads; i0 < s.items; i0 += step) {
    const bool live = i0 + tid < s.items;
    const Item it = item_of<D>(live ? i0 + tid : c, a.T, s.groups, s.span, a.rope);
    const T* x = static_cast<const T*>(s.x) + it.b * s.batch + it.t * s.token;
    const T* dy = static_cast<const T*>(s.y) + (static_cast<size_t>(it.b) * s.H * a.T + it.t) * D;
    T* dx = static_cast<T*>(s.dx) + it.b * s.dx_batch + it.t * s.dx_token;
    float cs[8], sn[8];
    angles(a, it, live, is_q && it.g0 == 0 && it.c == 0, th_hi, th_lo, cs, sn);
    for (int r = 0; r < s.span; ++r) {
      const int h = it.g0 + r;
      const bool mine = live && h < s.H;
      Piece<T> xl, xh, gl, gh;
      xl.clear(), xh.clear(), gl.clear(), gh.clear();
      if (mine) {
        xl.load(x + h * s.head + e0);
        xh.load(x + h * s.head + e1);
        gl.load(dy + static_cast<size_t>(h) * a.T * D + e0);
        gh.load(dy + static_cast<size_t>(h) * a.T * D + e1);
      }
      float g[16];
      gl.get(g);
      gh.get(g + 8);
      turn16(g, a.rope, cs, sn, -1.f);
      if (a.norm) {
        float y[16];
        xl.get(y);
        xh.get(y + 8);
        float sq = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          sq = fmaf(y[j], y[j], sq);
          dot = fmaf(g[j] * w[j], y[j], dot);
        }
        sq = row_sum<G>(sq);
        dot = row_sum<G>(dot);
        // (a lane without a row adds nothing: its gradient is 0, and eps > 0 or not, 0 * r must be)
        const float rs = mine ? rsqrtf(fmaf(sq, 1.f / D, a.eps)) : 0.f;
        const float m = dot * rs * (1.f / D);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float n = y[j] * rs;
          dw[j] = fmaf(g[j], n, dw[j]);
          g[j] = rs * fmaf(-n, m, g[j] * w[j]);
        }
      }
      if (mine) {
        Piece<T>::store(dx + h * s.dx_head + e0, g);
        Piece<T>::store(dx + h * s.dx_head + e1, g + 8);
      }
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
    if (lane < G) s_dw[warp][j < 8 ? e0 + j : e1 + j - 8] = dw[j];
  }
  __syncthreads();
  for (int j = tid; j < D; j += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += s_dw[v][j];
    a.partial[static_cast<size_t>(blockIdx.x) * D + j] = sum;
  }
}

// dw of the queries' (block 0) or the keys' gain: the blocks' sums in a fixed order
template <int D>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const float* __restrict__ partial,
                                                          int q_blocks, int blocks,
                                                          float* __restrict__ dqw,
                                                          float* __restrict__ dkw) {
  constexpr int kParts = kSumThreads / D;
  __shared__ float s[kParts][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool is_q = blockIdx.x == 0;
  float* out = is_q ? dqw : dkw;
  if (out == nullptr) return;
  const int ch = threadIdx.x % D, part = threadIdx.x / D;
  const int first = is_q ? 0 : q_blocks, last = is_q ? q_blocks : blocks;
  float sum = 0.f;
#pragma unroll 8
  for (int i = first + part; i < last; i += kParts) sum += partial[static_cast<size_t>(i) * D + ch];
  s[part][ch] = sum;
  __syncthreads();
  if (part != 0) return;
#pragma unroll
  for (int v = 1; v < kParts; ++v) sum += s[v][ch];
  out[ch] = sum;
}

// heads per thread and threads of a side: all heads of a token in one thread while that still
// fills the GPU, otherwise `least` of them
void share(QkNormSide& s, const QkNormArgs& a, int least) {
  const long long tokens = static_cast<long long>(a.B) * a.T * (a.d / 16);
  int groups = 1;
  while (groups * least < s.H && tokens * groups < 8LL * kSms * kThreads) groups *= 2;
  s.span = (s.H + groups - 1) / groups;
  s.groups = (s.H + s.span - 1) / s.span;
  s.items = static_cast<unsigned>(tokens * s.groups);
}
unsigned blocks_of(const QkNormSide& s) { return (s.items + kThreads - 1) / kThreads; }

template <typename T>
cudaError_t forward(const QkNormArgs& a, unsigned grid, cudaStream_t stream) {
  if (a.d == 128) return launch_behind(qk_norm_kernel<T, 128>, dim3(grid), kThreads, stream, a);
  if (a.d == 64) return launch_behind(qk_norm_kernel<T, 64>, dim3(grid), kThreads, stream, a);
  if constexpr (sizeof(T) == 4) {
    if (a.d == 32) return launch_behind(qk_norm_kernel<T, 32>, dim3(grid), kThreads, stream, a);
    return launch_behind(qk_norm_kernel<T, 16>, dim3(grid), kThreads, stream, a);
  }
  return cudaErrorInvalidValue;
}
template <typename T, int D>
cudaError_t backward_t(const QkNormArgs& a, unsigned grid, float* dqw, float* dkw,
                       cudaStream_t stream) {
  cudaError_t e = launch_behind(qk_norm_bwd_kernel<T, D>, dim3(grid), kThreads, stream, a);
  if (e != cudaSuccess || a.partial == nullptr) return e;
  return launch_behind(sum_kernel<D>, dim3(2), kSumThreads, stream,
                       static_cast<const float*>(a.partial), a.q_blocks, static_cast<int>(grid),
                       dqw, dkw);
}
template <typename T>
cudaError_t backward(const QkNormArgs& a, unsigned grid, float* dqw, float* dkw,
                     cudaStream_t stream) {
  if (a.d == 128) return backward_t<T, 128>(a, grid, dqw, dkw, stream);
  if (a.d == 64) return backward_t<T, 64>(a, grid, dqw, dkw, stream);
  if constexpr (sizeof(T) == 4) {
    if (a.d == 32) return backward_t<T, 32>(a, grid, dqw, dkw, stream);
    return backward_t<T, 16>(a, grid, dqw, dkw, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_qk_norm(QkNormArgs a, bool bf16, cudaStream_t stream) {
  const int least = bf16 ? 2 : 1;
  share(a.q, a, least);
  share(a.k, a, least);
  a.q_blocks = static_cast<int>(blocks_of(a.q));
  const unsigned grid = a.q_blocks + blocks_of(a.k);
  return bf16 ? forward<__nv_bfloat16>(a, grid, stream) : forward<float>(a, grid, stream);
}

cudaError_t launch_qk_norm_bwd(QkNormArgs a, bool bf16, float* dqw, float* dkw,
                               cudaStream_t stream) {
  share(a.q, a, 1);
  share(a.k, a, 1);
  // blocks by the heads, no more than there is work for
  const long long all = qk_norm_bwd_blocks();
  const int nq = static_cast<int>(std::min<long long>(
      blocks_of(a.q), std::max(1LL, all * a.q.H / (a.q.H + a.k.H))));
  const int nk = static_cast<int>(
      std::min<long long>(blocks_of(a.k), std::max(1LL, all - all * a.q.H / (a.q.H + a.k.H))));
  a.q_blocks = nq;
  return bf16 ? backward<__nv_bfloat16>(a, nq + nk, dqw, dkw, stream)
              : backward<float>(a, nq + nk, dqw, dkw, stream);
}

}  // namespace csattn
