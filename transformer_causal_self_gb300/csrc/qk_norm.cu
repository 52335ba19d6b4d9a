// RMS norm of every head's queries and keys, its gain and the rotation, in one pass; and the
// gradients of that pass.
//
//   forward:  y = R_pos (n o w),  n = x r,  r = 1 / sqrt(mean(x^2) + eps)   over a head's d channels
//   backward: g = R_pos^T dy,  dx = r (g o w - n mean(g o w o n)),  dw = sum over rows of g o n
//             (r is worked out again from x: that costs no traffic, x is read for n anyway)
//
// A thread has two runs of 16 bytes of a token, half a head apart, which hold whole pairs of the
// rotation in either layout: a row's lanes exchange nothing but the sums, and their loads touch.
// Its pairs' angles serve all heads that it takes of its token.  Everything between the load and
// the store is fp32, and each value is rounded once.
//
// Both directions move each value once.  Forward, 4 x 4096 tokens of 32 + 8 heads of 128 (bf16, out
// of a fused projection): 53.0 us for 336 MB, 6.3 TB/s, 94 % of a plain copy, with 76 % of the
// issue slots busy; 64 tokens 2.8 us.  Backward, 2 x 4096 tokens: 45.0 us for 252 MB, 5.6 TB/s, bound
// by the latency that 12 warps of 143 registers cover (with the rows in registers instead of shared
// memory 63.7 us, with runs half as long and more warps 67).  fp32, 8 x 1024 tokens of 24 heads of
// 64: 17.0 and 27.6 us for 101 and 151 MB.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"
#include "internal.h"
#include "rope_turns.cuh"

namespace csattn {
namespace {

constexpr int kThreads = 128;
// Channels of a piece: 16 bytes, so that neighbouring lanes' loads touch.
template <typename T>
constexpr int kPiece = 16 / sizeof(T);
constexpr int kSumThreads = 512;

// N channels as loaded
template <typename T, int N>
struct Piece {
  static_assert(N * sizeof(T) == 16, "one load");
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p) {
    *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void get(float* y) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 2)
        y[i] = i % 2 == 0 ? bf16lo_to_f32(w[i / 2]) : bf16hi_to_f32(w[i / 2]);
      else
        y[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void put(const float* y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2)
        w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
      else
        w[i] = __float_as_uint(y[i]);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
  }
};

// The pairs of 2 N channels (u 0..N-1, v N..2N-1): split-half (u_i, v_i) with angle i, adjacent
// (u_2i, u_2i+1) with angle i and (v_2i, v_2i+1) with angle N / 2 + i.  sign -1: turned back.
template <int N>
__device__ __forceinline__ void turn(float (&y)[2 * N], int layout, const float (&cs)[N],
                                     const float (&sn)[N], float sign) {
  auto one = [&](int p, int q, int i) {
    const float u = y[p], v = y[q], s = sign * sn[i];
    y[p] = fmaf(u, cs[i], -v * s);
    y[q] = fmaf(u, s, v * cs[i]);
  };
  if (layout == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) one(i, N + i, i);
  } else if (layout == 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) one(2 * i, 2 * i + 1, i);
  }
}

template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Whether a mean square (with eps; not negative) is outside [2^-80, 2^120), where squares may have been
// lost to either end of fp32's range, or is NaN: one comparison of its bits.
__device__ __forceinline__ bool out_of_range(float ms) {
  return __float_as_uint(ms) - (47u << 23) >= 200u << 23;
}

// mean(x^2) + eps of a row out of that range, from its channels y times a power of two f, which is
// returned (1 for the warp's other rows): of 1 / top, top the larger of the largest |y| and
// sqrt(eps), as far as f is a normal number.  ms becomes f^2 times the mean square with eps, so that
// y rsqrt(ms) is what it was, and 1 / sqrt(mean(x^2) + eps) is f rsqrt(ms).  A row with an
// infinity or NaN is left as it was.  All lanes of the warp call it.
template <int D, int N, int G>
__device__ __forceinline__ float rescale(float (&y)[2 * N], float eps, float& ms) {
  float top = sqrtf(eps);
#pragma unroll
  for (int j = 0; j < 2 * N; ++j) top = fmaxf(top, fabsf(y[j]));
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int e = static_cast<int>(__float_as_uint(top) >> 23);
  const float f = out_of_range(ms) && e < 255
                      ? __uint_as_float(static_cast<uint32_t>(min(max(254 - e, 27), 253)) << 23)
                      : 1.f;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 2 * N; ++j) {
    y[j] *= f;
    sum = fmaf(y[j], y[j], sum);
  }
  ms = fmaf(row_sum<G>(sum), 1.f / D, eps * f * f);
  return f;
}

// What one thread does: 2 N channels of a token in `span` heads from g0.
struct Item {
  int b, t, g0, c;
};
template <int G>
__device__ __forceinline__ Item item_of(unsigned i, int T, int groups, int span) {
  Item it;
  it.c = i % G;
  i /= G;
  it.t = i % T;
  i /= T;
  it.g0 = (i % groups) * span;
  it.b = i / groups;
  return it;
}

// cos and sin of the thread's N angles at the token's position: those of its pairs, channels N c..
// with D / 2 + N c.. (split-half), or the neighbours within either run (adjacent)
template <int D, int N>
__device__ __forceinline__ void angles(const QkNormArgs& a, const Item& it, bool tell,
                                       const float* th_hi, const float* th_lo, float (&cs)[N],
                                       float (&sn)[N]) {
  if (a.rope == 0) return;
  int pos = a.pos0 + it.t;
  if (a.positions != nullptr) {
    pos = a.positions[static_cast<size_t>(it.b) * a.T + it.t];
    if (pos < 0 || pos >= (1 << 24)) {  // (the token's outputs are then not meaningful)
      if (tell) atomicOr(a.status, kStatusDeviceArg);
      pos = 0;
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int at = a.rope == 1 ? N * it.c + j : N / 2 * it.c + j % (N / 2) + (2 * j < N ? 0 : D / 4);
    turn_cos_sin(pos, th_hi[at], th_lo[at], cs[j], sn[j]);
  }
}

// the lane's gains; 1 without any
template <typename T, int N>
__device__ __forceinline__ void gains(const void* w, int e0, int e1, float (&y)[2 * N]) {
#pragma unroll
  for (int j = 0; j < 2 * N; ++j) y[j] = 1.f;
  if (w == nullptr) return;
  Piece<T, N> p;
  p.load(static_cast<const T*>(w) + e0);
  p.get(y);
  p.load(static_cast<const T*>(w) + e1);
  p.get(y + N);
}

// 16 bytes to shared memory without a register between; zeros where `there` is false
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

// Blocks take items kThreads * (blocks of the side) apart; what a block has of dw is added up in
// it and left for sum_kernel, so that the order of all sums depends on the sizes alone.
// A thread's heads, of one item after the other, are a line of steps; their x (and dy) come
// kAhead steps ahead through shared memory, where each thread reads what it copied itself (in
// registers they leave room for too few threads to cover the memory's latency).
constexpr int kAhead = 2;
template <bool BWD>
constexpr int kStage = (BWD ? 4 : 2) * kThreads * 16;  // of a step: two pieces of x (and of dy)
template <bool BWD>
constexpr int kRing = (kAhead + 1) * kStage<BWD>;
// A thread adds its rows' terms of dw in fp32.  Past kMany of them (2^-14 of the sum, if all their
// roundings went one way) another kernel does it, LONG, which moves what it has to a sum of 64 bits
// behind the ring when an item begins and kFold rows or more were added: 8 x 8192 tokens of 32 + 8
// heads of 128, 576 rows a thread, 387 us with it and 366 without, 2 x 4096 tokens 47.6 and 45.0.
constexpr int kMany = 1024, kFold = 64;
template <typename T, bool BWD, bool LONG>
constexpr int kShared = kRing<BWD> + (LONG ? 2 * kPiece<T> * kThreads * 8 : 0);
template <typename T, int D, bool BWD, bool LONG>
__global__ void __launch_bounds__(kThreads, BWD ? 3 : 6)
    qk_norm_kernel(const __grid_constant__ QkNormArgs a) {
  constexpr int N = kPiece<T>, G = D / (2 * N);
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint8_t s_stage[];
  __shared__ float th_hi[64], th_lo[64];
  __shared__ float s_dw[BWD ? kWarps : 1][D];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  if (a.rope != 0 && tid < D / 2) {
    th_hi[tid] = a.turns.hi[tid];
    th_lo[tid] = a.turns.lo[tid];
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (BWD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool is_q = static_cast<int>(blockIdx.x) < a.q_blocks;
  const QkNormSide& s = is_q ? a.q : a.k;
  const unsigned first = (blockIdx.x - (is_q ? 0 : a.q_blocks)) * kThreads;
  const unsigned step = (is_q ? a.q_blocks : gridDim.x - a.q_blocks) * kThreads;
  const int c = tid % G;  // (the same in every round: kThreads is a multiple of G)
  const int e0 = N * c, e1 = D / 2 + N * c;

  const uint32_t mine_at = smem_u32(s_stage) + tid * 16;
  const int total =
      first < s.items ? static_cast<int>((s.items - first + step - 1) / step) * s.span : 0;
  float w[2 * N], dw[2 * N];
  gains<T, N>(s.w, e0, e1, w);
#pragma unroll
  for (int j = 0; j < 2 * N; ++j) dw[j] = 0.f;
  // The backward pass goes over its rows a second time where squares of one left fp32's range, for
  // those alone: with a branch in the first sweep all the others take 46 to 48 us instead of 45
  // (2 x 4096 tokens; 44 without either).
  bool again = false;
  double* far = reinterpret_cast<double*>(s_stage + kRing<BWD>) + tid;  // [2 N], kThreads apart
  bool folded = false;
  auto sweep = [&](auto second) {
    constexpr bool kAgain = decltype(second)::value;
    // the step that is loaded next
    unsigned li = first;
    int lr = 0, lh = 0, lbuf = 0;
    const T* lx = nullptr;
    const T* ly = nullptr;
    bool llive = false;
    auto load = [&](bool any) {
      if (any) {
        if (lr == 0) {
          llive = li + tid < s.items;
          const Item it = item_of<G>(llive ? li + tid : c, a.T, s.groups, s.span);
          lx = static_cast<const T*>(s.x) + it.b * s.batch + it.g0 * s.head + it.t * s.token;
          if (BWD)
            ly = static_cast<const T*>(s.dy) +
                 ((static_cast<size_t>(it.b) * s.H + it.g0) * a.T + it.t) * D;
          lh = it.g0;
        }
        const bool there = llive && lh < s.H;
        const uint32_t dst = mine_at + lbuf * kStage<BWD>;
        copy16(dst, lx + e0, there);
        copy16(dst + kThreads * 16, lx + e1, there);
        if (BWD) {
          copy16(dst + 2 * kThreads * 16, ly + e0, there);
          copy16(dst + 3 * kThreads * 16, ly + e1, there);
        }
        // (the pointers of a head that is not there are not followed: its 0 bytes are read)
        if (++lr == s.span) {
          lr = 0;
          li += step;
        } else {
          ++lh;
          lx += there ? s.head : 0;
          if (BWD) ly += there ? static_cast<size_t>(a.T) * D : 0;
        }
        if (++lbuf == kAhead + 1) lbuf = 0;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int n = 0; n < kAhead; ++n) load(n < total);
    unsigned i = first;
    int r = 0, h = 0, buf = 0;
    T* out = nullptr;
    bool live = false;
    float cs[N], sn[N];
    int next_fold = kFold;
    for (int n = 0; n < total; ++n) {
      load(n + kAhead < total);
      if (r == 0) {
        if (LONG && n >= next_fold) {
#pragma unroll
          for (int j = 0; j < 2 * N; ++j) {
            far[j * kThreads] = (folded ? far[j * kThreads] : 0.0) + static_cast<double>(dw[j]);
            dw[j] = 0.f;
          }
          folded = true;
          next_fold = n + kFold;
        }
        live = i + tid < s.items;
        const Item it = item_of<G>(live ? i + tid : c, a.T, s.groups, s.span);
        out = static_cast<T*>(s.y) + it.b * s.y_batch + it.g0 * s.y_head + it.t * s.y_token;
        h = it.g0;
        angles<D, N>(a, it, live && is_q && it.g0 == 0 && it.c == 0, th_hi, th_lo, cs, sn);
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
      const bool mine = live && h < s.H;
      auto fetch = [&](int piece, float* to) {
        Piece<T, N> p;
        *reinterpret_cast<uint4*>(p.w) = *reinterpret_cast<const uint4*>(
            s_stage + buf * kStage<BWD> + (piece * kThreads + tid) * 16);
        p.get(to);
      };
      bool keep = true;
      float y[2 * N];
      fetch(0, y);
      fetch(1, y + N);
      if constexpr (!BWD) {
        if (a.norm) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 2 * N; ++j) sum = fmaf(y[j], y[j], sum);
          float ms = fmaf(row_sum<G>(sum), 1.f / D, a.eps);
          if (__any_sync(0xffffffffu, out_of_range(ms))) rescale<D, N, G>(y, a.eps, ms);
          const float rs = rsqrtf(ms);
#pragma unroll
          for (int j = 0; j < 2 * N; ++j) y[j] *= rs * w[j];
        }
        turn<N>(y, a.rope, cs, sn, 1.f);
      } else {
        float g[2 * N];
        fetch(2, g);
        fetch(3, g + N);
        turn<N>(g, a.rope, cs, sn, -1.f);
        if (a.norm) {
          float sq = 0.f, dot = 0.f;
#pragma unroll
          for (int j = 0; j < 2 * N; ++j) {
            sq = fmaf(y[j], y[j], sq);
            dot = fmaf(g[j] * w[j], y[j], dot);
          }
          sq = row_sum<G>(sq);
          dot = row_sum<G>(dot);
          float ms = fmaf(sq, 1.f / D, a.eps), f = 1.f;
          const bool odd = mine && out_of_range(ms);
          if constexpr (kAgain) {
            f = rescale<D, N, G>(y, a.eps, ms);
            dot = 0.f;
#pragma unroll
            for (int j = 0; j < 2 * N; ++j) dot = fmaf(g[j] * w[j], y[j], dot);
            dot = row_sum<G>(dot);
          }
          const bool now = mine && odd == kAgain;
          again |= odd;
          // (a lane without a row, or with one of the other sweep's, adds nothing: 0 * r must be 0)
          const float rs = now ? rsqrtf(ms) : 0.f;
          const float m = dot * rs * (1.f / D);
#pragma unroll
          for (int j = 0; j < 2 * N; ++j) {
            const float v = y[j] * rs;
            dw[j] = fmaf(g[j], v, dw[j]);
            y[j] = rs * fmaf(-v, m, g[j] * w[j]);
            if (kAgain) y[j] *= f;
          }
          keep = !kAgain || odd;
        } else {
#pragma unroll
          for (int j = 0; j < 2 * N; ++j) y[j] = g[j];
        }
      }
      if (mine) {
        if (keep) {
          Piece<T, N> p;
          p.put(y);
          p.store(out + e0);
          p.put(y + N);
          p.store(out + e1);
        }
        out += s.y_head;
      }
      ++h;
      if (++r == s.span) {
        r = 0;
        i += step;
      }
      if (++buf == kAhead + 1) buf = 0;
    }
  };
  sweep(std::false_type{});
  if constexpr (BWD) {
    if (__syncthreads_or(again)) sweep(std::true_type{});
  }
  if constexpr (BWD) {
    if (a.partial == nullptr) return;
#pragma unroll
    for (int j = 0; j < 2 * N; ++j) {
      if (LONG && folded) dw[j] = static_cast<float>(far[j * kThreads] + static_cast<double>(dw[j]));
#pragma unroll
      for (int o = G; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
      if (lane < G) s_dw[warp][j < N ? e0 + j : e1 + j - N] = dw[j];
    }
    __syncthreads();
    for (int j = tid; j < D; j += kThreads) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) sum += s_dw[v][j];
      a.partial[static_cast<size_t>(blockIdx.x) * D + j] = sum;
    }
  }
}

// dw of the queries' (blockIdx.y = 0) or the keys' gain: the blocks' sums in a fixed order, 16
// channels per block
constexpr int kSumChannels = 16, kSumParts = kSumThreads / kSumChannels;
template <int D>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const float* __restrict__ partial,
                                                          int q_blocks, int blocks,
                                                          float* __restrict__ dqw,
                                                          float* __restrict__ dkw) {
  __shared__ float s[kSumParts][kSumChannels];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool is_q = blockIdx.y == 0;
  float* out = is_q ? dqw : dkw;
  if (out == nullptr) return;
  const int at = threadIdx.x % kSumChannels, part = threadIdx.x / kSumChannels;
  const int ch = blockIdx.x * kSumChannels + at;
  const int first = is_q ? 0 : q_blocks, last = is_q ? q_blocks : blocks;
  float sum = 0.f;
#pragma unroll 8
  for (int i = first + part; i < last; i += kSumParts)
    sum += partial[static_cast<size_t>(i) * D + ch];
  s[part][at] = sum;
  __syncthreads();
  if (part != 0) return;
#pragma unroll
  for (int v = 1; v < kSumParts; ++v) sum += s[v][at];
  out[ch] = sum;
}

unsigned blocks_of(const QkNormSide& s) { return (s.items + kThreads - 1) / kThreads; }

// Heads per item and blocks of the two sides; returns the grid.  `all`: blocks that fill the GPU.
// Items are of as many heads (which share their angles) as still give each of `all` blocks two of
// them, or four in the backward pass (`once` false), whose blocks' shares differ by one, and no more
// than kFold there.
int share(QkNormArgs& a, bool bf16, long long all, bool once) {
  const long long threads = static_cast<long long>(a.B) * a.T * (a.d / (bf16 ? 16 : 8));
  int span = std::min(std::max(a.q.H, a.k.H), once ? 1 << 20 : kFold);
  while (span > 1 && threads * ((a.q.H + span - 1) / span + (a.k.H + span - 1) / span) <
                         (once ? 2 : 4) * all * kThreads)
    span = (span + 1) / 2;
  for (QkNormSide* s : {&a.q, &a.k}) {
    s->span = std::min(span, s->H);
    s->groups = (s->H + s->span - 1) / s->span;
    s->items = static_cast<unsigned>(threads * s->groups);
  }
  const long long bq = blocks_of(a.q), bk = blocks_of(a.k);
  const long long rounds = once ? 1 : (bq + bk + all - 1) / all;
  a.q_blocks = static_cast<int>((bq + rounds - 1) / rounds);
  return a.q_blocks + static_cast<int>((bk + rounds - 1) / rounds);
}

template <typename T, int D, bool BWD, bool LONG>
cudaError_t launch_t(const QkNormArgs& a, int grid, float* dqw, float* dkw, cudaStream_t stream) {
  static SmemLimitOnce smem_limit;
  constexpr int kBytes = kShared<T, BWD, LONG>;
  cudaError_t e = smem_limit.set(qk_norm_kernel<T, D, BWD, LONG>, kBytes);
  if (e != cudaSuccess) return e;
  e = launch_behind(qk_norm_kernel<T, D, BWD, LONG>, dim3(static_cast<unsigned>(grid)), kThreads,
                    size_t{kBytes}, stream, a);
  if constexpr (BWD) {
    if (e == cudaSuccess && a.partial != nullptr)
      e = launch_behind(sum_kernel<D>, dim3(D / kSumChannels, 2), kSumThreads, stream,
                        static_cast<const float*>(a.partial), a.q_blocks, grid, dqw, dkw);
  }
  return e;
}
template <typename T, bool BWD, bool LONG>
cudaError_t launch_d(const QkNormArgs& a, int grid, float* dqw, float* dkw, cudaStream_t stream) {
  if (a.d == 128) return launch_t<T, 128, BWD, LONG>(a, grid, dqw, dkw, stream);
  if (a.d == 64) return launch_t<T, 64, BWD, LONG>(a, grid, dqw, dkw, stream);
  if constexpr (sizeof(T) == 4) {
    if (a.d == 32) return launch_t<T, 32, BWD, LONG>(a, grid, dqw, dkw, stream);
    return launch_t<T, 16, BWD, LONG>(a, grid, dqw, dkw, stream);
  }
  return cudaErrorInvalidValue;
}
template <bool BWD, bool LONG>
cudaError_t launch_type(const QkNormArgs& a, bool bf16, int grid, float* dqw, float* dkw,
                        cudaStream_t stream) {
  return bf16 ? launch_d<__nv_bfloat16, BWD, LONG>(a, grid, dqw, dkw, stream)
              : launch_d<float, BWD, LONG>(a, grid, dqw, dkw, stream);
}

// rows of a side's threads, at most
long long most_rows(const QkNormSide& s, int blocks) {
  return (blocks_of(s) + blocks - 1LL) / blocks * s.span;
}

}  // namespace

cudaError_t launch_qk_norm(QkNormArgs a, bool bf16, cudaStream_t stream) {
  const int grid = share(a, bf16, 6 * kSms, true);
  return launch_type<false, false>(a, bf16, grid, nullptr, nullptr, stream);
}

cudaError_t launch_qk_norm_bwd(QkNormArgs a, bool bf16, float* dqw, float* dkw,
                               cudaStream_t stream) {
  const int grid = share(a, bf16, qk_norm_bwd_blocks(), false);
  const bool many = a.partial != nullptr && std::max(most_rows(a.q, a.q_blocks),
                                                     most_rows(a.k, grid - a.q_blocks)) > kMany;
  return many ? launch_type<true, true>(a, bf16, grid, dqw, dkw, stream)
              : launch_type<true, false>(a, bf16, grid, dqw, dkw, stream);
}

}  // namespace csattn
