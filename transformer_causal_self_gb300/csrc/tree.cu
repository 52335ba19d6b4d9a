// A tree of drafted tokens over a KV cache: what a step does ahead of its attention, and the
// move of the accepted path afterwards.
//
// Draft t of sequence b (length L) has a parent p[t] < t among the drafts, -1 (its parent is
// the sequence's last token) or -2 (no token: padding).  Its depth is the number of drafts
// above it, its position L + depth, its cache row L + t.  With the position in the key, the
// rows of an accepted path need only be moved to L, L + 1, ... once the tree is verified.
#include <algorithm>

#include "fp8.cuh"
#include "internal.h"

namespace csattn {
namespace {

constexpr int kThreads = 256;  // >= the largest Tn
constexpr int kWords = kThreads / 32;
constexpr int kDrafts = 4;  // drafts of a CTA, where it has several
constexpr int kStride = kWords + 1;  // of a draft's mask words (odd: neighbours' in other banks)

// Ancestor masks (self included; zero for padding) of a sequence's drafts into s_anc and
// whether every parent is valid, by pointer doubling: after round r a token's mask holds
// its 2^r nearest, and its pointer the next one above.  All kThreads threads call it.
__device__ __forceinline__ bool tree_masks(const int32_t* parents, int Tn, int words,
                                           uint32_t (*s_anc)[kStride], int* s_up) {
  const int t = static_cast<int>(threadIdx.x);
  int up = t < Tn ? parents[t] : -2;
  bool bad = t < Tn && (up < -2 || up >= t);
  s_up[t] = up;
  __syncthreads();
  if (!bad && up >= 0) bad = s_up[up] == -2;  // below padding
  if (__syncthreads_or(bad)) return false;
#pragma unroll
  for (int w = 0; w < kWords; ++w)
    if (w < words) s_anc[t][w] = (up != -2 && (t >> 5) == w) ? 1u << (t & 31) : 0u;
  while (__syncthreads_or(up >= 0)) {
    uint32_t more[kWords];
    int next = -1;
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) more[w] = w < words ? s_anc[up][w] : 0u;
      next = s_up[up];
    }
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        if (w < words) s_anc[t][w] |= more[w];
      s_up[t] = next;
      up = next;
    }
  }
  return true;
}

// One CTA per draft of a sequence; several where few drafts leave SMs idle, and up to N drafts per
// CTA where there are many.  Every CTA works out the sequence's masks (a few rounds in shared
// memory), then its drafts' rows, 16 channels per thread: keys rotated at their positions and
// values to the cache (bf16 or e4m3), queries rotated into q_rot.  Bound by launch and memory
// latency for a few hundred drafts (3.1 us for 8 of one sequence, about 6 for 512; 128 channels,
// 48 heads), by the queries' bytes, in and out, for thousands.
template <int D, bool F8, int N>
__global__ void __launch_bounds__(kThreads) tree_prep_kernel(
    const __nv_bfloat16* __restrict__ q_new, const __nv_bfloat16* __restrict__ k_new,
    const __nv_bfloat16* __restrict__ v_new, void* __restrict__ k_cache,
    void* __restrict__ v_cache, uint8_t* __restrict__ k_scale, uint8_t* __restrict__ v_scale,
    const int32_t* __restrict__ cache_lens, const int32_t* __restrict__ parents, CacheRows rows,
    int Hq, int Tn, int max_seq_len, int rope, RopeTable theta, __nv_bfloat16* __restrict__ q_rot,
    float* __restrict__ q_factor, uint32_t* __restrict__ anc, int32_t* __restrict__ lens,
    uint8_t* __restrict__ vflag, int words, int drafts, uint32_t* status) {
  constexpr int G = D / 16;
  __shared__ uint32_t s_anc[kThreads][kStride];
  __shared__ int s_up[kThreads];
  __shared__ float s_cos[N][64], s_sin[N][64];
  if (N == 1) drafts = 1;
  const int t0 = blockIdx.x * drafts, b = blockIdx.y, tid = threadIdx.x, Hkv = rows.Hkv;
  const int rep = Hq / Hkv, items = (Hq + 2 * Hkv) * G, step = gridDim.z * kThreads;
  const int all = min(drafts, Tn - t0) * items;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the attention kernel may be scheduled; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int L = cache_lens[b];
  const bool fits = L >= 0 && L <= max_seq_len - Tn;
  // 16 channels of a row and, for a key or value, its cache row of KV head 0: each thread's first
  // while the masks are worked out, the next ones beside the arithmetic on the last
  auto load = [&](int i, uint4* lo, uint4* hi, long long* row0) {
    *lo = *hi = make_uint4(0u, 0u, 0u, 0u);
    *row0 = -1;
    if (i >= all) return;
    const int k = N == 1 ? 0 : i / items, t = t0 + k, j = i - k * items, head = j / G;
    const bool is_q = head < Hq, is_v = head >= Hq + Hkv;
    int e0, e1;
    rope_piece(is_v ? 0 : rope, D / 2, j % G, &e0, &e1);
    const int g = is_q ? head : head - Hq - (is_v ? Hkv : 0);
    const __nv_bfloat16* x = (is_q ? q_new : (is_v ? v_new : k_new)) +
                             ((static_cast<size_t>(b) * (is_q ? Hq : Hkv) + g) * Tn + t) * D;
    *lo = *reinterpret_cast<const uint4*>(x + e0);
    *hi = *reinterpret_cast<const uint4*>(x + e1);
    if (!is_q && fits) *row0 = rows.at(b, 0, L + t);
  };
  uint4 lo, hi;
  long long row0;
  load(blockIdx.z * kThreads + tid, &lo, &hi, &row0);
  const bool fine =
      tree_masks(parents + static_cast<size_t>(b) * Tn, Tn, words, s_anc, s_up) && fits;
  if (tid == 0 && t0 == 0 && blockIdx.z == 0) {
    lens[b] = fine ? L : -1;
    if (!fine) atomicOr(status, kStatusDeviceArg);
  }
  if (!fine) return;  // the sequence's cache is left as it was
  __syncthreads();
  if (blockIdx.z == 0 && tid < min(drafts, Tn - t0) * words)
    anc[(static_cast<size_t>(b) * Tn + t0) * words + tid] = s_anc[t0 + tid / words][tid % words];
  if (rope != 0) {
    for (int i = tid; i < min(drafts, Tn - t0) * (D / 2); i += kThreads) {
      const int k = i / (D / 2), c = i % (D / 2);
      int depth = -1;
      for (int w = 0; w < words; ++w) depth += __popc(s_anc[t0 + k][w]);
      // (padding is written like a first token, never seen)
      const int pos = L + max(depth, 0);
      // (a bf16 cache's rows are those of the other appends to it)
      if constexpr (F8)
        angle_cos_sin(pos, theta.hi[c], theta.lo[c], s_cos[k][c], s_sin[k][c]);
      else
        rope_cos_sin<false>(pos, theta.hi[c], theta.lo[c], s_cos[k][c], s_sin[k][c]);
    }
  }
  __syncthreads();
  // (whole warps take part in the shuffles)
  for (int i0 = blockIdx.z * kThreads; i0 < all; i0 += step) {
    const int i = i0 + tid;
    const bool live = i < all;
    const int k = N == 1 || !live ? 0 : i / items, t = t0 + k, j = live ? i - k * items : 0;
    const int head = j / G, c = i % G;
    const bool is_q = head < Hq, is_v = head >= Hq + Hkv;
    const int g = is_q ? head : head - Hq - (is_v ? Hkv : 0);
    const int layout = is_v ? 0 : rope;
    int e0, e1;
    rope_piece(layout, D / 2, c, &e0, &e1);
    uint4 next_lo, next_hi;
    long long next_row0;
    if (N > 1) load(i + step, &next_lo, &next_hi, &next_row0);
    if (N == 1 && i0 >= step) load(i, &lo, &hi, &row0);
    bool bad;
    const uint32_t top = row_absmax<G>(lo, hi, &bad);
    auto write = [&]() {
      float cs[8], sn[8], y[16];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        cs[n] = layout != 0 ? s_cos[k][8 * c + n] : 1.f;
        sn[n] = layout != 0 ? s_sin[k][8 * c + n] : 0.f;
      }
      const int code = scale_code(top, layout != 0);
      if (F8 && !is_q) {
        lo = scale_row(lo, code);
        hi = scale_row(hi, code);
      }
      rope16(lo, hi, layout, cs, sn, y);
      // (bf16: rounded to the cache's type, queries too: the products take both sides in one type)
      if (layout != 0) {
        lo = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                        pack_bf16x2(y[6], y[7]));
        hi = make_uint4(pack_bf16x2(y[8], y[9]), pack_bf16x2(y[10], y[11]),
                        pack_bf16x2(y[12], y[13]), pack_bf16x2(y[14], y[15]));
      }
      if (is_q) {
        // the rows of a KV head's queries one behind another, draft by draft
        const int kvh = g / rep;
        const size_t q_row =
            (static_cast<size_t>(b) * Hkv + kvh) * Tn * rep + t * rep + g - kvh * rep;
        if constexpr (F8) {  // (query_to_f16 with the angles at hand)
          const int E = min(max(static_cast<int>(top >> 7), 15), 254);
          const float f = __uint_as_float(static_cast<uint32_t>(268 - E) << 23);
          lo = make_uint4(pack_f16x2(y[0] * f, y[1] * f), pack_f16x2(y[2] * f, y[3] * f),
                          pack_f16x2(y[4] * f, y[5] * f), pack_f16x2(y[6] * f, y[7] * f));
          hi = make_uint4(pack_f16x2(y[8] * f, y[9] * f), pack_f16x2(y[10] * f, y[11] * f),
                          pack_f16x2(y[12] * f, y[13] * f), pack_f16x2(y[14] * f, y[15] * f));
          if (c == 0)
            q_factor[q_row] = __uint_as_float(static_cast<uint32_t>(E - 14) << 23);
        }
        __nv_bfloat16* dst = q_rot + q_row * D;
        *reinterpret_cast<uint4*>(dst + e0) = lo;
        *reinterpret_cast<uint4*>(dst + e1) = hi;
        return;
      }
      // (a row on a page outside the pool reads as zeros)
      if (is_v && c == 0)
        vflag[(static_cast<size_t>(b) * Hkv + g) * Tn + t] = bad && row0 >= 0 ? 1 : 0;
      if (row0 < 0) {
        if (c == 0) atomicOr(status, kStatusDeviceArg);
        return;
      }
      const int plane = rows.block_table != nullptr ? rows.page_size : rows.Lmax;  // rows of a head
      const long long row = row0 + static_cast<long long>(g) * plane;
      if constexpr (F8) {
        uint8_t* dst = static_cast<uint8_t*>(is_v ? v_cache : k_cache) + row * D;
        *reinterpret_cast<uint2*>(dst + e0) =
            make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3], code, bad),
                       pack_e4m3x4(y[4], y[5], y[6], y[7], code, bad));
        *reinterpret_cast<uint2*>(dst + e1) =
            make_uint2(pack_e4m3x4(y[8], y[9], y[10], y[11], code, bad),
                       pack_e4m3x4(y[12], y[13], y[14], y[15], code, bad));
        if (c == 0) (is_v ? v_scale : k_scale)[row] = static_cast<uint8_t>(code);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? v_cache : k_cache) + row * D;
        *reinterpret_cast<uint4*>(dst + e0) = lo;
        *reinterpret_cast<uint4*>(dst + e1) = hi;
      }
    };
    if (live) write();  // (no shuffle in it)
    if (N > 1) {
      lo = next_lo;
      hi = next_hi;
      row0 = next_row0;
    }
  }
}

// The path of accepted[b] (its ancestors and itself, a_0 < a_1 < ...): row L + i receives row
// L + a_i.  A CTA moves some KV heads of one sequence, kMoveRows rows at a time: all of their
// 16-byte pieces are read, then, behind a barrier, written.  a_i >= i, so what a group of rows
// overwrites has been read by it or by an earlier one.  Bound by latency (a walk up the tree,
// the block table, the rows): a few KB per sequence, 1.9 us for one, 4.0 for 256.
constexpr int kMoveRows = 8;
constexpr int kMoveBatch = 4;  // pieces per thread in flight

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(
    uint4* k_cache, uint4* v_cache, uint8_t* k_scale, uint8_t* v_scale,
    const int32_t* __restrict__ cache_lens, const int32_t* __restrict__ parents,
    const int32_t* __restrict__ accepted, int32_t* __restrict__ new_lens, CacheRows rows, int Tn,
    int pieces, int heads, uint32_t* status) {
  __shared__ int s_up[kThreads];
  __shared__ uint8_t s_path[kThreads];                   // the path, at its end
  __shared__ long long s_from[kThreads], s_to[kThreads];  // of row i, in rows, KV head 0
  __shared__ int s_n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g0 = blockIdx.x * heads, b = blockIdx.y, tid = threadIdx.x;
  const int nh = min(heads, rows.Hkv - g0);
  const int L = cache_lens[b], last = accepted[b];
  if (tid < Tn) s_up[tid] = parents[static_cast<size_t>(b) * Tn + tid];
  __syncthreads();
  if (tid == 0) {
    // a walk leaves the tree after at most Tn steps because each must go down in number
    int n = 0, t = last;
    bool bad = L < 0 || L > rows.Lmax - Tn || last < -1 || last >= Tn;
    while (!bad && t >= 0) {
      const int up = s_up[t];
      s_path[kThreads - ++n] = static_cast<uint8_t>(t);
      bad = up >= t || up < -1;
      t = up;
    }
    s_n = bad ? -1 : n;
  }
  __syncthreads();
  const int n = s_n;
  bool bad = n < 0;
  if (tid < n) {
    s_from[tid] = rows.at(b, 0, L + s_path[kThreads - n + tid]);
    s_to[tid] = rows.at(b, 0, L + tid);
    bad = s_from[tid] < 0 || s_to[tid] < 0;  // a page outside the pool: nothing is moved
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && g0 == 0) {
    new_lens[b] = bad ? L : L + n;
    if (bad) atomicOr(status, kStatusDeviceArg);
  }
  if (bad) return;
  const long long stride = rows.block_table == nullptr ? rows.Lmax : rows.page_size;  // of heads
  // tasks of a group of rows: (row, head, keys or values, piece), and the scale bytes
  const int per_head = 2 * pieces, per_row = nh * per_head;
  for (int i0 = 0; i0 < n; i0 += kMoveRows) {
    const int group = min(kMoveRows, n - i0);
    if (k_scale != nullptr) {
      const int e = tid, i = i0 + e / (2 * nh), gv = e % (2 * nh);
      // (2 * nh * kMoveRows scale bytes of a group: the launcher keeps them within the CTA)
      uint8_t x = 0;
      uint8_t* base = gv & 1 ? v_scale : k_scale;
      const bool mine = e < group * 2 * nh && s_from[i] != s_to[i];
      if (mine) x = base[s_from[i] + (g0 + gv / 2) * stride];
      __syncthreads();
      if (mine) base[s_to[i] + (g0 + gv / 2) * stride] = x;
    }
    for (int c0 = 0; c0 < per_row; c0 += kThreads * kMoveBatch / kMoveRows) {
      // columns c0.. of the group's rows; a barrier between their loads and their stores
      const int width = min(per_row - c0, kThreads * kMoveBatch / kMoveRows);
      uint4 x[kMoveBatch];
#pragma unroll
      for (int u = 0; u < kMoveBatch; ++u) {
        const int e = u * kThreads + tid, i = i0 + e / width, c = c0 + e % width;
        if (e >= group * width || s_from[i] == s_to[i]) continue;
        const int h = c / per_head, q = c - h * per_head;
        x[u] = (q < pieces ? k_cache : v_cache)[(s_from[i] + (g0 + h) * stride) * pieces +
                                                (q < pieces ? q : q - pieces)];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveBatch; ++u) {
        const int e = u * kThreads + tid, i = i0 + e / width, c = c0 + e % width;
        if (e >= group * width || s_from[i] == s_to[i]) continue;
        const int h = c / per_head, q = c - h * per_head;
        (q < pieces ? k_cache : v_cache)[(s_to[i] + (g0 + h) * stride) * pieces +
                                         (q < pieces ? q : q - pieces)] = x[u];
      }
    }
    __syncthreads();  // (the next group may read what this one has written only in order)
  }
}

CacheRows rows_of(const KvCache& c, int Hkv) {
  return CacheRows{c.block_table, Hkv, c.Lmax, c.page_size, c.num_pages, c.max_pages};
}

}  // namespace

cudaError_t launch_tree_prep(const TreePrepArgs& a, cudaStream_t stream) {
  const bool f8 = a.cache.k_scale != nullptr;
  // a draft's rows shared by several CTAs while these are all resident at once
  const int parts = ((a.Hq + 2 * a.Hkv) * (a.d / 16) + kThreads - 1) / kThreads;
  const bool few = static_cast<long long>(a.Tn) * a.B * parts <= 2 * kSms && parts <= 65535;
  // several drafts in a CTA where there are more than are resident at once: the masks are worked
  // out once for them (64 sequences of 500 rows, 64 drafts: 125 and 137 us for the whole step over
  // bf16 and e4m3, 8 and 13 more with one draft each; 512 drafts: 2 us less with one each)
  const int drafts = static_cast<int>(
      std::min<long long>(kDrafts, (static_cast<long long>(a.Tn) * a.B + 4 * kSms - 1) / (4 * kSms)));
  auto* kernel = a.d == 128
                     ? (f8 ? tree_prep_kernel<128, true, 1> : tree_prep_kernel<128, false, 1>)
                     : (f8 ? tree_prep_kernel<64, true, 1> : tree_prep_kernel<64, false, 1>);
  if (drafts > 1)
    kernel = a.d == 128 ? (f8 ? tree_prep_kernel<128, true, kDrafts>
                              : tree_prep_kernel<128, false, kDrafts>)
                        : (f8 ? tree_prep_kernel<64, true, kDrafts>
                              : tree_prep_kernel<64, false, kDrafts>);
  return launch_behind(kernel, dim3((a.Tn + drafts - 1) / drafts, a.B, few ? parts : 1), kThreads,
                       stream,
                       static_cast<const __nv_bfloat16*>(a.q_new),
                       static_cast<const __nv_bfloat16*>(a.k_new),
                       static_cast<const __nv_bfloat16*>(a.v_new), a.cache.k, a.cache.v,
                       static_cast<uint8_t*>(a.cache.k_scale),
                       static_cast<uint8_t*>(a.cache.v_scale), a.cache_lens, a.parents,
                       rows_of(a.cache, a.Hkv), a.Hq, a.Tn, a.max_seq_len, a.rope, a.theta,
                       static_cast<__nv_bfloat16*>(a.q_rot), a.q_factor, a.anc, a.lens, a.vflag,
                       a.words, drafts, a.status);
}

cudaError_t launch_tree_commit(const KvCache& cache, const int32_t* cache_lens,
                               const int32_t* parents, const int32_t* accepted, int32_t* new_lens,
                               int B, int Hkv, int Tn, int d, uint32_t* status,
                               cudaStream_t stream) {
  const int pieces = d * (cache.k_scale != nullptr ? 1 : 2) / 16;
  // heads per CTA: few while that leaves SMs idle, at most 16 (their scale bytes fill a CTA)
  const int heads = std::max(1, std::min({16, Hkv, static_cast<int>(
                                                       static_cast<long long>(Hkv) * B / kSms)}));
  return launch_behind(tree_commit_kernel, dim3((Hkv + heads - 1) / heads, B), kThreads, stream,
                       static_cast<uint4*>(cache.k), static_cast<uint4*>(cache.v),
                       static_cast<uint8_t*>(cache.k_scale), static_cast<uint8_t*>(cache.v_scale),
                       cache_lens, parents, accepted, new_lens, rows_of(cache, Hkv), Tn, pieces,
                       heads, status);
}

}  // namespace csattn
