// Block tables, slots and positions of a step's new tokens, from the requests' lengths.
//
// Request b holds held[b] rows in ceil(held / page_size) pages and gets new[b] tokens; the tokens
// of all requests, one request after the other, are the step's.  Two prefix sums over the requests
// say everything: the tokens ahead of a request (where its own begin) and the pages ahead of it
// (which of the free list it takes).  A page taken begins with a new token, so the thread of a
// page's first row writes the page down, and each token finds its page by itself.
//
// A CTA has a range of kTokens tokens.  It sums requests up, kThreads at a time, until it is past
// its tokens; those of the current kThreads requests find theirs by bisection in shared memory.
// The first CTA goes through all of them and writes what there is one of per request.  That every
// CTA adds up the lengths of those before it again costs less than a second launch: they are
// a few KB in L2.  64 requests of one token take 2.4 us, 512 with 65536 tokens 5.5 us (0.85 MB):
// a launch, the lengths, the sums, the table and the slot one after another.
#include "internal.h"

namespace csattn {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 1024;  // per CTA

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

__global__ void __launch_bounds__(kThreads)
    page_tables_kernel(const __grid_constant__ PageTablesArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ long long s_tok[kWarps], s_page[kWarps];
  __shared__ int s_end[kThreads], s_begin[kThreads], s_held[kThreads], s_nth[kThreads];
  __shared__ int s_taken;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const bool first = blockIdx.x == 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t0 = static_cast<int>(blockIdx.x) * kTokens;
  const int t1 = static_cast<int>(min(static_cast<long long>(a.N), t0 + 1LL * kTokens));
  const int ps = a.page_size;
  const int rows = a.max_pages * ps;  // (< 2^30)
  int num_free = *a.num_free;
  bool wrong = num_free < 0 || num_free > a.free_size;
  num_free = min(max(num_free, 0), a.free_size);
  if (tid == 0) s_taken = 0;
  long long tok_base = 0, page_base = 0;  // of the requests before the current ones
  int taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int held = 0, fresh = 0, want = 0;
    bool ok = true;
    if (b < a.B) {
      held = a.held[b];
      fresh = a.fresh[b];
      ok = held >= 0 && fresh >= 0 && held <= rows && fresh <= rows - held;
      if (ok) want = (held + fresh + ps - 1) / ps - (held + ps - 1) / ps;
      fresh = max(fresh, 0);
    }
    const long long tok_in = warp_scan(fresh, lane), page_in = warp_scan(want, lane);
    __syncthreads();  // (the last round's shared values are read)
    if (lane == 31) {
      s_tok[warp] = tok_in;
      s_page[warp] = page_in;
    }
    __syncthreads();
    long long tok_end = tok_base + tok_in, page_end = page_base + page_in;
    long long tok_sum = 0, page_sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        tok_end += s_tok[w];
        page_end += s_page[w];
      }
      tok_sum += s_tok[w];
      page_sum += s_page[w];
    }
    wrong |= !ok;
    // (no room in the step, or not enough pages; one that has no tokens needs neither)
    if (fresh > 0 && tok_end > a.N) ok = false;
    if (want > 0 && page_end > num_free) ok = false;
    if (ok && want > 0) taken = static_cast<int>(page_end);
    const int end = static_cast<int>(min(tok_end, static_cast<long long>(a.N)));
    const int begin = static_cast<int>(min(tok_end - fresh, static_cast<long long>(a.N)));
    s_end[tid] = end;
    s_begin[tid] = begin;
    s_held[tid] = ok ? held : -1;
    s_nth[tid] = static_cast<int>(min(page_end - want, 0x7fffffffLL));
    if (first && b < a.B) {
      wrong |= !ok;
      a.seq_lens[b] = ok ? held + fresh : (held >= 0 && held <= rows ? held : 0);
      a.starts[b + 1] = end;
      if (b == 0) a.starts[0] = 0;
    }
    __syncthreads();
    // the CTA's tokens among these requests'
    // (tok_base may be past 32 bits)
    const int lo = static_cast<int>(
        min(max(static_cast<long long>(t0), tok_base), static_cast<long long>(t1)));
    const int hi = static_cast<int>(min(static_cast<long long>(t1), tok_base + tok_sum));
    for (int t = lo + tid; t < hi; t += kThreads) {
      int r = 0;  // the first request that ends behind t
#pragma unroll
      for (int step = kThreads / 2; step > 0; step >>= 1)
        if (s_end[r + step - 1] <= t) r += step;
      const int had = s_held[r];
      long long slot = -1;
      int pos = 0;
      if (had >= 0) {
        const int row = had + (t - s_begin[r]);
        const int at = row / ps, off = row - at * ps, have = (had + ps - 1) / ps;
        int32_t* entry = a.block_table + static_cast<size_t>(b0 + r) * a.max_pages + at;
        const bool take = at >= have;
        const int page = take ? a.free_pages[num_free - 1 - (s_nth[r] + at - have)] : *entry;
        if (page >= 0 && page < a.num_pages) {
          slot = static_cast<long long>(page) * ps + off;
          if (take && off == 0) *entry = page;
        } else {
          wrong = true;
        }
        pos = row;
      }
      a.slots[t] = slot;
      a.positions[t] = pos;
    }
    tok_base += tok_sum;
    page_base += page_sum;
    if (!first && tok_base >= t1) break;
  }
  // tokens behind the last request's
  const long long from = max(tok_base, static_cast<long long>(t0));
  const int behind = static_cast<int>(min(from, static_cast<long long>(t1)));
  for (int t = behind + tid; t < t1; t += kThreads) {
    a.slots[t] = -1;
    a.positions[t] = 0;
  }
  if (wrong) atomicOr(a.status, kStatusDeviceArg);
  if (first) {
    // (the requests that take pages are the first that want some: the last one's sum is the largest)
    __syncthreads();
    atomicMax(&s_taken, taken);
    __syncthreads();
    if (tid == 0) *a.free_left = num_free - s_taken;
  }
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream) {
  const unsigned grid = (static_cast<unsigned>(a.N) + kTokens - 1) / kTokens;
  return launch_behind(page_tables_kernel, dim3(grid > 0 ? grid : 1), kThreads, stream, a);
}

}  // namespace csattn
