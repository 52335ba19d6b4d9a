// Whether two strided tensors have a place in common (host code).
#pragma once

#include <algorithm>
#include <cstdint>

namespace csattn {

// Where a tensor's elements are: rows of contiguous bytes, up to three strides apart.
struct Places {
  struct Step {
    long long stride, lo, hi;  // times lo..hi
  };
  long long at = 0, row = 0, end = 0;
  Step steps[3];
  int count = 0;

  Places() = default;
  Places(const void* p, long long bytes)
      : at(reinterpret_cast<intptr_t>(p)), row(p != nullptr ? bytes : 0), end(at + row) {}
  // [B, H, T, d] of elements of `size` bytes
  Places(const void* p, int B, int H, int T, int d, int size, long long batch, long long head,
         long long token)
      : Places(p, 1LL * d * size) {
    for (const Step& x : {Step{batch * size, 0, B - 1LL}, Step{head * size, 0, H - 1LL},
                          Step{token * size, 0, T - 1LL}})
      if (x.hi > 0 && x.stride > 0) steps[count++] = x;
    std::sort(steps, steps + count, [](const Step& a, const Step& b) { return a.stride < b.stride; });
    while (count > 0 && steps[0].stride == row) {  // dense
      row *= steps[0].hi + 1;
      std::copy(steps + 1, steps + count--, steps);
    }
    end = at + row;
    for (int i = 0; i < count; ++i) {
      // (past what an address reaches: not a tensor)
      long long reach = 0;
      if (__builtin_mul_overflow(steps[i].stride, steps[i].hi, &reach) || reach >= 1LL << 60)
        reach = 1LL << 60;
      end += reach;
    }
  }
};

// Whether lo < start + (a multiple of each of n strides) < hi is possible; the strides descend.
// Strides of one buffer's parts nest, so that few multiples are looked at; `budget` of them are.
inline bool reaches(long long start, const Places::Step* x, int n, long long lo, long long hi,
                    int* budget) {
  if (n == 0) return lo < start && start < hi;
  long long least = 0, most = 0;  // of the smaller strides
  for (int i = 1; i < n; ++i) {
    least += x[i].stride * x[i].lo;
    most += x[i].stride * x[i].hi;
  }
  // lo - start - most < stride * i < hi - start - least
  const auto floor_div = [](long long a, long long b) { return a / b - (a % b < 0 ? 1 : 0); };
  const long long first = std::max(x->lo, floor_div(lo - start - most, x->stride) + 1);
  const long long last = std::min(x->hi, -floor_div(start + least - hi, x->stride) - 1);
  for (long long i = first; i <= last && --*budget > 0; ++i)
    if (reaches(start + x->stride * i, x + 1, n - 1, lo, hi, budget)) return true;
  return false;
}

inline bool share_a_place(const Places& a, const Places& b) {
  if (a.row == 0 || b.row == 0 || a.end <= b.at || b.end <= a.at) return false;
  if (std::max(a.end - a.at, b.end - b.at) >= 1LL << 59) return false;
  // the differences of two rows' addresses
  Places::Step x[6];
  int n = 0;
  for (int i = 0; i < a.count; ++i) x[n++] = a.steps[i];
  for (int i = 0; i < b.count; ++i) {
    Places::Step* same = std::find_if(
        x, x + n, [&](const Places::Step& s) { return s.stride == b.steps[i].stride; });
    if (same == x + n) x[n++] = {b.steps[i].stride, 0, 0};
    same->lo -= b.steps[i].hi;
  }
  std::sort(x, x + n, [](const Places::Step& p, const Places::Step& q) {
    return p.stride > q.stride;
  });
  int budget = 1000;
  return reaches(a.at - b.at, x, n, -a.row, b.row, &budget);
}

}  // namespace csattn
