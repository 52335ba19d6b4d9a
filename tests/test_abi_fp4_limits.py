"""Refusals of overlapping tensors by the norm calls.  No GPU: every call here fails before any CUDA
call."""
import ctypes
import subprocess

import pytest

BASE = 1 << 30  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import transformer_causal_self_gb300 as csattn
    return csattn.load_library()


BRUTE = r"""
#include <cstdio>
#include <random>
#include <set>
#include <vector>
#include "places.h"
struct T { long long at; int n[3]; long long s[3]; int d; };
static void bytes(const T& t, std::set<long long>* out) {
  for (int b = 0; b < t.n[0]; ++b)
    for (int h = 0; h < t.n[1]; ++h)
      for (int i = 0; i < t.n[2]; ++i)
        for (int c = 0; c < 4 * t.d; ++c)
          out->insert(t.at + 4 * (b * t.s[0] + h * t.s[1] + i * t.s[2]) + c);
}
int main() {
  std::mt19937 rng(1);
  auto below = [&](int n) { return static_cast<int>(rng() % n); };
  int wrong = 0, apart = 0, together = 0;
  for (int round = 0; round < 40000; ++round) {
    T t[2];
    const int rows = 1 + below(6), T2 = 1 + below(4), B = 1 + below(3);
    for (T& x : t) {
      x.d = 4;
      x.n[0] = 1 + below(3), x.n[1] = 1 + below(4), x.n[2] = 1 + below(4);
      switch (below(4)) {
        case 0:  // parts of one projection's rows [B, T, rows, d]
          x.n[0] = B, x.n[2] = T2, x.n[1] = 1 + below(rows);
          x.s[0] = 4 * rows * T2, x.s[1] = 4, x.s[2] = 4 * rows;
          x.at = 4096 + 16 * below(rows - x.n[1] + 1);
          break;
        case 1:  // dense
          x.s[2] = 4, x.s[1] = 4 * x.n[2], x.s[0] = x.s[1] * x.n[1];
          x.at = 4096 + 16 * below(60) - 16 * below(2) * x.n[0] * x.n[1] * x.n[2];
          break;
        case 2:  // broadcast, and gaps
          x.s[2] = 4 * below(3), x.s[1] = 4 * below(20), x.s[0] = 4 * below(60);
          x.at = 4096 + 16 * below(90) - 16 * below(90);
          break;
        default:  // anything
          x.d = 4 * (1 + below(3));
          for (long long& s : x.s) s = 4 * below(30);
          x.at = 4096 + 4 * below(300) - 4 * below(300);
      }
    }
    std::set<long long> a, b;
    bytes(t[0], &a);
    bytes(t[1], &b);
    bool truth = false;
    for (long long v : a) truth = truth || b.count(v) != 0;
    csattn::Places p[2];
    for (int i = 0; i < 2; ++i)
      p[i] = csattn::Places(reinterpret_cast<void*>(t[i].at), t[i].n[0], t[i].n[1], t[i].n[2],
                            t[i].d, 4, t[i].s[0], t[i].s[1], t[i].s[2]);
    wrong += csattn::share_a_place(p[0], p[1]) != truth;
    wrong += csattn::share_a_place(p[1], p[0]) != truth;
    (truth ? together : apart) += 1;
  }
  std::printf("%d %d %d\n", wrong, apart, together);
}
"""


def test_places_against_all_bytes(tmp_path):
    """share_a_place against the sets of all bytes, over small tensors of every kind."""
    from transformer_causal_self_gb300 import build
    src, exe = tmp_path / "places.cpp", tmp_path / "places"
    src.write_text(BRUTE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    wrong, apart, together = map(int, subprocess.run(
        [str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert wrong == 0 and apart > 5000 and together > 5000


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


B, Hq, Hkv, T, D = 2, 4, 2, 5, 64
Q, K = 2 * B * Hq * T * D, 2 * B * Hkv * T * D  # bytes of dense bf16 tensors
ROWS = (Hq + 2 * Hkv) * D  # a fused projection's
FUSED = (ROWS * T, D, ROWS) * 2
STEP = 1 << 22  # between tensors that are apart


def forward(lib, strides=None, **kw):
    names = ("q", "k", "qw", "kw", "pos", "qo", "ko")
    at = {n: BASE + i * STEP for i, n in enumerate(names)}
    at.update(kw)
    rc = lib.csattn_qk_norm_rope(*[at[n] for n in names], B, Hq, Hkv, T, D, 1,
                                 i64(*strides) if strides else None, 0, 1, 1e-6, 1e4, 0, None)
    return rc, lib.csattn_last_error()


def backward(lib, strides=None, **kw):
    names = ("dqo", "dko", "q", "k", "qw", "kw", "pos", "dq", "dk", "dqw", "dkw")
    at = {n: BASE + i * STEP for i, n in enumerate(names)}
    at["ws"] = BASE + 20 * STEP
    at.update(kw)
    rc = lib.csattn_qk_norm_rope_bwd(*[at[n] for n in names], B, Hq, Hkv, T, D, 1,
                                     i64(*strides) if strides else None, 0, 1, 1e-6, 1e4, 0,
                                     at["ws"], 1 << 20, None)
    return rc, lib.csattn_last_error()


@pytest.mark.parametrize("kw,strides,what", [
    (dict(qo=BASE), None, b"input"),                      # in place
    (dict(qo=BASE + Q - 16), None, b"input"),
    (dict(ko=BASE + STEP + 2 * STEP), None, b"input"),    # a gain
    (dict(ko=BASE + 4 * STEP + 4 * B * T - 8), None, b"input"),  # a position
    (dict(ko=BASE + 5 * STEP + Q - 16), None, b"outputs"),
    (dict(k=BASE + 2 * Hq * D, qo=BASE + 2 * ROWS - 16), FUSED, b"input"),
    (dict(k=BASE + 2 * Hq * D, ko=BASE - K + 16), FUSED, b"input")])
def test_forward_refuses_overlaps(lib, kw, strides, what):
    rc, error = forward(lib, strides, **kw)
    assert rc == -1 and b"qk_norm_rope" in error and what in error, (rc, error)


@pytest.mark.parametrize("kw,strides,what", [
    (dict(dq=BASE + 2 * STEP), None, b"input"), (dict(dk=BASE + STEP), None, b"input"),
    (dict(dq=BASE), None, b"input"), (dict(dk=BASE + 7 * STEP + Q - 16), None, b"outputs"),
    (dict(dqw=BASE + 4 * STEP), None, b"input"),
    (dict(dkw=BASE + 9 * STEP + 4 * D - 4), None, b"outputs"),
    (dict(ws=BASE + 8 * STEP), None, b"outputs"), (dict(ws=BASE + 3 * STEP), None, b"input"),
    # parts of one gradient that overlap by a row, and the projection itself
    (dict(dk=BASE + 7 * STEP + 2 * (Hq - 1) * D), (Hq * T * D, T * D, D, Hkv * T * D, T * D, D)
     + FUSED, b"outputs"),
    (dict(k=BASE + 2 * STEP + 2 * Hq * D, dq=BASE + 2 * STEP, dk=BASE + 2 * STEP + 2 * Hq * D),
     FUSED * 2, b"input")])
def test_backward_refuses_overlaps(lib, kw, strides, what):
    rc, error = backward(lib, strides, **kw)
    assert rc == -1 and b"qk_norm_rope_bwd" in error and what in error, (rc, error)
