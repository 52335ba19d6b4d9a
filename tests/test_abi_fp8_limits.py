"""Limits of the 8-bit cache and token-tree calls that the host checks, and their RoPE angles on the
host.  No GPU: every call here fails before any CUDA call."""
import subprocess

import pytest

from tests.test_abi_fp8_tree import call, lib  # noqa: F401 (lib is the fixture)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw", [dict(B=32768, Hkv=32768), dict(B=65535, Hkv=32767)])
def test_read_of_too_many_heads(lib, kw, paged):  # noqa: F811
    """B * Hkv at 2^30 and above is past the limits, not a failed launch."""
    assert call(lib, "read", paged, Lout=1, pages=16, **kw) == -2
    assert b"too large" in lib.csattn_last_error()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("op", ["append", "decode", "tree"])
def test_rope_bases_below_one(lib, op, paged):  # noqa: F811
    """Angles past the range in which they are reduced exactly are refused; those within go on (to
    the check of something else)."""
    for kw in (dict(base=1e-3), dict(base=1e-3, d=128), dict(base=1e-30)):
        assert call(lib, op, paged, **kw) == -2
        assert b"RoPE" in lib.csattn_last_error()
    if op != "append":
        assert call(lib, op, paged, base=0.5, ws=None) == -5
        assert call(lib, op, paged, base=0.01, ws=None) == -5


ANGLES = r"""
#include <cmath>
#include <cstdio>
#include "fp8.cuh"
int main() {
  for (double base : {1.0, 1.5, 100.0, 10000.0, 500000.0, 1e8})
    for (int d : {64, 128}) {
      long double worst = 0;
      for (int p = 0; p < d / 2; ++p) {
        const double th = std::pow(base, -2.0 * p / d);
        const float hi = static_cast<float>(th), lo = static_cast<float>(th - hi);
        for (int pos = 0; pos < 49152; pos += pos < 256 ? 1 : 1 + (pos * 7 + p) % 61) {
          float c, s;
          csattn::angle_cos_sin(pos, hi, lo, c, s);
          const long double a = static_cast<long double>(pos) * th;
          worst = std::fmax(worst, std::fmax(std::fabs(c - std::cos(a)), std::fabs(s - std::sin(a))));
        }
      }
      std::printf("%g %d %.4f\n", base, d, static_cast<double>(worst * 8388608.0L));
    }
}
"""


def test_angles_are_good_to_their_bound(tmp_path):
    """angle_cos_sin, compiled for the host (the same fp32 operations and fused ones): off by less
    than 2^-23 at every frequency, over the positions that the calls accept."""
    from transformer_causal_self_gb300 import build
    src, exe = tmp_path / "angles.cu", tmp_path / "angles"
    src.write_text(ANGLES)
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    build.CSRC, str(src), "-o", str(exe)], check=True, capture_output=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    worst = [float(x.split()[2]) for x in lines if x]
    assert len(worst) == 12 and max(worst) < 1.0, lines
