"""Host-side refusals of the 4-bit cache, block-table and norm calls, their workspace sizes, the
rotation's angles on the host, and the oracle's rules.  No GPU: every call here fails before any
CUDA call."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from oracle import attn as OA
from oracle import step as OS

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import transformer_causal_self_gb300 as csattn
    return csattn.load_library()


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


CACHE = dict(q=FAKE, kn=FAKE, vn=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, lens=FAKE,
             slots=FAKE, strides=None, out=FAKE, ko=FAKE, vo=FAKE, B=2, Hq=4, Hkv=2, Tn=8, N=20,
             Lmax=256, Lout=200, page=16, pages=40, per=16, d=64, dtype=1, scale=0.0, msl=200,
             splits=0, ws=FAKE, wb=1 << 30)


def call(lib, op, paged, **kw):
    a = dict(CACHE)
    a.update(kw)
    cache = [a["k"], a["v"], a["ks"], a["vs"]]
    size = [a["page"], a["pages"], a["per"]] if paged else [a["Lmax"]]
    if op == "slots":
        return lib.csattn_cache_append_fp4_slots(
            a["kn"], a["vn"], a["strides"], *cache, a["slots"], a["N"], a["Hkv"], a["page"],
            a["pages"], a["d"], a["dtype"], None)
    if paged:
        cache.append(a["table"])
    sfx = "_paged" if paged else ""
    if op == "append":
        return getattr(lib, "csattn_cache_append_fp4" + sfx)(
            a["kn"], a["vn"], *cache, a["lens"], a["B"], a["Hkv"], a["Tn"], *size, a["d"],
            a["dtype"], None)
    if op == "read":
        return getattr(lib, "csattn_cache_read_fp4" + sfx)(
            *cache, a["lens"], a["ko"], a["vo"], a["B"], a["Hkv"], *size, a["Lout"], a["d"],
            a["dtype"], None)
    return getattr(lib, "csattn_attn_decode_fp4" + sfx)(
        a["q"], *cache, a["lens"], a["out"], a["B"], a["Hq"], a["Hkv"], *size, a["d"], a["dtype"],
        a["scale"], a["msl"], a["splits"], a["ws"], a["wb"], None)


ALL = ["append", "read", "decode"]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("ops,kw,status", [
    (ALL + ["slots"], dict(k=None), -1),
    (ALL + ["slots"], dict(v=None), -1),
    (ALL + ["slots"], dict(ks=None), -1),
    (ALL + ["slots"], dict(vs=None), -1),
    (ALL + ["slots"], dict(k=FAKE + 8), -1),
    (ALL + ["slots"], dict(ks=FAKE + 8), -1),
    (ALL + ["slots"], dict(vs=FAKE + 4), -1),
    (ALL + ["slots"], dict(Hkv=0), -1),
    (ALL + ["slots"], dict(d=96), -2),
    (ALL + ["slots"], dict(d=32), -2),
    (ALL + ["slots"], dict(dtype=0), -2),
    (ALL + ["slots"], dict(dtype=2), -1),
    (ALL, dict(lens=None), -1),
    (ALL, dict(lens=FAKE + 2), -1),
    (ALL, dict(B=0), -1),
    (ALL, dict(B=70000), -2),
    (["append", "slots"], dict(kn=None), -1),
    (["append", "slots"], dict(vn=FAKE + 4), -1),
    (["append"], dict(Tn=0), -1),
    (["append"], dict(Tn=257), -1),
    (["append"], dict(Tn=1 << 20, Lmax=1 << 20, per=1 << 16, B=100), -2),
    (["slots"], dict(slots=None), -1),
    (["slots"], dict(slots=FAKE + 4), -1),
    (["slots"], dict(N=0), -1),
    (["slots"], dict(N=1 << 27), -2),
    (["slots"], dict(page=48), -1),
    (["slots"], dict(pages=0), -1),
    (["slots"], dict(strides=i64(128, 64, 100, 64)), -1),
    (["slots"], dict(strides=i64(-128, 64, 128, 64)), -1),
    (["slots"], dict(strides=i64(128, 4, 128, 64)), -1),
    (["read"], dict(ko=None), -1),
    (["read"], dict(vo=FAKE + 2), -1),
    (["read"], dict(Lout=0), -1),
    (["read"], dict(Lout=1 << 24), -2),
    (["read"], dict(B=32768, Hkv=32768, pages=16, Lout=1), -2),
    (["decode"], dict(q=None), -1),
    (["decode"], dict(out=FAKE + 8), -1),
    (["decode"], dict(Hq=5), -1),
    (["decode"], dict(Hq=0), -1),
    (["decode"], dict(msl=257), -1),
    (["decode"], dict(msl=0), -1),
    (["decode"], dict(splits=-1), -1),
    (["decode"], dict(scale=float("nan")), -1),
    (["decode"], dict(ws=None), -5),
    (["decode"], dict(ws=FAKE + 4), -5),
    (["decode"], dict(wb=64), -5),
])
def test_cache_refusals(lib, ops, kw, status, paged):
    for op in ops:
        assert call(lib, op, paged, **kw) == status, (op, lib.csattn_last_error())
        assert b"fp4" in lib.csattn_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), -1), (dict(table=FAKE + 2), -1), (dict(page=24), -1), (dict(page=0), -1),
    (dict(pages=0), -1), (dict(per=0), -1), (dict(per=1 << 26), -2), (dict(pages=1 << 30), -2)])
def test_page_refusals(lib, kw, status):
    for op in ALL:
        assert call(lib, op, True, **kw) == status, op


def test_workspace_sizes(lib):
    size = lib.csattn_decode_fp4_workspace_size
    for bad in [(0, 4, 2, 256, 64, 0), (2, 5, 2, 256, 64, 0), (2, 4, 2, 256, 96, 0),
                (2, 4, 2, 0, 64, 0), (2, 4, 2, 256, 64, -1)]:
        assert size(*bad) == 0
    # enough for every smaller bound, and no more than a wave's partial results
    for splits in (0, 1, 5):
        for B, Hq, Hkv, d in [(1, 4, 1, 64), (3, 32, 8, 128), (2, 40, 2, 128)]:
            full = size(B, Hq, Hkv, 4096, d, splits)
            assert 0 < full
            for msl in (1, 63, 64, 65, 1000, 4095):
                assert size(B, Hq, Hkv, msl, d, splits) <= full
    assert lib.csattn_qk_norm_rope_bwd_workspace_size(128) >= 4 * 128
    assert lib.csattn_qk_norm_rope_bwd_workspace_size(0) == 0


TABLES = dict(held=FAKE, new=FAKE + 0x1000, table=FAKE + 0x2000, free=FAKE + 0x3000,
              nfree=FAKE + 0x4000, lens=FAKE + 0x5000, starts=FAKE + 0x6000, slots=FAKE + 0x7000,
              pos=FAKE + 0x8000, left=FAKE + 0x9000, B=2, N=20, page=16, pages=40, per=8, size=30)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, -1) for n in ("held", "new", "table", "free", "nfree", "lens", "starts", "slots",
                                "pos", "left")],
    *[({n: TABLES[n] + 2}, -1) for n in ("held", "new", "table", "free", "nfree", "lens", "starts",
                                         "pos", "left")],
    (dict(slots=TABLES["slots"] + 4), -1),
    (dict(B=0), -1), (dict(N=0), -1), (dict(page=17), -1), (dict(pages=0), -1), (dict(per=0), -1),
    (dict(size=-1), -1), (dict(B=65536), -2), (dict(N=(1 << 30) + 1), -2), (dict(per=1 << 26), -2),
    (dict(lens=TABLES["held"]), -1), (dict(lens=TABLES["held"] + 4), -1),
    (dict(left=TABLES["nfree"]), -1), (dict(starts=TABLES["lens"] + 4), -1),
    (dict(pos=TABLES["slots"] + 8), -1), (dict(slots=TABLES["table"] + 32), -1),
    (dict(free=TABLES["table"] + 4), -1), (dict(pos=TABLES["free"] + 116), -1)])
def test_table_refusals(lib, kw, status):
    a = dict(TABLES)
    a.update(kw)
    got = lib.csattn_page_tables(*(a[n] for n in (
        "held", "new", "table", "free", "nfree", "lens", "starts", "slots", "pos", "left", "B", "N",
        "page", "pages", "per", "size")), None)
    assert got == status, lib.csattn_last_error()
    assert b"page_tables" in lib.csattn_last_error()


NORM = dict(q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, pos=None, qo=FAKE, ko=FAKE, dq=FAKE, dk=FAKE,
            dqw=FAKE, dkw=FAKE, B=2, Hq=4, Hkv=2, T=8, d=64, dtype=1, strides=None, pos0=0, norm=1,
            eps=1e-6, base=10000.0, layout=0, ws=FAKE, wb=1 << 30)


def norm_call(lib, back, **kw):
    a = dict(NORM)
    a.update(kw)
    tail = [a["B"], a["Hq"], a["Hkv"], a["T"], a["d"], a["dtype"], a["strides"], a["pos0"],
            a["norm"], a["eps"], a["base"], a["layout"]]
    if back:
        return lib.csattn_qk_norm_rope_bwd(a["qo"], a["ko"], a["q"], a["k"], a["qw"], a["kw"],
                                           a["pos"], a["dq"], a["dk"], a["dqw"], a["dkw"], *tail,
                                           a["ws"], a["wb"], None)
    return lib.csattn_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["qo"], a["ko"],
                                   *tail, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(q=FAKE + 8), -1), (dict(kw=FAKE + 2), -1), (dict(ko=FAKE + 4), -1),
    (dict(pos=FAKE + 2), -1), (dict(B=0), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1),
    (dict(T=0), -1), (dict(dtype=2), -1), (dict(d=96), -2), (dict(d=32), -2),
    (dict(d=8, dtype=0), -2), (dict(T=1 << 24), -2), (dict(B=1 << 12, Hq=1 << 10, T=1 << 10), -2),
    (dict(norm=2), -1), (dict(norm=0), -1), (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(layout=2), -1), (dict(base=float("nan")), -1),
    (dict(base=0.5), -2), (dict(pos0=-1), -1), (dict(pos0=(1 << 24) - 7), -2),
    (dict(strides=i64(100, 64, 64, 1024, 512, 64, 2048, 512, 64, 1024, 512, 64)), -1),
    (dict(strides=i64(2048, -8, 64, 1024, 512, 64, 2048, 512, 64, 1024, 512, 64)), -1),
    (dict(strides=i64(2048, 512, 64, 1024, 512, 4, 2048, 512, 64, 1024, 512, 64)), -1)])
def test_norm_refusals(lib, kw, status):
    for back in (False, True):
        assert norm_call(lib, back, **kw) == status, (back, lib.csattn_last_error())
        assert b"qk_norm_rope" in lib.csattn_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), -1), (dict(dk=FAKE + 8), -1), (dict(dqw=None), -1), (dict(kw=None), -1),
    (dict(dkw=FAKE + 2), -1), (dict(ws=None), -5), (dict(ws=FAKE + 8), -5), (dict(wb=1000), -5),
    (dict(strides=i64(2048, 512, 64, 1024, 512, 64, 2048, 512, 12, 1024, 512, 64)), -1)])
def test_norm_backward_refusals(lib, kw, status):
    assert norm_call(lib, True, **kw) == status, lib.csattn_last_error()


ANGLES = r"""
#include <cmath>
#include <cstdio>
#include "rope_turns.cuh"
int main() {
  for (double base : {1.0, 1.5, 100.0, 10000.0, 500000.0, 1e8})
    for (int d : {16, 64, 128}) {
      long double worst = 0;
      for (int p = 0; p < d / 2; ++p) {
        const long double th = std::pow(base, -2.0 * p / d);
        const double q = std::pow(base, -2.0 * p / d) * 0.63661977236758134308;
        const float hi = static_cast<float>(q), lo = static_cast<float>(q - hi);
        for (int pos = 0; pos < (1 << 24); pos += pos < 256 ? 1 : 1 + (pos * 7LL + p) % 3001) {
          float c, s;
          csattn::turn_cos_sin(pos, hi, lo, c, s);
          const long double a = static_cast<long double>(pos) * th;
          worst = std::fmax(worst, std::fmax(std::fabs(c - std::cos(a)), std::fabs(s - std::sin(a))));
        }
      }
      std::printf("%g %d %.4f\n", base, d, static_cast<double>(worst * 4194304.0L));
    }
}
"""


def test_angles_are_good_to_their_bound(tmp_path):
    """turn_cos_sin, compiled for the host: off by less than 2^-22 at every position below 2^24.
    Its parts: the frequency as two floats, 2^-50 of at most 2^23.4 quarter turns; what is left of
    the angle, at most pi/4, rounded three times (2^-24 of it each); the Taylor sums, 2^-27 and
    their roundings, 2^-23."""
    from transformer_causal_self_gb300 import build
    src, exe = tmp_path / "angles.cu", tmp_path / "angles"
    src.write_text(ANGLES)
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    build.CSRC, str(src), "-o", str(exe)], check=True, capture_output=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    worst = [float(x.split()[2]) for x in lines if x]
    assert len(worst) == 18 and max(worst) < 1.0, lines


# ------------------------------------------------------------------ Python's own checks
def test_python_refuses_host_tensors_and_wrong_types():
    import transformer_causal_self_gb300 as csattn
    x = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16)
    c4, s4 = torch.zeros(2, 2, 8, 32, dtype=torch.uint8), torch.zeros(2, 2, 8, 4, dtype=torch.uint8)
    lens = torch.zeros(2, dtype=torch.int32)
    for call_ in (lambda: csattn.attn_decode_fp4(x, c4, c4, s4, s4, lens),
                  lambda: csattn.cache_append_fp4(x, x, c4, c4, s4, s4, lens),
                  lambda: csattn.cache_append_fp4_slots(x[:, :, 0], x[:, :, 0], c4, c4, s4, s4,
                                                        lens.long()),
                  lambda: csattn.cache_read_fp4(c4, c4, s4, s4, lens),
                  lambda: csattn.qk_norm_rope(x, x),
                  lambda: csattn.qk_norm_rope_bwd(x, x, x, x),
                  lambda: csattn.page_tables(lens, lens, lens.view(1, 2), lens, lens[:1], 4,
                                             page_size=16, num_pages=2)):
        with pytest.raises(ValueError, match="CUDA"):
            call_()


@pytest.mark.parametrize("shape,strides,shared", [
    ((2, 3, 5, 64), (3 * 5 * 64, 5 * 64, 64), False), ((2, 3, 5, 64), (5 * 512, 64, 512), False),
    ((2, 3, 5, 64), (0, 5 * 64, 64), True), ((1, 3, 5, 64), (0, 5 * 64, 64), False),
    ((2, 3, 5, 64), (5 * 512, 32, 512), True), ((2, 3, 5, 64), (512, 64, 512), True),
    ((2, 1, 5, 64), (5 * 64, 0, 64), False)])
def test_places_that_elements_share(shape, strides, shared):
    import transformer_causal_self_gb300 as csattn
    assert csattn._shares_places(shape, strides) == shared


# ------------------------------------------------------------------ the oracle's own rules
def test_fp4_scales_are_f16s_upper_bits():
    f16 = (np.arange(OS._TOP + 1).astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(OS.fp4_scales(), f16)
    assert f16[-1] == 10240 and 6 * f16[-1] < 65504 < 6 * f16[-1] * 11 / 10


def test_fp4_rounding():
    x = np.zeros((1, 16))
    x[0, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]   # a / 6 = 1: the borders are ties
    x[0, 8:] = [-6, -5.001, -3.501, -2.499, 1.751, 1.249, -0.751, 0.251]
    data, code, v = OS.quantise_fp4(x)
    assert code[0, 0] == 15 * 8
    assert list(v[0]) == [6, 4, 4, 2, 2, 1, 1, 0, -6, -6, -4, -2, 2, 1, -1, 0.5]
    assert np.array_equal(OS.fp4_values(data, code), v)
    # every product is a bf16 number
    s = OS.fp4_scales()[:, None] * OS.E2M1
    assert np.array_equal(OA.round_to_bf16(s), s)
    bad = np.full((1, 32), 6.0)
    bad[0, 3] = np.inf
    data, code, v = OS.quantise_fp4(bad)
    assert code[0, 0] == 255 and not data[0, :8].any() and np.isnan(v[0, :16]).all()
    assert np.all(v[0, 16:] == 6)


def test_fp4_quotients_are_on_a_border_or_far_from_one():
    """What the kernels' arithmetic rests on, for every magnitude of 8 significant bits: a / 6
    against the borders between scales, x / s against those between e2m1 values."""
    x = np.concatenate([np.arange(128, 256) * 2.0 ** e for e in range(-30, 12)])
    s = OS.fp4_scales()
    mid = (s[1:] + s[:-1]) / 2
    a = x[x / 6 < s[-1]] / 6
    near = np.abs(a[:, None] - mid[None, :]).min(1)
    assert np.all((near == 0) | (near > 2.0 ** -9 * a) | (a < mid[0] / 2))
    emid = (OS.E2M1[1:] + OS.E2M1[:-1]) / 2
    for sc in s[1:]:
        y = x / sc
        y = y[y < 8]
        near = np.abs(y[:, None] - emid[None, :]).min(1)
        assert np.all((near == 0) | (near >= 2.0 ** -10))


def test_norm_gradients_are_those_of_differences():
    rng = np.random.default_rng(5)
    x, dy = rng.normal(size=(2, 3, 4, 16)), rng.normal(size=(2, 3, 4, 16))
    w, pos = rng.normal(size=16), rng.integers(0, 100, size=(2, 4))
    for layout in ("split_half", "adjacent"):
        for norm in (True, False):
            args = (pos, 1e-3, 100.0, layout, norm)
            dx, dw = OS.qk_norm_rope_bwd(dy, x, w if norm else None, *args)
            f = lambda a, b: (OS.qk_norm_rope(a, b if norm else None, *args) * dy).sum()  # noqa
            u, h = rng.normal(size=x.shape), 1e-5
            assert np.isclose((f(x + h * u, w) - f(x - h * u, w)) / (2 * h), (dx * u).sum(),
                              rtol=1e-7, atol=1e-7)
            if norm:
                u = rng.normal(size=16)
                assert np.isclose((f(x, w + h * u) - f(x, w - h * u)) / (2 * h), (dw * u).sum(),
                                  rtol=1e-7, atol=1e-7)


def test_table_rules():
    t, lens, starts, slots, pos, left, wrong = OS.page_tables(
        [15, 0, 16, 3], [2, 0, 1, 1], [[5, -1], [-1, -1], [6, -1], [7, -1]], [9, 8, 4, 3], 3, 6, 16,
        10)
    assert t == [[5, 4], [-1, -1], [6, 8], [7, -1]] and lens == [17, 0, 17, 4]
    assert starts == [0, 2, 2, 3, 4] and left == 1 and not wrong
    assert slots == [5 * 16 + 15, 4 * 16, 8 * 16, 7 * 16 + 3, -1, -1] and pos == [15, 16, 16, 3, 0, 0]
