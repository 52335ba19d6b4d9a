"""Decode over a 4-bit cache against float64 on the cache's exact values."""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from tests import fp4_helpers as H
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hkv,page,splits", [
    (128, 32, 8, 64, 0), (128, 4, 1, 0, 0), (128, 8, 1, 16, 3), (128, 7, 1, 32, 0),
    (128, 2, 2, 128, 0), (128, 16, 1, 64, 0), (128, 9, 1, 0, 2), (128, 40, 2, 64, 0),
    (64, 8, 2, 64, 0), (64, 1, 1, 0, 0), (64, 12, 12, 16, 0), (64, 16, 1, 32, 5),
    (64, 24, 1, 192, 0)])
def test_decode_parity(d, Hq, Hkv, page, splits):
    """Lengths of one row, around a tile's and a page's ends, and none at all; NaN behind them."""
    lens = [1, 64, 200, 63, 0, 65, 17, 129, 16, 191]
    c, q = H.filled(len(lens), Hq, Hkv, d, page, lens, 200, seed=Hq)
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens), num_splits=splits)
    csattn.check_status()
    assert torch.all(out[4] == 0)
    H.assert_close(out, H.expect(c, q, lens))


@pytest.mark.parametrize("d,Lmax", [(64, 33), (64, 70), (64, 201), (128, 33), (128, 201), (64, 1)])
def test_contiguous_caches_of_odd_lengths(d, Lmax):
    """Planes of scale bytes that do not begin on 16 bytes."""
    lens = [Lmax, max(1, Lmax // 2), 1]
    c, q = H.filled(3, 4, 2, d, 0, lens, Lmax, seed=Lmax)
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens))
    csattn.check_status()
    H.assert_close(out, H.expect(c, q, lens))


@pytest.mark.parametrize("d,Hq,Hkv,page", [
    (128, 32, 8, 64), (128, 4, 1, 16), (128, 7, 1, 192), (128, 8, 8, 0), (128, 16, 1, 128),
    (128, 40, 2, 64), (64, 8, 2, 64), (64, 12, 12, 16), (64, 16, 1, 32), (64, 24, 1, 384),
    (64, 3, 3, 0)])
def test_long_tiles(d, Hq, Hkv, page):
    """Caches with room for so much that the tiles are of 192 rows: lengths around their ends, the
    pages' and the groups' of 16 rows within them."""
    lens = [192, 1, 193, 191, 0, 400, 48, 49, 160, 576, 577, 65, 384, 15, 240, 17]
    room = 6144 + (0 if page else 9)  # (contiguous planes whose scales are not on 16 bytes, too)
    c, q = H.filled(len(lens), Hq, Hkv, d, page, lens, 577 if page else 640, seed=Hq)
    if page:  # entries of pages that no row is on
        per = -(-room // page)
        table = torch.full((len(lens), per), -1, dtype=torch.int32)
        table[:, :c["table"].shape[1]] = c["table"]
        c["table"] = table
        out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens))
    else:
        big = H.empty_cache(len(lens), Hkv, room, d, 0, seed=1)
        for n in H.NAMES:
            big[n][:, :, :c[n].shape[2]] = c[n]
        c = big
        out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens))
    csattn.check_status()
    assert torch.all(out[4] == 0)
    H.assert_close(out, H.expect(c, q, lens))


@pytest.mark.parametrize("gain,scale", [(8.0, 0.0), (1e-3, 0.0), (1.0, 3.0), (1e30, 1e-30),
                                        (1e-30, 1e30), (30.0, 0.0)])
def test_large_and_small_scores(gain, scale):
    """Peaked and flat softmaxes, and queries at the ends of bf16's range."""
    lens = [300, 77]
    c, q = H.filled(2, 8, 2, 128, 64, lens, 320, seed=5, gain=gain)
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens), scale=scale)
    csattn.check_status()
    H.assert_close(out, H.expect(c, q, lens, scale or None))


def test_scores_that_grow_row_by_row():
    """Every tile raises the maximum; and a first row that takes nearly all of the weight."""
    L, d = 400, 128
    c, q = H.filled(2, 4, 1, d, 64, [L, L], L, seed=2)
    k = torch.ones(1, L, d, dtype=torch.bfloat16) * torch.arange(L).view(1, L, 1) / 40
    v = torch.randn(1, L, d, generator=H.gen(8))
    H.set_rows(c, 0, 0, k.to(torch.bfloat16), v.to(torch.bfloat16))
    H.set_rows(c, 1, 0, k.flip(1).to(torch.bfloat16), v.to(torch.bfloat16))
    q[:] = 1.5
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32([L, L]))
    csattn.check_status()
    H.assert_close(out, H.expect(c, q, [L, L]))


def test_values_of_very_different_sizes():
    """The format's largest and smallest values beside one another, under equal weights."""
    L, d = 130, 64
    c, q = H.filled(1, 4, 1, d, 0, [L], L, seed=2)
    v = torch.randn(1, L, d, generator=H.gen(8)) * 2.0 ** torch.randint(-15, 13, (1, L, 1),
                                                                        generator=H.gen(9))
    v[0, 3], v[0, 70] = 61440.0, -61440.0
    H.set_rows(c, 0, 0, torch.randn(1, L, d, generator=H.gen(7)).to(torch.bfloat16),
               v.to(torch.bfloat16))
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32([L]))
    csattn.check_status()
    H.assert_close(out, H.expect(c, q, [L]))


def test_nan_in_sight_and_out_of_it():
    """A NaN key makes its KV head's outputs NaN, a NaN value block its 16 channels; other heads and
    sequences, and rows behind the length, have no part in it."""
    lens = [100, 100]
    c, q = H.filled(2, 4, 2, 128, 64, lens, 192, seed=3)
    ref = H.expect(c, q, lens)
    p, o = H.place(c, 0, 70)
    c["ks"][p, 0, o, 3] = 255
    p, o = H.place(c, 1, 3)
    c["vs"][p, 1, o, 2] = 255
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens))
    csattn.check_status()
    assert torch.isnan(out[0, :2]).all()
    assert torch.isnan(out[1, 2:, 0, 32:48]).all()
    got = out.clone()
    for at in ((0, slice(0, 2)), (1, slice(2, 4), 0, slice(32, 48))):
        assert np.isfinite(ref[0][at]).all()
        got[at] = torch.from_numpy(ref[0][at]).to(got.dtype).to(dev())
    H.assert_close(got, ref)


def test_queries_that_are_not_finite():
    lens = [50, 50]
    c, q = H.filled(2, 4, 1, 64, 16, lens, 64, seed=3)
    q[0, 1, 0, 5], q[0, 2, 0, 6] = float("nan"), float("inf")
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens))
    csattn.check_status()
    assert torch.isnan(out[0, 1]).all() and not torch.isfinite(out[0, 2]).any()
    q[0, 1], q[0, 2] = q[0, 0], q[0, 0]
    ref = H.expect(c, q, lens)
    out[0, 1], out[0, 2] = out[0, 0], out[0, 0]
    H.assert_close(out, ref)


def test_lengths_and_pages_out_of_range():
    lens = [40, 40, 40]
    c, q = H.filled(3, 4, 2, 64, 16, lens, 48, seed=6)
    ref = H.expect(c, q, lens)
    cd, qd = H.to_dev(c), q.to(dev())
    for bad in (-1, 49, 2 ** 31 - 1, -2 ** 31):
        out = H.decode(cd, qd, H.i32([40, bad, 40]))
        H.refused()
        assert torch.all(out[1] == 0)
        H.assert_close(out[::2], tuple(x[::2] for x in ref))
    out = H.decode(cd, qd, H.i32([40, 0, 40]))
    csattn.check_status()
    assert torch.all(out[1] == 0)
    # a bound below a length
    out = H.decode(cd, qd, H.i32([40, 33, 40]), max_seq_len=39)
    H.refused()
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0) and torch.any(out[1] != 0)
    # rows on a page outside the pool read as zeros
    for bad in (-1, cd["k"].shape[0], 2 ** 31 - 1):
        cd["table"].copy_(c["table"])
        cd["table"][1, 1] = bad
        out = H.decode(cd, qd, H.i32(lens))
        H.refused()
        zero = {n: (x.clone() if isinstance(x, torch.Tensor) else x) for n, x in c.items()}
        for r in range(16, 32):
            p, o = H.place(c, 1, r)
            for n in H.NAMES:
                zero[n][p, :, o] = 0
        H.assert_close(out, H.expect(zero, q, lens))


def test_many_sequences_and_one_long_one():
    """More segments than CTAs, and a sequence over many CTAs among short ones."""
    lens = [(37 * i) % 70 for i in range(200)]
    lens[77] = 5000
    c, q = H.filled(200, 4, 2, 64, 64, lens, 5056, seed=4)
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens), max_seq_len=5000)
    csattn.check_status()
    H.assert_close(out, H.expect(c, q, lens))


@pytest.mark.parametrize("d,rep,splits", [(128, 4, 0), (128, 1, 1), (128, 9, 0), (64, 4, 0),
                                          (64, 5, 1), (64, 16, 0), (64, 1, 0)])
def test_many_tiles_per_cta_from_any_pages(d, rep, splits):
    """Ranges of more tiles than a warp's lanes read pages for at once: the same bits from pages of
    every size, from a contiguous cache and from one whose planes start anywhere; right for some
    sequences; and rows on pages outside the pool read as zeros whichever way they are copied."""
    B, Hkv, room = (24, 8, 6144) if splits == 0 else (2, 2, 6144)
    g = H.gen(rep)
    lens = [room - 131 * b for b in range(B)]
    lens[1] = 777
    c = {"table": None, "page": 0}
    for n in ("k", "v"):
        c[n] = torch.randint(0, 256, (B, Hkv, room, d // 2), generator=g, dtype=torch.uint8)
        c[n + "s"] = torch.randint(90, 130, (B, Hkv, room, d // 16), generator=g, dtype=torch.uint8)
    q = torch.randn(B, Hkv * rep, 1, d, generator=g).to(torch.bfloat16)
    qd, ld = q.to(dev()), H.i32(lens)
    want = H.decode(H.to_dev(c), qd, ld, num_splits=splits)
    csattn.check_status()
    for b in (1, B - 1):
        only = [n if i == b else 0 for i, n in enumerate(lens)]
        H.assert_close(want[b:b + 1], tuple(x[b:b + 1] for x in H.expect(c, q, only)))
    shifted = dict(c)
    for n in H.NAMES:
        shifted[n] = torch.cat([c[n], torch.full_like(c[n][:, :, :1], 255)], 2).contiguous()
    out = H.decode(H.to_dev(shifted), qd, ld, num_splits=splits, max_seq_len=room)
    csattn.check_status()
    assert H.same(out, want)
    for page in (16, 32, 64, 128, 192, 384, 1024):
        per = room // page
        order = torch.randperm(B * per, generator=g)
        paged = {"page": page, "table": torch.empty(B * per, dtype=torch.int32)}
        paged["table"][:] = order.argsort().to(torch.int32)
        paged["table"] = paged["table"].view(B, per)
        for n in H.NAMES:  # page p of the pool is piece order[p] of the sequences
            x = c[n].view(B, Hkv, per, page, -1).transpose(1, 2).reshape(B * per, Hkv, page, -1)
            paged[n] = x[order].contiguous()
        pd = H.to_dev(paged)
        out = H.decode(pd, qd, ld, num_splits=splits)
        csattn.check_status()
        assert H.same(out, want), page
        at = 5000 // page if page < 1024 else 1
        pd["table"][0, at] = B * per
        out = H.decode(pd, qd, ld, num_splits=splits)
        H.refused()
        zero = dict(c)
        for n in H.NAMES:
            zero[n] = c[n].clone()
            zero[n][0, :, at * page:(at + 1) * page] = 0
        other = H.decode(H.to_dev(zero), qd, ld, num_splits=splits)
        assert H.same(out, other) and not H.same(out, want), page


@pytest.mark.parametrize("B,heads", [(1, 1), (1, 3), (3, 5), (1, 4097)])
def test_odd_numbers_of_rows(B, heads):
    lens = [20] * B
    c, q = H.filled(B, heads, heads, 64, 0, lens, 24, seed=heads)
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens))
    csattn.check_status()
    H.assert_close(out, H.expect(c, q, lens))


def test_a_wait_that_runs_out_is_reported():
    lens = [100] * 300
    c, q = H.filled(300, 4, 2, 64, 0, [100], 102, seed=1)
    c = {n: (x[:1].expand(300, -1, -1, -1).contiguous() if isinstance(x, torch.Tensor) else x)
         for n, x in c.items()}
    cd, qd, ld = H.to_dev(c), q[:1].expand(300, -1, -1, -1).contiguous().to(dev()), H.i32(lens)
    need = csattn.decode_fp4_workspace_size(300, 4, 2, 102, 64)

    def run():
        return H.decode(cd, qd, ld, workspace=torch.full((need,), 0x7E, dtype=torch.uint8,
                                                         device=dev()))

    want = run().clone()
    csattn.check_status()
    csattn.selftest_lost_arrival()
    run()
    with pytest.raises(csattn.CsattnError) as e:
        csattn.check_status()
    assert e.value.status == -4
    again = run()
    csattn.check_status()
    assert H.same(again, want)


def test_graphs_streams_and_repeats():
    """Captured twice and replayed over other inputs in the same buffers; another stream; a stream
    inside a capture; equal inputs give equal bits."""
    lens = [100, 37]
    c, q = H.filled(2, 8, 2, 128, 64, lens, 128, seed=21)
    cd, qd, ld = H.to_dev(c), q.to(dev()), H.i32(lens)
    first = H.decode(cd, qd, ld)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = H.decode(cd, qd, ld, stream=side)
    side.synchronize()
    assert H.same(out, first)
    graphs = []
    for _ in range(2):
        o = torch.empty_like(first)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            H.decode(cd, qd, ld, out=o)
            side.wait_stream(torch.cuda.current_stream())
            two = H.decode(cd, qd, ld, stream=side)
            torch.cuda.current_stream().wait_stream(side)
        graphs.append((gr, o, two))
    qd.mul_(-1)
    ld.copy_(H.i32([3, 128]))
    for n in ("ks", "vs"):
        cd[n][cd[n] == 255] = 100
    other = H.decode(cd, qd, ld)
    for gr, _, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    csattn.check_status()
    for _, o, two in graphs:
        assert H.same(o, other) and H.same(two, other)
    assert not H.same(other, first)
