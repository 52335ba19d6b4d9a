"""Decode over a 4-bit cache where scores, weights and lengths go to their ends."""
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from tests import fp4_helpers as H
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("log2", [0, 4, 10, 16, 23, 40, 60, 80, 100])
@pytest.mark.parametrize("at", [0, 17, 130, 299])
def test_one_row_takes_all_at_any_size_of_scores(d, log2, at):
    """Scores of up to 2^119, where fp32 numbers are far apart: the row with the largest score, which
    is ahead of the others by at least half of it, is the output to the bit (the others' weights are
    below 2^-1000, the row's own divides out, and a value is a bf16 number); two such rows give
    their mean, which one rounding to bf16 (2^-8) and the weights' and sums' (2^-11, 2^-20) leave
    within 2^-7 of their magnitudes."""
    L, rep = 300, 4
    c, q = H.filled(2, rep, 1, d, 64, [L, L], L, seed=at)
    g = H.gen(log2)
    sign = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    k = sign * 4096 * torch.rand(L, 1, generator=g).repeat(1, d)  # up to half of the largest
    k[at] = 8192 * sign
    twin = (at + 61) % L
    two = k.clone()
    two[twin] = k[at]
    v = torch.randn(L, d, generator=g)
    for b, rows in enumerate((k, two)):
        H.set_rows(c, b, 0, rows[None].to(torch.bfloat16), v[None].to(torch.bfloat16))
    size = torch.tensor([1.0, 1.25, 1.5, 1.9375]) * 2.0 ** log2
    q[:] = (size.view(rep, 1, 1) * sign).to(torch.bfloat16)
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32([L, L])).cpu().double()
    csattn.check_status()
    held = torch.from_numpy(H.rows(c, 0, L)[1][0])
    assert torch.equal(out[0, :, 0], held[at].expand(rep, d))
    want, tol = (held[at] + held[twin]) / 2, (held[at].abs() + held[twin].abs()) * 2.0 ** -7
    assert torch.all((out[1, :, 0] - want).abs() <= tol)


@pytest.mark.parametrize("d", [64, 128])
def test_a_maximum_that_lags_behind_large_scores(d):
    """A later row whose score is 5 to 11 (in powers of two) above the first one's, at 2^24 and 2^26,
    where scores are rounded to steps of 2 and 8: they are off by half a step each, so the later row
    has a weight of 2^-(5 - 8) to 1 times the first one's; whichever it is, the output is between
    the two rows (the rest have no weight), within 2^-7 of their magnitudes."""
    L, rep = 300, 16
    c, q = H.filled(2, rep, 1, d, 0, [L, L], L, seed=d)
    g = H.gen(d)
    v = torch.randn(L, d, generator=g)
    for b, log2 in enumerate((24, 26)):
        # the score, in powers of two: size * 8192 * (d - 16) * log2(e) / sqrt(d)
        size = 1.1 * 2.0 ** (log2 - 13) * d ** 0.5 / ((d - 16) * 1.4427)
        k = torch.zeros(L, d)
        k[0] = k[256] = 8192.0
        k[0, :16] = -8192.0  # one block of small channels of the query
        x = torch.full((rep, d), size)
        x[:, :16] = 0.0
        ahead = torch.linspace(5.0, 11.0, rep)
        x[:, 3] = ahead * d ** 0.5 / (2 * 8192.0 * 1.4427)
        q[b, :, 0] = x.to(torch.bfloat16)
        H.set_rows(c, b, 0, k[None].to(torch.bfloat16), v[None].to(torch.bfloat16))
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32([L, L]), num_splits=1).cpu().double()
    csattn.check_status()
    held = torch.from_numpy(H.rows(c, 0, L)[1][0])
    lo, hi = torch.minimum(held[0], held[256]), torch.maximum(held[0], held[256])
    tol = (held[0].abs() + held[256].abs()) * 2.0 ** -7
    assert torch.all(out[:, :, 0] >= lo - tol) and torch.all(out[:, :, 0] <= hi + tol)


@pytest.mark.parametrize("d", [64, 128])
def test_many_small_weights_behind_a_dominant_one(d):
    """Weights of 2^-19 to 2^-34 of the first row's, whose value is 0: what is left of each is within
    2^-11 of it and 2^-32 of the largest; the other terms as in fp4_helpers.expect."""
    L, rep = 3000, 16
    c = H.empty_cache(1, 1, L, d, 0, seed=d)
    k, v = torch.zeros(1, L, d), torch.full((1, L, d), 24576.0)
    k[:, 0], v[:, 0] = 1.0, 0.0
    H.set_rows(c, 0, 0, k.to(torch.bfloat16), v.to(torch.bfloat16))
    ahead = torch.arange(19.0, 19.0 + rep) + 0.4  # (powers of two)
    q = (ahead / (d ** 0.5 * 1.442695)).view(1, rep, 1, 1).expand(1, rep, 1, d)
    q = q.to(torch.bfloat16).contiguous()
    for splits in (0, 1, 7):
        out = H.decode(H.to_dev(c), q.to(dev()), H.i32([L]), num_splits=splits)
        csattn.check_status()
        s = q[0, :, 0].double() @ torch.from_numpy(H.rows(c, 0, 1)[0][0, 0]) * d ** -0.5
        w = torch.exp(-s) * (L - 1)
        want = 24576.0 * w / (1 + w)
        off = 2.0 ** -17 * s
        tol = (want * (2.0 ** -11 + 2 * off + 2.0 ** -18 + 2.0 ** -8)
               + 24576.0 * (L - 1) * 2.0 ** -32) * (1 + 2.0 ** -7)
        got = out[0, :, 0].double().cpu()
        assert torch.all((got - want[:, None]).abs() <= tol[:, None]), (got[:, 0], want, tol)


@pytest.mark.parametrize("d,Hq,Hkv,page", [
    (128, 32, 8, 64), (128, 16, 1, 128), (128, 7, 1, 16), (128, 8, 8, 0), (64, 8, 2, 64),
    (64, 24, 1, 384), (64, 12, 12, 16), (64, 3, 3, 0)])
def test_lengths_at_the_long_tiles_ends(d, Hq, Hkv, page):
    """Caches with room for so much that the tiles are the long ones, of 128 rows (128 channels) or
    192 (64): lengths at the ends of one, two and three of them, and a row to either side."""
    lens = [127, 128, 129, 255, 256, 257, 383, 384, 385, 191, 192, 193, 575, 576, 577, 0, 1]
    room = 6144 + (0 if page else 9)
    c, q = H.filled(len(lens), Hq, Hkv, d, page, lens, 577 if page else room, seed=page + d)
    if page:
        table = torch.full((len(lens), room // page), -1, dtype=torch.int32)
        table[:, :c["table"].shape[1]] = c["table"]
        c["table"] = table
    out = H.decode(H.to_dev(c), q.to(dev()), H.i32(lens))
    csattn.check_status()
    assert torch.all(out[15] == 0)
    H.assert_close(out, H.expect(c, q, lens))


@pytest.mark.skipif(not hasattr(torch, "float4_e2m1fn_x2"), reason="no packed e2m1 type")
@pytest.mark.parametrize("page", [0, 64])
def test_caches_of_torchs_packed_type(page):
    """Appended to, read and decoded as torch.float4_e2m1fn_x2: the same bytes as of uint8."""
    lens = [70, 3]
    c, q = H.filled(2, 8, 2, 64, page, lens, 128, seed=3)
    kn, vn = (H.tokens(c, 2 * 9, 2, 64, s).view(2, 9, 2, 64).transpose(1, 2).contiguous().to(dev())
              for s in (1, 2))
    plain, packed = H.to_dev(c), H.to_dev(c)
    for n in ("k", "v"):
        packed[n] = packed[n].view(torch.float4_e2m1fn_x2)
    for x in (plain, packed):
        H.append(x, kn, vn, H.i32(lens))
    ends = H.i32([n + 9 for n in lens])
    for n in ("k", "v"):
        assert torch.equal(packed[n].view(torch.uint8), plain[n])
    for a, b in zip(H.read(plain, ends), H.read(packed, ends)):
        assert H.same(a[0, :, :79], b[0, :, :79]) and H.same(a[1, :, :12], b[1, :, :12])
    assert H.same(H.decode(plain, q.to(dev()), ends), H.decode(packed, q.to(dev()), ends))
    if page:
        slots = torch.tensor([5, -1, 64], device=dev())
        for x in (plain, packed):
            csattn.cache_append_fp4_slots(kn[0, :, :3].transpose(0, 1).contiguous(),
                                          vn[0, :, :3].transpose(0, 1).contiguous(), *H.cache(x),
                                          slots)
        assert torch.equal(packed["k"].view(torch.uint8), plain["k"])
    csattn.check_status()
