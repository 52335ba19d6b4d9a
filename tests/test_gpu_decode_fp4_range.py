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
