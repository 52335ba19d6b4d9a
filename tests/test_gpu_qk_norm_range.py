"""Norm of queries and keys at the ends of the numbers' range, and gains' gradients over many rows.

Tolerances as in test_gpu_qk_norm.py; a stored fp32 below 2^-126 is rounded to half a step of 2^-149.
"""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import step as OS
from tests.fp8_helpers import gen
from tests.gpu_helpers import dev
from tests.test_gpu_qk_norm import case, np64, pair_lengths, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64),
                                     (torch.float32, 64), (torch.float32, 16)])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-30, 1e-6])
def test_heads_whose_squares_leave_the_range(dtype, d, eps):
    """Heads of magnitudes 2^-130 to 2^124, with an eps far below them, beside them and far above."""
    eps = float(np.float32(eps))
    logs = [-130, -126, -100, -75, -64, -50, -41, 0, 50, 59, 63, 64, 100, 124]
    q, k, w, dy = case(2, len(logs), 3, 5, d, dtype, False, seed=d)
    for h, e in enumerate(logs):
        q[:, h] = (q[:, h].double() * 2.0 ** e).to(dtype)
        dy[0][:, h] *= 2.0 ** (-20 if e < 0 else 0)
    q[1, 3, 2] *= torch.where(torch.arange(d, device=dev()) % 3 == 0, 2.0 ** -40, 1.0).to(dtype)
    k[0, 1], k[1, 2] = k[0, 1] * 2.0 ** -70, k[1, 2] * 2.0 ** 70
    if eps == 0.0:
        assert (q.float() != 0).any(-1).all()
    kw = dict(eps=eps, rope_base=10000.0)
    out = csattn.qk_norm_rope(q, k, *w, **kw)
    grads = csattn.qk_norm_rope_bwd(*dy, q, k, *w, **kw)
    csattn.check_status()
    pos = np.tile(np.arange(5), (2, 1))
    least = 0.0 if dtype == torch.bfloat16 else 2.0 ** -149
    for i, (x, y, dx, dw) in enumerate(zip((q, k), out, grads[:2], grads[2:])):
        what, xn, wn, dyn = "qk"[i], np64(x), np64(w[i]), np64(dy[i])
        flat = OS.qk_norm_rope(xn, wn, pos, eps, 0.0, "split_half")
        within(y, OS.qk_norm_rope(xn, wn, pos, eps, 10000.0, "split_half"),
               2.0 ** -19 * pair_lengths(flat, 10000.0, "split_half") + least, what)
        rx, rw = OS.qk_norm_rope_bwd(dyn, xn, wn, pos, eps, 10000.0, "split_half")
        lg = pair_lengths(dyn, 10000.0, "split_half")
        r = 1 / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps)
        n, a = xn * r, np.abs(wn)
        g = OS._turn(dyn, pos, 10000.0, "split_half", back=True)
        size = r * (lg * a + np.abs(n) * np.mean(np.abs(g * a * n), -1, keepdims=True))
        assert size.max() < 3e38  # (nothing here is past the type's range)
        within(dx, rx, 2.0 ** -18 * size + least, "d" + what)
        within(dw, rw, 2.0 ** -16 * (lg * np.abs(n)).sum((0, 1, 2)), "d" + what + "w")


def test_a_head_of_zeros_without_eps():
    """0 / 0: NaN in that head and in what it is summed into, and nowhere else."""
    q, k, w, dy = case(1, 4, 2, 8, 64, torch.bfloat16, False, seed=5)
    kw = dict(eps=0.0, rope_base=10000.0)
    clean = csattn.qk_norm_rope(q, k, *w, **kw)
    grads = csattn.qk_norm_rope_bwd(*dy, q, k, *w, **kw)
    q[0, 1, 3] = 0
    got = csattn.qk_norm_rope(q, k, *w, **kw)
    back = csattn.qk_norm_rope_bwd(*dy, q, k, *w, **kw)
    csattn.check_status()
    assert torch.isnan(got[0][0, 1, 3]).all() and torch.isnan(back[0][0, 1, 3]).all()
    assert torch.isnan(back[2]).all()
    got[0][0, 1, 3], back[0][0, 1, 3] = clean[0][0, 1, 3], grads[0][0, 1, 3]
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    assert torch.equal(back[0], grads[0]) and torch.equal(back[1], grads[1])
    assert torch.equal(back[3], grads[3])


def test_gains_gradients_over_many_rows_per_thread():
    """Equal terms, whose roundings into one fp32 sum all go the same way (over 2300 rows in a
    thread: 2^-15 of the sum and more).  Here a thread adds at most 127 of them in fp32, then 4 steps
    of lanes' and 4 warps' sums are added, and 15 and 32 of the blocks': 2^-24 of the sum each,
    2^-16.5 in all, and the terms' 2^-18."""
    T, H, d = 1 << 20, 64, 16
    c = 1 + 2.0 ** -14 - 2.0 ** -20
    x = torch.ones(d, device=dev())
    q, k = x.expand(1, H, T, d), x.expand(1, 1, T, d)
    dy = [torch.full((1, h, T, d), c, device=dev()) for h in (H, 1)]
    grads = csattn.qk_norm_rope_bwd(*dy, q, k, x, x, eps=0.0)
    csattn.check_status()
    for h, dw in zip((H, 1), grads[2:]):
        want = float(np.float32(c)) * h * T
        assert np.abs(np64(dw) / want - 1).max() <= 2.0 ** -16


def test_many_rows_per_thread_parity():
    """Gradients of random rows where threads have over 1100 each, the last ones fewer."""
    T, H, d = (1 << 19) + 13, 63, 16
    x, xk = (torch.randn(T, d, generator=gen(s)).to(dev()) for s in (1, 2))
    w = [(1 + 0.3 * torch.randn(d, generator=gen(3))).to(dev()) for _ in range(2)]
    dy = [torch.randn(1, h, T, d, device=dev(), generator=torch.Generator(dev()).manual_seed(h))
          for h in (H, 1)]
    got = csattn.qk_norm_rope_bwd(*dy, x.expand(1, H, T, d), xk.expand(1, 1, T, d), *w, eps=1e-6)
    csattn.check_status()
    for i, (a, g) in enumerate(zip((x, xk), dy)):
        n = a.double() / (a.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
        want, size = torch.zeros(d, dtype=torch.float64, device=dev()), 0.0
        for h in range(g.shape[1]):
            gn = g[0, h].double() * n
            want += gn.sum(0)
            size = size + gn.abs().sum(0)
        assert ((got[2 + i].double() - want).abs() <= 2.0 ** -16 * size).all()
        for h in {0, g.shape[1] // 2, g.shape[1] - 1}:
            rx, _ = OS.qk_norm_rope_bwd(np64(g[:, h:h + 1]), np64(a)[None, None], np64(w[i]),
                                        np.zeros((1, T)), 1e-6, 0.0, "split_half")
            r = 1 / np.sqrt((np64(a) ** 2).mean(-1, keepdims=True) + 1e-6)
            gw = np.abs(np64(g[0, h]) * np64(w[i]))
            tol = 2.0 ** -18 * r * (gw + np64(n.abs()) * (gw * np64(n.abs())).mean(-1, keepdims=True))
            within(got[i][:, h:h + 1], rx, tol[None, None], "qk"[i])
