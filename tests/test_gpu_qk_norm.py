"""Norm of queries and keys with the rotation, and its gradients, against float64 and against
differences.

Tolerances, with L the length of a channel's pair ahead of the rotation (the channel's magnitude
without one), all operations between load and store in fp32 (2^-24 each):
  forward   2^-19 L: at most 24 additions of squares (half of their error in the root), rsqrt (2^-22),
            three products, the sine and cosine (2^-22 each);
  dx        2^-18 of r (Lg |w| + |n| mean |g w n|), Lg the length of the gradient's pair: as above
            twice;
  dw        2^-16 of sum |g n|: chains of at most 64 additions in a thread here, 5 + 2 in a block, and
            of a few in the second pass, each of 2^-24 of the sum at most, and the terms' 2^-18;
and for bf16 the stored value's rounding, 2^-8 of it, or of a subnormal one half a step of 2^-133.
"""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import step as OS
from tests.fp4_helpers import gen, i32, refused
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu
EPS = 1e-6


def pair_lengths(x, base, layout):
    if base <= 0:
        return np.abs(x)
    if layout == "split_half":
        return np.tile(np.hypot(*np.split(x, 2, -1)), 2)
    return np.repeat(np.hypot(x[..., 0::2], x[..., 1::2]), 2, -1)


def case(B, Hq, Hkv, T, d, dtype, fused, seed, gains=True):
    """Inputs on the device: q, k (parts of one tensor if fused), gains, the outputs' gradients."""
    g = gen(seed)
    if fused:
        x = torch.randn(B, T, Hq + 2 * Hkv, d, generator=g).to(dtype).to(dev())
        q, k = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv)))
    else:
        q, k = (torch.randn(B, H, T, d, generator=g).to(dtype).to(dev()) for H in (Hq, Hkv))
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype).to(dev()) if gains else None
         for _ in range(2)]
    dy = [torch.randn(B, H, T, d, generator=g).to(dtype).to(dev()) for H in (Hq, Hkv)]
    return q, k, w, dy


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def within(got, want, tol, what):
    off = np.abs(np64(got) - want)
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8 + 2.0 ** -134
    assert np.all(off <= tol), (what, float((off / np.maximum(tol, 1e-300)).max()))


def check(q, k, w, dy, positions, base, layout, norm=True, pos0=0, dxs=(None, None)):
    B, _, T, d = q.shape
    kw = dict(norm=norm, eps=EPS, rope_base=base, rope_layout=layout, pos0=pos0)
    out = csattn.qk_norm_rope(q, k, *w, positions, **kw)
    grads = csattn.qk_norm_rope_bwd(*dy, q, k, *w, positions, *dxs, **kw)
    csattn.check_status()
    pos = (np.tile(pos0 + np.arange(T), (B, 1)) if positions is None
           else positions.cpu().numpy())
    args = (pos, EPS, base, layout, norm)
    for i, (x, y, dx, dw) in enumerate(zip((q, k), out, grads[:2], grads[2:])):
        what = "qk"[i]
        assert y.is_contiguous() and y.shape == x.shape
        xn, wn, dyn = np64(x), np64(w[i]), np64(dy[i])
        flat = OS.qk_norm_rope(xn, wn, pos, EPS, 0.0, layout, norm)
        within(y, OS.qk_norm_rope(xn, wn, *args), 2.0 ** -19 * pair_lengths(flat, base, layout),
               what)
        rx, rw = OS.qk_norm_rope_bwd(dyn, xn, wn, *args)
        lg = pair_lengths(dyn, base, layout)
        if not norm:
            within(dx, rx, 2.0 ** -19 * lg, "d" + what)
            assert dw is None
            continue
        r = 1 / np.sqrt((xn * xn).mean(-1, keepdims=True) + EPS)
        n, a = xn * r, 1.0 if wn is None else np.abs(wn)
        g = OS._turn(dyn, pos, base, layout, back=True)
        size = r * (lg * a + np.abs(n) * np.mean(np.abs(g * a * n), -1, keepdims=True))
        within(dx, rx, 2.0 ** -18 * size, "d" + what)
        if wn is None:
            assert dw is None
        else:
            assert dw.dtype == torch.float32
            within(dw, rw, 2.0 ** -16 * (lg * np.abs(n)).sum((0, 1, 2)), "d" + what + "w")
    return out, grads


@pytest.mark.parametrize("B,Hq,Hkv,T,d,dtype,base,layout,fused,places", [
    (2, 8, 2, 37, 128, torch.bfloat16, 10000.0, "split_half", True, False),
    (2, 8, 2, 37, 128, torch.bfloat16, 10000.0, "adjacent", True, True),
    (64, 32, 8, 1, 128, torch.bfloat16, 500000.0, "split_half", True, True),
    (1, 1, 1, 1, 64, torch.bfloat16, 10000.0, "split_half", False, False),
    (3, 7, 1, 19, 64, torch.bfloat16, 10000.0, "adjacent", False, True),
    (1, 12, 12, 200, 64, torch.bfloat16, 0.0, "split_half", True, False),
    (2, 6, 3, 33, 128, torch.float32, 10000.0, "split_half", True, True),
    (2, 5, 5, 17, 64, torch.float32, 10000.0, "adjacent", False, False),
    (3, 2, 1, 11, 32, torch.float32, 100.0, "split_half", True, False),
    (3, 3, 1, 9, 16, torch.float32, 10000.0, "adjacent", True, True),
    (1, 4, 2, 5, 16, torch.float32, 1.0, "split_half", False, False),
    (5, 40, 4, 700, 128, torch.bfloat16, 10000.0, "split_half", True, False),
    (2, 13, 11, 1000, 64, torch.float32, 10000.0, "split_half", False, False)])
def test_parity(B, Hq, Hkv, T, d, dtype, base, layout, fused, places):
    q, k, w, dy = case(B, Hq, Hkv, T, d, dtype, fused, seed=T)
    positions = None
    if places:
        positions = torch.randint(0, 40000, (B, T), generator=gen(1)).to(torch.int32).to(dev())
    check(q, k, w, dy, positions, base, layout)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_without_gains_and_without_the_norm(dtype):
    q, k, w, dy = case(2, 4, 2, 21, 64, dtype, True, seed=1, gains=False)
    check(q, k, w, dy, None, 10000.0, "split_half", pos0=100)
    check(q, k, w, dy, None, 10000.0, "adjacent", norm=False, pos0=7)
    check(q, k, w, dy, None, 0.0, "split_half", norm=False)
    half = [torch.ones(64, dtype=dtype, device=dev()), None]
    check(q, k, half, dy, None, 10000.0, "split_half")
    check(q, k, half[::-1], dy, None, 10000.0, "split_half")


@pytest.mark.parametrize("layout", ["split_half", "adjacent"])
def test_far_positions(layout):
    """Up to the last that is accepted."""
    top = (1 << 24) - 1
    pos = i32([[0, 1, 49151, 49152, 1 << 20, top - 1, top]])
    q, k, w, dy = case(1, 2, 1, 7, 128, torch.float32, False, seed=4)
    for base in (1.0, 10000.0, 1e8):
        check(q, k, w, dy, pos, base, layout)
    check(q, k, w, dy, None, 10000.0, layout, pos0=(1 << 24) - 7)


def test_small_and_large_heads():
    """Zeros (eps alone decides), subnormals, and magnitudes far apart within a head."""
    q, k, w, dy = case(1, 4, 2, 8, 64, torch.bfloat16, False, seed=5)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -130
    q[0, 2] *= 2.0 ** 50
    q[0, 3, :, ::3] *= 2.0 ** -20
    k[0, 0] *= 2.0 ** -12
    out, grads = check(q, k, w, dy, None, 10000.0, "split_half")
    assert torch.all(out[0][0, 0] == 0)


def test_not_finite_stays_in_its_head():
    q, k, w, dy = case(1, 4, 2, 8, 64, torch.bfloat16, False, seed=5)
    clean = csattn.qk_norm_rope(q, k, *w, rope_base=10000.0)
    q[0, 1, 3, 7], k[0, 1, 2, 0] = float("nan"), float("inf")
    got = csattn.qk_norm_rope(q, k, *w, rope_base=10000.0)
    csattn.check_status()
    assert torch.isnan(got[0][0, 1, 3]).all() and torch.isnan(got[1][0, 1, 2]).any()
    got[0][0, 1, 3], got[1][0, 1, 2] = clean[0][0, 1, 3], clean[1][0, 1, 2]
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


def test_gradients_against_differences():
    """Of the kernel's own fp32 outputs: a central difference along a direction, whose error is a
    third derivative's h^2 / 6 and the outputs' roundings (2^-19 of about 1 each, of 3000 at
    random) over 2h."""
    q, k, w, dy = case(1, 3, 1, 5, 64, torch.float32, False, seed=9)
    kw = dict(eps=1e-3, rope_base=100.0)
    dq, dk, dqw, dkw = csattn.qk_norm_rope_bwd(*dy, q, k, *w, **kw)

    def f(q, k, w):
        y = csattn.qk_norm_rope(q, k, *w, **kw)
        return sum((a.double() * b.double()).sum().item() for a, b in zip(y, dy))

    g = gen(10)
    u = [torch.randn(t.shape, generator=g).to(dev()) for t in (q, k, *w)]
    h = 2.0 ** -8
    for i in range(4):
        s = [0.0] * 4
        s[i] = h
        ends = [f(q + a * s[0] * u[0], k + a * s[1] * u[1],
                  [w[0] + a * s[2] * u[2], w[1] + a * s[3] * u[3]]) for a in (1, -1)]
        want = ((dq, dk, dqw, dkw)[i].double() * u[i].double()).sum().item()
        assert abs((ends[0] - ends[1]) / (2 * h) - want) <= 2e-3 * max(1.0, abs(want)) + 0.02


def test_into_a_fused_gradient_and_the_same_bits_twice():
    """dq and dk as parts of the projection's gradient, whose other rows stay as they were."""
    B, Hq, Hkv, T, d = 3, 8, 2, 45, 128
    q, k, w, dy = case(B, Hq, Hkv, T, d, torch.bfloat16, True, seed=3)
    bufs = []
    for _ in range(2):
        x = torch.full((B, T, Hq + 2 * Hkv, d), 7.0, dtype=torch.bfloat16, device=dev())
        dxs = [x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv))]
        _, grads = check(q, k, w, dy, None, 10000.0, "split_half", dxs=dxs)
        assert grads[0] is dxs[0] and grads[1] is dxs[1]
        bufs.append((x, grads[2], grads[3]))
    assert torch.all(bufs[0][0][:, :, Hq + Hkv:] == 7.0)
    for a, b in zip(*bufs):
        assert torch.equal(a, b)


def test_positions_out_of_range():
    q, k, w, dy = case(1, 2, 1, 4, 64, torch.bfloat16, False, seed=3)
    good = csattn.qk_norm_rope(q, k, *w, i32([[5, 0, 9, 11]]), rope_base=10000.0)
    csattn.check_status()
    for bad in (-1, 1 << 24, 2 ** 31 - 1, -2 ** 31):
        pos = i32([[5, bad, 9, 11]])
        got = csattn.qk_norm_rope(q, k, *w, pos, rope_base=10000.0)
        refused()
        assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
        csattn.qk_norm_rope_bwd(*dy, q, k, *w, pos, rope_base=10000.0)
        refused()


def test_capture_and_streams():
    """Both directions captured and replayed over other inputs in the same buffers, and on another
    stream beside the current one; eager calls between the replays."""
    q, k, w, dy = case(4, 8, 2, 30, 128, torch.bfloat16, True, seed=6)
    pos = torch.randint(0, 9000, (4, 30), generator=gen(2)).to(torch.int32).to(dev())
    kw = dict(rope_base=10000.0)

    def run(**more):
        return [*csattn.qk_norm_rope(q, k, *w, pos, **kw, **more),
                *csattn.qk_norm_rope_bwd(*dy, q, k, *w, pos, **kw, **more)]

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = run()
        graphs.append((gr, o))
    q.mul_(0.5)
    dy[0].mul_(-1)
    w[1].add_(1)
    want = run()
    for gr, o in graphs:
        gr.replay()
        run()
    torch.cuda.synchronize()
    csattn.check_status()
    for _, o in graphs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_python_refusals():
    q, k, w, dy = case(2, 4, 2, 5, 64, torch.bfloat16, False, seed=1)
    fn, bwd = csattn.qk_norm_rope, csattn.qk_norm_rope_bwd
    for bad, kind in [
            (lambda: fn(q.half(), k.half()), TypeError), (lambda: fn(q, k.float()), TypeError),
            (lambda: fn(q, k[:1]), ValueError), (lambda: fn(q, k[..., :32]), ValueError),
            (lambda: fn(q[0], k[0]), ValueError), (lambda: fn(q, k, w[0].float()), TypeError),
            (lambda: fn(q, k, w[0][:32]), ValueError),
            (lambda: fn(q, k, positions=torch.zeros(2, 5, device=dev())), TypeError),
            (lambda: fn(q, k, positions=i32([[0] * 4] * 2)), ValueError),
            (lambda: fn(q.transpose(2, 3)[:, :, :5, :5], k), ValueError),
            (lambda: fn(q, k, w[0], norm=False), csattn.CsattnError),
            (lambda: fn(q, k, rope_base=0.5), csattn.CsattnError),
            (lambda: fn(q, k, rope_layout="other"), KeyError),
            (lambda: bwd(dy[0].transpose(1, 2).contiguous().transpose(1, 2), dy[1], q, k), ValueError),
            (lambda: bwd(*dy, q, k, dq=q[:, :, :1].expand(-1, -1, 5, -1)), ValueError),
            (lambda: bwd(*dy, q, k, dq_weight=torch.zeros(64, device=dev())), ValueError),
            (lambda: bwd(*dy, q, k, *w, workspace=torch.zeros(64, device=dev())), csattn.CsattnError)]:
        with pytest.raises(kind):
            bad()
    csattn.check_status()
