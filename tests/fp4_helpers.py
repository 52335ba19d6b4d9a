"""Inputs and expected values of the 4-bit cache tests."""
import numpy as np
import torch

import transformer_causal_self_gb300 as csattn
from oracle import step as OS
from tests.fp8_helpers import gen, i32, place, to_cpu, to_dev  # noqa: F401
from tests.gpu_helpers import dev

NAMES = ("k", "v", "ks", "vs")


def empty_cache(B, Hkv, rows, d, page, seed, spare=2):
    """A cache on the CPU whose every row is garbage (any values, NaN scales) with a shuffled block
    table (None: contiguous): dict(k, v, ks, vs, table, page)."""
    g = gen(seed)
    if page:
        per = -(-rows // page)
        n = B * per + spare
        table = torch.randperm(n, generator=g)[:B * per].to(torch.int32).view(B, per).contiguous()
        shape = (n, Hkv, page)
    else:
        table, shape = None, (B, Hkv, rows)
    c = {"table": table, "page": page}
    for n in ("k", "v"):
        c[n] = torch.randint(0, 256, (*shape, d // 2), generator=g, dtype=torch.uint8)
        c[n + "s"] = torch.full((*shape, d // 16), 255, dtype=torch.uint8)
    return c


def set_rows(c, b, r0, k, v):
    """Rows r0.. of sequence b from k, v [Hkv, n, d], quantised."""
    for name, x in (("k", k), ("v", v)):
        data, code, _ = OS.quantise_fp4(x.double().numpy())
        for i in range(x.shape[1]):
            p, o = place(c, b, r0 + i)
            c[name][p, :, o] = torch.from_numpy(data[:, i])
            c[name + "s"][p, :, o] = torch.from_numpy(code[:, i])


def rows(c, b, n):
    """Rows 0..n-1 of sequence b in float64: (k, v) [Hkv, n, d]."""
    at = [place(c, b, r) for r in range(n)]
    p, o = [a[0] for a in at], [a[1] for a in at]
    return [np.swapaxes(OS.fp4_values(c[n][p, :, o].numpy(), c[n + "s"][p, :, o].numpy()), 0, 1)
            for n in ("k", "v")]


def cache(c):
    return c["k"], c["v"], c["ks"], c["vs"]


def append(c, kn, vn, lens, **kw):
    if c["table"] is None:
        csattn.cache_append_fp4(kn, vn, *cache(c), lens, **kw)
    else:
        csattn.cache_append_fp4_paged(kn, vn, *cache(c), c["table"], lens, **kw)


def read(c, lens, *out, **kw):
    if c["table"] is None:
        return csattn.cache_read_fp4(*cache(c), lens, *out, **kw)
    return csattn.cache_read_fp4_paged(*cache(c), c["table"], lens, *out, **kw)


def decode(c, q, lens, **kw):
    if c["table"] is None:
        return csattn.attn_decode_fp4(q, *cache(c), lens, **kw)
    return csattn.attn_decode_fp4_paged(q, *cache(c), c["table"], lens, **kw)


def refused():
    import pytest
    with pytest.raises(csattn.CsattnError) as e:
        csattn.check_status()
    assert e.value.status == -6


def expect(c, q, lens, scale=None):
    """The decode in float64, out [B, Hq, 1, d], and how far a kernel's output may be from it.

    With p the weights and A = sum p |v|: the output's rounding is 2^-8 of it (2^-133 where it is
    subnormal), the weights' 2^-11 each, of A in all, and 2^-33 of the largest for those that
    vanish.  A score's fp32 sum is off by at most 2^-17 of sum |q_i k_i| (d products, added in
    groups of 16), which moves a weight relatively by as much as the score, and the sum of the
    weights again; 2^-18 for the exponentials.
    """
    B, Hq, _, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out, tol = np.zeros((B, Hq, 1, d)), np.zeros((B, Hq, 1, d))
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        k, v = rows(c, b, n)
        rep = Hq // k.shape[0]
        x = q[b, :, 0].double().numpy().reshape(k.shape[0], rep, d)
        s = np.einsum("grd,gnd->grn", x, k) * scale
        off = np.einsum("grd,gnd->grn", np.abs(x), np.abs(k)).max(-1) * scale * 2.0 ** -17
        p = np.exp(s - s.max(-1, keepdims=True))
        total = p.sum(-1, keepdims=True)
        p /= total
        o = np.einsum("grn,gnd->grd", p, v)
        a = np.einsum("grn,gnd->grd", p, np.abs(v))
        lost = 2.0 ** -33 / total * np.abs(v).sum(1)[:, None]
        out[b, :, 0] = o.reshape(Hq, d)
        tol[b, :, 0] = (a * (2.0 ** -11 + 2 * off[..., None] + 2.0 ** -18) + lost
                        + np.abs(o) * 2.0 ** -8 + 2.0 ** -133).reshape(Hq, d) * (1 + 2.0 ** -7)
    return out, tol


def assert_close(got, ref, what=""):
    out, tol = ref
    off = np.abs(got.double().cpu().numpy() - out)
    assert np.all(off <= tol), (what, float((off / np.maximum(tol, 1e-300)).max()))


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def filled(B, Hq, Hkv, d, page, lens, room, seed, gain=1.0):
    """A cache of random rows (garbage behind each length) and queries, on the CPU."""
    g = gen(seed)
    c = empty_cache(B, Hkv, room, d, page, seed)
    for b, n in enumerate(lens):
        if n > 0:
            k, v = (torch.randn(Hkv, n, d, generator=g) for _ in range(2))
            v = v * torch.exp(torch.randn(Hkv, n, 1, generator=g))
            set_rows(c, b, 0, k.to(torch.bfloat16), v.to(torch.bfloat16))
    return c, (gain * torch.randn(B, Hq, 1, d, generator=g)).to(torch.bfloat16)


def tokens(c, n, Hkv, d, seed):
    """n keys or values with blocks of very different sizes, ties and zeros among them."""
    g = gen(seed)
    x = torch.randn(n, Hkv, d, generator=g) * torch.exp(2 * torch.randn(n, Hkv, 1, generator=g))
    x[..., :16] = torch.round(4 * x[..., :16]) / 4
    x[..., 16] = 0.0
    return x.to(torch.bfloat16)
