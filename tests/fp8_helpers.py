"""Inputs and expected values of the 8-bit cache and token-tree tests."""
import numpy as np
import torch

from oracle import attn as OA
from tests.gpu_helpers import dev


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def round_query(x, e4m3):
    """The rotated query as the products take it: bf16, or 11 significant bits with an 8-bit
    cache (float64 in and out)."""
    if not e4m3:
        return OA.round_to_bf16(x)
    m, e = np.frexp(x)
    return np.ldexp(np.round(np.ldexp(m, 11)), e - 11)


def values(k8, code):
    """What e4m3 rows and scale codes stand for, in float64."""
    return k8.float().cpu().double().numpy() * np.exp2(
        code.cpu().view(torch.uint8).numpy().astype(np.float64) - 127)[..., None]


def quantise(x, rotated_from=None):
    """Exact quantisation of rows x [..., d]: (e4m3 tensor, codes uint8).  rotated_from: the rows
    before their rotation, which set the scale."""
    e = OA.e4m3_exponents(x if rotated_from is None else rotated_from, rotated_from is not None)
    y, _ = OA.quantise_rows(x, e)
    return (torch.from_numpy(y).float().to(torch.float8_e4m3fn),
            torch.from_numpy((e + 127).astype(np.uint8)))


def empty_cache(B, Hkv, rows, d, page, e4m3, seed, spare=2):
    """A cache on the CPU whose every row is garbage (NaN values, NaN or odd scale codes) with a
    shuffled block table (None: contiguous): dict(k, v[, ks, vs], table, page)."""
    g = gen(seed)
    if page:
        per = -(-rows // page)
        n = B * per + spare
        table = torch.randperm(n, generator=g)[:B * per].to(torch.int32).view(B, per).contiguous()
        shape = (n, Hkv, page, d)
    else:
        table, shape = None, (B, Hkv, rows, d)
    c = {"table": table, "page": page}
    if e4m3:
        nan = torch.full(shape, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn)
        c.update(k=nan, v=nan.clone(), ks=torch.full(shape[:3], 255, dtype=torch.uint8),
                 vs=torch.full(shape[:3], 255, dtype=torch.uint8))
    else:
        nan = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        c.update(k=nan, v=nan.clone())
    return c


def raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def set_rows(c, b, r0, k, v):
    """Rows r0.. of sequence b from k, v [Hkv, n, d] (bf16 tensors; quantised for an 8-bit cache)."""
    new = {"k": k, "v": v}
    if "ks" in c:
        for n in ("k", "v"):
            q, code = quantise(new[n].double().numpy())
            new[n], new[n + "s"] = q, code
    for n, x in new.items():
        for i in range(k.shape[1]):
            p, o = place(c, b, r0 + i)
            raw(c[n])[p, :, o] = raw(x)[:, i]


def place(c, b, r):
    if c["table"] is None:
        return b, r
    return int(c["table"][b, r // c["page"]]), r % c["page"]


def rows(c, b, n):
    """Rows 0..n-1 of sequence b in float64: (k, v) [Hkv, n, d]."""
    at = [place(c, b, r) for r in range(n)]
    p, o = [a[0] for a in at], [a[1] for a in at]
    out = []
    for name in ("k", "v"):
        if name + "s" in c:
            x = values(raw(c[name])[p, :, o].view(torch.float8_e4m3fn), c[name + "s"][p, :, o])
        else:
            x = c[name][p, :, o].double().numpy()
        out.append(np.swapaxes(x, 0, 1))
    return out


def to_dev(c):
    return {n: (x.to(dev()) if isinstance(x, torch.Tensor) else x) for n, x in c.items()}


def to_cpu(c):
    return {n: (x.cpu() if isinstance(x, torch.Tensor) else x) for n, x in c.items()}


def scales(c):
    return {"k_scale": c["ks"], "v_scale": c["vs"]} if "ks" in c else {}


def same_bits(a, b):
    a, b = raw(a), raw(b)
    if a.dtype == torch.bfloat16:
        a, b = a.view(torch.int16), b.view(torch.int16)
    return torch.equal(a, b)
