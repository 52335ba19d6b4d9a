"""The 4-bit cache as it is written and read: exactly the nearest values of the format, wherever
rows go, and nothing else."""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import step as OS
from tests import fp4_helpers as H
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def same_cache(a, b):
    return all(torch.equal(a[n], b[n]) for n in H.NAMES)


@pytest.mark.parametrize("d,Hkv,Tn,page", [
    (128, 8, 1, 0), (128, 2, 37, 0), (64, 3, 37, 0), (64, 1, 1, 16), (128, 3, 100, 16),
    (64, 12, 65, 32), (128, 1, 130, 64), (64, 2, 33, 192)])
def test_append_stores_the_nearest_values(d, Hkv, Tn, page):
    """Bit for bit, at rows that begin inside pages; the rest of the cache stays as it was."""
    B, held = 3, [0, 5, 61]
    c = H.empty_cache(B, Hkv, 70 + Tn, d, page, seed=Tn)
    kn, vn = (H.tokens(c, B * Tn, Hkv, d, s).view(B, Tn, Hkv, d).transpose(1, 2).contiguous()
              for s in (1, 2))
    cd = H.to_dev(c)
    H.append(cd, kn.to(dev()), vn.to(dev()), H.i32(held))
    csattn.check_status()
    for b in range(B):
        H.set_rows(c, b, held[b], kn[b], vn[b])
    assert same_cache(H.to_cpu(cd), c)


@pytest.mark.parametrize("d,Hkv,N,page,fused", [
    (128, 8, 64, 64, True), (64, 3, 1, 16, True), (128, 1, 77, 16, False), (64, 12, 33, 128, True)])
def test_append_to_slots(d, Hkv, N, page, fused):
    """Tokens in any order, some without a slot; keys and values may be parts of wider rows."""
    c = H.empty_cache(1, Hkv, N + 3 * page, d, page, seed=N, spare=1)
    n = c["k"].shape[0]
    g = H.gen(N)
    slots = torch.randperm(n * page, generator=g)[:N]
    slots[::5] = -1
    if N > 1:
        slots[1] = n * page - 1
        slots[2:][slots[2:] == n * page - 1] = -7
    kn, vn = H.tokens(c, N, Hkv, d, 3), H.tokens(c, N, Hkv, d, 4)
    if fused:
        both = torch.cat([torch.zeros(N, 1, d, dtype=torch.bfloat16), kn, vn], 1).to(dev())
        k, v = both[:, 1:1 + Hkv], both[:, 1 + Hkv:]
    else:
        k, v = kn.to(dev()), vn.transpose(0, 1).contiguous().to(dev()).transpose(0, 1)
    cd = H.to_dev(c)
    csattn.cache_append_fp4_slots(k, v, *H.cache(cd), slots.to(dev()))
    csattn.check_status()
    for name, x in (("k", kn), ("v", vn)):
        data, code, _ = OS.quantise_fp4(x.double().numpy())
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                c[name][s // page, :, s % page] = torch.from_numpy(data[i])
                c[name + "s"][s // page, :, s % page] = torch.from_numpy(code[i])
    assert same_cache(H.to_cpu(cd), c)


@pytest.mark.parametrize("d,Hkv,N,page", [(128, 5, 9001, 64), (64, 12, 5003, 16), (64, 7, 100, 32),
                                          (128, 1, 4097, 128), (64, 131, 700, 64)])
@pytest.mark.parametrize("fused", [False, True])
def test_append_to_many_slots(d, Hkv, N, page, fused):
    """The same rows as the append of one sequence to pages of that order."""
    g = H.gen(N)
    per = -(-N // page)
    table = torch.randperm(per + 3, generator=g)[:per].to(torch.int32).to(dev())
    at = torch.arange(N, device=dev())
    slots = table.long()[at // page] * page + at % page
    x = torch.randn(N, 3 * Hkv, d, generator=g).to(torch.bfloat16).to(dev())
    k, v = x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    new = [torch.full((per + 3, Hkv, page, n), 9, dtype=torch.uint8, device=dev())
           for n in (d // 2, d // 2, d // 16, d // 16)]
    want = [t.clone() for t in new]
    csattn.cache_append_fp4_slots(k, v, *new, slots)
    csattn.cache_append_fp4_paged(*(t.transpose(0, 1)[None].contiguous() for t in (k, v)), *want,
                                  table[None], H.i32([0]))
    csattn.check_status()
    for a, b in zip(new, want):
        assert torch.equal(a, b)


def test_append_every_magnitude():
    """Blocks that begin with every finite bf16 magnitude, beside fractions of it on and next to
    the borders between codes; infinities and NaN."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    top = (bits << 16).view(torch.float32).double()
    f = torch.tensor([1, -1 / 12, 1 / 12, 0.125, -0.25, 7 / 24, 5 / 12, 7 / 12, 5 / 6, -5 / 6,
                      0.0, -0.0, 0.9, 0.4, -0.03, 1 / 3], dtype=torch.float64)
    x = (top[:, None] * f).to(torch.bfloat16)           # [32640, 16]
    rows = x.view(-1, 1, 128)                           # tokens of one head
    odd = torch.randn(4, 1, 128, generator=H.gen(3)).to(torch.bfloat16)
    odd[0, 0, 5], odd[1, 0, 127], odd[2, 0, 64] = float("inf"), float("nan"), -float("inf")
    rows = torch.cat([rows, odd]).transpose(0, 1)[None].contiguous()  # [1, 1, n, 128]
    n = rows.shape[2]
    c = H.to_dev(H.empty_cache(1, 1, n, 128, 0, seed=1))
    H.append(c, rows.to(dev()), rows.flip(2).contiguous().to(dev()), H.i32([0]))
    ko, vo = H.read(c, H.i32([n]))
    csattn.check_status()
    data, code, want = OS.quantise_fp4(rows.double().numpy())
    assert np.array_equal(c["k"].cpu().numpy(), data)
    assert np.array_equal(c["ks"].cpu().numpy(), code)
    assert np.array_equal(c["v"].cpu().numpy(), data[:, :, ::-1])
    assert np.array_equal(ko.double().cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(vo.double().cpu().numpy(), want[:, :, ::-1], equal_nan=True)


def test_read_every_byte():
    """All pairs of codes with all scale bytes that are written."""
    d, n = 64, 227
    k = torch.arange(256, dtype=torch.uint8).repeat_interleave(1)[None, :, None].expand(n, 256, d // 2)
    k = k.transpose(0, 1).contiguous()[None].view(1, 256, n, d // 2)
    ks = torch.arange(n, dtype=torch.uint8)[None, None, :, None].expand(1, 256, n, 4).contiguous()
    ks[0, 0, :, 1] = 255
    v, vs = k.flip(1).contiguous(), ks.flip(2).contiguous()
    ko, vo = csattn.cache_read_fp4(*(t.to(dev()) for t in (k, v, ks, vs)), H.i32([n]))
    csattn.check_status()
    for got, x, s in ((ko, k, ks), (vo, v, vs)):
        assert np.array_equal(got.double().cpu().numpy(), OS.fp4_values(x.numpy(), s.numpy()),
                              equal_nan=True)


@pytest.mark.parametrize("B,Hkv,d,page,Lout", [(3, 4, 128, 0, 150), (2, 3, 64, 16, 100),
                                               (1, 1, 128, 64, 200), (2, 2, 64, 0, 77)])
def test_read_back_is_exact_and_leaves_the_rest(B, Hkv, d, page, Lout):
    lens = [0, Lout, 33][-B:]
    c, _ = H.filled(B, Hkv, Hkv, d, page, lens, 210, seed=B)
    out = [torch.full((B, Hkv, Lout, d), 7.0, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    got = H.read(H.to_dev(c), H.i32(lens), *out)
    csattn.check_status()
    assert got[0] is out[0] and got[1] is out[1]
    for b, n in enumerate(lens):
        for o, want in zip(out, H.rows(c, b, n) if n else (None, None)):
            if n:
                assert np.array_equal(o[b, :, :n].double().cpu().numpy(), want)
            assert torch.all(o[b, :, n:] == 7.0)


def test_device_side_refusals():
    B, Hkv, d, page = 3, 2, 64, 16
    c = H.to_dev(H.empty_cache(B, Hkv, 64, d, page, seed=1))
    x = H.tokens(c, B * 8, Hkv, d, 1).view(B, 8, Hkv, d).transpose(1, 2).contiguous().to(dev())
    before = {n: c[n].clone() for n in H.NAMES}
    for lens in ([-1, 57, 2 ** 31 - 1], [-2 ** 31, 64, 100]):
        H.append(c, x, x, H.i32(lens))
        H.refused()
        assert all(torch.equal(c[n], before[n]) for n in H.NAMES)
    # a page outside the pool: its rows are not written, others are
    good = c["table"].clone()
    c["table"][1, 0] = c["k"].shape[0]
    c["table"][2, 0] = -1
    H.append(c, x, x, H.i32([0, 12, 8]))
    H.refused()
    p = int(good[1, 1])
    touched = set(torch.nonzero((c["k"] != before["k"]).flatten(1).any(1)).flatten().tolist())
    assert touched == {int(good[0, 0]), p}
    assert torch.all((c["k"][p] != before["k"][p]).flatten(2).any(2).any(0)
                     == (torch.arange(16, device=dev()) < 4))
    # slots past the pool
    before = {n: c[n].clone() for n in H.NAMES}
    n = c["k"].shape[0] * page
    t = x.transpose(1, 2).reshape(-1, Hkv, d)[:4]
    bad = torch.tensor([n, n + 5, 2 ** 40, 2 ** 63 - 1], device=dev())
    csattn.cache_append_fp4_slots(t, t, *H.cache(c), bad)
    H.refused()
    csattn.cache_append_fp4_slots(t, t, *H.cache(c), -bad)
    csattn.check_status()
    assert all(torch.equal(c[n], before[n]) for n in H.NAMES)
    # reading
    c["table"].copy_(good)
    c["table"][0, 1] = -3
    out = [torch.full((B, Hkv, 40, d), 7.0, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    H.read(c, H.i32([32, -1, 41]), *out)
    H.refused()
    for o in out:
        assert torch.all(o[0, :, 16:32] == 0) and torch.all(o[0, :, 32:] == 7)
        assert torch.all(o[1:] == 7)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: the last page's rows are written, read and attended."""
    Hkv, d, page = 1, 128, 64
    n = (1 << 32) // (d // 2 * page) + 3
    k = torch.zeros(n, Hkv, page, d // 2, dtype=torch.uint8, device=dev())
    ks = torch.zeros(n, Hkv, page, d // 16, dtype=torch.uint8, device=dev())
    c = {"k": k, "v": k.clone(), "ks": ks, "vs": ks.clone(), "table": H.i32([[n - 1]]), "page": page}
    x = H.tokens(c, 50, Hkv, d, 9)
    xd = x.to(dev())
    slots = (n - 1) * page + torch.arange(50, device=dev())
    csattn.cache_append_fp4_slots(xd, xd, *H.cache(c), slots)
    _, _, want = OS.quantise_fp4(x.double().numpy())
    ko, vo = H.read(c, H.i32([50]))
    q = torch.randn(1, 4, 1, d, generator=H.gen(4)).to(torch.bfloat16)
    out = H.decode(c, q.to(dev()), H.i32([50]))
    csattn.check_status()
    assert np.array_equal(ko[0, 0, :50].double().cpu().numpy(), want[:, 0])
    assert torch.equal(ko[:, :, :50], vo[:, :, :50])
    small = {name: c[name][n - 1:].cpu() for name in H.NAMES}
    small.update(table=torch.zeros(1, 1, dtype=torch.int32), page=page)
    H.assert_close(out, H.expect(small, q, [50]))


def test_python_refusals():
    c = H.to_dev(H.empty_cache(2, 2, 32, 64, 16, seed=1))
    x = torch.zeros(2, 2, 4, 64, dtype=torch.bfloat16, device=dev())
    lens, t = H.i32([0, 0]), x[:, :, 0].contiguous()
    slots = torch.zeros(2, dtype=torch.int64, device=dev())
    k, v, ks, vs = H.cache(c)
    for bad, kind in [
            (lambda: csattn.cache_append_fp4_paged(x.float(), x, k, v, ks, vs, c["table"], lens), TypeError),
            (lambda: csattn.cache_append_fp4_paged(x, x[:1], k, v, ks, vs, c["table"], lens), ValueError),
            (lambda: csattn.cache_append_fp4_paged(x, x, k, v, ks[..., :2], vs, c["table"], lens), ValueError),
            (lambda: csattn.cache_append_fp4_paged(x, x, k, v[:, :1], ks, vs, c["table"], lens), ValueError),
            (lambda: csattn.cache_append_fp4_paged(x, x, k, v, ks, vs, c["table"].long(), lens), TypeError),
            (lambda: csattn.cache_append_fp4_paged(x, x, k, v, ks, vs, c["table"], lens[:1]), ValueError),
            (lambda: csattn.cache_append_fp4(x, x, k, v, ks, vs, lens), ValueError),
            (lambda: csattn.cache_append_fp4_slots(t, t, k, v, ks, vs, slots.int()), TypeError),
            (lambda: csattn.cache_append_fp4_slots(t[..., :32], t, k, v, ks, vs, slots), ValueError),
            (lambda: csattn.cache_append_fp4_slots(x.transpose(2, 3)[:, :, 0], t, k, v, ks, vs, slots), ValueError),
            (lambda: csattn.cache_read_fp4_paged(k, v, ks, vs, c["table"], lens, x), ValueError),
            (lambda: csattn.attn_decode_fp4_paged(x, k, v, ks, vs, c["table"], lens), ValueError)]:
        with pytest.raises(kind):
            bad()
    # rows that are not a multiple of 16 bytes apart: refused by the library
    wide = torch.zeros(2, 2, 68, dtype=torch.bfloat16, device=dev())[..., :64]
    with pytest.raises(csattn.CsattnError) as e:
        csattn.cache_append_fp4_slots(wide, wide, k, v, ks, vs, slots)
    assert e.value.status == -1
    csattn.check_status()
