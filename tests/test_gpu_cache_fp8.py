"""The 8-bit KV cache against float64: the quantising append, reading back, and decode.

Tolerances.  Reading back is exact.  A stored value is exact for v (bf16 in, one rounding);
a key is rounded from an fp32 rotation whose error is below 2^-20 of the pair's length
(angle reduction and __sincosf, 2^-21 each), so it may fall on the other side of a rounding
border: such a key is one e4m3 step away, 2^-3 of its value at most, and fewer than
1 in 1000 do (the border's width over a step's, 2^-20 / 2^-4, times the two sides).
A decode's output is bf16: it is held to the bounds of the bf16 decode (max-abs 2e-2, relative
L2 5e-3), which allow for the bf16 rounding of the output (2^-9); the weights' f16 rounding,
2^-11, is below it, and the query's 11 bits are the reference's, too.  Those bounds are for outputs below
4; test_decode_parity's values reach 8 |N(0,1)|, so outputs of 8 and more occur, whose storing in
bf16 alone costs half a step, 2^(e-8) for [2^e, 2^(e+1)): 2^-5 = 3.1e-2 at 8.  Its max-abs
bound is 2e-2 plus that half step of the largest expected output.
"""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import attn as OA
from tests import fp8_helpers as H
from tests.gpu_helpers import assert_bf16_close, dev, half_ulp_bf16, to_np

pytestmark = pytest.mark.gpu


def _append(c, kn, vn, lens, base, layout, stream=None):
    kw = dict(rope_base=base, rope_layout=layout, stream=stream)
    if c["table"] is None:
        csattn.cache_append_fp8(kn, vn, c["k"], c["v"], c["ks"], c["vs"], lens, **kw)
    else:
        csattn.cache_append_fp8_paged(kn, vn, c["k"], c["v"], c["ks"], c["vs"], c["table"], lens,
                                      **kw)


def _decode(c, q, lens, **kw):
    if c["table"] is None:
        return csattn.attn_decode_fp8(q, c["k"], c["v"], c["ks"], c["vs"], lens, **kw)
    return csattn.attn_decode_fp8_paged(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], lens,
                                        **kw)


def _read(c, lens, ko=None, vo=None):
    if c["table"] is None:
        return csattn.cache_read_fp8(c["k"], c["v"], c["ks"], c["vs"], lens, ko, vo)
    return csattn.cache_read_fp8_paged(c["k"], c["v"], c["ks"], c["vs"], c["table"], lens, ko, vo)


@pytest.mark.parametrize("d,Hkv,Tn,base,layout,page", [
    (128, 8, 300, 10000.0, "split_half", 0),
    (64, 2, 1, 500000.0, "adjacent", 16),
    (128, 3, 17, 0.0, "split_half", 64),
    (64, 5, 65, 10000.0, "split_half", 32),
    (128, 1, 33, 10000.0, "adjacent", 0),
])
def test_append_stores_the_rounded_rows(d, Hkv, Tn, base, layout, page):
    B, room = 3, 700
    lens = [0, 257, room - Tn]
    g = H.gen(d + Tn)
    kn = (torch.randn(B, Hkv, Tn, d, generator=g) * torch.exp2(
        torch.randint(-20, 20, (B, Hkv, Tn, 1), generator=g))).to(torch.bfloat16)
    vn = (torch.randn(B, Hkv, Tn, d, generator=g) * 0.1).to(torch.bfloat16)
    kn[0, 0, 0] = 0
    vn[0, 0, 0] = 0
    c = H.empty_cache(B, Hkv, room, d, page, True, seed=1)
    cd = H.to_dev(c)
    _append(cd, kn.to(dev()), vn.to(dev()), H.i32(lens), base, layout)
    csattn.check_status()
    got = H.to_cpu(cd)
    wrong = total = 0
    for b, L in enumerate(lens):
        k = kn[b].double().numpy()
        kr = OA.rope_rotate(k, L + np.arange(Tn), base, layout) if base > 0 else k
        ek, ev = OA.e4m3_exponents(k, base > 0), OA.e4m3_exponents(vn[b], False)
        k8, _ = OA.quantise_rows(kr, ek)
        v8, _ = OA.quantise_rows(vn[b].double().numpy(), ev)
        for t in range(Tn):
            p, o = H.place(c, b, L + t)
            assert np.array_equal(got["ks"][p, :, o].numpy(), ek[:, t] + 127)
            assert np.array_equal(got["vs"][p, :, o].numpy(), ev[:, t] + 127)
            assert np.array_equal(H.raw(got["v"])[p, :, o].view(torch.float8_e4m3fn).double(),
                                  v8[:, t])
            gk = H.raw(got["k"])[p, :, o].view(torch.float8_e4m3fn).double().numpy()
            off = gk != k8[:, t]
            wrong += int(off.sum())
            total += off.size
            assert np.all(np.abs(gk - k8[:, t]) <= np.maximum(np.abs(k8[:, t]) / 8, 2.0 ** -9))
            # written: nothing else is, below
            H.raw(got["k"])[p, :, o] = 0x7F
            H.raw(got["v"])[p, :, o] = 0x7F
            got["ks"][p, :, o] = 255
            got["vs"][p, :, o] = 255
    assert wrong <= 1e-3 * total, (wrong, total)
    for n in ("k", "v", "ks", "vs"):
        assert H.same_bits(got[n], c[n]), f"{n}: rows that are not the chunk's were written"


def test_append_extreme_and_non_finite_rows():
    """Largest and smallest bf16, scale limits, and rows with NaN or infinities: those are
    stored as NaN, and the others' scale comes from the finite values."""
    d = 64
    x = torch.zeros(1, 1, 8, d)
    x[0, 0, 0] = torch.finfo(torch.bfloat16).max
    x[0, 0, 1] = 2.0 ** -133
    x[0, 0, 2, 3] = float("inf")
    x[0, 0, 2, 4] = 5.0
    x[0, 0, 3, 5] = float("nan")
    x[0, 0, 3, 6] = -3.0
    x[0, 0, 4] = float("-inf")
    x[0, 0, 5] = 448.0
    x[0, 0, 6] = 452.0          # above 448: the next scale
    x[0, 0, 7, ::2] = -0.0
    x = x.to(torch.bfloat16)
    c = H.to_dev(H.empty_cache(1, 1, 8, d, 0, True, seed=2))
    _append(c, x.to(dev()), x.to(dev()), H.i32([0]), 0.0, "split_half")
    csattn.check_status()
    e = OA.e4m3_exponents(x[0, 0], False)
    want, stands = OA.quantise_rows(x[0, 0].double().numpy(), e)
    for n in ("k", "v"):
        assert np.array_equal(c[n + "s"][0, 0].cpu().numpy(), e + 127)
        np.testing.assert_array_equal(c[n][0, 0].cpu().double().numpy(), want)
    ko, vo = _read(c, H.i32([8]))
    for o in (ko, vo):
        np.testing.assert_array_equal(o[0, 0].cpu().double().numpy(), stands)


@pytest.mark.parametrize("B,Hkv,d,page,Lout", [(3, 4, 128, 0, 150), (2, 3, 64, 16, 100),
                                               (4, 1, 128, 64, 129), (1, 8, 64, 128, 1)])
def test_read_back_is_exact_and_leaves_the_rest(B, Hkv, d, page, Lout):
    room = 160
    lens = [Lout, 0, 1, Lout // 2][:B]
    c = H.empty_cache(B, Hkv, room, d, page, True, seed=d)
    g = H.gen(5)
    for b, L in enumerate(lens):
        k = (torch.randn(Hkv, L, d, generator=g) * 30).to(torch.bfloat16)
        if L:
            H.set_rows(c, b, 0, k, k * 2.0 ** -9)
    ko = torch.full((B, Hkv, Lout, d), 7.0, dtype=torch.bfloat16, device=dev())
    vo = torch.full_like(ko, -7.0)
    _read(H.to_dev(c), H.i32(lens), ko, vo)
    csattn.check_status()
    for b, L in enumerate(lens):
        k, v = H.rows(c, b, L) if L else (np.zeros((Hkv, 0, d)),) * 2
        assert np.array_equal(ko[b, :, :L].double().cpu().numpy(), k)
        assert np.array_equal(vo[b, :, :L].double().cpu().numpy(), v)
        assert torch.all(ko[b, :, L:] == 7.0) and torch.all(vo[b, :, L:] == -7.0)


def _filled(B, Hq, Hkv, d, page, lens, room, seed, gain=1.0):
    g = H.gen(seed)
    c = H.empty_cache(B, Hkv, room, d, page, True, seed=seed)
    for b, L in enumerate(lens):
        k = torch.randn(Hkv, L, d, generator=g).to(torch.bfloat16)
        v = (torch.randn(Hkv, L, d, generator=g) *
             torch.exp2(torch.randint(-3, 4, (Hkv, L, 1), generator=g))).to(torch.bfloat16)
        H.set_rows(c, b, 0, k, v)
    q = (torch.randn(B, Hq, 1, d, generator=g) * gain).to(torch.bfloat16)
    return c, q


def _expect(c, q, lens, base=0.0, layout="split_half", scale=None):
    out = np.zeros(tuple(q.shape))
    Hq = q.shape[1]
    for b, L in enumerate(lens):
        k, v = H.rows(c, b, L)
        x = q[b, :, 0].double().numpy()
        if base > 0:
            x = H.round_query(OA.rope_rotate(x[:, None], np.array([L - 1]), base, layout), True)[:, 0]
        out[b] = OA.decode(torch.from_numpy(x)[None, :, None], torch.from_numpy(k)[None],
                           torch.from_numpy(v)[None], [L], scale=scale)[0]
    return out


@pytest.mark.parametrize("d,Hq,Hkv,page,base,layout,splits", [
    (128, 8, 2, 0, 10000.0, "split_half", 0),
    (128, 32, 8, 64, 0.0, "split_half", 0),
    (64, 6, 2, 16, 10000.0, "adjacent", 3),
    (64, 12, 12, 32, 500000.0, "split_half", 0),
    (128, 16, 1, 256, 10000.0, "adjacent", 7),
    (128, 21, 1, 128, 0.0, "split_half", 1),     # more than 16 query heads per KV head
    (64, 48, 1, 0, 10000.0, "split_half", 2),
])
def test_decode_parity(d, Hq, Hkv, page, base, layout, splits):
    lens = [1, 15, 64, 65, 400, 701]
    c, q = _filled(6, Hq, Hkv, d, page, lens, 704, seed=Hq + d)
    out = _decode(H.to_dev(c), q.to(dev()), H.i32(lens), rope_base=base, rope_layout=layout,
                  num_splits=splits)
    csattn.check_status()
    got, ref = to_np(out), _expect(c, q, lens, base, layout)
    err, rl2 = np.max(np.abs(got - ref)), np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rl2 <= 5e-3 and err <= 2e-2 + half_ulp_bf16(np.max(np.abs(ref))), (err, rl2)


def test_decode_values_of_very_different_scales():
    """A row with all the weight and values 2^-30 of the others': its values are the output
    (relative L2 of the outputs' own scale, as everywhere)."""
    d, L = 128, 200
    c = H.empty_cache(1, 1, L, d, 0, True, seed=4)
    g = H.gen(9)
    q = torch.randn(1, 1, 1, d, generator=g).to(torch.bfloat16)
    k = torch.randn(1, L, d, generator=g).to(torch.bfloat16) * 0
    k[0, 77] = q[0, 0, 0] * 8            # score ~ 8 * |q|^2 / sqrt(d) ~ 90
    v = torch.randn(1, L, d, generator=g).to(torch.bfloat16)
    v[0, 77] *= 2.0 ** -30
    v[0, 3] = 0                          # an all-zero row among them
    H.set_rows(c, 0, 0, k, v)
    out = to_np(_decode(H.to_dev(c), q.to(dev()), H.i32([L])))
    ref = _expect(c, q, [L])
    assert np.max(np.abs(ref)) < 1e-7
    assert np.linalg.norm(out - ref) <= 5e-3 * np.linalg.norm(ref)


def test_decode_large_and_small_queries():
    """Queries at the ends of bf16's range: the scores come out of fp32 sums, 0 or decisive."""
    d, L = 64, 130
    c, q = _filled(1, 2, 1, d, 0, [L], L, seed=3)
    q = torch.cat([q[:, :1] * 2.0 ** -120, q[:, 1:] * 2.0 ** 40], 1)
    out = to_np(_decode(H.to_dev(c), q.to(dev()), H.i32([L])))
    ref = _expect(c, q, [L])
    assert np.linalg.norm(out - ref) <= 5e-3 * np.linalg.norm(ref)
    assert np.max(np.abs(out - ref)) <= 2e-2 + half_ulp_bf16(np.max(np.abs(ref)))


def test_decode_nan_in_sight_and_out_of_it():
    """Garbage past the length stays out; a NaN row, key or query in sight makes its outputs NaN."""
    d, L = 128, 100
    c, q = _filled(3, 4, 2, d, 64, [L, L, L], 128, seed=8)
    p, o = H.place(c, 1, 50)
    H.raw(c["k"])[p, 1, o, 3] = 0x7F
    q[2, 0, 0, 0] = float("nan")
    out = _decode(H.to_dev(c), q.to(dev()), H.i32([L] * 3)).cpu()
    csattn.check_status()
    assert torch.isfinite(out[0]).all()
    assert torch.isfinite(out[1, :2]).all() and torch.isnan(out[1, 2:]).all()
    assert torch.isnan(out[2, 0]).all() and torch.isfinite(out[2, 1:]).all()


def test_device_side_refusals():
    d, Hkv, page = 64, 2, 16
    c, q = _filled(3, 4, Hkv, d, page, [40, 40, 40], 48, seed=6)
    cd = H.to_dev(c)

    def refused():
        with pytest.raises(csattn.CsattnError) as e:
            csattn.check_status()
        assert e.value.status == -6

    good = _decode(cd, q.to(dev()), H.i32([40, 40, 40]))
    csattn.check_status()
    for bad in (0, -1, 49):
        out = _decode(cd, q.to(dev()), H.i32([40, bad, 40]))
        refused()
        assert torch.all(out[1] == 0)
        assert H.same_bits(out[0], good[0]) and H.same_bits(out[2], good[2])
    # lengths: the read leaves the outputs, the append the cache
    ko = torch.zeros(3, Hkv, 45, d, dtype=torch.bfloat16, device=dev())
    vo = torch.zeros_like(ko)
    _read(cd, H.i32([40, 46, -3]), ko, vo)
    refused()
    assert torch.all(ko[1:] == 0) and torch.any(ko[0] != 0)
    new = torch.ones(3, Hkv, 9, d, dtype=torch.bfloat16, device=dev())
    _append(cd, new, new, H.i32([40, -1, 2 ** 31 - 1]), 0.0, "split_half")
    refused()
    for n in ("k", "v", "ks", "vs"):
        assert H.same_bits(cd[n].cpu(), c[n])
    # a page index outside the pool
    cd["table"][1, 1] = c["k"].shape[0]
    cd["table"][2, 0] = -5
    out = _decode(cd, q.to(dev()), H.i32([40, 40, 40]))
    refused()
    assert H.same_bits(out[0], good[0])
    _read(cd, H.i32([40, 40, 40]), ko, vo)
    refused()
    assert torch.all(ko[1, :, 16:32] == 0) and torch.any(ko[1, :, :16] != 0)
    _append(cd, new, new, H.i32([0, 12, 0]), 0.0, "split_half")
    refused()
    csattn.check_status()


def test_append_then_decode_then_read_over_shared_and_long_caches():
    """A prompt in chunks into pages, decode, and a chunked prefill over the rows read back
    agree with the same steps over the cache the oracle keeps."""
    B, Hq, Hkv, d, page, n = 2, 8, 2, 128, 16, 200
    g = H.gen(12)
    k = torch.randn(B, Hkv, n, d, generator=g).to(torch.bfloat16)
    v = torch.randn(B, Hkv, n, d, generator=g).to(torch.bfloat16)
    q = torch.randn(B, Hq, 1, d, generator=g).to(torch.bfloat16)
    cd = H.to_dev(H.empty_cache(B, Hkv, n + 8, d, page, True, seed=3))
    L = 0
    for m in (1, 63, 136):
        kn, vn = (x[:, :, L:L + m].contiguous().to(dev()) for x in (k, v))
        _append(cd, kn, vn, H.i32([L] * B), 10000.0, "split_half")
        L += m
    out = _decode(cd, q.to(dev()), H.i32([n] * B), rope_base=10000.0)
    csattn.check_status()
    c = H.to_cpu(cd)
    assert_bf16_close(to_np(out), _expect(c, q, [n] * B, 10000.0), "decode of appended chunks")
    # the stored keys stand for the rotated ones: relative error of e4m3, 2^-4 per value
    kr = OA.rope_rotate(k.double().numpy(), np.arange(n), 10000.0)
    for b in range(B):
        have, _ = H.rows(c, b, n)
        assert np.all(np.abs(have - kr[b]) <= np.abs(kr[b]) * 2.0 ** -4 +
                      np.max(np.abs(kr[b]), -1, keepdims=True) * 2.0 ** -15)
    # the last 40 rows once more as a chunk of queries over the cache read back
    ko, vo = _read(cd, H.i32([n] * B))
    ko, vo = ko[:, :, :n].contiguous(), vo[:, :, :n].contiguous()
    qc = torch.randn(B, Hq, 40, d, generator=g).to(torch.bfloat16)
    got = csattn.attn_fwd_ext(qc.to(dev()), ko, vo, q_offset=n - 40, rope_base=10000.0,
                              k_prerotated=True)
    csattn.check_status()
    for b in range(B):
        kk, vv = H.rows(c, b, n)
        qr = OA.round_to_bf16(OA.rope_rotate(qc[b].double().numpy(), n - 40 + np.arange(40),
                                             10000.0))
        for h in range(Hq):
            z = qr[h] @ kk[h // 4].T / np.sqrt(d)
            z[np.arange(n)[None] > (n - 40 + np.arange(40))[:, None]] = -np.inf
            ref = OA.softmax_rows(z) @ vv[h // 4]
            assert_bf16_close(to_np(got[b, h]), ref, "prefill over rows read back")


def test_offsets_past_32_bits():
    """A pool of more than 2^31 bytes: the last page's rows are written, read and attended."""
    Hkv, d, page = 8, 128, 64
    n = (1 << 31) // (Hkv * d * page) + 3
    k8 = torch.zeros(n, Hkv, page, d, dtype=torch.float8_e4m3fn, device=dev())
    v8 = torch.zeros_like(k8)
    ks = torch.full((n, Hkv, page), 127, dtype=torch.uint8, device=dev())
    vs = ks.clone()
    table = H.i32([[n - 1]])
    g = H.gen(1)
    kn = torch.randn(1, Hkv, 50, d, generator=g).to(torch.bfloat16)
    csattn.cache_append_fp8_paged(kn.to(dev()), kn.to(dev()), k8, v8, ks, vs, table, H.i32([0]))
    ko, vo = csattn.cache_read_fp8_paged(k8, v8, ks, vs, table, H.i32([50]))
    q = torch.randn(1, Hkv, 1, d, generator=g).to(torch.bfloat16)
    out = csattn.attn_decode_fp8_paged(q.to(dev()), k8, v8, ks, vs, table, H.i32([50]))
    csattn.check_status()
    e = OA.e4m3_exponents(kn, False)
    _, x = OA.quantise_rows(kn.double().numpy(), e)
    assert np.array_equal(ko[:, :, :50].double().cpu().numpy(), x)
    ref = OA.decode(q, x, x, [50])
    assert_bf16_close(to_np(out), ref, "last page")


def test_graphs_streams_and_repeats():
    """Captured and replayed on a side stream with other inputs in the same buffers, each graph
    with its workspace; equal inputs give equal bits."""
    lens = [100, 37]
    c, q = _filled(2, 8, 2, 128, 64, lens, 128, seed=21)
    cd = H.to_dev(c)
    qd, ld = q.to(dev()), H.i32(lens)
    first = _decode(cd, qd, ld, rope_base=10000.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = _decode(cd, qd, ld, rope_base=10000.0, stream=side)
    side.synchronize()
    assert H.same_bits(out, first)
    graphs = []
    for _ in range(2):
        o = torch.empty_like(first)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            _decode(cd, qd, ld, out=o, rope_base=10000.0)
        graphs.append((gr, o))
    qd.mul_(-1)
    other = _decode(cd, qd, ld, rope_base=10000.0)
    for gr, o in graphs:
        gr.replay()
    torch.cuda.synchronize()
    csattn.check_status()
    for _, o in graphs:
        assert H.same_bits(o, other)
    assert not H.same_bits(other, first)
