"""Attention over an 8-bit cache at the ends of the scale codes' range and with rows of very
different scales beside one another, against float64.

Tolerance, per output element, with w_j a query's weights (of sum 1) and A = sum_j w_j |v_j|:
  2^-8 |out|           the output's rounding to bf16 (half a step, doubled)
  2^-11 A              weights rounded to 11 bits (half a step: 2^-12 A) and what is below f16's
                       least (2^-31 of the largest term for each row: < 2^-20 A for 1000 rows)
  2^-17 max|x| A       scores x as fp32 sums of d <= 128 products and one fp32 addition: off by
                       at most 2^-18 of sum |q_i k_i| * scale * log2(e), which is taken as x here
  2^-133               a step of bf16 below its normal numbers
The reference reads the rows the cache holds and rounds the query as the kernels do."""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import attn as OA
from tests import fp8_helpers as H
from tests import test_gpu_tree as T
from tests.gpu_helpers import dev, to_np

pytestmark = pytest.mark.gpu


def _reference(q, kk, vv, seen):
    """q [Hq, T, d] rounded, kk, vv [Hkv, n, d], seen [T, n]: (out, lse, bound) in float64."""
    Hq, n_t, d = q.shape
    rep = Hq // kk.shape[0]
    out, bound, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((Hq, n_t))
    for h in range(Hq):
        for t in range(n_t):
            k, v = kk[h // rep][seen[t]], vv[h // rep][seen[t]]
            z = (k @ q[h, t]) / np.sqrt(d)
            big = np.max(np.abs(k) @ np.abs(q[h, t])) / np.sqrt(d) * 1.4427
            w = np.exp(z - z.max())
            lse[h, t] = z.max() + np.log(w.sum())
            w /= w.sum()
            out[h, t] = w @ v
            a = w @ np.abs(v)
            bound[h, t] = (2.0 ** -8 * np.abs(out[h, t]) + (2.0 ** -11 + 2.0 ** -17 * big) * a +
                           2.0 ** -133)
    return out, lse, bound


def _close(got, ref, bound, what):
    assert np.all(np.isfinite(got)), what
    off = np.abs(got - ref) / bound
    assert off.max() <= 1.0, f"{what}: {off.max():.3g} times the bound"


def _check_tree(q, k, v, prefix_k, prefix_v, parents, d, page=0, queries=None, **kw):
    """A step over a prefix [Hkv, L, d] (float tensors of bf16 values); `queries`: the drafts
    whose outputs are checked."""
    Hkv, L, _ = prefix_k.shape
    Hq, Tn = q.shape[1:3]
    c = H.empty_cache(1, Hkv, L + Tn, d, page, True, seed=1)
    if L:
        H.set_rows(c, 0, 0, prefix_k, prefix_v)
    cd = H.to_dev(c)
    lse = torch.zeros(1, Hq, Tn, device=dev())
    out = T._step(cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32([L]), H.i32([parents]),
                  lse=lse, **kw)
    csattn.check_status()
    kk, vv = H.rows(H.to_cpu(cd), 0, L + Tn)
    anc = OA.tree_ancestors(parents)
    at = [t for t in range(Tn) if anc[t, t]] if queries is None else queries
    seen = [np.concatenate([np.arange(L), L + np.nonzero(anc[t])[0]]).astype(int) for t in at]
    ref, ref_lse, bound = _reference(H.round_query(q[0, :, at].double().numpy(), True), kk, vv,
                                     seen)
    _close(to_np(out)[0][:, at], ref, bound, "out")
    got = lse.double().cpu().numpy()[0][:, at]
    assert np.max(np.abs(got - ref_lse) / np.maximum(1.0, np.abs(ref_lse))) <= 1e-3
    return out


def _inputs(Hq, Hkv, L, Tn, d, seed):
    g = H.gen(seed)
    new = [torch.randn(1, h, Tn, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
    old = [torch.randn(Hkv, L, d, generator=g).to(torch.bfloat16) for _ in range(2)]
    return new + old


HUGE = [float(torch.finfo(torch.bfloat16).max), 1e30]


@pytest.mark.parametrize("L", [0, 30, 300])
@pytest.mark.parametrize("what", ["keys", "values", "both"])
@pytest.mark.parametrize("Tn,Hq,d", [(6, 2, 64), (6, 2, 128), (40, 4, 64), (40, 4, 128),
                                     (40, 8, 128)])
def test_finite_values_of_unseen_drafts_stay_out(Tn, Hq, d, what, L):
    """The largest finite values, and 1e30, in a branch and in padding: the drafts that see
    neither have the outputs of a run without them, but for the weights' rounding."""
    q, k, v, pk, pv = _inputs(Hq, 1, L, Tn, d, Tn + d + L)
    parents = [-1, 0, -1, 2] + [-1] * (Tn - 6) + [-2, -2]
    free = [t for t in range(Tn - 2) if t not in (2, 3)]
    for huge in HUGE:
        kb, vb = k.clone(), v.clone()
        for t in (2, 3, Tn - 2, Tn - 1):
            if what != "values":
                kb[0, 0, t] = torch.where(k[0, 0, t] < 0, -huge, huge)
            if what != "keys":
                vb[0, 0, t] = torch.where(v[0, 0, t] < 0, -huge, huge)
        _check_tree(q, kb, vb, pk, pv, parents, d, queries=free)


@pytest.mark.parametrize("Tn,Hq", [(6, 2), (40, 4)])
@pytest.mark.parametrize("base", [1e30, 1e10, 1e-20])
def test_rows_of_another_scale_in_sight(Tn, Hq, base):
    """A value row far from the others' scale, and keys far below them, in everybody's sight."""
    d, L = 128, 200
    q, k, v, pk, pv = _inputs(Hq, 1, L, Tn, d, 5)
    pv[0, 7] = pv[0, 7] * base
    pk[0, 11::16] = pk[0, 11::16] * 1e-12
    k[0, 0, 1] = 0
    _check_tree(q, k, v, pk, pv, [-1] * Tn, d)
    # a small value with nearly all of the weight beside large ones with hardly any
    q[:] = 1
    pk[0], k[0, 0] = 0, 0
    pk[0, 3] = 4.0                               # x = 4 * 128 / sqrt(128) = 45 nats = 65 octaves
    pv[0, 3] = pv[0, 3] * 2.0 ** -40
    pv[0, 4:] = pv[0, 4:] * 2.0 ** 20
    _check_tree(q, k, v, pk, pv, [-1] * Tn, d)


@pytest.mark.parametrize("v_shift", [0, -100, 100])
@pytest.mark.parametrize("L", [0, 300])
@pytest.mark.parametrize("Tn,Hq,d", [(4, 2, 64), (5, 8, 64), (40, 8, 128)])
def test_a_key_that_decides_alone(Tn, Hq, d, L, v_shift):
    """A draft's key of 1e30: scores of 1e30, beside which a scale's exponent is lost.  Its own
    query takes its value, exactly, where the score is positive, and the others' where it is not;
    without a prefix it has nothing else to see."""
    q, k, v, pk, pv = _inputs(Hq, 1, L, Tn, d, 9)
    v, pv = ((x.double() * 2.0 ** v_shift).to(torch.bfloat16) for x in (v, pv))
    k[0, 0, 2] = torch.where(k[0, 0, 2] < 0, -1e30, 1e30)
    others = [t for t in range(Tn) if t != 2]
    out = _check_tree(q, k, v, pk, pv, [-1] * Tn, d, queries=others)
    _, own = OA.quantise_rows(v[0, 0, 2].double().numpy(), OA.e4m3_exponents(v[0, 0, 2], False))
    got = to_np(out)[0, :, 2]
    score = (q[0, :, 2].double() @ k[0, 0, 2].double()).numpy()
    for h in range(Hq):
        if L == 0 or score[h] > 0:
            assert np.array_equal(got[h], own), h
        else:
            # (as if the draft were not there)
            kk, vv = pk[0].double().numpy(), pv[0].double().numpy()
            z = kk @ q[0, h, 2].double().numpy() / np.sqrt(d)
            w = np.exp(z - z.max())
            ref = w / w.sum() @ vv
            # (the prefix unquantised here: half a step of e4m3 in keys and values)
            assert np.linalg.norm(got[h] - ref) <= 2.0 ** -2 * np.linalg.norm(ref), h


@pytest.mark.parametrize("splits", [0, 1, 7])
@pytest.mark.parametrize("Hq", [2, 12])
def test_equal_large_scores_weigh_alike(Hq, splits):
    """300 equal keys whose score is past 2^24: the mean of the values, in whatever pieces."""
    d, L = 64, 300
    _, _, _, _, pv = _inputs(1, 1, L, 1, d, 2)
    c = H.empty_cache(1, 1, L, d, 0, True, seed=2)
    H.set_rows(c, 0, 0, torch.full((1, L, d), 2.0 ** 40, dtype=torch.bfloat16), pv)
    cd = H.to_dev(c)
    q = torch.ones(1, Hq, 1, d, dtype=torch.bfloat16, device=dev())
    out = csattn.attn_decode_fp8(q, cd["k"], cd["v"], cd["ks"], cd["vs"], H.i32([L]),
                                 num_splits=splits)
    csattn.check_status()
    vv = H.rows(c, 0, L)[1][0]
    bound = 2.0 ** -8 * np.abs(vv.mean(0)) + 2.0 ** -11 * np.abs(vv).mean(0)
    _close(to_np(out)[0, :, 0], np.broadcast_to(vv.mean(0), (Hq, d)), bound, "mean")


def _decode(q, k, v, **kw):
    """q [1, Hq, 1, d], k, v [Hkv, L, d]: checked decode over them."""
    Hkv, L, d = k.shape
    c = H.empty_cache(1, Hkv, L, d, 0, True, seed=2)
    H.set_rows(c, 0, 0, k, v)
    cd = H.to_dev(c)
    out = csattn.attn_decode_fp8(q.to(dev()), cd["k"], cd["v"], cd["ks"], cd["vs"], H.i32([L]),
                                 **kw)
    csattn.check_status()
    kk, vv = H.rows(c, 0, L)
    seen = [np.arange(L)]
    ref, _, bound = _reference(H.round_query(q[0].double().numpy(), True), kk, vv, seen)
    _close(to_np(out)[0], ref, bound, "decode")


# (a value of a row's largest code: 1.75 * 2^127 and more; of its least: 448 * 2^-124 and less)
SPANS = {"top": lambda x, n: torch.where(x < 0, -1.0, 1.0) * 2.0 ** 127 * 1.8,
         "bottom": lambda x, n: x * 2.0 ** -122,
         "least": lambda x, n: x * 2.0 ** -128,
         "low": lambda x, n: x * 2.0 ** -112,
         "halves": lambda x, n: torch.where(torch.arange(n)[:, None] < n // 2, x * 2.0 ** -118,
                                            x * 2.0 ** 100),
         "halves, upper first": lambda x, n: torch.where(torch.arange(n)[:, None] >= n // 2,
                                                         x * 2.0 ** -118, x * 2.0 ** 100),
         "top and one": lambda x, n: torch.where(torch.arange(n)[:, None] % 128 == 5,
                                                 1.9 * 2.0 ** 127, x),
         "both in every tile": lambda x, n: torch.where(torch.arange(n)[:, None] % 3 == 0,
                                                        x * 2.0 ** -118, x * 2.0 ** -90),
         "far apart, halves": lambda x, n: x * torch.exp2(
             20.0 * (torch.arange(n)[:, None] % 2) + torch.where(
                 torch.arange(n)[:, None] < n // 2, 90.0, -110.0)),
         "zeros and one large": lambda x, n: torch.where(torch.arange(n)[:, None] == 5,
                                                         x * 2.0 ** 60, 0.0)}


@pytest.mark.parametrize("splits", [0, 1, 7])
@pytest.mark.parametrize("span", SPANS)
@pytest.mark.parametrize("d,Hq", [(64, 4), (128, 4), (128, 12)])
def test_decode_over_the_range_of_values(d, Hq, span, splits):
    q, _, _, pk, pv = _inputs(Hq, 1, 512, 1, d, 3)
    _decode(q, pk, SPANS[span](pv.double(), 512).to(torch.bfloat16), num_splits=splits)


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("span", SPANS)
@pytest.mark.parametrize("d,Hq,Tn", [(128, 2, 4), (64, 4, 4), (64, 8, 12), (128, 8, 12),
                                       (128, 8, 20)])
def test_tree_over_the_range_of_values(d, Hq, Tn, span, splits):
    """In one tile, over the tiles of one CTA and over CTAs."""
    q, k, v, pk, pv = _inputs(Hq, 1, 512 - Tn, Tn, d, 4)
    both = SPANS[span](torch.cat([pv, v[0]], 1).double(), 512).to(torch.bfloat16)
    _check_tree(q, k, both[None, :, 512 - Tn:], pk, both[:, :512 - Tn].contiguous(),
                [t // 2 - 1 for t in range(Tn)], d, num_splits=splits)


@pytest.mark.parametrize("shift", [-116, -100, -40, 40, 100, 116])
@pytest.mark.parametrize("Hq,Tn", [(2, 4), (8, 12)])
def test_keys_and_queries_over_the_range(Hq, Tn, shift):
    """Keys and queries whose scales cancel."""
    q, k, v, pk, pv = _inputs(Hq, 1, 300, Tn, 128, 6)
    q = (q.double() * 2.0 ** -shift).to(torch.bfloat16)
    k, pk = ((x.double() * 2.0 ** shift).to(torch.bfloat16) for x in (k, pk))
    _check_tree(q, k, v, pk, pv, [-1] * Tn, 128)
    _decode(q[:, :, :1].contiguous(), pk, pv)
