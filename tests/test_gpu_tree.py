"""Token trees over a cache (csattn_attn_tree_step, csattn_tree_commit) against float64.

Tolerances: outputs as in the other bf16 attention tests (max-abs 2e-2, relative L2 5e-3);
lse: a sum of fp32 exponentials (each off by 2^-22) of scores that are off by the rounding of
the rotated query alone (bf16, or 11 bits with an 8-bit cache), which the reference makes too, so 1e-3 covers fp32 sums of the
d products (d * 2^-24 * |score| below 2^-10 here).  Appended rows: values bit-exact, rotated keys
as in the append tests.
"""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import attn as OA
from tests import fp8_helpers as H
from tests.gpu_helpers import assert_bf16_close, dev, to_np

pytestmark = pytest.mark.gpu

CHAIN = "chain"


def make_parents(kind, Tn, g):
    if kind == CHAIN:
        return [t - 1 for t in range(Tn)]
    if kind == "flat":
        return [-1] * Tn
    p = [int(torch.randint(-1, t, (1,), generator=g)) if t else -1 for t in range(Tn)]
    if kind == "padded":
        for t in range(Tn):
            if t >= 1 and (t % 5 == 4 or t >= Tn - 2) and t not in p:
                p[t] = -2
    return p


def _step(c, q, k, v, lens, parents, **kw):
    kw.update(H.scales(c))
    if c["table"] is None:
        return csattn.attn_tree_step(q, k, v, c["k"], c["v"], lens, parents, **kw)
    return csattn.attn_tree_step_paged(q, k, v, c["k"], c["v"], c["table"], lens, parents, **kw)


def _commit(c, lens, parents, accepted, new_lens=None):
    if c["table"] is None:
        return csattn.tree_commit(c["k"], c["v"], lens, parents, accepted, new_lens, **H.scales(c))
    return csattn.tree_commit_paged(c["k"], c["v"], c["table"], lens, parents, accepted, new_lens,
                                    **H.scales(c))


def _case(B, Hq, Hkv, d, Tn, lens, room, page, e4m3, kind, seed):
    g = H.gen(seed)
    c = H.empty_cache(B, Hkv, room, d, page, e4m3, seed=seed)
    for b, L in enumerate(lens):
        if L:
            H.set_rows(c, b, 0, torch.randn(Hkv, L, d, generator=g).to(torch.bfloat16),
                       torch.randn(Hkv, L, d, generator=g).to(torch.bfloat16))
    q = torch.randn(B, Hq, Tn, d, generator=g).to(torch.bfloat16)
    k = torch.randn(B, Hkv, Tn, d, generator=g).to(torch.bfloat16)
    v = torch.randn(B, Hkv, Tn, d, generator=g).to(torch.bfloat16)
    parents = [make_parents(kind, Tn, g) for _ in range(B)]
    return c, q, k, v, parents


def _check(c0, c1, q, k, v, parents, lens, out, lse, base, layout):
    """Outputs from the rows the cache holds; those rows against the drafts; nothing else moved."""
    B, Hq, Tn, d = q.shape
    wrong = total = 0
    ref = np.zeros(tuple(q.shape))
    ref_lse = np.zeros(tuple(q.shape[:3]))
    for b, L in enumerate(lens):
        anc = OA.tree_ancestors(parents[b])
        pos = L + np.maximum(anc.sum(1) - 1, 0)
        kk, vv = H.rows(c1, b, L + Tn)
        kr = k[b].double().numpy()
        if base > 0:
            kr = OA.rope_rotate(kr, pos, base, layout)
        if "ks" in c1:
            _, kw = OA.quantise_rows(kr, OA.e4m3_exponents(k[b], base > 0))
            _, vw = OA.quantise_rows(v[b].double().numpy(), OA.e4m3_exponents(v[b], False))
            step = 2.0 ** -3
        else:
            kw, vw, step = OA.round_to_bf16(kr), v[b].double().numpy(), 2.0 ** -7
        assert np.array_equal(vv[:, L:], vw)
        off = kk[:, L:] != kw
        wrong, total = wrong + int(off.sum()), total + off.size
        top = np.max(np.abs(kw), -1, keepdims=True)
        assert np.all(np.abs(kk[:, L:] - kw) <= np.maximum(np.abs(kw) * step, top * 2.0 ** -15))
        qr = q[b].double().numpy()
        if base > 0:
            qr = H.round_query(OA.rope_rotate(qr, pos, base, layout), "ks" in c1)
        ref[b], ref_lse[b] = OA.tree_attention(qr, kk, vv, L, anc)
    assert wrong <= max(2, 2e-3 * total), (wrong, total)
    assert_bf16_close(to_np(out), ref, "tree attention")
    if lse is not None:
        got = lse.double().cpu().numpy()
        assert np.array_equal(np.isinf(got), np.isinf(ref_lse))
        f = np.isfinite(ref_lse)
        assert np.max(np.abs(got[f] - ref_lse[f]), initial=0.0) <= 1e-3
    for n in [n for n in ("k", "v", "ks", "vs") if n in c0]:
        x, y = H.raw(c0[n]).clone(), H.raw(c1[n]).clone()
        for b, L in enumerate(lens):
            for t in range(Tn):
                p, o = H.place(c0, b, L + t)
                x[p, :, o] = 0
                y[p, :, o] = 0
        assert H.same_bits(x, y), f"{n}: other rows were written"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,Tn,page,kind,base,layout", [
    (128, 8, 2, 1, 0, CHAIN, 10000.0, "split_half"),
    (128, 4, 1, 8, 64, "random", 10000.0, "adjacent"),
    (64, 2, 2, 17, 16, "padded", 500000.0, "split_half"),
    (64, 6, 1, 33, 32, "random", 0.0, "split_half"),
    (128, 8, 2, 64, 128, "random", 10000.0, "split_half"),
    (128, 7, 1, 40, 0, "padded", 10000.0, "split_half"),
    (64, 3, 3, 100, 64, CHAIN, 10000.0, "adjacent"),
    (128, 2, 1, 256, 0, "padded", 10000.0, "split_half"),
    (64, 24, 1, 31, 0, "flat", 0.0, "split_half"),
])
def test_tree_step(d, Hq, Hkv, Tn, page, kind, base, layout, e4m3):
    lens = [0, 1, 63, 200]
    room = 200 + Tn
    c, q, k, v, parents = _case(4, Hq, Hkv, d, Tn, lens, room, page, e4m3, kind, seed=Tn + d)
    cd = H.to_dev(c)
    lse = torch.zeros(4, Hq, Tn, device=dev())
    out = _step(cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32(lens), H.i32(parents), lse=lse,
                rope_base=base, rope_layout=layout)
    csattn.check_status()
    _check(c, H.to_cpu(cd), q, k, v, parents, lens, out, lse, base, layout)


@pytest.mark.parametrize("splits", [1, 2, 5, 100])
@pytest.mark.parametrize("e4m3,Tn,Hq", [(False, 20, 4), (True, 20, 4), (False, 48, 8),
                                        (True, 48, 8)])
def test_tree_step_splits(splits, e4m3, Tn, Hq):
    lens = [700, 641, 5]
    c, q, k, v, parents = _case(3, Hq, 1, 128, Tn, lens, 800, 16, e4m3, "random", seed=splits)
    cd = H.to_dev(c)
    out = _step(cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32(lens), H.i32(parents),
                rope_base=10000.0, num_splits=splits, max_seq_len=780)
    csattn.check_status()
    _check(c, H.to_cpu(cd), q, k, v, parents, lens, out, None, 10000.0, "split_half")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Tn,Hq", [(6, 2), (40, 4)])
def test_values_of_unseen_drafts_stay_out(e4m3, Tn, Hq):
    """NaN, infinities and the largest values in one branch: the other branch's outputs are the
    same bits as without them, and the drafts that see them get them."""
    d, L = 64, 30
    c, q, k, v, _ = _case(1, Hq, 1, d, Tn, [L], L + Tn, 0, e4m3, "flat", seed=3)
    parents = [[-1, 0, -1, 2] + [-1] * (Tn - 4)]  # 0-1 and 2-3 are branches
    args = (q.to(dev()), k.to(dev()))
    cd = H.to_dev(c)
    clean = _step(cd, *args, v.to(dev()), H.i32([L]), H.i32(parents)).cpu()
    v2 = v.clone()
    v2[0, 0, 2, 5] = float("inf")
    v2[0, 0, 2, 6] = float("nan")
    v2[0, 0, 3, 5] = float("-inf")
    v2[0, 0, 3, 7] = float("-inf")
    k2 = k.clone()
    k2[0, 0, Tn - 1, 0] = float("nan")   # a key only its own draft sees
    cd = H.to_dev(c)
    out = _step(cd, args[0], k2.to(dev()), v2.to(dev()), H.i32([L]), H.i32(parents)).cpu()
    csattn.check_status()
    free = [t for t in range(Tn - 1) if t not in (2, 3)]
    assert H.same_bits(out[:, :, free], clean[:, :, free])
    assert torch.isnan(out[:, :, Tn - 1]).all()
    bad = torch.isfinite(out[0, :, 2]).logical_not()
    assert bad[:, [5, 6]].all() and bad.sum() == 2 * Hq
    if not e4m3:
        assert torch.all(out[0, :, 2, 5] == float("inf"))
        assert torch.all(out[0, :, 3, 7] == float("-inf"))
    assert torch.isnan(out[0, :, 3, [5, 6]]).all()
    bad = torch.isfinite(out[0, :, 3]).logical_not()
    assert bad[:, [5, 6, 7]].all() and bad.sum() == 3 * Hq


def test_single_draft_is_the_decode_step():
    """Tn = 1 with parent -1 over a bf16 cache: csattn_attn_decode_step's cache rows, and its
    output within the two kernels' roundings."""
    B, Hq, Hkv, d, lens = 3, 8, 2, 128, [0, 5, 99]
    c, q, k, v, _ = _case(B, Hq, Hkv, d, 1, lens, 100, 0, False, CHAIN, seed=14)
    one, two = H.to_dev(c), H.to_dev(c)
    args = (q.to(dev()), k.to(dev()), v.to(dev()))
    a = _step(one, *args, H.i32(lens), H.i32([[-1]] * B), rope_base=10000.0)
    b = csattn.attn_decode_step(*args, two["k"], two["v"], H.i32(lens), rope_base=10000.0)
    csattn.check_status()
    assert H.same_bits(one["k"], two["k"]) and H.same_bits(one["v"], two["v"])
    assert_bf16_close(to_np(a), to_np(b), "single draft")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page,Tn", [(64, 16, 12), (128, 0, 40), (128, 64, 256), (64, 0, 1)])
def test_commit_moves_the_path(e4m3, d, page, Tn):
    B, Hkv, lens = 5, 3, [0, 1, 14, 60, 100]
    c, _, k, v, parents = _case(B, 3, Hkv, d, Tn, lens, 100 + Tn, page, e4m3, "random", seed=Tn)
    parents[3] = make_parents(CHAIN, Tn, None)
    for b, L in enumerate(lens):
        H.set_rows(c, b, L, k[b], v[b])
    accepted = [-1, 0, Tn - 1, Tn - 1, Tn // 2]
    cd = H.to_dev(c)
    new = _commit(cd, H.i32(lens), H.i32(parents), H.i32(accepted))
    csattn.check_status()
    got = H.to_cpu(cd)
    want = {n: (x.clone() if isinstance(x, torch.Tensor) else x) for n, x in c.items()}
    for b, L in enumerate(lens):
        path = OA.tree_path(parents[b], accepted[b])
        assert int(new[b]) == L + len(path)
        for i, a in enumerate(path):
            p0, o0 = H.place(c, b, L + a)
            p1, o1 = H.place(c, b, L + i)
            for n in [n for n in ("k", "v", "ks", "vs") if n in c]:
                H.raw(want[n])[p1, :, o1] = H.raw(c[n])[p0, :, o0]
    for n in [n for n in ("k", "v", "ks", "vs") if n in c]:
        assert H.same_bits(got[n], want[n]), n


@pytest.mark.parametrize("e4m3", [False, True])
def test_speculative_loop(e4m3):
    """Draft, step, commit, draft again: the committed cache is what appending the accepted
    tokens one by one gives, and the next step attends to it."""
    B, Hq, Hkv, d, page, Tn, base = 2, 4, 2, 64, 16, 6, 10000.0
    lens, room = [3, 20], 64
    c, q, k, v, _ = _case(B, Hq, Hkv, d, Tn, lens, room, page, e4m3, "flat", seed=1)
    cd = H.to_dev(c)
    parents = [[-1, -1, 0, 1, 3, -2], [-1, 0, 1, 1, -1, 4]]
    accepted = [4, 3]
    _step(cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32(lens), H.i32(parents), rope_base=base)
    new = _commit(cd, H.i32(lens), H.i32(parents), H.i32(accepted))
    one = H.to_dev(c)
    for b in range(B):
        path = OA.tree_path(parents[b], accepted[b])
        kn, vn = k[b:b + 1, :, path].contiguous().to(dev()), v[b:b + 1, :, path].contiguous().to(dev())
        at, tab = H.i32([lens[b]]), one["table"][b:b + 1].contiguous()
        if e4m3:
            csattn.cache_append_fp8_paged(kn, vn, one["k"], one["v"], one["ks"], one["vs"], tab,
                                          at, rope_base=base)
        else:
            csattn.cache_append_paged(kn, vn, one["k"], one["v"], tab, at, rope_base=base)
    csattn.check_status()
    assert new.tolist() == [lens[0] + 3, lens[1] + 3]
    x, y = H.to_cpu(cd), H.to_cpu(one)
    for b in range(B):
        for a, e in zip(H.rows(x, b, int(new[b])), H.rows(y, b, int(new[b]))):
            assert np.array_equal(a, e)
    q2, k2, v2 = (torch.roll(t, 1, 0).to(dev()) for t in (q, k, v))
    p2 = [[-1, 0, 0, 2, 2, 1]] * B
    for cc in (cd, one):
        cc["out"] = _step(cc, q2, k2, v2, new, H.i32(p2), rope_base=base)
    csattn.check_status()
    assert H.same_bits(cd["out"], one["out"])
    before = dict(x)
    _check(before, H.to_cpu(cd), q2.cpu(), k2.cpu(), v2.cpu(), p2, new.tolist(), cd["out"], None,
           base, "split_half")


def test_device_side_refusals():
    B, Hq, Hkv, d, Tn, lens, page = 4, 4, 2, 64, 5, [10, 10, 10, 10], 16
    c, q, k, v, _ = _case(B, Hq, Hkv, d, Tn, lens, 32, page, True, "flat", seed=5)
    good = [-1, 0, 0, 1, -2]
    args = (q.to(dev()), k.to(dev()), v.to(dev()))
    cd = H.to_dev(c)
    ref = _step(cd, *args, H.i32(lens), H.i32([good] * B))
    csattn.check_status()

    def refused():
        with pytest.raises(csattn.CsattnError) as e:
            csattn.check_status()
        assert e.value.status == -6

    bad_trees = [[-1, 1, 0, 0, 0], [-1, -3, 0, 0, 0], [-2, 0, -1, -1, -1]]
    for tree, L in [(t, 10) for t in bad_trees] + [(good, -1), (good, 28), (good, 2 ** 31 - 1)]:
        cd = H.to_dev(c)
        out = _step(cd, *args, H.i32([10, L, 10, 10]), H.i32([good, tree, good, good]),
                    rope_base=0.0)
        refused()
        assert torch.all(out[1] == 0)
        for b in (0, 2, 3):
            assert H.same_bits(out[b], ref[b])
        for b in (1,):
            for a, e in zip(H.rows(H.to_cpu(cd), b, 32), H.rows(c, b, 32)):
                assert np.array_equal(a, e, equal_nan=True)
    for acc, L, tree in [(5, 10, good), (-2, 10, good), (4, 10, good), (2, -1, good),
                         (2, 28, good), (3, 10, [-1, 1, 0, 1, 0]), (1, 10, [-1, -5, 0, 0, 0])]:
        cd = H.to_dev(c)
        new = _commit(cd, H.i32([10, L, 10, 10]), H.i32([good, tree, good, good]),
                      H.i32([-1, acc, -1, -1]))
        refused()
        assert new.tolist() == [10, L, 10, 10]
        for n in ("k", "v", "ks", "vs"):
            assert H.same_bits(cd[n].cpu(), c[n])
    # pages outside the pool: the drafts' rows there are not written, the others' outputs stand
    cd = H.to_dev(c)
    cd["table"][2, 0] = 10 ** 6
    out = _step(cd, *args, H.i32(lens), H.i32([good] * B))
    refused()
    assert H.same_bits(out[0], ref[0]) and torch.isfinite(out[2]).all()
    new = _commit(cd, H.i32(lens), H.i32([good] * B), H.i32([2, 2, 2, 2]))
    refused()
    assert new.tolist() == [12, 12, 10, 12]
    csattn.check_status()


def test_graph_of_step_and_commit_on_another_stream():
    """A step and its commit captured once, replayed with other inputs in the same buffers."""
    B, Hq, Hkv, d, Tn, lens = 2, 8, 2, 128, 9, [40, 7]
    c, q, k, v, parents = _case(B, Hq, Hkv, d, Tn, lens, 64, 0, True, "random", seed=2)
    acc = [Tn - 1, 3]
    cd, ce = H.to_dev(c), H.to_dev(c)
    qd, kd, vd = q.to(dev()), k.to(dev()), v.to(dev())
    ld, pd, ad = H.i32(lens), H.i32(parents), H.i32(acc)
    out = torch.zeros(B, Hq, Tn, d, dtype=torch.bfloat16, device=dev())
    new = torch.zeros(B, dtype=torch.int32, device=dev())
    ws = torch.empty(csattn.tree_workspace_size(B, Hq, Hkv, Tn, 64, d), dtype=torch.uint8,
                     device=dev())
    scratch = H.to_dev(c)
    _step(scratch, qd, kd, vd, ld, pd, rope_base=10000.0)  # (warm)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        _step(cd, qd, kd, vd, ld, pd, out=out, rope_base=10000.0, workspace=ws)
        _commit(cd, ld, pd, ad, new)
    for x in (qd, kd, vd):
        x.mul_(-0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        gr.replay()
        want = _step(ce, qd, kd, vd, ld, pd, rope_base=10000.0)
        new2 = _commit(ce, ld, pd, ad)
    side.synchronize()
    csattn.check_status()
    assert H.same_bits(out, want) and new.tolist() == new2.tolist()
    for n in ("k", "v", "ks", "vs"):
        assert H.same_bits(cd[n], ce[n])
