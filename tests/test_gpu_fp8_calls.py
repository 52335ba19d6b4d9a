"""Calls of the 8-bit cache and of token trees in their less usual circumstances: waits that
run out, memory that another stream still uses, pages and lengths out of range, streams of other
libraries, odd numbers of rows; and the bound of the log-sum-exp over a bf16 cache."""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import attn as OA
from tests import fp8_helpers as H
from tests import test_gpu_tree as T
from tests.gpu_helpers import assert_bf16_close, dev, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["decode", "tree", "tree_8bit", "wide", "wide_8bit", "pair_8bit"])
def test_a_wait_that_runs_out_is_reported(call):
    """Many sequences, so that every CTA begins several segments; a workspace of bytes that are no
    slots of it.  The merge finds what every segment left for it and the GPU stays usable."""
    B, Hkv, d, L = 300, 2, 64, 100
    Hq, Tn = {"wide": (16, 6), "wide_8bit": (16, 6), "pair_8bit": (16, 20)}.get(call, (4, 2))
    g = H.gen(1)
    c = H.to_dev(H.empty_cache(B, Hkv, L + Tn, d, 0, call.endswith("8bit") or call == "decode", 1))
    for n in ("k", "v"):
        H.raw(c[n]).zero_()
    for n in [n for n in ("ks", "vs") if n in c]:
        c[n].fill_(120)
    lens = H.i32([L] * B)
    q = torch.randn(B, Hq, Tn, d, generator=g).to(torch.bfloat16).to(dev())
    k, v = (torch.randn(B, Hkv, Tn, d, generator=g).to(torch.bfloat16).to(dev()) for _ in range(2))
    parents = H.i32([[-1] * Tn] * B)
    if call == "decode":
        need = csattn.decode_fp8_workspace_size(B, Hq, Hkv, L + Tn, d)
    else:
        need = csattn.tree_workspace_size(B, Hq, Hkv, Tn, L + Tn, d)

    def run():
        ws = torch.full((need,), 0x7E, dtype=torch.uint8, device=dev())
        if call == "decode":
            return csattn.attn_decode_fp8(q[:, :, :1].contiguous(), c["k"], c["v"], c["ks"],
                                          c["vs"], lens, workspace=ws)
        return T._step(c, q, k, v, lens, parents, workspace=ws)

    want = run().clone()
    csattn.check_status()
    csattn.selftest_lost_arrival()
    run()
    with pytest.raises(csattn.CsattnError) as e:
        csattn.check_status()
    assert e.value.status == -4
    again = run()
    csattn.check_status()
    assert H.same_bits(again, want)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("which", ["out", "workspace"])
def test_stream_argument_beside_memory_in_use(which, raw):
    """A block that was freed while work queued on the current stream still reads it does not
    become the output or workspace of a call on another stream."""
    B, Hq, d, Tn, L = 2, 64, 128, 64, 500
    c, q, k, v, p = T._case(B, Hq, 8, d, Tn, [L] * B, 600, 64, False, "random", seed=8)
    cd = H.to_dev(c)
    args = (cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32([L] * B), H.i32(p))
    want = T._step(*args, rope_base=10000.0)
    need = csattn.tree_workspace_size(B, Hq, 8, Tn, cd["table"].shape[1] * 64, d)
    given = (dict(workspace=torch.empty(need, dtype=torch.uint8, device=dev())) if which == "out"
             else dict(out=torch.empty_like(want)))
    size = want.numel() * 2 if which == "out" else need
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.full((size,), 7, dtype=torch.uint8, device=dev())
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # (about 50 ms)
    y.copy_(x)
    del x
    got = T._step(*args, rope_base=10000.0, stream=s.cuda_stream if raw else s, **given)
    torch.cuda.synchronize()
    csattn.check_status()
    assert H.same_bits(got, want)
    assert bool((y == 7).all())


def _refused():
    with pytest.raises(csattn.CsattnError) as e:
        csattn.check_status()
    assert e.value.status == -6


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Tn,Hq", [(5, 2), (20, 4)])
def test_draft_rows_on_a_page_outside_the_pool_read_as_zeros(Tn, Hq, e4m3):
    """Their values do not reach the outputs, infinities and NaN among them neither."""
    L, page, d = 16, 16, 64
    c, q, k, v, _ = T._case(1, Hq, 1, d, Tn, [L], 48, page, e4m3, "flat", seed=5)
    k[:] = 0  # (what is read as zero as well: the outputs with and without the page compare)
    v[0, 0, 1, 3], v[0, 0, 2, 4] = float("inf"), float("nan")
    cd = H.to_dev(c)
    cd["table"][0, 1] = -1
    out = T._step(cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32([L]), H.i32([[-1] * Tn]))
    _refused()
    zero = H.to_dev(c)
    v0 = v.clone()
    v0[:, :, :16] = 0
    if Tn > 16:
        v0[:, :, 16:] = v[:, :, 16:]
    want = T._step(zero, q.to(dev()), k.to(dev()), v0.to(dev()), H.i32([L]), H.i32([[-1] * Tn]))
    csattn.check_status()
    assert torch.isfinite(out).all()
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6


def test_every_length_out_of_range_is_reported():
    d, B = 64, 3
    c, q, _, _, _ = T._case(B, 2, 1, d, 1, [10] * B, 32, 0, True, T.CHAIN, seed=6)
    cd = H.to_dev(c)
    for bad in (0, -1, -2, 33, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1):
        out = csattn.attn_decode_fp8(q.to(dev()), cd["k"], cd["v"], cd["ks"], cd["vs"],
                                     H.i32([10, bad, 10]))
        _refused()
        assert torch.all(out[1] == 0) and torch.isfinite(out).all() and torch.any(out[2] != 0)
        c2, q2, k2, v2, _ = T._case(B, 2, 1, d, 3, [10] * B, 32, 0, True, T.CHAIN, seed=6)
        if bad in (0,):
            continue
        out = T._step(H.to_dev(c2), q2.to(dev()), k2.to(dev()), v2.to(dev()),
                      H.i32([10, bad, 10]), H.i32([[-1, 0, 1]] * B))
        _refused()
        assert torch.all(out[1] == 0)


def test_workspaces_are_kept_for_torch_streams_and_can_be_let_go():
    c, q, _, _, _ = T._case(1, 4, 1, 64, 1, [40], 64, 0, True, T.CHAIN, seed=3)
    cd, qd, lens = H.to_dev(c), q.to(dev()), H.i32([40])

    def run():
        return csattn.attn_decode_fp8(qd, cd["k"], cd["v"], cd["ks"], cd["vs"], lens)

    csattn.release_workspaces()
    want = run()
    assert len(csattn._kept.__dict__) == 1
    mine = torch.cuda.Stream()
    with torch.cuda.stream(mine):
        mine.wait_stream(torch.cuda.default_stream())
        assert H.same_bits(run(), want)
    assert len(csattn._kept.__dict__) == 2
    # a stream that torch does not own: no workspace is kept under its handle
    other = torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream)
    with torch.cuda.stream(other):
        other.wait_stream(torch.cuda.default_stream())
        assert H.same_bits(run(), want)
    assert len(csattn._kept.__dict__) == 2
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    csattn.release_workspaces()
    assert not csattn._kept.__dict__ and torch.cuda.memory_allocated() < held
    assert H.same_bits(run(), want)
    csattn.check_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,heads", [(1, 1), (1, 3), (3, 5), (1, 4097)])
def test_odd_numbers_of_rows(B, heads, d):
    """The last block of the merge has fewer rows than it has room for (and a barrier, but for the
    last case)."""
    L = 20
    c, q, _, _, _ = T._case(B, heads, heads, d, 1, [L] * B, 24, 0, True, T.CHAIN, seed=heads)
    cd = H.to_dev(c)
    out = csattn.attn_decode_fp8(q.to(dev()), cd["k"], cd["v"], cd["ks"], cd["vs"], H.i32([L] * B))
    csattn.check_status()
    kk, vv = (torch.stack([torch.from_numpy(H.rows(c, b, L)[i]) for b in range(B)])
              for i in range(2))
    s = torch.einsum("bhqd,bhkd->bhqk", q.double(), kk) / d ** 0.5
    ref = torch.softmax(s, -1) @ vv
    assert_bf16_close(to_np(out), ref.numpy(), "decode")


def test_stream_argument_in_a_capture():
    """A stream that the capture has been forked to: its outputs and workspaces are the graph's."""
    B, L = 2, 200
    c, q, k, v, p = T._case(B, 8, 1, 64, 20, [L] * B, 300, 64, True, "random", seed=9)
    cd, ce = H.to_dev(c), H.to_dev(c)
    args = (q.to(dev()), k.to(dev()), v.to(dev()), H.i32([L] * B), H.i32(p))
    want = T._step(ce, *args, rope_base=10000.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        side.wait_stream(torch.cuda.current_stream())
        out = T._step(cd, *args, rope_base=10000.0, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        two = T._step(cd, *args, rope_base=10000.0, stream=torch.cuda.current_stream())
        both = out + two
    for _ in range(3):
        gr.replay()
        # (calls in between, which take memory from the same streams)
        T._step(ce, *args, rope_base=10000.0, stream=side)
        T._step(ce, *args, rope_base=10000.0)
    torch.cuda.synchronize()
    csattn.check_status()
    assert H.same_bits(out, want) and H.same_bits(two, want)
    assert H.same_bits(both, want + want)


def _rotation_ties(x, pos, base, layout):
    """Rotated queries x [Hq, T, d] in float64, and for each channel the bf16 step that a
    rotation in fp32 may fall off by: its angles' sine and cosine are good to 2^-20, so that a value
    within 2^-19 of its pair's length of the middle of two bf16 numbers may go to either."""
    r = OA.rope_rotate(x, pos, base, layout)
    half = x.shape[-1] // 2
    if layout == "split_half":
        pair = np.tile(np.hypot(x[..., :half], x[..., half:]), 2)
    else:
        pair = np.repeat(np.hypot(x[..., 0::2], x[..., 1::2]), 2, axis=-1)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -126))) - 7)
    off = np.abs(np.abs(r) / step - np.floor(np.abs(r) / step) - 0.5) * step
    return r, np.where(off <= 2.0 ** -19 * pair, step, 0.0)


@pytest.mark.parametrize("factor", [1.0, 4.0])
@pytest.mark.parametrize("Hq,Tn,d", [(4, 4, 128), (8, 40, 128), (4, 32, 64)])
def test_lse_over_a_bf16_cache(Hq, Tn, d, factor):
    """lse against float64 over many seeds: off by at most what the channels that fall on the other
    side of a bf16 tie move a score by, and the fp32 sums (2^-17 of sum |q_i k_i| * scale, and 2^-18
    for exponentials and logarithm)."""
    L = 300
    for seed in range(12):
        c, q, k, v, p = T._case(1, Hq, 1, d, Tn, [L], L + Tn, 0, False, "random", seed=seed)
        q = (q.float() * factor).to(torch.bfloat16)
        cd = H.to_dev(c)
        lse = torch.zeros(1, Hq, Tn, device=dev())
        T._step(cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32([L]), H.i32(p), lse=lse,
                rope_base=10000.0)
        csattn.check_status()
        anc = OA.tree_ancestors(p[0])
        pos = L + np.maximum(anc.sum(1) - 1, 0)
        kk, vv = H.rows(H.to_cpu(cd), 0, L + Tn)
        r, tie = _rotation_ties(q[0].double().numpy(), pos, 10000.0, "split_half")
        qr = OA.round_to_bf16(r)
        _, ref = OA.tree_attention(qr, kk, vv, L, anc)
        a = np.abs(kk[0]).T / np.sqrt(d)
        bound = (tie @ a).max(-1) + 2.0 ** -17 * (np.abs(qr) @ a).max(-1) + 2.0 ** -18
        off = np.abs(lse.double().cpu().numpy()[0] - ref) / bound
        assert off.max() <= 1.0, (seed, off.max())
