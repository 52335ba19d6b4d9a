"""Token trees with many query rows per KV head, long prefixes and many sequences, and 8-bit
decode beside them, against float64 (tolerances: tests/test_gpu_tree.py); calls at the same time
and captured calls against the same calls one after another, bit by bit."""
import threading

import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from tests import fp8_helpers as H
from tests import test_gpu_tree as T
from tests.gpu_helpers import assert_bf16_close, dev, to_np

pytestmark = pytest.mark.gpu


def _run_and_check(case, lens, base, **kw):
    c, q, k, v, parents = case
    cd = H.to_dev(c)
    lse = torch.zeros(q.shape[:3], device=dev())
    out = T._step(cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32(lens), H.i32(parents), lse=lse,
                  rope_base=base, **kw)
    csattn.check_status()
    T._check(c, H.to_cpu(cd), q, k, v, parents, lens, out, lse, base, "split_half")
    return out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,Hq,Tn", [(128, 8, 64), (64, 7, 40), (128, 5, 52), (64, 16, 33)])
def test_more_query_rows_than_a_block(d, Hq, Tn, e4m3):
    """512, 280, 260 and 528 rows: whole, begun and all but empty second and third blocks."""
    lens = [0, 130, 300]
    case = T._case(3, Hq, 1, d, Tn, lens, 300 + Tn, 0, e4m3, "random", seed=Hq + Tn)
    _run_and_check(case, lens, 10000.0)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page,d,Hq,Tn", [(16, 128, 8, 12), (32, 64, 8, 12), (64, 128, 4, 70),
                                          (192, 64, 8, 12), (256, 128, 8, 12), (0, 128, 8, 12),
                                          (32, 128, 2, 7)])
def test_long_prefix(page, d, Hq, Tn, e4m3):
    """Prefixes of many tiles that the CTAs share, pages smaller and larger than a tile, and ends
    inside of them."""
    lens = [1500, 1024, 767]
    case = T._case(3, Hq, 1, d, Tn, lens, 1600, page, e4m3, "random", seed=page + d)
    _run_and_check(case, lens, 10000.0)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,Tn", [(2, 3), (4, 9)])
def test_many_sequences(Hq, Tn, e4m3):
    lens = [(37 * b) % 41 if b % 3 else 0 for b in range(75)]
    case = T._case(75, Hq, 1, 64, Tn, lens, 41 + Tn, 0, e4m3, "padded", seed=Hq)
    _run_and_check(case, lens, 0.0)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv,Tn,page,kind", [(64, 2, 1, 33, 16, "padded"),
                                                   (128, 3, 3, 18, 0, "random"),
                                                   (128, 10, 2, 11, 32, "flat")])
def test_many_drafts(d, Hq, Hkv, Tn, page, kind, e4m3):
    """More drafts than CTAs at once: several of them in one, the last ones of a sequence fewer."""
    lens = [(37 * b) % 41 for b in range(80)]
    case = T._case(80, Hq, Hkv, d, Tn, lens, 41 + Tn, page, e4m3, kind, seed=Tn)
    _run_and_check(case, lens, 10000.0)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 0)])
def test_decode_many_sequences(d, page):
    lens = [1 + (37 * b) % 150 for b in range(75)]
    c, q, _, _, _ = T._case(75, 4, 2, d, 1, lens, 150, page, True, T.CHAIN, seed=d)
    cd = H.to_dev(c)
    if page:
        out = csattn.attn_decode_fp8_paged(q.to(dev()), cd["k"], cd["v"], cd["ks"], cd["vs"],
                                           cd["table"], H.i32(lens))
    else:
        out = csattn.attn_decode_fp8(q.to(dev()), cd["k"], cd["v"], cd["ks"], cd["vs"],
                                     H.i32(lens))
    csattn.check_status()
    ref = np.zeros(tuple(q.shape))
    for b, L in enumerate(lens):
        kk, vv = H.rows(c, b, L)
        s = np.einsum("gjd,gkd->gjk", q[b].double().numpy().reshape(2, 2, d), kk) / np.sqrt(d)
        w = np.exp(s - s.max(-1, keepdims=True))
        ref[b] = (w / w.sum(-1, keepdims=True) @ vv).reshape(4, 1, d)
    assert_bf16_close(to_np(out), ref, "decode")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,L", [(1, 4, 1, 20000), (1, 4, 2, 3000), (2, 8, 4, 1500),
                                        (4, 8, 8, 600), (16, 16, 8, 130), (130, 64, 8, 20)])
def test_decode_from_one_to_many_partial_results(B, Hq, Hkv, L, d):
    """Rows with hundreds of partial results to merge (one long sequence) down to a few."""
    g = H.gen(L + d)
    k, v = (torch.randn(B, Hkv, L, d, generator=g, dtype=torch.float32).to(torch.bfloat16).to(dev())
            for _ in range(2))
    q = torch.randn(B, Hq, 1, d, generator=g).to(torch.bfloat16).to(dev())
    c = {n: x.to(dev()) for n, x in H.empty_cache(B, Hkv, L, d, 0, True, seed=1).items()
         if isinstance(x, torch.Tensor)}
    csattn.cache_append_fp8(k, v, c["k"], c["v"], c["ks"], c["vs"], H.i32([0] * B))
    lens = [max(1, L - 7 * b) for b in range(B)]
    out = csattn.attn_decode_fp8(q, c["k"], c["v"], c["ks"], c["vs"], H.i32(lens))
    csattn.check_status()
    kk, vv = (c[n].double() * torch.exp2(c[n + "s"].double() - 127)[..., None] for n in ("k", "v"))
    s = torch.einsum("bgjd,bgkd->bgjk", q.double().view(B, Hkv, Hq // Hkv, d), kk) / np.sqrt(d)
    s.masked_fill_(torch.arange(L, device=dev()) >= torch.tensor(lens, device=dev()).view(B, 1, 1, 1),
                   float("-inf"))
    ref = (torch.softmax(s, -1) @ vv).view(B, Hq, 1, d)
    assert_bf16_close(to_np(out), ref.cpu().numpy(), "decode")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,Tn", [(2, 6), (8, 12), (8, 40)])
def test_rows_of_zeros(Hq, Tn, e4m3):
    """Zero queries (a plain mean), keys and values."""
    lens = [200, 3]
    c, q, k, v, parents = T._case(2, Hq, 1, 128, Tn, lens, 260, 0, e4m3, "random", seed=9)
    q[0, :, Tn // 2] = 0
    k[:, :, 1::2] = 0
    v[:, :, ::2] = 0
    zero = torch.zeros(1, 130, 128, dtype=torch.bfloat16)
    H.set_rows(c, 0, 0, zero, zero)
    _run_and_check((c, q, k, v, parents), lens, 10000.0)


@pytest.mark.parametrize("shift", [-60, 60])
@pytest.mark.parametrize("Hq,Tn", [(2, 6), (8, 12), (8, 40)])
def test_powers_of_two(Hq, Tn, shift):
    """Values times 2^shift and keys times 2^shift with the scale 2^-shift of it: scales of an
    8-bit cache that move the outputs by that power.

    Up to 16 query rows the weights' exponents are the same numbers, so the outputs are the same
    bits.  Above, the tile's value exponent is part of a weight's exponent x + e - R; sums of
    numbers up to 2^7 are off by 2^-17 each, so a weight by 2^-16 relative before it is rounded
    to f16 (half a step: 2^-11).  Two evaluations differ by at most one step of that rounding,
    2^-10 relative, the outputs by 2^-10 of the largest value and a step of bf16 (2^-8 of the
    output for half of it): within the tolerances of one evaluation against the exact values.
    """
    d, lens = 64, [200, 3]
    c, q, k, v, parents = T._case(2, Hq, 1, d, Tn, lens, 260, 0, True, "random", seed=4)
    outs = []
    for s in (0, shift):
        cd = H.to_dev(c)
        for n in ("ks", "vs"):
            for b, L in enumerate(lens):
                cd[n][b, :, :L] += s
        f = 2.0 ** s
        outs.append(T._step(cd, q.to(dev()), (k * f).to(dev()), (v * f).to(dev()), H.i32(lens),
                            H.i32(parents), rope_base=10000.0, scale=0.125 / f))
    csattn.check_status()
    assert torch.isfinite(outs[1]).all()
    back = outs[1] * 2.0 ** -shift
    if Hq * Tn <= 16:
        assert H.same_bits(outs[0], back)
    else:
        assert_bf16_close(to_np(outs[0]), to_np(back), "powers of two")


@pytest.mark.parametrize("Hq,Tn", [(2, 6), (8, 12), (8, 40)])
def test_scale_bytes_at_odd_addresses(Hq, Tn):
    lens, room = [300, 77], 361
    c, q, k, v, parents = T._case(2, Hq, 1, 128, Tn, lens, room, 0, True, "random", seed=6)
    args = (q.to(dev()), k.to(dev()), v.to(dev()), H.i32(lens), H.i32(parents))
    one, two = H.to_dev(c), H.to_dev(c)
    for n in ("ks", "vs"):
        x = torch.empty(two[n].numel() + 1, dtype=torch.uint8, device=dev())[1:].view(two[n].shape)
        two[n] = x.copy_(two[n])
    a = T._step(one, *args, rope_base=10000.0)
    b = T._step(two, *args, rope_base=10000.0)
    csattn.check_status()
    assert H.same_bits(a, b)
    for n in ("k", "v", "ks", "vs"):
        assert H.same_bits(one[n], two[n])


def _calls(seed, e4m3):
    """A tree step (many rows), a tree step (few rows) and a decode, each with its own caches and
    the output it gives alone: [(call, output)]."""
    made = []
    for Hq, Tn, d in ((8, 24, 128), (2, 4, 64)):
        lens = [900, 333]
        c, q, k, v, p = T._case(2, Hq, 1, d, Tn, lens, 1000, 64, e4m3, "random", seed=seed + Tn)
        cd = H.to_dev(c)
        args = (cd, q.to(dev()), k.to(dev()), v.to(dev()), H.i32(lens), H.i32(p))
        made.append(lambda args=args: T._step(*args, rope_base=10000.0))
    c, q, _, _, _ = T._case(2, 8, 1, 128, 1, [900, 333], 1000, 0, True, T.CHAIN, seed=seed)
    cd, qd, ld = H.to_dev(c), q.to(dev()), H.i32([900, 333])
    made.append(lambda: csattn.attn_decode_fp8(qd, cd["k"], cd["v"], cd["ks"], cd["vs"], ld,
                                               rope_base=10000.0))
    # (a step writes the same rows each time it is run)
    out = [(f, f().clone()) for f in made]
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("e4m3", [False, True])
def test_calls_on_several_streams_and_threads(e4m3):
    sets = [_calls(seed, e4m3) for seed in (1, 2, 3)]
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(10):
                got[i].append([f() for f, _ in sets[i]])

    work(0)   # one thread, two streams ...
    work(1)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]  # ... and three
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    csattn.check_status()
    for i, s in enumerate(sets):
        assert len(got[i]) == (10 if i == 2 else 20)
        for outs in got[i]:
            for out, (_, want) in zip(outs, s):
                assert H.same_bits(out, want)


def test_two_graphs_at_once_beside_eager_calls():
    """Calls that bring no workspace, captured into two graphs: replayed side by side, with eager
    calls in between, they do not touch one another's."""
    sets = [_calls(seed, True) for seed in (4, 5, 6)]
    graphs, outs = [], []
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([f() for f, _ in s])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    eager = []
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager.append([f() for f, _ in sets[2]])
    torch.cuda.synchronize()
    csattn.check_status()
    for s, got in list(zip(sets, outs)) + [(sets[2], e) for e in eager]:
        for out, (_, want) in zip(got, s):
            assert H.same_bits(out, want)


def test_stream_argument():
    """The `stream` argument, from a thread whose current stream is another."""
    s = torch.cuda.Stream()
    lens = [500, 20]
    c, q, k, v, p = T._case(2, 8, 1, 128, 24, lens, 600, 64, True, "random", seed=8)
    one, two = H.to_dev(c), H.to_dev(c)
    args = (q.to(dev()), k.to(dev()), v.to(dev()), H.i32(lens), H.i32(p))
    a = T._step(one, *args, rope_base=10000.0)
    torch.cuda.synchronize()
    b = T._step(two, *args, rope_base=10000.0, stream=s)
    e = T._step(two, *args, rope_base=10000.0, stream=s.cuda_stream)
    s.synchronize()
    csattn.check_status()
    assert H.same_bits(a, b) and H.same_bits(a, e)


@pytest.mark.parametrize("graph", [False, True])
def test_calls_behind_kernels_that_write_their_inputs(graph):
    """A generation loop on one stream without a wait on the host: every call's inputs are written
    by the kernel right before it (their blocks may be scheduled while that one still runs)."""
    B, Hq, Hkv, d, Tn, steps, base = 2, 8, 2, 128, 12, 12, 10000.0
    g = H.gen(11)
    xs = [[torch.randn(B, h, n, d, generator=g).to(torch.bfloat16).to(dev())
           for h, n in ((Hkv, 1), (Hkv, 1), (Hq, 1), (Hq, Tn), (Hkv, Tn), (Hkv, Tn))]
          for _ in range(steps)]
    parents = H.i32([[t // 2 - 1 for t in range(Tn)]] * B)

    c0 = {n: x.to(dev()) for n, x in H.empty_cache(B, Hkv, 256, d, 0, True, seed=2).items()
          if isinstance(x, torch.Tensor)}
    zero, first = H.i32([0, 0]), H.i32([0, 3])

    def loop(wait):
        def do(f):
            if wait:
                torch.cuda.synchronize()
            return f()

        c = {n: x.clone() for n, x in c0.items()}
        cache, scales = (c["k"], c["v"], c["ks"], c["vs"]), dict(k_scale=c["ks"], v_scale=c["vs"])
        buf = [torch.zeros_like(x) for x in xs[0]]
        lens, acc, outs = first.clone(), zero.clone(), []
        prompt = torch.ones(B, Hkv, 3, d, dtype=torch.bfloat16, device=dev())
        do(lambda: csattn.cache_append_fp8(prompt, prompt, *cache, zero))
        for i, x in enumerate(xs):
            for to, new in zip(buf, x):
                do(lambda: to.copy_(new))
            do(lambda: csattn.cache_append_fp8(buf[0], buf[1], *cache, lens, rope_base=base))
            do(lambda: lens.add_(1))
            outs.append(do(lambda: csattn.attn_decode_fp8(buf[2], *cache, lens, rope_base=base)))
            outs.append(do(lambda: csattn.attn_tree_step(buf[3], buf[4], buf[5], c["k"], c["v"],
                                                         lens, parents, rope_base=base, **scales)))
            do(lambda: acc.fill_(i % Tn))
            new_lens = do(lambda: csattn.tree_commit(c["k"], c["v"], lens, parents, acc, **scales))
            do(lambda: lens.copy_(new_lens))
        ko, vo = (torch.zeros(B, Hkv, 256, d, dtype=torch.bfloat16, device=dev()) for _ in range(2))
        do(lambda: csattn.cache_read_fp8(*cache, lens, ko, vo))
        return outs + [ko, vo, lens]

    want = loop(True)
    if graph:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got = loop(False)
        gr.replay()
        gr.replay()
    else:
        got = loop(False)
    torch.cuda.synchronize()
    csattn.check_status()
    for a, b in zip(got, want):
        assert H.same_bits(a, b)
