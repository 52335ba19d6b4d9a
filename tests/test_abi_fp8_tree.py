"""Host-side refusals of the 8-bit cache and token-tree calls, their workspace sizes, and the
oracle's e4m3 and tree rules.  No GPU: every call here fails before any CUDA call."""
import numpy as np
import pytest
import torch

from oracle import attn as OA

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import transformer_causal_self_gb300 as csattn
    return csattn.load_library()


BASE = dict(q=FAKE, kn=FAKE, vn=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, lens=FAKE,
            parents=FAKE, acc=FAKE + 0x1000, new=FAKE + 0x2000, out=FAKE, ko=FAKE, vo=FAKE, lse=None,
            B=2, Hq=4, Hkv=2, Tn=8, Lmax=256, Lout=200, page=16, pages=40, per=16, d=64, dtype=1,
            cache=2, base=10000.0, layout=0, scale=0.0, msl=200, splits=0, ws=FAKE, wb=1 << 30)


def call(lib, op, paged, **kw):
    a = dict(BASE)
    a.update(kw)
    cache = [a["k"], a["v"], a["ks"], a["vs"]] + ([a["table"]] if paged else [])
    size = [a["page"], a["pages"], a["per"]] if paged else [a["Lmax"]]
    rope, tail = [a["base"], a["layout"]], [a["scale"], a["msl"], a["splits"], a["ws"], a["wb"]]
    sfx = "_paged" if paged else ""
    if op == "append":
        return getattr(lib, "csattn_cache_append_fp8" + sfx)(
            a["kn"], a["vn"], *cache, a["lens"], a["B"], a["Hkv"], a["Tn"], *size, a["d"],
            a["dtype"], *rope, None)
    if op == "read":
        return getattr(lib, "csattn_cache_read_fp8" + sfx)(
            *cache, a["lens"], a["ko"], a["vo"], a["B"], a["Hkv"], *size, a["Lout"], a["d"],
            a["dtype"], None)
    if op == "decode":
        return getattr(lib, "csattn_attn_decode_fp8" + sfx)(
            a["q"], *cache, a["lens"], a["out"], a["B"], a["Hq"], a["Hkv"], *size, a["d"],
            a["dtype"], *rope, *tail, None)
    if op == "tree":
        return getattr(lib, "csattn_attn_tree_step" + sfx)(
            a["q"], a["kn"], a["vn"], *cache, a["lens"], a["parents"], a["out"], a["lse"], a["B"],
            a["Hq"], a["Hkv"], a["Tn"], *size, a["d"], a["cache"], *rope, *tail, None)
    return getattr(lib, "csattn_tree_commit" + sfx)(
        *cache, a["lens"], a["parents"], a["acc"], a["new"], a["B"], a["Hkv"], a["Tn"], *size,
        a["d"], a["cache"], None)


OPS = ["append", "read", "decode", "tree", "commit"]
NAMES = dict(append=b"cache_append_fp8", read=b"cache_read_fp8", decode=b"attn_decode_fp8",
             tree=b"attn_tree_step", commit=b"tree_commit")


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("ops,kw,status", [
    (OPS, dict(k=None), -1),
    (OPS, dict(v=None), -1),
    (OPS, dict(ks=None), -1),
    (OPS, dict(lens=None), -1),
    (OPS, dict(k=FAKE + 8), -1),
    (OPS, dict(lens=FAKE + 2), -1),
    (OPS, dict(B=0), -1),
    (OPS, dict(Hkv=0), -1),
    (OPS, dict(d=96), -2),
    (OPS, dict(d=32), -2),
    (OPS, dict(B=70000), -2),
    (["append"], dict(kn=None), -1),
    (["append"], dict(vn=FAKE + 4), -1),
    (["append", "commit"], dict(Tn=0), -1),
    (["append", "commit"], dict(Tn=257), -1),
    (["append", "read", "decode"], dict(dtype=0), -2),
    (["append", "read", "decode"], dict(dtype=2), -1),
    (["append", "decode", "tree"], dict(layout=4), -1),
    (["append", "decode", "tree"], dict(base=float("inf")), -1),
    (["read"], dict(ko=None), -1),
    (["read"], dict(vo=FAKE + 2), -1),
    (["read"], dict(Lout=0), -1),
    (["read"], dict(Lout=1 << 24), -2),
    (["decode", "tree"], dict(q=None), -1),
    (["decode", "tree"], dict(out=FAKE + 8), -1),
    (["decode", "tree"], dict(Hq=5), -1),
    (["decode", "tree"], dict(Hq=0), -1),
    (["decode", "tree"], dict(msl=257), -1),
    (["decode"], dict(msl=0), -1),
    (["tree"], dict(msl=7), -1),
    (["decode", "tree"], dict(splits=-1), -1),
    (["decode", "tree"], dict(scale=float("nan")), -1),
    (["decode", "tree"], dict(ws=None), -5),
    (["decode", "tree"], dict(ws=FAKE + 4), -5),
    (["decode", "tree"], dict(wb=64), -5),
    (["tree"], dict(Tn=0), -1),
    (["tree"], dict(Tn=300), -2),
    (["tree"], dict(parents=None), -1),
    (["tree"], dict(parents=FAKE + 1), -1),
    (["tree"], dict(lse=FAKE + 2), -1),
    (["tree", "commit"], dict(cache=0), -2),
    (["tree", "commit"], dict(cache=3), -1),
    (["tree", "commit"], dict(cache=1), -1),                 # bf16 with scales
    (["commit"], dict(acc=None), -1),
    (["commit"], dict(new=None), -1),
    (["commit"], dict(new=FAKE), -1),                        # overlaps the lengths
    (["commit"], dict(new=BASE["acc"] + 4), -1),
    (["commit"], dict(parents=BASE["new"] - 60), -1),
])
def test_refusals(lib, ops, kw, status, paged):
    for op in ops:
        assert call(lib, op, paged, **kw) == status, (op, kw, lib.csattn_last_error())
        assert NAMES[op] + (b"_paged" if paged else b"") + b":" in lib.csattn_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), -1), (dict(table=FAKE + 2), -1), (dict(page=8), -1), (dict(page=48), -1),
    (dict(page=65600), -1), (dict(pages=0), -1), (dict(per=0), -1), (dict(pages=1 << 30), -2),
    (dict(page=65536, per=1 << 15), -2),
])
def test_page_refusals(lib, kw, status):
    for op in OPS:
        assert call(lib, op, True, **kw) == status, (op, kw, lib.csattn_last_error())


@pytest.mark.parametrize("kw", [dict(Lmax=60000), dict(Lmax=60000, msl=50000)])
def test_rope_positions(lib, kw):
    ops = ["append"] + (["decode", "tree"] if "msl" in kw else [])
    for op in ops:
        assert call(lib, op, False, **kw) == -2
        assert b"RoPE" in lib.csattn_last_error()


def test_workspace_sizes_cover_every_length():
    import transformer_causal_self_gb300 as csattn
    # a call with less than the workspace it names is refused: find what each length needs by
    # offering 0 bytes and reading the message
    import re
    lib_ = csattn.load_library()
    for op, size in (("decode", lambda a, n: csattn.decode_fp8_workspace_size(*a, 64, n)),
                     ("tree", lambda a, n: csattn.tree_workspace_size(a[0], a[1], a[2], 8, a[3], 64,
                                                                      n))):
        for B, Hq, Hkv, Lmax in ((1, 8, 8, 4096), (1, 4, 1, 100), (64, 32, 8, 8192), (3, 7, 1, 30000)):
            for n in (0, 1, 3, 50):
                have = size((B, Hq, Hkv, Lmax), n)
                for msl in (8, 63, 64, 65, 255, 256, 257, Lmax // 2 + 1, Lmax - 1, Lmax):
                    if msl > Lmax:
                        continue
                    assert call(lib_, op, False, B=B, Hq=Hq, Hkv=Hkv, Lmax=Lmax, msl=msl, splits=n,
                                wb=0) == -5
                    need = int(re.search(rb"workspace of (\d+) bytes",
                                         lib_.csattn_last_error()).group(1))
                    assert 0 < need <= have, (op, B, Hq, Hkv, Lmax, n, msl, need, have)
    assert csattn.decode_fp8_workspace_size(0, 8, 8, 100, 64) == 0
    assert csattn.decode_fp8_workspace_size(1, 7, 2, 100, 64) == 0
    assert csattn.tree_workspace_size(1, 8, 8, 257, 1000, 64) == 0


@pytest.mark.parametrize("d,Hq,Tn", [(64, 8, 1), (128, 8, 2), (128, 12, 1), (128, 8, 12), (64, 32, 64)])
def test_tree_workspace_covers_both_caches(lib, d, Hq, Tn):
    import re
    for splits in (0, 3):
        for msl in (256, 3000, 30000):
            have = lib.csattn_tree_workspace_size(4, Hq, 1, Tn, 30000, d, splits)
            for cache, scales in ((1, None), (2, FAKE)):
                assert call(lib, "tree", False, B=4, Hq=Hq, Hkv=1, Tn=Tn, Lmax=30000, msl=msl, d=d,
                            cache=cache, ks=scales, vs=scales, splits=splits, wb=0) == -5
                need = int(re.search(rb"workspace of (\d+) bytes",
                                     lib.csattn_last_error()).group(1))
                assert 0 < need <= have


def test_sizes_past_the_limits(lib):
    for kw in (dict(Hq=2 * ((1 << 20) + 2), wb=1 << 60), dict(B=65535, Hq=8192, Tn=8, wb=1 << 60)):
        for op in (["decode", "tree"] if "B" not in kw else ["tree"]):
            assert call(lib, op, False, **kw) == -2, op
            assert b"too large" in lib.csattn_last_error()
    assert lib.csattn_decode_fp8_workspace_size(1, 1 << 21, 1, 100, 64, 0) == 0
    assert lib.csattn_decode_fp8_workspace_size(1 << 20, 8, 8, 100, 64, 0) == 0
    assert lib.csattn_decode_fp8_workspace_size(1, 8, 8, 1 << 30, 64, 0) == 0
    assert lib.csattn_decode_fp8_workspace_size(1, 8, 8, 100, 96, 0) == 0
    assert lib.csattn_tree_workspace_size(65535, 8192, 8, 8, 100, 64, 0) == 0


def test_binding_refuses_wrong_tensors():
    """CPU tensors, before anything is launched."""
    import transformer_causal_self_gb300 as csattn
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 2, 8, 64, dtype=torch.float8_e4m3fn)
    s = torch.zeros(1, 2, 8, dtype=torch.uint8)
    i = torch.zeros(1, dtype=torch.int32)
    p = torch.zeros(1, 3, dtype=torch.int32)
    for f in (lambda: csattn.cache_append_fp8(x, x, c, c, s, s, i),
              lambda: csattn.cache_read_fp8(c, c, s, s, i),
              lambda: csattn.attn_decode_fp8(x[:, :, :1], c, c, s, s, i),
              lambda: csattn.attn_tree_step(x, x, x, c, c, i, p, k_scale=s, v_scale=s),
              lambda: csattn.tree_commit(c, c, i, p, i, k_scale=s, v_scale=s)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


# ------------------------------------------------------------------ the oracle's own rules
def test_e4m3_rounding_matches_the_type():
    codes = np.arange(256, dtype=np.uint8)
    vals = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    fin = np.unique(vals[np.isfinite(vals)])
    assert np.array_equal(OA.round_to_e4m3(fin), fin)
    mids = (fin[1:] + fin[:-1]) / 2
    for x in np.concatenate([mids, mids * (1 + 1e-9), mids * (1 - 1e-9)]):
        d = np.abs(fin - x)
        near = fin[d == d.min()]
        y = float(OA.round_to_e4m3(x))
        assert y in near
        if len(near) == 2:  # a tie goes to the even code
            code = torch.tensor(y).to(torch.float8_e4m3fn).view(torch.uint8).item()
            assert code % 2 == 0
    assert np.all(np.isnan(OA.round_to_e4m3([np.inf, -np.inf, np.nan])))


@pytest.mark.parametrize("rotated", [False, True])
def test_scale_rule_from_bf16_bits(rotated):
    """The kernels' integer rule, code = exponent field - 8 (+ 1 above a mantissa), clamped to
    [3, 247], is the definition of e4m3_exponents for every finite bf16 magnitude."""
    bits = np.arange(0x7F80, dtype=np.int32)
    x = torch.from_numpy((bits << 16).astype(np.int32)).view(torch.float32).double().numpy()
    code = np.clip((bits >> 7) - 8 + ((bits & 0x7F) > (30 if rotated else 96)), 3, 247)
    assert np.array_equal(OA.e4m3_exponents(x[:, None], rotated) + 127, code)
    # nothing saturates but the very largest rows, whose scale is at its limit
    room = np.sqrt(2.0) if rotated else 1.0
    assert np.all(x * room <= 448.0 * 2.0 ** (code - 127.0))


def test_tree_rules():
    anc = OA.tree_ancestors([-1, 0, 0, 2, -2, -1])
    assert [list(np.nonzero(r)[0]) for r in anc] == [[0], [0, 1], [0, 2], [0, 2, 3], [], [5]]
    assert OA.tree_path([-1, 0, 0, 2, -2, -1], 3) == [0, 2, 3]
    assert OA.tree_path([-1], -1) == []
    for bad in ([0], [-1, 1], [-1, -3], [-2, 0]):
        with pytest.raises(ValueError):
            OA.tree_ancestors(bad)


def test_tree_attention_of_a_chain_is_causal_attention():
    """A chain after L rows sees what a chunk of queries after a cached prefix sees."""
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(2, 5, 16)), rng.normal(size=(1, 12, 16)), rng.normal(size=(1, 12, 16))
    out, lse = OA.tree_attention(q, k, v, 7, OA.tree_ancestors([-1, 0, 1, 2, 3]))
    for t in range(5):
        z = q[:, t] @ k[0, :8 + t].T / 4.0
        assert np.allclose(out[:, t], OA.softmax_rows(z) @ v[0, :8 + t], atol=1e-12)
        assert np.allclose(lse[:, t], np.log(np.exp(z).sum(-1)), atol=1e-12)

