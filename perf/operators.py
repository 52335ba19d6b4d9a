"""Measured cases of the 8-bit KV cache and of speculative decoding over a cache.

Five operators of one serving path:

  append  a prompt chunk or a token quantised to e4m3 as it enters the cache
  read    a quantised prefix read back to bf16 (a chunked prefill reads it)
  decode  one new query per sequence over the quantised cache
  tree    a tree of drafted tokens: appended to the cache (bf16 or e4m3), and
          attention of every draft over the prefix and its own ancestors
  commit  the accepted path of a verified tree moved to follow the prefix

A cache is a pool of pages [num_pages, Hkv, page, d]; a contiguous cache
[B, Hkv, Lmax, d] is the same memory with one page per sequence.  A row in 8 bits
is e4m3 values times 2^(code - 127), one code per row and KV head.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BASE = 10000.0


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # the new token of a batch in generation enters the paged cache (latency)
        dict(name="append_token", op="append", B=64, Hkv=8, d=128, Tn=1, Lmin=64, Lmax=256,
             page=64, base=BASE, layout="split_half"),
        # whole prompts enter a contiguous cache at once
        dict(name="append_prompt", op="append", B=4, Hkv=8, d=128, Tn=4096, Lmin=0, Lmax=4160,
             page=0, base=BASE, layout="split_half"),
        # short ragged prefixes of a small multi-head model, 16-row pages
        dict(name="read_short", op="read", B=8, Hkv=12, d=64, Lmin=17, Lmax=1024, page=16),
        # one long prefix, read back for the next chunk of its prefill
        dict(name="read_long", op="read", B=1, Hkv=8, d=128, Lmin=32768, Lmax=32768, page=128),
        # a single user's generation step (latency)
        dict(name="decode_one", op="decode", B=1, Hq=32, Hkv=8, d=128, Lmin=1000, Lmax=1000,
             page=0, base=BASE, layout="split_half"),
        # a served batch with ragged lengths over a paged cache
        dict(name="decode_batch", op="decode", B=64, Hq=32, Hkv=8, d=128, Lmin=512, Lmax=8192,
             page=64, base=BASE, layout="split_half"),
        # a few long contexts
        dict(name="decode_long", op="decode", B=4, Hq=32, Hkv=8, d=128, Lmin=30000, Lmax=32768,
             page=256, base=500000.0, layout="split_half"),
        # a single user's draft of eight tokens (latency)
        dict(name="tree_one", op="tree", B=1, Hq=32, Hkv=8, d=128, Tn=8, Lmin=1000, Lmax=1000,
             page=0, cache="bf16", base=BASE, layout="split_half"),
        # a served batch with drafts of 32 tokens over the quantised paged cache
        dict(name="tree_batch_8bit", op="tree", B=16, Hq=32, Hkv=8, d=128, Tn=32, Lmin=512,
             Lmax=8192, page=64, cache="e4m3", base=BASE, layout="split_half"),
        # wide trees after long prefixes
        dict(name="tree_wide", op="tree", B=8, Hq=32, Hkv=8, d=128, Tn=64, Lmin=8192, Lmax=16384,
             page=128, cache="bf16", base=BASE, layout="split_half"),
        # the accepted path of a single user's draft (latency)
        dict(name="commit_one", op="commit", B=1, Hkv=8, d=128, Tn=8, Lmin=100, Lmax=192, page=0,
             cache="bf16"),
        # the accepted paths of a served batch, quantised pages
        dict(name="commit_batch", op="commit", B=256, Hkv=8, d=128, Tn=64, Lmin=1, Lmax=192,
             page=64, cache="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "tree", "tree", "tree", "commit"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([0, 16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    base, layout = rng.choice([(BASE, "split_half"), (BASE, "adjacent"), (500000.0, "split_half"),
                               (0.0, "split_half")])
    if op == "append":
        B = _log(rng, 1, 64)
        Tn = _log(rng, 1, 4096)
        Tn = max(1, min(Tn, 16384 * 8 // (B * Hkv)))
        return dict(op=op, B=B, Hkv=Hkv, d=d, Tn=Tn, Lmin=0, Lmax=Tn + rng.randint(0, 200),
                    page=page, base=base, layout=layout)
    if op == "read":
        B = _log(rng, 1, 16)
        Lmax = _log(rng, 1, max(1, 32768 * 8 // (B * Hkv)))
        Lmax = min(Lmax, 32768)
        return dict(op=op, B=B, Hkv=Hkv, d=d, Lmin=max(1, Lmax // 4), Lmax=Lmax, page=page)
    if op == "commit":
        B = _log(rng, 1, 256)
        Tn = _log(rng, 1, 64)
        return dict(op=op, B=B, Hkv=min(Hkv, 8), d=d, Tn=Tn, Lmin=0, Lmax=rng.randint(1, 128) + Tn,
                    page=page, cache=rng.choice(["bf16", "e4m3"]))
    rep = rng.choice([1, 2, 4, 4, 7, 8])
    B = _log(rng, 1, 64)
    if op == "decode":
        Lmax = min(32768, _log(rng, 1, max(2, 8192 * 64 * 8 // (B * Hkv))))
        return dict(op=op, B=B, Hq=Hkv * rep, Hkv=Hkv, d=d, Lmin=max(1, Lmax // 8), Lmax=Lmax,
                    page=page, base=base, layout=layout)
    B = _log(rng, 1, 16)
    Tn = _log(rng, 1, 64)
    top = 8 * 32 * 64 * 12288 // (B * Hkv * rep * Tn)  # the work of the widest listed tree
    Lmax = _log(rng, 1, max(2, min(16384, top, 8 * 8 * 16384 // (B * Hkv))))
    return dict(op=op, B=B, Hq=Hkv * rep, Hkv=Hkv, d=d, Tn=Tn, Lmin=Lmax // 4, Lmax=Lmax,
                page=page, cache=rng.choice(["bf16", "e4m3"]), base=base, layout=layout)


def _rows(case):
    """Cache rows a sequence has room for: drafts come after the longest prefix."""
    return case["Lmax"] + (case["Tn"] if case["op"] == "tree" else 0)


def work(case):
    op, d, Hkv, B = case["op"], case["d"], case["Hkv"], case["B"]
    mean = (case["Lmin"] + case["Lmax"]) / 2
    row8, row16 = 2 * (d + 1), 2 * 2 * d  # bytes of a key and a value
    if op == "append":
        n = B * Hkv * case["Tn"]
        return {"bytes": n * (row16 + row8), "flops": n * d * 8}
    if op == "read":
        return {"bytes": B * Hkv * mean * (row16 + row8), "flops": B * Hkv * mean * d * 2}
    row = row8 if case.get("cache", "e4m3") == "e4m3" else row16
    if op == "commit":
        n = B * Hkv * _accepted_depth(case["Tn"])
        return {"bytes": 2 * n * row, "flops": 0}
    Hq = case["Hq"]
    if op == "decode":
        return {"bytes": B * Hkv * mean * row + 2 * B * Hq * d * 2,
                "flops": 4.0 * B * Hq * d * mean}
    Tn = case["Tn"]
    return {"bytes": B * Hkv * mean * row + B * Tn * (2 * Hq * d * 2 + Hkv * (row16 + row)),
            "flops": 4.0 * B * Hq * Tn * d * (mean + 4)}


# ---------------------------------------------------------------------- inputs
def _accepted_depth(Tn):
    return max(1, min(6, Tn // 4))


def _quantise(x, room):
    """e4m3 values and scale codes of rows x [..., d] (any float type): code - 127 is the
    least e in [-124, 120] with max|x| * room <= 448 * 2^e."""
    top = x.double().abs().amax(-1) * room
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / E4M3_MAX))
    e = torch.where(torch.ldexp(torch.full_like(top, E4M3_MAX), e - 1) >= top, e - 1, e)
    e = torch.where(torch.ldexp(torch.full_like(top, E4M3_MAX), e) < top, e + 1, e)
    e = e.clamp(-124, 120)
    return e


def _pools(case, g, rows, dev):
    """Keys and values of every row of every sequence's pages, in pools with shuffled pages."""
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    ps = page if page else rows
    per = -(-rows // ps)
    n = B * per
    if page:
        table = torch.randperm(n, generator=g, device=dev).to(torch.int32).view(B, per)
    else:
        table = torch.arange(B, dtype=torch.int32, device=dev).view(B, 1)
    s = {"table": table, "page": ps, "per": per}
    # keys have strong and weak channels, values strong and weak rows
    gain = torch.exp(0.5 * torch.randn(Hkv, 1, d, generator=g, device=dev))
    k = torch.randn(n, Hkv, ps, d, generator=g, device=dev, dtype=torch.bfloat16) * gain.bfloat16()
    v = torch.randn(n, Hkv, ps, d, generator=g, device=dev, dtype=torch.bfloat16)
    v *= torch.exp(0.5 * torch.randn(n, Hkv, ps, 1, generator=g, device=dev)).bfloat16()
    if case.get("cache", "e4m3") == "bf16":
        s["k"], s["v"] = k, v
        return s
    for name, x in (("k", k), ("v", v)):
        m = x.abs().amax(-1).float()
        e = torch.floor(torch.log2(m.clamp(min=2.0 ** -126))) - 7  # 448 * 2^e over max|x|
        s[name] = torch.ldexp(x, -e.unsqueeze(-1).to(torch.int32)).to(torch.float8_e4m3fn)
        s[name + "s"] = (e + 127).to(torch.uint8)
    return s


def _tree(case, g, dev):
    """Parents of a drafted tree per sequence: a level order with up to eight branches a level."""
    B, Tn = case["B"], case["Tn"]
    t = torch.arange(Tn, device=dev)
    width = max(1, min(8, Tn // 2))
    pick = torch.randint(0, width, (B, Tn), generator=g, device=dev)
    start = (t // width - 1) * width  # the level above
    return torch.where(t < width, -1, start + pick).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, d, op = case["B"], case["d"], case["op"]
    rows = _rows(case)
    s = {"case": case}
    s.update(_pools(case, g, rows, dev))
    top = case["Lmax"] - (case["Tn"] if op in ("append", "commit") else 0)
    low = min(case["Lmin"], top)
    s["lens"] = torch.randint(low, top + 1, (B,), generator=g, device=dev, dtype=torch.int32)

    def new(H, T):
        return torch.randn(B, H, T, d, generator=g, device=dev, dtype=torch.bfloat16)

    if op == "append":
        s["kn"], s["vn"] = new(case["Hkv"], case["Tn"]), new(case["Hkv"], case["Tn"])
    elif op == "read":
        s["ko"] = torch.zeros(B, case["Hkv"], case["Lmax"], d, dtype=torch.bfloat16, device=dev)
        s["vo"] = torch.zeros_like(s["ko"])
    elif op == "decode":
        s["q"] = new(case["Hq"], 1)
    elif op == "tree":
        s["q"] = new(case["Hq"], case["Tn"])
        s["kn"], s["vn"] = new(case["Hkv"], case["Tn"]), new(case["Hkv"], case["Tn"])
        s["parents"] = _tree(case, g, dev)
    else:
        # A chain that hangs below the first token or below one behind the accepted rows, so
        # that a second pass over the moved rows moves the same values again.
        Tn, n = case["Tn"], _accepted_depth(case["Tn"])
        pick = torch.rand(B, Tn, generator=g, device=dev)
        if 2 * n <= Tn:
            pick[:, :n] = 2.0
            chain = pick.argsort(1)[:, :n].sort(1).values
        else:
            chain = torch.arange(n, device=dev).expand(B, n)
        parents = torch.full((B, Tn), -1, dtype=torch.int64, device=dev)
        parents.scatter_(1, chain[:, 1:], chain[:, :-1])
        s["parents"] = parents.to(torch.int32)
        s["accepted"] = chain[:, -1].to(torch.int32)
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------- plain forms
def _rotated(x, pos, base, layout):
    """RoPE of x [B, H, T, d] at positions pos [B, T]: angles in 64 bits, the rest in 32."""
    x = x.float()
    if base <= 0:
        return x
    d = x.shape[-1]
    freq = base ** (-2.0 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    ang = pos.double()[:, None, :, None] * freq
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    if layout == "split_half":
        a, b = x[..., : d // 2], x[..., d // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _put(s, name, r, rows, e=None):
    """Rows [B, H, T, d] to cache rows r [B, T]; e: scale exponents [B, H, T] of e4m3 rows."""
    page = torch.gather(s["table"].long(), 1, r // s["page"])
    off = r % s["page"]
    if e is None:
        s[name][page, :, off] = rows.to(torch.bfloat16).transpose(1, 2)
        return
    q = torch.ldexp(rows, -e.unsqueeze(-1).to(rows.dtype)).to(torch.float8_e4m3fn)
    s[name].view(torch.uint8)[page, :, off] = q.view(torch.uint8).transpose(1, 2)
    s[name + "s"][page, :, off] = (e + 127).to(torch.uint8).transpose(1, 2)


def _all_rows(s, name):
    """The cache in 32 bits, [B, Hkv, rows, d] in order."""
    p = s["table"].long()
    x = s[name][p].float()  # [B, per, Hkv, page, d]
    if name + "s" in s:
        x = torch.ldexp(x, s[name + "s"][p].float().unsqueeze(-1) - 127)
    return x.transpose(1, 2).flatten(2, 3)


def _append(s, pos, r):
    c = s["case"]
    k = _rotated(s["kn"], pos, c["base"], c["layout"])
    v = s["vn"].float()
    if "ks" in s:
        _put(s, "k", r, k, _quantise(s["kn"], math.sqrt(2.0) if c["base"] > 0 else 1.0))
        _put(s, "v", r, v, _quantise(s["vn"], 1.0))
    else:
        _put(s, "k", r, k)
        _put(s, "v", r, v)


def _cache(s):
    return [s["k"], s["v"]] + ([s["ks"], s["vs"]] if "ks" in s else [])


def _attend(q, k, v, seen):
    """softmax over the seen rows: q [B, Hkv, rep, T, d], k, v [B, Hkv, R, d], seen [B, T, R]."""
    B, Hkv, rep, T, d = q.shape
    x = (q.flatten(2, 3) @ k.transpose(-1, -2)).view(B, Hkv, rep, T, -1) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x.flatten(2, 3) @ v).view(B, Hkv, rep, T, -1) / x.sum(-1, keepdim=True)
    return o.flatten(1, 2).to(torch.bfloat16)


def _ancestors(parents):
    """[B, T, T]: whether token j is token t or above it.  With A the parent relation, that is
    I + A + A^2 + ... = (I - A)^-1."""
    B, T = parents.shape
    a = (parents.unsqueeze(-1) == torch.arange(T, device=parents.device)).float()
    eye = torch.eye(T, device=parents.device).expand(B, T, T)
    return torch.linalg.solve_triangular(eye - a, eye, upper=False, unitriangular=True) > 0.5


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    lens = s["lens"].long()
    dev = lens.device
    if op == "append":
        r = lens[:, None] + torch.arange(c["Tn"], device=dev)
        _append(s, r, r)
        return _cache(s)
    if op == "read":
        live = (torch.arange(c["Lmax"], device=dev) < lens[:, None])[:, None, :, None]
        for name, o in (("k", s["ko"]), ("v", s["vo"])):
            o.copy_(torch.where(live, _all_rows(s, name)[:, :, : c["Lmax"]].to(o.dtype), o))
        return [s["ko"], s["vo"]]
    if op == "commit":
        T = c["Tn"]
        anc = _ancestors(s["parents"])
        path = torch.gather(anc, 1, s["accepted"].long()[:, None, None].expand(-1, 1, T))[:, 0]
        n = path.sum(1)
        i = torch.arange(T, device=dev)
        # the path's tokens first, then every other row onto itself
        src = torch.where(i < n[:, None], (~path).long().argsort(dim=1, stable=True), i)
        frm, to = lens[:, None] + src, lens[:, None] + i
        p, ps = s["table"].long(), s["page"]
        pf, pt = torch.gather(p, 1, frm // ps), torch.gather(p, 1, to // ps)
        for x in _cache(s):
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[pt, :, to % ps] = x[pf, :, frm % ps]
        s["new_lens"].copy_(lens + n)
        return _cache(s) + [s["new_lens"]]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    at = torch.arange(s["per"] * s["page"], device=dev)
    if op == "decode":
        q = _rotated(s["q"], lens[:, None] - 1, c["base"], c["layout"])
        seen = (at < lens[:, None])[:, None]
        T = 1
    else:
        T = c["Tn"]
        anc = _ancestors(s["parents"])
        pos = lens[:, None] + anc.sum(-1) - 1
        _append(s, pos, lens[:, None] + torch.arange(T, device=dev))
        q = _rotated(s["q"], pos, c["base"], c["layout"])
        rel = at - lens[:, None]  # [B, R]
        own_rows = torch.gather(anc, 2, rel.clamp(0, T - 1)[:, None].expand(-1, T, -1))
        seen = torch.where((rel < 0)[:, None], True, own_rows & (rel < T)[:, None])
    live = seen.any(1)[:, None, :, None]
    k, v = (torch.where(live, _all_rows(s, name), 0.0) for name in ("k", "v"))
    out = _attend(q.view(B, Hkv, Hq // Hkv, T, d), k, v, seen)
    return [out] if op == "decode" else [out] + _cache(s)


# ---------------------------------------------------------------------- the framework's calls
def _kernels(s):
    import transformer_causal_self_gb300 as csattn

    c, op = s["case"], s["case"]["op"]
    rope = dict(rope_base=c.get("base", 0.0), rope_layout=c.get("layout", "split_half"))
    if op == "append":
        if c["page"]:
            csattn.cache_append_fp8_paged(s["kn"], s["vn"], s["k"], s["v"], s["ks"], s["vs"],
                                          s["table"], s["lens"], **rope)
        else:
            csattn.cache_append_fp8(s["kn"], s["vn"], s["k"], s["v"], s["ks"], s["vs"], s["lens"],
                                    **rope)
        return _cache(s)
    if op == "read":
        if c["page"]:
            csattn.cache_read_fp8_paged(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"],
                                        s["ko"], s["vo"])
        else:
            csattn.cache_read_fp8(s["k"], s["v"], s["ks"], s["vs"], s["lens"], s["ko"], s["vo"])
        return [s["ko"], s["vo"]]
    if op == "decode":
        if c["page"]:
            return [csattn.attn_decode_fp8_paged(s["q"], s["k"], s["v"], s["ks"], s["vs"],
                                                 s["table"], s["lens"], max_seq_len=c["Lmax"],
                                                 **rope)]
        return [csattn.attn_decode_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["lens"],
                                       max_seq_len=c["Lmax"], **rope)]
    scales = dict(k_scale=s["ks"], v_scale=s["vs"]) if "ks" in s else {}
    if op == "tree":
        if c["page"]:
            out = csattn.attn_tree_step_paged(s["q"], s["kn"], s["vn"], s["k"], s["v"], s["table"],
                                              s["lens"], s["parents"],
                                              max_seq_len=c["Lmax"] + c["Tn"], **scales, **rope)
        else:
            out = csattn.attn_tree_step(s["q"], s["kn"], s["vn"], s["k"], s["v"], s["lens"],
                                        s["parents"], max_seq_len=c["Lmax"] + c["Tn"], **scales,
                                        **rope)
        return [out] + _cache(s)
    if c["page"]:
        csattn.tree_commit_paged(s["k"], s["v"], s["table"], s["lens"], s["parents"],
                                 s["accepted"], s["new_lens"], **scales)
    else:
        csattn.tree_commit(s["k"], s["v"], s["lens"], s["parents"], s["accepted"], s["new_lens"],
                           **scales)
    return _cache(s) + [s["new_lens"]]


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------- 64 bits
def _turn(vec, pos, base, layout):
    """R_pos of rows vec [T, d] (64 bits) as a complex product, pos [T]."""
    if base <= 0:
        return vec
    T, d = vec.shape
    half = d // 2
    theta = torch.exp(-math.log(base) * 2.0 * torch.arange(half, device=vec.device).double() / d)
    unit = torch.polar(torch.ones(T, half, device=vec.device, dtype=torch.float64),
                       pos.double()[:, None] * theta)
    if layout == "split_half":
        z = torch.complex(vec[:, :half], vec[:, half:]) * unit
        return torch.cat([z.real, z.imag], 1)
    z = torch.view_as_complex(vec.reshape(T, half, 2).contiguous()) * unit
    return torch.view_as_real(z).reshape(T, d)


def _exponents(x, room):
    """The least e in [-124, 120] with room * max|row| <= 448 * 2^e, by search over powers."""
    top = room * x.abs().amax(-1)
    e = torch.arange(-124, 121, device=x.device)
    fits = top.unsqueeze(-1) <= E4M3_MAX * torch.pow(2.0, e.double())
    return e[fits.long().argmax(-1)]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    B, Hkv, d, ps = c["B"], c["Hkv"], c["d"], s["page"]
    lens = s["lens"].tolist()
    eight = "ks" in s
    if op == "commit":
        return None  # values are moved, none is computed
    if not eight:
        s["k"], s["v"] = s["k"].double(), s["v"].double()

    def where(b, r):
        return s["table"][b].long()[r // ps], r % ps

    def store(b, r, pos):
        page, off = where(b, r)
        for h in range(Hkv):
            k = _turn(s["kn"][b, h].double(), pos, c["base"], c["layout"])
            for name, x, room, raw in (("k", k, math.sqrt(2.0) if c["base"] > 0 else 1.0, s["kn"]),
                                       ("v", s["vn"][b, h].double(), 1.0, s["vn"])):
                if eight:
                    e = _exponents(raw[b, h].double(), room)
                    y = (x / torch.pow(2.0, e.double())[:, None]).to(torch.float8_e4m3fn)
                    s[name].view(torch.uint8)[page, h, off] = y.view(torch.uint8)
                    s[name + "s"][page, h, off] = (e + 127).to(torch.uint8)
                else:
                    s[name][page, h, off] = x

    def load(name, b, h, r):
        page, off = where(b, r)
        if not eight:
            x = s[name][page, h, off]
            return x.bfloat16().double()  # what the cache holds
        y = s[name].view(torch.uint8)[page, h, off].view(torch.float8_e4m3fn).double()
        return y * torch.pow(2.0, s[name + "s"][page, h, off].double() - 127)[:, None]

    dev = s["lens"].device
    if op == "append":
        for b in range(B):
            r = lens[b] + torch.arange(c["Tn"], device=dev)
            store(b, r, r)
        return _cache(s)
    if op == "read":
        ko, vo = s["ko"].double(), s["vo"].double()
        for b in range(B):
            r = torch.arange(lens[b], device=dev)
            for h in range(Hkv):
                ko[b, h, : lens[b]], vo[b, h, : lens[b]] = load("k", b, h, r), load("v", b, h, r)
        return [ko, vo]
    rep, T = c["Hq"] // Hkv, c.get("Tn", 1)
    out = torch.zeros(B, c["Hq"], T, d, dtype=torch.float64, device=dev)
    for b in range(B):
        L = lens[b]
        if op == "tree":
            up = s["parents"][b].tolist()
            line = [[] for _ in range(T)]
            for t in range(T):
                line[t] = (line[up[t]] if up[t] >= 0 else []) + [t]
            pos = torch.tensor([L + len(x) - 1 for x in line], device=dev)
            hide = torch.ones(T, L + T, dtype=torch.bool, device=dev)
            hide[:, :L] = False
            for t in range(T):
                hide[t, [L + j for j in line[t]]] = False
            store(b, L + torch.arange(T, device=dev), pos)
            n = L + T
        else:
            n, pos = L, torch.tensor([L - 1], device=dev)
            hide = torch.zeros(1, n, dtype=torch.bool, device=dev)
        r = torch.arange(n, device=dev)
        for h in range(Hkv):
            k, v = load("k", b, h, r), load("v", b, h, r)
            for i in range(h * rep, (h + 1) * rep):
                q = _turn(s["q"][b, i].double(), pos, c["base"], c["layout"])
                z = (q @ k.t() / math.sqrt(d)).masked_fill(hide, -math.inf)
                out[b, i] = torch.softmax(z, -1) @ v
    return [out] if op == "decode" else [out] + _cache(s)
