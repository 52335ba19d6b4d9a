"""Measured cases of a 4-bit paged KV cache and of what goes ahead of it in a step.

Operators of one path, from the requests' lengths to their outputs:

  tables  block tables, slots and positions of a batch's new tokens, from the lengths alone
  norm    RMS norm of every head's queries and keys and the rotation (RoPE), in one pass
  grad    the same and its backward pass
  chunk   new keys and values quantised into the 4-bit cache, and the sequences read back to
          bf16 (as the prefill of a chunk reads them)
  decode  one new query per sequence over the 4-bit cache

A row in 4 bits is e2m1 values, two channels to a byte (the even one low), and for every 16
channels a scale byte: the upper bits of an f16 without its sign (5 of exponent, 3 of mantissa).
A block of largest magnitude a has the scale s nearest to a / 6 (ties to even, at most 10240),
its values are the e2m1 nearest to x / s (ties to even, at most 6 in magnitude).
"""
import math

import torch

own = False

BASE = 10000.0
EPS = 1e-6
TOP_SCALE = 226  # the byte of 10240: 6 * 10240 still is an f16


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # every request of a batch in generation gets one more token (latency)
        dict(name="tables_token", op="tables", B=64, N=64, L=4096, page=64),
        # prompts of all lengths join a large batch: a full step of a server
        dict(name="tables_mixed", op="tables", B=512, N=65536, L=8192, page=16),
        # the new token of a batch in generation, straight from the fused projection (latency)
        dict(name="norm_token", op="norm", B=64, T=1, Hq=32, Hkv=8, d=128, dtype="bf16", base=BASE,
             layout="split_half", fused=True, places=True),
        # whole prompts
        dict(name="norm_prompt", op="norm", B=4, T=4096, Hq=32, Hkv=8, d=128, dtype="bf16",
             base=500000.0, layout="split_half", fused=True, places=False),
        # a small multi-head model in training, 32 bits, interleaved pairs
        dict(name="grad_small", op="grad", B=8, T=1024, Hq=12, Hkv=12, d=64, dtype="fp32",
             base=BASE, layout="adjacent", fused=False, places=False),
        # a training step's sequences
        dict(name="grad_long", op="grad", B=2, T=4096, Hq=32, Hkv=8, d=128, dtype="bf16",
             base=BASE, layout="split_half", fused=True, places=False),
        # one token for each of a batch of short sequences (latency)
        dict(name="chunk_token", op="chunk", B=64, Hkv=8, d=128, Tn=1, Lmin=64, Lmax=256, page=64,
             slots=True),
        # short ragged sequences of a small multi-head model
        dict(name="chunk_short", op="chunk", B=8, Hkv=12, d=64, Tn=100, Lmin=117, Lmax=1024,
             page=16, slots=False),
        # the last chunk of a long prompt
        dict(name="chunk_long", op="chunk", B=1, Hkv=8, d=128, Tn=4096, Lmin=32768, Lmax=32768,
             page=128, slots=True),
        # a single user's generation step (latency)
        dict(name="decode_one", op="decode", B=1, Hq=32, Hkv=8, d=128, Lmin=1000, Lmax=1000,
             page=0),
        # a served batch with ragged lengths over a paged cache
        dict(name="decode_batch", op="decode", B=64, Hq=32, Hkv=8, d=128, Lmin=512, Lmax=8192,
             page=64),
        # a few long contexts
        dict(name="decode_long", op="decode", B=4, Hq=32, Hkv=8, d=128, Lmin=30000, Lmax=32768,
             page=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "norm", "grad", "chunk", "chunk", "decode", "decode", "decode"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "tables":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, N=rng.choice([B, max(B, _log(rng, B, 65536))]),
                    L=_log(rng, 1, 8192), page=page)
    Hkv = rng.choice([1, 2, 4, 8, 12])
    rep = rng.choice([1, 2, 4, 4, 7, 8])
    if op in ("norm", "grad"):
        d, dtype = rng.choice([(64, "bf16"), (128, "bf16"), (128, "bf16"), (64, "fp32"),
                               (128, "fp32")])
        base, layout = rng.choice([(BASE, "split_half"), (BASE, "adjacent"),
                                   (500000.0, "split_half")])
        top = (16384 if op == "norm" else 8192) * 40 * 128 // (Hkv * (rep + 1) * d)
        top = max(1, top // (1 if dtype == "bf16" else 2))
        B = _log(rng, 1, min(64, top))
        T = _log(rng, 1, min(8192, max(1, top // B)))
        return dict(op=op, B=B, T=T, Hq=Hkv * rep, Hkv=Hkv, d=d, dtype=dtype, base=base,
                    layout=layout, fused=rng.random() < 0.7, places=rng.random() < 0.5)
    d = rng.choice([64, 128, 128])
    page = rng.choice([0, page, page])
    if op == "chunk":
        B = _log(rng, 1, 64)
        Lmax = _log(rng, 2, max(2, min(32768, 32768 * 8 // (B * Hkv))))
        Tn = _log(rng, 1, max(1, min(4096, Lmax, 4096 * 8 // (B * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, d=d, Tn=Tn, Lmin=max(Tn, Lmax // 4), Lmax=Lmax,
                    page=page, slots=page > 0 and rng.random() < 0.5)
    B = _log(rng, 1, 64)
    Lmax = min(32768, _log(rng, 1, max(2, 7500 * 64 * 8 // (B * Hkv))))
    return dict(op=op, B=B, Hq=Hkv * rep, Hkv=Hkv, d=d, Lmin=max(1, Lmax // 8), Lmax=Lmax,
                page=page)


def work(case):
    op, B = case["op"], case["B"]
    if op == "tables":
        # lengths in and out, offsets; a slot and a position per token; a page taken, written down
        # and read again
        return {"bytes": 16 * B + 12 * case["N"] + 12 * (case["N"] / case["page"] + B),
                "flops": 0}
    d, Hkv = case["d"], case["Hkv"]
    if op in ("norm", "grad"):
        n = B * case["T"] * (case["Hq"] + Hkv) * d
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            return {"bytes": 2 * n * size, "flops": 8 * n}
        # the forward pass, then x and the outputs' gradients in, the inputs' out
        return {"bytes": 5 * n * size, "flops": 24 * n}
    row4, row16 = 2 * (d // 2 + d // 16), 2 * 2 * d  # bytes of a key and a value
    mean = (case["Lmin"] + case["Lmax"]) / 2
    if op == "chunk":
        new = B * Hkv * case["Tn"]
        return {"bytes": new * row16 + B * Hkv * mean * row4 + B * Hkv * mean * row16,
                "flops": new * d * 8 + B * Hkv * mean * d * 4}
    return {"bytes": B * Hkv * mean * row4 + 2 * B * case["Hq"] * d * 2,
            "flops": 4.0 * B * case["Hq"] * d * mean}


# ---------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _prepare_tables(case, g):
    B, N, ps, dev = case["B"], case["N"], case["page"], g.device
    # what the sequences hold, and their new tokens: some prompts take most of the step
    held = torch.randint(0, case["L"] + 1, (B,), generator=g, device=dev)
    share = torch.rand(B, generator=g, device=dev).pow(6) + 1e-9
    new = 1 + torch.floor(share / share.sum() * ((N - B) * 0.98)).long()
    per = -(-(case["L"] + N) // ps)
    pages = -(-held // ps)
    first = torch.cumsum(pages, 0) - pages
    num_pages = int(pages.sum()) + N // ps + 2 * B + 8
    order = torch.randperm(num_pages, generator=g, device=dev)
    col = torch.arange(per, device=dev)
    table = torch.where(col < pages[:, None], order[(first[:, None] + col).clamp(max=num_pages - 1)],
                        -1)
    free = order[int(pages.sum()):]
    return {"held": held.to(torch.int32), "new": new.to(torch.int32),
            "table": table.to(torch.int32), "free": free.to(torch.int32),
            "num_free": torch.tensor([free.numel()], dtype=torch.int32, device=dev),
            "num_pages": num_pages}


def _prepare_norm(case, g):
    B, T, Hq, Hkv, d = (case[n] for n in ("B", "T", "Hq", "Hkv", "d"))
    dev = g.device
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt)

    # projections: strong and weak channels
    gain = torch.exp(0.5 * torch.randn(Hq + 2 * Hkv, d, generator=g, device=dev)).to(dt)
    s = {}
    if case["fused"]:
        qkv = rand(B, T, Hq + 2 * Hkv, d) * gain
        s["q"], s["k"] = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv)))
    else:
        s["q"], s["k"] = rand(B, Hq, T, d), rand(B, Hkv, T, d)
    for n in ("qw", "kw"):
        s[n] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
    s["pos"] = None
    if case["places"]:  # each sequence has a prefix of its own
        start = torch.randint(0, 32768, (B, 1), generator=g, device=dev)
        s["pos"] = (start + torch.arange(T, device=dev)).to(torch.int32)
    if case["op"] == "grad":
        s["dqo"], s["dko"] = rand(B, Hq, T, d), rand(B, Hkv, T, d)
        if case["fused"]:  # the gradient of the fused projection (that of v comes from elsewhere)
            s["dqkv"] = torch.zeros(B, T, Hq + 2 * Hkv, d, device=dev, dtype=dt)
            s["dq"], s["dk"] = (s["dqkv"][:, :, a:b].transpose(1, 2)
                                for a, b in ((0, Hq), (Hq, Hq + Hkv)))
        else:
            s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    return s


def _pools(case, g, rows):
    """A cache of random rows for every sequence, in pools with shuffled pages."""
    B, Hkv, d, page, dev = case["B"], case["Hkv"], case["d"], case["page"], g.device
    ps = page if page else rows
    per = -(-rows // ps)
    n = B * per
    if page:
        table = torch.randperm(n, generator=g, device=dev).to(torch.int32).view(B, per)
    else:
        table = torch.arange(B, dtype=torch.int32, device=dev).view(B, 1)
    s = {"table": table, "ps": ps, "per": per}
    # keys have strong and weak channels, values strong and weak rows
    gain = torch.exp(0.5 * torch.randn(Hkv, 1, d, generator=g, device=dev))
    k = torch.randn(n, Hkv, ps, d, generator=g, device=dev, dtype=torch.bfloat16) * gain.bfloat16()
    s["k"], s["ks"] = _quantise(k)
    del k
    v = torch.randn(n, Hkv, ps, d, generator=g, device=dev, dtype=torch.bfloat16)
    v *= torch.exp(0.5 * torch.randn(n, Hkv, ps, 1, generator=g, device=dev)).bfloat16()
    s["v"], s["vs"] = _quantise(v)
    return s


def prepare(case, seed):
    g = _generator(seed)
    op, dev = case["op"], g.device
    s = {"case": case}
    if op == "tables":
        s.update(_prepare_tables(case, g))
        return s
    if op in ("norm", "grad"):
        s.update(_prepare_norm(case, g))
        return s
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    s.update(_pools(case, g, case["Lmax"]))
    s["lens"] = torch.randint(case["Lmin"], case["Lmax"] + 1, (B,), generator=g, device=dev,
                              dtype=torch.int32)
    if op == "decode":
        s["q"] = 1.5 * torch.randn(B, case["Hq"], 1, d, generator=g, device=dev,
                                   dtype=torch.bfloat16)
        return s
    Tn = case["Tn"]
    s["held"] = s["lens"] - Tn
    rows = s["held"].long()[:, None] + torch.arange(Tn, device=dev)
    if case["slots"]:
        s["slots"] = (torch.gather(s["table"].long(), 1, rows // s["ps"]) * s["ps"]
                      + rows % s["ps"]).view(-1)
        # tokens of the batch in a row, as the projection leaves them
        s["kn"], s["vn"] = (torch.randn(B * Tn, Hkv, d, generator=g, device=dev,
                                        dtype=torch.bfloat16) for _ in range(2))
    else:
        s["kn"], s["vn"] = (torch.randn(B, Hkv, Tn, d, generator=g, device=dev,
                                        dtype=torch.bfloat16) for _ in range(2))
    s["ko"] = torch.zeros(B, Hkv, case["Lmax"], d, dtype=torch.bfloat16, device=dev)
    s["vo"] = torch.zeros_like(s["ko"])
    return s


# ---------------------------------------------------------------------- plain forms
def _quantise(x):
    """(bytes [..., d/2], scale bytes [..., d/16]) of x [..., d].  The quotients that decide are
    exact enough in 32 bits: x has 8 significant bits, a border between two codes or scales times
    its divisor 7 or fewer, so what is not a tie is 2^-10 away from one."""
    b = x.float().unflatten(-1, (-1, 16))
    a = b.abs().amax(-1)
    h = (a / 6.0).clamp(max=10240.0).half().view(torch.int16).int()  # (exact at the ties)
    code = ((h + 63 + ((h >> 7) & 1)) >> 7).clamp(max=TOP_SCALE)
    s = (code << 7).to(torch.int16).view(torch.float16).float().unsqueeze(-1)
    y = torch.where(s > 0, b.abs() / s, 0.0)
    e = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int()
         + (y > 2.5).int() + (y >= 3.5).int() + (y > 5.0).int())
    e = (e | (torch.signbit(b).int() << 3)).flatten(-2)
    return (e[..., 0::2] | (e[..., 1::2] << 4)).to(torch.uint8), code.to(torch.uint8)


def _values(x, scale):
    """What bytes and scale bytes stand for, in 32 bits."""
    e = torch.stack([x & 15, x >> 4], -1).flatten(-2)
    size = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    value = torch.cat([size, -size])[e.long()]
    s = (scale.int() << 7).to(torch.int16).view(torch.float16).float()
    return (value.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _all_rows(s, name):
    """The cache in 32 bits, [B, Hkv, rows, d] in order."""
    p = s["table"].long()
    return _values(s[name][p], s[name + "s"][p]).transpose(1, 2).flatten(2, 3)


def _angles(s, sign):
    """cos and sin of every position and pair, from 64 bits, [B, 1, T, d/2]."""
    c, dev = s["case"], s["q"].device
    pos = torch.arange(c["T"], device=dev).expand(c["B"], -1) if s["pos"] is None else s["pos"]
    freq = c["base"] ** (-2.0 * torch.arange(c["d"] // 2, device=dev, dtype=torch.float64) / c["d"])
    a = (pos.double()[:, :, None] * freq)[:, None]
    return torch.cos(a).float(), sign * torch.sin(a).float()


def _turned(x, cs, sn, layout):
    if layout == "split_half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cs - b * sn, a * sn + b * cs], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)


def _forward(s):
    lay = s["case"]["layout"]
    cs, sn = _angles(s, 1.0)

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        return _turned(y, cs, sn, lay).to(w.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _backward(s):
    lay = s["case"]["layout"]
    cs, sn = _angles(s, -1.0)

    def one(x, w, dy, dx):
        x, g = x.float(), _turned(dy.float(), cs, sn, lay)
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n, gw = x * r, g * w.float()
        dx.copy_((gw - n * (gw * n).mean(-1, keepdim=True)) * r)
        return (g * n).sum((0, 1, 2), dtype=torch.float64).float()

    return one(s["q"], s["qw"], s["dqo"], s["dq"]), one(s["k"], s["kw"], s["dko"], s["dk"])


def _gradients(s, dqw, dkw):
    return ([s["dqkv"]] if "dqkv" in s else [s["dq"], s["dk"]]) + [dqw, dkw]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "tables":
        ps, N, dev = c["page"], c["N"], s["held"].device
        held, new = s["held"].long(), s["new"].long()
        have, want = -(-held // ps), -(-(held + new) // ps) + (-held // ps)
        upto = torch.cumsum(want, 0)
        ends = torch.cumsum(new, 0)
        t = torch.arange(N, device=dev)
        live = t < ends[-1]
        t = torch.minimum(t, ends[-1] - 1)
        r = torch.searchsorted(ends, t, right=True)
        row = held[r] + t - (ends - new)[r]
        at = row // ps
        fresh = at >= have[r]
        nth = (upto - want)[r] + at - have[r]
        page = torch.where(fresh, s["free"][torch.where(fresh, s["num_free"] - 1 - nth, 0)].long(),
                           s["table"][r, at].long())
        s["table"][r, at] = page.to(torch.int32)  # (tokens of one page write the same)
        zero = torch.zeros(1, dtype=torch.int64, device=dev)
        return [s["table"], s["held"] + s["new"], torch.cat([zero, ends]).to(torch.int32),
                torch.where(live, page * ps + row % ps, -1),
                torch.where(live, row, 0).to(torch.int32),
                s["num_free"] - upto[-1:].to(torch.int32)]
    if op == "norm":
        return list(_forward(s))
    if op == "grad":
        return list(_forward(s)) + _gradients(s, *_backward(s))
    dev, ps = s["lens"].device, s["ps"]
    lens = s["lens"].long()
    if op == "chunk":
        Tn = c["Tn"]
        for name, x in (("k", s["kn"]), ("v", s["vn"])):
            if c["slots"]:
                page, off = s["slots"] // ps, s["slots"] % ps
            else:
                x = x.transpose(1, 2).flatten(0, 1)
                row = (s["held"].long()[:, None] + torch.arange(Tn, device=dev))
                page = torch.gather(s["table"].long(), 1, row // ps).view(-1)
                off = (row % ps).view(-1)
            s[name][page, :, off], s[name + "s"][page, :, off] = _quantise(x)
        live = (torch.arange(c["Lmax"], device=dev) < lens[:, None])[:, None, :, None]
        for name, o in (("k", s["ko"]), ("v", s["vo"])):
            o.copy_(torch.where(live, _all_rows(s, name)[:, :, : c["Lmax"]].to(o.dtype), o))
        return [s["ko"], s["vo"]]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    live = torch.arange(s["per"] * ps, device=dev) < lens[:, None]
    k, v = (torch.where(live[:, None, :, None], _all_rows(s, name), 0.0) for name in ("k", "v"))
    x = (s["q"].float().view(B, Hkv, Hq // Hkv, d) @ k.transpose(-1, -2)) / math.sqrt(d)
    x = x.masked_fill(~live[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x @ v) / x.sum(-1, keepdim=True)
    return [o.view(B, Hq, 1, d).to(torch.bfloat16)]


# ---------------------------------------------------------------------- the framework's calls
def _kernels(s):
    import transformer_causal_self_gb300 as csattn

    c = s["case"]
    op = c["op"]
    if op == "tables":
        t = csattn.page_tables(s["held"], s["new"], s["table"], s["free"], s["num_free"], c["N"],
                               page_size=c["page"], num_pages=s["num_pages"])
        return [s["table"], t.seq_lens, t.starts, t.slots, t.positions, t.free_left]
    if op in ("norm", "grad"):
        rope = dict(eps=EPS, rope_base=c["base"], rope_layout=c["layout"])
        out = csattn.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["pos"], **rope)
        if op == "norm":
            return list(out)
        _, _, dqw, dkw = csattn.qk_norm_rope_bwd(s["dqo"], s["dko"], s["q"], s["k"], s["qw"],
                                                 s["kw"], s["pos"], s["dq"], s["dk"], **rope)
        return list(out) + _gradients(s, dqw, dkw)
    cache = (s["k"], s["v"], s["ks"], s["vs"])
    if op == "chunk":
        if c["slots"]:
            csattn.cache_append_fp4_slots(s["kn"], s["vn"], *cache, s["slots"])
        elif c["page"]:
            csattn.cache_append_fp4_paged(s["kn"], s["vn"], *cache, s["table"], s["held"])
        else:
            csattn.cache_append_fp4(s["kn"], s["vn"], *cache, s["held"])
        if c["page"]:
            csattn.cache_read_fp4_paged(*cache, s["table"], s["lens"], s["ko"], s["vo"])
        else:
            csattn.cache_read_fp4(*cache, s["lens"], s["ko"], s["vo"])
        return [s["ko"], s["vo"]]
    if c["page"]:
        return [csattn.attn_decode_fp4_paged(s["q"], *cache, s["table"], s["lens"],
                                             max_seq_len=c["Lmax"])]
    return [csattn.attn_decode_fp4(s["q"], *cache, s["lens"], max_seq_len=c["Lmax"])]


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------- 64 bits
def _sizes(dev):
    """e2m1's magnitudes and the scales of all bytes, by the fields' definitions (powers of two
    from the host: pow of a GPU may be off by a unit in the last place)."""
    e2m1 = [(c % 2) * 0.5 if c < 2 else 2.0 ** (c // 2 - 1) * (1 + (c % 2) / 2) for c in range(8)]
    scale = [2.0 ** -14 * b / 8 if b < 8 else 2.0 ** (b // 8 - 15) * (1 + b % 8 / 8)
             for b in range(TOP_SCALE + 1)]
    return (torch.tensor(e2m1, dtype=torch.float64, device=dev),
            torch.tensor(scale, dtype=torch.float64, device=dev))


def _dequantised(data, scale):
    """Rows [n, d] in 64 bits from bytes and scale bytes, by the fields' definitions."""
    e = torch.empty(data.shape[0], 2 * data.shape[1], dtype=torch.int64, device=data.device)
    e[:, 0::2], e[:, 1::2] = data.long() % 16, data.long() // 16
    sizes, scales = _sizes(data.device)
    value = torch.where(e >= 8, -sizes[e % 8], sizes[e % 8])
    return value * scales[scale.long()].repeat_interleave(16, 1)


def _rounded(x):
    """Rows [n, d] as the cache gives them back, in 64 bits, by the nearest of all values."""
    n, d = x.shape
    a = x.double().view(n, d // 16, 16)
    size, scales = _sizes(x.device)
    top = a.abs().amax(-1) / 6

    def nearest(values, y):
        """The index of the nearest of sorted values; of two as near, the even one."""
        hi = torch.searchsorted(values, y.contiguous()).clamp(1, values.numel() - 1)
        up, down = values[hi] - y, y - values[hi - 1]
        return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)

    s = scales[nearest(scales, top)].unsqueeze(-1)
    # (x / s is rounded, but no quotient that is not a tie comes within 2^-10 of one)
    y = size[nearest(size, torch.where(s > 0, a.abs() / s, 0.0))]
    return (torch.sign(a) * y * s).view(n, d)


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if op in ("norm", "grad"):
        return _exact_norm(s)
    B, Hkv, d, ps = case["B"], case["Hkv"], case["d"], s["ps"]
    lens, dev = s["lens"].tolist(), s["lens"].device

    def load(name, b, h, r):
        page, off = s["table"][b].long()[r // ps], r % ps
        return _dequantised(s[name][page, h, off], s[name + "s"][page, h, off])

    if op == "chunk":
        Tn = case["Tn"]
        out = []
        for name, new, o in (("k", s["kn"], s["ko"]), ("v", s["vn"], s["vo"])):
            o = o.double()
            for b in range(B):
                L = lens[b] - Tn
                for h in range(Hkv):
                    if L > 0:
                        o[b, h, :L] = load(name, b, h, torch.arange(L, device=dev))
                    x = new[b * Tn:(b + 1) * Tn, h] if case["slots"] else new[b, h]
                    o[b, h, L:L + Tn] = _rounded(x)
            out.append(o)
        return out
    rep = case["Hq"] // Hkv
    out = torch.zeros(B, case["Hq"], 1, d, dtype=torch.float64, device=dev)
    for b in range(B):
        r = torch.arange(lens[b], device=dev)
        for h in range(Hkv):
            k, v = load("k", b, h, r), load("v", b, h, r)
            q = s["q"][b, h * rep:(h + 1) * rep, 0].double()
            out[b, h * rep:(h + 1) * rep, 0] = torch.softmax(q @ k.t() * d ** -0.5, -1) @ v
    return [out]


def _exact_norm(s):
    """By differentiation of the forward pass, the rotation as a complex product."""
    c = s["case"]
    T, d, dev = c["T"], c["d"], s["q"].device
    theta = torch.exp(-math.log(c["base"]) * torch.arange(0, d, 2, device=dev).double() / d)

    def one(x, w, dy):
        x = x.double().requires_grad_()
        w = w.double().requires_grad_()
        outs, dw = [], torch.zeros(d, dtype=torch.float64, device=dev)
        dx = torch.zeros(x.shape, dtype=torch.float64, device=dev)
        for b in range(c["B"]):
            p = torch.arange(T, device=dev) if s["pos"] is None else s["pos"][b]
            unit = torch.polar(torch.ones(T, d // 2, dtype=torch.float64, device=dev),
                               p.double()[:, None] * theta)
            xb = x[b]
            y = w * xb / torch.sqrt(xb.pow(2).sum(-1, keepdim=True) / d + EPS)
            if c["layout"] == "split_half":
                z = torch.complex(y[..., : d // 2], y[..., d // 2:]) * unit
                y = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.view_as_complex(y.reshape(-1, T, d // 2, 2).contiguous()) * unit
                y = torch.view_as_real(z).reshape(-1, T, d)
            outs.append(y.detach())
            if dy is not None:
                gx, gw = torch.autograd.grad(y, (xb, w), dy[b].double())
                dx[b] = gx
                dw += gw
        return torch.stack(outs), dx, dw

    q, dq, dqw = one(s["q"], s["qw"], s.get("dqo"))
    k, dk, dkw = one(s["k"], s["kw"], s.get("dko"))
    if c["op"] == "norm":
        return [q, k]
    if "dqkv" not in s:
        return [q, k, dq, dk, dqw, dkw]
    both = torch.cat([dq, dk, torch.zeros_like(dk)], 1).transpose(1, 2)
    return [q, k, both, dqw, dkw]
