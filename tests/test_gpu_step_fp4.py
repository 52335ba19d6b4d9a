"""A server's steps from the requests' lengths to the outputs: block tables, norm and rotation,
the quantising append and the decode, eager and as one captured graph."""
import numpy as np
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import step as OS
from tests import fp4_helpers as H
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu
B, Hq, Hkv, d, page, per = 5, 8, 2, 128, 16, 8
EPS, BASE = 1e-6, 10000.0


class Server:
    def __init__(self, N):
        self.N = N
        self.c = H.to_dev(H.empty_cache(B, Hkv, per * page, d, page, seed=1))
        self.pages = self.c["k"].shape[0]
        self.c["table"] = torch.full((B, per), -1, dtype=torch.int32, device=dev())
        self.free = torch.randperm(self.pages, generator=H.gen(2)).to(torch.int32).to(dev())
        self.left = H.i32([self.pages])
        self.lens, self.new = H.i32([0] * B), H.i32([0] * B)
        self.qkv = torch.zeros(N, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device=dev())
        g = H.gen(3)
        self.w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).to(dev())
                  for _ in range(2)]

    def step(self):
        """Keys and values of the N tokens into the cache, and each sequence's last query over it."""
        N, qkv = self.N, self.qkv
        t = csattn.page_tables(self.lens, self.new, self.c["table"], self.free, self.left, N,
                               page_size=page, num_pages=self.pages)
        q, k = csattn.qk_norm_rope(qkv[:, :Hq].unsqueeze(2), qkv[:, Hq:Hq + Hkv].unsqueeze(2),
                                   *self.w, t.positions.view(N, 1), eps=EPS, rope_base=BASE)
        csattn.cache_append_fp4_slots(k.view(N, Hkv, d), qkv[:, Hq + Hkv:], *H.cache(self.c),
                                      t.slots)
        last = (t.starts[1:].long() - 1).clamp(min=0)
        out = csattn.attn_decode_fp4_paged(q[last], *H.cache(self.c), self.c["table"], t.seq_lens)
        self.lens.copy_(t.seq_lens)
        self.left.copy_(t.free_left)
        return out, k, t


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_a_server(captured):
    N = 60
    s = Server(N)
    g = H.gen(5)
    news = [[30, 0, 7, 1, 16], [1, 1, 1, 0, 1], [1, 20, 1, 15, 1], [1, 1, 1, 1, 0], [17, 0, 0, 0, 1]]
    rows = [[np.zeros((Hkv, 0, d)) for _ in range(2)] for _ in range(B)]
    lens = [0] * B
    if captured:
        s.new.copy_(H.i32([0] * B))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out, k, t = s.step()
    for new in news:
        s.new.copy_(H.i32(new))
        s.qkv.copy_(torch.randn(N, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16))
        if captured:
            gr.replay()
        else:
            out, k, t = s.step()
        csattn.check_status()
        x = s.qkv.double().cpu().numpy()
        begin = np.concatenate([[0], np.cumsum(new)])
        assert t.starts.tolist() == begin.tolist()
        pos = np.zeros((N, 1), dtype=np.int64)
        for b in range(B):
            pos[begin[b]:begin[b + 1], 0] = lens[b] + np.arange(new[b])
        assert t.positions.tolist() == pos[:, 0].tolist()
        # keys: a rotation of what the norm leaves, within its tolerance; what is stored is the
        # nearest of the kernel's own bf16 keys
        want = OS.qk_norm_rope(x[:, Hq:Hq + Hkv, None], s.w[1].double().cpu().numpy(), pos, EPS, BASE,
                               "split_half")
        got = k.double().cpu().numpy()
        assert np.all(np.abs(got - want)[:begin[-1]] <= 2.0 ** -8 * np.abs(want[:begin[-1]]) + 2e-5)
        kq = OS.quantise_fp4(got[:, :, 0])[2]
        vq = OS.quantise_fp4(x[:, Hq + Hkv:])[2]
        for b in range(B):
            for i, new_rows in enumerate((kq, vq)):
                part = np.swapaxes(new_rows[begin[b]:begin[b + 1]], 0, 1)
                rows[b][i] = np.concatenate([rows[b][i], part], 1)
            lens[b] += new[b]
        assert s.lens.tolist() == lens
        cpu = H.to_cpu(s.c)
        for b in range(B):
            for have, exp in zip(H.rows(cpu, b, lens[b]) if lens[b] else (), rows[b]):
                assert np.array_equal(have, exp)
        last = [max(e - 1, 0) for e in begin[1:]]
        q = csattn.qk_norm_rope(s.qkv[:, :Hq].unsqueeze(2), s.qkv[:, Hq:Hq + Hkv].unsqueeze(2), *s.w,
                                t.positions.view(N, 1), eps=EPS, rope_base=BASE)[0][last].cpu()
        H.assert_close(out, H.expect(cpu, q, lens))
        for b in range(B):
            assert lens[b] or torch.all(out[b] == 0)
    used = sum(-(-n // page) for n in lens)
    assert s.left.item() == s.pages - used
    table = s.c["table"].cpu()
    taken = [int(table[b, i]) for b in range(B) for i in range(-(-lens[b] // page))]
    assert len(set(taken)) == used and not set(taken) & set(s.free[:s.left.item()].tolist())


def test_a_chunk_of_a_prompt_over_a_quantised_prefix():
    """The prefix read back to bf16, then the chunk's prefill over it."""
    L, Tn = 40, 24
    c, _ = H.filled(2, Hq, Hkv, d, page, [L, L], L + Tn, seed=8)
    cd = H.to_dev(c)
    g = H.gen(9)
    q, k, v = (torch.randn(2, n, Tn, d, generator=g).to(torch.bfloat16) for n in (Hq, Hkv, Hkv))
    H.append(cd, k.to(dev()), v.to(dev()), H.i32([L, L]))
    ko, vo = H.read(cd, H.i32([L + Tn] * 2))
    out = csattn.attn_fwd_ext(q.to(dev()), ko[:, :, :L + Tn].contiguous(),
                              vo[:, :, :L + Tn].contiguous(), q_offset=L, rope_base=0.0,
                              k_prerotated=True)
    csattn.check_status()
    cpu = H.to_cpu(cd)
    for b in range(2):
        kk, vv = H.rows(cpu, b, L + Tn)
        for h in range(Hq):
            z = q[b, h].double().numpy() @ kk[h // 4].T / np.sqrt(d)
            z[np.arange(L + Tn)[None] > L + np.arange(Tn)[:, None]] = -np.inf
            p = np.exp(z - z.max(-1, keepdims=True))
            ref = p @ vv[h // 4] / p.sum(-1, keepdims=True)
            assert np.abs(out[b, h].double().cpu().numpy() - ref).max() <= 2e-2
