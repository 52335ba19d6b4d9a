"""Block tables, slots and positions from lengths, equal to one token after the other."""
import pytest
import torch

import transformer_causal_self_gb300 as csattn
from oracle import step as OS
from tests.fp4_helpers import gen, i32, refused
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def check(held, new, table, free, num_free, N, page, num_pages):
    """Runs the call and compares all that it leaves; whether it reported an error."""
    want = OS.page_tables(held, new, table.tolist(), free.tolist(), num_free, N, page, num_pages)
    t, f = table.to(dev()), free.to(dev())
    r = csattn.page_tables(i32(held), i32(new), t, f, i32([num_free]), N, page_size=page,
                           num_pages=num_pages)
    if want[6]:
        refused()
    else:
        csattn.check_status()
    assert torch.equal(t.cpu(), torch.tensor(want[0], dtype=torch.int32))
    assert torch.equal(f.cpu(), free)
    for got, x in zip(r, want[1:5]):
        assert got.tolist() == x
    assert r.free_left.item() == want[5]
    assert r.slots.dtype == torch.int64
    return want[6]


def pools(held, new, page, seed, spare=3):
    """A table and a free list of shuffled pages for these lengths."""
    g = gen(seed)
    have = [-(-max(h, 0) // page) for h in held]
    per = max(-(-(max(h, 0) + max(n, 0)) // page) for h, n in zip(held, new)) + 2
    want = sum(-(-(max(h, 0) + max(n, 0)) // page) for h, n in zip(held, new)) - sum(have)
    total = sum(have) + want + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(held), per), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:].contiguous(), total


@pytest.mark.parametrize("held,new,page,more", [
    ([0], [1], 16, 0), ([15], [1], 16, 0), ([16], [1], 16, 0), ([16], [0], 16, 1),
    ([0, 0, 0], [0, 0, 0], 16, 5), ([5, 31, 32, 0], [1, 1, 1, 1], 32, 0),
    ([5, 0, 100, 63, 64], [0, 200, 1, 1, 64], 64, 100), ([1000, 3], [5000, 2], 16, 1),
    ([70000], [70000], 65536, 0), (list(range(300)), [1] * 300, 16, 12),
    ([7] * 513, [i % 40 for i in range(513)], 16, 0), ([0] * 256, [4] * 256, 64, 1),
    ([9] * 1000, [0] * 999 + [3], 16, 2000)])
def test_tables(held, new, page, more):
    table, free, total = pools(held, new, page, seed=len(held))
    assert not check(held, new, table, free, len(free), sum(new) + more or 1, page, total)


def test_an_empty_free_list():
    """Steps that fit into the pages at hand, and one that does not."""
    table = torch.tensor([[3, 1], [0, 2]], dtype=torch.int32)
    none = torch.empty(0, dtype=torch.int32)
    assert not check([17, 5], [3, 11], table, none, 0, 14, 16, 4)
    assert check([16, 16], [1, 0], table[:, :1].repeat(1, 3), none, 0, 4, 16, 4)


@pytest.mark.parametrize("seed", range(6))
def test_random_steps(seed):
    g = gen(seed)
    B, page = [1, 40, 257, 600, 64, 30][seed], [16, 32, 64, 16, 128, 192][seed]
    held = torch.randint(0, 500, (B,), generator=g).tolist()
    new = (torch.rand(B, generator=g).pow(4) * 700).long().tolist()
    table, free, total = pools(held, new, page, seed)
    N = sum(new) + int(torch.randint(0, 3000, (1,), generator=g))
    # pages beyond num_free belong to someone else
    check(held, new, table, torch.cat([free, torch.tensor([0, 1], dtype=torch.int32)]), len(free),
          max(N, 1), page, total)


@pytest.mark.parametrize("short", [1, 2, 7, 30, 10 ** 6])
def test_too_few_pages(short):
    """The sequences from the first that finds too few on take none; those without need go on."""
    held, new = [0, 16, 15, 3, 40, 16, 2], [5, 1, 1, 30, 8, 0, 100]
    table, free, total = pools(held, new, 16, 3, spare=0)
    assert check(held, new, table, free, max(0, len(free) - short), sum(new), 16, total)


@pytest.mark.parametrize("N", [1, 5, 36, 44, 143, 144])
def test_too_small_a_step(N):
    held, new = [0, 16, 15, 3, 40, 16, 2], [5, 1, 1, 30, 8, 0, 100]
    table, free, total = pools(held, new, 16, 3)
    assert check(held, new, table, free, len(free), N, 16, total)


@pytest.mark.parametrize("b,h,n", [(0, -1, 2), (2, 3, -1), (1, 10 ** 6, 1), (1, 2, 2 ** 31 - 1),
                                   (3, -2 ** 31, -2 ** 31), (0, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_lengths_out_of_range(b, h, n):
    held, new = [5, 17, 0, 30], [3, 1, 16, 2]
    table, free, total = pools(held, new, 16, 7)
    held[b], new[b] = h, n
    assert check(held, new, table, free, len(free), 40, 16, total)


@pytest.mark.parametrize("big", [[2 ** 31 - 1] * 2, [2 ** 31 - 1] * 2 + [2], [2 ** 31 - 1] * 3,
                                 [2 ** 31 - 1] * 4, [2 ** 31 - 5], [2 ** 30] * 4])
@pytest.mark.parametrize("B,N", [(257, 8), (600, 2100)])
def test_lengths_that_add_up_past_32_bits(big, B, N):
    """No token of the step: all slots are -1, and nothing is written around them."""
    held, new = [3] * B, big + [0] * (256 - len(big)) + [1] * (B - 256)
    table, free, total = pools(held, [0] * B, 16, 5)
    slots = torch.full((N + 512,), 77, dtype=torch.int64, device=dev())
    positions = torch.full((N + 512,), 77, dtype=torch.int32, device=dev())
    z = torch.zeros(B + 1, dtype=torch.int32, device=dev())
    out = csattn.PageTables(z[:B].clone(), z, slots[256:256 + N], positions[256:256 + N],
                            z[:1].clone())
    csattn.page_tables(i32(held), i32(new), table.to(dev()), free.to(dev()), i32([len(free)]), N,
                       page_size=16, num_pages=total, out=out)
    refused()
    for x, inside in ((slots, -1), (positions, 0)):
        assert (x[256:256 + N] == inside).all()
        assert (x[:256] == 77).all() and (x[256 + N:] == 77).all()
    assert out.seq_lens.tolist() == held and out.free_left.item() == len(free)
    assert out.starts.tolist() == [0] + [N] * B


def test_pages_out_of_range():
    held, new = [5, 17, 0, 30], [3, 1, 40, 4]
    for where in range(4):
        table, free, total = pools(held, new, 16, 7)
        if where == 0:
            table[0, 0] = -1
        elif where == 1:
            table[1, 1] = total
        elif where == 2:
            free[-1] = total
        else:
            free[-2] = -5
        assert check(held, new, table, free, len(free), 48, 16, total)
    table, free, total = pools(held, new, 16, 7)
    assert check(held, new, table, free, -1, 48, 16, total)
    assert check(held, new, table, free, len(free) + 1, 48, 16, total)


def test_out_and_capture_and_streams():
    """Into the caller's tensors; replayed over the lengths of later steps (the free list's height is
    handed on); on another stream."""
    B, page, N = 40, 16, 64
    held, new = [3 * b for b in range(B)], [1] * B
    table, free, total = pools(held, [30] * B, page, seed=2)
    t, f, h, n = table.to(dev()), free.to(dev()), i32(held), i32(new)
    left = i32([len(free)])
    out = csattn.page_tables(h, n, t, f, left, N, page_size=page, num_pages=total)
    t.copy_(table.to(dev()))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        r = csattn.page_tables(h, n, t, f, left, N, page_size=page, num_pages=total, out=out)
        h.copy_(r.seq_lens)
        left.copy_(r.free_left)
    assert r is out
    now, at, height = list(held), table.tolist(), len(free)
    for _ in range(20):
        gr.replay()
        torch.cuda.synchronize()
        want = OS.page_tables(now, new, at, free.tolist(), height, N, page, total)
        assert t.tolist() == want[0] and out.slots.tolist() == want[3]
        assert out.positions.tolist() == want[4]
        now, at, height = want[1], want[0], want[5]
        assert h.tolist() == now and left.item() == height
    csattn.check_status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = csattn.page_tables(h, n, t, f, left, N, page_size=page, num_pages=total, stream=side)
    side.synchronize()
    csattn.check_status()
    want = OS.page_tables(now, new, at, free.tolist(), height, N, page, total)
    assert r.slots.tolist() == want[3] and t.tolist() == want[0]


def test_python_refusals():
    h, t, f = i32([1, 2]), i32([[0, 1], [2, 3]]), i32([4, 5])
    kw = dict(page_size=16, num_pages=6)
    for bad, kind in [(lambda: csattn.page_tables(h, h[:1], t, f, f[:1], 4, **kw), ValueError),
                      (lambda: csattn.page_tables(h, h.long(), t, f, f[:1], 4, **kw), TypeError),
                      (lambda: csattn.page_tables(h, h, t[:1], f, f[:1], 4, **kw), ValueError),
                      (lambda: csattn.page_tables(h, h, t[0], f, f[:1], 4, **kw), ValueError),
                      (lambda: csattn.page_tables(h, h, t, f, f, 4, **kw), ValueError),
                      (lambda: csattn.page_tables(h, h, t.t(), f, f[:1], 4, **kw), ValueError),
                      (lambda: csattn.page_tables(h, h, t, f, f[:1].clone(), 0, **kw),
                       csattn.CsattnError)]:
        with pytest.raises(kind):
            bad()
    csattn.check_status()
