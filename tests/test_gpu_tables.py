"""mxsa_build_tables on the GPU against a plain statement of its definition,
number by number."""
import numpy as np
import pytest
import torch

import block_sparse_attention_builder_gb300 as mx

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def dev(x, dt=I32):
    return torch.tensor(np.asarray(x), dtype=dt, device="cuda")


def reference(old, new, held, table, free, count, ps, total_q, pages):
    table, free, held = table.copy(), list(free), list(held)
    old = [0 if n < 0 else o for o, n in zip(old, new)]
    for s, n in enumerate(new):
        if n < 0:
            for p in table[s, :held[s]]:
                free[count] = int(p)
                count += 1
            held[s] = 0
    cu, pos, loc = [0], [], []
    for s, n in enumerate(new):
        n = max(n, 0)
        while held[s] * ps < old[s] + n:
            count -= 1
            table[s, held[s]] = free[count]
            held[s] += 1
        for p in range(old[s], old[s] + n):
            pos.append(p)
            page = int(table[s, p // ps])
            loc.append(page * ps + p % ps if 0 <= page < pages else -1)
        cu.append(len(pos))
    pad = [-1] * (total_q - len(pos))
    return cu, [o + max(n, 0) for o, n in zip(old, new)], pos + pad, loc + pad, table, free, held, count


class State:
    def __init__(self, r, B, ps, old_max, spare=2, extra=30):
        self.ps, self.B = ps, B
        self.old = [int(x) for x in r.randint(0, old_max + 1, B)]
        self.held = [-(-o // ps) + int(r.randint(0, 2)) for o in self.old]
        self.width = max(self.held) + spare
        self.pages = sum(self.held) + extra
        order = r.permutation(self.pages)
        self.table, at = np.full((B, self.width), -1, np.int32), 0
        for s, h in enumerate(self.held):
            self.table[s, :h] = order[at:at + h]
            at += h
        self.count = self.pages - at
        self.free = np.concatenate([order[at:], np.full(at, -4)]).astype(np.int32)

    def run(self, new, total_q, alias=False, **over):
        prob = mx.make_problem(self.B, total_q, 8, 8, 0, self.ps, self.pages, self.width)
        a = dict(kv_lens=dev(self.old), new_lens=dev(new), pages_held=dev(self.held), block_tables=dev(self.table),
                 free_pages=dev(self.free), free_count=dev([self.count]))
        a.update(over)
        o = dict(cu_seqlens_q=dev([7] * (self.B + 1), I64), used_kv_lens=a["kv_lens"] if alias else dev([7] * self.B),
                 positions=dev([7] * total_q, I64), loc=dev([7] * total_q, I64),
                 pages_held_out=None if alias else dev([7] * self.B), free_count_out=None if alias else dev([7]),
                 flags=dev([0]))
        mx.build_tables(prob, **a, **o)
        torch.cuda.synchronize()
        get = lambda n: a[{"pages_held_out": "pages_held", "free_count_out": "free_count"}[n]] if o[n] is None else o[n]
        return (o["flags"].item(), o["cu_seqlens_q"].tolist(), o["used_kv_lens"].tolist(), o["positions"].tolist(),
                o["loc"].tolist(), a["block_tables"].cpu().numpy(), a["free_pages"].tolist(),
                get("pages_held_out").tolist(), get("free_count_out").item())


def same(got, want):
    flags, cu, used, pos, loc, table, free, held, count = got
    assert flags == 0
    assert (cu, used, pos, loc, held, count) == (want[0], want[1], want[2], want[3], want[6], want[7])
    assert np.array_equal(table, want[4]) and free == want[5]


@pytest.mark.parametrize("B,ps,old_max,new_max,done,pad,alias", [
    (1, 64, 0, 1, 0, 0, False), (1, 64, 1000, 3, 0, 5, True), (1, 128, 500, 9000, 0, 1, False),
    (64, 64, 3000, 1, 0, 0, True), (33, 128, 900, 70, 5, 3, False), (200, 64, 700, 130, 40, 77, True),
    (1024, 64, 300, 2, 100, 9, False), (1024, 128, 200, 40, 0, 0, True), (7, 64, 100, 4097, 1, 0, False),
    (3, 64, 5, 0, 1, 4, False), (5, 64, 200, 0, 5, 0, True),
])
def test_against_the_definition(B, ps, old_max, new_max, done, pad, alias):
    r = np.random.RandomState(B * 7 + new_max)
    s = State(r, B, ps, old_max, spare=new_max // ps + 2, extra=B * (new_max // ps + 1) + 3)
    new = [int(x) for x in r.randint(0, new_max + 1, B)]
    new[r.randint(B)] = new_max
    for i in r.permutation(B)[:done]:
        new[i] = -1
    total = sum(max(n, 0) for n in new)
    want = reference(s.old, new, s.held, s.table, s.free, s.count, ps, total + pad, s.pages)
    same(s.run(new, total + pad, alias), want)


def test_pages_given_back_serve_the_same_step():
    s = State(np.random.RandomState(1), 4, 64, 300, spare=9, extra=0)
    assert s.count == 0
    s.held[0] = s.table.shape[1] - 9
    s.table[0, :s.held[0]] = np.arange(s.held[0])
    s.old[0] = 0
    new = [-1, 1, 0, s.held[0] * 64 - 63 - s.old[3] % 64]
    over = reference(s.old, new, s.held, s.table, list(s.free), 0, 64, 2000, s.pages)
    same(s.run(new, 2000), over)


def refused(s, new, total, flag, **over):
    flags, cu, used, pos, loc, table, free, held, count = s.run(new, total, **over)
    assert flags == flag
    assert cu == [0] * (s.B + 1) and pos == [-1] * total and loc == [-1] * total
    keep = lambda name, mine: over[name].tolist() if name in over else list(mine)
    assert used == keep("kv_lens", s.old) and held == keep("pages_held", s.held)
    assert count == (over["free_count"].item() if "free_count" in over else s.count)
    assert np.array_equal(table, s.table) and free == list(s.free)


@pytest.mark.parametrize("total", [600, 6000])  # one launch, two
def test_what_does_not_fit_moves_nothing(total):
    spare = total // 64 + 3
    s = State(np.random.RandomState(2), 6, 64, 500, spare=spare, extra=spare)
    refused(s, [total] + [0] * 5, total - 1, 128)                # more tokens than the step holds
    refused(s, [64 * 3] * 3 + [0, 0, 0], total, 2048, free_count=dev([2]))
    refused(s, [64 * s.width + 1] + [0] * 5, total, 16)          # more than the row's entries
    refused(s, [1] * 6, total, 16, kv_lens=dev([-1] + s.old[1:]))
    refused(s, [1] * 6, total, 16, kv_lens=dev([s.held[0] * 64 + 1] + s.old[1:]))
    refused(s, [1] * 6, total, 16, pages_held=dev(s.held[:5] + [s.width + 1]))
    refused(s, [1] * 5 + [-1], total, 16, pages_held=dev(s.held[:5] + [-1]))
    refused(s, [0] * 6, total, 2048, free_count=dev([-1]))
    refused(s, [0] * 6, total, 2048, free_count=dev([s.pages + 1]))
    refused(s, [0] * 5 + [-1], total, 2048, free_count=dev([s.pages]))  # the list would outgrow the cache
    refused(s, [2 ** 31 - 1] * 6, total, 16)


def test_a_page_outside_the_cache_has_no_slot():
    s = State(np.random.RandomState(3), 2, 64, 500, spare=3, extra=5)
    s.free[s.count - 1] = s.pages
    new = [s.held[0] * 64 - s.old[0] + 3, 0]
    flags, cu, used, pos, loc, *_ = s.run(new, new[0])
    assert flags == 4 and loc[-3:] == [-1] * 3 and all(x >= 0 for x in loc[:-3])
    assert pos == list(range(s.old[0], s.old[0] + new[0])) and cu == [0, new[0], new[0]]


def test_captured_decode_steps():
    """A captured step, replayed: lengths, held pages and list are its own inputs."""
    r = np.random.RandomState(5)
    s = State(r, 9, 64, 200, spare=4, extra=40)
    prob = mx.make_problem(9, 9, 8, 8, 0, 64, s.pages, s.width)
    lens, held, table, free, count = dev(s.old), dev(s.held), dev(s.table), dev(s.free), dev([s.count])
    one, cu, pos, loc, f = dev([1] * 9), dev([0] * 10, I64), dev([0] * 9, I64), dev([0] * 9, I64), dev([0])
    run = lambda: mx.build_tables(prob, lens, one, held, table, free, count, cu, lens, pos, loc, flags=f)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        run()
    old, hd, tb, fr, n = s.old, s.held, s.table, list(s.free), s.count
    for _ in range(100):
        g.replay()
        w = reference(old, [1] * 9, hd, tb, fr, n, 64, 9, s.pages)
        torch.cuda.synchronize()
        assert pos.tolist() == w[2] and loc.tolist() == w[3] and lens.tolist() == w[1]
        old, tb, fr, hd, n = w[1], w[4], w[5], w[6], w[7]
    assert f.item() == 0 and count.item() == n and held.tolist() == hd
