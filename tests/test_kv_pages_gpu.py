"""Page bookkeeping of the key/value cache on the GPU against plain Python: reserve with copy on write,
fork, truncate, compact; refusals that change nothing; and a serving run of all operators together."""
import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_block_scaled_mx_b200 import mxq

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """The same state as plain Python and on the device."""

    def __init__(self, rows, cols, pages, page, layers=2, seed=0, heads=2, dim=64, fmt="mxfp4"):
        self.pool = kh.Pool(rows, cols, pages, page)
        self.table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
        self.lens, self.refs, self.page = _dev([0] * rows), _dev([0] * pages), page
        g = torch.Generator().manual_seed(seed)
        shape = mxq.kv_cache_shape(pages, heads, dim, fmt, page, layers)
        self.cache = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()
        self.model = self.cache.cpu().numpy().copy()

    def same(self, what=""):
        torch.cuda.synchronize()
        assert self.table.cpu().tolist() == self.pool.table, what
        assert self.lens.cpu().tolist() == self.pool.lens, what
        assert self.refs.cpu().tolist() == self.pool.refs, what
        assert np.array_equal(self.cache.cpu().numpy(), self.model), what
        assert mxq.mxq_device_status() == 0, what

    def reserve(self, seqs, add, cap=None):
        slots = None if cap is None else torch.full((cap,), 77, dtype=torch.int32, device="cuda")
        info = mxq.kv_reserve(_dev(seqs), _dev(add), self.table, self.lens, self.refs, self.cache, self.page, slots=slots)
        code, n, want, moved = self.pool.reserve(seqs, add, cap)
        for a, b in moved:
            self.model[:, b] = self.model[:, a]
        assert info.tolist() == [code, n]
        if slots is not None:
            want = want or []
            assert slots.tolist() == want + [-1] * (cap - len(want))
        return code, slots

    def fork(self, parents, children):
        info = mxq.kv_fork(_dev(parents), _dev(children), self.table, self.lens, self.refs, self.page)
        want = self.pool.fork(parents, children)
        assert info.tolist() == list(want)
        return want[0]

    def truncate(self, seqs, to):
        info = mxq.kv_truncate(_dev(seqs), _dev(to), self.table, self.lens, self.refs, self.page)
        want = self.pool.truncate(seqs, to)
        assert info.tolist() == list(want)
        return want[0]

    def compact(self):
        info = mxq.kv_compact(self.table, self.lens, self.refs, self.cache, self.page)
        live, moved = self.pool.compact()
        for a, b in moved:
            self.model[:, b] = self.model[:, a]
        assert info.tolist() == [0, live]


@pytest.mark.parametrize("page,layers,heads,dim,fmt", [(16, 1, 1, 64, "mxfp4"), (48, 3, 2, 128, "nvfp4"), (64, 2, 8, 256, "mxfp4")])
def test_a_life_of_sequences(page, layers, heads, dim, fmt):
    s = Both(9, 12, 60, page, layers, 1, heads, dim, fmt)
    s.reserve([0, 3], [5 * page + 3, 1], 5 * page + 10)
    s.same("first")
    s.fork([0, 0, 3], [1, 2, 8])
    s.same("fork")
    s.reserve([1, 2, 0, 8], [1, page, 2, 0], page + 3)     # all holders of the tail page copy it
    s.same("copy on write")
    s.truncate([1, 0], [2 * page, 0])
    s.same("truncate")
    s.fork([2], [0])
    s.truncate([0], [page + 1])                            # ends inside a shared page
    s.reserve([0], [3], 3)
    s.same("shared middle page")
    s.compact()
    s.same("compact")
    s.compact()
    s.same("nothing left to move")
    s.truncate([0, 1, 2, 3, 8], [0] * 5)
    s.compact()
    s.same("empty")
    assert not any(s.pool.refs)


@pytest.mark.parametrize("seed", range(3))
def test_random_operations(seed):
    rng = np.random.RandomState(seed)
    s = Both(40, 9, 150, 16, 2, seed)
    for step in range(40):
        rows = rng.permutation(40)[:rng.randint(1, 25)].tolist()
        kind = rng.randint(4)
        if kind == 0:
            s.reserve(rows, [int(x) for x in rng.randint(0, 40, len(rows))], 1000)
        elif kind == 1:
            empty = [r for r in range(40) if s.pool.lens[r] == 0][:5]
            if empty:
                parents = [int(rng.choice([r for r in range(40) if r not in empty])) for _ in empty]
                s.fork(parents, empty)
        elif kind == 2:
            s.truncate(rows, [int(rng.randint(0, s.pool.lens[r] + 1)) for r in rows])
        else:
            s.compact()
        s.same("seed %d step %d kind %d" % (seed, step, kind))


def test_refusals_change_nothing():
    s = Both(6, 4, 7, 16)
    assert s.reserve([0, 1], [33, 16], 60)[0] == 0
    assert s.reserve([2, 2], [1, 1], 8)[0] == -1            # the same row twice
    assert s.reserve([6], [1], 8)[0] == -1
    assert s.reserve([-1], [1], 8)[0] == -1
    assert s.reserve([2], [-1], 8)[0] == -2
    assert s.reserve([2], [65], 80)[0] == -2                # more than a table row holds
    assert s.reserve([2], [9], 8)[0] == -2                  # more than slots holds
    assert s.reserve([2, 3], [48, 16], 64)[0] == -3         # four pages wanted, three free
    assert s.fork([0, 1], [2, 2]) == -1
    assert s.fork([0], [1]) == -1                           # not empty
    assert s.fork([2], [2]) == -1
    assert s.fork([0, 2], [2, 3]) == -1                     # a parent that is a child of the same call
    assert s.fork([9], [2]) == -1
    assert s.truncate([0, 0], [1, 1]) == -1
    assert s.truncate([0], [34]) == -2
    assert s.truncate([0], [-1]) == -2
    s.same()
    assert s.reserve([2, 3], [32, 16], 48)[0] == 0
    s.same("exactly what is free")
    none = _dev([])
    for call in (lambda: mxq.kv_fork(none, none, s.table, s.lens, s.refs, 16), lambda: mxq.kv_truncate(none, none, s.table, s.lens, s.refs, 16)):
        call()
    s.same("no rows")


def test_large_calls():
    """All 4096 rows of a call, and a pool that every thread of the cluster has several pages of."""
    n = 4096
    s = Both(5000, 3, 20000, 16, 1, 5, 1, 64)
    s.reserve(list(range(n)), [20] * n, 20 * n + 7)
    s.same("reserve")
    s.fork([0] * 900, list(range(n, n + 900)))
    s.same("fork")
    s.reserve(list(range(n, n + 900)), [1] * 900, 900)
    s.same("copies")
    s.truncate(list(range(0, n, 2)), [0] * (n // 2))
    s.same("truncate")
    s.compact()
    s.same("compact")


def test_captured_calls():
    s = Both(6, 6, 30, 16)
    s.reserve([0, 1], [20, 40], 60)
    state = [x.clone() for x in (s.table, s.lens, s.refs, s.cache)]
    of, kids, one, zero = _dev([0, 1, 1]), _dev([2, 3, 4]), _dev([1, 1, 1]), _dev([0, 0, 0])
    slots, info, ws = _dev([0] * 3), _dev([0, 0]), torch.empty(4096, dtype=torch.uint8, device="cuda")

    def step():
        mxq.kv_truncate(kids, zero, s.table, s.lens, s.refs, 16, info=info)
        mxq.kv_fork(of, kids, s.table, s.lens, s.refs, 16, info=info)
        mxq.kv_reserve(kids, one, s.table, s.lens, s.refs, s.cache, 16, slots=slots, info=info, workspace=ws)
        mxq.kv_compact(s.table, s.lens, s.refs, s.cache, 16, info=info, workspace=ws)

    step()
    for x, y in zip((s.table, s.lens, s.refs, s.cache), state):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        s.pool.truncate([2, 3, 4], [0] * 3)
        s.pool.fork([0, 1, 1], [2, 3, 4])
        for a, b in s.pool.reserve([2, 3, 4], [1] * 3, 3)[3]:
            s.model[:, b] = s.model[:, a]
        live, moved = s.pool.compact()
        for a, b in moved:
            s.model[:, b] = s.model[:, a]
        s.same("replay")
        assert info.tolist() == [0, live]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_a_serving_run(orc, fmt):
    """Prefill, branch, decode steps, a drop and a compaction, as a user runs them: every step's attention
    against 64 bits over the tokens that each sequence was given, whatever pages hold them."""
    H, G, D, page, P, R = 2, 3, 128, 16, 24, 5
    g = torch.Generator().manual_seed(3)
    rand = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16)  # noqa: E731
    gk = gv = None
    if fmt == "nvfp4":
        gk = gv = torch.tensor([6.0 / 2688], device="cuda")
    table, lens, refs = _dev(np.full((R, 6), -1)), _dev([0] * R), _dev([0] * P)
    cache = torch.randint(0, 256, mxq.kv_cache_shape(P, H, D, fmt, page), generator=g, dtype=torch.uint8).cuda()
    seqs = {0: [], 1: []}  # row -> [(k, v) of each token]

    def step(counts, causal_chunk=True):
        rows = sorted(counts)
        T = sum(counts.values())
        k, v, q = rand(T, H, D), rand(T, H, D), rand(T, H * G, D)
        slots = _dev([0] * (T + 3))
        info = mxq.kv_reserve(_dev(rows), _dev([counts[r] for r in rows]), table, lens, refs, cache, page, slots=slots)
        pad = torch.zeros((3, H, D), dtype=torch.bfloat16)
        mxq.kv_append(torch.cat([k, pad]).cuda(), torch.cat([v, pad]).cuda(), cache, slots, fmt, g_k=gk, g_v=gv)
        assert info.tolist()[0] == 0
        start = np.concatenate([[0], np.cumsum([counts[r] for r in rows])])
        out, lse = mxq.kv_attention(q.cuda(), cache, table[_dev(rows).long()].contiguous(), lens[_dev(rows).long()], fmt,
                                    q_start=_dev(start), max_q=max(counts.values()), g_k=gk, g_v=gv)
        at = 0
        for r in rows:
            seqs[r] = seqs[r] + [(k[at + i], v[at + i]) for i in range(counts[r])]
            at += counts[r]
        # the same tokens in a cache of their own, written by the oracle
        n = [len(seqs[r]) for r in rows]
        cols = max(-(-x // page) for x in n)
        own = np.zeros(mxq.kv_cache_shape(cols * len(rows), H, D, fmt, page), np.uint8)
        for i, r in enumerate(rows):
            kh.append(own, torch.stack([x for x, _ in seqs[r]]), torch.stack([x for _, x in seqs[r]]),
                      np.arange(n[i]) + i * cols * page, fmt, "ceil", *([np.float32(6.0 / 2688)] * 2 if gk is not None else [None] * 2))
        ref = kh.attention(q.double().numpy(), own, np.arange(cols * len(rows)).reshape(len(rows), cols), n, start, fmt,
                           np.float64(np.float32(D ** -0.5)), True, 0, *([np.float32(6.0 / 2688)] * 2 if gk is not None else [None] * 2))
        kh.check_attention(out, lse, ref, "%s %s" % (fmt, counts))
        assert mxq.mxq_device_status() == 0

    step({0: 37, 1: 20})
    step({0: 1, 1: 1})
    mxq.kv_fork(_dev([0, 0]), _dev([2, 3]), table, lens, refs, page)
    seqs[2], seqs[3] = list(seqs[0]), list(seqs[0])
    step({0: 1, 1: 1, 2: 1, 3: 1})
    step({0: 3, 1: 1, 2: 2, 3: 12})
    mxq.kv_truncate(_dev([1, 2]), _dev([0, 39]), table, lens, refs, page)
    seqs[1], seqs[2] = [], seqs[2][:39]
    info = mxq.kv_compact(table, lens, refs, cache, page)
    assert int(table.max()) == info.tolist()[1] - 1
    step({0: 1, 2: 1, 3: 1})
    step({0: 1, 1: 9, 2: 2, 3: 1})
