"""Calls at the edge of what the key/value cache's documentation allows: pages outside the cache, windows and scores of
any size, values of very different scale, page calls that name nothing, and arguments left at their defaults."""
import numpy as np
import pytest
import torch

import kv_helpers as kh
from test_kv_cache_gpu import FMTS, Problem, _rand, _status
from test_kv_rows_gpu import _dev, _rewrite

from nvfp4_block_scaled_mx_b200 import mxq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def orc():
    import oracle

    oracle.build()
    return oracle


def _reference(p, hidden, scale=None, causal=True, window=0):
    """kh.attention's results where the tokens hidden[b] of sequence b are seen by no row."""
    scale = np.float64(np.float32(p.D ** -0.5 if scale is None else scale))
    q = p.q.double().numpy()
    T, Hq, D = q.shape
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    absv, mass, floor = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq, 1))
    for b, n in enumerate(p.lens):
        table = np.where((p.table[b] >= 0) & (p.table[b] < p.cache.shape[0]), p.table[b], 0)
        k, v = kh.tokens(p.cache, table, n, D, p.fmt, p.gk, p.gv)
        shown = np.ones(n, bool)
        shown[list(hidden.get(b, []))] = False
        rows = range(p.q_start[b], p.q_start[b + 1])
        for i in rows:
            seen = n - len(rows) + (i - rows[0]) + 1
            span = np.arange(n)
            at = np.flatnonzero(shown & (span < (seen if causal else n)) & (span >= (seen - window if window else 0)))
            for h in range(Hq):
                out[i, h], lse[i, h] = 0, -np.inf
                if len(at):
                    kk, vv = k[at, h // p.G], v[at, h // p.G]
                    x = kk @ q[i, h] * scale
                    e = np.exp(x - x.max())
                    out[i, h], lse[i, h] = e @ vv / e.sum(), x.max() + np.log(e.sum())
                    absv[i, h], floor[i, h] = e @ np.abs(vv) / e.sum(), len(vv) * np.abs(vv).max()
                    mass[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, absv, mass, floor


# rows of a sequence and heads that take each kernel and its row tiles
SHAPES = [(64, 1, 3), (128, 5, 1), (128, 5, 2), (256, 2, 2), (256, 5, 4), (128, 1, 20), (128, 5, 11), (64, 5, 20), (128, 1, 150)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,q", SHAPES)
@pytest.mark.parametrize("page", [16, 48])
def test_tokens_of_pages_outside_the_cache_are_skipped(orc, fmt, D, G, q, page):
    p = Problem(fmt, D, 2, G, page, [301, 200, 37, 150], [q, q, 1, q], seed=q + D)
    P = p.cache.shape[0]
    p.table[0, [1, 4]] = P, -1
    p.table[1, 0] = 2 ** 31 - 1
    p.table[2, :-(-37 // page)] = -3
    hidden = {b: [t for t in range(n) if not 0 <= p.table[b, t // page] < P] for b, n in enumerate(p.lens)}
    cache, qd = torch.from_numpy(p.cache).cuda(), p.q.cuda()
    for causal, window in ((True, 0), (False, 0), (True, 170)):
        out, lse = mxq.kv_attention(qd, cache, _dev(p.table), _dev(p.lens), fmt, q_start=_dev(p.q_start), max_q=p.max_q,
                                    causal=causal, window=window, g_k=p.dk, g_v=p.dv)
        assert _status() == 0x201
        kh.check_attention(out, lse, _reference(p, hidden, causal=causal, window=window), "%s %s %d" % (fmt, causal, window))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,q", [(64, 1, 9), (128, 1, 9), (256, 1, 9), (128, 2, 30), (64, 4, 40)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_window_wider_than_any_sequence(orc, fmt, D, G, q, causal):
    # more query tokens than cached ones: the first rows' own places lie in front of the first token
    p = Problem(fmt, D, 2, G, 16, [5, 300, 0, 70], [q, q, q, 1], seed=D + q)
    want = p.run(causal=causal)
    kh.check_attention(*want, p.ref(causal=causal), "no window")
    for window in (2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30, 400):
        out, lse = p.run(causal=causal, window=window)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), window


def _levels(fmt, D, q, levels, seed):
    """One sequence of 700 tokens whose scores rise in steps of 32 tokens, by other amounts in each row, in units of
    log 2; tokens of step s have values in channel s % 32 (and s % 32 + 32) alone, so that each step's weight shows."""
    n = 700
    p = Problem(fmt, D, 1, 1, 16, [n], [q], seed=seed)
    step = np.minimum(np.arange(n) // 32, len(levels) - 1)
    k, v = torch.zeros((n, 1, D), dtype=torch.bfloat16), torch.zeros((n, 1, D), dtype=torch.bfloat16)
    k[:, 0, 0] = torch.tensor(levels, dtype=torch.bfloat16)[step]
    for c in (0, 32):
        v[np.arange(n), 0, step % 32 + c] = 1.0
    if fmt == "nvfp4":
        p.gk, p.gv = np.float32(1 / 64), np.float32(1 / 64)
        p.dk, p.dv = torch.tensor([p.gk], device="cuda"), torch.tensor([p.gv], device="cuda")
    _rewrite(p, k, v)
    p.q.zero_()
    p.q[:, 0, 0] = (0.9 + 0.2 * torch.arange(q) / q).to(torch.bfloat16)
    return p


LN2 = float(np.float32(np.log(2.0)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q", [20, 150])
@pytest.mark.parametrize("up", [9, 12, 24])
def test_a_maximum_that_rises_inside_a_tile(orc, fmt, D, q, up):
    """The probabilities of a tile's first tokens are written before a later one raises the row's base."""
    p = _levels(fmt, D, q, [-up, -up / 2, up / 2, up] + [up - 3] * 4 + [up + 9, 2 * up + 9, 0, 2 * up + 30], seed=q)
    for causal in (True, False):
        out, lse = p.run(scale=LN2, causal=causal, out_dtype=torch.float32)
        kh.check_attention(out, lse, p.ref(scale=LN2, causal=causal), "%s D%d q%d" % (fmt, D, q))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_probabilities_are_rounded_once(orc, fmt, D):
    """A probability is rounded when it is written, by at most half a step of f16, 2^-11 of it (all stay in f16's normal
    range here); raising the base afterwards is a power of two.  So each step's weight is off by 2^-11, by 2 d (scores, see
    check_attention), and by 2^-17 for fp32 sums of 128 terms and the quotient."""
    p = _levels(fmt, D, 150, [-8, -3, 5, 9], seed=7)
    p.lens[0] = 128  # one tile
    out, lse = p.run(scale=LN2, causal=False, out_dtype=torch.float32)
    r, l, absv, mass, _ = p.ref(scale=LN2, causal=False)
    d = (2.0 ** -20 + 2.0 ** -22) * mass + 2.0 ** -22 * np.abs(l)
    tol = (2 * d[..., None] + 2.0 ** -11 + 2.0 ** -17) * absv
    err = np.abs(out.double().cpu().numpy() - r)
    assert (err <= tol).all(), "off by %g of its tolerance" % np.nanmax(err / np.maximum(tol, 1e-300))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,q", [(64, 1, 3), (128, 5, 1), (256, 2, 2), (256, 5, 4), (128, 1, 20), (64, 1, 60), (128, 1, 150)])
def test_large_scores(orc, fmt, D, G, q):
    """Scores of 10^6 to 10^30, finite, and equal for every third token: those share the weight evenly, so the result is
    known to the rounding of the probabilities however coarse fp32 is at such scores.  The log-sum-exp has fewer than 16
    roundings of half a step of 2^-23, or as much where an exponent is held at the largest that f16 takes: 2^-20."""
    n = 300
    p = Problem(fmt, D, 1, G, 16, [n], [q], seed=5)
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16)
    k[:, 0, 3] = -4.0
    k[::3, 0, 3] = 4.0
    v = _rand((n, 1, D), 6)
    if fmt == "nvfp4":
        p.gk, p.gv = np.float32(4 * 1.01 / 2688), np.float32(float(v.float().abs().max()) * 1.01 / 2688)
        p.dk, p.dv = torch.tensor([p.gk], device="cuda"), torch.tensor([p.gv], device="cuda")
    _rewrite(p, k, v)
    p.q.zero_()
    for x in (2e5, 3e6, 5.1e6, 7.7e6, 2.3e7, 9e8, 2e9, 1e12, 3e29):
        p.q[..., 3] = x * (1 + torch.arange(p.q.shape[0] * G).reshape(-1, G) / 997.0)
        out, lse = p.run(scale=1.0, causal=False, out_dtype=torch.float32)
        r, l, absv, mass, floor = p.ref(scale=1.0, causal=False)
        z = lse.double().cpu().numpy()
        assert (np.abs(z - l) <= 2.0 ** -20 * np.abs(l)).all(), x
        tol = 2.0 ** -24 * np.abs(r) + (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -16) * absv + 2.0 ** -28 * floor
        err = np.abs(out.double().cpu().numpy() - r)
        assert (err <= tol).all(), "%g: off by %g of its tolerance" % (x, np.nanmax(err / np.maximum(tol, 1e-300)))


@pytest.mark.parametrize("D,G,q", SHAPES)
@pytest.mark.parametrize("big,small", [(24, 0), (60, 0), (90, 0), (0, -60), (60, -40), (110, 0), (100, -80)])
def test_mxfp4_values_of_any_scale(orc, D, G, q, big, small):
    """Values of 2^small beside ones of 2^big: tokens that a row does not see, and ones whose probability is 0, leave the
    others' values as they are.  In every second block of 32 channels the large values are elsewhere."""
    n = 150
    p = Problem("mxfp4", D, 1, G, 16, [n, 40], [q, 1], seed=D + q)
    f = np.full((n, D), 2.0 ** small)
    block = np.arange(D) // 32 % 2
    loud = [n - 1, n - max(q // 2, 1), 7, 100]  # seen by the last rows alone, and by all
    for t in loud:
        f[t, block == (t == 100)] = 2.0 ** big
    k = _rand((n, 1, D), 1)
    for t in (7, 100):
        k[t, 0, 3] = -2.0 ** 16  # so that its probability is 0
    p.q[..., 3] = 4.0
    v = (_rand((n, 1, D), 2).double() * torch.from_numpy(f)[:, None]).to(torch.bfloat16)
    _rewrite(p, k, v)
    out, lse = p.run(out_dtype=torch.float32)
    kh.check_attention(out, lse, _reference(p, {0: [7, 100]}), "2^%d beside 2^%d" % (big, small))


@pytest.mark.parametrize("D,G,q", [(64, 1, 3), (128, 5, 4), (256, 2, 3), (64, 1, 60), (128, 1, 70)])
def test_mxfp4_values_that_are_no_numbers_stay_with_the_rows_that_see_them(orc, D, G, q):
    p = Problem("mxfp4", D, 1, G, 16, [90], [q], seed=12)
    pos = kh.positions(D, "mxfp4")
    ref = p.ref()
    t = 89  # seen by the last row alone
    p.cache[p.table[0, t // 16], :, 0, pos[3][t % 16]] = 0xFF
    out, lse = p.run(out_dtype=torch.float32)
    kh.check_attention(out[:-1], lse[:-1], tuple(x[:-1] for x in ref), "0xFF")


@pytest.mark.parametrize("D,G,q", SHAPES)
@pytest.mark.parametrize("exp", [30, 80])
def test_mxfp4_keys_of_any_scale(orc, D, G, q, exp):
    """Blocks of keys 2^exp above and below the others, under queries that are 0 there or as much smaller."""
    n = 150
    p = Problem("mxfp4", D, 1, G, 16, [n, 40], [q, 1], seed=D + q)
    k = _rand((n, 1, D), 1)
    k[::2, :, :32] = (k[::2, :, :32].double() * 2.0 ** exp).to(torch.bfloat16)
    k[1::3, :, 32:] = (k[1::3, :, 32:].double() * 2.0 ** -exp).to(torch.bfloat16)
    p.q[..., :32] = 0
    _rewrite(p, k, _rand((n, 1, D), 2))
    out, lse = p.run(out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(), "2^%d" % exp)


def test_page_calls_that_name_no_row(orc):
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    lens, refs = _dev([0, 0, 0]), _dev([0] * 6)
    cache = torch.zeros(mxq.kv_cache_shape(6, 1, 64, "mxfp4", 16), dtype=torch.uint8, device="cuda")
    none = _dev([])
    state = (table, lens, refs)
    slots = torch.empty(21, dtype=torch.int32, device="cuda")
    assert mxq.kv_reserve(_dev([1]), _dev([20]), *state, cache, 16, slots=slots).tolist() == [0, 2]
    before = [x.clone() for x in (*state, cache)]
    for call in (lambda i: mxq.kv_reserve(none, none, *state, cache, 16, slots=slots, info=i),
                 lambda i: mxq.kv_reserve(none, none, *state, cache, 16, info=i),
                 lambda i: mxq.kv_fork(none, none, *state, 16, info=i),
                 lambda i: mxq.kv_truncate(none, none, *state, 16, info=i)):
        assert call(_dev([7, 7])).tolist() == [0, 0]
        assert call(None).tolist() == [0, 0]
    assert slots.tolist() == [-1] * 21  # an append that follows writes nothing
    assert all(torch.equal(x, y) for x, y in zip((*state, cache), before)) and _status() == 0
    # a captured call that names none
    info = _dev([7, 7])
    slots.fill_(3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mxq.kv_reserve(none, none, *state, cache, 16, slots=slots, info=info)
    g.replay()
    assert info.tolist() == [0, 0] and slots.tolist() == [-1] * 21


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G", [(64, 1), (128, 5), (256, 2)])
def test_query_rows_without_a_bound(orc, fmt, D, G):
    p = Problem(fmt, D, 2, G, 16, [100, 33, 0, 70], [3, 0, 2, 30], seed=D)
    out, lse = p.run(max_q=None)
    kh.check_attention(out, lse, p.ref(), fmt)


@pytest.mark.parametrize("max_q", [3, 40])
def test_starts_that_fall_are_reported(orc, max_q):
    p = Problem("nvfp4", 128, 1, 1, 16, [40, 33], [3, 3], seed=14)
    want = p.run(max_q=max_q)[0]
    out, _ = mxq.kv_attention(p.q.cuda(), torch.from_numpy(p.cache).cuda(), _dev(p.table), _dev(p.lens), "nvfp4",
                              q_start=_dev([0, 3, 2]), max_q=max_q, g_k=p.dk, g_v=p.dv)
    assert _status() == 0x202 and torch.equal(out[:3], want[:3])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,q", SHAPES)
def test_pages_in_front_of_the_window_are_not_looked_at(orc, fmt, D, G, q):
    """A page all of whose tokens lie in front of every row's window may have been given to others."""
    p = Problem(fmt, D, 2, G, 16, [300, 64, 17, 233], [q, 1, 1, q], seed=D + q)
    want = p.run(window=20)
    for b, n in enumerate(p.lens):
        first = max(n - int(p.q_start[b + 1] - p.q_start[b]) + 1 - 20, 0)
        p.table[b, :first // 16] = -7
    out, lse = p.run(window=20)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("exp", range(-14, 4))
def test_mxfp4_small_probabilities_of_small_values(orc, D, exp):
    """A probability of about 2^-24 keeps 2^-28 of the largest one, whatever the values' scale, when a row's values are
    all of that scale: two tokens, each with a value in a channel of its own."""
    p = Problem("mxfp4", D, 1, 7, 16, [2], [1], seed=3)
    k, v = torch.zeros((2, 1, D), dtype=torch.bfloat16), torch.zeros((2, 1, D), dtype=torch.bfloat16)
    k[0, 0, 0] = -24.0
    v[0, 0, 0] = v[1, 0, 1] = 2.0 ** exp
    _rewrite(p, k, v)
    p.q.zero_()
    p.q[0, :, 0] = (0.9 + 0.03 * torch.arange(7)).to(torch.bfloat16)
    out, lse = p.run(scale=LN2, out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(scale=LN2), "2^%d" % exp)
