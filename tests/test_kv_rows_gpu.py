"""Attention over the 4-bit cache with many rows a sequence (drafted tokens, chunks of a prompt): row tiles of every
fill, on both sides of each kernel's sizes, scores that keep rising, masks, graphs and streams."""
import numpy as np
import pytest
import torch

import kv_helpers as kh
from test_kv_cache_gpu import FMTS, Problem, _rand, _status

from nvfp4_block_scaled_mx_b200 import mxq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def orc():
    import oracle

    oracle.build()
    return oracle


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,q", [(1, 9), (16, 1), (17, 1), (1, 32), (3, 11), (4, 16), (5, 13), (2, 64), (3, 43), (1, 257)])
def test_row_tiles_of_every_fill(orc, fmt, D, G, q):
    # lengths in front of, at and behind a tile of tokens; fewer tokens than queries; none at all
    p = Problem(fmt, D, 2, G, 32, [385, 0, 128, 7], [q, max(q // 2, 1), q, q], seed=G * q)
    out, lse = p.run(out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(), "%s D%d G%d q%d" % (fmt, D, G, q))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,q", [(5, 6), (5, 40)])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 37), (True, 200), (False, 0), (False, 150)])
def test_masks_in_row_tiles(orc, fmt, D, G, q, causal, window):
    p = Problem(fmt, D, 1, G, 16, [530, 33, 256], [q, 3, 1], seed=q)
    out, lse = p.run(causal=causal, window=window)
    kh.check_attention(out, lse, p.ref(causal=causal, window=window), "%s D%d %s %d" % (fmt, D, causal, window))


def _rewrite(p, k, v, rule="ceil"):
    """The problem's cache with new keys and values [tokens of sequence 0, H, D]."""
    slots = np.full(p.cache.shape[0] * p.page, -1)
    pos = np.arange(p.lens[0])
    kk = torch.zeros((len(slots), p.H, p.D), dtype=torch.bfloat16)
    vv = torch.zeros_like(kk)
    at = p.table[0, pos // p.page] * p.page + pos % p.page
    kk[at], vv[at] = k, v
    slots[at] = at
    p.cache[:] = 0
    kh.append(p.cache, kk, vv, slots, p.fmt, rule, p.gk, p.gv)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q", [20, 150])
@pytest.mark.parametrize("step", [0.05, 0.6, 40.0])
def test_scores_that_keep_rising(orc, fmt, D, q, step):
    """Every token's score exceeds the last one's by about `step`: the running maximum moves inside tiles
    and from tile to tile, in some rows up and in others down."""
    p = Problem(fmt, D, 1, 1, 16, [700], [q], seed=21)
    n = p.lens[0]
    top = step * n
    k = _rand((n, 1, D), 22) * 0.01
    k[:, 0, 3] = (torch.arange(n) / n * 4).to(torch.bfloat16)
    _rewrite(p, k, _rand((n, 1, D), 23))
    p.q[..., 3] = top / 4
    p.q[::3, :, 3] = -top / 4
    out, lse = p.run(scale=1.0, out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(scale=1.0), "%s %g" % (fmt, step))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q", [20, 150])
def test_mxfp4_scales_that_move(orc, D, q):
    """V's scales rise by 2^20 along the tokens in some channels and fall in others; keys' scales jump from
    token to token and from block to block."""
    p = Problem("mxfp4", D, 1, 1, 16, [640], [q], seed=31)
    n = p.lens[0]
    pos = np.arange(n)
    side = np.where(np.arange(D) % 64 < 32, 1, -1)
    f = np.exp2((pos[:, None] / 32.0).round() * side[None])
    v = (_rand((n, 1, D), 32).float() * torch.from_numpy(f)[:, None].float()).to(torch.bfloat16)
    f = np.exp2(pos[:, None] * 7 % 13 * side[None] - 8.0)
    k = (_rand((n, 1, D), 33).float() * torch.from_numpy(f)[:, None].float()).to(torch.bfloat16)
    _rewrite(p, k, v, "even")
    out, lse = p.run(out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(), "scales")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kscale,vscale", [(1e-6, 1e-6), (40.0, 1e-3), (3.0, 3e4), (1e3, 1e20)])
@pytest.mark.parametrize("q", [20, 80])
def test_magnitudes_in_row_tiles(orc, fmt, kscale, vscale, q):
    p = Problem(fmt, 128, 1, 1, 16, [300], [q], seed=3, kscale=kscale, vscale=vscale)
    p.q[::2, :, 5] *= 1000
    out, lse = p.run(out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(), "%s %g %g" % (fmt, kscale, vscale))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("q", [20, 70])
def test_what_no_row_sees_may_hold_anything(orc, fmt, q):
    p = Problem(fmt, 128, 2, 1, 16, [237, 164, 0], [q, 1, 2], seed=11)
    ref = p.ref(window=50)
    clean = p.run(window=50)
    pos = kh.positions(128, fmt)
    for b, n in enumerate(p.lens):
        first = max(n - [q, 1, 2][b] + 1 - 50, 0)
        for t in range(-(-n // 16) * 16):
            if not first <= t < n:
                for x in pos:
                    p.cache[p.table[b, t // 16], :, 0, x[t % 16]] = 0xFF
    out, lse = p.run(window=50)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    kh.check_attention(out, lse, ref, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,most", [(5, 4), (2, 48)])
def test_many_ragged_sequences_captured_and_on_two_streams(orc, fmt, G, most):
    rng = np.random.RandomState(5)
    B = 70
    lens = [int(x) for x in rng.randint(0, 400, B)]
    qlens = [int(x) for x in rng.randint(0, most + 1, B)]
    p = Problem(fmt, 128, 2, G, 16, lens, qlens, seed=41, extra_rows=3)
    wide = torch.zeros((p.q.shape[0], 2 * G + 3, 128), dtype=torch.bfloat16)
    wide[:, 2:2 + 2 * G] = p.q
    q = wide.cuda()[:, 2:2 + 2 * G]
    cache, table, dl, qs = torch.from_numpy(p.cache).cuda(), _dev(p.table), _dev(p.lens), _dev(p.q_start)
    live = p.q_start[-1]
    ref = p.ref()
    ws = torch.full((mxq.kv_attention_workspace(B, most, 2 * G, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")

    def call(out=None, lse=None, workspace=None):
        return mxq.kv_attention(q, cache, table, dl, fmt, g_k=p.dk, g_v=p.dv, q_start=qs, max_q=most, out=out, lse=lse,
                                workspace=workspace)

    out = torch.full((live + 3, 2 * G, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((live + 3, 2 * G), 7.0, device="cuda")
    call(out, lse, ws)
    kh.check_attention(out[:live], lse[:live], tuple(x[:live] for x in ref), "batch")
    assert (out[live:] == 7).all() and (lse[live:] == 7).all()
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream(), torch.cuda.Stream()] * 2:
        with torch.cuda.stream(s):
            outs.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(o[:live], out[:live]) and torch.equal(z[:live], lse[:live]) for o, z in outs)
    # two captured calls that share a workspace, replayed with other lengths and starts
    o2, z2 = torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, lse, ws)
        call(o2, z2, ws)
    p.lens = [int(x) for x in rng.permutation(lens)]
    p.lens = [min(n, 16 * int((p.table[b] >= 0).sum())) for b, n in enumerate(p.lens)]
    qlens = [min(x, most) for x in reversed(qlens)]
    p.q_start = np.concatenate([[0], np.cumsum(qlens)])
    dl.copy_(_dev(p.lens))
    qs.copy_(_dev(p.q_start))
    g.replay()
    torch.cuda.synchronize()
    assert _status() == 0 and torch.equal(out[:live], o2[:live])
    kh.check_attention(out[:live], lse[:live], tuple(x[:live] for x in p.ref()), "replayed")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("q", [20, 70])
def test_bad_pages_in_row_tiles_are_reported(orc, fmt, q):
    p = Problem(fmt, 128, 1, 1, 16, [300, 200], [q, q], seed=14)
    cache, qd, qs = torch.from_numpy(p.cache).cuda(), p.q.cuda(), _dev(p.q_start)

    def call(table, lens, starts=qs):
        out, _ = mxq.kv_attention(qd, cache, _dev(table), _dev(lens), fmt, g_k=p.dk, g_v=p.dv, q_start=starts, max_q=q)
        return out, _status()

    good, st = call(p.table, p.lens)
    assert st == 0
    for bad_page in (p.cache.shape[0], -1, 2 ** 31 - 1):
        bad = p.table.copy()
        bad[1, 3] = bad_page
        out, st = call(bad, p.lens)
        assert st == 0x201 and torch.equal(out[:q], good[:q])
    assert call(p.table, [300, 10 ** 9])[1] in (0x201, 0x203)
    out, st = call(p.table, [300, -3])
    assert st == 0 and not out[q:].any() and torch.equal(out[:q], good[:q])
    for starts in ([0, q, 2 * q + 1], [-1, q, 2 * q], [0, 2 * q, q], [0, q + 1, 2 * q]):
        assert call(p.table, p.lens, _dev(starts))[1] == 0x202, starts


@pytest.mark.parametrize("q", [1, 20, 70])
def test_memory_of_a_call_on_a_given_stream(orc, q):
    """What a call allocates for a stream it is given is not handed to the current stream meanwhile."""
    p = Problem("nvfp4", 128, 8, 1, 64, [3000] * 4, [q] * 4, seed=51)
    want, _ = p.run()
    cache, table, lens, qd = torch.from_numpy(p.cache).cuda(), _dev(p.table), _dev(p.lens), p.q.cuda()
    size = mxq.kv_attention_workspace(4, q, 8, 8, 128)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs, others = [], []
    for _ in range(30):
        outs.append(mxq.kv_attention(qd, cache, table, lens, "nvfp4", max_q=q, g_k=p.dk, g_v=p.dv, stream=s)[0])
        others.append(torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
        del others[:-1]
    torch.cuda.synchronize()
    assert _status() == 0 and all(torch.equal(o, want) for o in outs)


def test_pages_and_tokens_on_a_given_stream(orc):
    """Reserve, append, attention, fork and compaction in a row on a stream that is not the current one."""
    D, H, page, P = 128, 2, 16, 12
    s = torch.cuda.Stream()
    cache = torch.zeros(mxq.kv_cache_shape(P, H, D, "mxfp4", page), dtype=torch.uint8, device="cuda")
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    slots = torch.empty(37, dtype=torch.int32, device="cuda")
    k, v, q = _rand((37, H, D), 1).cuda(), _rand((37, H, D), 2).cuda(), _rand((1, 2 * H, D), 3).cuda()
    rows = [_dev([i]) for i in range(3)]
    count, none = _dev([37]), _dev([0])
    torch.cuda.synchronize()
    state = (table, lens, refs)
    infos = [mxq.kv_reserve(rows[1], count, *state, cache, page, slots=slots, stream=s)]
    mxq.kv_append(k, v, cache, slots, "mxfp4", stream=s)
    infos.append(mxq.kv_fork(rows[1], rows[2], *state, page, stream=s))
    infos.append(mxq.kv_truncate(rows[1], none, *state, page, stream=s))
    infos.append(mxq.kv_compact(*state, cache, page, stream=s))
    out, lse = mxq.kv_attention(q, cache, table[2:], lens[2:], "mxfp4", stream=s)
    torch.cuda.synchronize()
    assert [i.tolist() for i in infos] == [[0, 3], [0, 3], [0, 3], [0, 3]] and _status() == 0
    ref = kh.attention(q.double().cpu().numpy(), cache.cpu().numpy(), table[2:].cpu().numpy(), [37], [0, 1], "mxfp4",
                       np.float64(np.float32(D ** -0.5)), True, 0, None, None)
    kh.check_attention(out, lse, ref, "stream")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,q", [(5, 1), (1, 20), (1, 80)])
def test_scales_of_zero_and_below(orc, fmt, G, q):
    p = Problem(fmt, 128, 1, G, 16, [200, 1], [q, 1], seed=61)
    for scale in (0.0, -0.3):
        out, lse = p.run(scale=scale, out_dtype=torch.float32)
        kh.check_attention(out, lse, p.ref(scale=scale), "%s %g" % (fmt, scale))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,q", [(5, 1), (1, 20), (1, 80)])
def test_a_query_that_is_not_finite_leaves_the_other_rows(orc, fmt, G, q):
    p = Problem(fmt, 128, 1, G, 16, [200, 33], [q, 1], seed=62)
    ref = p.ref()
    bad = p.q.clone()
    flat = bad.view(-1, 128)
    hurt = [1, flat.shape[0] - 1]
    flat[hurt[0], 7] = float("inf")
    flat[hurt[1], 9] = float("nan")
    out, lse = p.run(bad, out_dtype=torch.float32)
    keep = [i for i in range(flat.shape[0]) if i not in hurt]
    kh.check_attention(out.view(-1, 1, 128)[keep], lse.view(-1, 1)[keep],
                       tuple(x.reshape(-1, 1, x.shape[-1])[keep] if x.ndim == 3 else x.reshape(-1, 1)[keep] for x in ref), fmt)
    assert not torch.isfinite(out.view(-1, 128)[hurt[1]]).any()


def _guarded(shape, dtype):
    """A tensor inside an allocation of 0xA5 bytes, 4096 on either side."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    return raw, raw[4096:4096 + n].view(dtype).view(shape)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,q", [(64, 3, 1), (128, 5, 1), (256, 5, 3), (128, 5, 4), (128, 5, 31), (64, 1, 129), (256, 2, 40)])
def test_nothing_around_the_outputs_is_written(orc, fmt, D, G, q):
    p = Problem(fmt, D, 2, G, 16, [700, 0, 33, 1201, 5], [q, q, 1, q, 1], seed=71)
    rows = int(p.q_start[-1])
    raws = []

    def guarded(shape, dtype):
        raw, t = _guarded(shape, dtype)
        raws.append((raw, t.numel() * t.element_size()))
        return t

    cache = guarded(p.cache.shape, torch.uint8)
    cache.zero_()
    k, v = _rand((p.cache.shape[0] * 16, 2, D), 71), _rand((p.cache.shape[0] * 16, 2, D), 72)
    slots = torch.arange(k.shape[0], dtype=torch.int32, device="cuda")
    mxq.kv_append(k.cuda(), v.cuda(), cache, slots, fmt, g_k=p.dk, g_v=p.dv)
    assert np.array_equal(cache.cpu().numpy(), p.cache)
    ko, vo = guarded(k.shape, torch.bfloat16), guarded(v.shape, torch.bfloat16)
    mxq.kv_read(cache, slots, fmt, D, g_k=p.dk, g_v=p.dv, k_out=ko, v_out=vo)
    out, lse = guarded((rows, 2 * G, D), torch.bfloat16), guarded((rows, 2 * G), torch.float32)
    ws = guarded((mxq.kv_attention_workspace(5, q, 2 * G, 2, D),), torch.uint8)
    mxq.kv_attention(p.q.cuda(), cache, _dev(p.table), _dev(p.lens), fmt, q_start=_dev(p.q_start), max_q=q, g_k=p.dk, g_v=p.dv,
                     out=out, lse=lse, workspace=ws)
    assert _status() == 0
    kh.check_attention(out, lse, p.ref(), "guarded")
    for raw, n in raws:
        assert (raw[:4096] == 0xA5).all() and (raw[4096 + n:] == 0xA5).all()
