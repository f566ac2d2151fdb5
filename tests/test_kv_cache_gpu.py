"""The 4-bit key/value cache on the GPU: append (bytes against the oracle's quantizer), read, attention
against 64-bit sums, over formats, head sizes, page sizes, lengths, masks, strides and streams."""
import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_block_scaled_mx_b200 import mxq

pytestmark = pytest.mark.gpu

FMTS = ["nvfp4", "mxfp4"]


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def _g(fmt, *xs):
    """Global scales (numpy fp32) and their device tensors; None for MXFP4."""
    if fmt == "mxfp4":
        return (None, None), (None, None)
    h = [np.float32(max(float(x.float().abs().max()), 1e-3) * 1.01 / 2688) for x in xs]
    return tuple(h), tuple(torch.tensor([v], device="cuda") for v in h)


def _status():
    torch.cuda.synchronize()
    return mxq.mxq_device_status(reset=True)


@pytest.mark.parametrize("fmt,rule", [("nvfp4", "even"), ("mxfp4", "ceil"), ("mxfp4", "even")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (37, 3, 48), (130, 8, 64), (17, 2, 1024)])
def test_append_matches_the_oracle_byte_for_byte(orc, fmt, rule, D, T, H, page):
    k, v = _rand((T, H, D), T + D), _rand((T, H, D), T + D + 1, 0.01)
    v[T // 2] = 0
    k[0, 0, :4] = torch.tensor([3e38, -1e-38, 0.0, -0.0])
    (gk, gv), (dk, dv) = _g(fmt, k, v)
    pages = -(-T // page) + 2
    rng = np.random.RandomState(T)
    slots = rng.permutation(pages * page)[:T]
    slots[T // 3] = -1 if T > 1 else slots[0]
    start = rng.randint(0, 256, mxq.kv_cache_shape(pages, H, D, fmt, page)).astype(np.uint8)
    cache = torch.from_numpy(start.copy()).cuda()
    mxq.kv_append(k.cuda(), v.cuda(), cache, torch.tensor(slots, dtype=torch.int32, device="cuda"), fmt, rule, dk, dv)
    kh.append(start, k, v, slots, fmt, rule, gk, gv)
    assert np.array_equal(cache.cpu().numpy(), start)
    assert _status() == 0
    # reading back gives what fake quantization gives
    ks, vs = mxq.kv_read(cache, torch.tensor(slots, dtype=torch.int32, device="cuda"), fmt, D, dk, dv)
    for x, got, g in ((k, ks, dk), (v, vs, dv)):
        want = mxq.fake_quantize(x.cuda().reshape(T * H, D), fmt, rule, g).reshape(T, H, D)
        want[torch.tensor(slots < 0).cuda()] = 0
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
def test_append_takes_strided_rows_and_leaves_the_rest(orc, fmt):
    T, H, D, page = 33, 4, 128, 32
    rows = _rand((T, 3 * H + 1, D), 5).cuda()
    k, v = rows[:, 1:1 + H], rows[:, 1 + 2 * H:]
    (gk, gv), (dk, dv) = _g(fmt, k, v)
    cache = torch.full(mxq.kv_cache_shape(3, H, D, fmt, page), 0xA5, dtype=torch.uint8, device="cuda")
    want = cache.cpu().numpy()
    slots = np.arange(T) + 20
    mxq.kv_append(k, v, cache, torch.tensor(slots, dtype=torch.int32, device="cuda"), fmt, "ceil", dk, dv)
    kh.append(want, k, v, slots, fmt, "ceil", gk, gv)
    assert np.array_equal(cache.cpu().numpy(), want)
    # one token for all slots: a broadcast input (stride 0)
    one = _rand((1, H, D), 6).cuda().expand(T, H, D)
    mxq.kv_append(one, one, cache, torch.tensor(slots, dtype=torch.int32, device="cuda"), fmt, "ceil", dk, dk)
    kh.append(want, one, one, slots, fmt, "ceil", gk, gk)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_bad_slots_are_skipped_and_reported(orc):
    T, H, D, page, pages = 6, 2, 64, 16, 2
    k = _rand((T, H, D), 7).cuda()
    cache = torch.zeros(mxq.kv_cache_shape(pages, H, D, "mxfp4", page), dtype=torch.uint8, device="cuda")
    want = cache.cpu().numpy()
    slots = np.array([3, pages * page, 5, 2 ** 31 - 1, -7, 31])
    ds = torch.tensor(slots, dtype=torch.int32, device="cuda")
    mxq.kv_append(k, k, cache, ds, "mxfp4")
    assert _status() == 0x200
    kh.append(want, k, k, np.where(slots < pages * page, slots, -1), "mxfp4", "ceil", None, None)
    assert np.array_equal(cache.cpu().numpy(), want)
    ks, _ = mxq.kv_read(cache, ds, "mxfp4", D)
    assert _status() == 0x200
    assert not ks[[1, 3, 4]].any() and ks[[0, 2, 5]].any()
    assert mxq.kv_append(k[:0], k[:0], cache, ds[:0], "mxfp4") is None and _status() == 0


class Problem:
    """A filled cache, queries and their 64-bit result."""

    def __init__(self, fmt, D, H, G, page, lens, qlens=None, seed=0, kscale=1.0, vscale=1.0, extra_rows=0):
        self.fmt, self.D, self.H, self.G, self.page, self.lens = fmt, D, H, G, page, lens
        self.B = len(lens)
        rng = np.random.RandomState(seed + 1)
        used = [-(-max(n, 0) // page) for n in lens]
        P = sum(used) + 2
        order = rng.permutation(P)
        cols = max(used + [1]) + 1
        self.table = np.full((self.B, cols), -5)  # behind a sequence's end: never looked at
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        k, v = _rand((P * page, H, D), seed, kscale), _rand((P * page, H, D), seed + 1, vscale)
        (self.gk, self.gv), (self.dk, self.dv) = _g(fmt, k, v)
        self.cache = np.zeros(mxq.kv_cache_shape(P, H, D, fmt, page), np.uint8)
        kh.append(self.cache, k, v, np.arange(P * page), fmt, "ceil", self.gk, self.gv)
        qlens = qlens or [1] * self.B
        self.q_start = np.concatenate([[0], np.cumsum(qlens)])
        self.max_q = max(qlens + [1])
        self.q = _rand((self.q_start[-1] + extra_rows, H * G, D), seed + 2)

    def ref(self, scale=None, causal=True, window=0, q=None):
        q = self.q if q is None else q
        return kh.attention(q.double().numpy(), self.cache, self.table, self.lens, self.q_start, self.fmt,
                            np.float64(np.float32(self.D ** -0.5 if scale is None else scale)), causal, window, self.gk,
                            self.gv)

    def run(self, q=None, **kw):
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        kw.setdefault("q_start", dev(self.q_start))
        kw.setdefault("max_q", self.max_q)
        out = mxq.kv_attention((self.q if q is None else q).cuda(), torch.from_numpy(self.cache).cuda(), dev(self.table),
                               dev(self.lens), self.fmt, g_k=self.dk, g_v=self.dv, **kw)
        assert _status() == 0
        return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G,page,lens", [
    (1, 1, 16, [1]), (2, 5, 16, [15, 16, 17, 0, 1]), (8, 5, 64, [1009]), (2, 8, 48, [31, 700, 33]), (1, 16, 32, [257, 64]),
    (3, 12, 128, [130, 1, 999]), (2, 40, 1024, [1025, 5])])
def test_attention_single_tokens(orc, fmt, D, H, G, page, lens):
    p = Problem(fmt, D, H, G, page, lens, seed=D + G)
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = p.run(out_dtype=dtype)
        kh.check_attention(out, lse, p.ref(), "%s D%d G%d %s" % (fmt, D, G, dtype))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 37), (False, 0), (False, 20)])
def test_attention_several_tokens_and_masks(orc, fmt, D, causal, window):
    # more query tokens than cached ones, none at all, one, a chunk over several row tiles
    p = Problem(fmt, D, 2, 3, 32, [3, 200, 40, 130, 0], [5, 4, 0, 33, 2], seed=D + window)
    out, lse = p.run(causal=causal, window=window)
    kh.check_attention(out, lse, p.ref(causal=causal, window=window), "%s D%d %s %d" % (fmt, D, causal, window))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,q", [(1, 8), (1, 9), (5, 4), (8, 2), (5, 70)])
def test_attention_row_tiles(orc, fmt, G, q):
    p = Problem(fmt, 128, 2, G, 16, [333, 90], [q, q], seed=q)
    out, lse = p.run(q_start=None)
    kh.check_attention(out, lse, p.ref(), "%s G%d q%d" % (fmt, G, q))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kscale,vscale", [(1e-6, 1e-6), (40.0, 1e-3), (3.0, 3e4), (1e3, 1e20)])
def test_attention_magnitudes(orc, fmt, kscale, vscale):
    p = Problem(fmt, 128, 1, 4, 16, [150], seed=3, kscale=kscale, vscale=vscale)
    q = p.q.clone()
    q[..., 5] *= 1000
    out, lse = p.run(q, out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(q=q), "%s %g %g" % (fmt, kscale, vscale))


def test_attention_mxfp4_values_of_rising_and_falling_scale(orc):
    # the reference scale of V moves up along the tokens by 2^20 in all, in some channels down
    p = Problem("mxfp4", 128, 1, 5, 16, [640], seed=9)
    P, page, H, D = p.cache.shape[0], 16, 1, 128
    pos = np.empty(P * page, np.int64)
    pos[:] = 0
    for c, pg in enumerate(p.table[0][:40]):
        pos[pg * page:(pg + 1) * page] = np.arange(page) + c * page
    f = np.exp2((pos[:, None] / 32.0).round() * np.where(np.arange(D) % 64 < 32, 1, -1)[None])
    v = (_rand((P * page, H, D), 4).float() * torch.from_numpy(f)[:, None].float()).to(torch.bfloat16)
    k = _rand((P * page, H, D), 5)
    p.cache[:] = 0
    kh.append(p.cache, k, v, np.arange(P * page), "mxfp4", "even", None, None)
    out, lse = p.run(out_dtype=torch.float32)
    kh.check_attention(out, lse, p.ref(), "scales")


@pytest.mark.parametrize("fmt", FMTS)
def test_what_is_masked_may_hold_anything(orc, fmt):
    """Bytes of all ones (scales that are not numbers) behind the end, in front of the window, and in the
    pages of no sequence do not reach the result; pages behind the last one are not looked at."""
    p = Problem(fmt, 128, 2, 5, 16, [37, 64, 0], [3, 1, 2], seed=11)
    ref = p.ref(window=20)
    clean = p.run(window=20)
    pos = [x for x in kh.positions(128, fmt)]
    seen = np.zeros((p.cache.shape[0], 16), bool)
    for b, n in enumerate(p.lens):
        first = max(n - [3, 1, 2][b] + 1 - 20, 0)
        for t in range(first, n):
            seen[p.table[b, t // 16], t % 16] = True
    for pg in range(p.cache.shape[0]):
        for r in range(16):
            if not seen[pg, r]:
                for x in pos:
                    p.cache[pg, :, 0, x[r]] = 0xFF
    out, lse = p.run(window=20)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    kh.check_attention(out, lse, ref, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_values_of_a_later_token_do_not_reach_earlier_rows(orc, fmt):
    p = Problem(fmt, 128, 1, 5, 16, [50], [4], seed=12)
    clean = p.run(out_dtype=torch.float32)
    pos = kh.positions(128, fmt)
    t = 49  # seen by the last row alone
    p.cache[p.table[0, t // 16], :, 0, pos[3][t % 16]] = 0x7F if fmt == "nvfp4" else 0xFF
    out, lse = p.run(out_dtype=torch.float32)
    # (the row that sees such a scale, which the quantizer never writes, may get anything)
    if fmt == "nvfp4":  # (an MXFP4 scale of 2^128 moves the reference of its 32 channels)
        assert torch.equal(out[:3], clean[0][:3])
    assert torch.equal(lse[:3], clean[1][:3])


def test_rows_behind_the_last_sequence_are_left(orc):
    p = Problem("nvfp4", 64, 2, 2, 16, [20, 30], [2, 3], seed=13, extra_rows=4)
    out = torch.full((9, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 4), 7.0, device="cuda")
    p.run(out=out, lse=lse)
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    ref = p.ref()
    kh.check_attention(out[:5], lse[:5], tuple(x[:5] for x in ref), "head")


def test_out_of_range_state_is_reported(orc):
    p = Problem("mxfp4", 128, 1, 5, 16, [40, 33], seed=14)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, q = torch.from_numpy(p.cache).cuda(), p.q.cuda()
    good = mxq.kv_attention(q, cache, dev(p.table), dev(p.lens), "mxfp4")
    assert _status() == 0
    bad = p.table.copy()
    bad[1, 1] = p.cache.shape[0]
    out, _ = mxq.kv_attention(q, cache, dev(bad), dev(p.lens), "mxfp4")
    assert _status() == 0x201
    assert torch.equal(out[0], good[0][0])
    mxq.kv_attention(q, cache, dev(p.table), dev([40, 10 ** 9]), "mxfp4")
    assert _status() in (0x203, 0x201)
    out, _ = mxq.kv_attention(q, cache, dev(p.table), dev([40, -3]), "mxfp4")
    assert _status() == 0 and not out[1].any() and torch.equal(out[0], good[0][0])
    for starts in ([0, 1, 3], [-1, 1, 2], [0, 2, 1]):
        mxq.kv_attention(q, cache, dev(p.table), dev(p.lens), "mxfp4", q_start=dev(starts))
        assert _status() == 0x202, starts


@pytest.mark.parametrize("fmt", FMTS)
def test_strided_queries_streams_graphs_and_repetition(orc, fmt):
    p = Problem(fmt, 128, 8, 5, 64, [3000, 777, 64], seed=15)
    wide = torch.zeros((3, 56, 128), dtype=torch.bfloat16)
    wide[:, 8:48] = p.q
    want = p.run()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, table, lens = torch.from_numpy(p.cache).cuda(), dev(p.table), dev(p.lens)
    q = wide.cuda()[:, 8:48]
    ws = torch.full((mxq.kv_attention_workspace(3, 1, 40, 8, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = mxq.kv_attention(q, cache, table, lens, fmt, g_k=p.dk, g_v=p.dv, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # another stream, and two streams at once with a workspace each
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2, s1, s2):
        with torch.cuda.stream(s):
            outs.append(mxq.kv_attention(q, cache, table, lens, fmt, g_k=p.dk, g_v=p.dv))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(z, want[1]) for o, z in outs)
    # a captured call, replayed with other lengths
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = mxq.kv_attention(q, cache, table, lens, fmt, g_k=p.dk, g_v=p.dv, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    lens.copy_(dev([100, 7, 0]))
    g.replay()
    torch.cuda.synchronize()
    p.lens = [100, 7, 0]
    kh.check_attention(out, lse, p.ref(), "replayed")
    assert _status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences_and_long_ones(orc, fmt):
    # uneven batch: cuts inside and between row tiles everywhere; one long sequence
    rng = np.random.RandomState(1)
    p = Problem(fmt, 64, 2, 2, 16, [int(x) for x in rng.randint(0, 300, 150)], seed=16)
    out, lse = p.run()
    kh.check_attention(out, lse, p.ref(), "batch")
    p = Problem(fmt, 128, 1, 5, 64, [30011], seed=17)
    out, lse = p.run()
    kh.check_attention(out, lse, p.ref(), "long")


def test_an_offset_past_32_bits(orc):
    """Pages whose bytes lie behind 4 GiB of the cache."""
    H, D, page, fmt = 8, 256, 64, "nvfp4"
    per = H * 4 * kh.unit_bytes(D, fmt)
    P = (1 << 32) // per + 40
    cache = torch.zeros(mxq.kv_cache_shape(P, H, D, fmt, page), dtype=torch.uint8, device="cuda")
    k, v = _rand((70, H, D), 1), _rand((70, H, D), 2)
    (gk, gv), (dk, dv) = _g(fmt, k, v)
    pages = [P - 1, P - 3]
    slots = [pages[t // page] * page + t % page for t in range(70)]
    ds = torch.tensor(slots, dtype=torch.int32, device="cuda")
    mxq.kv_append(k.cuda(), v.cuda(), cache, ds, fmt, "even", dk, dv)
    ks, _ = mxq.kv_read(cache, ds, fmt, D, dk, dv)
    want = mxq.fake_quantize(k.cuda().reshape(-1, D), fmt, "even", dk).reshape(k.shape)
    assert torch.equal(ks.view(torch.int16), want.view(torch.int16))
    small = cache[[P - 3, P - 1]].cpu().numpy()
    q = _rand((1, 2 * H, D), 3)
    ref = kh.attention(q.double().numpy(), small, np.array([[1, 0]]), [70], [0, 1], fmt, np.float64(np.float32(1 / 16)), True,
                       0, gk, gv)
    out, lse = mxq.kv_attention(q.cuda(), cache, torch.tensor([pages], dtype=torch.int32, device="cuda"),
                                torch.tensor([70], dtype=torch.int32, device="cuda"), fmt, g_k=dk, g_v=dv)
    assert _status() == 0
    kh.check_attention(out, lse, ref, "far")
