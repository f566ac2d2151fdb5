"""CPU checks of the key/value cache's entry points: sizes, refusals before any launch, and the
binding's guards on types, shapes and buffer sizes."""
import ctypes

import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_block_scaled_mx_b200 import build as mxq_build
from nvfp4_block_scaled_mx_b200 import mxq

P = 0x10000  # never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def L():
    mxq_build.build()
    return mxq.lib()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_unit_layout_is_a_bijection(L, fmt, D):
    n = ctypes.c_size_t()
    assert L.mxq_kv_unit_bytes(D, mxq.FMT[fmt], ctypes.byref(n)) == 0 and n.value == kh.unit_bytes(D, fmt)
    at = np.concatenate([p.ravel() for p in kh.positions(D, fmt)])
    assert sorted(at.tolist()) == list(range(n.value))


def test_sizes_and_unsupported(L):
    n = ctypes.c_size_t()
    assert L.mxq_kv_unit_bytes(128, mxq.MXFP8, ctypes.byref(n)) == -4
    assert L.mxq_kv_unit_bytes(96, mxq.MXFP4, ctypes.byref(n)) == -2
    assert L.mxq_kv_unit_bytes(128, mxq.MXFP4, None) == -1
    assert L.mxq_kv_attention_workspace_size(4, 1, 40, 8, 128) > 0
    for bad in ((-1, 1, 40, 8, 128), (4, 0, 40, 8, 128), (4, 1, 41, 8, 128), (4, 1, 40, 8, 96), (4, 1 << 28, 40, 8, 128),
                (4, 1, 0, 8, 128), (4, 1, 8, 0, 128)):
        assert L.mxq_kv_attention_workspace_size(*bad) == 0
    assert L.mxq_kv_reserve_workspace_size(4097) == 0 and L.mxq_kv_reserve_workspace_size(4) >= 36
    assert L.mxq_kv_compact_workspace_size(0) == 0 and L.mxq_kv_compact_workspace_size(10) >= 124
    assert mxq.kv_cache_shape(7, 8, 128, "nvfp4", 64, 3) == (3, 7, 8, 4, 2304)
    with pytest.raises(ValueError):
        mxq.kv_cache_shape(7, 8, 128, "nvfp4", 24)


def _append(L, **kw):
    a = dict(k=P, v=P, tokens=4, heads=8, dim=128, kt=1024, kh=128, vt=1024, vh=128, slots=P, fmt=0, rule=1, gk=None, gv=None,
             cache=P, pages=4, page=16)
    a.update(kw)
    return L.mxq_kv_append(*a.values(), None)


def test_append_refusals(L):
    for kw, code in ((dict(fmt=2), -4), (dict(fmt=5), -4), (dict(rule=7), -4), (dict(k=None), -1), (dict(slots=None), -1),
                     (dict(cache=None), -1), (dict(fmt=1), -1), (dict(fmt=1, gk=P), -1), (dict(dim=96), -2),
                     (dict(heads=0), -2), (dict(page=24), -2), (dict(page=2048), -2), (dict(pages=0), -2),
                     (dict(pages=1 << 27), -2), (dict(tokens=-1), -2), (dict(tokens=1 << 27), -2), (dict(kt=1023), -2),
                     (dict(vh=-128), -2), (dict(k=P + 8), -3), (dict(cache=P + 4), -3), (dict(slots=P + 2), -3)):
        assert _append(L, **kw) == code, kw
        if "rule" in kw or "kt" in kw or "vh" in kw or kw.get("k", P) is None:
            continue
        r = dict(cache=P, pages=4, page=16, heads=8, dim=128, fmt=0, slots=P, tokens=4, gk=None, gv=None, ko=P, vo=P)
        r.update({("ko" if x == "k" else x): y for x, y in kw.items()})
        assert L.mxq_kv_read(*r.values(), None) == code, kw
    # what is in order reaches the device check, tokens = 0 too
    if not torch.cuda.is_available():
        assert _append(L) in (-6, -8) and _append(L, tokens=0, k=None, v=None, slots=None) in (-6, -8)


def _attention(L, **kw):
    a = dict(q=P, rows=4, qt=5120, qh=128, cache=P, pages=64, page=16, heads=40, kv=8, dim=128, fmt=0, table=P, ts=16, cols=16,
             lens=P, batch=4, start=None, max_q=1, scale=0.1, causal=1, window=0, gk=None, gv=None, ot=0, out=P, lse=None,
             ws=P, wb=1 << 30)
    a.update(kw)
    return L.mxq_kv_attention(*a.values(), None)


def test_attention_refusals(L):
    for kw, code in ((dict(fmt=2), -4), (dict(ot=2), -4), (dict(q=None), -1), (dict(table=None), -1), (dict(lens=None), -1),
                     (dict(out=None), -1), (dict(ws=None), -1), (dict(fmt=1, gk=P), -1), (dict(heads=41), -2),
                     (dict(kv=0), -2), (dict(dim=80), -2), (dict(page=8), -2), (dict(rows=5), -2), (dict(rows=-1), -2),
                     (dict(max_q=0), -2), (dict(ts=15), -2), (dict(cols=0, ts=16), -2), (dict(cols=1 << 27, ts=1 << 27), -2),
                     (dict(window=-1), -2), (dict(qt=5121), -2), (dict(batch=-1), -2), (dict(max_q=1 << 27, start=P), -2),
                     (dict(q=P + 2), -3), (dict(out=P + 8), -3), (dict(ws=P + 4), -3), (dict(start=P + 1), -3)):
        assert _attention(L, **kw) == code, kw
    if not torch.cuda.is_available():
        assert _attention(L) in (-6, -8) and _attention(L, rows=0, batch=0, q=None, out=None) in (-6, -8)


def _pages(L, call, **kw):
    a = dict(s=P, o=P, n=4, table=P, rows=8, stride=16, cols=16, lens=P, refs=P, pages=64, page=16)
    if call == "mxq_kv_reserve":
        a.update(cache=P, layers=2, ls=64 * 4352, pb=4352, slots=P, cap=4, info=P, ws=P, wb=1 << 20)
    elif call == "mxq_kv_compact":
        for x in ("s", "o", "n"):
            del a[x]
        a.update(cache=P, layers=2, ls=64 * 4352, pb=4352, info=P, ws=P, wb=1 << 20)
    else:
        a.update(info=P)
    if not set(kw) <= set(a):
        return None
    a.update(kw)
    return getattr(L, call)(*a.values(), None)


@pytest.mark.parametrize("call", ["mxq_kv_reserve", "mxq_kv_fork", "mxq_kv_truncate", "mxq_kv_compact"])
def test_page_refusals(L, call):
    for kw, code in ((dict(s=None), -1), (dict(o=None), -1), (dict(table=None), -1), (dict(lens=None), -1),
                     (dict(refs=None), -1), (dict(info=None), -1), (dict(cache=None), -1), (dict(ws=None), -1),
                     (dict(n=4097), -2), (dict(n=-1), -2), (dict(rows=0), -2), (dict(rows=65537), -2), (dict(stride=15), -2),
                     (dict(cols=0), -2), (dict(pages=0), -2), (dict(pages=1 << 28), -2), (dict(page=17), -2),
                     (dict(layers=0), -2), (dict(ls=63 * 4352), -2), (dict(pb=4351), -2), (dict(cap=-1), -2),
                     (dict(table=P + 2), -3), (dict(info=P + 1), -3), (dict(cache=P + 8), -3), (dict(ws=P + 4), -3),
                     (dict(wb=16), -5)):
        got = _pages(L, call, **kw)
        assert got in (None, code), (call, kw, got)
    if not torch.cuda.is_available():
        assert _pages(L, call) in (-6, -8)


def test_binding_guards(monkeypatch):
    mxq_build.build()
    calls = []
    monkeypatch.setattr(mxq, "_call", lambda name, device, stream, *args: calls.append(name))
    i32 = lambda *x: torch.zeros(x, dtype=torch.int32)  # noqa: E731
    bf = lambda *x: torch.zeros(x, dtype=torch.bfloat16)  # noqa: E731
    cache = torch.zeros(mxq.kv_cache_shape(4, 2, 64, "mxfp4", 32), dtype=torch.uint8)
    k = bf(5, 2, 64)
    mxq.kv_append(k, k, cache, i32(5), "mxfp4")
    mxq.kv_append(bf(5, 6, 64)[:, 2:4], k, cache, i32(5), "mxfp4")
    mxq.kv_read(cache, i32(5), "mxfp4", 64)
    mxq.kv_attention(bf(3, 4, 64), cache, i32(3, 2), i32(3), "mxfp4")
    mxq.kv_attention(bf(3, 4, 64), cache, i32(3, 4)[:, :2], i32(3), "mxfp4")
    state = (i32(3, 2), i32(3), i32(4))
    mxq.kv_reserve(i32(2), i32(2), *state, cache, 32, slots=i32(4))
    mxq.kv_fork(i32(2), i32(2), *state, 32)
    mxq.kv_truncate(i32(2), i32(2), *state, 32)
    mxq.kv_compact(*state, cache, 32)
    n = len(calls)
    assert n == 9
    for bad in (lambda: mxq.kv_append(k.float(), k, cache, i32(5), "mxfp4"),
                lambda: mxq.kv_append(k, k[:4], cache, i32(5), "mxfp4"),
                lambda: mxq.kv_append(k, bf(5, 3, 64), cache, i32(5), "mxfp4"),
                lambda: mxq.kv_append(bf(5, 3, 64), bf(5, 3, 64), cache, i32(5), "mxfp4"),
                lambda: mxq.kv_append(bf(5, 2, 128), bf(5, 2, 128), cache, i32(5), "mxfp4"),
                lambda: mxq.kv_append(bf(5, 2, 128)[..., ::2], k, cache, i32(5), "mxfp4"),
                lambda: mxq.kv_append(k, k, cache, i32(4), "mxfp4"),
                lambda: mxq.kv_append(k, k, cache, i32(5).long(), "mxfp4"),
                lambda: mxq.kv_append(k, k, cache.float(), i32(5), "mxfp4"),
                lambda: mxq.kv_append(k, k, cache, i32(5), "nvfp4", g_k=torch.ones(1), g_v=torch.ones(1)),
                lambda: mxq.kv_read(cache, i32(5), "mxfp4", 64, k_out=bf(4, 2, 64)),
                lambda: mxq.kv_attention(bf(3, 4, 64), cache, i32(3, 2), i32(2), "mxfp4"),
                lambda: mxq.kv_attention(bf(3, 4, 64), cache, i32(2, 3).t(), i32(3), "mxfp4"),
                lambda: mxq.kv_attention(bf(3, 4, 64), cache, i32(3, 2), i32(3), "mxfp4", q_start=i32(3)),
                lambda: mxq.kv_attention(bf(3, 4, 64), cache, i32(3, 2), i32(3), "mxfp4", out=bf(3, 4, 63)),
                lambda: mxq.kv_attention(bf(3, 4, 64), cache, i32(3, 2), i32(3), "mxfp4", lse=torch.zeros(11)),
                lambda: mxq.kv_attention(bf(3, 4, 64), cache, i32(3, 2), i32(3), "mxfp4", out=torch.zeros(3, 4, 64).half()),
                lambda: mxq.kv_reserve(i32(2), i32(1), *state, cache, 32),
                lambda: mxq.kv_reserve(i32(2), i32(2), *state, cache, 16),
                lambda: mxq.kv_reserve(i32(2), i32(2), state[0], state[1], i32(5), cache, 32),
                lambda: mxq.kv_reserve(i32(2), i32(2), i32(3, 4)[:, :2], *state[1:], cache, 32),
                lambda: mxq.kv_fork(i32(2), i32(1), *state, 32),
                lambda: mxq.kv_fork(i32(2), i32(2), state[0], i32(2), state[2], 32),
                lambda: mxq.kv_truncate(i32(2), i32(2).long(), *state, 32),
                lambda: mxq.kv_truncate(i32(2), i32(2), *state, 32, info=i32(1)),
                lambda: mxq.kv_append(k, k, cache[:, :, :, ::2], i32(5), "mxfp4"),
                lambda: mxq.kv_append(k, k, cache.transpose(0, 2), i32(5), "mxfp4"),
                lambda: mxq.kv_compact(*state, cache[:3], 32)):
        with pytest.raises(ValueError):
            bad()
    assert len(calls) == n


def test_host_tensors_are_refused():
    if torch.cuda.is_available():
        pytest.skip("a device is there: the call would name it")
    cache = torch.zeros(mxq.kv_cache_shape(4, 2, 64, "mxfp4", 32), dtype=torch.uint8)
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        mxq.kv_append(k, k, cache, torch.zeros(5, dtype=torch.int32), "mxfp4")
