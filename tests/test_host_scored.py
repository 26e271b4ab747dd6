"""Refusals of the scored decode, of the weights it accumulates and of the
eviction, and their host-side sizes.  No call reaches a GPU: each is rejected
by the host's checks, or is empty."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_kv_cache_04_gb300 as tq
from quantized_kv_cache_04_gb300 import _lib

INV, UNS, WS = -1, -2, -3
P = 0x10000          # a pointer that no rejected call reads


def _decode_args(mods=None, **kw):
    a = dict(preset=2, D=128, B=2, Hq=32, Hk=8, bs=16, qd=0, q=P, cache=P, nb=10, bt=P, bts=4, sl=P, maxlen=64,
             scale=0.1, S=1, signs=P, cent=P, out=P, od=2, lse=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return tuple(a.values()) + (ctypes.byref(mods) if mods is not None else None,)


def _mods(**kw):
    m = _lib.TQScoreMods()
    for k, v in kw.items():
        setattr(m, k, v)
    return m


BAD = [dict(B=-1), dict(Hq=31), dict(Hk=0), dict(q=0), dict(cache=0), dict(bt=0), dict(sl=0), dict(out=0),
       dict(ws=0), dict(ws=P + 4), dict(signs=0), dict(cent=0), dict(maxlen=-1), dict(maxlen=2 ** 30 + 1), dict(S=-1), dict(S=257), dict(nb=-1)]


@pytest.mark.parametrize("bad", range(len(BAD)))
def test_arguments_out_of_range(bad):
    m = _mods(softcap=5.0)
    assert tq.tq_decode_attention_scored(*_decode_args(m, **BAD[bad]), None) == INV
    assert tq.tq_decode_attention_weights(*_decode_args(m, **BAD[bad]), P, 8 * 64, 64, None) == INV


@pytest.mark.parametrize("bad", [dict(softcap=-1.0), dict(softcap=1e-31), dict(softcap=2e30), dict(softcap=float("nan")), dict(softcap=float("inf")),
                                 dict(window=-1), dict(prefix=-1), dict(window=4, prefix=-2)])
def test_modifiers_out_of_range(bad):
    assert tq.tq_decode_attention_scored(*_decode_args(_mods(**bad)), None) == INV
    assert tq.tq_decode_attention_weights(*_decode_args(_mods(**bad)), P, 8 * 64, 64, None) == INV


@pytest.mark.parametrize("bad", [dict(D=64), dict(bs=24), dict(qd=2), dict(od=7), dict(preset=9), dict(Hq=136)])
def test_unsupported(bad):
    assert tq.tq_decode_attention_scored(*_decode_args(_mods(window=3), **bad), None) == UNS
    assert tq.tq_decode_attention_weights(*_decode_args(None, **bad), P, 8 * 64, 64, None) == UNS


def test_workspace_too_small():
    n = tq.tq_decode_scored_workspace_bytes(2, 32, 1)
    assert tq.tq_decode_attention_scored(*_decode_args(_mods(window=3), wsb=n - 1), None) == WS
    n = tq.tq_decode_weights_workspace_bytes(2, 32, 8, 1, 128, 64)
    assert tq.tq_decode_attention_weights(*_decode_args(None, wsb=n - 1), P, 8 * 64, 64, None) == WS


@pytest.mark.parametrize("acc,sb,sh", [(0, 512, 64), (P, 512, 63), (P, 511, 64), (P, 0, 64), (P, 512, 0),
                                       (P, -512, 64), (P, 63, 128), (P, 64, 127)])
def test_sums_that_overlap(acc, sb, sh):
    assert tq.tq_decode_attention_weights(*_decode_args(None), acc, sb, sh, None) == INV
    assert _select(acc=acc, sb=sb, sh=sh) == INV
    if acc:
        assert _compact(acc=acc, sb=sb, sh=sh) == INV


def _select(**kw):
    a = dict(B=2, Hk=8, acc=P, sb=512, sh=64, sl=P, maxlen=64, budget=16, prefix=4, recent=4, keep=P, new=2 * P)
    a.update(kw)
    return tq.tq_evict_select(*a.values(), None)


def _compact(**kw):
    a = dict(preset=2, D=128, B=2, Hk=8, bs=16, cache=P, nb=10, bt=P, bts=4, keep=P, budget=16, sl=P, maxlen=64,
             acc=0, sb=0, sh=0)
    a.update(kw)
    return tq.tq_evict_compact(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(Hk=0), dict(budget=0), dict(prefix=-1), dict(recent=-1),
                                 dict(prefix=10, recent=7), dict(prefix=2 ** 31 - 1, recent=2 ** 31 - 1),
                                 dict(maxlen=-1), dict(maxlen=2 ** 30 + 1, sb=2 ** 40, sh=2 ** 31), dict(sl=0), dict(keep=0), dict(new=0), dict(new=P), dict(new=P + 4), dict(new=P - 4)])
def test_select_arguments(bad):
    assert _select(**bad) == INV


@pytest.mark.parametrize("bad", [dict(B=-1), dict(Hk=0), dict(budget=0), dict(maxlen=-1), dict(maxlen=2 ** 30 + 1), dict(cache=0), dict(bt=0),
                                 dict(keep=0), dict(sl=0), dict(cache=P + 8), dict(nb=-1), dict(bts=-1), dict(D=0)])
def test_compact_arguments(bad):
    assert _compact(**bad) == INV


@pytest.mark.parametrize("bad", [dict(D=64), dict(bs=8), dict(preset=5), dict(preset=2 | 0x200)])
def test_compact_unsupported(bad):
    assert _compact(**bad) == UNS


def test_empty_batches():
    assert tq.tq_decode_attention_scored(*_decode_args(_mods(softcap=1.0), B=0), None) == 0
    assert _select(B=0) == 0 and _compact(B=0) == 0


@pytest.mark.parametrize("max_len,window,prefix", [(0, 0, 0), (1, 0, 0), (64, 0, 5), (1000, 1, 0), (1000, 33, 7),
                                                   (100, 4096, 64), (2 ** 30, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_every_visible_token_has_a_place(max_len, window, prefix):
    """The scores' share of the workspace holds every 32-token tile with a visible token."""
    n = tq.tq_decode_weights_workspace_bytes(1, 4, 4, 1, 128, max_len, window, prefix)
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    tiles = (n - up(4 * 129 * 4) - 256) // (4 * 32 * 4)
    if max_len > 2000:
        assert tiles == -(-max_len // 32)
        return
    for L in range(max_len + 1):
        for lo in range(0, max(1, L), 29):
            first = max(lo, L - window) if window else lo
            see = {t // 32 for t in range(first, L)}
            if window:
                see |= {t // 32 for t in range(lo, min(L, lo + prefix))}
            assert len(see) <= tiles, (L, lo)


def test_python_refusals():
    """Tensors of the wrong place, type or shape raise before any call."""
    B, Hk, T = 2, 4, 64
    acc = torch.zeros((B, Hk, T))
    with pytest.raises(ValueError):                       # not on a GPU
        tq.evict_select(acc, torch.zeros(B, dtype=torch.int32), T, 8, torch.zeros((B, Hk, 8), dtype=torch.int32),
                        torch.zeros(B, dtype=torch.int32))
    with pytest.raises(ValueError):
        tq.evict_compact(2, torch.zeros((B, Hk, 8), dtype=torch.int32), torch.zeros(B, dtype=torch.int32),
                         torch.zeros((4, 16, Hk, 118), dtype=torch.uint8), torch.zeros((B, 4), dtype=torch.int32), Hk, 16)
    q = torch.zeros((B, 8, 128), dtype=torch.float16)
    args = (2, q, torch.zeros((4, 16, Hk, 118), dtype=torch.uint8), torch.zeros((B, 4), dtype=torch.int32),
            torch.zeros(B, dtype=torch.int32), T, Hk, 16, None, None, torch.zeros_like(q), None,
            torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        tq.decode_attention_scored(*args, softcap=3.0)
    with pytest.raises(ValueError):
        tq.decode_attention_weights(*args, acc)


def test_workspace_sizes():
    assert tq.tq_decode_weights_workspace_bytes(0, 32, 8, 1, 128, 64) == 0
    assert tq.tq_decode_weights_workspace_bytes(1, 31, 8, 1, 128, 64) == 0
    assert tq.tq_decode_weights_workspace_bytes(1, 32, 8, 1, 64, 64) == 0
    a = tq.scored_workspace_bytes(2, 4, 32, 8, 4096, weights=True)
    b = tq.scored_workspace_bytes(2, 4, 32, 8, 4096)
    assert a - b >= 4 * 32 * 4096 * 4
    # a window needs no more than a short sequence
    assert tq.scored_workspace_bytes(2, 4, 32, 8, 1 << 20, window=256, weights=True) < \
        tq.scored_workspace_bytes(2, 4, 32, 8, 4096, weights=True)
    assert np.all([tq.scored_workspace_bytes(p, 1, 4, 4, 0) >= 16 for p in range(5)])
