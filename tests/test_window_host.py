"""Refusals of the window attention call and its plan, on the host."""
import ctypes

import numpy as np
import pytest

import paged_prefix_shared_decode_gb300 as kvp

A = 1 << 20


def call(desc=None, q=A, q_lens=None, k=A, v=A, tables=((0, 1),), lens=(20,), win=8, sinks=0, out=A, lse=A, ws=A,
         ws_bytes=1 << 16):
    desc = desc or kvp.AttnDesc(1, 4, 2, 64, 16, 8, 0.0, 1)
    t = np.ascontiguousarray(tables, np.int32)
    ln = np.ascontiguousarray(lens, np.int32)
    ql = None if q_lens is None else np.ascontiguousarray(q_lens, np.int32)
    return kvp.load().paged_window_attention(q, None if ql is None else ql.ctypes.data, k, v, t.ctypes.data,
                                             ln.ctypes.data, t.shape[0], t.shape[1], win, sinks, ctypes.byref(desc),
                                             out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(ws=None), dict(ws=A + 128), dict(ws_bytes=256),
    dict(q=A + 8), dict(k=A + 8), dict(v=A + 8), dict(out=A + 8), dict(lse=A + 2), dict(win=0), dict(win=-1),
    dict(sinks=-1), dict(lens=(33,)), dict(lens=(-1,)), dict(lens=(0,)), dict(q_lens=(21,)), dict(q_lens=(-1,)),
    dict(tables=((0, 8),)), dict(tables=((0, -1),)),
    dict(desc=kvp.AttnDesc(1, 4, 2, 96, 16, 8, 0.0, 1)), dict(desc=kvp.AttnDesc(1, 4, 2, 64, 16, 8, 0.0, 1, 1)),
])
def test_refusals(bad):
    assert call(**bad) == kvp.KVP_ERR_INVALID


def test_nothing_asked_is_ok():
    assert call(lens=(20,), q_lens=(0,), q=None) == kvp.KVP_OK


def test_workspace_does_not_grow_with_the_cache():
    # a window bounds the plan: the same workspace for 1000 and 100000 cached tokens
    desc = kvp.AttnDesc(1, 32, 8, 128, 16, 8000, 0.0, 1)
    t = np.arange(8000, dtype=np.int32)[None]
    size = lambda n, q: kvp.kvp_window_workspace_size(desc, t, [n], [q], 512, 4)
    assert size(1000, 1) == size(100000, 1)
    assert size(2000, 300) == size(100000, 300)
    for bad in (dict(window=0, sinks=0), dict(window=4, sinks=-1)):
        with pytest.raises(kvp.KvpError):
            kvp.kvp_window_workspace_size(desc, t, [1000], [1], **bad)


def test_longest_window_and_sinks():
    # (the plan is made on the host: no sum of a position and a window overflows)
    desc = kvp.AttnDesc(1, 32, 8, 128, 16, 200, 0.0, 1)
    t = np.arange(200, dtype=np.int32)[None]
    top = 2 ** 31 - 1
    for n, q in ((1000, 1), (1000, 300), (3200, 3200), (1, 1), (0, 0)):
        size = lambda w, s: kvp.kvp_window_workspace_size(desc, t, [n], [q], w, s)
        assert size(top, 0) == size(5000, 0) and size(top, top) == size(5000, 5000) == size(5000, 0), (n, q)
        assert size(1, top) == size(1, 5000)
    assert call(lens=(top,), tables=np.zeros((1, 2 ** 27), np.int32)) == kvp.KVP_ERR_INVALID


@pytest.mark.parametrize("G", [32, 64])
def test_more_partial_rows_than_32_bits_hold_are_refused(G):
    # a causal prompt: a query row has one partial row per 8192 keys that it sees
    desc = kvp.AttnDesc(1, G, 1, 128, 16, 1 << 16, 0.0, 1)
    t = np.arange(1 << 16, dtype=np.int32)[None]
    size = lambda n: kvp.kvp_window_workspace_size(desc, t, [n], [n], n, 0)
    n = 1 << 17
    rows = G * sum((p // 256 * 256 + 256 + 8191) // 8192 if p >= 8192 else 0 for p in range(0, n, 256)) * 256
    assert size(n) >= rows * 129 * 4
    with pytest.raises(kvp.KvpError):
        size(1 << 20)
    assert call(desc=desc, tables=t, lens=(1 << 20,), q_lens=(1 << 20,), win=1 << 20) == kvp.KVP_ERR_INVALID
