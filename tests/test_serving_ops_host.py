"""Refusals and bookkeeping of rotated appends, sequence reordering, page
selection, sparse attention and beam selection, on the host."""
import ctypes

import numpy as np
import pytest

import paged_prefix_shared_decode_gb300 as kvp

A = 1 << 20     # any 256-byte aligned address: nothing here reaches the device
B = 1 << 24
OK, INVALID, STATE, OOM = kvp.KVP_OK, kvp.KVP_ERR_INVALID, kvp.KVP_ERR_STATE, kvp.KVP_ERR_OOM


def pool(storage=True, nb=16, bs=16, seqs=6, mb=8):
    d = kvp.PoolDesc(2, nb, bs, 2, 64, seqs, mb, 3)
    return kvp.kv_pool_create(d, A, A) if storage else kvp.kv_pool_create(d)


def append(p, seqs=(0,), ntoks=(5,), k=A, v=A, rope=None, positions=None, q=None, q_out=None, hq=4):
    s, n = (np.ascontiguousarray(x, np.int32) for x in (seqs, ntoks))
    rope = kvp.rope_desc(64) if rope is None else rope
    return kvp.load().seq_append_rope(p, len(s), s.ctypes.data, n.ctypes.data, k, v,
                                      ctypes.byref(rope) if rope else None, positions, q, q_out, hq, None)


def rope(rot=64, base=10000.0, scale=1.0, freqs=None):
    return kvp.rope_desc(rot, base=base, scale=scale, freqs=freqs)


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 2), dict(rope=False), dict(rope=rope(0)), dict(rope=rope(66)),
    dict(rope=rope(63)), dict(rope=rope(-2)), dict(rope=rope(base=0.0)), dict(rope=rope(base=-1.0)),
    dict(rope=rope(base=float("nan"))), dict(rope=rope(scale=float("inf"))),
    dict(rope=rope(4, freqs=[1.0, float("nan")])), dict(positions=A + 2),
    dict(q=A), dict(q_out=A), dict(q=A, q_out=B + 8), dict(q=A + 8, q_out=B), dict(q=A, q_out=B, hq=0),
    dict(q=A, q_out=B, hq=1 << 20),
    dict(q=A, q_out=A + 16),            # overlaps without being it
    dict(seqs=(3,)), dict(seqs=(0, 0), ntoks=(1, 1)), dict(ntoks=(-1,)), dict(ntoks=(8 * 16,)),
])
def test_append_rope_refusals_change_nothing(bad):
    p = pool()
    for _ in range(2):
        kvp.seq_reserve(p, kvp.seq_alloc(p), 20)
    assert append(p, **bad) == INVALID
    assert [kvp.seq_len(p, s) for s in (0, 1)] == [20, 20] and kvp.kvp_free_block_count(p) == 12
    kvp.kv_pool_destroy(p)


def test_append_rope_states():
    p = pool(storage=False)
    kvp.seq_alloc(p)
    assert append(p) == STATE
    kvp.kv_pool_destroy(p)
    assert append(None) == INVALID
    p = pool(nb=4)
    kvp.seq_alloc(p)
    assert append(p, ntoks=(65,)) == OOM
    assert append(p, ntoks=(0,), k=None, v=None) == OK      # nothing to append: nothing runs
    assert append(p, seqs=(), ntoks=()) == OK
    assert kvp.seq_len(p, 0) == 0 and kvp.kvp_free_block_count(p) == 4
    kvp.kv_pool_destroy(p)


def test_rope_desc_checks_freqs():
    with pytest.raises(ValueError):
        kvp.rope_desc(8, freqs=[1.0, 2.0])


def state(p, n):
    live = []
    for s in range(n):
        try:
            live.append((kvp.seq_len(p, s), kvp.seq_block_table(p, s).tolist()))
        except kvp.KvpError:
            live.append(None)
    return live, [kvp.block_refcount(p, b) for b in range(64)], kvp.kvp_free_block_count(p)


@pytest.mark.parametrize("seed", range(6))
def test_reorder_against_tables(seed):
    g = np.random.default_rng(seed)
    bs = int(g.choice([1, 4, 16]))
    p = pool(storage=False, nb=64, bs=bs, seqs=8, mb=16)
    root = kvp.seq_alloc(p)
    kvp.seq_reserve(p, root, int(g.integers(0, 3 * bs + 1)))
    seqs = [root] + [kvp.seq_fork(p, root) for _ in range(5)]
    for step in range(20):
        for s in seqs:
            if kvp.kvp_free_block_count(p) > 3 and kvp.seq_len(p, s) < 10 * bs:
                kvp.seq_reserve(p, s, int(g.integers(0, bs + 2)))
        dst = g.permutation(seqs)[:int(g.integers(0, 7))]
        src = g.choice(seqs, len(dst))
        before, _, _ = state(p, 8)
        kvp.seq_reorder(p, dst, src)
        after, ref, free = state(p, 8)
        want = list(before)
        for a, b in zip(dst, src):
            want[a] = before[b]
        assert after == want
        held = np.zeros(64, int)
        for x in after:
            if x:
                np.add.at(held, x[1], 1)
        assert ref == held.tolist() and free == int((held == 0).sum())
    kvp.kv_pool_destroy(p)


def test_reorder_then_append_repeats_its_blocks():
    # beams set back to their parents take the same blocks in every pass
    p = pool(storage=False, nb=40, bs=4, seqs=8, mb=8)
    parents = [kvp.seq_alloc(p) for _ in range(3)]
    for i, s in enumerate(parents):
        kvp.seq_reserve(p, s, 3 + 4 * i)
    kids = [kvp.seq_fork(p, s) for s in parents]
    seen = []
    for _ in range(3):
        kvp.seq_reorder(p, kids, parents)
        for s in kids:
            kvp.seq_reserve(p, s, 6)
        seen.append([kvp.seq_block_table(p, s).tolist() for s in kids])
    assert seen[0] == seen[1] == seen[2]
    kvp.kv_pool_destroy(p)


def test_reorder_refusals_change_nothing():
    p = pool(storage=False, nb=64)
    for _ in range(3):
        kvp.seq_reserve(p, kvp.seq_alloc(p), 20)
    before = state(p, 6)
    for dst, src in (((0, 0), (1, 2)), ((0, 4), (1, 1)), ((0, 1), (1, 5)), ((-1,), (0,)), ((0,), (6,))):
        with pytest.raises(kvp.KvpError) as e:
            kvp.seq_reorder(p, dst, src)
        assert e.value.code == INVALID
    assert kvp.load().seq_reorder(p, None, None, 1) == INVALID
    assert kvp.load().seq_reorder(None, None, None, 0) == INVALID
    assert kvp.load().seq_reorder(p, None, None, 0) == OK
    with pytest.raises(ValueError):
        kvp.seq_reorder(p, [0, 1], [0])
    assert state(p, 6) == before
    kvp.kv_pool_destroy(p)


def desc(L=1, hq=4, hkv=2, d=64, bs=16, nb=8, fmt=0):
    return kvp.AttnDesc(L, hq, hkv, d, bs, nb, 0.0, 0, fmt)


BAD_DESC = [desc(d=96), desc(hkv=3), desc(bs=8), desc(bs=24), desc(fmt=1), desc(L=40000), desc(nb=0), desc(L=0)]
BAD_BATCH = [dict(tables=None), dict(lens=None), dict(lens=A + 2), dict(S=0), dict(S=-1), dict(MB=0),
             dict(MB=1 << 27)] + [dict(desc=d) for d in BAD_DESC]


def bounds(k=A, tables=A, lens=A, S=2, MB=3, n_new=5, desc=desc(), out=B):
    return kvp.load().kvp_page_bounds(k, tables, lens, S, MB, n_new, ctypes.byref(desc), out, None)


@pytest.mark.parametrize("bad", BAD_BATCH + [dict(k=None), dict(k=A + 8), dict(out=None), dict(out=B + 4), dict(n_new=-1),
                                             dict(S=70000)])
def test_bounds_refusals(bad):
    assert bounds(**bad) == INVALID


def test_bounds_of_nothing():
    assert bounds(n_new=0) == OK


def scores(q=A, q_start=None, T=2, bnd=A, tables=A, lens=A, S=2, MB=3, desc=desc(), out=B, stride=3):
    return kvp.load().kvp_page_scores(q, q_start, T, bnd, tables, lens, S, MB, ctypes.byref(desc), out, stride, None)


@pytest.mark.parametrize("bad", BAD_BATCH + [
    dict(q=None), dict(q=A + 8), dict(bnd=None), dict(bnd=A + 8), dict(out=None), dict(out=B + 2), dict(stride=2),
    dict(T=-1), dict(T=3), dict(q_start=A + 2)])
def test_scores_refusals(bad):
    assert scores(**bad) == INVALID


def test_rows_of_nothing():
    assert scores(q=None, q_start=A, T=0, out=None) == OK
    assert select(q_start=A, T=0, sc=None, out=None) == OK
    assert sparse(q=None, q_start=A, T=0, out=None) == OK


def select(sc=A, stride=3, q_start=None, T=2, lens=A, S=2, MB=3, desc=desc(), budget=3, sink=1, recent=1, out=B):
    return kvp.load().kvp_page_select(sc, stride, q_start, T, lens, S, MB, ctypes.byref(desc), budget, sink, recent, out,
                                      None)


@pytest.mark.parametrize("bad", [x for x in BAD_BATCH if "tables" not in x] + [
    dict(sc=None), dict(sc=A + 2), dict(out=None), dict(out=B + 1), dict(stride=2), dict(T=-1), dict(T=1),
    dict(q_start=A + 1), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=2, recent=2),
    dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(T=2 ** 31 - 1, q_start=A)])
def test_select_refusals(bad):
    assert select(**bad) == INVALID


def sparse(q=A, q_start=None, T=2, k=A, v=A, tables=A, lens=A, S=2, MB=3, sel=A, budget=3, desc=desc(), out=B, lse=B):
    return kvp.load().paged_sparse_attention(q, q_start, T, k, v, tables, lens, S, MB, sel, budget, ctypes.byref(desc),
                                             out, lse, None)


@pytest.mark.parametrize("bad", [x for x in BAD_BATCH if x.get("desc") is not BAD_DESC[5]] + [
    dict(q=None), dict(q=A + 8), dict(k=None), dict(k=A + 2), dict(v=None), dict(v=A + 8), dict(sel=None), dict(sel=A + 2),
    dict(out=None), dict(out=B + 8), dict(lse=B + 2), dict(budget=0), dict(T=-1), dict(T=1), dict(q_start=A + 2),
    dict(T=2 ** 31 - 1, q_start=A)])
def test_sparse_refusals(bad):
    assert sparse(**bad) == INVALID


def beam(x=A, typ=0, stride=100, sc=A, done=None, pad=0, G=2, K=4, V=100, n=4, os=B, orow=B, ot=B, ws=A, ws_bytes=1 << 20):
    return kvp.load().kvp_beam_select(x, typ, stride, sc, done, pad, G, K, V, n, os, orow, ot, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=A + 2), dict(x=A + 1, typ=1), dict(typ=3), dict(typ=-1), dict(stride=-1), dict(sc=None),
    dict(sc=A + 2), dict(os=None), dict(os=B + 2), dict(orow=None), dict(orow=B + 1), dict(ot=None), dict(ot=B + 2),
    dict(ws=None), dict(ws=A + 8), dict(ws_bytes=100), dict(G=0), dict(K=0), dict(K=129), dict(V=0), dict(n=0),
    dict(n=129), dict(G=2 ** 31 - 1, K=128)])
def test_beam_refusals(bad):
    assert beam(**bad) == INVALID


def test_beam_workspace():
    assert kvp.kvp_beam_workspace_size(2, 4, 100, 4) <= kvp.kvp_beam_workspace_size(2, 4, 100000, 4)
    with pytest.raises(kvp.KvpError):
        kvp.kvp_beam_workspace_size(2, 4, 100, 0)


def test_reorder_state_refusals():
    f = kvp.load().kvp_state_reorder
    for bad in ((None, B, A, 1, 4, 4, 64), (A, None, A, 1, 4, 4, 64), (A, B, None, 1, 4, 4, 64), (A, B, A + 2, 1, 4, 4, 64),
                (A, B, A, -1, 4, 4, 64), (A, B, A, 1, -4, 4, 64), (A, B, A, 1, 4, -4, 64), (A, B, A, 1, 4, 4, -64),
                (A, A + 64, A, 1, 4, 4, 64), (A + 64, A, A, 1, 4, 4, 64), (A, B, A, 2 ** 62, 4, 4, 64),
                (A, B, A, 2 ** 20, 1, 2 ** 20, 16)):
        assert f(*bad, None) == INVALID, bad
    for none in ((A, B, A, 0, 4, 4, 64), (A, B, A, 1, 0, 4, 64), (A, B, A, 1, 4, 0, 64), (A, B, A, 1, 4, 4, 0)):
        assert f(*none, None) == OK
