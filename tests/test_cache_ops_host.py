"""Refusals of the accumulated-weight and eviction calls, on the host."""
import numpy as np
import pytest

import paged_prefix_shared_decode_gb300 as kvp

A = 1 << 20     # any 256-byte aligned address: nothing here reaches the device


def mass(desc=None, q=A, q_lens=None, lse=A, k=A, tables=((0, 1),), lens=(20,), decay=1.0, mass_in=None, prev=None,
         out=A, stride=32, ws=A, ws_bytes=1 << 16):
    import ctypes
    desc = desc or kvp.AttnDesc(1, 4, 2, 64, 16, 8, 0.0, 1)
    t = np.ascontiguousarray(tables, np.int32)
    arr = [None if x is None else np.ascontiguousarray(x, np.int32) for x in (lens, q_lens, prev)]
    p = [None if x is None else x.ctypes.data for x in arr]
    return kvp.load().kvp_attention_mass(q, p[1], lse, k, t.ctypes.data, p[0], t.shape[0], t.shape[1],
                                         ctypes.byref(desc), decay, mass_in, p[2], out, stride, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(lse=None), dict(k=None), dict(out=None), dict(ws=None), dict(ws=A + 128), dict(ws_bytes=256),
    dict(q=A + 8), dict(k=A + 8), dict(lse=A + 2), dict(out=A + 1), dict(mass_in=A + 2),
    dict(mass_in=A + 4),        # overlaps the output without being it
    dict(lens=(33,)), dict(lens=(-1,)), dict(lens=(0,)), dict(q_lens=(21,)), dict(q_lens=(-1,)),
    dict(prev=(21,)), dict(prev=(-1,)), dict(stride=19), dict(tables=((0, 8),)), dict(tables=((0, -1),)),
    dict(decay=float("inf")), dict(decay=float("nan")),
    dict(desc=kvp.AttnDesc(1, 4, 2, 96, 16, 8, 0.0, 1)), dict(desc=kvp.AttnDesc(1, 4, 3, 64, 16, 8, 0.0, 1)),
    dict(desc=kvp.AttnDesc(1, 4, 2, 64, 8, 8, 0.0, 1)), dict(desc=kvp.AttnDesc(1, 4, 2, 64, 16, 8, 0.0, 1, 1)),
    dict(desc=kvp.AttnDesc(40000, 4, 2, 64, 16, 8, 0.0, 1)),
])
def test_mass_refusals(bad):
    assert mass(**bad) == kvp.KVP_ERR_INVALID


def test_mass_empty_batch_is_ok():
    # nothing cached, nothing asked: no device work
    assert mass(lens=(0,), q_lens=(0,), q=None, lse=None) == kvp.KVP_OK


def test_mass_workspace():
    d = kvp.AttnDesc(1, 4, 2, 64, 16, 8, 0.0, 1)
    t = np.array([[0, 1], [2, -1]], np.int32)
    n = kvp.kvp_mass_workspace_size(d, t, [20, 3])
    assert n % 256 == 0 and n >= 256 + 2 * 24 + 3 * 4
    with pytest.raises(kvp.KvpError):
        kvp.kvp_mass_workspace_size(d, t, [20, 17])         # its second block is not there
    with pytest.raises(ValueError):
        kvp.kvp_mass_workspace_size(d, t, [20])


def test_evict_refusals_change_nothing():
    lib = kvp.load()
    p = kvp.kv_pool_create(kvp.PoolDesc(1, 16, 16, 2, 64, 4, 8, 0), A, A)
    s = kvp.seq_alloc(p)
    kvp.seq_reserve(p, s, 100)
    seqs = np.array([s], np.int32)
    twice = np.array([s, s], np.int32)
    dead = np.array([3], np.int32)
    ok = dict(pool=p, seqs=seqs.ctypes.data, n=1, mass=A, stride=128, budget=40, sink=4, recent=8, kept=A + (1 << 16),
              out=None, ws=A, ws_bytes=1 << 16, stream=None)
    for bad in (dict(pool=None), dict(seqs=None), dict(n=0), dict(seqs=twice.ctypes.data, n=2),
                dict(seqs=dead.ctypes.data), dict(mass=None), dict(mass=A + 2), dict(kept=None), dict(kept=A + 2),
                dict(stride=99), dict(budget=0), dict(budget=-1), dict(sink=-1), dict(recent=-1),
                dict(sink=33), dict(ws=None), dict(ws=A + 64), dict(ws_bytes=300),
                dict(out=A + 4)):       # overlaps mass without being it
        assert lib.seq_evict(*{**ok, **bad}.values()) == kvp.KVP_ERR_INVALID, bad
    assert kvp.seq_len(p, s) == 100 and kvp.kvp_free_block_count(p) == 9
    kvp.kv_pool_destroy(p)
    # no storage, or 4-bit pages
    p = kvp.kv_pool_create(kvp.PoolDesc(1, 16, 16, 2, 64, 4, 8, 0))
    s = kvp.seq_alloc(p)
    kvp.seq_reserve(p, s, 100)
    assert lib.seq_evict(*{**ok, "pool": p}.values()) == kvp.KVP_ERR_STATE
    kvp.kv_pool_destroy(p)
    p = kvp.kv_pool_create_kv4(kvp.PoolDesc(1, 16, 16, 2, 64, 4, 8, 0), A, A, A, A)
    s = kvp.seq_alloc(p)
    kvp.seq_reserve(p, s, 100)
    assert lib.seq_evict(*{**ok, "pool": p}.values()) == kvp.KVP_ERR_STATE
    assert kvp.seq_len(p, s) == 100
    kvp.kv_pool_destroy(p)


def test_evict_workspace():
    p = kvp.kv_pool_create(kvp.PoolDesc(1, 16, 16, 2, 64, 4, 8, 0))
    s = kvp.seq_alloc(p)
    kvp.seq_reserve(p, s, 100)
    n = kvp.seq_evict_workspace_size(p, [s], 40)
    assert n % 256 == 0 and n >= 256 + 16 + (7 + 3) * 4
    for seqs, budget in (([s], 0), ([2], 4), ([], 4)):
        with pytest.raises(kvp.KvpError):
            kvp.seq_evict_workspace_size(p, seqs, budget)
    kvp.kv_pool_destroy(p)


class Tensor:
    """What the binding asks of a tensor on the current device, at an address that nothing here may reach."""

    def __init__(self, dtype, *shape, device=0):
        import torch
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), device
        self.is_cuda = True

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 4

    def data_ptr(self):
        return A


@pytest.mark.parametrize("wrong", ["mass", "kept", "mass_out"])
@pytest.mark.parametrize("shape", [(1, 1, 3, 128), (2, 1, 1, 128), (2, 1, 2, 128), (3, 1, 3, 128), (2, 1, 4, 128),
                                   (2, 2, 3, 128), (2, 3, 128)])
def test_evict_weights_are_of_the_pool_s_layers_and_heads(wrong, shape):
    import torch
    p = kvp.kv_pool_create(kvp.PoolDesc(2, 16, 16, 3, 64, 4, 8, 0), A, A)
    s = kvp.seq_alloc(p)
    kvp.seq_reserve(p, s, 100)
    good = dict(mass=(2, 1, 3, 128), kept=(2, 1, 3, 40), mass_out=(2, 1, 3, 128))
    # one tensor too small or too large, and all of them of the same wrong layers and heads
    for names in ([wrong], list(good)):
        sh = {**good, **{n: shape[:-1] + good[n][-1:] for n in names}}
        with pytest.raises(ValueError, match="expected"):
            kvp.seq_evict(p, [s], Tensor(torch.float32, *sh["mass"]), 40, 4, 8, Tensor(torch.int32, *sh["kept"]),
                          Tensor(torch.float32, *sh["mass_out"]), A, 1 << 16, stream=0)
    assert kvp.seq_len(p, s) == 100 and kvp.kvp_free_block_count(p) == 9
    kvp.kv_pool_destroy(p)


def test_pool_shape():
    p = kvp.kv_pool_create(kvp.PoolDesc(2, 16, 16, 3, 64, 4, 8, 0))
    assert kvp.kvp_pool_shape(p) == (2, 3)
    kvp.kv_pool_destroy(p)
    for bad in ((None, A, A), (A, None, A), (A, A, None)):
        assert kvp.load().kvp_pool_shape(*bad) == kvp.KVP_ERR_INVALID
