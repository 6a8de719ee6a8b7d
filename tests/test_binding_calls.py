"""What the C++ part of the binding accepts and refuses, on the host."""
import array

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

A = 1 << 20     # any aligned address: nothing here reaches the device
DESC = kvp.AttnDesc(1, 8, 2, 64, 16, 16, 0.0, 0)


def pool(n=4):
    p = kvp.kv_pool_create(kvp.PoolDesc(1, 64, 16, 2, 64, 8, 8, 3), A, A)
    for i in range(n):
        kvp.seq_reserve(p, kvp.seq_alloc(p), 20 + i)
    return p


@pytest.mark.parametrize("make", [
    list, tuple, lambda x: np.array(x), lambda x: np.array(x, np.int32), lambda x: np.array(x, np.uint8),
    lambda x: np.repeat(np.array(x, np.int32), 2)[::2], lambda x: [np.int64(i) for i in x],
    lambda x: array.array("i", x), lambda x: array.array("q", x), lambda x: torch.tensor(x)])
def test_host_integers(make):
    p = pool()
    kvp.seq_reorder(p, make([0, 1, 2]), make([3, 3, 0]))
    assert [kvp.seq_len(p, i) for i in range(4)] == [23, 23, 20, 23]
    kvp.seq_reorder(p, [], [])
    kvp.kv_pool_destroy(p)


@pytest.mark.parametrize("dst,src,error", [
    ([0], [1, 2], ValueError), ([1 << 40], [0], ValueError), (np.array([1 << 40]), [0], ValueError),
    ([0.5], [0], TypeError), (3, [0], TypeError), (None, [0], TypeError), (np.zeros((1, 1), np.int32), [0], ValueError),
    ([0], ["1"], TypeError)])
def test_host_integers_refused(dst, src, error):
    p = pool()
    with pytest.raises(error):
        kvp.seq_reorder(p, dst, src)
    assert [kvp.seq_len(p, i) for i in range(4)] == [20, 21, 22, 23]
    kvp.kv_pool_destroy(p)


def test_library_refusals_are_errors_with_their_code():
    p = pool()
    with pytest.raises(kvp.KvpError) as e:
        kvp.seq_reorder(p, [0, 0], [1, 2])
    assert e.value.code == kvp.KVP_ERR_INVALID and "seq_reorder" in str(e.value)
    with pytest.raises(kvp.KvpError):
        kvp.seq_reorder(None, [0], [1])
    kvp.kv_pool_destroy(p)


def sparse(**kw):
    a = dict(q=torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16), q_start=None, k_pool=A, v_pool=A,
             block_tables=torch.zeros(2, 4, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32),
             selected=torch.zeros(1, 2, 2, 3, dtype=torch.int32), desc=DESC, out=A, lse=None, stream=0)
    a.update(kw)
    kvp.paged_sparse_attention(**a)


@pytest.mark.parametrize("bad,what", [
    (dict(), "block_tables: on cpu"), (dict(block_tables=torch.zeros(2, 4)), "block_tables: expected torch.int32, got torch.float32"),
    (dict(block_tables=torch.zeros(3, 4, dtype=torch.int32)), r"block_tables: expected shape \(2, 4\), got \(3, 4\)"),
    (dict(seq_lens=torch.zeros((), dtype=torch.int32)), "seq_lens: too few dimensions"),
    (dict(seq_lens=[1, 2]), "seq_lens: expected a tensor, got list"),
    (dict(desc=kvp.rope_desc(64)), "desc: not the structure")])
def test_tensors_refused(bad, what):
    with pytest.raises(ValueError, match=what):
        sparse(**bad)


def test_other_refusals():
    with pytest.raises(TypeError):
        sparse(desc=None)
    with pytest.raises(AttributeError):
        sparse(stream="0")
    x = torch.zeros(1, 2, 5)
    with pytest.raises(ValueError, match="logits: expected float32, bfloat16 or float16 on cuda"):
        kvp.kvp_beam_select(x, A, None, 0, x, A, A, A, 100, 0)
    with pytest.raises(ValueError, match="dim: no such dimension"):
        kvp.kvp_state_reorder(x, x, torch.zeros(2, dtype=torch.int32), 3, 0)
    with pytest.raises(ValueError, match="index: expected 2 entries, got 3"):
        kvp.kvp_state_reorder(x, x, torch.zeros(3, dtype=torch.int32), 1, 0)
    p = pool()
    with pytest.raises(ValueError, match="rope: not the structure"):
        kvp.seq_append_rope(p, [0], [0], None, None, DESC, stream=0)
    with pytest.raises(ValueError, match="ntoks: expected 1 entries, got 2"):
        kvp.seq_append_rope(p, [0], [0, 1], None, None, kvp.rope_desc(64), stream=0)
    kvp.seq_append_rope(p, [0], [0], None, None, kvp.rope_desc(64), stream=0)     # nothing to append: no tensors
    kvp.kv_pool_destroy(p)
