"""Tensors whose sizes do not fit the pool or the call are refused by the
binding, on the host."""
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

A = 1 << 20     # any aligned address: nothing here reaches the device


def test_rotated_append_takes_the_pools_head_dim():
    # k, v and q that agree with one another, but are narrower than the pool's rows
    p = kvp.kv_pool_create(kvp.PoolDesc(2, 16, 16, 2, 64, 4, 4, 3), A, A)
    s = kvp.seq_alloc(p)
    t = lambda h, d: torch.zeros(2, 3, h, d, dtype=torch.bfloat16)
    for d in (32, 128):
        with pytest.raises(ValueError, match=r"k: expected shape \(2, 3, 2, 64\), got \(2, 3, 2, %d\)" % d):
            kvp.seq_append_rope(p, [s], [3], t(2, d), t(2, d), kvp.rope_desc(32), None, t(4, d), t(4, d), stream=0)
    with pytest.raises(ValueError, match="k: on cpu"):          # (the right shape goes on to the next check)
        kvp.seq_append_rope(p, [s], [3], t(2, 64), t(2, 64), kvp.rope_desc(32), stream=0)
    with pytest.raises(ValueError, match=r"q: expected shape \(2, 3, 4, 64\), got \(2, 3, 4, 32\)"):
        kvp.seq_append_rope(p, [s], [3], A, A, kvp.rope_desc(32), None, t(4, 32), t(4, 32), stream=0)
    assert kvp.seq_len(p, s) == 0 and kvp.kvp_pool_head_dim(p) == 64
    with pytest.raises(kvp.KvpError):
        kvp.kvp_pool_head_dim(None)
    kvp.kv_pool_destroy(p)
