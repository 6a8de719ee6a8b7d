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


def beam(x, workspace, ws_bytes=None):
    kvp.kvp_beam_select(x, A, None, 0, torch.zeros(1, 4, device=x.device), A, A, workspace, ws_bytes, 0)


def test_beam_workspace_is_what_it_is_said_to_be():
    x, room = torch.zeros(1, 2, 100), torch.zeros(64, dtype=torch.uint8)
    for ws, n, what in ((room, 65, "ws_bytes: 65, but the workspace has 64"), (room, -1, "ws_bytes: out of range"),
                        (A, -1, "ws_bytes: out of range"), (A, None, "ws_bytes: needed"), (None, None, "ws_bytes: needed"),
                        (room, 1 << 70, "ws_bytes: out of range")):
        with pytest.raises(ValueError, match=what):
            beam(x, ws, n)
    for ws, n in ((room, 64), (room, 0), (room, None), (A, 64)):        # (these go on to the next check)
        with pytest.raises(ValueError, match="logits: expected float32"):
            beam(x, ws, n)


@pytest.mark.gpu
def test_beam_workspace_is_on_the_device():
    x = torch.zeros(1, 2, 100, device="cuda")
    out = torch.zeros(1, 4, device="cuda"), *(torch.zeros(1, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    cum = torch.zeros(1, 2, device="cuda")
    n = kvp.kvp_beam_workspace_size(1, 2, 100, 4)
    with pytest.raises(ValueError, match="workspace: on cpu"):
        kvp.kvp_beam_select(x, cum, None, 0, *out, torch.zeros(n, dtype=torch.uint8))
    ws = torch.zeros(2 * n, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace: expected a contiguous"):
        kvp.kvp_beam_select(x, cum, None, 0, *out, ws[::2])
    with pytest.raises(kvp.KvpError):
        kvp.kvp_beam_select(x, cum, None, 0, *out, ws, n - 1)
    kvp.kvp_beam_select(x, cum, None, 0, *out, ws, n)
    assert out[1].tolist() == [[0, 0, 0, 0]] and out[2].tolist() == [[0, 1, 2, 3]]
