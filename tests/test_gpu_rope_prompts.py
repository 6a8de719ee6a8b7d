"""Rotated appends of prompts: several tokens to a CTA, heads in 16-byte pieces."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp
from test_gpu_rope import Cache, close, rotated

pytestmark = pytest.mark.gpu


# tokens times layers: above 16 and above 32 to an SM, in numbers that no CTA's
# share divides; heads with an odd count of pieces, pairs for a part of the dims
@pytest.mark.parametrize("L,bs,Hkv,Hq,d,rot,adjacent,pre,new", [
    (3, 16, 2, 6, 64, 64, False, [5, 0, 33], [700, 1, 211]),         # 2 tokens a CTA
    (3, 16, 4, 8, 128, 128, False, [0, 7], [1501, 302]),             # 4
    (2, 32, 1, 3, 128, 64, True, [40], [4003]),
    (5, 16, 3, 5, 72, 16, False, [1, 2, 3], [1001, 1, 998]),
    (1, 16, 1, 7, 256, 256, True, [9], [5001]),
    (4, 64, 2, 0, 64, 32, False, [70], [2999]),                      # no queries
    (2, 16, 8, 64, 128, 96, False, [3], [2600])])
def test_prompts(L, bs, Hkv, Hq, d, rot, adjacent, pre, new):
    T = sum(new)
    nb = sum((p + n) // bs + 3 for p, n in zip(pre, new))
    c = Cache(L, nb, bs, Hkv, d, 16, nb, 11)
    parents = [kvp.seq_alloc(c.pool) for _ in pre]
    for s, n in zip(parents, pre):
        kvp.seq_reserve(c.pool, s, n)
    kids = [kvp.seq_fork(c.pool, s) for s in parents]
    before = [(c.rows(c.k, s).clone(), c.rows(c.v, s).clone()) for s in parents]
    k, v = c.normal(L, T, Hkv, d), c.normal(L, T, Hkv, d)
    q = c.normal(L, T, Hq, d) if Hq else None
    q_out = torch.full_like(q, 7.0) if Hq else None
    base, scale = 10000.0, 0.75
    freqs = base ** (-np.arange(rot // 2) * 2.0 / rot)
    pos = np.concatenate([np.arange(p, p + n) for p, n in zip(pre, new)])
    kvp.seq_append_rope(c.pool, kids, new, k, v, kvp.rope_desc(rot, base, None, adjacent, scale), None, q, q_out)
    want, mag = rotated(k, pos, rot, adjacent, freqs, scale)
    at = 0
    for i, s in enumerate(kids):
        got_k, got_v = c.rows(c.k, s), c.rows(c.v, s)
        assert torch.equal(got_k[:, :pre[i]], before[i][0]) and torch.equal(got_v[:, :pre[i]], before[i][1])
        assert torch.equal(got_v[:, pre[i]:], v[:, at:at + new[i]])
        close(got_k[:, pre[i]:], want[:, at:at + new[i]], mag[:, at:at + new[i]])
        assert torch.equal(c.rows(c.k, parents[i]), before[i][0])
        at += new[i]
    if Hq:
        close(q_out, *rotated(q, pos, rot, adjacent, freqs, scale))
        assert torch.equal(q_out[..., rot:], q[..., rot:])
        kvp.seq_reorder(c.pool, kids, parents)           # once more, in place and with the positions given
        kvp.seq_append_rope(c.pool, kids, new, k, v, kvp.rope_desc(rot, base, None, adjacent, scale),
                            torch.from_numpy(pos.astype(np.int32)).cuda(), q, q)
        assert torch.equal(q, q_out)
    kvp.kv_pool_destroy(c.pool)
