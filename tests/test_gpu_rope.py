"""Appends with the position rotation against the formula in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu


def rotated(x, pos, rot, adjacent, freqs, scale):
    """x [L][T][H][d] by the formula in 64 bits, and the sum of magnitudes that
    each result is made of."""
    x = x.double().cpu().numpy()
    y, mag = x.copy(), np.abs(x)
    a = np.asarray(pos, np.float64)[:, None] * freqs
    c, s = scale * np.cos(a)[:, None], scale * np.sin(a)[:, None]
    i = np.arange(rot // 2)
    i, j = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    mag[..., i] = mag[..., j] = scale * (np.abs(x[..., i]) + np.abs(x[..., j]))
    return y, mag


def close(got, want, mag):
    """One rounding to bf16 (2^-8 of the value) of a result whose cos and sin
    are off by at most the angle's rounding to fp32 (pi 2^-24), the angle's
    own 64-bit rounding (2^-22 at positions of 2^31) and a few 2^-24."""
    got = got.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag).all()


class Cache:
    """A pool on the device and a host copy of its K and V, kept by the formula."""

    def __init__(self, L, NB, bs, Hkv, d, seqs, mb, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.L, self.bs, self.Hkv, self.d = L, bs, Hkv, d
        self.k, self.v = self.normal(L, NB, Hkv, bs, d), self.normal(L, NB, Hkv, bs, d)
        self.pool = kvp.kv_pool_create(kvp.PoolDesc(L, NB, bs, Hkv, d, seqs, mb, seed + 1), self.k, self.v)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda", dtype=torch.bfloat16)

    def rows(self, which, s):
        """[L][len][Hkv][d] of a sequence."""
        t = torch.from_numpy(kvp.seq_block_table(self.pool, s).astype(np.int64)).cuda()
        x = which[:, t].transpose(2, 3).flatten(1, 2)
        return x[:, :kvp.seq_len(self.pool, s)]


CASES = [
    # L, bs, Hkv, Hq, d, rot, adjacent, prefix lengths, new tokens
    (1, 16, 4, 32, 64, 64, False, [0], [1]),
    (3, 16, 8, 32, 128, 128, False, [15, 16, 17, 1], [1, 1, 1, 1]),
    (2, 32, 2, 6, 64, 32, True, [5, 0, 40], [70, 1, 33]),
    (1, 16, 1, 1, 128, 48, False, [3], [200]),
    (1, 5, 3, 3, 24, 6, True, [7, 2], [11, 4]),       # rot_dim no multiple of 16, odd block size
    (2, 1, 2, 5, 40, 10, False, [3, 0], [4, 2]),
    (1, 16, 2, 4, 256, 256, True, [9], [20]),
    (1, 16, 2, 4, 64, 2, False, [9], [20]),
    (1, 16, 2, 4, 72, 16, False, [9], [3]),           # an odd number of 16-byte chunks
]


@pytest.mark.parametrize("L,bs,Hkv,Hq,d,rot,adjacent,pre,new", CASES)
@pytest.mark.parametrize("far", [None, 0, 900001, -77, 2 ** 31 - 300])
def test_append_rope(L, bs, Hkv, Hq, d, rot, adjacent, pre, new, far):
    c = Cache(L, 200, bs, Hkv, d, 16, 80, 3) if bs > 1 else Cache(L, 400, bs, Hkv, d, 16, 80, 3)
    parents = [kvp.seq_alloc(c.pool) for _ in pre]
    for s, n in zip(parents, pre):
        kvp.seq_reserve(c.pool, s, n)
    kids = [kvp.seq_fork(c.pool, s) for s in parents]       # last pages shared: copied on write
    before = [(c.rows(c.k, s).clone(), c.rows(c.v, s).clone()) for s in parents]
    T = sum(new)
    k, v, q = c.normal(L, T, Hkv, d), c.normal(L, T, Hkv, d), c.normal(L, T, Hq, d)
    q_out = torch.full_like(q, 7.0)
    own = np.concatenate([np.arange(p, p + n) for p, n in zip(pre, new)])
    pos = own if far is None else (np.arange(T) * 3 % 256 + far)
    positions = None if far is None else torch.from_numpy(pos.astype(np.int32)).cuda()
    base, scale = 10000.0, 1.25
    freqs = base ** (-np.arange(rot // 2) * 2.0 / rot)
    kvp.seq_append_rope(c.pool, kids, new, k, v, kvp.rope_desc(rot, base, None, adjacent, scale), positions, q, q_out)
    want, mag = rotated(k, pos, rot, adjacent, freqs, scale)
    at = 0
    for i, s in enumerate(kids):
        got_k, got_v = c.rows(c.k, s), c.rows(c.v, s)
        assert torch.equal(got_k[:, :pre[i]], before[i][0]) and torch.equal(got_v[:, :pre[i]], before[i][1])
        assert torch.equal(got_v[:, pre[i]:], v[:, at:at + new[i]])
        close(got_k[:, pre[i]:], want[:, at:at + new[i]], mag[:, at:at + new[i]])
        at += new[i]
        assert torch.equal(c.rows(c.k, parents[i]), before[i][0])
    close(q_out, *rotated(q, pos, rot, adjacent, freqs, scale))
    # dims behind rot_dim are what they were
    assert torch.equal(q_out[..., rot:], q[..., rot:])
    kvp.kv_pool_destroy(c.pool)


def test_other_slots_stay():
    c = Cache(2, 12, 16, 2, 64, 4, 6, 1)
    s = kvp.seq_alloc(c.pool)
    kvp.seq_reserve(c.pool, s, 21)
    k0, v0 = c.k.clone(), c.v.clone()
    k, v = c.normal(2, 3, 2, 64), c.normal(2, 3, 2, 64)
    kvp.seq_append_rope(c.pool, [s], [3], k, v, kvp.rope_desc(64))
    b = int(kvp.seq_block_table(c.pool, s)[1])
    for now, old in ((c.k, k0), (c.v, v0)):
        same = (now == old).all(-1)
        same[:, b, :, 5:8] = True
        assert bool(same.all())
    assert torch.equal(c.v[:, b, :, 5:8], v.transpose(1, 2))
    kvp.kv_pool_destroy(c.pool)


def test_given_frequencies_in_place_and_streams():
    c = Cache(1, 12, 16, 2, 64, 4, 6, 2)
    s = kvp.seq_alloc(c.pool)
    freqs = np.array([3.0, -0.5, 0.0, 1e-9, 100.25, 0.1, 0.01, 2 * math.pi])
    k, v, q = c.normal(1, 50, 2, 64), c.normal(1, 50, 2, 64), c.normal(1, 50, 4, 64)
    want_q, mag_q = rotated(q, np.arange(50), 16, False, freqs, 1.0)
    want_k, mag_k = rotated(k, np.arange(50), 16, False, freqs, 1.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kvp.seq_append_rope(c.pool, [s], [50], k, v, kvp.rope_desc(16, freqs=freqs, scale=0.0), None, q, q, stream=st)
    st.synchronize()
    close(q, want_q, mag_q)
    close(c.rows(c.k, s), want_k, mag_k)
    kvp.kv_pool_destroy(c.pool)


@pytest.mark.parametrize("n,each,bs", [(700, 1, 1), (3, 2500, 1), (90, 3, 16), (600, 2, 16), (1, 9000, 2)])
def test_more_than_one_launch_holds(n, each, bs):
    # sequences, pages and copy-on-write blocks beyond one launch's parameters
    d, L = 8, 1
    c = Cache(L, 12000, bs, 1, d, 2 * n + 1, 9100, 5)
    root = kvp.seq_alloc(c.pool)
    kvp.seq_reserve(c.pool, root, 5)
    kids = [kvp.seq_fork(c.pool, root) for _ in range(n)]
    head = c.rows(c.k, root).clone()
    T = n * each
    k, v = c.normal(L, T, 1, d), c.normal(L, T, 1, d)
    kvp.seq_append_rope(c.pool, kids, [each] * n, k, v, kvp.rope_desc(d))
    pos = np.tile(np.arange(5, 5 + each), n)
    want, mag = rotated(k, pos, d, False, 10000.0 ** (-np.arange(d // 2) * 2.0 / d), 1.0)
    for i in (0, n // 2, n - 1):
        got = c.rows(c.k, kids[i])
        assert torch.equal(got[:, :5], head)
        close(got[:, 5:], want[:, i * each:(i + 1) * each], mag[:, i * each:(i + 1) * each])
        assert torch.equal(c.rows(c.v, kids[i])[:, 5:], v[:, i * each:(i + 1) * each])
    kvp.kv_pool_destroy(c.pool)


@pytest.mark.parametrize("d,rot,adjacent", [(64, 64, False), (128, 96, True), (128, 20, False)])
def test_4bit_pages_hold_the_rotated_keys(d, rot, adjacent):
    # bit for bit what seq_append makes of the keys that a bf16 pool would hold
    L, NB, bs, Hkv, Hq = 2, 16, 16, 2, 6
    gen = torch.Generator(device="cuda").manual_seed(4)
    bytes_ = lambda *sh: torch.zeros(sh, dtype=torch.uint8, device="cuda")
    pre, new = [0, 21], [37, 1]
    T = sum(new)
    norm = lambda *sh: torch.randn(sh, generator=gen, device="cuda", dtype=torch.bfloat16)
    k, v, q = norm(L, T, Hkv, d), norm(L, T, Hkv, d), norm(L, T, Hq, d)
    old_k, old_v = norm(L, 21, Hkv, d), norm(L, 21, Hkv, d)
    r = kvp.rope_desc(rot, 500.0, None, adjacent)
    plain = Cache(L, NB, bs, Hkv, d, 4, 8, 7)
    pools = []
    for how in ("append", "rope"):
        st = [bytes_(L, NB, Hkv, bs, d // 2), bytes_(L, NB, Hkv, bs).view(torch.int8),
              bytes_(L, NB, Hkv, bs, d // 2), bytes_(L, NB, Hkv, bs).view(torch.int8)]
        p = kvp.kv_pool_create_kv4(kvp.PoolDesc(L, NB, bs, Hkv, d, 6, 8, 8), *st)
        pools.append((p, st))
    outs = []
    for p, st in pools + [(plain.pool, None)]:
        a, b = kvp.seq_alloc(p), kvp.seq_alloc(p)
        kvp.seq_append(p, b, old_k, old_v, 21)
        kid = kvp.seq_fork(p, b)
        outs.append((p, a, kid))
    q1, q2 = torch.empty_like(q), torch.empty_like(q)
    p, a, kid = outs[2]
    kvp.seq_append_rope(p, [a, kid], new, k, v, r, None, q, q1)
    turned = torch.cat([plain.rows(plain.k, a), plain.rows(plain.k, kid)[:, 21:]], 1).contiguous()
    p, a, kid = outs[0]
    kvp.seq_append_batch(p, [a, kid], new, turned, v)
    p, a, kid = outs[1]
    kvp.seq_append_rope(p, [a, kid], new, k, v, r, None, q, q2)
    for x, y in zip(pools[0][1], pools[1][1]):
        assert torch.equal(x, y)
    assert torch.equal(q1, q2)
    for p in (pools[0][0], pools[1][0], plain.pool):
        kvp.kv_pool_destroy(p)


def test_refused_while_captured():
    c = Cache(1, 12, 16, 2, 64, 4, 6, 2)
    s = kvp.seq_alloc(c.pool)
    k = c.normal(1, 3, 2, 64)
    g = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        x += 1
        with pytest.raises(kvp.KvpError) as e:
            kvp.seq_append_rope(c.pool, [s], [3], k, k, kvp.rope_desc(64))
    assert e.value.code == kvp.KVP_ERR_STATE and kvp.seq_len(c.pool, s) == 0
    kvp.kv_pool_destroy(c.pool)


def test_wrong_tensors_are_refused():
    c = Cache(1, 12, 16, 2, 64, 4, 6, 2)
    s = kvp.seq_alloc(c.pool)
    k, q = c.normal(1, 3, 2, 64), c.normal(1, 3, 4, 64)
    for bad in (dict(k=k.float()), dict(k=k[:, :2].contiguous()), dict(v=c.normal(1, 3, 2, 32)), dict(q=q.cpu()),
                dict(q_out=q[..., :32]), dict(positions=torch.zeros(3, device="cuda")),
                dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(k=k.transpose(0, 1))):
        a = dict(k=k, v=k, q=q, q_out=q, positions=None)
        a.update(bad)
        with pytest.raises(ValueError):
            kvp.seq_append_rope(c.pool, [s], [3], a["k"], a["v"], kvp.rope_desc(64), a["positions"], a["q"], a["q_out"])
    assert kvp.seq_len(c.pool, s) == 0
    kvp.kv_pool_destroy(c.pool)
