"""Accumulated attention weight and eviction over the pool, against plain
64-bit forms, and a run of them with the attention whose cache they keep."""
import math

import numpy as np
import pytest
import torch

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu


def make_pool(L, NB, Hkv, bs, d, seqs=16, MB=None, seed=3, gen=None):
    gen = gen or torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(L, NB, Hkv, bs, d, device="cuda", dtype=torch.bfloat16, generator=gen)
    v = torch.randn(L, NB, Hkv, bs, d, device="cuda", dtype=torch.bfloat16, generator=gen)
    return kvp.kv_pool_create(kvp.PoolDesc(L, NB, bs, Hkv, d, seqs, MB or NB, seed), k, v), k, v


def rows_of(pool_t, table, bs, n):
    """Token rows [L][n][Hkv][d] of one sequence's pages."""
    t = torch.as_tensor(np.asarray(table), device="cuda").long()
    pos = torch.arange(n, device="cuda")
    return pool_t[:, t[pos // bs], :, pos % bs].transpose(0, 1)   # indexing puts tokens first


# -------------------------------------------------------------------- mass

def mass_case(d, G, Hkv, bs, L, lens, qlens, seed=0, scale=0.0, mul=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S, Hq = len(lens), G * Hkv
    nb = [-(-n // bs) for n in lens]
    NB, MB = sum(nb) + 3, max(1, max(nb)) + 1
    order = torch.randperm(NB, generator=torch.Generator().manual_seed(seed)).numpy().astype(np.int32)
    tables, at = np.full((S, MB), -1, np.int32), 0
    for s, m in enumerate(nb):
        tables[s, :m] = order[at:at + m]
        at += m
    k = torch.full((L, NB, Hkv, bs, d), float("nan"), device="cuda", dtype=torch.bfloat16)   # unwritten slots
    T = sum(qlens)
    q = (torch.randn(L, T, Hq, d, device="cuda", generator=gen) * mul).to(torch.bfloat16)
    keys, lse, q0 = [], torch.zeros(L, T, Hq, device="cuda"), 0
    for s, n in enumerate(lens):
        x = torch.randn(L, n, Hkv, d, device="cuda", generator=gen).to(torch.bfloat16)
        keys.append(x)
        pos = torch.arange(n, device="cuda")
        blk = torch.from_numpy(tables[s].astype(np.int64)).cuda()[pos // bs]
        k[:, blk, :, pos % bs] = x.transpose(0, 1)
    sc = scale if scale > 0 else 1 / math.sqrt(d)
    want, size = [], 0.0     # [L][Hkv][n] per sequence; largest scale * sum |q k|
    for s, (n, m) in enumerate(zip(lens, qlens)):
        qs = q[:, q0:q0 + m].double().view(L, m, Hkv, G, d)
        ks = keys[s].double()
        sco = torch.einsum("lmhgd,lnhd->lmhgn", qs, ks) * sc
        if n and m:
            size = max(size, float(torch.einsum("lmhgd,lnhd->lmhgn", qs.abs(), ks.abs()).max() * sc))
        see = torch.arange(n, device="cuda") <= torch.arange(n - m, n, device="cuda")[:, None]
        sco = sco.masked_fill(~see[None, :, None, None], -math.inf)
        z = torch.logsumexp(sco, -1).float() if n else torch.zeros(L, m, Hkv, G, device="cuda")
        lse[:, q0:q0 + m] = z.reshape(L, m, Hq)
        want.append(torch.exp(sco - z.double()[..., None]).sum((1, 3)))
        q0 += m
    desc = kvp.AttnDesc(L, Hq, Hkv, d, bs, NB, scale, 1)
    # A score is a sum of d products (exact in 32 bits) with at most d + 2
    # roundings, of values up to scale * sum |q k|; its error is the weight's
    # relative error, to which lse's rounding (|lse| 2^-23 with the change of
    # base), two for the exponent's argument and 2^-21 for exp2 itself add.
    rtol = (d + 2) * 2.0 ** -24 * size + 2.0 ** -22 * (float(lse.abs().max()) if T else 0) + 2.0 ** -20
    return desc, q, lse, k, tables, want, rtol


def run_mass(desc, q, qlens, lse, k, tables, lens, decay, mass_in, prev, out):
    n = kvp.kvp_mass_workspace_size(desc, tables, lens, qlens)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    kvp.kvp_attention_mass(q, qlens, lse, k, tables, lens, desc, decay, mass_in, prev, out, ws)
    torch.cuda.synchronize()
    assert kvp.kvp_device_error(ws) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Hkv,bs,L,lens,qlens", [
    (1, 2, 16, 1, [1], [1]),
    (8, 4, 16, 2, [1, 15, 16, 17, 31, 33, 129, 640], None),
    (4, 2, 32, 1, [500, 3, 1000, 127, 128], [1, 1, 1, 1, 1]),
    (7, 3, 64, 2, [200, 70], [2, 1]),                  # 14 rows, then 7
    (16, 1, 16, 1, [257], [1]),                        # a full row tile
    (24, 1, 16, 1, [100, 40], [1, 1]),                 # two row tiles
    (4, 2, 16, 2, [0, 90, 5, 300, 64], [0, 5, 5, 33, 0]),
    (2, 2, 32, 1, [700, 140], [140, 140]),             # queries over several stages
    (64, 1, 16, 1, [77], [3]),
    (4, 2, 128, 1, [500, 129, 128], [20, 129, 5]),     # blocks as long as a tile of tokens, and longer
    (3, 2, 256, 2, [700, 256, 1], [50, 7, 1]),
])
def test_mass(d, G, Hkv, bs, L, lens, qlens):
    ql = qlens or [1] * len(lens)
    desc, q, lse, k, tables, want, rtol = mass_case(d, G, Hkv, bs, L, lens, ql, seed=len(lens) + d)
    S, stride = len(lens), max(lens) + 3
    old = torch.rand(L, S, Hkv, stride, device="cuda")
    out = torch.full_like(old, -5.0)
    decay = 0.75
    run_mass(desc, q, qlens, lse, k, tables, lens, decay, old, None, out)
    for s, n in enumerate(lens):
        assert (out[:, s, :, n:] == -5).all()          # behind the sequence: as it was
        prev = n - ql[s]
        w = want[s] + decay * old[:, s, :, :n].double() * (torch.arange(n, device="cuda") < prev)
        err = (out[:, s, :, :n].double() - w).abs()
        # + the sum over rows (at most rows roundings) and the last fma
        assert (err <= (rtol + (ql[s] * G + 2) * 2.0 ** -24) * w).all(), (s, float((err / w.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("d,G,lse", [(64, 16, 9.0), (128, 16, 7.3), (64, 5, 11.7)])
def test_mass_of_a_long_chunk_of_equal_weights(d, G, lse):
    """Up to 131072 rows give a token the same weight: roundings of one running sum all go the same way and add up."""
    lens, ql = [8200, 300], [8192, 300]
    desc, q, z, k, tables, _, _ = mass_case(d, 1, 1, 16, 1, lens, [1, 1])
    desc.num_q_heads = G
    q = torch.zeros(1, sum(ql), G, d, device="cuda", dtype=torch.bfloat16)      # every score is 0
    z = torch.full((1, sum(ql), G), lse, device="cuda")
    out = torch.full((1, 2, 1, 8200), -5.0, device="cuda")
    run_mass(desc, q, ql, z, k, tables, lens, 1.0, None, None, out)
    w = float(torch.exp(-z.double()[0, 0, 0]))
    # the exponent's argument: log2 e and its product with lse, half a step each
    # (relative 2^-24, of |lse| as a natural exponent); exp2 itself 2^-21; the
    # sum: 32 terms to an accumulator, two steps to join them, and the sum over
    # the chunks and its last step, whatever the number of rows
    tol = lse * 2.0 ** -23 + 2.0 ** -21 + 38 * 2.0 ** -24
    for s, (n, m) in enumerate(zip(lens, ql)):
        pos = torch.arange(n, device="cuda")
        want = (n - pos.clamp(min=n - m)).double() * G * w
        err = (out[0, s, 0, :n].double() - want).abs() / want
        assert (err <= tol).all(), (s, float(err.max()), tol)
        assert (out[0, s, 0, n:] == -5).all()


def test_mass_of_a_long_chunk():
    lens, ql = [4400, 1000], [4096, 999]
    desc, q, lse, k, tables, want, rtol = mass_case(128, 4, 1, 16, 1, lens, ql, seed=3)
    out = torch.zeros(1, 2, 1, 4400, device="cuda")
    run_mass(desc, q, ql, lse, k, tables, lens, 1.0, None, None, out)
    for s, n in enumerate(lens):
        err = (out[:, s, :, :n].double() - want[s]).abs()
        assert (err <= (rtol + 38 * 2.0 ** -24) * want[s]).all(), s


@pytest.mark.parametrize("d,G,L,Hkv", [(64, 8, 3, 3), (128, 4, 2, 5), (128, 5, 1, 2)])
def test_mass_many_sequences(d, G, L, Hkv):
    """More tiles than CTAs, every run of them crossing sequences and heads of
    one to many row chunks, some without queries or tokens."""
    g = np.random.default_rng(d + G)
    lens = [int(x) for x in g.integers(0, 1500, 30)]
    ql = [min(n, int(g.choice([0, 1, 3, 40, 150]))) for n in lens]
    desc, q, lse, k, tables, want, rtol = mass_case(d, G, Hkv, 16, L, lens, ql, seed=5)
    old = torch.rand(L, 30, Hkv, 1500, device="cuda")
    out = torch.full_like(old, -5.0)
    for _ in range(2):      # the workspace and its barriers are used again
        run_mass(desc, q, ql, lse, k, tables, lens, 0.5, old, None, out)
    for s, n in enumerate(lens):
        w = want[s] + 0.5 * old[:, s, :, :n].double() * (torch.arange(n, device="cuda") < n - ql[s])
        assert ((out[:, s, :, :n].double() - w).abs() <= (rtol + (ql[s] * G + 2) * 2.0 ** -24) * w).all(), s
        assert (out[:, s, :, n:] == -5).all()


def test_mass_in_place_prev_and_none():
    lens, ql = [50, 200], [1, 4]
    desc, q, lse, k, tables, want, rtol = mass_case(64, 4, 2, 16, 1, lens, ql, seed=9)
    base = torch.rand(1, 2, 2, 200, device="cuda")
    a = base.clone()
    run_mass(desc, q, ql, lse, k, tables, lens, 1.0, a, [50, 100], a)          # in place
    b = torch.zeros_like(base)
    run_mass(desc, q, ql, lse, k, tables, lens, 1.0, None, None, b)
    for s, n in enumerate(lens):
        prev = [50, 100][s]
        w = want[s] + base[:, s, :, :n].double() * (torch.arange(n, device="cuda") < prev)
        assert ((a[:, s, :, :n].double() - w).abs() <= (rtol + 2.0 ** -19) * w).all()
        assert ((b[:, s, :, :n].double() - want[s]).abs() <= (rtol + 2.0 ** -19) * want[s]).all()
    # the weights of one step sum to the query heads of the group: each softmax row sums to 1
    assert (b[0, 0, :, :50].sum(-1) - 4).abs().max() < 50 * 4 * rtol


def test_mass_rows_without_keys_add_nothing_and_large_scores():
    lens, ql = [90], [3]
    desc, q, lse, k, tables, want, rtol = mass_case(128, 2, 2, 16, 1, lens, ql, seed=4, mul=12.0)
    lse[0, 1] = -math.inf
    desc2, *_ = mass_case(128, 2, 2, 16, 1, lens, ql, seed=4, mul=12.0)
    out = torch.zeros(1, 1, 2, 90, device="cuda")
    run_mass(desc, q, ql, lse, k, tables, lens, 1.0, None, None, out)
    assert torch.isfinite(out).all()
    # the other two rows alone
    ks = rows_of(k, tables[0], 16, 90).double()[0]
    qs = q[0].double().view(3, 2, 2, 128)
    w = torch.zeros(2, 90, dtype=torch.float64, device="cuda")
    for i in (0, 2):
        e = torch.exp(torch.einsum("hgd,nhd->hgn", qs[i], ks) / math.sqrt(128) - lse[0, i].double().view(2, 2, 1))
        w += e.sum(1) * (torch.arange(90, device="cuda") <= 87 + i)
    assert ((out[0, 0].double() - w).abs() <= (rtol + 2.0 ** -19) * w).all()


def test_mass_after_decode_attention():
    # the lse that the library's own attention leaves
    lens = [333, 64, 1000]
    desc, q, lse, k, tables, want, rtol = mass_case(128, 4, 8, 16, 2, lens, [1, 1, 1], seed=21)
    k = torch.nan_to_num(k)
    v = torch.randn_like(k)
    out, z = torch.empty_like(q), torch.empty_like(lse)
    ws = torch.empty(kvp.kvp_decode_workspace_size(desc, tables, lens), dtype=torch.uint8, device="cuda")
    kvp.paged_decode_attention(q, k, v, tables, lens, desc, out, z, ws)
    mass = torch.zeros(2, 3, 8, 1000, device="cuda")
    run_mass(desc, q, None, z, k, tables, lens, 1.0, None, None, mass)
    tol = rtol + float((z - lse).abs().max()) + 2.0 ** -20
    assert tol < 2e-3
    for s, n in enumerate(lens):
        assert ((mass[:, s, :, :n].double() - want[s]).abs() <= tol * want[s]).all()


def test_mass_refuses_capture():
    lens = [40]
    desc, q, lse, k, tables, *_ = mass_case(64, 4, 1, 16, 1, lens, [1])
    out = torch.zeros(1, 1, 1, 40, device="cuda")
    ws = torch.empty(kvp.kvp_mass_workspace_size(desc, tables, lens), dtype=torch.uint8, device="cuda")
    x = torch.zeros(4, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x += 1
        with pytest.raises(kvp.KvpError) as e:
            kvp.kvp_attention_mass(q, None, lse, k, tables, lens, desc, 1.0, None, None, out, ws)
    assert e.value.code == kvp.KVP_ERR_STATE


# ------------------------------------------------------------------- evict

def pick(mass, n, budget, sink, recent):
    """Kept positions of one row: plain, in 64 bits."""
    if n <= budget:
        return np.arange(n)
    w = mass[:n].astype(np.float64)
    w = np.where(np.isnan(w), -np.inf, w)
    nan = np.isnan(mass[:n])
    mid = [i for i in range(n) if sink <= i < n - recent]
    mid.sort(key=lambda i: (-w[i], nan[i], i))
    return np.sort(np.array(list(range(sink)) + mid[:budget - sink - recent] + list(range(n - recent, n))))


def evict(pool, seqs, mass, budget, sink, recent, mass_out="new"):
    L, n, Hkv, stride = mass.shape
    kept = torch.full((L, n, Hkv, budget), -9, dtype=torch.int32, device="cuda")
    mo = torch.full_like(mass, -3.0) if isinstance(mass_out, str) else mass_out
    ws = torch.empty(kvp.seq_evict_workspace_size(pool, seqs, budget), dtype=torch.uint8, device="cuda")
    kvp.seq_evict(pool, seqs, mass, budget, sink, recent, kept, mo, ws)
    torch.cuda.synchronize()
    return kept, mo


def check_evicted(pool, k, v, seqs, before, mass, budget, sink, recent, kept, mo, bs):
    """before: per sequence (len, K rows, V rows) from before the call."""
    L, _, Hkv, stride = mass.shape
    m = mass.cpu().numpy()
    for i, s in enumerate(seqs):
        n, K, V = before[i]
        keep = min(n, budget)
        assert kvp.seq_len(pool, s) == keep
        table = kvp.seq_block_table(pool, s)
        assert len(table) == -(-keep // bs)
        K1, V1 = rows_of(k, table, bs, keep), rows_of(v, table, bs, keep)
        for l in range(L):
            for h in range(Hkv):
                want = pick(m[l, i, h], n, budget, sink, recent)
                got = kept[l, i, h].cpu().numpy()
                assert (got[:keep] == want).all() and (got[keep:] == -1).all()
                if n == 0:
                    continue
                ix = torch.from_numpy(want).cuda()
                assert torch.equal(K1[l, :, h], K[l, ix, h]) and torch.equal(V1[l, :, h], V[l, ix, h])
                if mo is not None:
                    a = mo[l, i, h, :keep].cpu().numpy()
                    assert np.array_equal(a, m[l, i, h, want], equal_nan=True)


def snapshot(pool, k, v, seqs, bs):
    out = []
    for s in seqs:
        n = kvp.seq_len(pool, s)
        t = kvp.seq_block_table(pool, s)
        out.append((n, rows_of(k, t, bs, n).clone(), rows_of(v, t, bs, n).clone()) if n else (0, None, None))
    return out


def weights(L, n, Hkv, stride, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.empty(L, n, Hkv, stride, device="cuda").exponential_(generator=g) ** 3
    return torch.where(m < 0.3, torch.round(m * 20) / 20, m)     # ties


@pytest.mark.parametrize("L,Hkv,bs,d", [(1, 1, 16, 64), (2, 3, 32, 128), (1, 2, 8, 24), (2, 2, 1, 8)])
@pytest.mark.parametrize("n,budget,sink,recent", [(40, 39, 0, 0), (100, 7, 3, 4), (257, 64, 4, 16), (600, 599, 17, 33),
                                                  (1000, 500, 0, 100), (2500, 1, 0, 0), (2500, 1, 1, 0),
                                                  (90, 90, 4, 4), (33, 64, 2, 2)])
def test_evict_in_place(L, Hkv, bs, d, n, budget, sink, recent):
    nb = -(-n // bs)
    pool, k, v = make_pool(L, nb + 2, Hkv, bs, d)
    s = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, s, n)
    before = snapshot(pool, k, v, [s], bs)
    t0 = list(kvp.seq_block_table(pool, s))
    free0 = kvp.kvp_free_block_count(pool)
    mass = weights(L, 1, Hkv, n + 3)
    kept, mo = evict(pool, [s], mass, budget, sink, recent)
    check_evicted(pool, k, v, [s], before, mass, budget, sink, recent, kept, mo, bs)
    t1 = list(kvp.seq_block_table(pool, s))
    assert t1 == t0[:len(t1)]                                        # its own pages, in place
    assert kvp.kvp_free_block_count(pool) == free0 + len(t0) - len(t1)
    kvp.kv_pool_destroy(pool)


def test_evict_shared_pages():
    L, Hkv, bs, d, n, budget, sink = 2, 2, 16, 64, 700, 200, 37
    pool, k, v = make_pool(L, 200, Hkv, bs, d)
    a = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, a, n)
    b = kvp.seq_fork(pool, a)
    kvp.seq_reserve(pool, b, 20)          # a copied last page: b's pages past it are its own
    k0, v0 = k.clone(), v.clone()
    ta = list(kvp.seq_block_table(pool, a))
    before = snapshot(pool, k, v, [b], bs)
    mass = weights(L, 1, Hkv, 720)
    kept, mo = evict(pool, [b], mass, budget, sink, 20)
    check_evicted(pool, k, v, [b], before, mass, budget, sink, 20, kept, mo, bs)
    tb = list(kvp.seq_block_table(pool, b))
    assert tb[:2] == ta[:2] and not set(tb[2:]) & set(ta)            # 32 sink tokens stay shared
    assert list(kvp.seq_block_table(pool, a)) == ta                  # the parent is whole
    for x in ta:
        assert torch.equal(k[:, x], k0[:, x]) and torch.equal(v[:, x], v0[:, x])
        assert kvp.block_refcount(pool, x) == (2 if x in tb else 1)
    kvp.seq_free(pool, a)
    kvp.seq_free(pool, b)
    assert kvp.kvp_free_block_count(pool) == 200
    kvp.kv_pool_destroy(pool)


def test_evict_siblings_in_one_call_and_mixed_pages():
    """Siblings that share pages with each other alone, one sequence whose
    first pages the prefix cache holds (fresh and in-place pages in one
    table), one that fits the budget and one that is empty."""
    L, Hkv, bs, d = 1, 2, 16, 128
    pool, k, v = make_pool(L, 300, Hkv, bs, d)
    a = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, a, 500)
    b = kvp.seq_fork(pool, a)
    c = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, c, 411)
    cache = kvp.kvp_radix_create(pool)
    tc = list(kvp.seq_block_table(pool, c))
    kvp.kvp_radix_insert(cache, np.arange(48), tc[:3])               # three pages of c are cached
    small, empty = kvp.seq_alloc(pool), kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, small, 60)
    seqs = [a, b, c, small, empty]
    before = snapshot(pool, k, v, seqs, bs)
    k0 = k.clone()
    ta = list(kvp.seq_block_table(pool, a))
    mass = weights(L, 5, Hkv, 501)
    kept, mo = evict(pool, seqs, mass, 130, 5, 30)
    check_evicted(pool, k, v, seqs, before, mass, 130, 5, 30, kept, mo, bs)
    na, nb, nc = (list(kvp.seq_block_table(pool, s)) for s in (a, b, c))
    assert not set(na) & set(ta) and not set(nb) & set(ta) and not set(na) & set(nb)
    assert not set(nc[:3]) & set(tc) and nc[3:] == tc[3:9]           # cached pages left alone, the rest in place
    for x in tc[:3]:
        assert torch.equal(k[:, x], k0[:, x]) and kvp.block_refcount(pool, x) == 1
    assert all(kvp.block_refcount(pool, x) == 0 for x in ta)
    kvp.kvp_radix_destroy(cache)
    for s in seqs:
        kvp.seq_free(pool, s)
    assert kvp.kvp_free_block_count(pool) == 300
    kvp.kv_pool_destroy(pool)


@pytest.mark.parametrize("same", [True, False])
def test_evict_odd_weights_and_mass_in_place(same):
    n, budget = 300, 150
    pool, k, v = make_pool(1, 40, 2, 16, 64)
    s = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, s, n)
    mass = weights(1, 1, 2, n)
    mass[0, 0, 0, ::3] = float("nan")
    mass[0, 0, 0, 1::3] = 0.0
    mass[0, 0, 0, 4::9] = -0.0
    mass[0, 0, 1, :250] = 1.0                                       # ties across warps
    mass[0, 0, 1, 7] = float("inf")
    mass[0, 0, 1, 8] = -float("inf")
    before = snapshot(pool, k, v, [s], 16)
    ref = mass.clone()
    kept, mo = evict(pool, [s], mass, budget, 2, 3, mass if same else None)
    check_evicted(pool, k, v, [s], before, ref, budget, 2, 3, kept, mo, 16)
    if not same:
        assert torch.equal(mass.nan_to_num(9.0), ref.nan_to_num(9.0))
    kvp.kv_pool_destroy(pool)


@pytest.mark.parametrize("same", [True, False])
def test_evict_long_rows(same):
    # past what a CTA holds of a row's weights
    n, budget = 70001, 20000
    pool, k, v = make_pool(1, -(-n // 64) + 1, 1, 64, 8)
    s = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, s, n)
    mass = weights(1, 1, 1, n)
    before, ref = snapshot(pool, k, v, [s], 64), mass.clone()
    kept, mo = evict(pool, [s], mass, budget, 4, 100, mass if same else None)
    check_evicted(pool, k, v, [s], before, ref, budget, 4, 100, kept, mo, 64)
    kvp.kv_pool_destroy(pool)


def test_evict_many_sequences():
    # an image of sequences and tables too long for the kernel parameters
    pool, k, v = make_pool(1, 1500, 2, 16, 64, seqs=40)
    seqs = [kvp.seq_alloc(pool) for _ in range(20)]
    for i, s in enumerate(seqs):
        kvp.seq_reserve(pool, s, 300 + 37 * i)
    seqs += [kvp.seq_fork(pool, s) for s in seqs[:5]]
    before = snapshot(pool, k, v, seqs, 16)
    mass = weights(1, 25, 2, 1100)
    kept, mo = evict(pool, seqs, mass, 333, 17, 40)
    check_evicted(pool, k, v, seqs, before, mass, 333, 17, 40, kept, mo, 16)
    for s in seqs:
        kvp.seq_free(pool, s)
    assert kvp.kvp_free_block_count(pool) == 1500
    kvp.kv_pool_destroy(pool)


def test_evict_out_of_blocks_changes_nothing():
    pool, k, v = make_pool(1, 12, 1, 16, 64)
    a = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, a, 10 * 16)
    b = kvp.seq_fork(pool, a)
    k0, t0 = k.clone(), list(kvp.seq_block_table(pool, b))
    mass = weights(1, 1, 1, 160)
    with pytest.raises(kvp.KvpError) as e:
        evict(pool, [b], mass, 48, 0, 0)                             # three fresh blocks, two free
    assert e.value.code == kvp.KVP_ERR_OOM
    assert list(kvp.seq_block_table(pool, b)) == t0 and kvp.kvp_free_block_count(pool) == 2
    assert torch.equal(k, k0)
    evict(pool, [b], mass, 48, 16, 0)                                # a sink page stays: two are enough
    kvp.kv_pool_destroy(pool)


def test_evict_refuses_capture():
    pool, k, v = make_pool(1, 12, 1, 16, 64)
    a = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, a, 100)
    mass = weights(1, 1, 1, 100)
    kept = torch.zeros(1, 1, 1, 50, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvp.seq_evict_workspace_size(pool, [a], 50), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mass += 1
        with pytest.raises(kvp.KvpError) as e:
            kvp.seq_evict(pool, [a], mass, 50, 0, 0, kept, None, ws)
    assert e.value.code == kvp.KVP_ERR_STATE and kvp.seq_len(pool, a) == 100
    kvp.kv_pool_destroy(pool)


# ------------------------------------------------------------- run together

def test_decode_with_a_bounded_cache():
    """Four branches decode, their weights accumulate, and every few steps
    their caches are cut back; attention over the cut cache is checked against
    the kept tokens in 64 bits."""
    L, Hq, Hkv, bs, d, budget = 2, 8, 2, 16, 64, 96
    pool, k, v = make_pool(L, 120, Hkv, bs, d)
    root = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, root, 200)
    seqs = [kvp.seq_fork(pool, root) for _ in range(4)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    desc = kvp.AttnDesc(L, Hq, Hkv, d, bs, 120, 0.0, 1)
    mass = torch.zeros(L, 4, Hkv, 256, device="cuda")
    prev = [0] * 4
    held = [rows_of(k, kvp.seq_block_table(pool, s), bs, 200).clone() for s in seqs]
    heldv = [rows_of(v, kvp.seq_block_table(pool, s), bs, 200).clone() for s in seqs]
    rnd = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16, generator=gen)
    for step in range(10):
        kn, vn, q = rnd(L, 4, Hkv, d), rnd(L, 4, Hkv, d), rnd(L, 4, Hq, d)
        kvp.seq_append_batch(pool, seqs, [1] * 4, kn, vn)
        held = [torch.cat([h, kn[:, i:i + 1]], 1) for i, h in enumerate(held)]
        heldv = [torch.cat([h, vn[:, i:i + 1]], 1) for i, h in enumerate(heldv)]
        t, ln = kvp.kvp_gather_tables(pool, seqs, 16)
        out, lse = torch.empty_like(q), torch.empty(L, 4, Hq, device="cuda")
        ws = torch.empty(kvp.kvp_decode_workspace_size(desc, t, ln), dtype=torch.uint8, device="cuda")
        kvp.paged_decode_attention(q, k, v, t, ln, desc, out, lse, ws)
        ws2 = torch.empty(kvp.kvp_mass_workspace_size(desc, t, ln), dtype=torch.uint8, device="cuda")
        kvp.kvp_attention_mass(q, None, lse, k, t, ln, desc, 0.9, mass, prev, mass, ws2)
        prev = [int(x) for x in ln]
        for i in range(4):
            K, V = held[i].double(), heldv[i].double()
            x = torch.einsum("lhgd,lnhd->lhgn", q[:, i].double().view(L, Hkv, Hq // Hkv, d), K) / math.sqrt(d)
            o = torch.einsum("lhgn,lnhd->lhgd", torch.softmax(x, -1), V).reshape(L, Hq, d)
            err = (out[:, i].double() - o).abs()
            # P and out are rounded to bf16: 2^-8 of sum p |v| and of |out| at most, half of each
            assert (err <= 2.0 ** -8 * (V.abs().max() + o.abs())).all()
        if step % 4 == 3:
            kept, _ = evict(pool, seqs, mass, budget, 4, 16, mass)
            for i in range(4):
                ix = kept[:, i].long().transpose(1, 2)[..., None].expand(-1, -1, -1, d)   # [L][budget][Hkv][d]
                held[i], heldv[i] = held[i].gather(1, ix), heldv[i].gather(1, ix)
            prev = [budget] * 4
    for s in [root] + seqs:
        kvp.seq_free(pool, s)
    assert kvp.kvp_free_block_count(pool) == 120
    kvp.kv_pool_destroy(pool)


def test_default_stream_beside_a_capture_is_refused_whole():
    """The legacy default stream cannot be used while a stream that synchronises with it is captured: the calls say
    so before anything changes, and the capture goes on."""
    import ctypes
    pool, k, v = make_pool(1, 12, 1, 16, 64)
    a = kvp.seq_alloc(pool)
    kvp.seq_reserve(pool, a, 100)
    mass = weights(1, 1, 1, 100)
    kept = torch.zeros(1, 1, 1, 50, dtype=torch.int32, device="cuda")
    t, ln = kvp.kvp_gather_tables(pool, [a], 8)
    desc = kvp.AttnDesc(1, 2, 1, 64, 16, 12, 0.0, 1)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(1, 1, 2, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    cu = ctypes.CDLL("libcuda.so.1")
    s, g = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(s), 0) == 0
    assert cu.cuStreamBeginCapture_v2(s, 1) == 0         # a capture of this thread's
    codes = []
    for call in (lambda: kvp.seq_evict(pool, [a], mass, 50, 0, 0, kept, None, ws, stream=0),
                 lambda: kvp.kvp_attention_mass(q, None, z, k, t, ln, desc, 1.0, None, None, mass, ws, stream=0),
                 lambda: kvp.paged_window_attention(q, None, k, v, t, ln, 8, 0, desc, out, z, ws, stream=0)):
        try:
            call()
            codes.append(kvp.KVP_OK)
        except kvp.KvpError as e:
            codes.append(e.code)
    ended = cu.cuStreamEndCapture(s, ctypes.byref(g))
    assert cu.cuGraphDestroy(g) == 0 if ended == 0 else True
    assert cu.cuStreamDestroy_v2(s) == 0
    assert codes == [kvp.KVP_ERR_STATE] * 3 and kvp.seq_len(pool, a) == 100
    assert ended == 0
    torch.cuda.synchronize()
    kvp.seq_evict(pool, [a], mass, 50, 0, 0, kept, None, ws, stream=0)
    torch.cuda.synchronize()
    assert kvp.seq_len(pool, a) == 50
    kvp.kv_pool_destroy(pool)
