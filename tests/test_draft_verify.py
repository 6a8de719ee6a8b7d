"""Verification of drafted tokens: the kernel against the walk written out on
the host in 64 bits, its refusals, and the distribution that it samples."""
import math

import numpy as np
import pytest

import paged_prefix_shared_decode_gb300 as kvp


def walk(target, draft, parent, token, u, u_next):
    """One sequence: (accepted, count, next).  Sums by math.fsum."""
    n = len(parent)
    V = target.shape[1]
    clean = lambda r: np.clip(np.nan_to_num(r.astype(np.float64), nan=0.0), 0.0, 1.0)
    par = [p if -1 <= p < i else -1 for i, p in enumerate(parent)]
    node, count = -1, 0
    while True:
        p = clean(target[node + 1])
        left, c, Z, took = p.copy(), 0.0, 1.0, None
        q = None
        for i in range(n):
            x = token[i]
            if par[i] != node or not 0 <= x < V:
                continue
            if draft is not None:
                q = clean(draft[node + 1])
                yes = float(u[i]) * q[x] * Z < p[x] - c * q[x]
            else:
                yes = float(u[i]) * Z < left[x]
            if yes:
                took = i
                break
            if draft is not None:
                c += Z
                left = np.maximum(p - c * q, 0.0)
                Z = math.fsum(left)
            else:
                Z = max(Z - left[x], 0.0)
                left[x] = 0.0
        if took is None:
            break
        node, count = took, count + 1
    if not left.any():
        left = p
    cum = np.cumsum(left)
    if cum[-1] == 0:
        return node, count, -1
    return node, count, int(np.searchsorted(cum, float(u_next) * cum[-1], side="right"))


def inputs(seed, B, n, V, tree=True, sharp=2.0):
    import torch
    g = np.random.default_rng(seed)
    x = g.normal(size=(B, n + 1, V)) * sharp
    y = x + 0.7 * g.normal(size=x.shape)
    soft = lambda z: (np.exp(z - z.max(-1, keepdims=True)) / np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)).astype(np.float32)
    p, q = soft(x), soft(y)
    par = np.zeros((B, n), np.int32)
    for i in range(n):
        par[:, i] = g.integers(-1, i, B) if tree else i - 1
    tok = np.zeros((B, n), np.int32)
    for b in range(B):
        for i in range(n):
            tok[b, i] = g.choice(V, p=q[b, par[b, i] + 1].astype(np.float64) / q[b, par[b, i] + 1].astype(np.float64).sum())
    u = g.random((B, n)).astype(np.float32)
    return dict(p=p, q=q, par=par, tok=tok, u=u, un=g.random(B).astype(np.float32))


def gpu(d, draft=True, p=None, q=None):
    import torch
    B = d["par"].shape[0]
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    out = [torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(3)]
    kvp.kvp_draft_verify(t(d["p"]) if p is None else p, (t(d["q"]) if q is None else q) if draft else None, t(d["par"]),
                         t(d["tok"]), t(d["u"]), t(d["un"]), *out)
    return np.stack([o.cpu().numpy() for o in out], 1)


def check(d, draft=True, **kw):
    got = gpu(d, draft, **kw)
    want = [walk(d["p"][b], d["q"][b] if draft else None, d["par"][b], d["tok"][b], d["u"][b], d["un"][b])
            for b in range(len(d["un"]))]
    assert got.tolist() == [list(w) for w in want]
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,n,V,tree", [(1, 1, 1, False), (3, 5, 2, True), (2, 7, 31, True), (5, 64, 33, True),
                                        (4, 9, 1000, True), (2, 63, 4097, True), (9, 4, 32003, False),
                                        (1, 6, 50000, True), (2, 3, 131071, True)])
def test_against_the_walk(B, n, V, tree, draft):
    check(inputs(B * 1000 + n, B, n, V, tree), draft)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,n,V", [(60, 3, 6001), (100, 3, 20001), (200, 2, 20000), (200, 2, 9001), (400, 1, 300)])
def test_batches_on_smaller_clusters(B, n, V, draft):
    check(inputs(B + V, B, n, V, True), draft)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_many_siblings(draft):
    # 40 children of the root, most of them rejected, equal tokens among them
    d = inputs(5, 6, 40, 300)
    d["par"][:] = -1
    d["u"] = np.sqrt(d["u"]).astype(np.float32)
    d["tok"][:, 1::7] = d["tok"][:, :1]
    got = check(d, draft)
    assert (got[:, 1] <= 1).all()


def sharp_siblings(n, V, pairs, u_next):
    """n children of the root, all of one token that the draft row is nearly
    certain of and the target rejects: c q(x) grows past n / 2.  pairs: (p, q)
    of that token, one per sequence; the rest of p lies on one other token."""
    B = len(pairs)
    d = dict(p=np.zeros((B, n + 1, V), np.float32), q=np.zeros((B, n, V), np.float32),
             par=np.full((B, n), -1, np.int32), tok=np.zeros((B, n), np.int32),
             u=np.full((B, n), 1.0 - 2.0 ** -24, np.float32), un=np.full(B, u_next, np.float32))
    for b, (p, q) in enumerate(pairs):
        x, y = (7 * b + 3) % V, (V - 1 - 5 * b) % V
        d["tok"][b] = x
        d["p"][b, 0, x], d["p"][b, 0, y] = p, np.float32(1) - np.float32(p)
        d["q"][b, 0, x], d["q"][b, 0, y] = q, np.float32(1) - np.float32(q)
    return d


# rows held in registers (up to 32768 tokens a sequence of a small batch), read
# as vectors (a length that is a multiple of 4) and element by element
@pytest.mark.gpu
@pytest.mark.parametrize("V", [40, 301, 40000, 40001])
@pytest.mark.parametrize("n,p,q", [(17, 1 / 16, 1.0), (31, 0.5, 1.0), (61, 0.75, 1.0), (64, 1 / 16, 1.0),
                                   (64, 0.25, 0.96875), (24, 0.125, 0.9375)])
def test_many_siblings_under_a_sharp_draft(V, n, p, q):
    # c q(x) reaches 16 and more: the token is spent, its residual stays 0
    for un in (0.0, 0.03, 0.4):
        d = sharp_siblings(n, V, [(p, q), (p / 2, q), (p, 1.0)], un)
        got = check(d)
        assert (got[:, 1] == 0).all() and (got[:, 2] != d["tok"][:, 0]).all()


@pytest.mark.gpu
def test_sharp_siblings_over_random_rows():
    # p(x) of 0.05 to 0.3 and q(x) of 0.9 to 0.99 on one token, the rest spread
    g = np.random.default_rng(11)
    B, n, V = 24, 64, 33
    d = sharp_siblings(n, V, [(0.1, 0.9)] * B, 0.5)
    for b in range(B):
        x = d["tok"][b, 0]
        for name, top in (("p", g.uniform(0.05, 0.3)), ("q", g.uniform(0.9, 0.99))):
            r = g.random(V)
            r[x] = 0
            r *= (1 - top) / r.sum()
            r[x] = top
            d[name][b, 0] = r
    d["un"] = g.random(B).astype(np.float32)
    check(d)


@pytest.mark.gpu
def test_no_drafts_is_sampling():
    d = inputs(6, 5, 3, 777)
    d.update(par=d["par"][:, :0], tok=d["tok"][:, :0], u=d["u"][:, :0])
    got = check(d)
    assert (got[:, 0] == -1).all() and (got[:, 1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("V", [64, 3003])
def test_strided_and_broadcast_rows(V):
    import torch
    d = inputs(7, 4, 6, V)
    # rows inside a wider buffer that starts off a 16-byte boundary; NaN around
    wide = torch.full((4, 9, V + 5), float("nan"), device="cuda")
    wide[:, 1:8, 3:V + 3] = torch.from_numpy(d["p"]).cuda()
    dw = torch.full((4, 7, V + 8), float("nan"), device="cuda")
    dw[:, :, 4:V + 4] = torch.from_numpy(d["q"]).cuda()
    check(d, p=wide[:, 1:8, 3:V + 3], q=dw[:, :6, 4:V + 4])
    # one distribution for the whole batch (batch stride 0)
    d["p"][:] = d["p"][:1]
    check(d, p=torch.from_numpy(d["p"][:1]).cuda().expand(4, -1, -1))


@pytest.mark.gpu
def test_borders():
    V = 130
    d = inputs(8, 8, 3, V, tree=False)
    d["un"][:] = [0.0, 1.0 - 2.0 ** -24, 0.5, 0.0, 0.25, 0.75, 0.0, 1.0 - 2.0 ** -24]
    d["u"][0] = 0.0                     # accepts whatever has p > c q
    d["u"][1] = 1.0 - 2.0 ** -24
    d["p"][2] = 0.0                     # nothing to sample
    d["p"][3, 0] = np.eye(V, dtype=np.float32)[17]       # greedy rows
    d["q"][3, 0] = np.eye(V, dtype=np.float32)[17]
    d["tok"][3, 0] = 17
    d["p"][4, 0] = np.eye(V, dtype=np.float32)[V - 1]
    d["q"][4, 0] = np.eye(V, dtype=np.float32)[3]
    d["tok"][4, 0] = 3
    d["q"][5] = d["p"][5]               # the draft is the target: never rejected
    d["par"][6] = [-1, 5, -9]           # bad parents are roots
    d["tok"][7] = [V, -1, 2 ** 30]      # no such tokens: left out
    got = check(d)
    assert got[2].tolist() == [-1, 0, -1]
    assert got[3, 1] >= 1 and got[4].tolist() == [-1, 0, V - 1]
    assert got[5, 1] == 3
    assert got[7, 0] == -1
    check(d, draft=False)


@pytest.mark.gpu
def test_all_of_p_taken_off():
    # p == q at the root and a child rejected by hand (its q is larger):
    # max(p - q, 0) is zero, so the token comes from p
    V = 50
    d = inputs(9, 2, 2, V)
    d["par"][:] = -1
    d["q"][:] = 1.0
    d["u"][:] = 0.99
    check(d)


@pytest.mark.gpu
def test_nan_and_negative_entries_count_as_zero():
    d = inputs(10, 4, 5, 515)
    d["p"][:, :, 5::17] = np.nan
    d["p"][:, :, 6::17] = -0.25
    d["q"][:, :, 7::17] = np.nan
    check(d)
    check(d, draft=False)


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
def test_sampled_distribution(draft):
    """The first token out (accepted child of the root, or the next token) has
    the target's distribution when the siblings are drawn from q (with a
    certain draft: any fixed siblings).  40000 walks; a frequency's standard
    deviation is sqrt(p (1 - p) / N), and 5 of them are allowed."""
    import torch
    N, V = 40000, 6
    p = np.array([0.4, 0.25, 0.2, 0.1, 0.05, 0.0], np.float32)
    q = np.array([0.1, 0.3, 0.05, 0.25, 0.2, 0.1], np.float32)
    g = np.random.default_rng(3)
    tok = g.choice(V, (N, 3), p=q / q.sum()).astype(np.int32) if draft else np.tile(np.int32([3, 1, 3]), (N, 1))
    d = dict(p=np.broadcast_to(p, (N, 4, V)), q=np.broadcast_to(q, (N, 4, V)), par=np.full((N, 3), -1, np.int32),
             tok=tok, u=g.random((N, 3)).astype(np.float32), un=g.random(N).astype(np.float32))
    t = lambda r: torch.from_numpy(r).cuda().expand(N, 4, V)
    acc, cnt, nxt = gpu(d, draft, p=t(p), q=t(q)).T
    first = np.where(acc >= 0, tok[np.arange(N), np.maximum(acc, 0)], nxt)
    f = np.bincount(first, minlength=V) / N
    assert (np.abs(f - p) <= 5 * np.sqrt(p * (1 - p) / N) + 1e-12).all(), f


@pytest.mark.gpu
def test_replayed_and_on_another_stream():
    import torch
    d = inputs(11, 4, 8, 5000)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    bufs = [t(d[k]) for k in ("p", "q", "par", "tok", "u", "un")]
    out = [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(3)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kvp.kvp_draft_verify(*bufs, *out)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvp.kvp_draft_verify(*bufs, *out)
    for seed in (12, 13):
        d = inputs(seed, 4, 8, 5000)
        for b, k in zip(bufs, ("p", "q", "par", "tok", "u", "un")):
            b.copy_(t(d[k]))
        for o in out:
            o.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        want = [walk(d["p"][b], d["q"][b], d["par"][b], d["tok"][b], d["u"][b], d["un"][b]) for b in range(4)]
        assert np.stack([o.cpu().numpy() for o in out], 1).tolist() == [list(w) for w in want]


def test_refusals():
    lib = kvp.load()
    a = 1 << 20
    ok = dict(target=a, tb=700, tr=100, draft=a, db=700, dr=100, par=a, tok=a, u=a, un=a, B=2, n=6, V=100, acc=a,
              cnt=a, nxt=a, stream=None)
    for bad in (dict(target=None), dict(un=None), dict(par=None), dict(tok=None), dict(u=None), dict(acc=None),
                dict(cnt=None), dict(nxt=None), dict(B=0), dict(B=-1), dict(n=-1), dict(n=65), dict(V=0),
                dict(V=2 ** 30 + 1, tr=2 ** 31, dr=2 ** 31), dict(tr=-1), dict(dr=-1), dict(tb=-1), dict(db=-1),
                dict(target=a + 2), dict(nxt=a + 1)):
        assert lib.kvp_draft_verify(*{**ok, **bad}.values()) == kvp.KVP_ERR_INVALID, bad


def test_refused_tensors():
    import torch
    i, f = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    o = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):   # host tensors
        kvp.kvp_draft_verify(torch.zeros(2, 4, 9), None, i, i, f, torch.zeros(2), o, o, o)
    with pytest.raises(ValueError):   # 16-bit probabilities
        kvp.kvp_draft_verify(torch.zeros(2, 4, 9, dtype=torch.bfloat16), None, i, i, f, torch.zeros(2), o, o, o)
