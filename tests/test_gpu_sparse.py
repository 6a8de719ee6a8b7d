"""Page bounds, page scores, page selection and attention over selected pages
against their definitions in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences with scattered pages; the last page's free slots and a spare
    table entry hold what must not matter."""

    def __init__(self, lens, q_lens=None, heads=(8, 2), d=64, bs=16, L=1, seed=0, spare=2, poison=True):
        g = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.q_lens = list(lens), q_lens
        nq = [1] * len(lens) if q_lens is None else list(q_lens)
        self.nq, self.T, self.S = nq, sum(nq), len(lens)
        (self.Hq, self.Hkv), self.d, self.bs, self.L = heads, d, bs, L
        pages = [-(-n // bs) for n in lens]
        self.NB, self.MB = sum(pages) + 3, max(pages + [1]) + spare
        order = g.permutation(self.NB)
        self.tables = np.full((self.S, self.MB), -1, np.int32)
        at = 0
        for s, n in enumerate(pages):
            self.tables[s, :n] = order[at:at + n]
            at += n
        norm = lambda *sh: torch.randn(sh, generator=gen, device="cuda", dtype=torch.bfloat16)
        self.k, self.v = norm(L, self.NB, self.Hkv, bs, d), norm(L, self.NB, self.Hkv, bs, d)
        self.q = norm(L, self.T, self.Hq, d)
        if poison:
            for s, n in enumerate(lens):
                if n % bs:
                    b = int(self.tables[s, n // bs])
                    self.k[:, b, :, n % bs:] = math.nan
                    self.v[:, b, :, n % bs:] = math.inf
        self.t, self.n = torch.from_numpy(self.tables).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.start = None
        if q_lens is not None:
            self.start = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device="cuda")
        self.desc = kvp.AttnDesc(L, self.Hq, self.Hkv, d, bs, self.NB, 0.0, 0)
        # (sequence, position) of every query row
        self.rows = [(s, lens[s] - nq[s] + i) for s in range(self.S) for i in range(nq[s])]

    def seen(self, t):
        s, p = self.rows[t]
        return p // self.bs + 1 if p >= 0 else 0

    def bounds(self, n_new=None, out=None):
        out = torch.full((self.L, self.NB, self.Hkv, 2, self.d), 9.0, dtype=torch.bfloat16,
                         device="cuda") if out is None else out
        kvp.kvp_page_bounds(self.k, self.t, self.n, max(self.lens) + 1 if n_new is None else n_new, self.desc, out)
        return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs,lens", [(16, [1, 16, 17, 0, 100]), (32, [31, 200]), (128, [5, 300]), (1024, [1500])])
def test_bounds(d, bs, lens):
    b = Batch(lens, d=d, bs=bs, L=2)
    for n_new in (None, 1, 2, 17):
        got = b.bounds(n_new)
        want = torch.full_like(got, 9.0)
        for s, n in enumerate(lens):
            for j in range(-(-n // bs)):
                if n_new is not None and (j + 1) * bs <= n - n_new:
                    continue
                x = b.k[:, int(b.tables[s, j]), :, :min(bs, n - j * bs)]
                want[:, int(b.tables[s, j])] = torch.stack([x.amin(2), x.amax(2)], 2)
        assert torch.equal(got, want)
    untouched = b.bounds(0)
    assert bool((untouched == 9.0).all())


def test_bounds_show_nan_and_skip_bad_entries():
    b = Batch([40, 20], d=64)
    blk = int(b.tables[0, 1])
    b.k[0, blk, 1, 3, 7] = math.nan
    b.t[1, 0] = b.NB            # not a block
    got = b.bounds()
    assert torch.isnan(got[0, blk, 1, :, 7]).all() and not torch.isnan(got[0, blk, 0]).any()
    assert bool((got[0, int(b.tables[1, 0])] == 9.0).all())


def scores_want(b, bounds, t):
    """Scores of row t [L][Hkv][pages] and the sum of the terms' magnitudes."""
    s, _ = b.rows[t]
    blocks = b.tables[s, :b.seen(t)]
    x = bounds[:, blocks].double().cpu().numpy()                    # [L][P][Hkv][2][d]
    q = b.q[:, t].double().cpu().numpy().reshape(b.L, 1, b.Hkv, -1, 1, b.d)
    prod = q * x[:, :, :, None]                                     # [L][P][Hkv][G][2][d]
    scale = 1 / math.sqrt(b.d)
    return (scale * prod.max(4).sum((3, 4)).swapaxes(1, 2),
            scale * np.abs(prod).max(4).sum((3, 4)).swapaxes(1, 2))


@pytest.mark.parametrize("heads,d", [((8, 2), 64), ((32, 8), 128), ((6, 2), 128), ((64, 1), 64), ((1, 1), 64)])
@pytest.mark.parametrize("bs,lens,q_lens", [
    (16, [1, 300, 17, 2500], None), (32, [100, 4500], None), (16, [40, 333, 16, 9], [17, 33, 0, 9]),
    (32, [600], [131]), (16, [5], [1])])
def test_scores(heads, d, bs, lens, q_lens):
    b = Batch(lens, q_lens, heads, d, bs, L=2, seed=3)
    bounds = b.bounds()
    got = torch.full((b.L, b.T, b.Hkv, b.MB + 5), 7.0, device="cuda")
    kvp.kvp_page_scores(b.q, b.start, bounds, b.t, b.n, b.desc, got)
    got = got.double().cpu().numpy()
    # the query sums are fp32 (G roundings), their three bf16 parts whole, the
    # products exact; 2 d / 16 accumulations of at most two units in the last
    # place each (2^-22), and a few more at the end
    eps = (heads[0] // heads[1] + 4 * 2 * d / 16 + 16) * 2.0 ** -24
    for t in range(b.T):
        want, mag = scores_want(b, bounds, t)
        n = b.seen(t)
        assert (np.abs(got[:, t, :, :n] - want) <= eps * mag).all()
        assert (got[:, t, :, n:] == 7.0).all()


def test_scores_bound_every_key():
    b = Batch([500], heads=(8, 2), d=64, seed=5)
    sc = torch.zeros(1, 1, 2, b.MB, device="cuda")
    kvp.kvp_page_scores(b.q, None, b.bounds(), b.t, b.n, b.desc, sc)
    for j in range(31):
        k = b.k[0, int(b.tables[0, j])].double()                    # [Hkv][bs][d]
        z = torch.einsum("hgd,hkd->hgk", b.q[0, 0].double().view(2, 4, 64), k).sum(1) / 8
        assert bool((z.amax(-1) <= sc[0, 0, :, j] + 1e-4).all())


def test_scores_of_bad_entries_and_padded_rows():
    b = Batch([100, 60], [3, 2], seed=6)
    bounds = b.bounds()
    b.t[0, 2], b.t[0, 3] = -1, b.NB
    q = torch.cat([b.q, b.q], 1).contiguous()                       # five rows behind the batch's
    got = torch.full((1, 10, b.Hkv, b.MB), 7.0, device="cuda")
    kvp.kvp_page_scores(q, b.start, bounds, b.t, b.n, b.desc, got)
    assert bool((got[0, :3, :, 2:4] == -math.inf).all()) and bool((got[0, 5:] == 7.0).all())
    assert bool(torch.isfinite(got[0, :5]).logical_or(got[0, :5] == -math.inf).all())


def select_want(sc, n, budget, sink, recent):
    must = set(range(min(sink, n))) | set(range(max(0, n - recent), n))
    key = np.where(np.isnan(sc[:n]), np.inf, sc[:n])
    order = np.lexsort((np.arange(n), -key, ~np.isnan(sc[:n])))
    pick = sorted((sorted(must) + [int(j) for j in order if int(j) not in must])[:budget])
    return pick + [-1] * (budget - len(pick))


def values(kind, shape, g):
    if kind == "normal":
        return g.normal(size=shape)
    if kind == "ties":
        return g.integers(-2, 3, shape).astype(np.float64) * np.where(g.random(shape) < 0.5, -1.0, 1.0)   # zeros of both signs
    if kind == "equal":
        return np.full(shape, -3.25)
    if kind == "up":        # the best ones next to each other
        return np.broadcast_to(np.arange(shape[-1]), shape).astype(np.float64)
    if kind == "close":     # neighbours in fp32
        return 1.0 + g.integers(0, 50, shape) * 2.0 ** -23
    if kind == "wide":      # a few huge ones among small ones
        return g.normal(size=shape) * 10.0 ** g.integers(-30, 30, shape)
    x = g.normal(size=shape)
    x[g.random(shape) < 0.1] = np.nan
    x[g.random(shape) < 0.1] = np.inf
    x[g.random(shape) < 0.3] = -np.inf
    return x


@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "up", "close", "wide", "odd"])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (8, 1, 2), (8, 8, 0), (8, 0, 8), (64, 4, 7),
                                               (300, 0, 1), (700, 2, 9), (2000, 1, 1)])
def test_select(kind, budget, sink, recent):
    lens = [1, 16 * 7, 16 * 9 + 1, 16 * 100, 16 * 513, 16 * 1025, 16 * 4095 + 3, 16 * 9001]
    for q_lens in (None, [1, 3, 0, 2, 1, 1, 1, 2]):
        nq = [1] * 8 if q_lens is None else q_lens
        T, MB = sum(nq), 9003
        g = np.random.default_rng(budget + sink)
        sc = values(kind, (1, T, 2, MB), g).astype(np.float32)
        desc = kvp.AttnDesc(1, 4, 2, 64, 16, 8, 0.0, 0)
        start = None if q_lens is None else torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device="cuda")
        out = torch.full((1, T + 2, 2, budget), 77, dtype=torch.int32, device="cuda")
        rows = T if q_lens is None else T + 2
        full = np.concatenate([sc, sc[:, :2]], 1)[:, :rows]
        kvp.kvp_page_select(torch.from_numpy(np.ascontiguousarray(full)).cuda(), start,
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), desc, sink, recent, out[:, :rows])
        got = out.cpu().numpy()
        t = 0
        for s in range(8):
            for i in range(nq[s]):
                n = (lens[s] - nq[s] + i) // 16 + 1 if lens[s] - nq[s] + i >= 0 else 0
                for h in range(2):
                    assert got[0, t, h].tolist() == select_want(sc[0, t, h], n, budget, sink, recent), (s, i, h, n)
                t += 1
        assert (got[0, T:] == 77).all()         # rows behind the last sequence


def test_select_reads_only_what_is_seen():
    # a NaN behind the query's pages is not chosen
    sc = torch.zeros(1, 1, 1, 40, device="cuda")
    sc[..., 10:] = math.nan
    out = torch.zeros(1, 1, 1, 4, dtype=torch.int32, device="cuda")
    kvp.kvp_page_select(sc, None, torch.tensor([160], dtype=torch.int32, device="cuda"),
                        kvp.AttnDesc(1, 1, 1, 64, 16, 8, 0.0, 0), 0, 1, out)
    assert out.flatten().tolist() == [0, 1, 2, 9]


def sparse_want(b, sel, scale=None):
    """out, lse and sum p |v| in 64 bits."""
    G = b.Hq // b.Hkv
    out = np.zeros((b.L, b.T, b.Hq, b.d))
    mag, lse = np.zeros_like(out), np.full((b.L, b.T, b.Hq), -np.inf)
    k, v = b.k.double().cpu().numpy(), b.v.double().cpu().numpy()
    q = b.q.double().cpu().numpy()
    scale = scale or 1 / math.sqrt(b.d)
    table = b.t.cpu().numpy()
    for l, t, h in np.ndindex(b.L, b.T, b.Hkv):
        s, p = b.rows[t]
        kk, vv = [], []
        for j in sel[l, t, h]:
            if 0 <= j < b.seen(t) and 0 <= table[s, j] < b.NB:
                m = min(b.bs, p + 1 - j * b.bs)
                kk.append(k[l, table[s, j], h, :m])
                vv.append(v[l, table[s, j], h, :m])
        if not kk:
            continue
        K, V = np.concatenate(kk), np.concatenate(vv)
        hq = slice(h * G, h * G + G)
        z = scale * q[l, t, hq] @ K.T
        m = z.max(1, keepdims=True)
        e = np.exp(z - m)
        lse[l, t, hq] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
        pr = e / e.sum(1, keepdims=True)
        out[l, t, hq], mag[l, t, hq] = pr @ V, pr @ np.abs(V)
    return out, lse, mag


def check_sparse(b, sel, scale=None, lse=True):
    out = torch.full_like(b.q, 5.0)
    ls = torch.full((b.L, b.T, b.Hq), 5.0, device="cuda") if lse else None
    dev = torch.from_numpy(np.ascontiguousarray(sel, np.int32)).cuda()
    kvp.paged_sparse_attention(b.q, b.start, b.k, b.v, b.t, b.n, dev, b.desc, out, ls)
    want, want_lse, mag = sparse_want(b, sel, scale)
    got = out.double().cpu().numpy()
    # out is rounded to bf16 once (2^-8); the weights keep 16 bits (2^-17), and
    # a score of magnitude 8 in fp32 and the exponential's argument are off by
    # at most 2^-18 or so, which doubles in a normalised weight: 2^-12 of sum p
    # |v| leaves room
    # (a NaN that a row sees shows in it.  An infinite value meets the weight's
    # two parts one by one: the second is 0 or of either sign, 0 * inf is NaN and
    # inf - inf too, so that the result is an infinity or a NaN)
    assert np.array_equal(np.isfinite(got), np.isfinite(want)) and np.isnan(got)[np.isnan(want)].all()
    ok = np.isfinite(want)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mag)[ok].all()
    if lse:
        g = ls.double().cpu().numpy()
        assert np.array_equal(np.isneginf(g), np.isneginf(want_lse)) and np.array_equal(np.isnan(g), np.isnan(want_lse))
        ok = np.isfinite(want_lse)
        # a score's rounding (2^-18 or so) and lse's own to fp32
        assert (np.abs(g - want_lse)[ok] <= 2.0 ** -15 + 2.0 ** -22 * np.abs(want_lse[ok])).all()
    return out, ls


def some_pages(b, budget, seed=0, fill=0.8):
    g = np.random.default_rng(seed)
    sel = np.full((b.L, b.T, b.Hkv, budget), -1, np.int32)
    for l, t, h in np.ndindex(b.L, b.T, b.Hkv):
        n = b.seen(t)
        m = min(n, max(0, int(round(budget * fill))))
        pick = g.permutation(n)[:m]
        sel[l, t, h, :m] = np.sort(pick) if (t + h) % 2 else pick
        if m and (t + h) % 3 == 0:
            sel[l, t, h, 0] = n - 1         # the query's own page
        sel[l, t, h] = np.where(np.isin(np.arange(budget), g.permutation(budget)[:m]), -1, sel[l, t, h]) \
            if (t + h) % 5 == 0 else sel[l, t, h]
    return sel


@pytest.mark.parametrize("heads,d", [((32, 4), 64), ((32, 8), 128), ((1, 1), 64), ((6, 2), 128), ((12, 1), 64), ((16, 1), 128),
                                     ((40, 2), 128), ((64, 1), 64)])
@pytest.mark.parametrize("bs,lens,q_lens,budget", [
    (16, [1, 300, 17, 2000], None, 16), (32, [100, 1500], None, 9), (16, [2500], None, 150), (64, [640, 63], None, 3),
    (16, [40, 333, 16, 9], [17, 5, 0, 9], 6), (16, [90], [1], 1)])
def test_sparse(heads, d, bs, lens, q_lens, budget):
    b = Batch(lens, q_lens, heads, d, bs, L=2, seed=8)
    check_sparse(b, some_pages(b, budget))


def test_sparse_equals_decode_over_all_pages():
    b = Batch([1000, 333], heads=(32, 8), d=128, seed=9)
    sel = np.full((1, 2, 8, b.MB), -1, np.int32)
    for s, n in enumerate(b.lens):
        sel[:, s, :, :-(-n // 16)] = np.arange(-(-n // 16))
    out, lse = check_sparse(b, sel)
    o2, l2 = torch.empty_like(b.q), torch.empty(1, 2, 32, device="cuda")
    b.k.nan_to_num_(0, 0, 0), b.v.nan_to_num_(0, 0, 0)
    t = np.where(b.tables < 0, 0, b.tables)
    ws = torch.empty(kvp.kvp_decode_workspace_size(b.desc, t, b.lens), dtype=torch.uint8, device="cuda")
    kvp.paged_decode_attention(b.q, b.k, b.v, t, b.lens, b.desc, o2, l2, ws)
    assert float((out.float() - o2.float()).abs().max()) <= 2e-2 and float((lse - l2).abs().max()) <= 1e-3


def test_sparse_rows_without_keys_and_wrong_entries():
    b = Batch([100, 60, 0, 33], seed=10)
    sel = np.full((1, 4, 2, 7), -1, np.int32)
    sel[0, 0, 0] = [-1, 99, 2 ** 31 - 1, -2 ** 31, 7, 3, 3]         # 7 pages (0..6) are seen; page 3 twice
    sel[0, 1, :, 2] = 1
    sel[0, 2] = 0                                                   # an empty sequence
    b.t[0, 3] = 5
    sel[0, 3] = [0, 1, 2, 0, 1, 2, 2]
    b.t[3, 1] = b.NB + 3                                            # its second page is no block
    b.t[3, 0] = -4
    out, lse = check_sparse(b, sel)
    assert bool((out[0, 0, 4:] == 0).all()) and bool((lse[0, 0, 4:] == -math.inf).all())
    assert bool((out[0, 2] == 0).all())


def test_sparse_padded_rows_and_no_lse():
    b = Batch([100, 60], [3, 2], seed=11)
    q = torch.cat([b.q, b.q], 1).contiguous()
    sel = torch.zeros(1, 10, 2, 2, dtype=torch.int32, device="cuda")
    sel[..., 1] = -1
    out = torch.full_like(q, 5.0)
    kvp.paged_sparse_attention(q, b.start, b.k, b.v, b.t, b.n, sel, b.desc, out, None)
    assert bool((out[0, 5:] == 5.0).all()) and not bool((out[0, :5] == 5.0).any())


def test_sparse_scores_that_grow_and_peak():
    # every page raises the maximum; then one key holds all the weight
    b = Batch([320], heads=(8, 2), d=64, seed=12, poison=False)
    for j in range(20):
        b.k[0, int(b.tables[0, j])] = b.q[0, 0].view(2, 4, 1, 64)[:, 0] * (j / 4)
    sel = np.arange(20, dtype=np.int32)[None, None, None].repeat(2, 2)
    out = torch.empty_like(b.q)
    lse = torch.empty(1, 1, 8, device="cuda")
    kvp.paged_sparse_attention(b.q, None, b.k, b.v, b.t, b.n, torch.from_numpy(sel).cuda(), b.desc, out, lse)
    want, wl, mag = sparse_want(b, sel)
    # scores up to about 40: fp32 rounding of those reaches 2^-16
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mag).all()
    assert np.abs(lse.double().cpu().numpy() - wl).max() <= 2.0 ** -14


def test_sparse_same_bits_and_scale():
    b = Batch([3000], heads=(32, 4), d=64, seed=13)
    b.desc = kvp.AttnDesc(1, 32, 4, 64, 16, b.NB, 0.25, 0)
    sel = some_pages(b, 100)
    x = check_sparse(b, sel, 0.25)
    y = check_sparse(b, sel, 0.25)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_captured_calls_follow_tables_and_lengths():
    b = Batch([200, 90], heads=(8, 2), d=64, seed=14, poison=False)
    bounds = b.bounds()
    sc = torch.zeros(1, 2, 2, b.MB, device="cuda")
    sel = torch.zeros(1, 2, 2, 4, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(b.q), torch.empty(1, 2, 8, device="cuda")

    def step():
        kvp.kvp_page_bounds(b.k, b.t, b.n, 1, b.desc, bounds)
        kvp.kvp_page_scores(b.q, None, bounds, b.t, b.n, b.desc, sc)
        kvp.kvp_page_select(sc, None, b.n, b.desc, 1, 1, sel)
        kvp.paged_sparse_attention(b.q, None, b.k, b.v, b.t, b.n, sel, b.desc, out, lse)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in ([200, 90], [150, 17], [31, 64]):
        b.n.copy_(torch.tensor(n, dtype=torch.int32))
        b.q.normal_()
        g.replay()
        got = [x.clone() for x in (bounds, sel, out, lse)]
        step()
        for x, y in zip(got, (bounds, sel, out, lse)):
            assert torch.equal(x, y)
        b.lens, b.rows = n, [(s, n[s] - 1) for s in range(2)]
        want, wl, mag = sparse_want(b, sel.cpu().numpy())
        assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mag).all()


def test_two_streams_at_once():
    b = [Batch([700 + 100 * i], heads=(8, 2), d=64, seed=15 + i) for i in range(2)]
    sel = [some_pages(x, 20) for x in b]
    dev = [torch.from_numpy(s).cuda() for s in sel]
    outs = [torch.empty_like(x.q) for x in b]
    st = [torch.cuda.Stream() for _ in b]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, s, o, e in zip(b, dev, outs, st):
            kvp.paged_sparse_attention(x.q, None, x.k, x.v, x.t, x.n, s, x.desc, o, None, stream=e)
    torch.cuda.synchronize()
    for x, s, o in zip(b, sel, outs):
        want, _, mag = sparse_want(x, s)
        assert (np.abs(o.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mag).all()


def test_wrong_tensors_are_refused():
    b = Batch([100, 60])
    sel = torch.zeros(1, 2, 2, 4, dtype=torch.int32, device="cuda")
    call = lambda **kw: kvp.paged_sparse_attention(*{**dict(q=b.q, qs=None, k=b.k, v=b.v, t=b.t, n=b.n, s=sel, d=b.desc,
                                                           o=torch.empty_like(b.q), l=None), **kw}.values())
    call()
    for bad in (dict(q=b.q.float()), dict(k=b.k[:, :-1].contiguous()), dict(t=b.t.long()), dict(n=b.n.cpu()),
                dict(s=sel[:, :1].contiguous()), dict(s=sel.float()), dict(qs=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(o=torch.empty(1, 2, 8, 128, device="cuda", dtype=torch.bfloat16)), dict(t=b.t[:, ::2]),
                dict(l=torch.empty(1, 2, 4, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)


CHUNKS = [((8, 2), 64, 16, [300, 350], [280, 260]), ((8, 2), 128, 32, [1000, 9], [306, 3]),
          ((8, 1), 128, 16, [700], [650]), ((16, 4), 64, 16, [90, 400], [90, 88]), ((4, 4), 64, 16, [2000], [640]),
          ((6, 2), 128, 16, [500], [480]), ((5, 1), 64, 64, [950], [930]), ((16, 8), 128, 16, [340, 60, 200], [300, 1, 77])]


def like_neighbours(b, budget, seed=1):
    """Every 13 rows choose from one set of pages, with the newest and a few of
    their own; ascending as kvp_page_select leaves them."""
    g = np.random.default_rng(seed)
    sel = np.full((b.L, b.T, b.Hkv, budget), -1, np.int32)
    for l, h in np.ndindex(b.L, b.Hkv):
        for t in range(b.T):
            n = b.seen(t)
            if t % 13 == 0 or b.rows[t][0] != b.rows[t - 1][0]:
                common = g.permutation(n)[:budget]
            pick = np.unique(np.concatenate([common, [n - 1], g.integers(0, n, 3)]))
            pick = g.permutation(pick)[:min(budget, n)]
            sel[l, t, h, :len(pick)] = np.sort(pick)
    return sel


@pytest.mark.parametrize("heads,d,bs,lens,q_lens", CHUNKS)
def test_chunks(heads, d, bs, lens, q_lens):
    b = Batch(lens, q_lens, heads, d, bs, L=2, seed=20)
    x = check_sparse(b, like_neighbours(b, 9))
    y = check_sparse(b, like_neighbours(b, 9))
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    check_sparse(b, some_pages(b, 7))           # no order, nothing in common, entries of -1


@pytest.mark.parametrize("heads,d,bs,lens,q_lens", CHUNKS[:3])
def test_chunks_with_a_page_twice(heads, d, bs, lens, q_lens):
    b = Batch(lens, q_lens, heads, d, bs, L=2, seed=21)
    sel = like_neighbours(b, 9)
    sel[:, 5, 0, 3] = sel[:, 5, 0, 2]
    sel[1, 40] = 0                              # nine times
    sel[0, 50] = -1                             # none at all
    sel[0, 51, 0] = [-3, 2 ** 31 - 1, -2 ** 31, 5000, 20000, -1, 16384, 1 << 24, 0]
    check_sparse(b, sel)


def test_chunks_with_values_that_some_rows_do_not_see():
    b = Batch([400], [380], (8, 2), 64, 16, L=2, seed=22, poison=False)
    sel = like_neighbours(b, 6)
    for l in range(2):
        sel[l, 100:200, 0] = np.array([0, 1, 2, 3, 4, -1])
        sel[l, 120, 0] = [0, 1, 2, 3, 5, -1]    # one row alone names page 5, which holds a NaN
        sel[l, 150:153, 0, 4] = -1
    b.v[:, int(b.tables[0, 5]), 0, 3, 7] = math.nan
    b.k[:, int(b.tables[0, 4]), 0, 1, 1] = math.nan
    b.v[0, int(b.tables[0, 4]), 0, 2] = math.inf
    sel[:, 300:, 0] = np.array([0, 1, 2, 3, 19, 20])
    b.v[:, int(b.tables[0, 20]), 0, 5] = -math.inf      # token 325: seen from row 305 on
    check_sparse(b, sel)


def test_chunks_of_padded_rows_and_short_sequences():
    # more queries than tokens: the first rows have no position
    b = Batch([400, 10], [300, 40], (8, 2), 64, 16, L=2, seed=23)
    q = torch.cat([b.q, b.q[:, :9]], 1).contiguous()
    sel = np.zeros((2, 349, 2, 3), np.int32)
    sel[..., 1], sel[..., 2] = 2, -1
    out = torch.full_like(q, 5.0)
    lse = torch.full((2, 349, 8), 5.0, device="cuda")
    kvp.paged_sparse_attention(q, b.start, b.k, b.v, b.t, b.n, torch.from_numpy(sel).cuda(), b.desc, out, lse)
    assert bool((out[:, 340:] == 5.0).all()) and bool((lse[:, 340:] == 5.0).all())
    assert bool((out[:, 300:330] == 0).all()) and bool((lse[:, 300:330] == -math.inf).all())
    want, wl, mag = sparse_want(b, sel[:, :340])
    got = out[:, :340].double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mag).all()


# shapes whose tiles hold more than 16 (query, head) rows
WIDE = [((32, 8), 128, 32, [1000, 77, 600], [333, 1, 316]), ((16, 4), 64, 16, [400], [330]),
        ((24, 2), 128, 16, [300], [170]), ((16, 2), 64, 64, [2000, 90], [290, 60]), ((10, 2), 128, 16, [520], [470])]


@pytest.mark.parametrize("heads,d,bs,lens,q_lens", WIDE)
def test_wide_chunks(heads, d, bs, lens, q_lens):
    b = Batch(lens, q_lens, heads, d, bs, L=2, seed=24)
    sel = like_neighbours(b, 9)
    x = check_sparse(b, sel)
    y = check_sparse(b, sel)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    check_sparse(b, some_pages(b, 7))


@pytest.mark.parametrize("heads,d,bs,lens,q_lens", WIDE)
def test_wide_chunks_with_repeated_and_unseen(heads, d, bs, lens, q_lens):
    b = Batch(lens, q_lens, heads, d, bs, L=2, seed=25)
    sel = like_neighbours(b, 9)
    sel[:, 5, 0, 3] = sel[:, 5, 0, 2]
    sel[1, 40] = 0
    sel[0, 50] = -1
    sel[0, 51, 0] = [-3, 2 ** 31 - 1, -2 ** 31, 5000, 20000, -1, 4096, 1 << 24, 0]
    # a page that one row of its tile names holds a NaN and an infinite value
    sel[:, 64:96, 1] = -1
    sel[:, 64:96, 1, 0] = 0
    sel[:, 70, 1, 1] = 1
    b.v[:, int(b.tables[0, 1]), 1, 2, 3] = math.nan
    b.v[:, int(b.tables[0, 1]), 1, 4] = math.inf
    check_sparse(b, sel)


# tiles of the tensor-core kernel: groups that fill 128 rows and that do not, rows
# of several tiles, pages from 16 tokens to more than a step's 128, steps that end
# inside a page, budgets above a warp's lanes
LARGE = [((64, 1), 128, 16, [900], [640], 9), ((40, 1), 64, 32, [1500, 3000], [700, 640], 5),
         ((16, 8), 64, 128, [1000, 40, 900], [150, 0, 75], 4), ((8, 8), 128, 256, [2000], [97], 3),
         ((12, 4), 128, 1024, [1500, 2049], [33, 180], 2), ((32, 8), 64, 16, [1200], [160], 40),
         ((7, 1), 128, 64, [4000], [641], 6), ((4, 2), 128, 16, [330], [330], 33)]


@pytest.mark.parametrize("heads,d,bs,lens,q_lens,budget", LARGE)
def test_large_tiles(heads, d, bs, lens, q_lens, budget):
    b = Batch(lens, q_lens, heads, d, bs, seed=30)
    sel = like_neighbours(b, budget)
    x = check_sparse(b, sel)
    y = check_sparse(b, sel)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    sel = sel[:, :, :, g_perm(budget)]          # no order
    sel[:, 3:40] = -1                           # a tile's rows without keys, then a whole tile's
    sel[:, 64:130, 0] = -1
    check_sparse(b, sel, lse=False)


def g_perm(n):
    return np.random.default_rng(n).permutation(n)


@pytest.mark.parametrize("heads,d,bs,lens,q_lens,budget", LARGE)
def test_large_tiles_with_repeated_and_unseen(heads, d, bs, lens, q_lens, budget):
    b = Batch(lens, q_lens, heads, d, bs, seed=31)
    sel = like_neighbours(b, budget)
    sel[:, 5, 0, -1] = sel[:, 5, 0, 0]          # twice
    h = b.Hkv - 1
    sel[:, 32:64, h] = -1
    sel[:, 32:64, h, 0] = 0
    sel[:, 40, h, 1] = 1                        # one row of its tile names page 1
    b.v[:, int(b.tables[0, 1]), h, 2, 3] = math.nan
    b.k[:, int(b.tables[0, 1]), h, 4, 1] = math.inf
    check_sparse(b, sel)


def test_large_tiles_whose_scores_grow():
    # every page's scores are above those before it, by far more than the
    # reference's slack, and fall again: both chains raise theirs and are joined
    b = Batch([2000], [80], (16, 8), 128, 16, seed=32, poison=False)
    rise = torch.linspace(-1, 1, 125, device="cuda")
    rise = torch.where(rise > 0.6, -rise, rise)
    unit = b.q[:, :, ::2].float().mean(1)                                   # [L][Hkv][d]
    for j in range(125):
        blk = int(b.tables[0, j])
        b.k[:, blk] = (b.k[:, blk].float() * 0.1 + 30 * rise[j] * unit[:, :, None] / unit.norm(dim=-1)[:, :, None, None]).bfloat16()
    b.q[:] = (b.q.float() * 0.2 + unit.repeat_interleave(2, 1)[:, None] / unit.norm() * 5).bfloat16()
    sel = np.broadcast_to(np.arange(0, 120, 2, dtype=np.int32), (1, 80, 8, 60)).copy()
    check_sparse(b, sel)


def test_large_tiles_far_in_a_long_table():
    b = Batch([65000], [100], (8, 8), 128, 16, seed=33)
    sel = np.broadcast_to(np.array([4062, 0, 2047, 2048, 3999, 1, 4061], np.int32), (1, 100, 8, 7)).copy()
    check_sparse(b, sel)
    wide = torch.full((1, 4096), -1, dtype=torch.int32, device="cuda")      # the widest table, and one more
    wide[:, :b.MB] = b.t
    for more in (0, 1):
        b.t = torch.cat([wide, wide[:, :more]], 1).contiguous()
        check_sparse(b, sel)


# a few rows each of many sequences: tiles of 32 and of 16 (query, head) rows
@pytest.mark.parametrize("heads,d,bs,S", [((16, 4), 128, 16, 120), ((16, 2), 64, 32, 230), ((8, 4), 128, 16, 130),
                                          ((4, 4), 64, 16, 200)])
def test_few_rows_of_many_sequences(heads, d, bs, S):
    g = np.random.default_rng(S)
    q_lens = g.integers(3, 6, S)
    b = Batch([int(n) for n in g.integers(5, 180, S)], [int(n) for n in q_lens], heads, d, bs, L=3, seed=34)
    assert b.T < 5 * S
    sel = like_neighbours(b, 5)
    x = check_sparse(b, sel)
    y = check_sparse(b, sel)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    sel = some_pages(b, 4)
    sel[0, 11] = 0                              # a page four times
    sel[:, 20:30, 1] = -1
    sel[:, 20:30, 1, 0] = 0
    sel[:, 23, 1, 1] = 1
    s = b.rows[23][0]
    if b.tables[s, 1] >= 0:
        b.v[:, int(b.tables[s, 1]), 1, 0, 5] = math.nan
    check_sparse(b, sel)


def test_large_tiles_captured_twice_and_on_two_streams():
    b = Batch([500, 700], [300, 200], (8, 2), 128, 16, seed=35)
    sel = torch.from_numpy(like_neighbours(b, 6)).cuda()
    want = torch.empty_like(b.q)
    kvp.paged_sparse_attention(b.q, b.start, b.k, b.v, b.t, b.n, sel, b.desc, want, None)
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        outs.append(torch.zeros_like(b.q))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for _ in range(3):
                kvp.paged_sparse_attention(b.q, b.start, b.k, b.v, b.t, b.n, sel, b.desc, outs[-1], None)
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    b.n -= 17                                   # a graph follows the lengths: their pages' ends, rows without a position
    b.lens = [n - 17 for n in b.lens]
    b.rows = [(s, p - 17) for s, p in b.rows]
    graphs[0].replay()
    torch.cuda.synchronize()
    out, _, mag = sparse_want(b, sel.cpu().numpy())
    got = outs[0].double().cpu().numpy()
    assert (np.abs(got - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -12 * mag).all()
