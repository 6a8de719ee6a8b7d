"""Cases that measure four operators over the paged KV pool: sliding-window
attention with sink tokens, accumulated attention weight per cached token,
eviction by that weight, and verification of drafted tokens.

`own` false runs the operators in plain torch operations (32-bit, or 64-bit
where a comparison or a long sum decides a token); `own` true makes the calls
of the package.  Pools are bf16 with scattered blocks; K, V and Q ~ N(0, 1).
"""
import math

import numpy as np
import torch

own = False

# head shapes of the repository's workloads
HEADS = {"64": (32, 4, 64), "128": (32, 8, 128)}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one agent's next token over a short window: latency
        dict(name="window_decode_1", op="window", heads="64", bs=16, L=1, S=1, q=1, len=4100, win=1024, sinks=4),
        # a serving batch's decode step, several layers, mixed lengths
        dict(name="window_decode_64", op="window", heads="128", bs=16, L=4, S=64, q=1, len=12000, win=4096, sinks=4),
        # chunked prefill of a mixed batch, odd window, 32-token pages
        dict(name="window_extend", op="window", heads="64", bs=32, L=2, S=5, q=777, len=3001, win=1000, sinks=3),
        # a long document's prefill chunk
        dict(name="window_prefill", op="window", heads="128", bs=16, L=1, S=1, q=8192, len=16384, win=4096, sinks=16),
        # one sequence's running weights after its decode step
        dict(name="mass_decode_1", op="mass", heads="64", bs=16, L=1, S=1, q=1, len=1500),
        # a batch's running weights after a decode step over long caches
        dict(name="mass_decode_32", op="mass", heads="128", bs=16, L=2, S=32, q=1, len=12000),
        # the weights that a prompt's last tokens give the whole prompt
        dict(name="mass_prompt", op="mass", heads="128", bs=32, L=1, S=2, q=64, len=8191),
        # one branch pruned to a quarter
        dict(name="evict_1", op="evict", heads="64", bs=16, L=1, S=1, len=1023, budget=256, sink=4, recent=64),
        # eight branches of a long context pruned at once, several layers
        dict(name="evict_8", op="evict", heads="128", bs=16, L=4, S=8, len=16000, budget=4096, sink=4, recent=512),
        # one chain of drafts
        dict(name="verify_chain_1", op="verify", B=1, n=5, vocab=32000, tree=False, draft=True),
        # full draft trees, vocabulary rows of odd length
        dict(name="verify_tree_8", op="verify", B=8, n=64, vocab=32003, tree=True, draft=True),
        # a batch of chains over a large vocabulary
        dict(name="verify_chain_64", op="verify", B=64, n=7, vocab=131072, tree=False, draft=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "mass", "evict", "verify"])
    c = dict(op=op)
    if op in ("window", "mass", "evict"):
        c.update(heads=rng.choice(["64", "128"]), bs=rng.choice([16, 32]), L=rng.randint(1, 4))
    if op == "window":
        if rng.random() < 0.5:   # decode
            c.update(S=_log(rng, 1, 64), q=1, len=_log(rng, 20, 12000), win=_log(rng, 16, 4096))
        else:                    # extend
            c.update(S=_log(rng, 1, 8), q=_log(rng, 2, 1500), win=_log(rng, 16, 4096))
            c.update(len=c["q"] + _log(rng, 1, 6000), L=1)
        c.update(sinks=rng.choice([0, 1, 4, 17, 100]))
    elif op == "mass":
        c.update(S=_log(rng, 1, 32), q=rng.choice([1, 1, 5, 33]), len=_log(rng, 40, 12000), L=rng.randint(1, 2))
    elif op == "evict":
        n = _log(rng, 100, 16000)
        keep = max(40, int(n * rng.uniform(0.1, 0.9)))
        c.update(S=_log(rng, 1, 8), len=n, budget=keep, sink=rng.choice([0, 4, 19]), recent=rng.randint(0, keep // 3))
    else:
        n = _log(rng, 1, 64)
        c.update(B=_log(rng, 1, 64), n=n, tree=rng.random() < 0.5, draft=rng.random() < 0.7)
        c.update(vocab=min(_log(rng, 500, 131072), 60_000_000 // (c["B"] * (n + 1))))
    return c


# ------------------------------------------------------------------ inputs

def _lens(c):
    """Cached tokens and query tokens of each sequence, the case's alone (they
    set the outputs' shapes): the first has the case's own, the others down to
    half of them."""
    g = np.random.Generator(np.random.Philox(key=[c["len"], c["S"]]))
    f = g.uniform(0.5, 1.0, c["S"])
    f[0] = 1.0
    q = np.maximum(1, (c.get("q", 1) * f).astype(np.int32)).astype(np.int32)
    if c.get("q", 1) > 64 and c["S"] > 2:
        q[1], q[2] = 1, 17      # a decoding sequence and a short chunk ride along
    n = np.maximum(q, (c["len"] * f).astype(np.int32)).astype(np.int32)
    return n, q


def _shuffled(nb, seed):
    """The pool's allocation order for alloc_seed `seed`."""
    a, s, m = list(range(nb)), seed, (1 << 64) - 1
    for i in range(nb - 1, 0, -1):
        s = (s + 0x9E3779B97F4A7C15) & m
        z = ((s ^ (s >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        j = (z ^ (z >> 31)) % (i + 1)
        a[i], a[j] = a[j], a[i]
    return np.array(a, np.int32)


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _tables(n, bs, order):
    """Block tables [S][MB]: sequence after sequence takes `order`'s blocks."""
    nb = (n + bs - 1) // bs
    t = np.full((len(n), int(nb.max())), -1, np.int32)
    at = 0
    for s, k in enumerate(nb):
        t[s, :k] = order[at:at + k]
        at += k
    return t, at


def _slots(tables, bs, width, device="cuda"):
    """Pool slot (block * bs + offset) of token positions 0 .. width-1; the
    positions past a sequence's table give slot 0."""
    t = torch.from_numpy(tables.astype(np.int64)).to(device).clamp_(min=0)
    pos = torch.arange(width, device=device)
    blk = (pos // bs).clamp_(max=t.shape[1] - 1)
    return t[:, blk] * bs + pos % bs


class _Pool:
    """A pool handle that goes with its state."""

    def __init__(self, kvp, handle):
        self.kvp, self.handle = kvp, handle

    def __del__(self):
        self.kvp.kv_pool_destroy(self.handle)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    st = dict(c=c)
    if own:
        import paged_prefix_shared_decode_gb300 as kvp
        st["kvp"] = kvp
    if c["op"] == "verify":
        return _prepare_verify(c, seed, gen, st)
    Hq, Hkv, d = HEADS[c["heads"]]
    n, nq = _lens(c)
    bs, L, S = c["bs"], c["L"], c["S"]
    nb = (n + bs - 1) // bs
    extra = S * -(-c["budget"] // bs) if c["op"] == "evict" else 0
    NB = int(nb.sum()) + extra
    order = _shuffled(NB, 1 + seed)
    tables, used = _tables(n, bs, order)
    st.update(Hq=Hq, Hkv=Hkv, d=d, n=n, nq=nq, NB=NB, tables=tables,
              slots=_slots(tables, bs, int(n.max())), lens=torch.from_numpy(n.astype(np.int64)).cuda())
    st["k"] = _normal(gen, L, NB, Hkv, bs, d)
    if c["op"] != "mass":
        st["v"] = _normal(gen, L, NB, Hkv, bs, d)
    if c["op"] != "evict":
        T = int(nq.sum())
        st["q"] = _normal(gen, L, T, Hq, d)
        first = np.concatenate([[0], np.cumsum(nq)[:-1]])
        seq = np.repeat(np.arange(S), nq)
        col = np.arange(T) - first[seq]
        st["seq"], st["col"] = torch.from_numpy(seq).cuda(), torch.from_numpy(col).cuda()
        st["pos"] = torch.from_numpy((n - nq)[seq] + col).cuda()
    if own:
        st["desc"] = kvp.AttnDesc(L, Hq, Hkv, d, bs, NB, 0.0, 1, kvp.KVP_KV_BF16)
    stride = int(n.max()) + 5
    if c["op"] == "window":
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(L, T, Hq, device="cuda")
        if own:
            need = kvp.kvp_window_workspace_size(st["desc"], tables, n, nq, c["win"], c["sinks"])
            st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    elif c["op"] == "mass":
        st["decay"] = 0.95
        # tokens appended since the weights were last updated start at zero
        st["prev"] = n - nq
        st["mass"] = torch.rand(L, S, Hkv, stride, generator=gen, device="cuda") * 4
        st["mass_out"] = torch.zeros_like(st["mass"])
        s = _scores(st, _padded_q(st), _dense(st, "k", st["slots"]), torch.float32)
        seen = _seen(st)
        lse = torch.logsumexp(s.masked_fill(~seen, -math.inf), -1)      # [L][S][Hkv][G][nq]
        st["lse"] = _rows(st, lse).contiguous()
        if own:
            need = kvp.kvp_mass_workspace_size(st["desc"], tables, n, nq)
            st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    else:
        # weights as sums of softmax rows leave them: a few heavy tokens, a
        # long tail, and tokens that tie
        m = torch.empty(L, S, Hkv, stride, device="cuda").exponential_(1.0, generator=gen) ** 3
        st["mass"] = torch.where(m < 0.05, torch.round(m * 100) / 100, m)
        st["mass_out"] = torch.zeros_like(m)
        st["kept"] = torch.zeros(L, S, Hkv, c["budget"], dtype=torch.int32, device="cuda")
        # the evicted sequences' tables: a page that holds sink tokens alone
        # stays shared with the parent, every other one is fresh
        keep = np.minimum(n, c["budget"])
        dst = np.full((S, max(1, int(-(-keep // bs).max()))), -1, np.int32)
        at = used
        for s in range(S):
            for j in range(-(-int(keep[s]) // bs)):
                if n[s] <= c["budget"] or (j + 1) * bs <= c["sink"]:
                    dst[s, j] = tables[s, j]
                else:
                    dst[s, j] = order[at]
                    at += 1
        st["dst"] = _slots(dst, bs, c["budget"])
        if own:
            h = kvp.kv_pool_create(kvp.PoolDesc(L, NB, bs, Hkv, d, 2 * S, tables.shape[1], 1 + seed), st["k"], st["v"])
            st["pool"] = _Pool(kvp, h)
            st["parents"] = []
            for s in range(S):
                i = kvp.seq_alloc(h)
                kvp.seq_reserve(h, i, int(n[s]))
                st["parents"].append(i)
            need = kvp.seq_evict_workspace_size(h, st["parents"], c["budget"])
            st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return st


def _prepare_verify(c, seed, gen, st):
    B, n, V = c["B"], c["n"], c["vocab"]
    g = np.random.Generator(np.random.Philox(key=[seed, 13]))
    if c["tree"]:   # random parents, the first nodes at the root
        par = np.array([[int(g.integers(-1, max(0, i - 1))) if i else -1 for i in range(n)] for _ in range(B)], np.int32)
    else:
        par = np.broadcast_to(np.arange(-1, n - 1, dtype=np.int32), (B, n)).copy()
    x = _normal(gen, B, n + 1, V, dtype=torch.float32) * 2.5
    st["target"] = torch.softmax(x, -1)
    # the draft model: close to the target
    q = torch.softmax(x + 0.6 * _normal(gen, B, n + 1, V, dtype=torch.float32), -1)
    row = torch.from_numpy(par.astype(np.int64)).cuda() + 1
    b = torch.arange(B, device="cuda")[:, None]
    st["tokens"] = torch.multinomial(q[b, row].view(B * n, V), 1, generator=gen).view(B, n).int()
    st["draft"] = q if c["draft"] else None
    st["parent"] = torch.from_numpy(par).cuda()
    st["u"] = torch.rand(B, n, generator=gen, device="cuda")
    st["u_next"] = torch.rand(B, generator=gen, device="cuda")
    for k in ("accepted", "count", "next"):
        st[k] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------- plain forms

def _dense(st, name, slots):
    """Rows of a pool at slots [S][N], in 32 bits: [L][S][Hkv][N][d]."""
    p = st[name]
    L, NB, Hkv, bs, d = p.shape
    rows = p[:, slots // bs, :, slots % bs]            # [S][N][L][Hkv][d]
    return rows.permute(2, 0, 3, 1, 4).float()


def _padded_q(st):
    """Queries as [L][S][Hkv][G][most queries][d], in 32 bits; padding is 0."""
    q = st["q"].float()
    L, T, Hq, d = q.shape
    p = q.new_zeros(L, len(st["n"]), int(st["nq"].max()), Hq, d)
    p[:, st["seq"], st["col"]] = q
    return p.view(*p.shape[:3], st["Hkv"], Hq // st["Hkv"], d).permute(0, 1, 3, 4, 2, 5)


def _rows(st, x):
    """Back from [L][S][Hkv][G][queries] (and values) to [L][T][Hq]."""
    x = x.permute(0, 1, 4, 2, 3, *range(5, x.dim()))
    x = x.reshape(*x.shape[:3], -1, *x.shape[5:])
    return x[:, st["seq"], st["col"]]


def _scores(st, q, k, dtype):
    L, S, Hkv, G, N, d = q.shape
    s = q.reshape(L, S, Hkv, G * N, d).to(dtype) @ k.to(dtype).transpose(-1, -2)
    return s.view(L, S, Hkv, G, N, -1) * (1.0 / math.sqrt(d))


def _seen(st):
    """Keys that a query sees: those at or before its position."""
    n, nq = st["lens"], torch.from_numpy(st["nq"].astype(np.int64)).cuda()
    pos = (n - nq)[:, None] + torch.arange(int(nq.max()), device="cuda")        # [S][queries]
    j = torch.arange(int(n.max()), device="cuda")
    return ((j <= pos[..., None]) & (j < n[:, None, None]))[:, None, None]


def _window(st):
    c = st["c"]
    W, sinks = c["win"], c["sinks"]
    n = st["lens"]
    nq = torch.from_numpy(st["nq"].astype(np.int64)).cuda()
    # the sinks, then every position some query's window reaches
    width = min(W - 1, int(st["n"].max())) + int(st["nq"].max())
    lo = (n - nq - W + 1).clamp(min=sinks)
    j = torch.cat([torch.arange(sinks, device="cuda").expand(len(n), -1),
                   lo[:, None] + torch.arange(width, device="cuda")], 1)        # [S][keys]
    slots = st["slots"].gather(1, j.clamp(max=st["slots"].shape[1] - 1))
    s = _scores(st, _padded_q(st), _dense(st, "k", slots), torch.float32)
    pos = (n - nq)[:, None, None] + torch.arange(s.shape[4], device="cuda")[:, None]
    jj = j[:, None]
    see = (jj <= pos) & (jj < n[:, None, None]) & ((jj > pos - W) | (jj < sinks))
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    # a padded query past its sequence sees the last keys or none; it is dropped
    e = torch.exp(s - m.clamp(min=-1e30))
    del s
    l = e.sum(-1, keepdim=True)
    L, S, Hkv, G, N, K = e.shape
    o = (e.view(L, S, Hkv, G * N, K) @ _dense(st, "v", slots)).view(L, S, Hkv, G, N, -1) / l
    lse = (m + torch.log(l)).squeeze(-1)
    return dict(out=_rows(st, o).to(torch.bfloat16), lse=_rows(st, lse))


def _mass(st):
    s = _scores(st, _padded_q(st), _dense(st, "k", st["slots"]), torch.float32)
    L, S, Hkv, G, N, K = s.shape
    lse = s.new_full((L, S, N, Hkv * G), math.inf)         # a padded query gives exp(-inf)
    lse[:, st["seq"], st["col"]] = st["lse"]
    lse = lse.view(L, S, N, Hkv, G).permute(0, 1, 3, 4, 2)
    p = torch.where(_seen(st), torch.exp(s - lse[..., None]), s.new_zeros(())).sum((3, 4))      # [L][S][Hkv][K]
    j = torch.arange(K, device="cuda")
    prev = torch.from_numpy(st["prev"].astype(np.int64)).cuda()[:, None, None]
    old = torch.where(j < prev, st["mass"][..., :K] * st["decay"], p.new_zeros(()))
    out = st["mass_out"]
    out[..., :K] = torch.where(j < st["lens"][:, None, None], old + p, out[..., :K])
    return dict(mass=out)


def _evict(st):
    c = st["c"]
    L, S, Hkv, stride = st["mass"].shape
    n, budget = st["lens"][:, None], c["budget"]
    j = torch.arange(stride, device="cuda")
    # sinks and recent tokens before every other, tokens past the end after
    rank = torch.where((j < c["sink"]) | (j >= n - c["recent"]), math.inf, 0.0)
    w = st["mass"] + rank[:, None]
    w.masked_fill_((j >= n)[:, None], -math.inf)
    by = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.sort(by, dim=-1).values
    have = torch.arange(budget, device="cuda") < n.clamp(max=budget)         # [S][budget]
    kept = torch.where(have[:, None], kept, -1)
    st["kept"].copy_(kept)
    at = kept.clamp(min=0)
    torch.where(have[:, None], st["mass"].gather(-1, at), st["mass_out"][..., :budget],
                out=st["mass_out"][..., :budget])
    bs = c["bs"]
    src = st["slots"][:, None].expand(L, S, Hkv, -1).gather(-1, at)
    dst = st["dst"][:, None].expand(L, S, Hkv, -1)
    # sequences that fit the budget keep their pages
    move = (have & (n > budget))[:, None].expand(L, S, Hkv, -1)
    l = torch.arange(L, device="cuda")[:, None, None, None].expand_as(src)[move]
    h = torch.arange(Hkv, device="cuda")[:, None].expand_as(src)[move]
    src, dst = src[move], dst[move]
    for p in (st["k"], st["v"]):
        p[l, dst // bs, h, dst % bs] = p[l, src // bs, h, src % bs]
    return dict(kept=st["kept"], mass=st["mass_out"], k=st["k"], v=st["v"])


def _verify(st):
    c = st["c"]
    B, n, V = c["B"], c["n"], c["vocab"]
    b = torch.arange(B, device="cuda")
    cur = torch.full((B,), -1, device="cuda")
    count = torch.zeros(B, dtype=torch.int64, device="cuda")
    p = st["target"][:, 0].double()
    q = st["draft"][:, 0].double() if st["draft"] is not None else torch.zeros_like(p)
    a = torch.zeros(B, dtype=torch.float64, device="cuda")      # weight of q taken off p
    z = torch.ones(B, dtype=torch.float64, device="cuda")
    for i in range(n):
        x = st["tokens"][:, i].long()
        here = st["parent"][:, i] == cur
        u = st["u"][:, i].double()
        px = p[b, x]
        if st["draft"] is not None:
            qx = q[b, x]
            yes = here & (u * qx * z < px - a * qx)
            no = here & ~yes
            a = torch.where(no, a + z, a)
            z = torch.where(no, (p - a[:, None] * q).clamp_(min=0).sum(-1), z)
        else:   # the draft was certain of x: x itself leaves the distribution
            yes = here & (u * z < px)
            no = here & ~yes
            z = torch.where(no, (z - px).clamp(min=0), z)
            p[b, x] = torch.where(no, 0.0, px)
        cur = torch.where(yes, i, cur)
        count += yes
        p = torch.where(yes[:, None], st["target"][:, i + 1].double(), p)
        if st["draft"] is not None:
            q = torch.where(yes[:, None], st["draft"][:, i + 1].double(), q)
        a, z = torch.where(yes, 0.0, a), torch.where(yes, 1.0, z)
    cdf = (p - a[:, None] * q).clamp_(min=0).cumsum(-1)
    t = st["u_next"].double() * cdf[:, -1]
    nxt = torch.searchsorted(cdf, t[:, None], right=True)[:, 0]
    return dict(accepted=cur.int(), count=count.int(), next=nxt.int())


PLAIN = dict(window=_window, mass=_mass, evict=_evict, verify=_verify)


def run(state):
    st, c = state, state["c"]
    if not own:
        return PLAIN[c["op"]](st)
    kvp = st["kvp"]
    if c["op"] == "window":
        kvp.paged_window_attention(st["q"], st["nq"], st["k"], st["v"], st["tables"], st["n"], c["win"], c["sinks"],
                                   st["desc"], st["out"], st["lse"], st["ws"])
        return dict(out=st["out"], lse=st["lse"])
    if c["op"] == "mass":
        kvp.kvp_attention_mass(st["q"], st["nq"], st["lse"], st["k"], st["tables"], st["n"], st["desc"], st["decay"],
                               st["mass"], st["prev"], st["mass_out"], st["ws"])
        return dict(mass=st["mass_out"])
    if c["op"] == "evict":
        # pruned branches of the parents, which stay whole
        h = st["pool"].handle
        kids = [kvp.seq_fork(h, s) for s in st["parents"]]
        kvp.seq_evict(h, kids, st["mass"], c["budget"], c["sink"], c["recent"], st["kept"], st["mass_out"], st["ws"])
        for s in reversed(kids):
            kvp.seq_free(h, s)
        return dict(kept=st["kept"], mass=st["mass_out"], k=st["k"], v=st["v"])
    kvp.kvp_draft_verify(st["target"], st["draft"], st["parent"], st["tokens"], st["u"], st["u_next"],
                         st["accepted"], st["count"], st["next"])
    return dict(accepted=st["accepted"], count=st["count"], next=st["next"])


# --------------------------------------------------------------- work, exact

def _pairs(n, q, W, sinks):
    """Visible (query, key) pairs of one sequence, and the distinct keys."""
    pos = np.arange(n - q, n, dtype=np.int64)
    lo = np.maximum(pos - W + 1, 0)
    pairs = int((pos - lo + 1 + np.minimum(lo, sinks)).sum())
    return pairs, int(n - lo[0] + min(int(lo[0]), sinks))


def work(case):
    c = dict(case)
    if c["op"] == "verify":
        # the row at which the walk stops: target's, and the draft's with it
        return dict(bytes=float(c["B"] * (c["vocab"] * (8 if c["draft"] else 4) + 16 * c["n"] + 12)),
                    flops=float(c["B"] * c["vocab"] * 4))
    Hq, Hkv, d = HEADS[c["heads"]]
    L = c["L"]
    n, nq = _lens(c)
    if c["op"] == "window":
        pk = [_pairs(int(a), int(b), c["win"], c["sinks"]) for a, b in zip(n, nq)]
        T = int(nq.sum())
        return dict(bytes=float(L * (T * Hq * (4 * d + 4) + sum(k for _, k in pk) * Hkv * 4 * d)),
                    flops=float(L * Hq * 4 * d * sum(p for p, _ in pk)))
    if c["op"] == "mass":
        pk = [_pairs(int(a), int(b), int(a), 0) for a, b in zip(n, nq)]
        T, K = int(nq.sum()), int(n.sum())
        return dict(bytes=float(L * (T * Hq * (2 * d + 4) + K * Hkv * (2 * d + 8))),
                    flops=float(L * Hq * 2 * d * sum(p for p, _ in pk)))
    keep = int(np.minimum(n, c["budget"])[n > c["budget"]].sum())
    return dict(bytes=float(L * Hkv * (4 * int(n.sum()) + keep * (8 * d + 8))), flops=float(L * Hkv * int(n.sum())))


def exact(case, seed):
    global own
    was, own = own, False       # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = was
    c = st["c"]
    f64 = torch.float64
    if c["op"] == "verify":
        return _exact_verify(st)
    Hkv, G = st["Hkv"], st["Hq"] // st["Hkv"]
    bs, L = c["bs"], c["L"]
    if c["op"] == "evict":
        kept = np.full((L, c["S"], Hkv, c["budget"]), -1, np.int32)
        mass, old = st["mass_out"].cpu().numpy().copy(), st["mass"].cpu().numpy()
        k, v = st["k"].clone(), st["v"].clone()
        at = int(sum(-(-int(x) // bs) for x in st["n"]))
        order = _shuffled(st["NB"], 1 + seed)
        for s, n in enumerate(int(x) for x in st["n"]):
            m = min(n, c["budget"])
            if n <= m:
                kept[:, s, :, :m] = np.arange(m)
                mass[:, s, :, :m] = old[:, s, :, :m]
                continue
            pages = []
            for j in range(-(-m // bs)):
                if (j + 1) * bs <= c["sink"]:
                    pages.append(int(st["tables"][s, j]))
                else:
                    pages.append(int(order[at]))
                    at += 1
            i = np.arange(m)
            to = torch.from_numpy(np.array(pages)[i // bs]).cuda(), torch.from_numpy(i % bs).cuda()
            for l in range(L):
                for h in range(Hkv):
                    first = set(range(min(c["sink"], n))) | set(range(max(0, n - c["recent"]), n))
                    rest = [t for t in np.argsort(-old[l, s, h, :n], kind="stable") if t not in first]
                    pick = np.array(sorted(list(first) + rest[:m - len(first)]))
                    kept[l, s, h, :m] = pick
                    mass[l, s, h, :m] = old[l, s, h, pick]
                    blk = torch.from_numpy(st["tables"][s, pick // bs].astype(np.int64)).cuda()
                    off = torch.from_numpy(pick % bs).cuda()
                    k[l, to[0], h, to[1]] = st["k"][l, blk, h, off]
                    v[l, to[0], h, to[1]] = st["v"][l, blk, h, off]
        return dict(kept=kept, mass=mass, k=k, v=v)
    if c["op"] == "window":
        out = torch.zeros(*st["q"].shape, dtype=f64, device="cuda")
        lse = torch.zeros(*st["q"].shape[:3], dtype=f64, device="cuda")
    else:
        out = st["mass_out"].double()
    at = 0
    for s in range(c["S"]):
        n, m = int(st["n"][s]), int(st["nq"][s])
        blocks = torch.from_numpy(st["tables"][s, :-(-n // bs)].astype(np.int64)).cuda()
        j = torch.arange(n, device="cuda")
        p = torch.arange(n - m, n, device="cuda")[:, None]
        see = j <= p
        if c["op"] == "window":
            see = see & ((p - j < c["win"]) | (j < c["sinks"]))
        for l in range(L):
            for h in range(Hkv):
                K = st["k"][l, blocks, h].reshape(-1, st["d"])[:n].to(f64)
                total = torch.zeros(n, dtype=f64, device="cuda")
                for g in range(G):
                    x = (st["q"][l, at:at + m, h * G + g].to(f64) @ K.T) / math.sqrt(st["d"])
                    if c["op"] == "mass":
                        e = torch.exp(x - st["lse"][l, at:at + m, h * G + g].to(f64)[:, None])
                        total += torch.where(see, e, 0.0).sum(0)
                        continue
                    x = torch.where(see, x, -math.inf)
                    z = torch.logsumexp(x, 1)
                    V = st["v"][l, blocks, h].reshape(-1, st["d"])[:n].to(f64)
                    out[l, at:at + m, h * G + g] = torch.exp(x - z[:, None]) @ V
                    lse[l, at:at + m, h * G + g] = z
                if c["op"] == "mass":
                    keep = st["mass"][l, s, h, :n].double() * (j < int(st["prev"][s]))
                    out[l, s, h, :n] = st["decay"] * keep + total
        at += m
    return dict(out=out, lse=lse) if c["op"] == "window" else dict(mass=out)


def _exact_verify(st):
    """The walk from the root, node by node, on the host in 64 bits."""
    c = st["c"]
    par, tok = st["parent"].cpu().numpy(), st["tokens"].cpu().numpy()
    u, un = st["u"].cpu().numpy().astype(np.float64), st["u_next"].cpu().numpy().astype(np.float64)
    res = np.zeros((3, c["B"]), np.int32)
    for b in range(c["B"]):
        node, depth = -1, 0
        while True:
            p = st["target"][b, node + 1].cpu().numpy().astype(np.float64)
            q = st["draft"][b, node + 1].cpu().numpy().astype(np.float64) if st["draft"] is not None else None
            a, z, took = 0.0, 1.0, -1
            r = p.copy()        # what is left of p, unnormalised
            for i in np.flatnonzero(par[b] == node):
                x = tok[b, i]
                ok = u[b, i] * z < r[x] if q is None else u[b, i] * q[x] * z < p[x] - a * q[x]
                if ok:
                    took = int(i)
                    break
                if q is None:
                    z = max(z - r[x], 0.0)
                    r[x] = 0.0
                else:
                    a += z
                    r = np.maximum(p - a * q, 0.0)
                    z = math.fsum(r)
            if took < 0:
                break
            node, depth = took, depth + 1
        cdf = np.cumsum(r)
        res[:, b] = node, depth, int(np.searchsorted(cdf, un[b] * cdf[-1], side="right"))
    return dict(accepted=res[0], count=res[1], next=res[2])
