"""Cases that measure operators over the paged KV pool beside those of
operators.py: appending with the position rotation on the way, page bounds and
page scores, selection of pages by score, attention over selected pages, and
beam search's selection with the reordering of the beams' states.

`own` false runs the operators in plain torch operations (32-bit; 64-bit for
the rotation's angles and for beam scores, whose order decides a token); `own`
true makes the calls of the package.  Pools are bf16 with scattered blocks.
"""
import math

import numpy as np
import torch

own = False

# head shapes of the repository's workloads
HEADS = {"64": (32, 4, 64), "128": (32, 8, 128)}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one agent's next token in every layer: latency
        dict(name="rope_decode_1", op="rope", heads="64", bs=16, L=22, S=1, q=1, len=700, rot=64, pairs="half", far=0),
        # a batch of beams, each taken over from its parent: copy-on-write of
        # the last page, positions far behind the evicted cache's slots
        dict(name="rope_decode_64", op="rope", heads="128", bs=16, L=8, S=64, q=1, len=520, rot=128, pairs="half",
             far=900000),
        # ragged prompts of a mixed batch, half of each head rotated, adjacent pairs
        dict(name="rope_prompt", op="rope", heads="128", bs=32, L=2, S=5, q=8191, len=1, rot=64, pairs="adjacent",
             far=0),
        # decode step over long caches: the newest page's bounds, then every page's score
        dict(name="score_decode_64", op="score", heads="128", bs=16, L=1, S=64, q=1, len=40000, new=1),
        # a prompt's chunk: all bounds of the prompt, scores of a few hundred queries
        dict(name="score_extend", op="score", heads="64", bs=32, L=2, S=3, q=257, len=9001, new=9001),
        # one sequence's page choice: latency
        dict(name="select_1", op="select", heads="64", bs=16, L=1, S=1, q=1, len=33000, budget=64, sink=1, recent=4),
        # a batch over very long caches, all layers at once
        dict(name="select_64", op="select", heads="128", bs=16, L=4, S=64, q=1, len=131072, budget=128, sink=1,
             recent=8),
        # one sequence's next token over its chosen pages
        dict(name="sparse_decode_1", op="sparse", heads="64", bs=16, L=1, S=1, q=1, len=33000, budget=64, sink=1,
             recent=4),
        # a serving batch's decode step, two layers
        dict(name="sparse_decode_64", op="sparse", heads="128", bs=16, L=2, S=64, q=1, len=12000, budget=128, sink=1,
             recent=8),
        # chunks of ragged prompts, larger pages, every query with its own choice
        dict(name="sparse_extend", op="sparse", heads="128", bs=32, L=1, S=3, q=333, len=8001, budget=32, sink=1,
             recent=2),
        # one request with four beams
        dict(name="beam_4", op="beam", G=1, B=4, vocab=32000, type="bf16", n=4, hist=200, done=False),
        # a batch of requests with eight beams, twice as many candidates, some beams finished
        dict(name="beam_256", op="beam", G=32, B=8, vocab=131072, type="f32", n=16, hist=4096, done=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "score", "select", "sparse", "beam"])
    c = dict(op=op)
    if op == "beam":
        c.update(B=rng.randint(1, 12), vocab=_log(rng, 200, 131072), type=rng.choice(sorted(TYPES)))
        c.update(G=min(_log(rng, 1, 64), max(1, 32_000_000 // (c["B"] * c["vocab"]))), hist=_log(rng, 8, 4096))
        c.update(n=c["B"] * rng.randint(1, 2), done=rng.random() < 0.5)
        return c
    c.update(heads=rng.choice(sorted(HEADS)), bs=rng.choice([16, 32]))
    chunk = rng.random() < 0.35
    if op == "rope":
        c.update(L=rng.randint(1, 4), S=_log(rng, 1, 8) if chunk else _log(rng, 1, 64))
        c.update(q=_log(rng, 2, 2000) if chunk else 1, len=_log(rng, 1, 600), pairs=rng.choice(["half", "adjacent"]))
        c.update(rot=rng.choice([16, 32, 64, int(c["heads"])]), far=rng.choice([0, _log(rng, 1000, 1000000)]))
        return c
    if op == "score":
        c.update(L=1, S=_log(rng, 1, 4) if chunk else _log(rng, 1, 64), q=_log(rng, 2, 250) if chunk else 1)
        c.update(len=c["q"] + _log(rng, 1, 8000 if chunk else 40000))
        c.update(new=c["len"] if chunk else rng.choice([1, 1, 5, 40]))
        return c
    c.update(L=1, S=_log(rng, 1, 3) if chunk else _log(rng, 1, 64), q=_log(rng, 2, 300) if chunk else 1)
    # some pages by score beside those by position, and more pages than are chosen
    c.update(budget=_log(rng, 2, 32 if chunk else 128))
    c.update(sink=min(rng.choice([0, 1, 2]), c["budget"] - 1))
    c.update(recent=rng.randint(0, min(8, c["budget"] - c["sink"] - 1)))
    c.update(len=c["q"] + 4 * c["bs"] * c["budget"] + _log(rng, 20, 8000))
    return c


# ------------------------------------------------------------------ inputs

def _lens(c):
    """Cached tokens (those of this call among them) and query tokens of each
    sequence, the case's alone: the first has the case's own, the others down
    to half of them."""
    g = np.random.Generator(np.random.Philox(key=[c["len"], c["S"]]))
    f = g.uniform(0.5, 1.0, c["S"])
    f[0] = 1.0
    q = np.maximum(1, (c["q"] * f).astype(np.int64))
    if c["q"] > 64 and c["S"] > 2:
        q[1] = 1                # a decoding sequence rides along
    n = np.maximum(q, (c["len"] * f).astype(np.int64))
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


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class _Pool:
    """A pool handle that goes with its state."""

    def __init__(self, kvp, handle):
        self.kvp, self.handle = kvp, handle

    def __del__(self):
        self.kvp.kv_pool_destroy(self.handle)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 23)
    st = dict(c=c)
    if own:
        import paged_prefix_shared_decode_gb300 as kvp
        st["kvp"] = kvp
    if c["op"] == "beam":
        return _prepare_beam(c, gen, st)
    Hq, Hkv, d = HEADS[c["heads"]]
    st.update(Hq=Hq, Hkv=Hkv, d=d)
    if c["op"] == "rope":
        return _prepare_rope(c, seed, gen, st)
    n, nq = _lens(c)
    bs, L, S = c["bs"], c["L"], c["S"]
    pages = -(-n // bs)
    T, NB, MB = int(nq.sum()), int(pages.sum()), int(pages.max())
    seq = np.repeat(np.arange(S), nq)
    first = np.concatenate([[0], np.cumsum(nq)])
    pos = (n - nq)[seq] + np.arange(T) - first[seq]
    st.update(NB=NB, n=n, nq=nq, T=T, MB=MB, seq=_cuda(seq), col=_cuda(np.arange(T) - first[seq]), pos=_cuda(pos),
              lens=_cuda(n.astype(np.int32)), q_start=None if c["q"] == 1 else _cuda(first.astype(np.int32)))
    if own:
        st["desc"] = kvp.AttnDesc(L, Hq, Hkv, d, bs, NB, 0.0, 0, kvp.KVP_KV_BF16)
    if c["op"] != "select":
        # block tables as kvp_export_tables leaves them on the device
        order = torch.randperm(NB, generator=gen, device="cuda").int()
        at = _cuda(np.concatenate([[0], np.cumsum(pages)[:-1]]))[:, None] + torch.arange(MB, device="cuda")
        st["tables"] = torch.where(torch.arange(MB, device="cuda") < _cuda(pages)[:, None],
                                   order[at.clamp(max=NB - 1)], -1).int()
        st["k"] = _normal(gen, L, NB, Hkv, bs, d)
        st["q"] = _normal(gen, L, T, Hq, d)
    if c["op"] == "score":
        # keys of trained models have large channels: a per-head offset
        st["k"] += 2 * _normal(gen, L, 1, Hkv, 1, d)
        st["bounds"] = torch.zeros(L, NB, Hkv, 2, d, dtype=torch.bfloat16, device="cuda")
        _bounds(st, 0, st["lens"] - c["new"])          # as they were before the newest tokens
        st["scores"] = torch.zeros(L, T, Hkv, MB + 3, device="cuda")
        return st
    # neighbouring queries choose alike: a score per page and 32 queries, and a query's own part
    own_part = torch.rand(L, T, Hkv, MB, generator=gen, device="cuda")
    common = torch.rand(L, S, T // 32 + 1, Hkv, MB, generator=gen, device="cuda")
    st["scores"] = own_part * 0.3 + common[:, st["seq"], st["col"] // 32]
    st["selected"] = torch.zeros(L, T, Hkv, c["budget"], dtype=torch.int32, device="cuda")
    if c["op"] == "sparse":
        _select(st)
        del st["scores"]
        st["v"] = _normal(gen, L, NB, Hkv, bs, d)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(L, T, Hq, device="cuda")
    return st


def _prepare_rope(c, seed, gen, st):
    """Parents of `len` tokens (fewer for some) and a branch of each, which
    every pass sets back to its parent and then appends to."""
    kvp = st.get("kvp")
    n, nq = _lens(dict(c, len=c["len"] + c["q"]))
    n0 = np.maximum(0, n - nq)
    bs, L, S, d, Hkv, Hq = c["bs"], c["L"], c["S"], st["d"], st["Hkv"], st["Hq"]
    pages0, pages1 = -(-n0 // bs), -(-(n0 + nq) // bs)
    NB = int(pages1.sum() + pages0.sum()) + S
    order = _shuffled(NB, 1 + seed)
    T, at = int(nq.sum()), int(pages0.sum())
    begin = np.concatenate([[0], np.cumsum(pages0)[:-1]])
    slots, cow = [], []
    for s in range(S):          # where the pool's allocation puts the new tokens
        used = int(n0[s] % bs)
        table = list(order[begin[s]:begin[s] + pages0[s]])
        if used:                # the parent's last page is shared and not full
            cow.append((int(table[-1]), int(order[at]), used))
            table[-1] = order[at]
            at += 1
        more = int(pages1[s]) - len(table)
        table += list(order[at:at + more])
        at += more
        p = np.arange(n0[s], n0[s] + nq[s])
        slots.append(np.array(table, np.int64)[p // bs] * bs + p % bs)
    seq = np.repeat(np.arange(S), nq)
    pos = n0[seq] + np.arange(T) - np.concatenate([[0], np.cumsum(nq)[:-1]])[seq] + c["far"]
    st.update(nq=nq, slots=_cuda(np.concatenate(slots)), T=T, pos=_cuda(pos))
    st["cow_src"] = _cuda(np.array([x[0] for x in cow for _ in range(x[2])] or [0], np.int64))
    st["cow_dst"] = _cuda(np.array([x[1] for x in cow for _ in range(x[2])] or [0], np.int64))
    st["cow_off"] = _cuda(np.array([i for x in cow for i in range(x[2])] or [0], np.int64))
    st["k"], st["v"] = _normal(gen, L, NB, Hkv, bs, d), _normal(gen, L, NB, Hkv, bs, d)
    st["k_new"], st["v_new"] = _normal(gen, L, T, Hkv, d), _normal(gen, L, T, Hkv, d)
    st["q"] = _normal(gen, L, T, Hq, d)
    st["q_out"] = torch.empty_like(st["q"])
    st["base"] = 500000.0
    if kvp:
        h = kvp.kv_pool_create(kvp.PoolDesc(L, NB, bs, Hkv, d, 2 * S, int(pages1.max()) + 1, 1 + seed),
                               st["k"], st["v"])
        st["pool"] = _Pool(kvp, h)
        st["parents"] = [kvp.seq_alloc(h) for _ in range(S)]
        for s, i in enumerate(st["parents"]):
            kvp.seq_reserve(h, i, int(n0[s]))
        st["kids"] = [kvp.seq_fork(h, i) for i in st["parents"]]
        st["rope"] = kvp.rope_desc(c["rot"], base=st["base"], interleaved=c["pairs"] == "adjacent")
        st["positions"] = st["pos"].int() if c["far"] else None     # without: the cache's own positions
    return st


def _prepare_beam(c, gen, st):
    G, B, V = c["G"], c["B"], c["vocab"]
    # beams of one request share most of their text: common logits and a part of their own
    x = 2.5 * _normal(gen, G, 1, V, dtype=torch.float32) + _normal(gen, G, B, V, dtype=torch.float32)
    st["logits"] = x.to(TYPES[c["type"]])
    st["cum"] = -20 - 4 * torch.rand(G, B, generator=gen, device="cuda")
    st["done"] = (torch.rand(G, B, generator=gen, device="cuda") < 0.2) if c["done"] else None
    st["hist"] = torch.randint(0, V, (G * B, c["hist"]), generator=gen, device="cuda", dtype=torch.int32)
    st["hist_out"] = torch.zeros(G * c["n"], c["hist"], dtype=torch.int32, device="cuda")
    st["best"] = torch.zeros(G, c["n"], device="cuda")
    st["row"], st["token"] = (torch.zeros(G, c["n"], dtype=torch.int32, device="cuda") for _ in range(2))
    if own:
        need = st["kvp"].kvp_beam_workspace_size(G, B, V, c["n"])
        st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- plain forms

def _rotate(st, x):
    """x [L][T][H][d] turned by its tokens' positions, in 32 bits."""
    rot, half = st["c"]["rot"], st["c"]["rot"] // 2
    f = st["base"] ** (-torch.arange(half, dtype=torch.float64, device="cuda") * 2 / rot)
    a = st["pos"].double()[:, None] * f
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]     # [T][1][half]
    x = x.float()
    y = x.clone()
    i = torch.arange(half, device="cuda")
    i, j = (i, i + half) if st["c"]["pairs"] == "half" else (2 * i, 2 * i + 1)
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., j] * cos + x[..., i] * sin
    return y.to(torch.bfloat16)


def _rope(st):
    bs = st["c"]["bs"]
    blk, off = st["slots"] // bs, st["slots"] % bs
    for p, new in ((st["k"], _rotate(st, st["k_new"])), (st["v"], st["v_new"])):
        # (without a shared page: a page copied onto itself)
        p[:, st["cow_dst"], :, st["cow_off"]] = p[:, st["cow_src"], :, st["cow_off"]]
        p[:, blk, :, off] = new.transpose(0, 1)
    st["q_out"].copy_(_rotate(st, st["q"]))
    return dict(k=st["k"], v=st["v"], q=st["q_out"])


def _valid(st, lens):
    """Tokens of each table entry's page: [S][MB]."""
    j = torch.arange(st["MB"], device="cuda")
    return (lens[:, None] - j * st["c"]["bs"]).clamp(0, st["c"]["bs"])


def _bounds(st, since, lens):
    """Smallest and largest key of each page that holds tokens from `since` on."""
    bs, tables = st["c"]["bs"], st["tables"]
    end = (torch.arange(st["MB"], device="cuda") + 1) * bs
    s, j = torch.nonzero((_valid(st, lens) > 0) & (end > torch.as_tensor(since, device="cuda").reshape(-1, 1)),
                         as_tuple=True)
    blk = tables[s, j].long()
    k = st["k"][:, blk]                                         # [L][pages][Hkv][bs][d]
    ok = (torch.arange(bs, device="cuda") < _valid(st, lens)[s, j][:, None])[:, None, :, None]
    st["bounds"][:, blk, :, 0] = torch.where(ok, k, math.inf).amin(-2)
    st["bounds"][:, blk, :, 1] = torch.where(ok, k, -math.inf).amax(-2)


def _seen(st):
    """Pages that query row t sees, [T][MB]: those that begin at or before it."""
    return torch.arange(st["MB"], device="cuda") <= (st["pos"] // st["c"]["bs"])[:, None]


def _score(st):
    c = st["c"]
    L, S, Hkv, d, MB = c["L"], c["S"], st["Hkv"], st["d"], st["MB"]
    _bounds(st, st["lens"] - c["new"], st["lens"])
    q = st["q"].float().view(L, st["T"], Hkv, -1, d)
    pad = q.new_zeros(2, L, S, int(st["nq"].max()), Hkv, d)
    pad[:, :, st["seq"], st["col"]] = torch.stack([q.clamp(max=0).sum(3), q.clamp(min=0).sum(3)])
    b = st["bounds"][:, st["tables"].clamp(min=0)].float()      # [L][S][MB][Hkv][2][d]
    b = b.permute(4, 0, 1, 3, 5, 2)                             # [2][L][S][Hkv][d][MB]
    s = (pad.transpose(3, 4) @ b).sum(0) * (1 / math.sqrt(d))   # [L][S][Hkv][queries][MB]
    s = s.transpose(2, 3)[:, st["seq"], st["col"]]              # [L][T][Hkv][MB]
    out = st["scores"]
    out[..., :MB] = torch.where(_seen(st)[:, None], s, out[..., :MB])
    return dict(bounds=st["bounds"], scores=out)


def _select(st):
    c, j = st["c"], torch.arange(st["MB"], device="cuda")
    last = (st["pos"] // c["bs"])[:, None]
    must = (j < c["sink"]) | (j > last - c["recent"])
    w = st["scores"].masked_fill(must[:, None], math.inf).masked_fill(~_seen(st)[:, None], -math.inf)
    by = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    have = by <= last[:, None]                                  # a short sequence has fewer pages
    by = torch.where(have, by, st["MB"]).sort(-1).values
    by = torch.where(by < st["MB"], by, -1).int()
    st["selected"].fill_(-1)[..., :by.shape[-1]] = by
    return dict(selected=st["selected"])


def _sparse(st):
    c, L, Hkv, d, bs = st["c"], st["c"]["L"], st["Hkv"], st["d"], st["c"]["bs"]
    sel, T = st["selected"].long(), st["T"]
    at = sel.clamp(min=0)
    blk = st["tables"].long()[st["seq"]][None, :, None].expand(L, T, Hkv, -1).gather(-1, at)
    l = torch.arange(L, device="cuda")[:, None, None, None]
    h = torch.arange(Hkv, device="cuda")[:, None]
    key = (at[..., None] * bs + torch.arange(bs, device="cuda")).flatten(-2)        # [L][T][Hkv][keys]
    see = (sel >= 0)[..., None].expand(*sel.shape, bs).flatten(-2) & (key <= st["pos"][:, None, None])
    k = st["k"][l, blk, h].flatten(3, 4).float()                                    # [L][T][Hkv][keys][d]
    q = st["q"].float().view(L, T, Hkv, -1, d)
    s = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(d))
    del k
    s.masked_fill_(~see[..., None, :], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)               # a query may have no page
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    o = (e @ st["v"][l, blk, h].flatten(3, 4).float()) / torch.where(z > 0, z, 1.0)
    return dict(out=o.to(torch.bfloat16).view(L, T, -1, d), lse=(m + torch.log(z)).view(L, T, -1))


def _beam(st):
    c = st["c"]
    G, B, V, n = c["G"], c["B"], c["vocab"], c["n"]
    x = st["logits"].double()
    m = x.amax(-1, keepdim=True)
    s = st["cum"].double()[..., None] + (x - (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))))
    if st["done"] is not None:      # a finished beam goes on with token 0 alone, at no cost
        s.masked_fill_(st["done"][..., None], -math.inf)
        s[..., 0] = torch.where(st["done"], st["cum"].double(), s[..., 0])
    best, at = torch.sort(s.view(G, B * V), dim=-1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    none = best == -math.inf
    row = torch.where(none, -1, at // V + B * torch.arange(G, device="cuda")[:, None]).int()
    token = torch.where(none, -1, at % V).int()
    keep = (row.view(-1) >= 0)[:, None]
    st["hist_out"].copy_(torch.where(keep, st["hist"][row.view(-1).clamp(min=0).long()], st["hist_out"]))
    return dict(best=best.float(), row=row, token=token, hist=st["hist_out"])


PLAIN = dict(rope=_rope, score=_score, select=_select, sparse=_sparse, beam=_beam)


def run(state):
    st, c = state, state["c"]
    if not own:
        return PLAIN[c["op"]](st)
    kvp = st["kvp"]
    if c["op"] == "rope":
        h = st["pool"].handle
        kvp.seq_reorder(h, st["kids"], st["parents"])
        kvp.seq_append_rope(h, st["kids"], st["nq"], st["k_new"], st["v_new"], st["rope"], positions=st["positions"],
                            q=st["q"], q_out=st["q_out"])
        return dict(k=st["k"], v=st["v"], q=st["q_out"])
    if c["op"] == "score":
        kvp.kvp_page_bounds(st["k"], st["tables"], st["lens"], c["new"], st["desc"], st["bounds"])
        kvp.kvp_page_scores(st["q"], st["q_start"], st["bounds"], st["tables"], st["lens"], st["desc"], st["scores"])
        return dict(bounds=st["bounds"], scores=st["scores"])
    if c["op"] == "select":
        kvp.kvp_page_select(st["scores"], st["q_start"], st["lens"], st["desc"], c["sink"], c["recent"],
                            st["selected"])
        return dict(selected=st["selected"])
    if c["op"] == "sparse":
        kvp.paged_sparse_attention(st["q"], st["q_start"], st["k"], st["v"], st["tables"], st["lens"], st["selected"],
                                   st["desc"], st["out"], st["lse"])
        return dict(out=st["out"], lse=st["lse"])
    kvp.kvp_beam_select(st["logits"], st["cum"], st["done"], 0, st["best"], st["row"], st["token"], st["ws"])
    kvp.kvp_state_reorder(st["hist"], st["hist_out"], st["row"])
    return dict(best=st["best"], row=st["row"], token=st["token"], hist=st["hist_out"])


# --------------------------------------------------------------- work, exact

def work(case):
    c = dict(case)
    if c["op"] == "beam":
        rows, size = c["G"] * c["B"], 4 if c["type"] == "f32" else 2
        out = c["G"] * c["n"]
        return dict(bytes=float(rows * (c["vocab"] * size + 4) + out * (12 + 8 * c["hist"])),
                    flops=float(3 * rows * c["vocab"]))
    Hq, Hkv, d = HEADS[c["heads"]]
    L, bs = c["L"], c["bs"]
    if c["op"] == "rope":
        n, nq = _lens(dict(c, len=c["len"] + c["q"]))
        T, copied = int(nq.sum()), int((np.maximum(0, n - nq) % bs).sum())
        return dict(bytes=float(4 * L * d * (T * (2 * Hkv + Hq) + copied * 2 * Hkv)),
                    flops=float(3 * L * T * (Hkv + Hq) * c["rot"]))
    n, nq = _lens(c)
    T = int(nq.sum())
    pages = -(-n // bs)
    rows = int((nq * pages).sum())       # (query, page) pairs, a few more than are seen
    if c["op"] == "score":
        fresh = int(np.minimum(n, c["new"] + bs).sum())
        return dict(bytes=float(L * Hkv * (int(pages.sum()) * 4 * d + fresh * 2 * d + rows * 4) + L * T * Hq * 2 * d),
                    flops=float(L * Hkv * rows * 4 * d))
    if c["op"] == "select":
        return dict(bytes=float(L * Hkv * (rows + T * c["budget"]) * 4), flops=float(L * Hkv * rows))
    chosen = np.minimum(pages, c["budget"])
    read = int(np.minimum(pages, nq * chosen).sum()) * bs
    return dict(bytes=float(L * (Hkv * (read * 4 * d + T * 4 * c["budget"]) + T * Hq * (4 * d + 4))),
                flops=float(L * Hq * 4 * d * bs * int((nq * chosen).sum())))


def exact(case, seed):
    global own
    was, own = own, False       # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return dict(rope=_exact_rope, score=_exact_score, select=_exact_select, sparse=_exact_sparse,
                beam=_exact_beam)[st["c"]["op"]](st)


def _exact_rope(st):
    c, f64 = st["c"], torch.float64
    k, v = st["k"].to(f64), st["v"].to(f64)
    src, dst, off = (st[x].cpu().numpy() for x in ("cow_src", "cow_dst", "cow_off"))
    for a, b, o in zip(src, dst, off):
        k[:, b, :, o], v[:, b, :, o] = k[:, a, :, o].clone(), v[:, a, :, o].clone()
    z = []
    for x in (st["k_new"], st["q"]):
        x = x.to(f64)
        y = x.clone()
        for i in range(c["rot"] // 2):      # one pair of dimensions as a complex number
            a, b = (i, i + c["rot"] // 2) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
            t = st["pos"].to(f64) * math.exp(-math.log(st["base"]) * 2 * i / c["rot"])
            w = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(t), t)[:, None]
            y[..., a], y[..., b] = w.real, w.imag
        z.append(y)
    blk, off = st["slots"] // c["bs"], st["slots"] % c["bs"]
    for l in range(c["L"]):
        k[l, blk, :, off] = z[0][l]
        v[l, blk, :, off] = st["v_new"][l].to(f64)
    return dict(k=k, v=v, q=z[1])


def _exact_score(st):
    c, f64 = st["c"], torch.float64
    bs, G = c["bs"], st["Hq"] // st["Hkv"]
    bounds, scores = st["bounds"].clone(), st["scores"].to(f64)
    row = 0
    for s in range(c["S"]):
        n, m = int(st["n"][s]), int(st["nq"][s])
        np_ = -(-n // bs)
        blocks = st["tables"][s, :np_].long()
        for j in range(max(0, n - c["new"]) // bs, np_):
            keys = st["k"][:, blocks[j], :, :min(bs, n - j * bs)]
            bounds[:, blocks[j], :, 0], bounds[:, blocks[j], :, 1] = keys.amin(2), keys.amax(2)
        lo, hi = bounds[:, blocks, :, 0].to(f64), bounds[:, blocks, :, 1].to(f64)      # [L][pages][Hkv][d]
        for t in range(m):
            seen = (n - m + t) // bs + 1
            q = st["q"][:, row + t].to(f64).view(c["L"], 1, st["Hkv"], G, -1)
            x = torch.maximum(q * lo[:, :seen, :, None], q * hi[:, :seen, :, None])
            scores[:, row + t, :, :seen] = x.sum((3, 4)).transpose(1, 2) / math.sqrt(st["d"])
        row += m
    return dict(bounds=bounds, scores=scores)


def _exact_select(st):
    c = st["c"]
    w, pos = st["scores"].cpu().numpy(), st["pos"].cpu().numpy()
    out = np.full((c["L"], st["T"], st["Hkv"], c["budget"]), -1, np.int32)
    for l, t, h in np.ndindex(out.shape[:3]):
        m = int(pos[t]) // c["bs"] + 1
        first = set(range(min(c["sink"], m))) | set(range(max(0, m - c["recent"]), m))
        rest = [p for p in np.argsort(-w[l, t, h, :m], kind="stable")[:c["budget"] + len(first)] if p not in first]
        pick = sorted((list(first) + rest)[:c["budget"]])
        out[l, t, h, :len(pick)] = pick
    return dict(selected=out)


def _exact_sparse(st):
    c, f64 = st["c"], torch.float64
    bs, G = c["bs"], st["Hq"] // st["Hkv"]
    out, lse = st["out"].to(f64), st["lse"].to(f64)
    sel, seq, pos = st["selected"].cpu().numpy(), st["seq"].cpu().numpy(), st["pos"].cpu().numpy()
    tables = st["tables"].cpu().numpy()
    for l, t, h in np.ndindex(sel.shape[:3]):
        p = sel[l, t, h][sel[l, t, h] >= 0]
        key = (p[:, None] * bs + np.arange(bs)).reshape(-1)
        key = _cuda(np.flatnonzero(key <= pos[t]))
        blk = _cuda(tables[seq[t], p].astype(np.int64))
        K = st["k"][l, blk, h].flatten(0, 1)[key].to(f64)
        V = st["v"][l, blk, h].flatten(0, 1)[key].to(f64)
        x = st["q"][l, t, h * G:(h + 1) * G].to(f64) @ K.T / math.sqrt(st["d"])
        lse[l, t, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
        out[l, t, h * G:(h + 1) * G] = torch.softmax(x, -1) @ V
    return dict(out=out, lse=lse)


def _exact_beam(st):
    c = st["c"]
    best = np.full((c["G"], c["n"]), -np.inf)
    row, token = (np.full((c["G"], c["n"]), -1, np.int32) for _ in range(2))
    hist, out = st["hist"].cpu().numpy(), st["hist_out"].cpu().numpy().reshape(c["G"], c["n"], -1)
    cum = st["cum"].cpu().numpy().astype(np.float64)
    done = st["done"].cpu().numpy() if st["done"] is not None else np.zeros(cum.shape, bool)
    for g in range(c["G"]):
        found = []
        for b in range(c["B"]):
            x = st["logits"][g, b].float().cpu().numpy().astype(np.float64)
            if done[g, b]:
                found.append((-cum[g, b], b, 0))
                continue
            x = x - np.logaddexp.reduce(x)
            top = np.argsort(-x, kind="stable")[:c["n"]]
            found += [(-(cum[g, b] + x[t]), b, int(t)) for t in top]
        for i, (s, b, t) in enumerate(sorted(found)[:c["n"]]):
            best[g, i], row[g, i], token[g, i] = -s, g * c["B"] + b, t
            out[g, i] = hist[g * c["B"] + b]
    return dict(best=best, row=row, token=token, hist=out.reshape(st["hist_out"].shape))
