"""Beam search over a paged cache with all of it together: prompts appended with
the rotation, then per token the beams' append, page bounds, scores, selection,
attention over the chosen pages, beam selection, and sequences, histories and
running attention weights reordered; each step against a dense 64-bit cache."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu

L, Hq, Hkv, d, bs, V = 2, 8, 2, 64, 16, 700
G, B, BUDGET, SINK, RECENT = 2, 3, 5, 1, 1
NB, MB = 400, 20


class Model:
    """Fixed random maps from a token and the attention's output."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.k, self.v, self.q = r(V, L, Hkv, d), r(V, L, Hkv, d), r(V, L, Hq, d)
        self.out = r(L * Hq * d, V) / 8

    def project(self, tokens):
        pick = lambda w: w[tokens].transpose(0, 1).contiguous().to(torch.bfloat16)
        return pick(self.k), pick(self.v), pick(self.q)

    def logits(self, o):                                    # [L][T][Hq][d]
        return o.transpose(0, 1).flatten(1).float() @ self.out


def turn(x, pos):
    """[L][T][H][d] rotated in 64 bits, rounded to bf16 once, as 64-bit numbers."""
    a = np.asarray(pos, np.float64)[:, None] * 10000.0 ** (-np.arange(d // 2) * 2.0 / d)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    x = x.double().cpu().numpy()
    y = np.concatenate([x[..., :d // 2] * c - x[..., d // 2:] * s, x[..., d // 2:] * c + x[..., :d // 2] * s], -1)
    return torch.from_numpy(y).to(torch.bfloat16).double().numpy()


def test_beam_search_loop():
    m = Model(3)
    dev = "cuda"
    kp, vp = (torch.zeros(L, NB, Hkv, bs, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    pool = kvp.kv_pool_create(kvp.PoolDesc(L, NB, bs, Hkv, d, 2 * G * B, MB, 5), kp, vp)
    desc = kvp.AttnDesc(L, Hq, Hkv, d, bs, NB, 0.0, 0)
    rope = kvp.rope_desc(d)
    rows = G * B
    bounds = torch.zeros(L, NB, Hkv, 2, d, dtype=torch.bfloat16, device=dev)
    tables = torch.zeros(rows, MB, dtype=torch.int32, device=dev)
    lens = torch.zeros(rows, dtype=torch.int32, device=dev)
    scores = torch.zeros(L, rows, Hkv, MB, device=dev)
    selected = torch.zeros(L, rows, Hkv, BUDGET, dtype=torch.int32, device=dev)
    out = torch.zeros(L, rows, Hq, d, dtype=torch.bfloat16, device=dev)
    lse = torch.zeros(L, rows, Hq, device=dev)
    hist = torch.full((rows, 64), -1, dtype=torch.int32, device=dev)
    ws = torch.empty(kvp.kvp_beam_workspace_size(G, B, V, B), dtype=torch.uint8, device=dev)
    best = torch.zeros(G, B, device=dev)
    new_row, token = (torch.zeros(G, B, dtype=torch.int32, device=dev) for _ in range(2))

    # prompts: one sequence a request, then its beams as forks
    g = np.random.default_rng(1)
    n0 = [75, 133]
    prompts = [torch.from_numpy(g.integers(0, V, n)).to(dev) for n in n0]
    k, v, _ = m.project(torch.cat(prompts))
    roots = [kvp.seq_alloc(pool) for _ in range(G)]
    kvp.seq_append_rope(pool, roots, n0, k, v, rope)
    cache, at = [], 0            # dense reference: [K, V] per row
    for r in range(G):
        K, Vr = turn(k[:, at:at + n0[r]], np.arange(n0[r])), v[:, at:at + n0[r]].double().cpu().numpy()
        at += n0[r]
        cache += [[K.copy(), Vr.copy()] for _ in range(B)]
    beams = [kvp.seq_fork(pool, roots[r // B]) for r in range(rows)]
    kvp.kvp_export_tables(pool, beams, MB, tables, lens)
    kvp.kvp_page_bounds(kp, tables, lens, max(n0), desc, bounds)        # the whole prompts
    score = torch.tensor([[0.0] + [-math.inf] * (B - 1)] * G, device=dev)    # equal beams: one in use
    tokens = torch.tensor([int(prompts[r // B][-1]) for r in range(rows)], device=dev)
    ref_hist = [[] for _ in range(rows)]

    for step in range(24):
        k, v, q = m.project(tokens)
        pos = [kvp.seq_len(pool, s) for s in beams]
        kvp.seq_append_rope(pool, beams, [1] * rows, k, v, rope, None, q, q)
        kvp.kvp_export_tables(pool, beams, MB, tables, lens)
        kvp.kvp_page_bounds(kp, tables, lens, 1, desc, bounds)
        kvp.kvp_page_scores(q, None, bounds, tables, lens, desc, scores)
        kvp.kvp_page_select(scores, None, lens, desc, SINK, RECENT, selected)
        kvp.paged_sparse_attention(q, None, kp, vp, tables, lens, selected, desc, out, lse)
        logits = m.logits(out).view(G, B, V)
        kvp.kvp_beam_select(logits, score, None, 0, best, new_row, token, ws)

        # the dense cache and what each row should have chosen
        nk, nv, nq = turn(k, pos), v.double().cpu().numpy(), q.double().cpu().numpy()
        sel, sc = selected.cpu().numpy(), scores.cpu().numpy()
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for r in range(rows):
            K = cache[r][0] = np.concatenate([cache[r][0], nk[:, r:r + 1]], 1)
            Vr = cache[r][1] = np.concatenate([cache[r][1], nv[:, r:r + 1]], 1)
            n = K.shape[1]
            pages = -(-n // bs)
            for l, h in np.ndindex(L, Hkv):
                qh = nq[l, r, 4 * h:4 * h + 4]
                bound = np.array([np.maximum(qh * K[l, j * bs:(j + 1) * bs, h].min(0),
                                             qh * K[l, j * bs:(j + 1) * bs, h].max(0)).sum() for j in range(pages)]) / 8
                # (a key that rounds the other way moves a bound by 2^-8 of it)
                assert np.abs(sc[l, r, h, :pages] - bound).max() <= 2.0 ** -5
                mid = [j for j in range(SINK, pages - RECENT)]
                order = sorted(mid, key=lambda j: (-sc[l, r, h, j], j))[:BUDGET - SINK - RECENT]
                pick = sorted(list(range(SINK)) + order + list(range(pages - RECENT, pages)))
                assert sel[l, r, h].tolist() == pick + [-1] * (BUDGET - len(pick))
                t = np.concatenate([np.arange(j * bs, min(n, (j + 1) * bs)) for j in pick])
                z = qh @ K[l, t, h].T / 8
                e = np.exp(z - z.max(1, keepdims=True))
                want = e @ Vr[l, t, h] / e.sum(1, keepdims=True)
                assert np.abs(got[l, r, 4 * h:4 * h + 4] - want).max() <= 2e-2
                assert np.abs(got_lse[l, r, 4 * h:4 * h + 4] - z.max(1) - np.log(e.sum(1))).max() <= 1e-2
        x = logits.double().cpu().numpy()
        rows_, toks, bests = new_row.cpu().numpy(), token.cpu().numpy(), best.cpu().numpy()
        for r in range(G):
            lp = score[r].double().cpu().numpy()[:, None] + x[r] - np.logaddexp.reduce(x[r], 1)[:, None]
            top = np.argsort(-lp, axis=None, kind="stable")[:B]
            assert rows_[r].tolist() == [r * B + i // V for i in top] and toks[r].tolist() == [i % V for i in top]
            assert np.abs(bests[r] - lp.flat[top]).max() <= 1e-4

        # on to the chosen beams
        parent = rows_.reshape(-1).tolist()
        kvp.seq_reorder(pool, beams, [beams[i] for i in parent])
        moved = hist.clone()
        kvp.kvp_state_reorder(hist, moved, new_row)
        hist = moved
        hist[:, step] = token.view(-1)
        cache = [[cache[i][0].copy(), cache[i][1].copy()] for i in parent]
        ref_hist = [ref_hist[i] + [t] for i, t in zip(parent, toks.reshape(-1).tolist())]
        score, tokens = best.clone(), token.view(-1).long()
        assert hist[:, :step + 1].cpu().numpy().tolist() == ref_hist

    # the pages hold the beams' caches, shared prefixes once
    t, n = kvp.kvp_gather_tables(pool, beams, MB)
    for r in range(rows):
        blocks = torch.from_numpy(t[r, :-(-n[r] // bs)].astype(np.int64)).cuda()
        for p, which in ((kp, 0), (vp, 1)):
            rows_of = p[:, blocks].transpose(2, 3).flatten(1, 2)[:, :n[r]].double().cpu().numpy()
            assert np.abs(rows_of - cache[r][which]).max() <= 2.0 ** -8 * 4.5
    assert len(set(t[t >= 0].tolist())) < sum(-(-x // bs) for x in n)
    for s in beams + roots:
        kvp.seq_free(pool, s)
    assert kvp.kvp_free_block_count(pool) == NB
    kvp.kv_pool_destroy(pool)


def test_default_stream_beside_a_capture_is_refused():
    """The legacy default stream cannot be used while a stream that synchronises with it is captured: every call says
    so before anything changes, and the capture goes on."""
    import ctypes
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    kp, vp, bounds = torch.zeros(1, 8, 1, bs, d, **bf16), torch.zeros(1, 8, 1, bs, d, **bf16), torch.zeros(1, 8, 1, 2, d, **bf16)
    pool = kvp.kv_pool_create(kvp.PoolDesc(1, 8, bs, 1, d, 2, 8, 0), kp, vp)
    a = kvp.seq_alloc(pool)
    desc = kvp.AttnDesc(1, 2, 1, d, bs, 8, 0.0, 0)
    q, out = torch.zeros(1, 1, 2, d, **bf16), torch.zeros(1, 1, 2, d, **bf16)
    new = torch.zeros(1, 3, 1, d, **bf16)
    t, n = torch.zeros(1, 8, dtype=torch.int32, device="cuda"), torch.full((1,), 40, dtype=torch.int32, device="cuda")
    sc, sel = torch.zeros(1, 1, 1, 8, device="cuda"), torch.zeros(1, 1, 1, 2, dtype=torch.int32, device="cuda")
    x, cum = torch.zeros(1, 2, 100, device="cuda"), torch.zeros(1, 2, device="cuda")
    best, row, tok = torch.zeros(1, 2, device="cuda"), *(torch.zeros(1, 2, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    src, dst = torch.zeros(2, 8, device="cuda"), torch.ones(2, 8, device="cuda")
    torch.cuda.synchronize()
    cu = ctypes.CDLL("libcuda.so.1")
    s, g = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(s), 0) == 0
    assert cu.cuStreamBeginCapture_v2(s, 1) == 0         # a capture of this thread's
    codes = []
    for call in (lambda: kvp.seq_append_rope(pool, [a], [3], new, new, kvp.rope_desc(d), stream=0),
                 lambda: kvp.kvp_page_bounds(kp, t, n, 1, desc, bounds, stream=0),
                 lambda: kvp.kvp_page_scores(q, None, bounds, t, n, desc, sc, stream=0),
                 lambda: kvp.kvp_page_select(sc, None, n, desc, 0, 1, sel, stream=0),
                 lambda: kvp.paged_sparse_attention(q, None, kp, vp, t, n, sel, desc, out, None, stream=0),
                 lambda: kvp.kvp_beam_select(x, cum, None, 0, best, row, tok, ws, stream=0),
                 lambda: kvp.kvp_state_reorder(src, dst, row.view(-1), stream=0)):
        try:
            call()
            codes.append(0)
        except kvp.KvpError as e:
            codes.append(e.code)
    ended = cu.cuStreamEndCapture(s, ctypes.byref(g))
    cu.cuStreamDestroy_v2(s)
    assert codes == [kvp.KVP_ERR_STATE] * 7 and ended == 0
    assert kvp.seq_len(pool, a) == 0 and kvp.kvp_free_block_count(pool) == 8
    torch.cuda.synchronize()
    assert float(dst.sum()) == 16
    kvp.kv_pool_destroy(pool)
