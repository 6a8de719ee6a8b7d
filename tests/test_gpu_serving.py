"""The operators as a serving loop uses them, one after the other on one pool:
a prompt in chunks and decode steps under a sliding window, drafts verified
and accepted between them, and at the end the cache cut back to its heaviest
tokens."""
import math

import numpy as np
import pytest
import torch

import paged_prefix_shared_decode_gb300 as kvp
from test_draft_verify import walk

pytestmark = pytest.mark.gpu

L, Hq, Hkv, d, bs, V = 1, 8, 2, 64, 16, 50
WIN, SINKS = 48, 3


class Model:
    """Fixed random maps from a token and its position to K, V and Q, and from
    attention outputs to next-token probabilities."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(2)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.k, self.v, self.q = r(V, Hkv, d), r(V, Hkv, d), r(V, Hq, d)
        self.pos, self.out = r(512, d), r(Hq * d, V) * 0.06

    def kvq(self, tokens, pos):
        t, p = torch.as_tensor(tokens, device="cuda").long(), torch.as_tensor(pos, device="cuda").long()
        return tuple((m[t] + (self.pos[p][:, None] if i != 1 else 0)).to(torch.bfloat16)[None].contiguous()
                     for i, m in enumerate((self.k, self.v, self.q)))

    def probs(self, out):       # [T][Hq][d] -> [T][V]
        return torch.softmax(out.float().reshape(out.shape[0], -1) @ self.out, -1)


def attend(K, V_, q, see):
    """Plain attention in 64 bits: K, V_ [n][Hkv][d], q [m][Hq][d], see [m][n]."""
    Q = q.double().view(q.shape[0], Hkv, Hq // Hkv, d)
    x = torch.einsum("mhgd,nhd->hgmn", Q, K.double()) / math.sqrt(d)
    p = torch.softmax(x.masked_fill(~see, -math.inf), -1)
    return torch.einsum("hgmn,nhd->mhgd", p, V_.double()).reshape(q.shape[0], Hq, d)


def close(got, want, V_):
    # P and out in bf16: half a step of each (2^-9 of at most max |v|, and of out), doubled
    assert ((got.double() - want).abs() <= 2.0 ** -8 * (V_.double().abs().max() + want.abs())).all()


def test_prompt_drafts_and_decode():
    m = Model()
    NB = 64
    k = torch.zeros(L, NB, Hkv, bs, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    pool = kvp.kv_pool_create(kvp.PoolDesc(L, NB, bs, Hkv, d, 4, 32, 5), k, v)
    desc = kvp.AttnDesc(L, Hq, Hkv, d, bs, NB, 0.0, 1)
    seq = kvp.seq_alloc(pool)
    g = np.random.default_rng(8)
    tokens = []

    def append(new):
        K, V_, Q = m.kvq(new, range(len(tokens), len(tokens) + len(new)))
        kvp.seq_append(pool, seq, K, V_, len(new))
        tokens.extend(int(t) for t in new)
        return Q

    def held():
        K, V_, _ = m.kvq(tokens, range(len(tokens)))
        return K[0], V_[0]

    def windowed(Q, n):
        t, ln = kvp.kvp_gather_tables(pool, [seq], 32)
        ws = torch.empty(kvp.kvp_window_workspace_size(desc, t, ln, [n], WIN, SINKS), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(Q)
        kvp.paged_window_attention(Q, [n], k, v, t, ln, WIN, SINKS, desc, out, None, ws)
        p, j = np.arange(len(tokens) - n, len(tokens))[:, None], np.arange(len(tokens))
        see = torch.from_numpy((j <= p) & ((j > p - WIN) | (j < SINKS))).cuda()
        K, V_ = held()
        close(out[0], attend(K, V_, Q[0], see), V_)
        return out[0]

    # the prompt, in chunks
    prompt = g.integers(0, V, 150)
    for a, b in ((0, 70), (70, 71), (71, 150)):
        last = windowed(append(prompt[a:b]), b - a)[-1:]
    accepted_total = 0
    for step in range(6):
        # a draft tree after the context: the draft model is the target's
        # output, tempered
        n = 6
        parent = np.array([-1, 0, 0, 1, -1, 4], np.int32)
        root = m.probs(last)[0]
        draft_rows = torch.softmax(torch.log(root) * 0.7, -1).expand(n + 1, V).contiguous()
        gen = torch.Generator(device="cuda").manual_seed(step)
        drafts = torch.multinomial(draft_rows[parent + 1], 1, generator=gen)[:, 0].int()
        ctx = len(tokens)
        depth = [0] * n
        for i in range(n):
            depth[i] = 0 if parent[i] < 0 else depth[parent[i]] + 1
        Kd, Vd, Qd = m.kvq(drafts.cpu().numpy(), [ctx + x for x in depth])
        kvp.seq_append(pool, seq, Kd, Vd, n)
        t, _ = kvp.kvp_gather_tables(pool, [seq], 32)
        ws = torch.empty(kvp.kvp_verify_workspace_size(desc, t, [ctx], n), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(Qd), torch.empty(L, n, Hq, device="cuda")
        par = torch.from_numpy(parent).cuda()[None].contiguous()
        kvp.tree_verify_attention(Qd, par, n, k, v, t, [ctx], desc, out, lse, ws)
        target = torch.cat([root[None], m.probs(out[0])])[None].contiguous()
        u, un = torch.rand(1, n, generator=gen, device="cuda"), torch.rand(1, generator=gen, device="cuda")
        acc, cnt, nxt = (torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(3))
        kvp.kvp_draft_verify(target, draft_rows[None], par, drafts[None].contiguous(), u, un, acc, cnt, nxt)
        want = walk(target[0].cpu().numpy(), draft_rows.cpu().numpy(), parent, drafts.cpu().numpy(),
                    u[0].cpu().numpy(), un[0].cpu().numpy())
        assert (int(acc), int(cnt), int(nxt)) == want
        path = kvp.seq_accept_draft(pool, seq, ctx, parent, int(acc))
        assert len(path) == int(cnt)
        accepted_total += len(path)
        tokens.extend(int(drafts[i]) for i in path)
        assert kvp.seq_len(pool, seq) == len(tokens)
        # the sampled token: a decode step under the window
        last = windowed(append([int(nxt)]), 1)
    assert accepted_total > 0

    # the cache is cut back to the tokens that the last queries of attention
    # over all of it gave the most weight, and decoding goes on
    held_k, held_v = held()
    mass = torch.zeros(L, 1, Hkv, 512, device="cuda")
    prev, budget = None, 40
    for token in (3, 1, 4):
        Q = append([token])
        K, V_, _ = m.kvq([token], [len(tokens) - 1])
        held_k, held_v = torch.cat([held_k, K[0]]), torch.cat([held_v, V_[0]])
        t, ln = kvp.kvp_gather_tables(pool, [seq], 32)
        out, lse = torch.empty_like(Q), torch.empty(L, 1, Hq, device="cuda")
        ws = torch.empty(kvp.kvp_decode_workspace_size(desc, t, ln), dtype=torch.uint8, device="cuda")
        kvp.paged_decode_attention(Q, k, v, t, ln, desc, out, lse, ws)
        see = torch.ones(1, len(tokens), dtype=torch.bool, device="cuda")
        close(out[0], attend(held_k, held_v, Q[0], see), held_v)
        ws = torch.empty(kvp.kvp_mass_workspace_size(desc, t, ln), dtype=torch.uint8, device="cuda")
        kvp.kvp_attention_mass(Q, None, lse, k, t, ln, desc, 1.0, mass, prev, mass, ws)
        prev = [len(tokens)]
    # each query's weights sum to one for every query head
    total = mass[..., :len(tokens)].double().sum(-1)
    assert ((total - 3 * Hq // Hkv).abs() <= 1e-3 * total).all()
    kept = torch.empty(L, 1, Hkv, budget, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvp.seq_evict_workspace_size(pool, [seq], budget), dtype=torch.uint8, device="cuda")
    kvp.seq_evict(pool, [seq], mass, budget, SINKS, 8, kept, mass, ws)
    assert kvp.seq_len(pool, seq) == budget
    ix = kept[0, 0].long().t()[..., None].expand(-1, -1, d)
    held_k, held_v = held_k.gather(0, ix), held_v.gather(0, ix)
    Kn, Vn, Q = m.kvq([9], [len(tokens)])
    kvp.seq_append(pool, seq, Kn, Vn, 1)
    t, ln = kvp.kvp_gather_tables(pool, [seq], 32)
    out = torch.empty_like(Q)
    ws = torch.empty(kvp.kvp_decode_workspace_size(desc, t, ln), dtype=torch.uint8, device="cuda")
    kvp.paged_decode_attention(Q, k, v, t, ln, desc, out, None, ws)
    held_k, held_v = torch.cat([held_k, Kn[0]]), torch.cat([held_v, Vn[0]])
    close(out[0], attend(held_k, held_v, Q[0], torch.ones(1, budget + 1, dtype=torch.bool, device="cuda")), held_v)
    kvp.seq_free(pool, seq)
    assert kvp.kvp_free_block_count(pool) == NB
    kvp.kv_pool_destroy(pool)
