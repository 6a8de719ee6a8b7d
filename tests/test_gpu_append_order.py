"""Batched appends in which one sequence copies a shared page and another, cut
back in that page, writes in it: every cache holds what appends one after the
other leave."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu

L, BS, HKV, HQ, D = 2, 16, 2, 4, 64


class Pool:
    def __init__(self, fourbit, seqs=8, nb=64, seed=3):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.fourbit, self.nb = fourbit, nb
        desc = kvp.PoolDesc(L, nb, BS, HKV, D, seqs, 8, seed)
        zeros = lambda *sh: torch.zeros(sh, dtype=torch.uint8, device="cuda")
        if fourbit:
            self.store = [zeros(L, nb, HKV, BS, D // 2), zeros(L, nb, HKV, BS).view(torch.int8),
                          zeros(L, nb, HKV, BS, D // 2), zeros(L, nb, HKV, BS).view(torch.int8)]
            self.h = kvp.kv_pool_create_kv4(desc, *self.store)
        else:
            self.store = [torch.zeros(L, nb, HKV, BS, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            self.h = kvp.kv_pool_create(desc, *self.store)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda", dtype=torch.bfloat16)

    def rows(self, s):
        """What a sequence holds, per storage array."""
        t = torch.from_numpy(kvp.seq_block_table(self.h, s).astype(np.int64)).cuda()
        return [x[:, t].transpose(2, 3).flatten(1, 2)[:, :kvp.seq_len(self.h, s)].clone() for x in self.store]

    def family(self, kids, used, cut):
        """A sequence of `used` tokens, its forks, and a last one cut back to `cut`."""
        root = kvp.seq_alloc(self.h)
        kvp.seq_append(self.h, root, self.normal(L, used, HKV, D), self.normal(L, used, HKV, D), used)
        seqs = [root] + [kvp.seq_fork(self.h, root) for _ in range(kids)]
        if cut < used:
            kvp.seq_accept_draft(self.h, seqs[-1], cut, list(range(-1, used - cut - 1)), -1)
        return seqs


def append(p, how, seqs, ntoks, k, v):
    if how == "batch":
        kvp.seq_append_batch(p.h, seqs, ntoks, k, v)
    elif how == "rope":
        kvp.seq_append_rope(p.h, seqs, ntoks, k, v, kvp.rope_desc(D))
    else:
        q = p.normal(L, len(seqs), HQ, D)
        out = torch.empty_like(q)
        lse = torch.empty(L, len(seqs), HQ, device="cuda")
        ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
        desc = kvp.AttnDesc(L, HQ, HKV, D, BS, p.nb, 0.0, 0, int(p.fourbit))
        kvp.DecodeStep(p.h, seqs, 1, kvp.step_io(q, out, lse, k, v), desc, ws)()


def both(fourbit, how, kids, used, cut, order, ntoks):
    """The batch in one call, and its sequences one after the other in a pool
    of the same blocks (the same operator, so that bits are equal)."""
    rows = []
    for one_call in (True, False):
        p = Pool(fourbit, kids + 2, 2 * kids + 64)
        seqs = p.family(kids, used, cut)
        seqs = [seqs[i] for i in order]
        before = [p.rows(s) for s in seqs]
        T = sum(ntoks)
        k, v = p.normal(L, T, HKV, D), p.normal(L, T, HKV, D)
        torch.cuda.synchronize()
        n = kvp.kvp_kernel_launches()
        if one_call:
            append(p, how, seqs, ntoks, k, v)
            launches = kvp.kvp_kernel_launches() - n
        else:
            at = 0
            for s, m in zip(seqs, ntoks):
                append(p, "rope" if how == "rope" else "batch", [s], [m], k[:, at:at + m].contiguous(),
                       v[:, at:at + m].contiguous())
                at += m
        rows.append([p.rows(s) for s in seqs])
        # (what was there stays)
        for s, old in zip(seqs, before):
            for x, y in zip(p.rows(s), old):
                assert torch.equal(x[:, :y.shape[1]], y)
        kvp.kv_pool_destroy(p.h)
    for x, y in zip(*rows):
        for a, b in zip(x, y):
            assert torch.equal(a, b)
    return launches


@pytest.mark.parametrize("fourbit", [False, True])
@pytest.mark.parametrize("how", ["batch", "rope", "step"])
@pytest.mark.parametrize("used,cut", [(26, 22), (26, 17), (12, 1), (31, 25)])
@pytest.mark.parametrize("order", [[0, 1], [1, 0]])
def test_a_sequence_cut_back_in_a_shared_page(fourbit, how, used, cut, order):
    both(fourbit, how, 1, used, cut, order, [1, 1])


@pytest.mark.parametrize("fourbit", [False, True])
@pytest.mark.parametrize("how", ["batch", "rope"])
@pytest.mark.parametrize("ntoks", [[3, 40, 9], [1, 1, 20]])
@pytest.mark.parametrize("order", [[0, 1, 2], [2, 0, 1], [1, 2, 0]])
def test_several_tokens(fourbit, how, ntoks, order):
    both(fourbit, how, 2, 27, 20, order, ntoks)


@pytest.mark.parametrize("fourbit", [False, True])
@pytest.mark.parametrize("how", ["batch", "rope"])
def test_more_copies_than_a_launch_holds(fourbit, how):
    n = 700
    both(fourbit, how, n, 28, 20, list(range(n + 1)), [1] * (n + 1))


@pytest.mark.parametrize("fourbit", [False, True])
@pytest.mark.parametrize("how", ["batch", "rope"])
def test_copies_come_first_only_where_they_have_to(fourbit, how):
    assert both(fourbit, how, 1, 26, 22, [0, 1], [1, 1]) == 2
    assert both(fourbit, how, 1, 26, 22, [1, 0], [1, 1]) == 1       # the longer one goes on in the page, behind the copy
    assert both(fourbit, how, 1, 26, 26, [0, 1], [1, 1]) == 1
    assert both(fourbit, how, 1, 26, 22, [0, 1], [1, 0]) == 1
