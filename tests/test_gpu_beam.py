"""Beam selection and state reordering against their definitions in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def want(x, cum, done, pad, n):
    """score, row, token by the definition; the order of equal scores too."""
    G, B, V = x.shape
    out = np.full((G, n), -np.inf), np.full((G, n), -1, np.int64), np.full((G, n), -1, np.int64)
    for g in range(G):
        found = []
        for b in range(B):
            if not np.isfinite(cum[g, b]):
                continue
            if done is not None and done[g, b]:
                found.append((-float(cum[g, b]), b, 0.0, pad))
                continue
            r = x[g, b].astype(np.float64)
            if np.isnan(r).any() or (r == np.inf).any() or (r == -np.inf).all():
                continue
            m = r.max()
            z = m + math.log(np.exp(r - m).sum())
            top = np.argsort(-r, kind="stable")[:n]
            found += [(-(float(cum[g, b]) - z + r[t]), b, -r[t], int(t)) for t in top if r[t] > -np.inf]
        for i, (s, b, _, t) in enumerate(sorted(found)[:n]):
            out[0][g, i], out[1][g, i], out[2][g, i] = -s, g * B + b, t
    return out


def run(x, cum, done, pad, n):
    G, B, V = x.shape
    os = torch.full((G, n), 3.0, device="cuda")
    orow, ot = (torch.full((G, n), 3, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.full((kvp.kvp_beam_workspace_size(G, B, V, n),), 255, dtype=torch.uint8, device="cuda")
    kvp.kvp_beam_select(x, cum, done, pad, os, orow, ot, ws)
    return os, orow, ot


def check(x, cum, done=None, pad=0, n=4):
    got = [y.cpu().numpy() for y in run(x, cum, done, pad, n)]
    w = want(x.float().cpu().numpy(), cum.cpu().numpy(), None if done is None else done.cpu().numpy(), pad, n)
    assert np.array_equal(got[1], w[1]) and np.array_equal(got[2], w[2])
    none = np.isneginf(w[0])
    assert np.array_equal(np.isneginf(got[0]), none)
    # the log-sum-exp's exponentials are fp32 (2^-22 of the sum), the score is
    # rounded to fp32 once (2^-24)
    assert (np.abs(got[0] - w[0])[~none] <= 2.0 ** -24 * np.abs(w[0][~none]) + 2.0 ** -21).all()


def inputs(G, B, V, dtype, seed=0, scale=2.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (scale * torch.randn((G, B, V), generator=gen, device="cuda")).to(dtype)
    return x, -20 - 4 * torch.rand((G, B), generator=gen, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,B,V,n", [(1, 1, 1, 1), (1, 4, 32000, 4), (3, 5, 50257, 10), (2, 8, 131072, 16), (4, 1, 7, 7), (1, 3, 5, 20),
                                     (2, 2, 8192, 128), (1, 2, 8193, 64), (1, 128, 300, 128), (40, 2, 1000, 3)])
def test_beam_select(dtype, G, B, V, n):
    check(*inputs(G, B, V, dtype), n=n)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties(dtype):
    # equal logits: the lower beam, then the lower token
    for V in (10, 300, 9000, 40000):
        x = torch.zeros(2, 3, V, device="cuda", dtype=dtype)
        cum = torch.tensor([[-1.0, -1.0, -0.5], [-2.0, -3.0, -3.0]], device="cuda")
        check(x, cum, n=8)
        check(x, cum, n=128)
        g = torch.Generator(device="cuda").manual_seed(V)
        check(torch.randint(0, 3, (2, 3, V), generator=g, device="cuda").to(dtype), cum, n=20)


def test_first_step_and_unused_beams():
    x, cum = inputs(2, 4, 1000, torch.float32)
    cum[:, 1:] = -math.inf          # one beam in use
    check(x, cum, n=8)
    cum[1, 0] = math.nan            # and none
    check(x, cum, n=8)
    cum[1, 0] = math.inf
    check(x, cum, n=8)


@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
def test_finished_beams(dtype):
    x, cum = inputs(3, 4, 500, torch.bfloat16)
    done = torch.tensor([[0, 1, 0, 0], [1, 1, 1, 1], [0, 0, 0, 1]], device="cuda").to(dtype)
    x[1] = math.nan                 # their logits are not read
    cum[0, 1] = -10.0
    check(x, cum, done, pad=499, n=6)


def test_masked_and_broken_logits():
    x, cum = inputs(4, 2, 9000, torch.float32)
    x[0, 0, 5:] = -math.inf         # five tokens allowed
    x[0, 1] = -math.inf             # none
    x[1, 0, 8999] = math.nan
    x[1, 1, 0] = math.inf
    x[2, :, 100:] = -math.inf
    x[3, 0] = torch.finfo(torch.float32).min
    x[3, 0, 17] = -1e30
    check(x, cum, n=9)
    # masks of the type's lowest value
    for t in TYPES:
        y = torch.full((1, 2, 300), torch.finfo(t).min, device="cuda", dtype=t)
        y[0, 1, 3] = 2.0
        check(y, torch.tensor([[-5.0, -6.0]], device="cuda"), n=12)


def test_large_logits_next_to_each_other():
    # the best ones in a few threads' hands
    x, cum = inputs(1, 2, 30000, torch.float32)
    x[0, 0, 1000:1400] = 20 + torch.arange(400, device="cuda") / 50
    x[0, 1, ::256] = 25.0
    check(x, cum, n=64)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_and_unaligned_rows(dtype):
    full, cum = inputs(2, 3, 1010, dtype)
    check(full[:, :, :1003], cum, n=6)             # a row stride that is no multiple of 16 bytes
    check(full[:, :, 1:1002], cum, n=6)            # rows that begin off a 16-byte boundary
    flat = full.view(6, 1010)[:, 3:500]
    check(flat.view(2, 3, 497), cum, n=6)


def test_same_row_for_all():
    x, cum = inputs(1, 1, 5000, torch.float32)
    one = x.expand(1, 3, 5000)
    os, orow, ot = (torch.empty(1, 4, device="cuda"), *(torch.empty(1, 4, dtype=torch.int32, device="cuda") for _ in range(2)))
    ws = torch.empty(kvp.kvp_beam_workspace_size(1, 3, 5000, 4), dtype=torch.uint8, device="cuda")
    cum = torch.tensor([[-1.0, -1.0, -1.0]], device="cuda")
    kvp.kvp_beam_select(one, cum, None, 0, os, orow, ot, ws)
    w = want(one.cpu().numpy(), cum.cpu().numpy(), None, 0, 4)
    assert np.array_equal(orow.cpu().numpy(), w[1]) and np.array_equal(ot.cpu().numpy(), w[2])


def test_captured():
    x, cum = inputs(2, 4, 20000, torch.bfloat16)
    n = 8
    os, orow, ot = (torch.empty(2, n, device="cuda"), *(torch.empty(2, n, dtype=torch.int32, device="cuda") for _ in range(2)))
    ws = torch.empty(kvp.kvp_beam_workspace_size(2, 4, 20000, n), dtype=torch.uint8, device="cuda")
    hist = torch.arange(8 * 33, dtype=torch.int32, device="cuda").view(8, 33)
    out = torch.zeros(16, 33, dtype=torch.int32, device="cuda")

    def step():
        kvp.kvp_beam_select(x, cum, None, 0, os, orow, ot, ws)
        kvp.kvp_state_reorder(hist, out, orow)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
        step()                      # the same workspace twice in one graph
    for seed in range(3):
        x.copy_(inputs(2, 4, 20000, torch.bfloat16, seed + 5)[0])
        g.replay()
        torch.cuda.synchronize()
        w = want(x.float().cpu().numpy(), cum.cpu().numpy(), None, 0, n)
        assert np.array_equal(orow.cpu().numpy(), w[1]) and np.array_equal(ot.cpu().numpy(), w[2])
        assert torch.equal(out, hist[orow.view(-1).long()])


def test_wrong_tensors_are_refused():
    x, cum = inputs(2, 3, 100, torch.float32)
    with pytest.raises(ValueError):
        run(x.double(), cum, None, 0, 4)
    with pytest.raises(ValueError):
        run(x, cum[:, :2].contiguous(), None, 0, 4)
    with pytest.raises(ValueError):
        run(x[:, :2], cum[:, :2].contiguous(), None, 0, 4)      # rows not evenly spaced
    with pytest.raises(ValueError):
        run(x[:, :, ::2], cum, None, 0, 4)
    with pytest.raises(ValueError):
        run(x, cum, torch.zeros(2, 3, device="cuda"), 0, 4)
    with pytest.raises(kvp.KvpError):
        kvp.kvp_beam_select(x, cum, None, 0, torch.empty(2, 4, device="cuda"),
                            *(torch.empty(2, 4, dtype=torch.int32, device="cuda") for _ in range(2)),
                            torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype,shape,dim,n_dst", [
    (torch.float32, (8, 100), 0, 8), (torch.int32, (5, 4097), 0, 10), (torch.bfloat16, (3, 6, 7), 1, 6),
    (torch.uint8, (2, 9, 13), 1, 4), (torch.float32, (2, 16, 4, 5000), 1, 16), (torch.int64, (1, 1), 0, 3),
    (torch.float32, (4, 70000), 0, 4)])
def test_state_reorder(dtype, shape, dim, n_dst):
    g = torch.Generator(device="cuda").manual_seed(1)
    src = torch.randint(0, 100, shape, generator=g, device="cuda").to(dtype)
    dst = torch.full((*shape[:dim], n_dst, *shape[dim + 1:]), 101, device="cuda").to(dtype)
    idx = torch.randint(0, shape[dim], (n_dst,), generator=g, device="cuda", dtype=torch.int32)
    idx[0] = -1
    if n_dst > 3:
        idx[3] = shape[dim]
        idx[2] = 2 ** 31 - 1
    w = dst.clone()
    for i, j in enumerate(idx.tolist()):
        if 0 <= j < shape[dim]:
            w.select(dim, i).copy_(src.select(dim, j))
    kvp.kvp_state_reorder(src, dst, idx, dim)
    assert torch.equal(dst, w)
    with pytest.raises(ValueError):
        kvp.kvp_state_reorder(src, dst, idx.repeat(2), dim)
    with pytest.raises(ValueError):
        kvp.kvp_state_reorder(src, dst, idx.long(), dim)


def test_state_reorder_unaligned():
    src = torch.arange(1000, dtype=torch.uint8, device="cuda")[1:901].view(9, 100)
    dst = torch.zeros(901, dtype=torch.uint8, device="cuda")[1:].view(9, 100)
    idx = torch.tensor([8, 7, 6, 5, 4, 3, 2, 1, 0], dtype=torch.int32, device="cuda")
    kvp.kvp_state_reorder(src, dst, idx)
    assert torch.equal(dst, src.flip(0))
