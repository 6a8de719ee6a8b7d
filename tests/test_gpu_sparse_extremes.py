"""Sparse attention where scores are very large, and where the scale is next to
nothing, by single rows, by tiles and on the tensor cores."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp
from test_gpu_sparse import Batch, like_neighbours, sparse_want

pytestmark = pytest.mark.gpu


def batch(how):
    if how == "single":
        return Batch([300, 500], None, (8, 2), 64, 16, seed=1, poison=False)
    if how == "tensor":
        return Batch([700, 400], [300, 350], (8, 2), 128, 16, L=2, seed=4, poison=False)
    S, heads, d = (120, (16, 4), 128) if how == "tile of 32" else (200, (4, 4), 64)
    g = np.random.default_rng(S)
    q_lens = [int(n) for n in g.integers(3, 6, S)]
    return Batch([int(n) for n in g.integers(60, 180, S)], q_lens, heads, d, 16, L=3, seed=2, poison=False)


def check(b, sel, scale, lse_rel):
    b.desc = kvp.AttnDesc(b.L, b.Hq, b.Hkv, b.d, b.bs, b.NB, scale, 0)
    out, lse = torch.full_like(b.q, 5.0), torch.full((b.L, b.T, b.Hq), 5.0, device="cuda")
    kvp.paged_sparse_attention(b.q, b.start, b.k, b.v, b.t, b.n, torch.from_numpy(sel).cuda(), b.desc, out, lse)
    want, want_lse, mag = sparse_want(b, sel, scale)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    # (the tolerance of ordinary scores: below, the weights are equal or far apart)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * mag).all()
    assert (np.abs(got_lse - want_lse) <= 2.0 ** -15 + lse_rel * np.abs(want_lse)).all()


HOW = ["single", "tile of 32", "tile of 16", "tensor"]


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("size", [1.0, 2.0 ** 10, 2.0 ** 13, 2.0 ** 14, 2.0 ** 15, 2.0 ** 17, 2.0 ** 20, 2.0 ** 30])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(how, size, sign):
    # keys along one direction, each token's a power of two of the next one's: a
    # row's scores are equal in every bit or a factor of two apart.  A sum of d
    # products of one sign has d / 16 accumulations of two units in the last place
    # (2^-22), and lse three roundings more
    b = batch(how)
    gen = torch.Generator(device="cuda").manual_seed(5)
    u = torch.randn(b.L, 1, b.Hkv, 1, b.d, generator=gen, device="cuda").bfloat16().float()
    b.k[:] = (size * u * 0.5 ** (torch.arange(b.bs, device="cuda") % 4)[:, None]).bfloat16()
    f = 0.5 + torch.rand(b.L, b.T, b.Hq, 1, generator=gen, device="cuda")
    b.q[:] = (sign * size * f * u[:, :, :, 0].repeat_interleave(b.Hq // b.Hkv, 2)).bfloat16()
    check(b, like_neighbours(b, 5), 0.125, (b.d / 16 + 1) * 2.0 ** -22)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("scale", [1e-30, 1e-37, 1e-38, 1e-39, 1e-42])
def test_scales_next_to_nothing(how, scale):
    b = batch(how)
    check(b, like_neighbours(b, 5), scale, 2.0 ** -22)
