"""Beam selection whose new scores take the old ones' places."""
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,K,V", [(1, 4, 32000), (64, 8, 5000), (3, 128, 300), (200, 1, 40)])
def test_scores_in_place(G, K, V):
    gen = torch.Generator(device="cuda").manual_seed(G)
    x = torch.randn(G, K, V, generator=gen, device="cuda")
    cum = -10 * torch.rand(G, K, generator=gen, device="cuda")
    done = torch.rand(G, K, generator=gen, device="cuda") < 0.2
    ws = torch.empty(kvp.kvp_beam_workspace_size(G, K, V, K), dtype=torch.uint8, device="cuda")
    apart, rows, tokens = torch.empty_like(cum), *(torch.empty(G, K, dtype=torch.int32, device="cuda") for _ in range(2))
    kvp.kvp_beam_select(x, cum, done, 7, apart, rows, tokens, ws)
    r2, t2 = torch.empty_like(rows), torch.empty_like(tokens)
    for _ in range(5):
        here = cum.clone()
        kvp.kvp_beam_select(x, here, done, 7, here, r2, t2, ws)
        assert torch.equal(here, apart) and torch.equal(r2, rows) and torch.equal(t2, tokens)
