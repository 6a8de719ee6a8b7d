"""Sizes of beam selection that its 32-bit counts do not hold are refused, on
the host."""
import pytest

import paged_prefix_shared_decode_gb300 as kvp

A, B = 1 << 20, 1 << 24     # any aligned addresses: nothing here reaches the device


@pytest.mark.parametrize("G,K,V,n", [
    (2 ** 25, 128, 100, 4),             # 2^32 rows
    (2 ** 31 - 1, 128, 100, 4), (2 ** 26, 64, 100, 4), (2 ** 31 - 1, 3, 100, 4), (2 ** 24, 128, 100, 4),
    (2 ** 22, 128, 131072, 4),          # rows that fit, chunks that do not
    (1, 128, 2 ** 30 + 1, 4), (1, 1, 2 ** 31 - 1, 1), (2, 128, 2 ** 30, 128)])
def test_rows_and_chunks_beyond_32_bits(G, K, V, n):
    lib = kvp.load()
    assert lib.kvp_beam_workspace_size(G, K, V, n) == 0
    with pytest.raises(kvp.KvpError):
        kvp.kvp_beam_workspace_size(G, K, V, n)
    assert lib.kvp_beam_select(A, 0, V, A, None, 0, G, K, V, n, B, B, B, A, 2 ** 63, None) == kvp.KVP_ERR_INVALID


@pytest.mark.parametrize("G,K,V,n", [(2 ** 23, 128, 100, 4), (2 ** 31 - 1, 1, 8184, 1), (1, 128, 2 ** 25, 128)])
def test_the_largest_sizes_have_a_workspace(G, K, V, n):
    # a head of 16 bytes and n candidates of 8 for every row and chunk of 8184
    assert kvp.kvp_beam_workspace_size(G, K, V, n) == G * K * -(-V // 8184) * (16 + 8 * n)


def select(scores=A, done=None, K=4, n=4, out=B, rows=B + 4096, tokens=B + 8192, G=3):
    return kvp.load().kvp_beam_select(A, 0, 100, scores, done, 0, G, K, 100, n, out, rows, tokens, A, 1 << 20, None)


@pytest.mark.parametrize("bad", [
    dict(scores=B, n=5), dict(scores=B, n=3), dict(scores=B, K=5),      # in place, but not as many as beams
    dict(scores=B + 4), dict(scores=B + 44), dict(scores=B - 44),       # overlaps without being it
    dict(scores=B + 4096), dict(scores=B + 8192), dict(scores=B + 4096, rows=B + 4096, out=B + 4096),
    dict(done=B), dict(done=B + 47), dict(done=B - 11), dict(done=B + 4096), dict(done=B + 8200)])
def test_results_over_inputs_that_are_still_read(bad):
    assert select(**bad) == kvp.KVP_ERR_INVALID
