"""Page selection in tables of every width that has a kernel of its own: widths
on both sides of each limit, rows that fill the table and that do not, budgets
from one page to more than the row has."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu

BS = 16
LIMITS = [256, 1024, 2048, 4096, 8192, 32768]
WIDTHS = [2, 255] + [w + i for w in LIMITS for i in (0, 1)] + [50000]
KINDS = ["normal", "ties", "equal", "up", "down", "close", "wide", "odd", "negative", "two"]


def values(kind, n, g):
    if kind == "normal":
        return g.normal(size=n)
    if kind == "ties":          # zeros of both signs among few values
        return g.integers(-2, 3, n) * np.where(g.random(n) < 0.5, -1.0, 1.0)
    if kind == "equal":
        return np.full(n, -3.25)
    if kind == "up":
        return np.arange(n) * 0.5
    if kind == "down":
        return -np.arange(n) * 0.25
    if kind == "close":         # neighbours in fp32, equal in bf16
        return 1.0 + g.integers(0, 50, n) * 2.0 ** -23
    if kind == "wide":
        return g.normal(size=n) * 10.0 ** g.integers(-30, 30, n)
    if kind == "negative":      # below zero, where keys and numbers run against one another
        return -np.exp(4 * g.normal(size=n))
    if kind == "two":           # a few large ones, in one thread's places
        x = np.full(n, -1.0)
        x[::256] = 5.0 + g.integers(0, 3, len(x[::256]))
        return x
    x = g.normal(size=n)
    x[g.random(n) < 0.1] = np.nan
    x[g.random(n) < 0.1] = np.inf
    x[g.random(n) < 0.3] = -np.inf
    return x


def want(x, n, budget, sink, recent):
    """By the definition: the first and last pages, then the best, the lower
    page first among equal ones, a NaN above everything."""
    if n <= budget:
        return np.concatenate([np.arange(n), np.full(budget - n, -1)])
    mid = x[sink:n - recent].astype(np.float64)
    high = np.isnan(mid)
    order = np.lexsort((np.arange(len(mid)), -np.where(high, 0.0, mid), ~high))
    pick = np.sort(order[:budget - sink - recent]) + sink
    return np.concatenate([np.arange(sink), pick, np.arange(n - recent, n)])


def budgets(width):
    """(budget, sinks, last ones): small, around the threads of a kernel (128, 256,
    1024) and four times as many, and around the row's own length."""
    sizes = [1, 2, 9, 63, 128, 131, 257, 300, 519, 700, 1030, 1100, 2051, 4100, 4500, width // 2, width - 3, width - 1, width, width + 5]
    for b in sorted({s for s in sizes if 0 < s <= width + 5}):
        yield b, 0, 0
        if b > 3:
            yield b, 2, 1


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", KINDS)
def test_every_width(width, kind):
    g = np.random.default_rng(width)
    # pages that the rows see; the last one's length is cut to the table
    pages = sorted({max(1, p) for p in (width, width - 1, width - 2, width // 2, width // 3 + 1, 1, 40, 200)} & set(range(width + 1)))
    lens = [p * BS - int(g.integers(0, BS)) for p in pages] + [width * BS + 7]
    pages = pages + [width]
    x = np.stack([values(kind, width, g) for _ in pages])[None, :, None].astype(np.float32)     # [1][rows][1][width]
    dev, n = torch.from_numpy(x).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    desc = kvp.AttnDesc(1, 1, 1, 64, BS, 8, 0.0, 0)
    for budget, sink, recent in budgets(width):
        out = torch.full((1, len(pages), 1, budget), 77, dtype=torch.int32, device="cuda")
        kvp.kvp_page_select(dev, None, n, desc, sink, recent, out)
        got = out[0, :, 0].cpu().numpy()
        for i, p in enumerate(pages):
            assert np.array_equal(got[i], want(x[0, i, 0], p, budget, sink, recent)), (p, budget, sink, recent)


@pytest.mark.parametrize("width", [w + i for w in LIMITS for i in (0, 1)])
def test_rows_of_chunks_layers_and_heads(width):
    # several rows a sequence, rows behind the last one, scores wider than the table
    g = np.random.default_rng(width)
    L, H, q_lens = 2, 2, [3, 0, 5]
    lens = [width * BS, 100, (width // 2) * BS + 2]
    T, stride = sum(q_lens), width + 3
    x = g.normal(size=(L, T + 2, H, stride)).astype(np.float32)
    start = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda")
    budget, sink, recent = min(70, width // 3), 1, 2
    out = torch.full((L, T + 2, H, budget), 77, dtype=torch.int32, device="cuda")
    kvp.kvp_page_select(torch.from_numpy(x).cuda(), start, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                        kvp.AttnDesc(L, 4, H, 64, BS, 8, 0.0, 0), sink, recent, out, max_blocks=width)
    got, t = out.cpu().numpy(), 0
    for s, n in enumerate(q_lens):
        for i in range(n):
            p = (lens[s] - n + i) // BS + 1
            for l, h in np.ndindex(L, H):
                assert np.array_equal(got[l, t, h], want(x[l, t, h], p, budget, sink, recent)), (s, i, l, h)
            t += 1
    assert (got[:, T:] == 77).all()
