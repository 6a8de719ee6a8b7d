"""Sliding-window attention with sink tokens against a plain 64-bit form."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_prefix_shared_decode_gb300 as kvp

pytestmark = pytest.mark.gpu


def case(d, G, Hkv, bs, L, lens, qlens, win, sinks, seed=0, scale=0.0, share=None, mul=1.0):
    """Inputs whose unwritten slots, and tokens that no query sees, are NaN.
    share: sequence 0's first `share` tokens (whole blocks) lead every table."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S = len(lens)
    nb = [-(-n // bs) for n in lens]
    NB, MB = sum(nb) + 2, max(1, max(nb))
    order = torch.randperm(NB, generator=torch.Generator().manual_seed(seed)).numpy().astype(np.int32)
    tables, at = np.full((S, MB), -1, np.int32), 0
    for s, m in enumerate(nb):
        tables[s, :m] = order[at:at + m]
        at += m
        if share and s:
            tables[s, :share // bs] = tables[0, :share // bs]
    k = torch.full((L, NB, Hkv, bs, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    v = k.clone()
    for s, n in enumerate(lens):
        lo = max(0, n - qlens[s] - win + 1) if qlens[s] else n
        pos = torch.cat([torch.arange(0, min(sinks, n) if qlens[s] else 0), torch.arange(max(lo, 0), n)]).unique().cuda()
        blk = torch.from_numpy(tables[s].astype(np.int64)).cuda()[pos // bs]
        new = torch.isnan(k[0, blk, 0, pos % bs, 0])          # shared slots are written once
        blk, off = blk[new], (pos % bs)[new]
        for t in (k, v):
            t[:, blk, :, off] = torch.randn(len(blk), L, Hkv, d, device="cuda", generator=gen).to(torch.bfloat16)
    T = sum(qlens)
    q = (torch.randn(L, T, G * Hkv, d, device="cuda", generator=gen) * mul).to(torch.bfloat16)
    return kvp.AttnDesc(L, G * Hkv, Hkv, d, bs, NB, scale, 1), q, k, v, tables


def plain(q, k, v, tables, lens, qlens, win, sinks, scale):
    L, T, Hq, d = q.shape
    _, _, Hkv, bs, _ = k.shape
    G, sc = Hq // Hkv, scale if scale > 0 else 1 / math.sqrt(d)
    out = torch.zeros(L, T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(L, T, Hq, dtype=torch.float64, device="cuda")
    vmax, at = 0.0, 0
    for s, (n, m) in enumerate(zip(lens, qlens)):
        if m == 0:
            continue
        pos = torch.arange(n, device="cuda")
        blk = torch.from_numpy(tables[s].astype(np.int64)).cuda()[pos // bs]
        K = k[:, blk, :, pos % bs].double()       # [n][L][Hkv][d]
        V = v[:, blk, :, pos % bs].double()
        p = torch.arange(n - m, n, device="cuda")[:, None]
        see = (pos <= p) & ((pos > p - win) | (pos < sinks))
        Q = q[:, at:at + m].double().view(L, m, Hkv, G, d)
        x = torch.einsum("lmhgd,nlhd->lmhgn", Q, K.nan_to_num()) * sc
        x = x.masked_fill(~see[None, :, None, None], -math.inf)
        z = torch.logsumexp(x, -1)
        out[:, at:at + m] = torch.einsum("lmhgn,nlhd->lmhgd", torch.exp(x - z[..., None]), V.nan_to_num()).reshape(L, m, Hq, d)
        lse[:, at:at + m] = z.reshape(L, m, Hq)
        vmax = max(vmax, float(V.nan_to_num().abs().max()))
        at += m
    return out, lse, vmax


def call(desc, q, qlens, k, v, tables, lens, win, sinks):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    n = kvp.kvp_window_workspace_size(desc, tables, lens, qlens, win, sinks)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    kvp.paged_window_attention(q, qlens, k, v, tables, lens, win, sinks, desc, out, lse, ws)
    torch.cuda.synchronize()
    assert kvp.kvp_device_error(ws) == 0
    return out, lse


def check(d, G, Hkv, bs, L, lens, qlens, win, sinks, none=False, scale=0.0, **kw):
    desc, q, k, v, tables = case(d, G, Hkv, bs, L, lens, qlens, win, sinks, scale=scale, **kw)
    desc.use_sharing = 0 if kw.get("share") == 0 else 1
    out, lse = call(desc, q, None if none else qlens, k, v, tables, lens, win, sinks)
    want, z, vmax = plain(q, k, v, tables, lens, qlens, win, sinks, scale)
    # P is rounded to bf16 (2^-9 of each p, so of sum p |v| <= max |v|) and so
    # is out (2^-9 of it); the rest is fp32: twice that covers everything
    err = (out.double() - want).abs()
    assert (err <= 2.0 ** -8 * (vmax + want.abs())).all(), float(err.max())
    # as a whole the roundings of P average out: 5e-3 is the bound of the
    # library's other attention calls
    assert float(err.norm() / want.norm().clamp(min=1e-30)) <= 5e-3
    assert (lse.double() - z).abs().max() <= 1e-3


DECODE = [
    ([1], 1, 0), ([1], 5, 3), ([2, 17, 64, 65], 1, 0), ([2, 17, 64, 65], 16, 1), ([100, 333, 1000, 15], 64, 4),
    ([100, 333, 1000, 15], 65, 0), ([500, 77], 1 << 30, 0), ([500, 77], 100, 1 << 30), ([900, 901, 902], 300, 129),
    ([5000], 4000, 4), ([12000, 700], 9000, 64),
]


@pytest.mark.parametrize("d,G,Hkv,bs,L", [(64, 8, 4, 16, 1), (128, 4, 2, 16, 2), (128, 1, 2, 32, 1), (64, 16, 1, 64, 1),
                                          (128, 7, 1, 128, 1)])
@pytest.mark.parametrize("lens,win,sinks", DECODE)
def test_decode(d, G, Hkv, bs, L, lens, win, sinks):
    check(d, G, Hkv, bs, L, lens, [1] * len(lens), win, sinks, none=True, seed=win % 97 + d)


@pytest.mark.parametrize("d,G,Hkv", [(64, 8, 2), (128, 4, 2), (128, 16, 1)])
@pytest.mark.parametrize("share", [256, 512])
@pytest.mark.parametrize("win,sinks", [(100, 4), (400, 33), (700, 0), (5000, 0)])
def test_decode_over_shared_blocks(d, G, Hkv, share, win, sinks):
    lens = [share + 1 + 53 * i for i in range(20)]
    check(d, G, Hkv, 16, 1, lens, [1] * 20, win, sinks, none=True, share=share, seed=win)


EXTEND = [
    ([5], [5], 3, 0), ([130], [130], 1, 0), ([200, 64, 1], [2, 64, 1], 50, 4), ([700], [300], 128, 5),
    ([300, 0, 40, 65], [1, 0, 40, 0], 64, 1), ([1000, 257], [513, 257], 1 << 30, 0), ([900], [257], 1, 1),
    ([2000, 333], [33, 7], 777, 65), ([1500], [1500], 100, 0), ([640], [640], 640, 640), ([9000], [70], 8500, 200),
    ([10000], [10], 1 << 30, 0),
]


@pytest.mark.parametrize("d,G,Hkv,bs", [(64, 8, 2, 16), (128, 4, 2, 16), (128, 1, 1, 32), (64, 3, 1, 64), (128, 64, 1, 128),
                                        (64, 2, 2, 256)])
@pytest.mark.parametrize("lens,qlens,win,sinks", EXTEND)
def test_extend(d, G, Hkv, bs, lens, qlens, win, sinks):
    check(d, G, Hkv, bs, 1, lens, qlens, win, sinks, seed=len(lens) + d + G)


def test_layers_scale_and_peaked_rows():
    check(128, 4, 2, 16, 3, [600, 90], [200, 1], 250, 7, scale=0.3, mul=4.0)
    check(64, 8, 2, 16, 3, [600, 90], [1, 1], 250, 7, scale=0.3, mul=4.0)


@pytest.mark.parametrize("win,sinks", [(2 ** 31 - 1, 0), (1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_longest_window_and_sinks(win, sinks):
    check(64, 8, 2, 16, 1, [700, 65], [300, 1], win, sinks)
    check(128, 4, 2, 16, 1, [700, 65], [1, 1], win, sinks)


SCORES = {   # of 320 keys, 64-token tiles
    "all far down": lambda j: -300,
    "all far up": lambda j: 300,
    "first tile far down": lambda j: -300 if j < 64 else 0,
    "second tile far down": lambda j: -300 if 64 <= j < 128 else 0,
    "odd tiles far down": lambda j: -200 if j // 64 % 2 else -3,
    "even tiles far down": lambda j: -3 if j // 64 % 2 else -200,
    "rising": lambda j: j - 250,
    "falling": lambda j: 100 - j,
    "around the bounds": lambda j: (-12, 22, -11, 23, -14)[j // 64],
    "down, then up": lambda j: -256 if j < 250 else 256,
}


@pytest.mark.parametrize("name", SCORES)
@pytest.mark.parametrize("d,m", [(64, 20), (64, 10), (128, 30), (128, 12)])
def test_prescribed_scores(name, d, m):
    """Rows whose scores lie far from 0 or jump between tiles, in units of one
    and of two row tiles."""
    n, G, bs = 320, 8, 16
    gen = torch.Generator(device="cuda").manual_seed(d)
    k = torch.zeros(1, n // bs, 1, bs, d, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(1, n // bs, 1, bs, d, device="cuda", generator=gen).to(torch.bfloat16)
    score = torch.tensor([float(SCORES[name](j)) for j in range(n)], device="cuda")
    k[0, :, 0, :, 0] = score.view(n // bs, bs).to(torch.bfloat16)
    q = torch.zeros(1, m, G, d, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1
    score = k[0, :, 0, :, 0].reshape(n).double()
    desc = kvp.AttnDesc(1, G, 1, d, bs, n // bs, 1.0, 1)
    tables = np.arange(n // bs, dtype=np.int32)[None]
    see = torch.arange(n, device="cuda") <= torch.arange(n - m, n, device="cuda")[:, None]
    for win, sinks in ((n, 0), (100, 70)):
        vis = see & ((torch.arange(n, device="cuda") > torch.arange(n - m, n, device="cuda")[:, None] - win)
                     | (torch.arange(n, device="cuda") < sinks))
        x = score.expand(m, n).masked_fill(~vis, -math.inf)
        want = torch.softmax(x, -1) @ v[0].double().view(n, d)
        ws = torch.empty(kvp.kvp_window_workspace_size(desc, tables, [n], [m], win, sinks), dtype=torch.uint8,
                         device="cuda")
        out, lse = torch.empty_like(q), torch.empty(1, m, G, device="cuda")
        kvp.paged_window_attention(q, [m], k, v, tables, [n], win, sinks, desc, out, lse, ws)
        assert kvp.kvp_device_error(ws) == 0
        # P and out in bf16 (2^-9 each, doubled); scores of up to 433 in base 2
        # round by 433 * 2^-24, which the lse carries
        err = (out[0].double() - want[:, None]).abs()
        assert (err <= 2.0 ** -8 * (v.double().abs().max() + want[:, None].abs())).all(), (win, float(err.max()))
        lw = torch.logsumexp(x, -1)[:, None]
        assert ((lse[0].double() - lw).abs() <= 2.0 ** -18 * (1 + lw.abs())).all(), win


def test_unshared_plan():
    check(64, 8, 2, 16, 1, [400, 300, 64], [1, 1, 1], 100, 20, share=0)


def test_whole_window_is_decode_attention():
    lens = [300, 64, 1000, 17]
    desc, q, k, v, tables = case(128, 4, 2, 16, 2, lens, [1] * 4, 1 << 30, 0)
    out, lse = call(desc, q, None, k, v, tables, lens, 1 << 30, 0)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(kvp.kvp_decode_workspace_size(desc, tables, lens), dtype=torch.uint8, device="cuda")
    kvp.paged_decode_attention(q, k, v, tables, lens, desc, o2, l2, ws)
    assert (out.float() - o2.float()).abs().max() <= 2.0 ** -7 and (lse - l2).abs().max() <= 1e-4


def test_no_lse_and_another_stream():
    lens, ql = [500, 200], [100, 3]
    desc, q, k, v, tables = case(128, 4, 2, 16, 1, lens, ql, 64, 4)
    want, _ = call(desc, q, ql, k, v, tables, lens, 64, 4)
    out = torch.zeros_like(q)
    ws = torch.empty(kvp.kvp_window_workspace_size(desc, tables, lens, ql, 64, 4), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kvp.paged_window_attention(q, ql, k, v, tables, lens, 64, 4, desc, out, None, ws)
    s.synchronize()
    assert torch.equal(out, want)


def test_capture_is_refused():
    lens = [40]
    desc, q, k, v, tables = case(64, 4, 1, 16, 1, lens, [1], 8, 0)
    out = torch.zeros_like(q)
    ws = torch.empty(kvp.kvp_window_workspace_size(desc, tables, lens, None, 8, 0), dtype=torch.uint8, device="cuda")
    g, x = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
    with torch.cuda.graph(g):
        x += 1
        with pytest.raises(kvp.KvpError) as e:
            kvp.paged_window_attention(q, None, k, v, tables, lens, 8, 0, desc, out, None, ws)
    assert e.value.code == kvp.KVP_ERR_STATE


@pytest.mark.parametrize("path", ["tc", "mma"])
def test_forced_kernels(path):
    """The same cases on one kernel alone (the switch is read once a process)."""
    code = ("import sys; sys.path.insert(0, 'tests'); import test_gpu_window as t\n"
            "for d, G, Hkv in ((64, 8, 2), (128, 4, 2)):\n"
            "    for lens, qlens, win, sinks in t.EXTEND[:9]: t.check(d, G, Hkv, 16, 1, lens, qlens, win, sinks)\n"
            "    t.check(d, G, Hkv, 16, 1, [257 + 53 * i for i in range(20)], [1] * 20, 100, 4, share=256)\n"
            "print('same')")
    r = subprocess.run([sys.executable, "-c", code], env={**os.environ, "KVP_ATTN_PATH": path}, capture_output=True,
                       text=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("d,lens,qlens", [(128, [3000, 900], [1, 1]), (64, [3000, 900, 70], [777, 1, 70]),
                                          (128, [3000, 900], [1000, 40])])
def test_twice_gives_the_same_bits(d, lens, qlens):
    desc, q, k, v, tables = case(d, 8, 2, 16, 2, lens, qlens, 500, 4)
    ws = torch.empty(kvp.kvp_window_workspace_size(desc, tables, lens, qlens, 500, 4), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(5):
        out = torch.full_like(q, 7.0)
        lse = torch.zeros(q.shape[:3], device="cuda")
        kvp.paged_window_attention(q, qlens, k, v, tables, lens, 500, 4, desc, out, lse, ws)
        first = first or (out, lse)
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])
