"""The 8-bit cache's attention called again and again: outputs filled with other bits before each
call, on other streams, in graphs whose inputs change between replays; each call's result looked at."""
import math

import pytest
import torch

import _fp8_ref as R
import mxfp4_sparse_paged_gb300 as m
from test_gpu_fp8_kv import attention, clean, pool, tables  # noqa: F401 (clean: a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHAPES = [([70001], 1, 16, 1, None), ([40000, 3, 20000], 2, 16, 2, None), ([5000] * 3, 8, 32, 1, None),
          ([777], 1, 16, 1, None), ([3000, 0, 31, 500], 3, 24, 4, None), ([20000, 64, 0], 1, 16, 1, 16),
          ([9000, 257], 2, 40, 8, 5)]


def lists(lens, q, k):
    g = torch.Generator().manual_seed(k)
    out = []
    for L in lens:
        for j in range(q):
            n = max(0, (L - q + j) // 128 + 1) if L - q + j >= 0 else 0
            out.append(torch.randperm(n, generator=g)[:k].tolist() or [-1])
    return out


@pytest.mark.parametrize("lens,q,H,Hkv,k", SHAPES)
def test_every_call_writes_the_same_bits(lens, q, H, Hkv, k):
    """All of out and lse, NaN before each call, twenty times; each call's result is the first's."""
    out, lse, want, call = attention(lens, q, H, Hkv, seed=1, blocks=None if k is None else lists(lens, q, k))
    R.check_attention(out, lse, want)
    first = out.clone(), lse.clone()
    for i in range(20):
        out.fill_(math.nan)
        lse.fill_(math.nan)
        call()
        if i % 2:
            torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), i
    m.mx4_check_status()


def test_calls_on_two_streams_each_looked_at():
    """Two streams with a workspace each, twenty rounds; a copy of every round's result, NaN before it."""
    sides = [attention([9000, 30], 1, 16, 1, seed=20), attention([3000] * 5, 2, 20, 4, seed=21)]
    want = [(s[0].clone(), s[1].clone()) for s in sides]
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (s, (out, lse, _, call)) in enumerate(zip(streams, sides)):
            with torch.cuda.stream(s):
                out.fill_(math.nan)
                lse.fill_(math.nan)
                call()
                got[i].append((out.clone(), lse.clone()))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, w[0]) and torch.equal(b, w[1]) for a, b in g)
    m.mx4_check_status()


@pytest.mark.parametrize("k", [None, 3])
def test_replays_with_other_inputs(k):
    """A call on a side stream and a captured one: between replays the pages, scales, tables, lengths
    (to none and to the table's end), lists and queries become others."""
    q, H, Hkv, lens = 2, 16, 2, [600, 300]
    g = torch.Generator().manual_seed(19)
    _, P = tables(g, lens)
    new = lambda: (pool(g, P, Hkv, 118, 122), pool(g, P, Hkv, 118, 122), torch.randperm(P, generator=g)[:8].view(2, 4).to(torch.int32),
                   torch.randn((2 * q, H, 128), generator=g).to(torch.bfloat16))
    shapes = [t.to(DEV) for (a, b, t2, qq) in [new()] for t in (*a, *b, t2, qq)]
    kp, ks, vp, vs, table, qq = shapes
    sl = torch.zeros(2, dtype=torch.int32, device=DEV)
    idx = torch.full((2 * q, k or 1), -1, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(qq), torch.empty((2 * q, H), device=DEV)
    need = m.fp8_paged_decode_workspace(2 * q, q, H, Hkv) if k is None else m.fp8_block_decode_workspace(2 * q, k, H, Hkv)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def call():
        if k is None:
            m.fp8_paged_decode(qq, q, kp, vp, ks, vs, table, sl, 0.1, out, ws, lse=lse)
        else:
            m.fp8_block_decode(qq, q, kp, vp, ks, vs, table, sl, idx, 0.1, out, ws, lse=lse)

    def fill(lens):
        (a, b), (c, d), t, x = new()
        li = None if k is None else lists(lens, q, k)
        for dst, src in ((kp, a), (ks, b), (vp, c), (vs, d), (table, t), (qq, x), (sl, torch.tensor(lens, dtype=torch.int32))):
            dst.copy_(src)
        if li is not None:
            idx.copy_(torch.tensor([r + [-1] * (k - len(r)) for r in li], dtype=torch.int32))
        out.fill_(math.nan)
        lse.fill_(math.nan)
        return R.attend(x, q, R.values(a, b), R.values(c, d), t, lens, 0.1, li)

    want = fill([400, 37])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    R.check_attention(out, lse, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([100, 40], [512, 0], [0, 1], [300, 512], [0, 0], [33, 511]):
        want = fill(lens)
        graph.replay()
        R.check_attention(out, lse, want)
    m.mx4_check_status()


def test_two_graphs_share_a_workspace():
    """Two captured calls of different shapes over one workspace, replayed in turn on one stream."""
    shapes = [([9000, 30], 1, 16, 1), ([700, 64], 4, 20, 4)]
    ws = torch.empty(max(m.fp8_paged_decode_workspace(len(n) * q, q, H, Hkv) for n, q, H, Hkv in shapes),
                     dtype=torch.uint8, device=DEV)
    sides = []
    for lens, q, H, Hkv in shapes:
        g = torch.Generator().manual_seed(q)
        table, P = tables(g, lens)
        (kp, ks), (vp, vs) = pool(g, P, Hkv, 118, 122), pool(g, P, Hkv, 118, 122)
        x = torch.randn((len(lens) * q, H, 128), generator=g).to(torch.bfloat16)
        want = R.attend(x, q, R.values(kp, ks), R.values(vp, vs), table, lens, 0.1)
        args = [t.to(DEV) for t in (kp, vp, ks, vs, table, torch.tensor(lens, dtype=torch.int32))]
        qq, out, lse = x.to(DEV), torch.empty_like(x, device=DEV), torch.empty(x.shape[:2], device=DEV)
        m.fp8_paged_decode(qq, q, *args, 0.1, out, ws, lse=lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.fp8_paged_decode(qq, q, *args, 0.1, out, ws, lse=lse)
        sides.append((graph, out, lse, want, (args, qq)))
    for i in range(12):
        graph, out, lse, want, _ = sides[i % 2]
        out.fill_(math.nan)
        lse.fill_(math.nan)
        graph.replay()
        R.check_attention(out, lse, want)
    m.mx4_check_status()
