"""The 8-bit K/V cache on the GPU: append with the turn, attention, block scores, block choice,
each against 64-bit plain forms (tests/_fp8_ref.py), and a step of them together."""
import math

import numpy as np
import pytest
import torch

import _fp8_ref as R
import mxfp4_sparse_paged_gb300 as m

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64, E4M3 = torch.float64, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def clean():
    try:
        m.mx4_check_status()
    except m.Mx4Error:  # left by a test before
        pass
    yield
    torch.cuda.synchronize()


def flagged(bits):
    with pytest.raises(m.Mx4Error) as e:
        m.mx4_check_status()
    assert e.value.bits == bits, hex(e.value.bits)


def tables(g, lens, spare=2, width=None):
    n = [max(0, -(-L // 128)) for L in lens]
    P = sum(n) + spare
    perm = torch.randperm(P, generator=g)
    t = torch.full((len(lens), width or max(1, max(n))), -1, dtype=torch.int32)
    o = 0
    for s, k in enumerate(n):
        t[s, :k] = perm[o:o + k].to(torch.int32)
        o += k
    return t, P


def pool(g, P, Hkv, lo=110, hi=126):
    """Random rows and scales; no NaN code."""
    x = torch.randn((P, Hkv, 16384), generator=g).mul_(100).clamp_(-448, 448)
    return x.to(E4M3).view(torch.uint8), torch.randint(lo, hi, (P, Hkv, 4), generator=g, dtype=torch.uint8)


def poison(pages, scales, table, lens):
    """What no token has written: NaN codes past a length, NaN scales of blocks past it."""
    for s, L in enumerate(lens):
        if L > 0 and L % 128:
            p = table[s, L // 128]
            pages[p].view(-1, 128, 128)[:, L % 128:] = 255
            scales[p][:, -(-(L % 128) // 32):] = 255


# ------------------------------------------------------------------ attention

def attention(lens, q_per_seq, H, Hkv, seed=0, blocks=None, edit=None, scale=1 / math.sqrt(128),
              klo=118, khi=122, vlo=112, vhi=124, strided=False):
    g = torch.Generator().manual_seed(seed)
    table, P = tables(g, lens)
    kp, ks = pool(g, P, Hkv, klo, khi)
    vp, vs = pool(g, P, Hkv, vlo, vhi)
    poison(kp, ks, table, lens)
    poison(vp, vs, table, lens)
    T = len(lens) * q_per_seq
    q = torch.randn((T, H, 128), generator=g).mul_(2).to(torch.bfloat16)
    if edit:
        edit(q, kp, ks, vp, vs, table)
    want = R.attend(q, q_per_seq, R.values(kp, ks), R.values(vp, vs), table,
                    lens, scale, blocks)
    dk, dv = kp.to(DEV), vp.to(DEV)
    if strided:
        big = torch.full((2, P, Hkv + 1, 16384 + 16), 255, dtype=torch.uint8, device=DEV)
        big[0, :, :Hkv, :16384], big[1, :, :Hkv, :16384] = dk, dv
        dk, dv = big[0, :, :Hkv, :16384], big[1, :, :Hkv, :16384]
    out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, H), 7.0, device=DEV)
    args = (dk, dv, ks.to(DEV), vs.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    if blocks is None:
        ws = torch.empty(m.fp8_paged_decode_workspace(T, q_per_seq, H, Hkv), dtype=torch.uint8, device=DEV)
        call = lambda: m.fp8_paged_decode(q.to(DEV), q_per_seq, *args, scale, out, ws, lse=lse)
    else:
        k = max(len(x) for x in blocks)
        idx = torch.tensor([x + [-1] * (k - len(x)) for x in blocks], dtype=torch.int32, device=DEV)
        ws = torch.empty(m.fp8_block_decode_workspace(T, k, H, Hkv), dtype=torch.uint8, device=DEV)
        call = lambda: m.fp8_block_decode(q.to(DEV), q_per_seq, *args, idx, scale, out, ws, lse=lse)
    call()
    return out, lse, want, call


LENS = [0, 1, 2, 31, 32, 33, 127, 128, 129, 160, 500, 1500]


@pytest.mark.parametrize("q,H,Hkv", [(1, 1, 1), (1, 16, 1), (1, 40, 8), (1, 128, 8), (2, 7, 1), (3, 24, 4),
                                     (4, 20, 4), (8, 16, 2), (8, 128, 1), (5, 128, 2), (1, 128, 1)])
def test_paged_decode(q, H, Hkv):
    out, lse, want, _ = attention(LENS, q, H, Hkv, seed=q * 1000 + H)
    R.check_attention(out, lse, want)
    m.mx4_check_status()


@pytest.mark.parametrize("lens,q,H,Hkv", [([70001], 1, 16, 1), ([40000, 3, 20000], 2, 16, 2), ([9000], 4, 32, 1),
                                          ([5000] * 3, 8, 32, 1)])
def test_paged_decode_long(lens, q, H, Hkv):
    """Tiles cut over many CTAs."""
    out, lse, want, call = attention(lens, q, H, Hkv, seed=3)
    R.check_attention(out, lse, want)
    first, first_lse = out.clone(), lse.clone()
    call()  # joined in a fixed order: the same bits again
    assert torch.equal(first, out) and torch.equal(first_lse, lse)
    m.mx4_check_status()


def test_paged_decode_many_sequences():
    """More sequences than a launch takes, most of them short."""
    g = np.random.default_rng(0)
    lens = g.integers(0, 40, 2100).tolist()
    lens[2047:2050] = [300, 0, 200]
    out, lse, want, _ = attention(lens, 1, 4, 2, seed=5)
    R.check_attention(out, lse, want)


def test_paged_decode_strided_pools():
    out, lse, want, _ = attention([200, 129, 5], 2, 8, 2, seed=6, strided=True)
    R.check_attention(out, lse, want)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_paged_decode_scales(scale):
    out, lse, want, _ = attention([700, 64], 1, 16, 1, seed=7, scale=scale)
    R.check_attention(out, lse, want)


def test_paged_decode_wide_scales():
    """Blocks whose V scales lie 2^100 apart; K scales that make rows of tiny and of huge logits."""
    out, lse, want, _ = attention([300, 40], 1, 16, 1, seed=8, vlo=60, vhi=160)
    R.check_attention(out, lse, want)
    out, lse, want, _ = attention([300, 40], 1, 16, 1, seed=9, klo=1, khi=100)
    R.check_attention(out, lse, want)

    def big(q, kp, ks, vp, vs, table):
        ks[:] = 130  # logits of thousands: one token holds the row
        vs[:] = 0    # scale 2^-127
    out, lse, want, _ = attention([300, 40], 1, 16, 1, seed=10, edit=big)
    R.check_attention(out, lse, want)


@pytest.mark.parametrize("q,H", [(3, 8), (5, 8), (4, 16), (6, 16), (8, 16), (3, 64)])
def test_paged_decode_wide_scales_and_nan_many_rows(q, H):
    """24 to 192 rows a sequence, in one to eight warps a tile: V scales 2^100 apart, and NaN values and
    scales that only the last queries see."""
    out, lse, want, _ = attention([300, 41, 700], q, H, 1, seed=20 + q, vlo=60, vhi=160)
    R.check_attention(out, lse, want)

    def edit(qq, kp, ks, vp, vs, table):
        vp[table[0, 2]].view(1, 128, 128)[0, 299 - 256, 17] = 0x7F   # the last token
        vp[table[1, 0]].view(1, 128, 128)[0, 97, 100] = 0xFF         # the one before it, of 99
        vs[table[2, 1], 0, 0] = 255                                  # tokens 128 .. 129 of 130
    out, lse, want, _ = attention([300, 99, 130], q, H, 1, seed=30 + q, edit=edit)
    o = torch.isnan(out.cpu().float()).view(3, q, H, 128)
    assert o[0, -1, :, 17].all() and int(o[0].sum()) == H
    assert o[1, -2:, :, 100].all() and int(o[1].sum()) == 2 * H
    assert o[2, -2:].all() and int(o[2].sum()) == 2 * H * 128
    ok = ~torch.isnan(want[0]).any(-1).reshape(-1)
    fin = [w.flatten(0, 1)[ok] if w.dim() == 3 else w.reshape(-1)[ok] for w in want]
    R.check_attention(out.flatten(0, 1)[ok.to(DEV)], lse.reshape(-1)[ok.to(DEV)], fin)


def test_paged_decode_large_and_small_queries():
    def edit(q, kp, ks, vp, vs, table):
        q[0] *= 2.0**90
        q[1] *= 2.0**-80
        ks[table[0, 0]], ks[table[1, 0]] = 127 - 96, 127 + 70
        q[2, 3] = 0
    out, lse, want, _ = attention([100, 100, 100], 1, 16, 1, seed=11, edit=edit)
    R.check_attention(out, lse, want)


def test_paged_decode_nan_stays_where_it_is_seen():
    """A NaN key or value of the last tokens reaches only the rows that see it."""
    def edit(q, kp, ks, vp, vs, table):
        rows = vp[table[0, 2]].view(1, 128, 128)
        rows[0, 299 - 256, 17] = 0x7F          # token 299 of 300: the last query alone
        rows[0, 298 - 256, 100] = 0xFF         # token 298: the last two
        kp[table[1, 0]].view(1, 128, 128)[0, 97, 3] = 0x7F  # token 97 of 99: the last two queries
        vs[table[2, 1], 0, 0] = 255            # tokens 128 .. 129 of 130: the scale is NaN
    out, lse, want, _ = attention([300, 99, 130], 4, 16, 1, seed=12, edit=edit)
    o = torch.isnan(out.cpu().float()).view(3, 4, 16, 128)
    assert o[0, 3, :, 17].all() and o[0, 2:, :, 100].all() and int(o[0].sum()) == 16 * 3
    assert o[1, 2:].all() and not o[1, :2].any() and o[2, 2:].all() and not o[2, :2].any()
    ok = ~torch.isnan(want[1]).reshape(-1)
    fin = [w.flatten(0, 1)[ok] if w.dim() == 3 else w.reshape(-1)[ok] for w in want]
    R.check_attention(out.flatten(0, 1)[ok.to(DEV)], lse.reshape(-1)[ok.to(DEV)], fin)


def test_paged_decode_bad_data():
    """A page id outside the pool and lengths outside the table are reported, nothing else moves."""
    g = torch.Generator().manual_seed(13)
    lens = [300, 200, 100]
    table, P = tables(g, lens)
    kp, ks = pool(g, P, 1, 118, 122)
    vp, vs = pool(g, P, 1, 118, 122)
    q = torch.randn((3, 16, 128), generator=g).to(torch.bfloat16)
    ws = torch.empty(m.fp8_paged_decode_workspace(3, 1, 16, 1), dtype=torch.uint8, device=DEV)
    for page, lens2, bits in ((P, lens, 0x2), (-1, lens, 0x2), (None, [300, -1, 100], 0x4),
                              (None, [300, 385, 100], 0x4)):
        t = table.clone()
        if page is not None:
            t[1, 0] = page
        out = torch.full((3, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((3, 16), 7.0, device=DEV)
        m.fp8_paged_decode(q.to(DEV), 1, kp.to(DEV), vp.to(DEV), ks.to(DEV), vs.to(DEV), t.to(DEV),
                           torch.tensor(lens2, dtype=torch.int32, device=DEV), 0.1, out, ws, lse=lse)
        flagged(bits)
        if page is not None:  # the page's tokens are skipped: the rest is those of block 1
            blocks = [[0, 1, 2], [1], [0]]
            want = R.attend(q, 1, R.values(kp, ks), R.values(vp, vs), table, lens, 0.1, blocks)
        else:
            want = R.attend(q, 1, R.values(kp, ks), R.values(vp, vs), table, [300, 0, 100], 0.1)
        R.check_attention(out, lse, want)


def test_block_decode_lists():
    """Lists in any order, a block twice, padding anywhere, the token's own block, none at all."""
    lens = [1500, 1500, 129, 64, 0, 700]
    blocks = [[3, 0, 11, 7], [5, 5, 2], [-1, 1, -1, 0], [0], [-1], [-1, -1]]
    out, lse, want, _ = attention(lens, 1, 20, 4, seed=14, blocks=blocks)
    R.check_attention(out, lse, want)
    m.mx4_check_status()


@pytest.mark.parametrize("q,H,Hkv,k", [(1, 16, 1, 16), (3, 32, 2, 5), (8, 128, 1, 3), (2, 40, 8, 64)])
def test_block_decode(q, H, Hkv, k):
    r = np.random.default_rng(k)
    lens = [10000, 9000, 257, 30, 2]
    blocks = []
    for L in lens:
        for j in range(q):
            p = L - q + j
            n = p // 128 + 1 if p >= 0 else 0
            blocks.append(sorted(r.choice(n, min(n, k), replace=False).tolist()) if n else [-1])
    out, lse, want, call = attention(lens, q, H, Hkv, seed=15, blocks=blocks)
    R.check_attention(out, lse, want)
    first = out.clone()
    call()
    assert torch.equal(first, out)
    m.mx4_check_status()


def test_block_decode_all_blocks_are_the_dense_result():
    lens = [1000, 129, 3]
    a = attention(lens, 2, 16, 1, seed=16)
    b = attention(lens, 2, 16, 1, seed=16, blocks=[list(range(8))] * 2 + [[0], [0, 1]] + [[0]] * 2)
    R.check_attention(b[0], b[1], a[2])


def test_block_decode_bad_index():
    lens = [300, 300]
    out, lse, want, _ = attention(lens, 1, 16, 1, seed=17, blocks=[[0, 3], [2147483647, 2]])
    flagged(0x8)
    R.check_attention(out, lse, want)


def test_decode_in_a_graph_and_on_a_stream():
    """Captured: lengths that grow between replays, other values in the same pages."""
    out, lse, _, _ = attention([600, 300], 1, 16, 2, seed=18)
    g = torch.Generator().manual_seed(19)
    table, P = tables(g, [600, 300])
    kp, ks = (x.to(DEV) for x in pool(g, P, 2, 118, 122))
    vp, vs = (x.to(DEV) for x in pool(g, P, 2, 118, 122))
    q = torch.randn((2, 16, 128), generator=g).to(torch.bfloat16).to(DEV)
    lens = torch.tensor([100, 40], dtype=torch.int32, device=DEV)
    ws = torch.empty(m.fp8_paged_decode_workspace(2, 1, 16, 2), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((2, 16), device=DEV)
    td = table.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.fp8_paged_decode(q, 1, kp, vp, ks, vs, td, lens, 0.1, out, ws, lse=lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.fp8_paged_decode(q, 1, kp, vp, ks, vs, td, lens, 0.1, out, ws, lse=lse)
        lens.add_(100)
    for L in ([100, 40], [200, 140], [300, 240]):
        graph.replay()
        want = R.attend(q.cpu(), 1, R.values(kp.cpu(), ks.cpu()), R.values(vp.cpu(), vs.cpu()), table, L, 0.1)
        R.check_attention(out, lse, want)


def test_nothing_cached_and_full_tables():
    """Empty sequences alone, and lengths that fill the table to its last token; no lse."""
    for lens in ([0, 0, 0], [384, 384]):
        out, lse, want, _ = attention(lens, 3, 16, 2, seed=30)
        R.check_attention(out, lse, want)
    g = torch.Generator().manual_seed(31)
    table, P = tables(g, [384])
    kp, ks = (x.to(DEV) for x in pool(g, P, 1))
    q = torch.randn((1, 16, 128), generator=g).to(torch.bfloat16).to(DEV)
    ws = torch.empty(m.fp8_paged_decode_workspace(1, 1, 16, 1), dtype=torch.uint8, device=DEV)
    outs = []
    for lse in (torch.empty((1, 16), device=DEV), None):
        out = torch.empty_like(q)
        m.fp8_paged_decode(q, 1, kp, kp, ks, ks, table.to(DEV), torch.tensor([384], dtype=torch.int32, device=DEV),
                           0.1, out, ws, lse=lse)
        outs.append(out)
    assert torch.equal(*outs)
    m.mx4_check_status()


def test_two_streams_at_once():
    """Calls on two streams with a workspace each, again and again: the bits of calls one by one."""
    a = attention([9000, 30], 1, 16, 1, seed=20)
    b = attention([3000] * 5, 2, 20, 4, seed=21)
    wa, wb = (a[0].clone(), a[1].clone()), (b[0].clone(), b[1].clone())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a[3]()
        with torch.cuda.stream(s2):
            b[3]()
    torch.cuda.synchronize()
    assert torch.equal(a[0], wa[0]) and torch.equal(a[1], wa[1])
    assert torch.equal(b[0], wb[0]) and torch.equal(b[1], wb[1])


def test_pages_past_32_bits():
    """Pages whose bytes lie past 2^32 in the pool: append there and read back."""
    g = torch.Generator().manual_seed(22)
    P = (1 << 32) // 16384 + 100
    kp, vp = (torch.empty((P, 1, 16384), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((P, 1, 4), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    L = 300
    table = torch.tensor([[P - 1, P - 77, P - 3]], dtype=torch.int32)
    i = dict(dtype=torch.int32, device=DEV)
    k, v = (torch.randn((L, 1, 128), generator=g).to(torch.bfloat16) for _ in range(2))
    m.fp8_rope_append(None, k.to(DEV), v.to(DEV), torch.tensor([0, L], **i), table.to(DEV), torch.tensor([L], **i),
                      kp, vp, ks, vs, None)
    q = torch.randn((1, 16, 128), generator=g).to(torch.bfloat16)
    out, lse = torch.empty((1, 16, 128), dtype=torch.bfloat16, device=DEV), torch.empty((1, 16), device=DEV)
    ws = torch.empty(m.fp8_paged_decode_workspace(1, 1, 16, 1), dtype=torch.uint8, device=DEV)
    m.fp8_paged_decode(q.to(DEV), 1, kp, vp, ks, vs, table.to(DEV), torch.tensor([L], **i), 0.1, out, ws, lse=lse)
    at = table[0].long().to(DEV)
    rows = [R.values(x[at].cpu(), y[at].cpu()) for x, y in ((kp, ks), (vp, vs))]
    small = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    R.check_attention(out, lse, R.attend(q, 1, *rows, small, [L], 0.1))
    # stored values: within half a step of E4M3 (2^-4 of the value, 2^-10 of the scale) of the rows
    got = rows[1][:, 0].reshape(-1, 128)[:L]
    scale = torch.pow(2.0, vs[at].cpu().double() - 127).view(-1)[:, None].repeat_interleave(32, 0)[:L]
    assert ((got - v[:, 0].double()).abs() <= v[:, 0].double().abs() * 2.0**-4 + scale * 2.0**-10).all()
    m.mx4_check_status()


# ------------------------------------------------------------------ append

def append(lens, new, H, Hkv, dtype, rot, inter, seed, factor=1.0, shift=None, pad=0, fused=True, edit=None):
    """One append against the definition: q_out and every byte of the pools."""
    g = torch.Generator().manual_seed(seed)
    table, P = tables(g, lens)
    kp, ks = pool(g, P, Hkv, 100, 124)
    vp, vs = pool(g, P, Hkv, 100, 124)
    T = sum(new) + pad
    x = torch.randn((T, (H + 2 * Hkv) * 128), generator=g)
    x *= torch.exp2(torch.randint(-3, 6, (T, 1), generator=g))
    x = x.to(dtype)
    if edit:
        edit(x, kp, ks, vp, vs, table)
    parts = [t.unflatten(1, (-1, 128)) for t in x.split([H * 128, Hkv * 128, Hkv * 128], 1)]
    freq, _ = m.rope_frequencies(rot) if rot else (None, 1)
    ph = m.rope_phases(freq) if rot else None
    cu = np.concatenate([[0], np.cumsum(new)])
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)] + [np.zeros(pad)]).astype(np.int64)
    use = pos if shift is None else pos + shift
    d = [t.to(DEV) for t in parts]
    if fused:
        fx = x.to(DEV)
        d = [t.unflatten(1, (-1, 128)) for t in fx.split([H * 128, Hkv * 128, Hkv * 128], 1)]
    dk, dv, dks, dvs = kp.to(DEV), vp.to(DEV), ks.to(DEV), vs.to(DEV)
    qo = torch.full((T, H, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    m.fp8_rope_append(*d, torch.tensor(cu, dtype=torch.int32, device=DEV), table.to(DEV),
                      torch.tensor(lens, dtype=torch.int32, device=DEV), dk, dv, dks, dvs, qo,
                      phases=None if ph is None else ph.to(DEV),
                      positions=None if shift is None else torch.tensor(use, device=DEV),
                      interleaved=inter, factor=factor)
    n = sum(new)
    phl = None if ph is None else ph.tolist()
    # the turn in fp32: angles to 2^-24 of half a turn and sines to 2 ulp, two products and a sum
    # (the magnitude of the pair times 2^-21 holds all of it)
    q, k, v = (t[:n].double() for t in parts)
    yq, yk = (R.turned(t, use[:n], phl, inter, factor) for t in (q, k))
    bq, bk = (band(t, rot, inter, factor) for t in (q, k))
    got = qo.cpu()
    assert (got[n:] == 9).all()
    # (bf16 keeps 8 bits: half a step is up to 2^-8 of the value, as at 64.25 between 64 and 64.5)
    assert ((got[:n].double() - yq).abs() <= 2.0**-8 * yq.abs() + 1.01 * bq).all()
    check_pool(dk.cpu(), dks.cpu(), kp, ks, yk, bk, table, lens, new)
    check_pool(dv.cpu(), dvs.cpu(), vp, vs, v, torch.zeros_like(v), table, lens, new)


def band(x, rot, inter, factor):
    y = x.abs().clone()
    if rot == 0:
        return torch.zeros_like(y)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    y[..., a] = y[..., b] = x.abs()[..., a] + x.abs()[..., b]
    y[..., rot:] = 0
    return y * 2.0**-21 * max(1.0, abs(factor))


def check_pool(pages, scales, before, before_scales, rows, bands, table, lens, new):
    """rows float64 [n, Hkv, 128], right to bands.  Scales: the exponent of the block's largest, or of
    a value within the band.  New codes: within half a step (and the band) of the row.  Stored rows:
    the nearest codes at the new scale, bit for bit.  All other bytes: as before."""
    P, Hkv = pages.shape[:2]
    want, want_s = before.clone().view(P, Hkv, 128, 128), before_scales.clone()
    got = pages.view(P, Hkv, 128, 128)
    at = 0
    for s, (L, n) in enumerate(zip(lens, new)):
        p = L - n
        while p < L:
            cnt, r0 = min(L - p, 32 - p % 32), p % 128
            page, sub, st = int(table[s, p // 128]), p % 128 // 32, p % 32
            x, b = rows[at:at + cnt], bands[at:at + cnt]
            for h in range(Hkv):
                old = int(before_scales[page, h, sub])
                old = -127 if old == 255 else old - 127
                lo, hi = (R.exponent(float((x[:, h].abs() + sg * b[:, h]).clamp_min(0).max())) for sg in (-1, 1))
                if st:
                    lo, hi = max(lo, old), max(hi, old)
                e = int(scales[page, h, sub]) - 127
                assert lo <= e <= hi, (s, p, h, lo, e, hi)
                want_s[page, h, sub] = e + 127
                if st and e > old:
                    c = want[page, h, r0 - st:r0].contiguous()
                    y = torch.ldexp(c.view(E4M3).double(), torch.tensor(old - e)).float()
                    want[page, h, r0 - st:r0] = y.to(E4M3).view(torch.uint8)
                code = got[page, h, r0:r0 + cnt]
                y = torch.ldexp(code.contiguous().view(E4M3).double(), torch.tensor(e))
                step = torch.maximum(x[:, h].abs() * 2.0**-4, torch.tensor(2.0**(e - 10), dtype=F64))
                assert ((y - x[:, h]).abs() <= step + 2 * b[:, h]).all(), (s, p, h)
                exact = torch.ldexp(x[:, h], torch.tensor(-e)).float().to(E4M3).view(torch.uint8)
                if not b.any():
                    assert torch.equal(code, exact)
                else:  # only values next to a border may differ
                    assert (code != exact).float().mean() <= 0.01
                want[page, h, r0:r0 + cnt] = code
            p += cnt
            at += cnt
    assert torch.equal(scales, want_s)
    assert torch.equal(pages, want.view(P, Hkv, 16384))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,new,H,Hkv,rot,inter", [
    ([777], [1], 16, 1, 128, False), ([1, 32, 33, 128, 129, 64], [1] * 6, 8, 2, 64, True),
    ([40, 300, 128, 5], [7, 1, 3, 5], 4, 1, 96, False), ([700, 129, 96, 0], [650, 129, 1, 0], 5, 1, 128, True),
    ([9, 70], [1, 2], 2, 1, 8, False), ([90, 70], [50, 60], 2, 1, 24, False), ([33, 40], [33, 40], 3, 1, 120, True),
    ([100, 100], [40, 33], 3, 3, 0, False), ([257, 31], [256, 31], 16, 8, 16, False), ([64] * 9, [0] * 4 + [64] + [0] * 4, 1, 1, 8, True)])
def test_append(lens, new, H, Hkv, rot, inter, dtype):
    append(lens, new, H, Hkv, dtype, rot, inter, seed=len(lens) + rot)
    m.mx4_check_status()


def test_append_far_positions_and_padding():
    """Positions past 2^31, a factor, rows behind the last sequence, separate arrays."""
    append([50, 260], [50, 2], 4, 2, torch.bfloat16, 128, False, 1, factor=1.2, shift=1000003, pad=7)
    append([50, 260], [3, 9], 4, 2, torch.float32, 64, True, 2, shift=(1 << 33) + 12345, pad=1, fused=False)
    append([50], [50], 4, 2, torch.float32, 64, False, 3, shift=-40)  # negative positions turn back
    m.mx4_check_status()


def test_append_special_values():
    """Zeros, the format's ends, powers of two at a scale's border, huge and tiny rows, a block with a
    NaN scale, and rows that make the stored ones vanish."""
    def edit(x, kp, ks, vp, vs, table):
        x[:] = x.clamp(-100, 100)
        x[0] = 0                              # a block of zeros: the smallest scale
        x[1, -128:] = 448.0
        x[2, -128:] = 449.0
        x[3, -128:] = torch.tensor([2.0**120, -2.0**-126, 1.75 * 2.0**100, -0.0] * 32)
        x[4, -128:] = 2.0**-140               # below the smallest scale
        vs[table[3, 0]] = 40
        vs[table[5, 0]] = 255
        x[5, -128:] = torch.tensor([3.0, -448.0, 1e-30, 0.0] * 32)
    append([1, 1, 1, 8, 1, 31], [1] * 6, 1, 1, torch.float32, 0, False, 4, edit=edit)
    m.mx4_check_status()


def test_append_in_place():
    """q_out may be q: the bits of a call into another tensor."""
    g = torch.Generator().manual_seed(8)
    i = dict(dtype=torch.int32, device=DEV)
    for n in (3, 200):
        q = torch.randn((n, 20, 128), generator=g).to(torch.bfloat16).to(DEV)
        k = torch.randn((n, 1, 128), generator=g).to(torch.bfloat16).to(DEV)
        pools = [torch.zeros((2, 1, 16384), dtype=torch.uint8, device=DEV) for _ in range(2)]
        pools += [torch.zeros((2, 1, 4), dtype=torch.uint8, device=DEV) for _ in range(2)]
        rest = (torch.tensor([0, n], **i), torch.tensor([[0, 1]], **i), torch.tensor([n], **i), *pools)
        ph = m.rope_phases(m.rope_frequencies(128)[0]).to(DEV)
        other = torch.empty_like(q)
        m.fp8_rope_append(q, k, k, *rest, other, phases=ph)
        m.fp8_rope_append(q, k, k, *rest, q, phases=ph)
        assert torch.equal(q, other)
        with pytest.raises(m.Mx4Error, match="overlaps"):
            m.fp8_rope_append(q[:1], k[:1], k[:1], rest[0].clamp(max=1), *rest[1:], q.view(-1)[64:64 + 20 * 128].view(1, 20, 128),
                              phases=ph)


def test_append_non_finite():
    """Stored as NaN, reported, and without a say in the scale of the others."""
    g = torch.Generator().manual_seed(5)
    k = torch.randn((2, 1, 128), generator=g)
    v = torch.randn((2, 1, 128), generator=g)
    v[0, 0, 5], v[1, 0, 7] = math.inf, math.nan
    kp = torch.zeros((1, 1, 16384), dtype=torch.uint8, device=DEV)
    vp, ks = torch.zeros_like(kp), torch.zeros((1, 1, 4), dtype=torch.uint8, device=DEV)
    vs = torch.zeros_like(ks)
    i = dict(dtype=torch.int32, device=DEV)
    m.fp8_rope_append(None, k.to(DEV), v.to(DEV), torch.tensor([0, 2], **i), torch.zeros((1, 1), **i),
                      torch.tensor([2], **i), kp, vp, ks, vs, None)
    flagged(0x10)
    got = vp.cpu().view(128, 128)[:2]
    fin = torch.isfinite(v[:, 0])
    e = R.exponent(float(v[:, 0][fin].abs().max()))
    assert int(vs[0, 0, 0]) == e + 127 and ((got & 0x7F) == 0x7F).eq(~fin).all()
    exact = torch.ldexp(v[:, 0].nan_to_num(0, 0, 0), torch.tensor(-e)).to(E4M3).view(torch.uint8)
    assert torch.equal(got[fin], exact[fin])


def test_append_bad_data():
    """Bad lengths, offsets and pages are reported; the other sequences are written."""
    g = torch.Generator().manual_seed(6)
    v = torch.randn((4, 1, 128), generator=g).to(DEV)
    i = dict(dtype=torch.int32, device=DEV)
    for lens, cu, table, bits, written in (
            ([1, 0, 1, 1], [0, 1, 2, 3, 4], [0, 1, 2, 3], 0x4, [0, 2, 3]),
            ([1, 129, 1, 1], [0, 1, 2, 3, 4], [0, 1, 2, 3], 0x4, [0, 2, 3]),
            ([1, 1, 1, 1], [0, 1, 2, 3, 4], [0, 4, 2, -1], 0x2, [0, 2]),
            ([1, 1, 1, 9], [0, 1, 2, 3, 9], [0, 1, 2, 3], 0x4, [0, 1, 2]),
            ([1, 1, 1, 1], [1, 1, 2, 3, 3], [0, 1, 2, 3], None, [1, 2])):
        kp, vp = (torch.full((4, 1, 16384), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
        ks, vs = (torch.full((4, 1, 4), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
        m.fp8_rope_append(None, v, v, torch.tensor(cu, **i), torch.tensor(table, **i).view(4, 1),
                          torch.tensor(lens, **i), kp, vp, ks, vs, None)
        if bits:
            flagged(bits)
        else:
            m.mx4_check_status()
        for pages in (kp, vp):
            got = [p for p in range(4) if (pages[p, 0, :128] != 255).any()]
            assert got == written, (lens, cu, table, got)


# ------------------------------------------------------------------ block scores and choice

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q", [1, 2, 3, 5, 8])
def test_block_scores_are_the_scorers_maxima(q, fp8):
    """Bit for bit the largest index_score of each block."""
    g = torch.Generator().manual_seed(q)
    lens = [q, 127 + q, 128, 129, 700, 1500, 4100, 8192]
    table, P = tables(g, lens)
    iq = torch.randn((len(lens) * q, 128), generator=g).to(torch.bfloat16).to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    W = table.shape[1]
    sc = torch.zeros((len(lens) * q, W * 128), device=DEV)
    bs = torch.full((len(lens) * q, W), 7.0, device=DEV)
    if fp8:
        pages = pool(g, P, 1)[0][:, 0].to(DEV)
        m.index_score_fp8(iq, q, pages, table.to(DEV), sl, 0.03, sc)
        m.index_block_score_fp8(iq, q, pages, table.to(DEV), sl, 0.03, bs)
    else:
        pages = torch.randint(0, 256, (P, 8704), generator=g, dtype=torch.uint8)
        pages[:, 8192:] = torch.randint(115, 130, (P, 512), generator=g, dtype=torch.uint8)
        pages = pages.to(DEV)
        m.index_score(iq, q, pages, table.to(DEV), sl, sc)
        m.index_block_score(iq, q, pages, table.to(DEV), sl, bs)
    for s, L in enumerate(lens):
        n = -(-L // 128)
        for t in range(s * q, s * q + q):
            x = torch.full((n * 128,), -math.inf, device=DEV)
            x[:L] = sc[t, :L]
            assert torch.equal(bs[t, :n], x.view(n, 128).amax(1)), (s, t)
            assert (bs[t, n:] == 7).all()
    m.mx4_check_status()


@pytest.mark.parametrize("fp8,q", [(False, 1), (False, 4), (True, 1), (True, 8)])
def test_block_scores_of_many_pages(fp8, q):
    """Every CTA goes round its ring many times (11000 pages), lengths ragged, three times over."""
    g = torch.Generator().manual_seed(q)
    lens = np.random.default_rng(q).integers(q, 11000, 256).tolist()
    table, P = tables(g, lens)
    iq = torch.randn((len(lens) * q, 128), generator=g).to(torch.bfloat16).to(DEV)
    sl, td, W = torch.tensor(lens, dtype=torch.int32, device=DEV), table.to(DEV), table.shape[1]
    sc = torch.full((len(lens) * q, W * 128), -math.inf, device=DEV)
    gd = torch.Generator(DEV).manual_seed(q)
    if fp8:
        pages = torch.randn((P, 16384), generator=gd, device=DEV).mul_(100).to(E4M3).view(torch.uint8)
        run = lambda f, out: f(iq, q, pages, td, sl, 0.03, out)
        one, block = m.index_score_fp8, m.index_block_score_fp8
    else:
        pages = torch.randint(0, 256, (P, 8704), generator=gd, device=DEV, dtype=torch.uint8)
        pages[:, 8192:] = torch.randint(115, 130, (P, 512), generator=gd, device=DEV, dtype=torch.uint8)
        run = lambda f, out: f(iq, q, pages, td, sl, out)
        one, block = m.index_score, m.index_block_score
    run(one, sc)
    want = sc.view(len(lens) * q, W, 128).amax(-1)
    for _ in range(3):
        bs = torch.full((len(lens) * q, W), -math.inf, device=DEV)
        run(block, bs)
        # (the fp8 rows hold a few NaN codes, values past the format: their blocks are NaN on both sides)
        assert torch.equal(torch.isnan(bs), torch.isnan(want))
        assert torch.equal(bs.nan_to_num(nan=0.0, neginf=-1e9), want.nan_to_num(nan=0.0, neginf=-1e9))
    m.mx4_check_status()


def test_block_scores_of_many_sequences():
    """More sequences than a launch takes."""
    g = torch.Generator().manual_seed(40)
    lens = np.random.default_rng(3).integers(1, 400, 2100).tolist()
    table, P = tables(g, lens)
    pages = pool(g, P, 1)[0][:, 0].to(DEV)
    iq = torch.randn((2100, 128), generator=g).to(torch.bfloat16).to(DEV)
    sl, W = torch.tensor(lens, dtype=torch.int32, device=DEV), table.shape[1]
    sc = torch.full((2100, W * 128), -math.inf, device=DEV)
    bs = torch.full((2100, W), -math.inf, device=DEV)
    m.index_score_fp8(iq, 1, pages, table.to(DEV), sl, 1.0, sc)
    m.index_block_score_fp8(iq, 1, pages, table.to(DEV), sl, 1.0, bs)
    assert torch.equal(bs, sc.view(2100, W, 128).amax(-1))
    m.mx4_check_status()


def test_block_scores_edges():
    """Sequences shorter than their queries, NaN scores, bad pages and lengths."""
    g = torch.Generator().manual_seed(0)
    q, lens = 4, [0, 1, 3, 200, 300]
    table, P = tables(g, lens)
    pages = pool(g, P, 1)[0][:, 0]
    iq = torch.randn((len(lens) * q, 128), generator=g).to(torch.bfloat16)
    pages[table[3, 0]].view(128, 128)[5] = 0x7F   # a row of NaN
    table[4, 1] = P + 3
    bs = torch.full((len(lens) * q, 4), 7.0, device=DEV)
    m.index_block_score_fp8(iq.to(DEV), q, pages.to(DEV), table.to(DEV),
                            torch.tensor(lens, dtype=torch.int32, device=DEV), 1.0, bs)
    flagged(0x2)
    x = pages.view(E4M3).double().view(P, 128, 128)
    got = bs.cpu()
    for s, L in enumerate(lens):
        for j in range(q):
            p = L - q + j
            for b in range(4):
                v = got[s * q + j, b].item()
                if b >= -(-L // 128):
                    assert v == 7
                elif s == 4 and b == 1 or p < 128 * b:
                    assert v == -math.inf
                elif s == 3 and b == 0:
                    assert math.isnan(v)
                else:
                    w = (x[table[s, b], :min(128, p + 1 - 128 * b)] @ iq[s * q + j].double())
                    mag = (x[table[s, b]].abs() @ iq[s * q + j].double().abs()).max()
                    assert abs(v - w.max().item()) <= 4e-6 * mag  # 128 fp32 terms, as the scorer
    m.index_block_score_fp8(iq.to(DEV)[:4], q, pages.to(DEV), table[:1].to(DEV),
                            torch.tensor([-1], dtype=torch.int32, device=DEV), 1.0, bs)
    flagged(0x4)


@pytest.mark.parametrize("lens,q,k,first,last", [
    ([0, 1, 128, 129, 3000, 100000], 1, 16, 1, 2), ([500, 40000, 131072, 7], 3, 7, 0, 0),
    ([131072] * 3, 8, 1, 0, 1), ([300000, 520000, 90], 2, 500, 5, 5), ([8388608, 4000000], 1, 100, 1, 3),
    ([700000, 3], 1, 4096, 0, 0), ([1000] * 40, 1, 4, 2, 2)])
@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
def test_block_topk(lens, q, k, first, last, kind):
    g = torch.Generator().manual_seed(k)
    W = max(1, max(-(-L // 128) for L in lens))
    x = torch.randn((len(lens) * q, W), generator=g) * 3 + 5
    if kind == "ties":
        x = x.round().clamp(3, 6)
    if kind == "special":
        r = torch.rand(x.shape, generator=g)
        for i, v in enumerate((math.inf, -math.inf, math.nan, -0.0, 0.0, 1e-42, -3e38, 3e38)):
            x[(r > i / 40) & (r < (i + 1) / 40)] = v
    idx = torch.full((len(lens) * q, k), 99, dtype=torch.int32, device=DEV)
    m.block_topk(x.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), q, idx, first=first, last=last)
    assert idx.tolist() == R.topk(x, lens, q, k, first, last)
    m.mx4_check_status()


@pytest.mark.parametrize("W", [1000, 4096, 9000])
def test_block_topk_rows_off_16_bytes(W):
    """Rows of a multiple of four scores that begin one, two, three floats off a 16-byte boundary."""
    lens, q, k = [128 * W, 128 * W - 500, 128 * (W // 2)], 2, 33
    x = torch.randn((len(lens) * q, W), generator=torch.Generator().manual_seed(W))
    for off in range(4):
        flat = torch.full((x.numel() + off,), math.inf, device=DEV)
        rows = flat[off:].view(x.shape).copy_(x)
        idx = torch.full((len(lens) * q, k), 99, dtype=torch.int32, device=DEV)
        m.block_topk(rows, torch.tensor(lens, dtype=torch.int32, device=DEV), q, idx, first=1, last=2)
        assert idx.tolist() == R.topk(x, lens, q, k, 1, 2)
    m.mx4_check_status()


def test_block_topk_bad_lengths():
    x = torch.zeros((3, 4), device=DEV)
    idx = torch.full((3, 2), 9, dtype=torch.int32, device=DEV)
    m.block_topk(x, torch.tensor([-5, 513, 512], dtype=torch.int32, device=DEV), 1, idx, last=1)
    flagged(0x4)
    assert idx.tolist() == [[-1, -1], [-1, -1], [0, 3]]


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("blocks,q,dtype", [(4, 1, torch.bfloat16), (3, 2, torch.float32), (0, 4, torch.bfloat16)])
def test_steps_together(blocks, q, dtype):
    """Prompts of odd lengths, then steps, against 64-bit attention over the rows as they were
    appended (read back from the pages), with the blocks that 64-bit index scores choose."""
    from mxfp4_sparse_paged_gb300.fp8_step import Fp8Caches, Fp8Step
    g = torch.Generator().manual_seed(blocks)
    B, H, Hkv, prompt = 3, 8, 2, [1000, 37, 640]
    lens = list(prompt)
    table, P = tables(g, [L + 64 for L in lens])
    caches = Fp8Caches(P, Hkv, index_scale=0.02)
    freq, grow = m.rope_frequencies(64, scaling="bands", factor=4.0, original_context=512)
    step = Fp8Step(caches, table.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV), q, H, blocks,
                   first=1, last=1, phases=m.rope_phases(freq).to(DEV), factor=grow)
    draw = lambda *s: torch.randn(s, generator=g).to(dtype).to(DEV)
    n = sum(prompt)
    cu = torch.tensor([0] + list(np.cumsum(prompt)), dtype=torch.int32, device=DEV)
    step.append(draw(n, Hkv, 128), draw(n, Hkv, 128), torch.randn((n, 128), generator=g).to(DEV), cu,
                torch.tensor(prompt, dtype=torch.int32, device=DEV))
    graph = None
    for i in range(4):
        T = B * q
        ins = (draw(T, H, 128), draw(T, Hkv, 128), draw(T, Hkv, 128),
               torch.randn((T, 128), generator=g).to(torch.bfloat16).to(DEV),
               torch.randn((T, 128), generator=g).to(DEV))
        if i == 2:  # the rest from a graph
            held = [x.clone() for x in ins]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step.run(*held)
        if graph:
            for a, b in zip(held, ins):
                a.copy_(b)
            graph.replay()
        else:
            step.run(*ins)
        m.mx4_check_status()
        lens = [L + q for L in lens]
        assert step.seq_lens.tolist() == lens
        kv = [x.cpu() for x in caches.kv()]
        chosen = None
        if blocks:
            ik = caches.idx_pages.cpu().view(E4M3).double().view(P, 128, 128) * 0.02
            sc = torch.full((T, table.shape[1]), -math.inf, dtype=F64)
            for t in range(T):
                p = lens[t // q] - q + t % q
                for b in range(p // 128 + 1):
                    rows = ik[table[t // q, b], :min(128, p + 1 - 128 * b)]
                    sc[t, b] = (rows @ ins[3][t].cpu().double()).max()
            chosen = R.topk(sc, lens, q, blocks, 1, 1)
            assert step.block_idx.tolist() == chosen  # (no two of these scores are within 1e-6)
        want = R.attend(step.q_out.cpu(), q, R.values(kv[0], kv[2]), R.values(kv[1], kv[3]), table, lens,
                        step.scale, chosen)
        R.check_attention(step.out, step.lse, want)
        yq = R.turned(ins[0].cpu(), [lens[t // q] - q + t % q for t in range(T)], m.rope_phases(freq).tolist(),
                      False, grow)
        assert ((step.q_out.cpu().double() - yq).abs() <= 2.0**-8 * yq.abs() + band(ins[0].cpu().double(), 64, False, grow)).all()


def test_chain_without_waits():
    """Calls that read what the call before wrote, sixty steps without a wait between them: the bits
    of the same steps with one after every call."""
    from mxfp4_sparse_paged_gb300.fp8_step import Fp8Caches, Fp8Step
    g = torch.Generator(DEV).manual_seed(0)
    B, H, Hkv, prompt, steps = 24, 16, 2, 700, 60
    table, P = tables(torch.Generator().manual_seed(1), [prompt + steps] * B)
    ins = [(torch.randn((B, H, 128), generator=g, device=DEV).to(torch.bfloat16),
            torch.randn((B, Hkv, 128), generator=g, device=DEV).to(torch.bfloat16),
            torch.randn((B, Hkv, 128), generator=g, device=DEV).to(torch.bfloat16),
            torch.randn((B, 128), generator=g, device=DEV).to(torch.bfloat16),
            torch.randn((B, 128), generator=g, device=DEV)) for _ in range(steps)]
    pk = torch.randn((2, B * prompt, Hkv, 128), generator=g, device=DEV).to(torch.bfloat16)
    pi = torch.randn((B * prompt, 128), generator=g, device=DEV)
    phases = m.rope_phases(m.rope_frequencies(128)[0]).to(DEV)

    def go(wait):
        caches = Fp8Caches(P, Hkv, index_scale=0.02)
        step = Fp8Step(caches, table.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV), 1, H, 3, 1, 1, phases)
        step.append(pk[0], pk[1], pi, torch.arange(0, B * prompt + 1, prompt, dtype=torch.int32, device=DEV), prompt)
        outs = []
        for x in ins:
            if wait:
                torch.cuda.synchronize()
            outs.append(step.run(*x).clone())
            outs.append(step.block_idx.clone())
        return outs + [t.clone() for t in caches.kv()]

    quick, slow = go(False), go(True)
    assert all(torch.equal(a, b) for a, b in zip(quick, slow))
    m.mx4_check_status()
