"""GPU parity of the speculative decode step's calls, against the plain 64-bit
implementations of _spec_ref (tolerances derived there and below)."""
import numpy as np
import pytest
import torch

import _spec_ref as R
import mxfp4_sparse_paged_gb300 as m

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda"
SCALE = 128 ** -0.5


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


class Attn:
    """Inputs of one tree_paged_decode call on both sides."""

    def __init__(self, seed, lens, N, H=16, Hkv=1, kind="chain", window=0, sinks=0, counts=None,
                 scale=SCALE, q_std=2.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens = rng, np.asarray(lens, np.int32)
        B = len(lens)
        self.N, self.H, self.Hkv, self.window, self.sinks, self.scale = N, H, Hkv, window, sinks, scale
        self.bt, self.P = R.block_table(rng, lens)
        self.kp, self.vp = R.random_pages(rng, self.P, Hkv), R.random_pages(rng, self.P, Hkv)
        for s, L in enumerate(lens):  # rows past the length hold 0xFF, as an empty cache does
            if L % 128:
                p = self.bt[s, L // 128]
                for pool in (self.kp, self.vp):
                    parts = [x.copy() for x in R.row_parts(pool)]
                    for x in parts:
                        x[p, :, L % 128:] = 255
                    R.join_parts(pool, parts)
        self.counts = np.asarray(counts if counts is not None else [N] * B, np.int32)
        self.parents = [R.random_tree(rng, N) if kind == "tree" else list(range(-1, N - 1))
                        for _ in range(B)]
        self.mask = np.stack([R.masks_of(p) for p in self.parents])
        self.send_mask = kind == "tree"
        self.q = bf16(q_std * rng.standard_normal((B, N, H, 128)))

    def run(self, kp=None, vp=None, stream=None, lse=True):
        B = len(self.lens)
        out = torch.full((B, self.N, self.H, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        ls = torch.full((B, self.N, self.H), float("nan"), device=DEV) if lse else None
        ws = torch.empty(max(16, m.tree_paged_decode_workspace(B, self.N, self.H, self.Hkv)),
                         dtype=torch.uint8, device=DEV)
        ws.fill_(255)
        self.args = (self.q.to(DEV), dev(self.kp) if kp is None else kp,
                     dev(self.vp) if vp is None else vp, dev(self.bt), dev(self.lens), self.scale,
                     out, ws)
        self.kwargs = dict(tree_mask=dev(self.mask.view(np.int64)) if self.send_mask else None,
                           n_nodes=dev(self.counts), window=self.window, sinks=self.sinks, lse=ls)
        m.tree_paged_decode(*self.args, **self.kwargs)
        return out, ls

    def want(self):
        return R.attend(self.q.float().numpy(), self.kp, self.vp, self.bt, self.lens, self.counts,
                        self.mask, self.window, self.sinks, self.scale)

    def check(self, out, lse, want=None):
        o, l, to, tl = self.want() if want is None else want
        got, gl = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isneginf(gl), np.isneginf(l))
        assert np.array_equal(np.isnan(got), np.isnan(o))
        fin = np.isfinite(l)
        assert np.all(np.abs(gl[fin] - l[fin]) <= tl[fin]), float(np.max(np.abs(gl[fin] - l[fin]) / tl[fin]))
        err = np.abs(got - o) - to
        err[np.isnan(o)] = 0
        assert np.all(err <= 0), (float(np.nanmax(np.abs(got - o))), np.argwhere(err > 0)[:4])


CASES = [
    # lens, N, H, Hkv, kind, window, sinks, counts
    ([1], 1, 16, 1, "chain", 0, 0, None),
    ([1, 2, 127, 128, 129, 300], 1, 16, 1, "chain", 0, 0, None),
    ([5000, 40], 1, 16, 1, "chain", 0, 0, None),
    ([640, 128, 8], 8, 16, 1, "chain", 0, 0, None),
    ([64, 65, 700], 64, 16, 1, "tree", 0, 0, [64, 1, 37]),
    ([200, 33], 33, 4, 1, "tree", 0, 0, [33, 0]),
    ([300, 500], 3, 40, 8, "chain", 0, 0, None),
    ([260], 7, 6, 2, "tree", 0, 0, None),
    ([131, 400], 5, 7, 7, "tree", 0, 0, [5, 3]),
    ([900], 2, 128, 1, "chain", 0, 0, None),
    ([400], 64, 8, 8, "tree", 0, 0, None),
    ([1500, 90, 1], 1, 16, 1, "chain", 100, 0, None),
    ([1500, 90, 5], 4, 16, 2, "chain", 1, 0, None),
    ([1500, 600, 20], 6, 16, 1, "tree", 300, 4, [6, 6, 2]),
    ([1500, 600, 20], 16, 10, 2, "tree", 3, 200, None),
    ([2000], 20, 16, 1, "tree", 5, 1, None),
    ([700], 3, 16, 1, "chain", 5000, 130, None),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_tree_paged_decode(i):
    lens, N, H, Hkv, kind, window, sinks, counts = CASES[i]
    lens = [max(x, N if counts is None else 1) for x in lens]
    if counts is not None:
        lens = [max(x, c) for x, c in zip(lens, counts)]
    a = Attn(100 + i, lens, N, H, Hkv, kind, window, sinks, counts)
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)
    again, _ = a.run(lse=False)  # lse is optional; the same bits again
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_tree_many_sequences_and_long_split():
    # 70 short sequences and one long enough to be cut over many CTAs
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 400, 70)] + [30000]
    a = Attn(6, lens, 1, H=4, Hkv=2)
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)


def test_rows_that_see_nothing():
    # a mask of 0 over a cache that holds only the drafts; one with bits past n_nodes only;
    # an idle sequence
    a = Attn(7, [4, 4, 200], 4, kind="tree", counts=[4, 2, 0])
    a.lens[1] = 2
    a.mask[0, 1] = 0
    a.mask[0, 3] = 1 << 60
    a.mask[1, 1] = 1 << 2
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)
    o = out.float().cpu().numpy()
    assert not o[0, 1].any() and not o[0, 3].any() and not o[1, 1:].any() and not o[2].any()
    assert np.isneginf(lse.cpu().numpy()[2]).all()


def test_masked_places_may_hold_anything():
    # a draft that some nodes do not see holds NaN scales in K and V: only the nodes that see
    # it are NaN (a NaN key: all of the row; a NaN value block: its 32 dims); the same for
    # the tokens that a window leaves out
    a = Attn(8, [300], 4, kind="tree", window=150, sinks=2)
    a.mask[0] = [1, 3, 5, 9]  # a root and three children
    L, base = 300, 296
    p, r = a.bt[0, (base + 2) // 128], (base + 2) % 128
    a.vp[p, 0, 8192 + 4 * r + 1] = 255
    p3, r3 = a.bt[0, (base + 3) // 128], (base + 3) % 128
    a.kp[p3, 0, 8192 + 4 * r3 + 2] = 255
    far, fr = a.bt[0, 0], 60  # token 60: outside every window (296 - 150 > 60)
    a.kp[far, 0, 8192 + 4 * fr:8192 + 4 * fr + 4] = 255
    a.vp[far, 0, 8192 + 4 * fr:8192 + 4 * fr + 4] = 255
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    o, l = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(o[0, :2]).all() and np.isfinite(l[0, :3]).all()
    assert np.isnan(o[0, 2, :, 32:64]).all()
    assert np.isfinite(o[0, 2, :, :32]).all() and np.isfinite(o[0, 2, :, 64:]).all()
    assert np.isnan(o[0, 3]).all() and np.isnan(l[0, 3]).all()
    want = a.want()
    fin = [x[:, :2] for x in want]
    keep, a.N = a.N, 2
    a.check(out[:, :2], lse[:, :2], fin)
    a.N = keep


@pytest.mark.parametrize("klo,khi,vlo,vhi,qs", [
    (60, 70, 200, 230, 2.0 ** 55),   # tiny keys, huge values, a huge query
    (180, 190, 1, 12, 2.0 ** -58),   # huge keys, values near the smallest, a tiny query
    (110, 140, 120, 150, 0.5),       # values of both sides of 2^15
    (100, 128, 0, 3, 1.0),           # the smallest value scales
])
def test_scales_over_the_whole_range(klo, khi, vlo, vhi, qs):
    a = Attn(9, [500], 3, kind="chain", q_std=qs)
    a.kp[..., 8192:] = a.rng.integers(klo, khi, a.kp[..., 8192:].shape)
    a.vp[..., 8192:] = a.rng.integers(vlo, vhi, a.vp[..., 8192:].shape)
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    o, l, to, tl = a.want()
    # bf16's smallest subnormal: results below its normal range round on that grid, and
    # fp32 sums of them on theirs
    a.check(out, lse, (o, l, to + 2.0 ** -133, tl))


@pytest.mark.parametrize("slope", [40.0, -40.0, 400.0])
def test_logits_that_climb_and_fall(slope):
    # keys grow along the context, so that every page's largest logit is far above (below)
    # the last page's: by 40 and 400 in natural units
    a = Attn(10, [1500], 2, kind="chain")
    q = np.zeros((1, 2, 16, 128), np.float32)
    q[..., 0] = np.linspace(0.5, 1.0, 16)[None, None]
    a.q = bf16(q)
    a.scale = abs(slope) / 4
    for pg in range(12):
        c = pg if slope > 0 else 11 - pg
        p = a.bt[0, pg]
        d = a.kp[p, 0, :8192].reshape(128, 64)
        d[:, 0] = (d[:, 0] & 0xF0) | [0, 1, 2, 3, 4, 4, 5, 5, 6, 6, 7, 7][c]
        a.kp[p, 0, 8192:].reshape(128, 4)[:, 0] = 127
    if a.lens[0] % 128:
        p = a.bt[0, 11]
        a.kp[p, 0, 8192:].reshape(128, 4)[a.lens[0] % 128:] = 255
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)


@pytest.mark.parametrize("N", [1, 3, 8, 13])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_of_every_tile_size_with_references_that_move(N, sign):
    # 16, 48, 128 and 208 rows of a head: half of the heads' logits climb from page to page,
    # half fall
    a = Attn(19, [900 + N], N, kind="tree")
    q = np.zeros((1, N, 16, 128), np.float32)
    q[..., 0] = sign * np.linspace(0.5, 1.0, 16) * np.where(np.arange(16) % 2, 1, -1)
    a.q = bf16(q)
    a.scale = 10.0
    for pg in range(8):
        d = a.kp[a.bt[0, pg], 0, :8192].reshape(128, 64)
        d[:, 0] = (d[:, 0] & 0xF0) | pg
        a.kp[a.bt[0, pg], 0, 8192:].reshape(128, 4)[:, 0] = 127
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)


@pytest.mark.parametrize("N,H,kind", [(1, 16, "chain"), (6, 5, "tree"), (7, 16, "tree")])
def test_value_scales_that_change_from_page_to_page(N, H, kind):
    # blocks of some pages far above and far below the others, a page of zeros (scale byte 0)
    a = Attn(18, [1300], N, H=H, kind=kind)
    for pg, sc in ((0, 0), (2, 150), (3, 90), (6, 103), (7, 141), (9, 200)):
        p = a.bt[0, pg]
        a.vp[p, 0, 8192:].reshape(128, 4)[:, pg % 4] = sc
        if pg == 0:
            a.vp[p, 0, :8192] = 0
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)


def test_infinite_queries_are_nan():
    a = Attn(11, [200], 2)
    a.q[0, 1, 3, 5] = float("inf")
    a.q[0, 1, 4, 6] = float("nan")
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    o = out.float().cpu().numpy()
    bad = np.zeros((2, 16), bool)
    bad[1, 3] = bad[1, 4] = True
    assert np.array_equal(np.isnan(o[0]).all(-1), bad) and np.array_equal(np.isnan(o[0]).any(-1), bad)


def test_bad_pages_and_lengths_are_flagged_and_skipped():
    a = Attn(12, [600, 300, 400], 2)
    a.bt[0, 1] = a.P + 7
    a.bt[2, 0] = -1
    out, lse = a.run()
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x2
    # the tokens of the bad pages are not seen
    good = Attn(12, [600, 300, 400], 2)
    o, l, to, tl = good.want()
    want = [x.copy() for x in (o, l, to, tl)]
    for s, keep in ((0, np.r_[0:128, 256:600]), (2, np.r_[128:400])):
        k, v = R.rows_of(good.kp, good.bt[s], 0, int(good.lens[s])), R.rows_of(good.vp, good.bt[s], 0, int(good.lens[s]))
        for j in range(2):
            at = keep[keep <= good.lens[s] - 2 + j]
            for h in range(16):
                x = SCALE * (k[at] @ good.q[s, j, h].double().numpy())
                w = np.exp(x - x.max())
                want[0][s, j, h] = w @ v[at] / w.sum()
                want[1][s, j, h] = np.log(w.sum()) + x.max()
                want[2][s, j, h] = 2.0 ** -7 * 1.05 * (w @ np.abs(v[at]) / w.sum())
    a.check(out, lse, want)
    a = Attn(13, [600, 300], 2)
    a.lens[0] = 100000
    a.lens[1] = 1
    out, lse = a.run()
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x4
    assert not out.float().any() and torch.isneginf(lse).all()


def test_strided_pools_streams_and_graphs():
    # K and V as the halves of one pool (page stride 2 x heads x 8704), on a side stream, and
    # replayed from a graph with new contents
    a = Attn(14, [700, 90], 4, H=12, Hkv=3, kind="tree", window=200, sinks=3)
    both = torch.zeros((a.P, 2, 3, 8704), dtype=torch.uint8, device=DEV)
    both[:, 0], both[:, 1] = dev(a.kp), dev(a.vp)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out, lse = a.run(both[:, 0], both[:, 1])
    torch.cuda.current_stream().wait_stream(st)
    assert m.mx4_check_status() == 0
    want = a.want()
    a.check(out, lse, want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        m.tree_paged_decode(*a.args, **a.kwargs)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    a.check(out, lse, want)


def test_page_offsets_past_32_bits():
    # a pool of 4.6 GB a tensor, the sequence's pages at its two ends
    P = 530000
    a = Attn(15, [256], 2, H=4, Hkv=1)
    kp = torch.empty((P, 1, 8704), dtype=torch.uint8, device=DEV)
    vp = torch.empty((P, 1, 8704), dtype=torch.uint8, device=DEV)
    ids = np.array([P - 1, 3], np.int32)
    for i in range(2):
        kp[int(ids[i])] = dev(a.kp[a.bt[0, i]])
        vp[int(ids[i])] = dev(a.vp[a.bt[0, i]])
    want = a.want()
    a.bt[0, :2] = ids
    out, lse = a.run(kp, vp)
    assert m.mx4_check_status() == 0
    a.check(out, lse, want)


# ------------------------------------------------------------------ verify_drafts

def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def verify_inputs(seed, B, N, V, chain=False, noise=0.8, sharp=2.0):
    rng = np.random.default_rng(seed)
    x = sharp * rng.standard_normal((B, N, V))
    target, draft = softmax(x), softmax(x + noise * rng.standard_normal((B, N, V)))
    parents = np.array([list(range(-1, N - 1)) if chain else R.random_tree(rng, N) for _ in range(B)],
                       np.int32)
    tokens = np.zeros((B, N), np.int32)
    for s in range(B):
        for j in range(1, N):
            c = np.cumsum(draft[s, parents[s, j]].astype(np.float64))
            tokens[s, j] = min(V - 1, int(np.searchsorted(c, rng.random() * c[-1])))
    return target, draft, tokens, parents, rng.random((B, N), dtype=np.float32), rng.random(B, dtype=np.float32)


def run_verify(target, draft, tokens, parents, u, us, counts=None):
    B, N, V = target.shape
    path = torch.full((B, N), 77, dtype=torch.int32, device=DEV)
    acc = torch.full((B,), 77, dtype=torch.int32, device=DEV)
    nxt = torch.full((B,), 77, dtype=torch.int32, device=DEV)
    t = target if isinstance(target, torch.Tensor) else dev(target)
    d = draft if draft is None or isinstance(draft, torch.Tensor) else dev(draft)
    m.verify_drafts(t, d, dev(tokens), dev(parents), dev(u), dev(us), path, acc, nxt,
                    n_nodes=None if counts is None else dev(np.asarray(counts, np.int32)))
    return path.cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy()


def same(got, want):
    for g, w, name in zip(got, want, ("path", "n_accepted", "next_token")):
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:3])


@pytest.mark.parametrize("B,N,V,chain,given", [
    (1, 1, 1, True, False), (3, 1, 50, True, False), (40, 4, 7, True, False),
    (200, 12, 33, False, False), (200, 12, 33, False, True), (64, 8, 1000, True, True),
    (3, 64, 2049, False, False), (2, 5, 40001, False, False), (300, 6, 4500, False, True),
    (1, 3, 131072, True, False), (100, 4, 20011, False, False),
])
def test_verify_drafts(B, N, V, chain, given):
    a = verify_inputs(B * 7 + N, B, N, V, chain)
    if given:
        a = (a[0], None) + a[2:]
    rng = np.random.default_rng(V)
    counts = rng.integers(0, N + 1, B)
    counts[0] = N
    got = run_verify(*a, counts)
    assert m.mx4_check_status() == 0
    same(got, R.verify(*a, counts))
    same(run_verify(*a), R.verify(*a, np.full(B, N)))


def test_verify_rows_that_are_not_kept():
    # a vocabulary beyond what a cluster's registers hold, siblings of one node tested in turn
    a = verify_inputs(21, 3, 6, 140001, noise=2.0)
    a[3][:] = [-1, 0, 0, 0, 1, 1]
    a[5][1:] = 0
    same(run_verify(*a), R.verify(*a, np.full(3, 6)))
    assert m.mx4_check_status() == 0


@pytest.mark.parametrize("V,noise", [(40, 3.0), (700, 1e-3), (9000, 1.0), (30000, 1e-4)])
def test_verify_many_siblings(V, noise):
    # up to 63 rejections at one node, drafts far from the target and next to it
    N = 64
    a = verify_inputs(22, 5, N, V, noise=noise)
    a[3][:] = 0
    a[3][:, 0] = -1
    a[4][:4] = np.maximum(a[4][:4], 0.97)
    rng = np.random.default_rng(V)
    for s in range(5):
        c = np.cumsum(a[1][s, 0].astype(np.float64))
        a[2][s, 1:] = np.minimum(V - 1, np.searchsorted(c, rng.random(N - 1) * c[-1]))
    same(run_verify(*a), R.verify(*a, np.full(5, N)))
    b = (a[0], None) + a[2:]
    same(run_verify(*b), R.verify(*b, np.full(5, N)))
    assert m.mx4_check_status() == 0


def test_verify_borders():
    # u of 0 and next to 1, one-hot targets, drafts equal to the target, zero probabilities
    V, N = 300, 5
    target, draft, tokens, parents, u, us = verify_inputs(1, 8, N, V)
    u[0] = us[0] = 0
    u[1] = us[1] = np.float32(1) - np.float32(2.0 ** -24)
    target[2] = 0
    target[2, :, 123] = 1.0
    draft[3] = target[3]
    # p <= q everywhere and x outside both: rejected, nothing left, p itself is drawn from
    draft[4] = target[4] = 0
    target[4, :, 5] = draft[4, :, 5] = 0.5
    target[4, :, 290] = draft[4, :, 290] = 0.5
    tokens[4] = 7
    parents[4] = [-1, 0, 0, 1, 1]
    tokens[5, 1:] = tokens[5, 1]  # every child the same token
    parents[5] = [-1, 0, 0, 0, 0]
    target[6, :, :] = np.float32(1.0 / 300)
    draft[6, :, :] = 0
    draft[6, :, 0] = 1.0
    tokens[6] = 0
    parents[6] = [-1, 0, 0, 0, 0]
    u[6] = 0.9
    a = (target, draft, tokens, parents, u, us)
    got = run_verify(*a)
    assert m.mx4_check_status() == 0
    same(got, R.verify(*a, np.full(8, N)))
    assert got[2][0] >= 0 and got[2][2] == 123
    b = (target, None, tokens, parents, u, us)
    same(run_verify(*b), R.verify(*b, np.full(8, N)))
    assert m.mx4_check_status() == 0


def test_verify_strides_graph_and_stream():
    a = verify_inputs(2, 6, 4, 1001)
    big = torch.zeros((7, 5, 1003), device=DEV)
    big[:6, :4, 1:1002] = dev(a[0])
    dbig = torch.zeros((4, 6, 1001), device=DEV)
    dbig.copy_(dev(a[1]).transpose(0, 1))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run_verify(big[:6, :4, 1:1002], dbig.transpose(0, 1), *a[2:])
    same(got, R.verify(*a, np.full(6, 4)))
    assert m.mx4_check_status() == 0


def test_verify_bad_inputs_are_flagged():
    target, draft, tokens, parents, u, us = verify_inputs(3, 5, 4, 100, chain=True)
    want = R.verify(target, draft, tokens, parents, u, us, np.full(5, 4))
    tokens[1, 1] = 100
    parents[2, 2] = 2
    got = run_verify(target, draft, tokens, parents, u, us)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x8
    assert got[1][1] == 1 and got[1][2] <= 2
    for i in (0, 3, 4):
        assert np.array_equal(got[0][i], want[0][i]) and got[2][i] == want[2][i]
    target, draft, tokens, parents, u, us = verify_inputs(4, 3, 1, 100)
    target[1] = 0
    target[2, 0, 5] = np.nan
    want = R.verify(target[:1], draft[:1], tokens[:1], parents[:1], u[:1], us[:1], [1])
    got = run_verify(target, draft, tokens, parents, u, us)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x10
    assert got[2][0] == want[2][0] and got[2][1] == -1 and 0 <= got[2][2] < 100


# ------------------------------------------------------------------ rows and pages

def pools_of(rng, P, Hkv, fp8):
    idx = (rng.integers(0, 256, (P, 16384), dtype=np.uint8) if fp8
           else rng.integers(0, 256, (P, 8704), dtype=np.uint8))
    return [rng.integers(0, 256, (P, Hkv, 8704), dtype=np.uint8),
            rng.integers(0, 256, (P, Hkv, 8704), dtype=np.uint8), idx]


@pytest.mark.parametrize("B,N,Hkv,fp8,use_idx", [
    (1, 1, 1, False, True), (5, 8, 1, False, True), (7, 64, 8, True, True), (9, 33, 2, False, False),
    (40, 64, 1, True, True),
])
def test_accept_rows(B, N, Hkv, fp8, use_idx):
    rng = np.random.default_rng(B + N)
    counts = rng.integers(0, N + 1, B).astype(np.int32)
    counts[0] = N
    lens = (counts + rng.integers(0, 300, B)).astype(np.int32)
    bt, P = R.block_table(rng, np.maximum(lens, 1))
    pools = pools_of(rng, P, Hkv, fp8)[:3 if use_idx else 2]
    path = np.full((B, N), -1, np.int32)
    acc = np.array([rng.integers(0, c + 1) for c in counts], np.int32)
    for s in range(B):
        path[s, :acc[s]] = np.sort(rng.choice(int(counts[s]), int(acc[s]), replace=False))
    want, wl = R.accept(path, acc, lens, counts, bt, pools)
    d = [dev(p) for p in pools]
    new = torch.full((B,), -5, dtype=torch.int32, device=DEV)
    m.mx4_accept_rows(dev(path), dev(acc), dev(lens), dev(bt), d[0], d[1], d[2] if use_idx else None,
                      new, n_nodes=dev(counts))
    assert m.mx4_check_status() == 0
    for x, w in zip(d, want):
        assert np.array_equal(x.cpu().numpy(), w)
    assert np.array_equal(new.cpu().numpy(), wl)


def test_accept_rows_refuses_bad_paths_and_leaves_the_cache():
    rng = np.random.default_rng(9)
    B, N = 6, 8
    lens = np.array([200, 200, 200, 200, 5, 200], np.int32)
    bt, P = R.block_table(rng, lens)
    pools = pools_of(rng, P, 1, False)
    path = np.tile(np.array([0, 2, 5, -1, -1, -1, -1, -1], np.int32), (B, 1))
    acc = np.full(B, 3, np.int32)
    path[0, 1] = 0       # does not ascend
    path[1, 2] = 8       # past the nodes
    path[2, 0] = -3
    acc[3] = 9           # more than there are
    # sequence 4: shorter than its nodes
    d = [dev(p) for p in pools]
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    m.mx4_accept_rows(dev(path), dev(acc), dev(lens), dev(bt), *d, new)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0xC
    keep = np.array([0, 0, 0, 0, 0, 3], np.int32)
    want, _ = R.accept(path, keep, np.where(keep, lens, 8).astype(np.int32), np.full(B, 8), bt, pools)
    for x, w in zip(d, want):
        assert np.array_equal(x.cpu().numpy(), w)
    assert new.cpu().tolist() == [200, 200, 200, 200, 5, 195]


class PageState:
    def __init__(self, seed, lens, spare, Hkv=1, fp8=False):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        self.bt, self.P = R.block_table(rng, lens, spare)
        self.pools = pools_of(rng, self.P, Hkv, fp8)
        self.refs = np.zeros(self.P, np.int32)
        used = self.bt[self.bt >= 0]
        self.refs[used] = 1
        left = np.setdiff1d(np.arange(self.P), used).astype(np.int32)
        rng.shuffle(left)
        self.fl = np.full(self.P, -1, np.int32)
        self.fl[:len(left)] = left
        self.fc = len(left)
        self.d = dict(bt=dev(self.bt), lens=dev(self.lens), refs=dev(self.refs), fl=dev(self.fl),
                      fc=dev(np.array([self.fc], np.int32)), pools=[dev(p) for p in self.pools])

    def fork(self, rows):
        n, W = len(rows), self.bt.shape[1]
        ct = torch.full((n, W), 55, dtype=torch.int32, device=DEV)
        cl = torch.full((n,), 55, dtype=torch.int32, device=DEV)
        d = self.d
        m.mx4_fork_pages(dev(np.asarray(rows, np.int32)), d["bt"], d["lens"], d["refs"], d["fl"], d["fc"],
                         *d["pools"], ct, cl)
        want = R.fork(rows, self.bt, self.lens, self.refs, self.fl, self.fc, self.pools)
        self.refs, self.fc, self.pools = want[2], want[3], want[4]
        return ct, cl, want

    def check(self):
        d = self.d
        assert np.array_equal(d["refs"].cpu().numpy(), self.refs)
        assert int(d["fc"].cpu()) == self.fc
        assert np.array_equal(d["fl"].cpu().numpy()[:self.fc], self.fl[:self.fc])
        for x, w in zip(d["pools"], self.pools):
            assert np.array_equal(x.cpu().numpy(), w)


@pytest.mark.parametrize("n,B,Hkv,fp8", [(1, 1, 1, False), (4, 1, 1, True), (33, 5, 8, False),
                                         (2500, 60, 1, False)])
def test_fork_and_free_pages(n, B, Hkv, fp8):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 700, B)
    lens[0] = 300
    if B > 2:
        lens[1], lens[2] = 256, 0
    st = PageState(n + 1, lens, n + 4, Hkv, fp8)
    rows = rng.integers(0, B, n)
    ct, cl, want = st.fork(rows)
    assert m.mx4_check_status() == 0
    assert np.array_equal(ct.cpu().numpy(), want[0]) and np.array_equal(cl.cpu().numpy(), want[1])
    st.check()
    # half of the children end, then the parents and the rest
    h = n // 2
    d = st.d
    for t, l, tn, ln in ((ct[:h], cl[:h], want[0][:h], want[1][:h]),
                         (torch.cat((d["bt"], ct[h:])), torch.cat((d["lens"], cl[h:])),
                          np.concatenate((st.bt, want[0][h:])), np.concatenate((st.lens, want[1][h:])))):
        m.mx4_free_pages(t.contiguous(), l.contiguous(), d["refs"], d["fl"], d["fc"])
        st.refs, st.fl, st.fc = R.free(tn, ln, st.refs, st.fl, st.fc)
        assert m.mx4_check_status() == 0
        st.check()
    assert not st.refs.any() and st.fc == st.P


def test_fork_without_pages_and_bad_rows():
    st = PageState(3, [300, 128], 2)
    rows = np.array([0, 1, 0, 0, 1, 9], np.int64)
    ct, cl, want = st.fork(rows)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x48
    assert np.array_equal(ct.cpu().numpy(), want[0]) and np.array_equal(cl.cpu().numpy(), want[1])
    assert cl.cpu().tolist() == [300, 128, 300, 0, 128, 0]
    st.check()


def test_freeing_a_page_nobody_holds_is_flagged():
    st = PageState(4, [300, 128], 2)
    d = st.d
    m.mx4_free_pages(d["bt"], d["lens"], d["refs"], d["fl"], d["fc"])
    assert m.mx4_check_status() == 0
    m.mx4_free_pages(d["bt"], d["lens"], d["refs"], d["fl"], d["fc"])
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x80
    st.refs, st.fl, st.fc = R.free(st.bt, st.lens, st.refs, st.fl, st.fc)
    st.check()


def test_lengths_written_by_a_call_are_read_by_the_next():
    # accept -> attention and fork -> attention back to back on one stream, many times: the
    # attention reads the lengths and tables that the call before it wrote
    a = Attn(16, [400, 130, 700], 3, H=16)
    d = [dev(a.kp), dev(a.vp)]
    path = np.tile(np.array([0, 1, 2], np.int32), (3, 1))
    new = torch.zeros(3, dtype=torch.int32, device=DEV)
    out = torch.zeros((3, 3, 16, 128), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((3, 3, 16), device=DEV)
    ws = torch.empty(max(16, m.tree_paged_decode_workspace(3, 3, 16, 1)), dtype=torch.uint8, device=DEV)
    q, bt, p = a.q.to(DEV), dev(a.bt), dev(path)
    acc, lens = dev(np.full(3, 3, np.int32)), dev(a.lens)
    first = None
    for _ in range(30):
        new.zero_()
        m.mx4_accept_rows(p, acc, lens, bt, d[0], d[1], None, new)
        m.tree_paged_decode(q, d[0], d[1], bt, new, SCALE, out, ws, lse=lse)
        m.tree_paged_decode(q, d[0], d[1], bt, new, SCALE, out, ws, lse=lse)
        if first is None:
            first = out.clone()
        assert torch.equal(out, first)
    assert m.mx4_check_status() == 0
    a.check(out, lse)


@pytest.mark.parametrize("N,H,kind", [(1, 16, "chain"), (5, 7, "tree")])
def test_more_sequences_than_a_launch_holds(N, H, kind):
    # 300: a launch of 256 and one of 44 over the same workspace, masks, counts and lse with it;
    # two long ones at the launches' border and one idle
    rng = np.random.default_rng(N)
    lens = [int(x) for x in rng.integers(N, 200, 300)]
    lens[255], lens[256], lens[299] = 3000, 5000, 700
    counts = rng.integers(1, N + 1, 300)
    counts[7] = counts[290] = 0
    a = Attn(40 + N, lens, N, H=H, kind=kind, counts=counts, window=150 if kind == "tree" else 0, sinks=2)
    want = a.want()
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse, want)
    again, _ = a.run(lse=False)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
