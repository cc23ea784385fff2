"""GPU parity of the speculative step's calls at the ends of their ranges: the largest value
scales, logits far beyond fp32's integers, probabilities that are none (64-bit references of
_spec_ref; tolerances derived there and below)."""
import numpy as np
import pytest
import torch

import _spec_ref as R
import mxfp4_sparse_paged_gb300 as m
from test_gpu_speculate import DEV, Attn, bf16, dev, pools_of, run_verify, same, verify_inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def value_block(a, token, block, scale, codes):
    """The 32-dim block of the value of cached token `token` of sequence 0, head 0: a scale byte
    and one code for the even dims, one for the odd."""
    p, r = a.bt[0, token // 128], token % 128
    a.vp[p, 0, 64 * r + 16 * block:64 * r + 16 * block + 16] = codes[0] | codes[1] << 4
    a.vp[p, 0, 8192 + 4 * r + block] = scale


# ------------------------------------------------------------------ tree_paged_decode

@pytest.mark.parametrize("heads", [4, 16, 32])  # 16, 64 and 128 rows a tile
@pytest.mark.parametrize("scale,codes", [(253, (6, 7)), (253, (14, 7)), (254, (2, 4)), (254, (7, 15))])
def test_values_beyond_bf16_in_places_not_seen(heads, scale, codes):
    # codes whose value passes bf16's largest, in a sibling and in a token that the window leaves
    # out: the other nodes' results are those without them; the node that sees its own has a
    # result that bf16 holds, as its weight is small
    a = Attn(31, [300], 4, H=heads, kind="tree", window=150, sinks=2)
    a.mask[0] = [1, 3, 5, 9]  # a root and three children
    value_block(a, 296 + 2, 1, scale, codes)
    for block in range(4):
        value_block(a, 60, block, scale, codes)  # outside every window (296 - 150 > 60)
    want = a.want()
    assert np.abs(want[0][0, [0, 1, 3]]).max() < 100 and np.abs(want[0]).max() < 0.9 * BF16_MAX
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse, want)


def test_values_beyond_bf16_with_a_weight_of_zero():
    # seen, but 2^-200 of the row: no part in the result
    a = Attn(32, [200], 1)
    q = np.zeros((1, 1, 16, 128), np.float32)
    q[..., 0] = np.linspace(1.0, 2.0, 16)
    a.q, a.scale = bf16(q), 140.0
    d = a.kp[a.bt[0, 0], 0, :8192].reshape(128, 64)
    a.kp[a.bt[0, 0], 0, 8192:].reshape(128, 4)[:, 0] = 127
    a.kp[a.bt[0, 1], 0, 8192:].reshape(128, 4)[:72, 0] = 127
    d[:, 0] = d[:, 0] & 0xF0 | 1
    e = a.kp[a.bt[0, 1], 0, :8192].reshape(128, 64)
    e[:72, 0] = e[:72, 0] & 0xF0 | 1
    d[7, 0] = d[7, 0] & 0xF0 | 9  # -0.5: 140 below the others and more
    value_block(a, 7, 2, 254, (7, 6))
    seen = R.rows_of(a.kp, a.bt[0], 0, 200)[:, 0]
    assert (seen == np.where(np.arange(200) == 7, -0.5, 0.5)).all()
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)


def test_the_largest_values_that_bf16_holds():
    # one token: the result is its value, 3 x 2^126 and 1.5 x 2^127 exactly, and infinite past that
    a = Attn(33, [1], 1)
    for block, (scale, codes) in enumerate([(253, (5, 12)), (254, (3, 2)), (254, (1, 9)), (254, (7, 15))]):
        value_block(a, 0, block, scale, codes)
    out, _ = a.run()
    assert m.mx4_check_status() == 0
    o = out.float().cpu().numpy()[0, 0].astype(np.float64)
    want = R.rows_of(a.vp, a.bt[0], 0, 1)[0]
    assert np.array_equal(o[:, :96], np.broadcast_to(want[:96], (16, 96)))
    assert np.array_equal(o[:, 96:], np.broadcast_to(np.where(want[96:] > 0, np.inf, -np.inf), (16, 32)))


@pytest.mark.parametrize("N", [1, 2, 4, 13])  # 16, 32, 64 and 128 rows a tile
@pytest.mark.parametrize("power", [24, 30, 33, 36, 60])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_far_beyond_the_integers_of_fp32(N, power, sign):
    # one dim of q and of K: the logits are exact products, 2^power times a few, and lie so far
    # apart that the largest alone have a weight.  Six pages, larger keys in the later ones.
    a = Attn(34, [700], N, kind="tree")
    q = np.zeros((1, N, 16, 128), np.float32)
    q[..., 0] = (1 + np.arange(16) / 16) * np.where(np.arange(16) % 3 == 1, -1, 1)
    a.q = bf16(q)
    a.scale = sign * 2.0 ** power
    codes = np.zeros((6, 128), np.int64)
    for pg in range(6):
        codes[pg] = a.rng.integers(0, 4 + min(pg, 2), 128) | 8 * a.rng.integers(0, 2, 128)
        p = a.bt[0, pg]
        d = a.kp[p, 0, :8192].reshape(128, 64)
        d[:, 0] = d[:, 0] & 0xF0 | codes[pg]
        a.kp[p, 0, 8192:].reshape(128, 4)[:, 0] = 127
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    o, l, _, _ = a.want()
    got, gl = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    # the weights are 0 or 1, exactly; the mean rounds in fp32 and to bf16 (half a step), the
    # logsumexp by five fp32 operations
    v = R.rows_of(a.vp, a.bt[0], 0, 700)
    tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -16 * np.abs(v).max()
    assert np.all(np.abs(got - o) <= tol), float(np.nanmax(np.abs(got - o)))
    assert np.all(np.abs(gl - l) <= 2.0 ** -21 * np.abs(l))


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-30, -1e-30])
def test_scales_next_to_zero(scale):
    # every visible token has nearly the same weight, whatever the queries
    a = Attn(35, [300, 140], 3, kind="tree", scale=scale)
    a.q[0, 1] *= 2.0 ** 40
    out, lse = a.run()
    assert m.mx4_check_status() == 0
    a.check(out, lse)


# ------------------------------------------------------------------ verify_drafts

def flat_rows(a, rows, total):
    """Rows (s, j) of the target become flat with this sum."""
    V = a[0].shape[2]
    for s, j in rows:
        a[0][s, j] = np.float32(total / V)


@pytest.mark.parametrize("V", [40, 1000, 5000, 20001, 131072, 140001])
@pytest.mark.parametrize("given", [False, True])
def test_verify_rows_that_sum_to_two_and_more(V, given):
    # no probabilities: rows of 1.5 are worked with as they are, those of 3, 10 and (where that
    # many probabilities are) 40 are refused where their sum is needed: no next token
    B, N = 6, 3
    a = verify_inputs(V, B, N, V, chain=True)
    if given:
        a = (a[0], None) + a[2:]
    a[3][:] = [-1, 0, 0]
    a[4][1:5] = 0.999  # both drafts, the only token of the draft's row, are rejected at the root
    a[2][1:5, 1:] = 7
    if not given:
        a[1][1:5, 0] = np.arange(V) == 7
    for s, total in ((1, 1.5), (2, 3.0), (3, 10.0), (4, min(V / 2, 40.0))):
        flat_rows(a, [(s, 0)], total)
    want = R.verify(*a, np.full(B, N))
    got = run_verify(*a)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x10
    for g, w in zip(got, want):
        assert np.array_equal(g[[0, 1, 5]], w[[0, 1, 5]])
    assert (got[2][2:5] == -1).all() and (got[1][2:5] == 1).all()
    assert (got[0][2:5] == [0, -1, -1]).all()


def test_verify_rows_past_two_in_one_thread():
    # all of a large sum in the values of one thread, of one warp and of one CTA
    B, N, V = 4, 1, 70001
    a = verify_inputs(5, B, N, V)
    a[0][:3] = 0
    a[0][0, 0, 32 * np.arange(30)] = 0.9
    a[0][1, 0, :1000] = 0.5
    a[0][2, 0, 100:30000] = 0.5
    want = R.verify(*a, np.full(B, N))
    got = run_verify(*a)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x10
    assert (got[2][:3] == -1).all() and got[2][3] == want[2][3]


def test_verify_sums_just_below_two_are_exact():
    # two tokens of 1 and the number before it: drawn right up to the border between them
    V = 256
    a = verify_inputs(6, 5, 1, V)
    a[0][:] = 0
    a[0][:, 0, 3], a[0][:, 0, 200] = 1.0, np.float32(1) - np.float32(2.0 ** -24)
    a[5][:] = np.array([0.0, 0.499, 0.5, 0.50001, 1 - 2.0 ** -24], np.float32)
    same(run_verify(*a), R.verify(*a, np.full(5, 1)))
    assert m.mx4_check_status() == 0


@pytest.mark.parametrize("which,value", [("target", np.nan), ("target", -0.5), ("target", 1.5),
                                         ("draft", np.nan), ("draft", -0.5), ("draft", 1.5)])
def test_verify_flags_what_it_looks_up(which, value):
    # the probability of a tested draft, in a row that is not summed as the draft stands; the same
    # of a draft that is never tested is not looked at
    B, N, V = 2, 4, 50
    a = verify_inputs(7, B, N, V, chain=True)
    a[3][:] = [-1, 0, 1, 1]
    a[4][:] = 0  # every tested draft with a probability stands
    row = a[0] if which == "target" else a[1]
    a[0][0, 0, a[2][0, 1]] = 0.5
    clean = [np.copy(x) for x in a]
    row[0, 1, a[2][0, 3]] = value  # node 2 stands first: 3 is not tested
    a[2][0, 2] = (a[2][0, 3] + 1) % V
    clean[2][0, 2] = a[2][0, 2]
    a[0][0, 1, a[2][0, 2]] = clean[0][0, 1, a[2][0, 2]] = 0.5
    same(run_verify(*a), R.verify(*clean, np.full(B, N)))
    assert m.mx4_check_status() == 0
    row[0, 0, a[2][0, 1]] = value
    got = run_verify(*a)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x10
    assert got[1][0] == (1 if which == "target" and not value > 0 else 3)


# ------------------------------------------------------------------ mx4_accept_rows

@pytest.mark.parametrize("path", [[0, 1, 2, -1], [0, 1, 3, -1]])
@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_accepted_rows_have_to_be_on_a_page(path, page):
    # the drafts' second page is none: its rows were never cached, so a path over them is
    # refused, whether its rows move or stay; a path that ends before them stands
    rng = np.random.default_rng(1)
    lens = np.array([130, 130], np.int32)  # four nodes each, two on the second page
    bt, P = R.block_table(rng, lens)
    bt[:, 1] = page
    pools = pools_of(rng, P, 1, False)
    paths = np.array([path, [0, 1, -1, -1]], np.int32)
    d = [dev(p) for p in pools]
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    m.mx4_accept_rows(dev(paths), dev(np.array([3, 2], np.int32)), dev(lens), dev(bt), *d, new)
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x2
    assert new.cpu().tolist() == [130, 128]
    for x, w in zip(d, pools):
        assert np.array_equal(x.cpu().numpy(), w)
