"""The 8-bit cache's attention and append where numbers leave the usual range: logits of any size,
V scales any powers apart, results next to the least bf16, angles of slow pairs; against float64."""
import math

import pytest
import torch

import _fp8_ref as R
import mxfp4_sparse_paged_gb300 as m
from test_gpu_fp8_kv import append, attention, clean, tables  # noqa: F401 (clean: a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64, E4M3 = torch.float64, torch.float8_e4m3fn


def codes(x):
    return torch.as_tensor(x, dtype=torch.float32).to(E4M3).view(torch.uint8)


def near(out, lse, want, exact=False):
    """out: half a step of bf16 (2^-8 of the value, 2^-134 where it is subnormal), and of sum w |V| 2^-11
    (weights of 11 bits, 2^-12 each, and fp32 sums) and twice the logits' error: 2^-18 of sum |q| |K| for
    128 products summed in fp32, 0 where the sums are exact.  lse: that error, and fp32 of a logit (2^-22
    holds its product and two sums).  Nothing absolute: a small result is held to its own size."""
    w, wl, mag, big = want
    out, lse = out.double().cpu(), lse.double().cpu()
    dl = torch.zeros_like(big) if exact else 2.0**-18 * (big + 1)
    tol = 2.0**-8 * w.abs() + (2.0**-11 + 2 * dl[..., None]) * mag + 2.0**-134
    bad = ~((out - w).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4], out[bad][:4], w[bad][:4])
    fin = torch.isfinite(wl)
    assert torch.equal(lse == -math.inf, wl == -math.inf) and torch.isfinite(lse[fin]).all()
    assert ((lse - wl).abs()[fin] <= 2.0**-22 * wl.abs()[fin] + 1e-6 + dl[fin]).all()


# ------------------------------------------------------------------ logits

def one_dim(size, sign, lo=1.0):
    """Queries of one element, keys of E4M3 numbers in lo .. 448 there: every score is one exact
    product, tokens of one code tie, others lie 2^-4 of the logit apart."""
    def edit(q, kp, ks, vp, vs, table):
        g = torch.Generator().manual_seed(1)
        x = torch.exp2(torch.rand(kp.numel() // 128, generator=g) * math.log2(448 / lo)).mul_(lo).clamp_max_(448)
        kp.view(-1, 128).zero_()
        kp.view(-1, 128)[:, 5] = codes(x)
        ks[:] = 127
        q.zero_()
        q[:, :, 5] = sign * size / 448 * math.sqrt(128)  # scale is 1 / sqrt(128)
    return edit


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [9e7, 3e8, 5e8, 2e9, 1e12, 1e20, 1e30, 1e36])
def test_large_logits(size, sign):
    """Of logits far apart the largest alone counts, and those that tie with it, whatever its size."""
    for q, H, Hkv in ((1, 16, 1), (4, 20, 4), (3, 8, 1), (4, 16, 1)):
        out, lse, want, _ = attention([300, 40, 1, 129, 700], q, H, Hkv, seed=q, edit=one_dim(size, sign))
        near(out, lse, want, exact=True)
    m.mx4_check_status()


def test_large_logits_long():
    """Pieces of a row in many CTAs, and lists."""
    for size, sign in ((5e8, 1), (2e9, -1), (1e31, -1)):
        out, lse, want, _ = attention([30000, 5000], 1, 16, 1, seed=5, edit=one_dim(size, sign))
        near(out, lse, want, exact=True)
        blocks = [[3, 0, 30, 7], [5, 5, 2, 39]]
        out, lse, want, _ = attention([30000, 5000], 1, 16, 1, seed=5, blocks=blocks, edit=one_dim(size, sign))
        near(out, lse, want, exact=True)


@pytest.mark.parametrize("size,unit", [(2.0**20, 1), (2.0**23, 1), (2.0**25, 4)])
def test_logits_large_and_near(size, unit):
    """Logits of 2^20 to 2^25 that differ by `unit` up to 12: two exact products whose sum has 24 bits,
    so that the weights are as exact as those of small logits."""
    def edit(q, kp, ks, vp, vs, table):
        g = torch.Generator().manual_seed(2)
        rows = kp.view(-1, 128)
        rows.zero_()
        # larger ones later: references move again and again
        rank = torch.arange(rows.shape[0]) % 128 / 128.0
        x = 12 * torch.rand(rows.shape[0], generator=g) * (0.2 + rank)
        rows[:, 0] = codes(256.0)
        rows[:, 7] = codes((x / unit).round().mul(unit).clamp(0, 12))
        ks[:] = 127
        q.zero_()
        q[:, :, 0] = size / 256
        q[:, :, 7] = 1.0
    for q, H, Hkv in ((1, 16, 1), (4, 20, 4), (3, 8, 1)):
        out, lse, want, _ = attention([700, 64, 2000], q, H, Hkv, seed=7, scale=1.0, edit=edit)
        near(out, lse, want, exact=True)


# ------------------------------------------------------------------ V scales

def v_scale(blocks, low=20, rest=None):
    """V scales `low`, and those of 32-token blocks (sequence, block) `blocks[...]`."""
    def edit(q, kp, ks, vp, vs, table):
        vs[:] = low
        for (s, b), e in blocks.items():
            vs[table[s, b // 4], :, b % 4] = e
        if rest:
            rest(q, kp, ks, vp, vs, table)
    return edit


@pytest.mark.parametrize("high", [150, 200, 247])
@pytest.mark.parametrize("q,H,Hkv", [(2, 16, 1), (2, 4, 2), (8, 3, 1), (3, 16, 1), (8, 16, 1)])
def test_a_large_scale_out_of_sight(q, H, Hkv, high):
    """The last tokens begin a block whose V scale is far above the others: the queries before them
    keep their small results."""
    edit = v_scale({(0, 1): high, (1, 8): high, (2, 4): high})
    out, lse, want, _ = attention([33, 257, 128 + q - 1], q, H, Hkv, seed=3, edit=edit)
    near(out, lse, want)


@pytest.mark.parametrize("low,high", [(0, 130), (0, 247), (20, 150), (60, 240)])
@pytest.mark.parametrize("q,H,Hkv", [(1, 16, 1), (2, 12, 1), (4, 16, 1), (1, 8, 2)])
def test_a_large_scale_without_weight(q, H, Hkv, low, high):
    """Blocks of far larger V scales and logits 300 below the others' (weights of 2^-430), first, in the
    middle and last; every other head gives them all its weight."""
    def rest(qq, kp, ks, vp, vs, table):
        rows = kp.view(*kp.shape[:2], 128, 128)
        rows[..., 3] = 0
        for s, b in far:
            rows[table[s, b // 4], :, b % 4 * 32:b % 4 * 32 + 32, 3] = codes(-448.0)
        qq[:, :, 3] = 1000.0
        qq[:, 1::2, 3] = -1000.0
    far = [(0, 0), (0, 5), (1, 7), (2, 40), (2, 93)]
    edit = v_scale({x: high for x in far}, low, rest)
    out, lse, want, _ = attention([300, 256, 3000], q, H, Hkv, seed=4, klo=120, khi=121, edit=edit)
    near(out, lse, want)


@pytest.mark.parametrize("high", [140, 247])
def test_a_large_scale_in_another_piece(high):
    """Pieces of a row in several CTAs, one with a block of a far larger V scale and no weight."""
    def rest(qq, kp, ks, vp, vs, table):
        rows = kp.view(*kp.shape[:2], 128, 128)
        rows[..., 3] = 0
        rows[table[0, 61], :, 64:96, 3] = codes(-448.0)
        qq[:, :, 3] = 1000.0
    edit = v_scale({(0, 61 * 4 + 2): high}, 8, rest)
    for q in (1, 2):
        out, lse, want, _ = attention([20000], q, 16, 1, seed=6, klo=120, khi=121, edit=edit)
        near(out, lse, want)


def test_scales_climb():
    """V scales that grow by powers of 2^40 along a sequence, the weight on the first block."""
    def rest(qq, kp, ks, vp, vs, table):
        rows = kp.view(*kp.shape[:2], 128, 128)
        rows[..., 3] = codes(-448.0)
        rows[table[0, 0], :, :32, 3] = 0
        qq[:, :, 3] = 1000.0
    edit = v_scale({(0, b): 7 + 40 * b for b in range(1, 7)}, 10, rest)
    for q, H in ((1, 16), (3, 8), (4, 16)):
        out, lse, want, _ = attention([210], q, H, 1, seed=8, klo=120, khi=121, edit=edit)
        near(out, lse, want)


def test_some_weight_on_a_large_scale():
    """A weight of 2^-14 on a block whose V scale is 2^70 and more above: it decides the result."""
    def rest(qq, kp, ks, vp, vs, table):
        rows = kp.view(*kp.shape[:2], 128, 128)
        rows[..., 3] = 0
        rows[table[0, 1], :, 32:64, 3] = codes(-9.0)
        qq.zero_()
        qq[:, :, 3] = 1.0
    edit = v_scale({(0, 5): 180}, 90, rest)
    for q, H in ((1, 16), (3, 8), (4, 16)):
        out, lse, want, _ = attention([300], q, H, 1, seed=9, klo=127, khi=128, scale=1.0, edit=edit)
        near(out, lse, want, exact=True)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("q,H,Hkv", [(1, 16, 1), (3, 8, 2), (3, 8, 1), (8, 16, 1), (2, 20, 4)])
def test_scales_and_levels(q, H, Hkv, zeros):
    """Each block's V scale is any power of two (or a third of the blocks are zeros of the least scale,
    the others usual), its logits are about 0 or 309 above or below; odd heads see that upside down."""
    def edit(qq, kp, ks, vp, vs, table):
        g = torch.Generator().manual_seed(q)
        level = torch.randint(-1, 2, (*ks.shape[:2], 4, 1), generator=g) * 448.0
        rows = kp.view(*kp.shape[:2], 4, 32, 128)
        rows[..., 3] = codes(level).expand(-1, -1, -1, 32)
        if zeros:
            at = torch.rand(vs.shape, generator=g) < 1 / 3
            vs[at] = 0
            vp.view(*vs.shape, 4096)[at] = 0
        else:
            vs[:] = torch.randint(0, 248, vs.shape, generator=g, dtype=torch.uint8)
        qq[:, :, 3] = 1000.0
        qq[:, 1::2, 3] = -1000.0
    lens = [6000, 33, 700, 31, 64, 129]
    out, lse, want, _ = attention(lens, q, H, Hkv, seed=q, klo=120, khi=121, edit=edit)
    near(out, lse, want)
    g = torch.Generator().manual_seed(q)
    blocks = [torch.randperm((L - q + j) // 128 + 1, generator=g)[:12].tolist() for L in lens for j in range(q)]
    out, lse, want, _ = attention(lens, q, H, Hkv, seed=q, blocks=blocks, klo=120, khi=121, edit=edit)
    near(out, lse, want)


@pytest.mark.parametrize("byte", [0, 1, 6, 12, 20])
def test_small_results_of_long_contexts(byte):
    """Near-equal weights of many tokens, values next to the least normal number."""
    def edit(q, kp, ks, vp, vs, table):
        vs[:] = byte
        vp[:] = codes(100.0)
        q.mul_(0.01)
    for lens, q, H in (([12000], 1, 16), ([32768, 500], 1, 16), ([300, 40], 1, 16), ([9000], 4, 10)):
        out, lse, want, _ = attention(lens, q, H, 1, seed=10, edit=edit)
        near(out, lse, want)


def test_usual_values_held_to_their_size():
    """The bound without an absolute part on usual inputs, and on V scales of 2^-127."""
    for q, H, Hkv in ((1, 16, 1), (2, 7, 1), (4, 20, 4), (3, 24, 4), (8, 16, 1)):
        for v in (None, 0):
            def edit(qq, kp, ks, vp, vs, table):
                if v is not None:
                    vs[:] = v
            out, lse, want, _ = attention([0, 1, 33, 160, 700], q, H, Hkv, seed=q, edit=edit)
            near(out, lse, want)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("byte", [248, 251, 253, 254])
def test_append_behind_a_large_scale(byte):
    """A block that another writer gave a scale above 2^120 keeps it; new rows are its codes, in the
    form for single tokens and in that for prompts."""
    def edit(x, kp, ks, vp, vs, table):
        ks[:] = byte
        vs[:] = byte
        x[:, -256:] = torch.tensor([2.0**120, -2.0**119, 2.0**125, 2.0**117, 1.75 * 2.0**127, 0.0, 1.0, -2.0**118] * 32)
    for new in ([1, 2], [20, 9]):
        append([30, 50], new, 1, 1, torch.float32, 0, False, byte, edit=edit)
    m.mx4_check_status()


@pytest.mark.parametrize("base", [1e4, 5e5, 1e7])
@pytest.mark.parametrize("inter", [False, True])
def test_slow_pairs(base, inter):
    """Angles of pairs that turn by 1e-9 a position keep all bits of an fp32 number."""
    T, R_ = 10, 128
    f = m.rope_frequencies(R_, base, "linear", 8.0)[0]
    ph = m.rope_phases(f)
    x = torch.zeros((T, 1, 128))
    a = 2 * torch.arange(64) if inter else torch.arange(64)
    x[..., a] = 1.0
    pos = torch.tensor([0, 1, 2, 3, 17, 1000, -1, -5, 123456, 2**31 + 7])
    i = dict(dtype=torch.int32, device=DEV)
    pools = [torch.zeros((1, 1, 16384), dtype=torch.uint8, device=DEV) for _ in range(2)]
    pools += [torch.zeros((1, 1, 4), dtype=torch.uint8, device=DEV) for _ in range(2)]
    qo = torch.zeros((T, 1, 128), dtype=torch.bfloat16, device=DEV)
    m.fp8_rope_append(x.to(DEV), x.to(DEV), x.to(DEV), torch.tensor([0, T], **i), torch.zeros((1, 1), **i),
                      torch.tensor([T], **i), *pools, qo, phases=ph.to(DEV), positions=pos.to(DEV),
                      interleaved=inter)
    want = R.turned(x, pos.tolist(), ph.tolist(), inter, 1.0)
    # bf16; the angle (of -pi .. pi) as an fp32 number and times pi, 2^-23 of it; the sine's 2 ulp
    turns = torch.tensor([[((int(w) * int(p) + 2**63) % 2**64 - 2**63) / 2.0**64 for w in ph.tolist()]
                          for p in pos.tolist()], dtype=F64)
    angle = 2 * math.pi * turns.abs()
    tol = (2.0**-8 + 2.0**-21) * want.abs()
    for d in (a, a + 1 if inter else a + 64):
        tol[:, 0, d] += 2.0**-23 * angle
    got = qo.cpu().double()
    bad = (got - want).abs() > tol
    assert not bad.any(), (bad.nonzero()[:5], got[bad][:5], want[bad][:5])
