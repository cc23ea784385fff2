"""The 8-bit cache's calls without a GPU: refusals, rotary frequencies and phases, slots."""
import ctypes
import math

import pytest
import torch

import mxfp4_sparse_paged_gb300 as m
from mxfp4_sparse_paged_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return m._load()


def _args(T=4, H=16, Hkv=2, B=4, W=3, k=8):
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    return {"q": torch.zeros((T, H, 128), dtype=bf), "k": torch.zeros((T, Hkv, 128), dtype=bf),
            "v": torch.zeros((T, Hkv, 128), dtype=bf), "cu": torch.arange(B + 1, dtype=i32),
            "bt": torch.zeros((B, W), dtype=i32), "sl": torch.ones(B, dtype=i32),
            "kp": torch.zeros((3, Hkv, 16384), dtype=u8), "vp": torch.zeros((3, Hkv, 16384), dtype=u8),
            "ks": torch.zeros((3, Hkv, 4), dtype=u8), "vs": torch.zeros((3, Hkv, 4), dtype=u8),
            "qo": torch.zeros((T, H, 128), dtype=bf), "ph": torch.zeros(64, dtype=torch.int64),
            "pos": torch.zeros(T, dtype=torch.int64), "out": torch.zeros((T, H, 128), dtype=bf),
            "lse": torch.zeros((T, H)), "idx": torch.zeros((T, k), dtype=i32),
            "ws": torch.zeros(64, dtype=u8), "sc": torch.zeros((T, W)),
            "iq": torch.zeros((T, 128), dtype=bf), "ip": torch.zeros((3, 8704), dtype=u8),
            "fp8": torch.zeros((3, 16384), dtype=u8)}


def _calls(a):
    kv = ("kp", "vp", "ks", "vs")
    return {
        "append": lambda: m.fp8_rope_append(a["q"], a["k"], a["v"], a["cu"], a["bt"], a["sl"],
                                            *(a[n] for n in kv), a["qo"], phases=a["ph"],
                                            positions=a["pos"]),
        "paged": lambda: m.fp8_paged_decode(a["q"], 1, *(a[n] for n in kv), a["bt"], a["sl"], 0.1,
                                            a["out"], a["ws"], lse=a["lse"]),
        "block": lambda: m.fp8_block_decode(a["q"], 1, *(a[n] for n in kv), a["bt"], a["sl"],
                                            a["idx"], 0.1, a["out"], a["ws"], lse=a["lse"]),
        "score": lambda: m.index_block_score(a["iq"], 1, a["ip"], a["bt"], a["sl"], a["sc"]),
        "score8": lambda: m.index_block_score_fp8(a["iq"], 1, a["fp8"], a["bt"], a["sl"], 0.5,
                                                  a["sc"]),
        "topk": lambda: m.block_topk(a["sc"], a["sl"], 1, a["idx"]),
    }


def test_host_tensors_stop_at_the_device_check(lib):
    for name, call in _calls(_args()).items():
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("call,key,shape", [
    ("append", "v", (4, 1, 128)), ("append", "k", (3, 2, 128)), ("append", "cu", (4,)),
    ("append", "bt", (3, 3)), ("append", "ks", (3, 2, 3)), ("append", "vp", (3, 1, 16384)),
    ("append", "qo", (4, 8, 128)), ("append", "pos", (3,)), ("append", "k", (4, 2, 64)),
    ("paged", "out", (4, 8, 128)), ("paged", "lse", (4, 8)), ("paged", "q", (5, 16, 128)),
    ("paged", "bt", (3, 3)), ("paged", "vs", (2, 2, 4)), ("paged", "kp", (3, 2, 8704)),
    ("block", "idx", (3, 8)), ("block", "bt", (5, 3)), ("score", "sc", (3, 3)),
    ("score", "bt", (3, 3)), ("score8", "iq", (4, 64)), ("topk", "sc", (3, 3)),
    ("topk", "idx", (5, 8)),
])
def test_shapes_are_refused(lib, call, key, shape):
    a = _args()
    a[key] = torch.zeros(shape, dtype=a[key].dtype)
    with pytest.raises(ValueError) as e:
        _calls(a)[call]()
    assert "CUDA tensor" not in str(e.value), str(e.value)


@pytest.mark.parametrize("call,key,dtype", [
    ("append", "k", torch.float16), ("append", "q", torch.float32), ("append", "cu", torch.int64),
    ("append", "ks", torch.int8), ("append", "ph", torch.int32), ("append", "qo", torch.float32),
    ("paged", "q", torch.float32), ("paged", "out", torch.float32), ("block", "idx", torch.int64),
    ("score", "sc", torch.bfloat16), ("topk", "sc", torch.float64), ("paged", "kp", torch.int8),
])
def test_types_are_refused(lib, call, key, dtype):
    a = _args()
    a[key] = a[key].to(dtype)
    with pytest.raises(TypeError):
        _calls(a)[call]()


def test_strides(lib):
    a = _args()
    fused = torch.zeros((4, 20 * 128), dtype=torch.bfloat16).unflatten(1, (20, 128))
    a["q"], a["k"], a["v"] = fused[:, :16], fused[:, 16:18], fused[:, 18:]  # a fused projection
    with pytest.raises(ValueError, match="CUDA tensor"):
        _calls(a)["append"]()
    a["k"] = torch.zeros((4, 128, 2), dtype=torch.bfloat16).transpose(1, 2)
    with pytest.raises(ValueError, match="contiguous"):
        _calls(a)["append"]()
    a = _args()
    a["kp"] = torch.zeros((3, 4, 16384), dtype=torch.uint8)[:, ::2]  # (V's strides differ)
    with pytest.raises(ValueError, match="same shape and strides"):
        _calls(a)["paged"]()
    a["qo"] = None
    with pytest.raises(ValueError, match="together"):
        _calls(a)["append"]()


def _c(lib, name, **kw):
    """The C call with arguments that are fine but for kw; addresses are never read."""
    p, far = 1 << 20, 1 << 30
    f = ctypes.c_float
    base = {
        "fp8_rope_append": dict(q=p, qs=2048, k=p, kst=256, v=p, vst=256, fp32=0, T=4, H=16, Hkv=2,
                                cu=p, B=4, pos=None, ph=p, rot=128, inter=0, factor=f(1.0), bt=p,
                                W=3, sl=p, kp=p, vp=p, ps=32768, hs=16384, P=3, ks=p, vs=p, qo=far,
                                stream=None),
        "fp8_paged_decode": dict(q=p, T=4, qps=1, H=16, Hkv=2, kp=p, vp=p, ps=32768, hs=16384, P=3,
                                 ks=p, vs=p, bt=p, B=4, W=3, sl=p, scale=f(0.1), out=far, lse=p, ws=p,
                                 nws=1 << 40, stream=None),
        "fp8_block_decode": dict(q=p, T=4, qps=1, H=16, Hkv=2, kp=p, vp=p, ps=32768, hs=16384, P=3,
                                 ks=p, vs=p, bt=p, B=4, W=3, sl=p, idx=p, kb=8, scale=f(0.1), out=far,
                                 lse=p, ws=p, nws=1 << 40, stream=None),
        "block_topk": dict(sc=p, ld=3, sl=p, B=4, qps=1, k=8, first=1, last=2, idx=far, stream=None),
        "index_block_score": dict(iq=p, T=4, qps=1, ip=p, ps=8704, P=3, bt=p, B=4, W=3, sl=p, sc=p,
                                  ld=3, stream=None),
        "index_block_score_fp8": dict(iq=p, T=4, qps=1, ip=p, ps=16384, P=3, bt=p, B=4, W=3, sl=p,
                                      scale=f(0.1), sc=p, ld=3, stream=None),
    }[name]
    assert set(kw) <= set(base)
    args = list({**base, **kw}.values())
    rc = getattr(lib, name)(*args)
    # the binding's form of the call: one array of words
    how = {"fp8_rope_append": m._APPEND, "fp8_paged_decode": m._PAGED, "fp8_block_decode": m._BLOCK,
           "block_topk": m._TOPK, "index_block_score": m._SCORE, "index_block_score_fp8": m._SCORE_FP8}[name]
    why = m.mx4_last_error()
    words = how[1](*(0 if x is None else x.value if isinstance(x, f) else x for x in args))
    assert lib.mx4_call_words(how[0], words) == rc and m.mx4_last_error() == why
    return rc


INF, NAN = ctypes.c_float(math.inf), ctypes.c_float(math.nan)


@pytest.mark.parametrize("name,kw,code", [
    ("fp8_rope_append", dict(Hkv=9), -2), ("fp8_rope_append", dict(H=129), -2),
    ("fp8_rope_append", dict(rot=4), -2), ("fp8_rope_append", dict(rot=136), -2),
    ("fp8_rope_append", dict(T=-1), -2), ("fp8_rope_append", dict(T=(1 << 24) + 1), -2),
    ("fp8_rope_append", dict(factor=NAN), -1), ("fp8_rope_append", dict(k=None), -1),
    ("fp8_rope_append", dict(ph=None), -1), ("fp8_rope_append", dict(q=None), -1),
    ("fp8_rope_append", dict(qo=None), -1), ("fp8_rope_append", dict(kst=255), -1),
    ("fp8_rope_append", dict(kst=128), -1), ("fp8_rope_append", dict(qs=1024), -1),
    ("fp8_rope_append", dict(k=(1 << 20) + 4), -1), ("fp8_rope_append", dict(fp32=1, k=(1 << 20) + 8), -1),
    ("fp8_rope_append", dict(ps=16376), -1), ("fp8_rope_append", dict(hs=8192), -1),
    ("fp8_rope_append", dict(P=0), -1), ("fp8_rope_append", dict(vs=None), -1),
    ("fp8_rope_append", dict(W=0), -1), ("fp8_rope_append", dict(T=0), 0),
    ("fp8_paged_decode", dict(qps=0), -2), ("fp8_paged_decode", dict(qps=9), -2),
    ("fp8_paged_decode", dict(H=15), -2), ("fp8_paged_decode", dict(H=256), -2),
    ("fp8_paged_decode", dict(T=5), -1), ("fp8_paged_decode", dict(scale=INF), -1),
    ("fp8_paged_decode", dict(nws=100), -3), ("fp8_paged_decode", dict(ws=None), -1),
    ("fp8_paged_decode", dict(ws=(1 << 20) + 8), -1), ("fp8_paged_decode", dict(out=None), -1),
    ("fp8_paged_decode", dict(q=(1 << 20) + 8), -1), ("fp8_paged_decode", dict(W=(1 << 20) + 1), -2),
    ("fp8_paged_decode", dict(B=65536, T=65536), -2), ("fp8_paged_decode", dict(B=0, T=0), 0),
    ("fp8_paged_decode", dict(out=(1 << 20) + 4 * 16 * 256 - 16), -1),
    ("fp8_rope_append", dict(qo=(1 << 20) + 4 * 2048 * 2 - 8), -1),
    ("fp8_rope_append", dict(v=(1 << 30) + 4 * 16 * 256 - 8), -1),
    ("block_topk", dict(idx=(1 << 20) + 8), -1),
    ("fp8_block_decode", dict(kb=0), -2), ("fp8_block_decode", dict(kb=4097), -2),
    ("fp8_block_decode", dict(idx=None), -1), ("fp8_block_decode", dict(kp=(1 << 20) + 8), -1),
    ("block_topk", dict(k=0), -2), ("block_topk", dict(k=4097), -2), ("block_topk", dict(first=-1), -1),
    ("block_topk", dict(first=7), -1), ("block_topk", dict(last=9), -1),
    ("block_topk", dict(first=2147483647, last=2147483647), -1),
    ("block_topk", dict(ld=0), -2), ("block_topk", dict(ld=65537), -2), ("block_topk", dict(qps=9), -2),
    ("block_topk", dict(idx=None), -1), ("block_topk", dict(B=0), 0),
    ("index_block_score", dict(qps=9), -2), ("index_block_score", dict(T=3), -1),
    ("index_block_score", dict(ps=8703), -1), ("index_block_score", dict(B=0, T=0), 0),
    ("index_block_score_fp8", dict(scale=ctypes.c_float(0.0)), -1),
    ("index_block_score_fp8", dict(ps=8704), -1),
])
def test_c_refusals(lib, name, kw, code):
    assert _c(lib, name, **kw) == code
    assert code == 0 or name in m.mx4_last_error()


def test_call_of_words(lib):
    assert lib.mx4_call_words(99, b"") == -1 and "99" in m.mx4_last_error()


def test_workspaces(lib):
    # two pieces of a tile a CTA and one of each of its eight warps, rows of 132 floats (128 sums; a
    # reference, a total, a unit and nothing), and two words; without a GPU the SM count is taken as
    # 1024.  A tile's rows: M warps of NT times eight.
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 1024
    for rows, M, NT in ((1, 1, 1), (8, 1, 1), (16, 1, 2), (24, 1, 3), (25, 2, 2), (40, 2, 3), (64, 4, 2),
                        (65, 4, 3), (128, 8, 2), (1000, 8, 2)):
        want = sms * ((2 * 8 * NT * M + 8 * 8 * NT) * 132 * 4 + 8)
        if rows <= 128:
            assert m.fp8_block_decode_workspace(3, 16, rows, 1) == want
        if rows % 8 == 0:
            assert m.fp8_paged_decode_workspace(24, 8, rows // 8, 1) == want
    assert m.fp8_paged_decode_workspace(0, 1, 16, 1) == 0


def test_phases():
    """Turns a position in 64-bit fractions: the angle of a far position to 1e-9 turns (fp64's
    rounding of the frequency times the position), modulo one turn."""
    f, grow = m.rope_frequencies(128, base=10000.0)
    assert f.dtype == torch.float32 and grow == 1.0
    p = m.rope_phases(f)
    for i in (0, 1, 17, 63):
        for pos in (0, 1, 1000003, (1 << 31) - 1):
            turns = ((int(p[i]) % 2**64) * pos % 2**64) / 2.0**64
            from fractions import Fraction
            pi2 = Fraction(884279719003555, 140737488355328) + Fraction(24492935982947064, 10**32) * 1
            want = float(Fraction(float(f[i])) * pos / pi2 % 1)
            d = abs(turns - want)
            assert min(d, 1 - d) < 1e-15 * max(1, pos) + 1e-12
    assert m.rope_phases(torch.tensor([-2 * math.pi / 4])).item() % 2**64 == pytest.approx(3 * 2**62, rel=1e-6)


def test_frequencies():
    f, _ = m.rope_frequencies(64, 10000.0)
    lin, g = m.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert torch.equal(lin, (f.double() / 4).float()) or torch.allclose(lin, f / 4, rtol=2**-23)
    assert g == 1.0
    b, _ = m.rope_frequencies(64, 10000.0, "base", 4.0)
    assert b[0] == f[0] and abs(float(b[-1] / f[-1]) - 0.25) < 1e-6  # slowest by 4, fastest kept
    y, g = m.rope_frequencies(64, 10000.0, "bands", 4.0, original_context=4096)
    turns = 4096 * f.double() / (2 * math.pi)
    assert torch.equal(y[turns > 32], f[turns > 32])
    assert torch.allclose(y[turns < 1], f[turns < 1] / 4, rtol=2**-23)
    assert ((y <= f) & (y >= f / 4 * (1 - 2**-22))).all() and g == pytest.approx(0.1 * math.log(4) + 1)
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="what"),
                dict(rot_dim=8, factor=0.5), dict(rot_dim=8, scaling="bands"),
                dict(rot_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            m.rope_frequencies(**bad)


def test_slots():
    """Rows of a ragged append: their slots from the table, none for rows behind the last sequence,
    slots past the pool where there is no page."""
    from mxfp4_sparse_paged_gb300.fp8_step import Fp8Caches, Fp8Step
    caches = Fp8Caches(7, device="cpu")
    table = torch.tensor([[3, 5, -1], [1, 6, 2]], dtype=torch.int32)
    step = Fp8Step.__new__(Fp8Step)
    step.caches, step.block_table = caches, table
    step.seq_lens = torch.tensor([130, 257], dtype=torch.int32)
    cu = torch.tensor([0, 3, 5], dtype=torch.int32)
    assert step.slots(cu, 6).tolist() == [3 * 128 + 127, 5 * 128, 5 * 128 + 1, 6 * 128 + 127, 2 * 128, -1]
    step.seq_lens = torch.tensor([258, 400], dtype=torch.int32)
    got = step.slots(cu, 6)
    assert got[0].item() == 5 * 128 + 127 and (got[1:5] >= 7 * 128).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_phases_are_exact(dtype):
    """Phases to a unit of 2^-64 turns, so that a position of 2^36 keeps an angle to 2^-28 turns:
    against integers, pi to 60 digits."""
    from fractions import Fraction
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10**60)
    g = torch.Generator().manual_seed(0)
    f = torch.cat([m.rope_frequencies(128, b, s, 8.0)[0].to(dtype) for b in (1e4, 1e7) for s in (None, "linear")] + [
        torch.exp2(40 * torch.rand(200, generator=g, dtype=torch.float64) - 35).to(dtype),
        torch.tensor([0.0, 1.0, -1.0, -1e-9, 2 * math.pi, 0.3, -0.7, 3.5, 1e4, 2.0**-60, -2.0**-70], dtype=dtype)])
    got = m.rope_phases(f)
    assert got.dtype == torch.int64
    for x, p in zip(f.tolist(), got.tolist()):
        want = Fraction(x) / (2 * pi) * 2**64
        d = (want - p + 2**63) % 2**64 - 2**63
        assert abs(d) <= 1, (x, p, float(d))


@pytest.mark.parametrize("name,kw", [
    ("block_topk", dict(first=1 << 32)), ("block_topk", dict(last=(1 << 32) + 1)), ("block_topk", dict(k=(1 << 32) + 8)),
    ("block_topk", dict(qps=(1 << 32) + 1)), ("fp8_rope_append", dict(rot=(1 << 32) + 128)),
    ("fp8_rope_append", dict(H=(1 << 40) + 16)), ("fp8_rope_append", dict(Hkv=2 - (1 << 32))),
    ("fp8_block_decode", dict(kb=(1 << 32) + 8)), ("fp8_paged_decode", dict(qps=1 - (1 << 32))),
    ("index_block_score", dict(qps=(1 << 33) + 1))])
def test_numbers_past_32_bits_are_refused(lib, name, kw):
    """The array of words: numbers that would be others in 32 bits."""
    p, far, third = 1 << 20, 1 << 30, 0.1
    how, words = {
        "fp8_rope_append": (m._APPEND, dict(q=p, qs=2048, k=p, kst=256, v=p, vst=256, fp32=0, T=4, H=16, Hkv=2, cu=p, B=4,
                                            pos=0, ph=p, rot=128, inter=0, factor=1.0, bt=p, W=3, sl=p, kp=p, vp=p,
                                            ps=32768, hs=16384, P=3, ks=p, vs=p, qo=far, stream=0)),
        "fp8_paged_decode": (m._PAGED, dict(q=p, T=4, qps=1, H=16, Hkv=2, kp=p, vp=p, ps=32768, hs=16384, P=3, ks=p, vs=p,
                                            bt=p, B=4, W=3, sl=p, scale=third, out=far, lse=p, ws=p, nws=1 << 40, stream=0)),
        "fp8_block_decode": (m._BLOCK, dict(q=p, T=4, qps=1, H=16, Hkv=2, kp=p, vp=p, ps=32768, hs=16384, P=3, ks=p, vs=p,
                                            bt=p, B=4, W=3, sl=p, idx=p, kb=8, scale=third, out=far, lse=p, ws=p,
                                            nws=1 << 40, stream=0)),
        "block_topk": (m._TOPK, dict(sc=p, ld=3, sl=p, B=4, qps=1, k=8, first=1, last=2, idx=far, stream=0)),
        "index_block_score": (m._SCORE, dict(iq=p, T=4, qps=1, ip=p, ps=8704, P=3, bt=p, B=4, W=3, sl=p, sc=p, ld=3, stream=0)),
    }[name]
    assert set(kw) <= set(words)
    assert lib.mx4_call_words(how[0], how[1](*{**words, **kw}.values())) in (-1, -2)
    assert name in m.mx4_last_error()


def test_every_exported_call_is_declared(lib):
    """What the binding calls is in the header."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mx4sp.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    binding = open(m.__file__).read()
    for name in set(re.findall(r"lib\.(\w+)\.argtypes", binding)) | set(re.findall(r"_load\(\)\.(\w+)\(", binding)):
        assert re.search(rf"\b{name}\s*\(", src), name
