"""The speculative decode step's calls on the CPU: refusals of the C entries and the
binding, workspace sizes, and the reference implementations checked by themselves."""
import ctypes

import numpy as np
import pytest
import torch

import _spec_ref as R
import mxfp4_sparse_paged_gb300 as m
from mxfp4_sparse_paged_gb300 import build as B_


@pytest.fixture(scope="module")
def lib():
    B_.build()
    return m._load()


F = ctypes.c_float
ONE = ctypes.c_void_p(4096)  # a non-NULL address that is never read: every call stops before


def _tree(lib, **kw):
    a = dict(q=ONE, B=1, N=1, H=16, Hkv=1, k=ONE, v=ONE, ps=8704, hs=8704, P=1, bt=ONE, W=1, sl=ONE,
             nn=None, tm=None, win=0, sinks=0, scale=F(0.1), out=ONE, lse=None, ws=ONE,
             wsb=1 << 40, st=None)
    a.update(kw)
    return lib.tree_paged_decode(*a.values())


@pytest.mark.parametrize("kw,code,word", [
    (dict(N=0), -2, "N"), (dict(N=65), -2, "N"), (dict(H=15, Hkv=2), -2, "H"), (dict(H=129), -2, "H"),
    (dict(Hkv=9, H=18), -2, "Hkv"), (dict(Hkv=0), -2, "Hkv"), (dict(B=-1), -2, "B"),
    (dict(B=65536), -2, "B"),
    (dict(win=-1), -1, "window"), (dict(sinks=-1), -1, "sinks"),
    (dict(scale=F(float("nan"))), -1, "scale"), (dict(scale=F(float("inf"))), -1, "scale"),
    (dict(q=None), -1, "NULL"), (dict(out=None), -1, "NULL"), (dict(k=None), -1, "NULL"),
    (dict(bt=None), -1, "NULL"), (dict(sl=None), -1, "NULL"),
    (dict(q=ctypes.c_void_p(4104)), -1, "misaligned"), (dict(k=ctypes.c_void_p(4112)), -1, "32"),
    (dict(ps=8720), -1, "32"), (dict(ps=8192), -1, "stride"), (dict(P=0), -1, "num_pages"),
    (dict(Hkv=2, hs=8192), -1, "stride"), (dict(W=0), -1, "bt_width"),
    (dict(tm=ctypes.c_void_p(4100)), -1, "misaligned"),
])
def test_tree_paged_decode_refusals(lib, kw, code, word):
    assert _tree(lib, **kw) == code
    assert word in m.mx4_last_error()


def test_tree_paged_decode_empty_batch_and_workspace(lib):
    assert _tree(lib, B=0, q=None, k=None) == 0
    need = m.tree_paged_decode_workspace(4, 8, 16, 1)
    if need:
        assert _tree(lib, B=4, N=8, wsb=need - 1) == -3
        assert _tree(lib, B=4, N=8, ws=None) == -1
    assert m.tree_paged_decode_workspace(0, 8, 16, 1) == 0
    assert m.tree_paged_decode_workspace(4, 65, 16, 1) == 0


def _verify(lib, **kw):
    a = dict(t=ONE, tb=64, tn=16, d=ONE, db=64, dn=16, tok=ONE, par=ONE, u=ONE, us=ONE, nn=None, B=2,
             N=4, V=16, path=ONE, na=ONE, nx=ONE, st=None)
    a.update(kw)
    return lib.verify_drafts(*a.values())


@pytest.mark.parametrize("kw,code,word", [
    (dict(N=0), -2, "N"), (dict(N=65), -2, "N"), (dict(V=0), -2, "V"), (dict(V=(1 << 24) + 1), -2, "V"),
    (dict(B=65536), -2, "B"), (dict(t=None), -1, "NULL"), (dict(tok=None), -1, "NULL"),
    (dict(nx=None), -1, "NULL"), (dict(tn=15), -1, "stride"), (dict(dn=15), -1, "stride"),
    (dict(t=ctypes.c_void_p(4098)), -1, "misaligned"),
])
def test_verify_drafts_refusals(lib, kw, code, word):
    assert _verify(lib, **kw) == code
    assert word in m.mx4_last_error()
    assert _verify(lib, B=0, t=None) == 0


def _accept(lib, **kw):
    a = dict(path=ONE, na=ONE, sl=ctypes.c_void_p(8192), nn=None, B=2, N=4, bt=ONE, W=1, k=ONE, v=ONE,
             ps=8704, hs=8704, Hkv=1, idx=ONE, ips=8704, fp8=0, P=1, new=ctypes.c_void_p(16384),
             st=None)
    a.update(kw)
    return lib.mx4_accept_rows(*a.values())


@pytest.mark.parametrize("kw,code,word", [
    (dict(N=0), -2, "N"), (dict(N=65), -2, "N"), (dict(Hkv=9), -2, "Hkv"), (dict(B=-1), -2, "B"),
    (dict(path=None), -1, "NULL"), (dict(k=None), -1, "NULL"), (dict(new=None), -1, "NULL"),
    (dict(new=ctypes.c_void_p(8196)), -1, "overlap"), (dict(ips=8192), -1, "stride"),
    (dict(fp8=1), -1, "stride"), (dict(ps=8712), -1, "16-byte"), (dict(W=0), -1, "bt_width"),
])
def test_accept_rows_refusals(lib, kw, code, word):
    assert _accept(lib, **kw) == code
    assert word in m.mx4_last_error()
    assert _accept(lib, B=0, path=None) == 0


def test_accept_rows_without_heads_needs_index_pages(lib):
    assert _accept(lib, Hkv=0, k=None, v=None, idx=None) == -1
    assert "NULL" in m.mx4_last_error()
    assert _accept(lib, Hkv=-1) == -2


def _fork(lib, **kw):
    a = dict(rows=ONE, n=2, bt=ctypes.c_void_p(1 << 20), B=2, W=3, sl=ctypes.c_void_p(2 << 20), refs=ONE,
             fl=ONE, fc=ONE, k=ONE, v=ONE, ps=8704, hs=8704, Hkv=1, idx=None, ips=0, fp8=0, P=4,
             ct=ctypes.c_void_p(3 << 20), cl=ctypes.c_void_p(4 << 20), st=None)
    a.update(kw)
    return lib.mx4_fork_pages(*a.values())


@pytest.mark.parametrize("kw,code,word", [
    (dict(n=65536), -2, "n"), (dict(Hkv=0), -2, "Hkv"), (dict(rows=None), -1, "NULL"),
    (dict(refs=None), -1, "NULL"), (dict(B=0), -1, "B"), (dict(W=0), -1, "bt_width"),
    (dict(ct=ctypes.c_void_p((1 << 20) + 4)), -1, "overlap"),
    (dict(cl=ctypes.c_void_p((2 << 20) + 4)), -1, "overlap"), (dict(P=0), -1, "num_pages"),
])
def test_fork_pages_refusals(lib, kw, code, word):
    assert _fork(lib, **kw) == code
    assert word in m.mx4_last_error()
    assert _fork(lib, n=0, rows=None) == 0


def test_free_pages_refusals(lib):
    a = [ONE, 2, 3, ONE, ONE, 4, ONE, ONE, None]
    for i, v, code in ((0, None, -1), (3, None, -1), (6, None, -1), (2, 0, -1), (5, 0, -1), (1, 65536, -2)):
        b = list(a)
        b[i] = v
        assert lib.mx4_free_pages(*b) == code
    assert lib.mx4_free_pages(None, 0, 3, ONE, ONE, 4, ONE, ONE, None) == 0


def _host():
    i32, f32 = torch.int32, torch.float32
    B, N, H, V, P, W = 2, 4, 16, 10, 5, 3
    return dict(q=torch.zeros((B, N, H, 128), dtype=torch.bfloat16),
                out=torch.zeros((B, N, H, 128), dtype=torch.bfloat16),
                kp=torch.zeros((P, 1, 8704), dtype=torch.uint8),
                vp=torch.zeros((P, 1, 8704), dtype=torch.uint8),
                ip=torch.zeros((P, 8704), dtype=torch.uint8),
                bt=torch.zeros((B, W), dtype=i32), sl=torch.ones(B, dtype=i32),
                mask=torch.zeros((B, N), dtype=torch.int64), nn=torch.ones(B, dtype=i32),
                lse=torch.zeros((B, N, H)), ws=torch.zeros(64, dtype=torch.uint8),
                t=torch.zeros((B, N, V)), d=torch.zeros((B, N, V)), tok=torch.zeros((B, N), dtype=i32),
                par=torch.zeros((B, N), dtype=i32), u=torch.zeros((B, N)), us=torch.zeros(B),
                path=torch.zeros((B, N), dtype=i32), na=torch.zeros(B, dtype=i32),
                nx=torch.zeros(B, dtype=i32), new=torch.zeros(B, dtype=i32),
                rows=torch.zeros(3, dtype=i32), refs=torch.zeros(P, dtype=i32),
                fl=torch.zeros(P, dtype=i32), fc=torch.zeros(1, dtype=i32),
                ct=torch.zeros((3, W), dtype=i32), cl=torch.zeros(3, dtype=i32))


def _binding(a):
    return {
        "tree": lambda: m.tree_paged_decode(a["q"], a["kp"], a["vp"], a["bt"], a["sl"], 0.1, a["out"],
                                            a["ws"], a["mask"], a["nn"], 4, 1, a["lse"]),
        "verify": lambda: m.verify_drafts(a["t"], a["d"], a["tok"], a["par"], a["u"], a["us"],
                                          a["path"], a["na"], a["nx"], a["nn"]),
        "accept": lambda: m.mx4_accept_rows(a["path"], a["na"], a["sl"], a["bt"], a["kp"], a["vp"],
                                            a["ip"], a["new"], a["nn"]),
        "fork": lambda: m.mx4_fork_pages(a["rows"], a["bt"], a["sl"], a["refs"], a["fl"], a["fc"],
                                         a["kp"], a["vp"], a["ip"], a["ct"], a["cl"]),
        "free": lambda: m.mx4_free_pages(a["ct"], a["cl"], a["refs"], a["fl"], a["fc"]),
    }


@pytest.mark.parametrize("name", ["tree", "verify", "accept", "fork", "free"])
def test_bindings_refuse_host_tensors(lib, name):
    with pytest.raises(ValueError, match="CUDA tensor"):
        _binding(_host())[name]()


@pytest.mark.parametrize("name,key,shape,dtype", [
    ("tree", "out", (2, 4, 8, 128), torch.bfloat16), ("tree", "bt", (1, 3), torch.int32),
    ("tree", "mask", (2, 3), torch.int64), ("tree", "mask", (2, 4), torch.int32),
    ("tree", "nn", (3,), torch.int32), ("tree", "lse", (2, 4), torch.float32),
    ("tree", "q", (2, 4, 16, 64), torch.bfloat16), ("tree", "q", (2, 4, 16, 128), torch.float16),
    ("tree", "vp", (5, 2, 8704), torch.uint8), ("tree", "sl", (2,), torch.int64),
    ("verify", "d", (2, 4, 9), torch.float32), ("verify", "t", (2, 4, 10), torch.bfloat16),
    ("verify", "tok", (2, 3), torch.int32), ("verify", "u", (2, 4), torch.float64),
    ("verify", "us", (3,), torch.float32), ("verify", "path", (2, 5), torch.int32),
    ("accept", "na", (3,), torch.int32), ("accept", "ip", (4, 8704), torch.uint8),
    ("accept", "new", (1,), torch.int32), ("accept", "bt", (3, 3), torch.int32),
    ("fork", "ct", (3, 4), torch.int32), ("fork", "refs", (4,), torch.int32),
    ("fork", "fc", (2,), torch.int32), ("free", "cl", (2,), torch.int32),
    ("free", "fl", (6,), torch.int32),
])
def test_bindings_refuse_inconsistent_arguments(lib, name, key, shape, dtype):
    a = _host()
    a[key] = torch.zeros(shape, dtype=dtype)
    with pytest.raises((ValueError, TypeError)) as ei:
        _binding(a)[name]()
    assert "CUDA tensor" not in str(ei.value)


def test_reference_verify_follows_the_targets_distribution():
    # 40000 draws of a two-child tree over four tokens: the first token after the root is
    # distributed as the target's row whatever the draft's row is.  Expected counts of
    # 4000 or more; 5 standard deviations
    rng = np.random.default_rng(3)
    p = np.array([0.1, 0.2, 0.3, 0.4], np.float32)
    q = np.array([0.4, 0.3, 0.2, 0.1], np.float32)
    n = 40000
    target = np.broadcast_to(p, (n, 3, 4))
    draft = np.broadcast_to(q, (n, 3, 4))
    tokens = np.zeros((n, 3), np.int32)
    tokens[:, 1:] = rng.choice(4, size=(n, 2), p=q.astype(np.float64) / q.sum(dtype=np.float64))
    parents = np.tile(np.array([-1, 0, 0], np.int32), (n, 1))
    u, us = rng.random((n, 3), dtype=np.float32), rng.random(n, dtype=np.float32)
    path, acc, nxt = R.verify(target, draft, tokens, parents, u, us, np.full(n, 3))
    first = np.where(acc > 1, tokens[np.arange(n), np.maximum(path[:, 1], 0)], nxt)
    count = np.bincount(first, minlength=4)
    assert np.all(np.abs(count - n * p) <= 5 * np.sqrt(n * p * (1 - p)))


def test_reference_attention_is_the_plain_softmax():
    # everything visible and one head: the textbook softmax over the decoded rows
    rng = np.random.default_rng(4)
    kp, vp = R.random_pages(rng, 3, 1), R.random_pages(rng, 3, 1)
    bt = np.array([[2, 0, 1]], np.int32)
    q = rng.standard_normal((1, 1, 1, 128)).astype(np.float32)
    out, lse, _, _ = R.attend(q, kp, vp, bt, [300], [1], [[1]], 0, 0, 0.1)
    k, v = R.rows_of(kp, bt[0], 0, 300), R.rows_of(vp, bt[0], 0, 300)
    l = torch.from_numpy(0.1 * (k @ q[0, 0, 0]))
    assert np.allclose(out[0, 0, 0], (torch.softmax(l, 0).numpy() @ v), rtol=1e-12)
    assert np.isclose(lse[0, 0, 0], torch.logsumexp(l, 0).item(), rtol=1e-12)
