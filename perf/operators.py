"""The operators of a speculative decode step over the MXFP4 paged cache: cases, inputs and plain forms.

A speculative step inserts the drafted tokens' rows, attends with all of them at once
(tree_paged_decode: a tree of drafts, or a chain, or a single token; over the whole cache or
over a window and the first tokens), decides which drafts stand (verify_drafts), takes the
others' rows out of the cache (mx4_accept_rows); sequences branch and end by sharing pages
(mx4_fork_pages, mx4_free_pages).

`own` chooses between the plain forms below and the package's calls.  Page format: 128 token
rows of 64 bytes (two e2m1 codes a byte, low nibble first), then 128 rows of 4 e8m0 scale bytes.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
PT, HD, PB, FP8_PB = 128, 128, 8704, 16384
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
SCALE = 1.0 / math.sqrt(HD)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's single token over a short context: the smallest call, latency
        _attn("decode_one_short", B=1, N=1, H=16, Hkv=1, lens="fixed", lo=777, hi=777),
        # the decode batch of the repository's serving workload: 256 ragged contexts
        _attn("decode_batch_ragged", B=256, N=1, H=16, Hkv=1, lens="lognormal", lo=8192, hi=131072),
        # eight sequences of 8192 tokens, each checking a chain of eight drafts
        _attn("chain_of_8", B=8, N=8, H=16, Hkv=1, lens="fixed", lo=8192, hi=8192),
        # a sliding-window layer with visible first tokens, grouped heads of odd width
        _attn("window_sinks_gqa", B=64, N=4, H=40, Hkv=8, lens="uniform", lo=2048, hi=16384,
              window=1000, sinks=5),
        # trees of up to 64 drafts over long contexts: the largest, matrix-product bound
        _attn("tree_of_64_long", B=16, N=64, H=16, Hkv=1, lens="uniform", lo=4096, hi=65536,
              tree=True),
        # one user's chain of three drafts, a small vocabulary
        _verify("verify_one_chain", B=1, N=4, V=32000),
        # a batch of trees against a large vocabulary
        _verify("verify_batch_tree", B=64, N=32, V=131072, tree=True),
        # drafts looked up rather than sampled (no draft probabilities), odd vocabulary
        _verify("verify_given_drafts", B=256, N=8, V=50001, given=True),
        # one user's accepted chain moves together
        _accept("accept_one", B=1, N=8, Hkv=1),
        # a batch of 64-node trees, eight KV heads, fp8 index rows
        _accept("accept_batch_gqa", B=256, N=64, Hkv=8, fp8=True),
        # four samples of one prompt branch and end
        _fork("fork_four_samples", n=4, B=1, Hkv=1, lo=300, hi=300),
        # eight beams for each of 64 sequences, eight KV heads
        _fork("fork_beams_gqa", n=512, B=64, Hkv=8, lo=200, hi=4096),
    ]


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "verify", "verify", "accept", "fork"])
    seed = rng.randrange(1 << 30)
    if kind == "attn":
        Hkv = rng.choice([1, 1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 8, 16]) if Hkv > 1 else rng.choice([1, 4, 7, 16, 16, 16])
        N = _log(rng, 1, 64)
        B = _log(rng, 1, 64)
        # at most 500000 cached tokens of one head in all
        hi = min(65536, max(N + 1, 500000 // (B * Hkv)))
        lo = max(N, min(hi, _log(rng, 1, hi)))
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        c = _attn(None, B=B, N=N, H=G * Hkv, Hkv=Hkv, lens="uniform", lo=lo, hi=hi,
                  window=window, sinks=rng.choice([0, 1, 4, 130]) if window else 0,
                  tree=rng.random() < 0.5)
    elif kind == "verify":
        V = _log(rng, 100, 131072)
        N = _log(rng, 1, 64)
        B = min(_log(rng, 1, 256), max(1, (1 << 28) // (V * N)))
        c = _verify(None, B=B, N=N, V=V, tree=rng.random() < 0.5, given=rng.random() < 0.3)
    elif kind == "accept":
        c = _accept(None, B=_log(rng, 1, 256), N=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]),
                    fp8=rng.random() < 0.5)
    else:
        lo = _log(rng, 1, 4096)
        c = _fork(None, n=_log(rng, 1, 512), B=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]),
                  lo=lo, hi=rng.randint(lo, 4096))
    c["shape_seed"] = seed
    del c["name"]
    return c


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _attn(name, B, N, H, Hkv, lens, lo, hi, window=0, sinks=0, tree=False):
    return {"name": name, "kind": "attn", "B": B, "N": N, "H": H, "Hkv": Hkv, "lens": lens,
            "lo": lo, "hi": hi, "window": window, "sinks": sinks, "tree": tree, "shape_seed": 1}


def _verify(name, B, N, V, tree=False, given=False):
    return {"name": name, "kind": "verify", "B": B, "N": N, "V": V, "tree": tree, "given": given,
            "shape_seed": 2}


def _accept(name, B, N, Hkv, fp8=False):
    return {"name": name, "kind": "accept", "B": B, "N": N, "Hkv": Hkv, "fp8": fp8,
            "shape_seed": 3}


def _fork(name, n, B, Hkv, lo, hi):
    return {"name": name, "kind": "fork", "n": n, "B": B, "Hkv": Hkv, "lo": lo, "hi": hi,
            "shape_seed": 4}


# ------------------------------------------------------------------ shapes (from the case alone)

def _lens(c, at_least):
    r = random.Random(c["shape_seed"])
    if c["lens"] == "fixed":
        return [c["lo"]] * c["B"]
    if c["lens"] == "lognormal":
        return [max(at_least, min(c["hi"], int(c["lo"] * math.exp(r.gauss(0.0, 1.0)))))
                for _ in range(c["B"])]
    return [max(at_least, r.randint(c["lo"], c["hi"])) for _ in range(c["B"])]


def _tree(r, N, tree):
    """parents[j] < j (the root is node 0, parent -1); a chain, or a tree that widens near its root."""
    if not tree:
        return list(range(-1, N - 1))
    return [-1] + [min(j - 1, int(j * r.random() ** 1.5)) for j in range(1, N)]


def _trees(c):
    r = random.Random(c["shape_seed"] + 17)
    return [_tree(r, c["N"], c["tree"]) for _ in range(c["B"])]


def _counts(c):
    """Nodes of each sequence: all N, or (trees) now and then fewer."""
    r = random.Random(c["shape_seed"] + 29)
    if not c["tree"]:
        return [c["N"]] * c["B"]
    return [c["N"] if r.random() < 0.7 else r.randint(1, c["N"]) for _ in range(c["B"])]


def _masks(parents):
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | (1 << j))
    return out


def _visible_span(c, L, n):
    """Cached tokens before the drafts that some node sees: (sinks, first of the window, base)."""
    base = L - n
    lo = max(0, base + 1 - c["window"]) if c["window"] else 0
    return min(c["sinks"], lo), lo, base


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """fp32 rows [..., 128] -> codes uint8 [..., 64] and scale bytes uint8 [..., 4] (OCP MX)."""
    b = x.view(*x.shape[:-1], 4, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    y = torch.ldexp(b, -e.unsqueeze(-1))
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), mids).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    code = code.view(*x.shape[:-1], 64, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _random_pages(g, P, heads):
    pages = torch.empty((P, heads, PB), dtype=torch.uint8, device=DEV)
    for a in range(0, P, max(1, 4096 // heads)):
        b = min(P, a + max(1, 4096 // heads))
        x = torch.randn((b - a, heads, PT, HD), generator=g, device=DEV)
        code, sc = _quantise(x)
        pages[a:b, :, :8192] = code.reshape(b - a, heads, 8192)
        pages[a:b, :, 8192:] = sc.reshape(b - a, heads, 512)
    return pages


def _poison_tails(pages, table, lens, heads):
    """Rows past a sequence's length hold what an empty cache holds: 0xFF."""
    t = torch.tensor([[s, L // PT, L % PT] for s, L in enumerate(lens) if L % PT], device=DEV)
    if t.numel() == 0:
        return
    pid = table[t[:, 0], t[:, 1]].long()
    row = torch.arange(PT, device=DEV)
    dead = row[None] >= t[:, 2][:, None]  # [n, 128]
    v = pages[pid]
    d = v[..., :8192].view(-1, heads, PT, 64)
    s = v[..., 8192:].view(-1, heads, PT, 4)
    d[dead[:, None].expand(-1, heads, -1)] = 255
    s[dead[:, None].expand(-1, heads, -1)] = 255
    pages[pid] = v


def _tables(c, lens, spare, g):
    """Page ids a random permutation of the pool; int32 block table, -1 past a sequence's pages."""
    n = [(L + PT - 1) // PT for L in lens]
    P = sum(n) + spare
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(c["shape_seed"] + 5))
    table = torch.full((len(lens), max(n)), -1, dtype=torch.int32)
    o = 0
    for s, k in enumerate(n):
        table[s, :k] = perm[o:o + k].to(torch.int32)
        o += k
    return table.to(DEV), P, perm[o:].tolist()


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return {"attn": _prepare_attn, "verify": _prepare_verify, "accept": _prepare_accept,
            "fork": _prepare_fork}[c["kind"]](c, g)


def _prepare_attn(c, g):
    B, N, H, Hkv = c["B"], c["N"], c["H"], c["Hkv"]
    counts = _counts(c)
    lens = _lens(c, N)
    table, P, _ = _tables(c, lens, 2, g)
    k, v = _random_pages(g, P, Hkv), _random_pages(g, P, Hkv)
    _poison_tails(k, table, lens, Hkv)
    _poison_tails(v, table, lens, Hkv)
    # logits of standard deviation 2: some tokens stand out, as in a trained model
    q = (2.0 * torch.randn((B, N, H, HD), generator=g, device=DEV)).to(torch.bfloat16)
    masks = None
    if c["tree"]:
        m = np.array([_masks(p) for p in _trees(c)], dtype=np.uint64).view(np.int64)
        masks = torch.from_numpy(m).to(DEV)
    st = {"case": c, "q": q, "k": k, "v": v, "table": table,
          "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
          "n_nodes": torch.tensor(counts, dtype=torch.int32, device=DEV) if c["tree"] else None,
          "masks": masks, "lens": lens, "counts": counts,
          "out": torch.empty((B, N, H, HD), dtype=torch.bfloat16, device=DEV),
          "lse": torch.empty((B, N, H), dtype=torch.float32, device=DEV)}
    if own:
        import mxfp4_sparse_paged_gb300 as m
        n = m.tree_paged_decode_workspace(B, N, H, Hkv)
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return st


def _prepare_verify(c, g):
    B, N, V = c["B"], c["N"], c["V"]
    trees = torch.tensor(_trees(c), dtype=torch.int32)
    logits = torch.randn((B, N, V), generator=g, device=DEV).mul_(2.5)
    target = torch.softmax(logits, -1)
    logits.add_(torch.randn((B, N, V), generator=g, device=DEV), alpha=0.8)
    draft = torch.softmax(logits, -1)
    del logits
    parents = trees.to(DEV)
    tokens = torch.zeros((B, N), dtype=torch.int32, device=DEV)
    rows = torch.arange(B, device=DEV)
    for j in range(1, N):  # each draft drawn from its parent's draft distribution
        p = draft[rows, parents[:, j].long()]
        tokens[:, j] = torch.multinomial(p, 1, generator=g)[:, 0].to(torch.int32)
    st = {"case": c, "target": target, "draft": None if c["given"] else draft, "tokens": tokens,
          "parents": parents, "u": torch.rand((B, N), generator=g, device=DEV),
          "us": torch.rand((B,), generator=g, device=DEV),
          "n_nodes": torch.tensor(_counts(c), dtype=torch.int32, device=DEV),
          "path": torch.empty((B, N), dtype=torch.int32, device=DEV),
          "n_acc": torch.empty((B,), dtype=torch.int32, device=DEV),
          "next": torch.empty((B,), dtype=torch.int32, device=DEV)}
    return st


def _paths(c):
    """Accepted paths: node 0, then nodes whose rows lie past the accepted rows' places (or already
    in place), so that moving the rows again gives the same cache."""
    r = random.Random(c["shape_seed"] + 3)
    out = []
    for _ in range(c["B"]):
        N = c["N"]
        a = r.randint(1, max(1, min(N, 2 + N // 6)))
        stay = r.randint(1, a)
        far = sorted(r.sample(range(a, N), min(a - stay, max(0, N - a)))) if N > a else []
        p = list(range(stay)) + far
        out.append(p + [-1] * (N - len(p)))
    return out


def _prepare_accept(c, g):
    B, N, Hkv = c["B"], c["N"], c["Hkv"]
    r = random.Random(c["shape_seed"] + 4)
    lens = [N + r.randint(0, 500) for _ in range(B)]
    table, P, _ = _tables(c, lens, 1, g)
    paths = _paths(c)
    k, v = _random_pages(g, P, Hkv), _random_pages(g, P, Hkv)
    if c["fp8"]:
        idx = torch.randint(0, 127, (P, FP8_PB), generator=g, device=DEV, dtype=torch.uint8)
    else:
        idx = _random_pages(g, P, 1)[:, 0]
    return {"case": c, "k": k, "v": v, "idx": idx, "table": table,
            "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "path": torch.tensor(paths, dtype=torch.int32, device=DEV),
            "n_acc": torch.tensor([sum(x >= 0 for x in p) for p in paths], dtype=torch.int32,
                                  device=DEV),
            "new_lens": torch.empty((B,), dtype=torch.int32, device=DEV)}


def _fork_lens(c):
    r = random.Random(c["shape_seed"] + 6)
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def _fork_rows(c):
    return [i * c["B"] // c["n"] if c["n"] >= c["B"] else i for i in range(c["n"])]


def _prepare_fork(c, g):
    B, n, Hkv = c["B"], c["n"], c["Hkv"]
    lens = _fork_lens(c)
    table, P, free = _tables(c, lens, n + 3, g)
    free = sorted(free)
    refs = torch.zeros((P,), dtype=torch.int32, device=DEV)
    refs[table[table >= 0].long()] = 1
    fl = torch.full((P,), -1, dtype=torch.int32)
    fl[:len(free)] = torch.tensor(free, dtype=torch.int32)
    return {"case": c, "k": _random_pages(g, P, Hkv), "v": _random_pages(g, P, Hkv),
            "idx": _random_pages(g, P, 1)[:, 0], "table": table,
            "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "rows": torch.tensor(_fork_rows(c), dtype=torch.int32, device=DEV),
            "refs": refs, "free_list": fl.to(DEV),
            "free_count": torch.tensor([len(free)], dtype=torch.int32, device=DEV),
            "child": torch.empty((n, table.shape[1]), dtype=torch.int32, device=DEV),
            "child_lens": torch.empty((n,), dtype=torch.int32, device=DEV)}


# ------------------------------------------------------------------ one pass

def run(st):
    kind = st["case"]["kind"]
    if own:
        return {"attn": _own_attn, "verify": _own_verify, "accept": _own_accept,
                "fork": _own_fork}[kind](st)
    return {"attn": _plain_attn, "verify": _plain_verify, "accept": _plain_accept,
            "fork": _plain_fork}[kind](st)


def _own_attn(st):
    import mxfp4_sparse_paged_gb300 as m
    c = st["case"]
    m.tree_paged_decode(st["q"], st["k"], st["v"], st["table"], st["seq_lens"], SCALE, st["out"],
                        st["ws"], tree_mask=st["masks"], n_nodes=st["n_nodes"],
                        window=c["window"], sinks=c["sinks"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_verify(st):
    import mxfp4_sparse_paged_gb300 as m
    m.verify_drafts(st["target"], st["draft"], st["tokens"], st["parents"], st["u"], st["us"],
                    st["path"], st["n_acc"], st["next"], n_nodes=st["n_nodes"])
    return {"path": st["path"], "n_accepted": st["n_acc"], "next": st["next"]}


def _own_accept(st):
    import mxfp4_sparse_paged_gb300 as m
    m.mx4_accept_rows(st["path"], st["n_acc"], st["seq_lens"], st["table"], st["k"], st["v"],
                      st["idx"], st["new_lens"])
    return {"k": st["k"], "v": st["v"], "idx": st["idx"], "lens": st["new_lens"]}


def _own_fork(st):
    import mxfp4_sparse_paged_gb300 as m
    m.mx4_fork_pages(st["rows"], st["table"], st["seq_lens"], st["refs"], st["free_list"],
                     st["free_count"], st["k"], st["v"], st["idx"], st["child"], st["child_lens"])
    m.mx4_free_pages(st["child"], st["child_lens"], st["refs"], st["free_list"], st["free_count"])
    return _fork_out(st)


def _fork_out(st):
    return {"child": st["child"], "child_lens": st["child_lens"], "refs": st["refs"],
            "free_list": st["free_list"], "free_count": st["free_count"], "k": st["k"],
            "v": st["v"], "idx": st["idx"]}


# ------------------------------------------------------------------ plain forms

def _decode_pages(pages, dtype):
    """Bytes [..., 8704] of pages -> the values they stand for [..., 128 tokens, 128 dims]."""
    lut = torch.tensor(GRID + [-x for x in GRID], dtype=dtype, device=pages.device)
    d = pages[..., :8192].unflatten(-1, (PT, 64))
    x = lut[torch.stack((d & 15, d >> 4), -1).flatten(-2).int()]
    sc = pages[..., 8192:].unflatten(-1, (PT, 4)).to(torch.int32)
    f = torch.ldexp(torch.ones((), dtype=dtype, device=pages.device), sc - 127)
    f = torch.where(sc == 255, torch.full_like(f, float("nan")), f)
    return (x.unflatten(-1, (4, 32)) * f.unsqueeze(-1)).flatten(-2)


def _popcount(x, n):
    return sum(((x >> i) & 1) for i in range(n))


def _plain_attn(st, dtype=torch.float32):
    c = st["case"]
    B, N, H, Hkv = c["B"], c["N"], c["H"], c["Hkv"]
    G = H // Hkv
    out = torch.zeros((B, N, H, HD), dtype=dtype, device=DEV)
    lse = torch.full((B, N, H), -math.inf, dtype=dtype, device=DEV)
    for s in range(B):
        L, n = st["lens"][s], st["counts"][s]
        sk, lo, base = _visible_span(c, L, n)
        lo = (lo // PT) * PT if lo > (sk + PT - 1) // PT * PT else 0
        pages = list(range(0, (sk + PT - 1) // PT if lo else 0)) + list(range(lo // PT, (L + PT - 1) // PT))
        at = torch.tensor(pages, device=DEV)
        ids = st["table"][s, at].long()
        tok = (at[:, None] * PT + torch.arange(PT, device=DEV)).flatten()
        tok_ok = tok < L
        kk = _decode_pages(st["k"][ids], dtype).transpose(0, 1).flatten(1, 2)[:, tok_ok]
        vv = _decode_pages(st["v"][ids], dtype).transpose(0, 1).flatten(1, 2)[:, tok_ok]
        tok = tok[tok_ok]
        if st["masks"] is None:
            mask = (2 << torch.arange(n, device=DEV)) - 1
        else:
            mask = st["masks"][s, :n]
        depth = (_popcount(mask, n) - 1).clamp_min(0)
        i = tok - base
        drafted = i >= 0
        ic = i.clamp(0, n - 1)
        see = ((mask[:, None] >> ic[None]) & 1).bool() | ~drafted[None]
        if c["window"]:
            near = torch.where(drafted, depth[ic], i)[None] > depth[:, None] - c["window"]
            first = torch.where(drafted, base + depth[ic], tok) < c["sinks"]
            see = see & (near | first[None])
        qs = st["q"][s, :n].to(dtype).view(n, Hkv, G, HD).permute(1, 0, 2, 3).reshape(Hkv, n * G, HD)
        x = (qs @ kk.transpose(1, 2)).view(Hkv, n, G, -1) * SCALE
        x = torch.where(see[None, :, None, :], x, torch.full((), -math.inf, dtype=dtype, device=DEV))
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
        z = e.sum(-1, keepdim=True)
        o = (e.view(Hkv, n * G, -1) @ vv).view(Hkv, n, G, HD)
        o = torch.where(z > 0, o / z, torch.zeros_like(o))
        out[s, :n] = o.permute(1, 0, 2, 3).reshape(n, H, HD)
        lse[s, :n] = (torch.log(z) + top)[..., 0].permute(1, 0, 2).reshape(n, H)
    return {"out": out.to(torch.bfloat16) if dtype == torch.float32 else out, "lse": lse}


def _plain_verify(st):
    c = st["case"]
    B, N, V = c["B"], c["N"], c["V"]
    r = torch.arange(B, device=DEV)
    f64 = torch.float64
    cur = torch.zeros(B, dtype=torch.int64, device=DEV)
    W = st["target"][:, 0].to(f64)
    T = torch.ones(B, dtype=f64, device=DEV)
    shut = torch.zeros(B, dtype=torch.bool, device=DEV)  # no further child of this node is tested
    path = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    acc = torch.ones(B, dtype=torch.int64, device=DEV)
    vocab = torch.arange(V, device=DEV)
    for j in range(1, N):
        test = (st["parents"][:, j] == cur) & ~shut & (j < st["n_nodes"])
        x = st["tokens"][:, j].long()
        if st["draft"] is None:
            q = (vocab[None] == x[:, None]).to(f64)
        else:
            q = st["draft"][r, cur].to(f64)
        ok = st["u"][:, j].to(f64) * T * q[r, x] < W[r, x]
        yes, no = test & ok, test & ~ok
        W1 = torch.clamp_min(W - T[:, None] * q, 0.0)
        T1 = W1.sum(-1)
        none = no & (T1 <= 0)
        shut = shut | none
        W = torch.where((no & ~none)[:, None], W1, W)
        W = torch.where(none[:, None], st["target"][r, cur].to(f64), W)
        T = torch.where(no & ~none, T1, T)
        cur = torch.where(yes, torch.full_like(cur, j), cur)
        W = torch.where(yes[:, None], st["target"][:, j].to(f64), W)
        T = torch.where(yes, torch.ones_like(T), T)
        at = torch.where(yes, acc, torch.zeros_like(acc))
        path[r, at] = torch.where(yes, torch.full_like(at, j), torch.zeros_like(at)).to(torch.int32)
        acc = acc + yes
    cum = W.cumsum(-1)
    nxt = (cum <= (st["us"].to(f64) * cum[:, -1])[:, None]).sum(-1).clamp_max(V - 1)
    return {"path": path, "n_accepted": acc.to(torch.int32), "next": nxt.to(torch.int32)}


def _row_views(pages):
    """The row parts of a pool: MXFP4 [P, (heads,) 128, 64] and [..., 128, 4], or fp8 [P, 128, 128]."""
    if pages.shape[-1] == FP8_PB:
        return [pages.unflatten(-1, (PT, 128))]
    return [pages[..., :8192].unflatten(-1, (PT, 64)), pages[..., 8192:].unflatten(-1, (PT, 4))]


def _plain_accept(st):
    path, N = st["path"].long(), st["case"]["N"]
    i = torch.arange(N, device=DEV)[None]
    live = (i < st["n_acc"][:, None]) & (path > i)
    base = (st["seq_lens"].long() - N)[:, None]
    src = base + torch.where(live, path, torch.zeros_like(path))
    dst = base + torch.where(live, i.expand_as(path), torch.zeros_like(path))
    sp, dp = st["table"].gather(1, src // PT).long(), st["table"].gather(1, dst // PT).long()
    for pool in (st["k"], st["v"], st["idx"]):
        for x in _row_views(pool):
            if x.dim() == 4:
                x = x.transpose(1, 2)  # [P, 128, heads, bytes]
            x[dp, dst % PT] = x[sp, src % PT]
    st["new_lens"].copy_(st["seq_lens"] - N + st["n_acc"])
    return {"k": st["k"], "v": st["v"], "idx": st["idx"], "lens": st["new_lens"]}


def _plain_fork(st):
    rows = st["rows"].long()
    Wd = st["table"].shape[1]
    lens = st["seq_lens"][rows].long()
    P = st["refs"].shape[0]
    part = lens % PT != 0
    last = lens // PT
    rank = part.long().cumsum(0) - 1
    new = st["free_list"][(st["free_count"].long() - 1 - rank).clamp_min(0)].long()
    slot = torch.arange(Wd, device=DEV)[None]
    full = slot < last[:, None]
    src = st["table"][rows].long()
    child = torch.where(full, src, torch.full_like(src, -1))
    child = torch.where((slot == last[:, None]) & part[:, None], new[:, None], child)
    st["child"].copy_(child)
    st["child_lens"].copy_(lens)
    refs = torch.zeros(P + 1, dtype=torch.int32, device=DEV)
    refs[:P] = st["refs"]
    one = torch.ones((), dtype=torch.int32, device=DEV)
    refs.index_put_((torch.where(child >= 0, child, torch.full_like(child, P)),), one, accumulate=True)
    st["free_count"].sub_(part.sum().to(torch.int32))
    # the used rows of a partly filled last page; the others (and children without one) stay
    at = torch.where(part, last, torch.zeros_like(last))
    sp = src.gather(1, at[:, None])[:, 0]
    dp = torch.where(part, new, sp)
    keep = (torch.arange(PT, device=DEV)[None] >= (lens % PT)[:, None])
    for pool in (st["k"], st["v"], st["idx"]):
        for x in _row_views(pool):
            k = keep[:, None, :, None] if x.dim() == 4 else keep[:, :, None]
            x[dp] = torch.where(k, x[dp], x[sp])
    # the children end
    before = refs[:P] > 0
    refs.index_put_((torch.where(child >= 0, child, torch.full_like(child, P)),), -one, accumulate=True)
    gone = before & (refs[:P] == 0)
    to = torch.where(gone, st["free_count"].long() + gone.long().cumsum(0) - 1,
                     torch.full((P,), P, device=DEV))
    fl = torch.empty(P + 1, dtype=torch.int32, device=DEV)
    fl[:P] = st["free_list"]
    fl[to] = torch.arange(P, dtype=torch.int32, device=DEV)
    st["free_list"].copy_(fl[:P])
    st["free_count"].add_(gone.sum().to(torch.int32))
    st["refs"].copy_(refs[:P])
    return _fork_out(st)


# ------------------------------------------------------------------ floors

def work(c):
    if c["kind"] == "attn":
        B, N, H, Hkv = c["B"], c["N"], c["H"], c["Hkv"]
        by, fl = 0, 0
        for L, n in zip(_lens(c, N), _counts(c)):
            sk, lo, base = _visible_span(c, L, n)
            tok = sk + (L - lo)
            by += tok * Hkv * 2 * 68
            pairs = n * (sk + min(base, c["window"]) if c["window"] else base) + n * (n + 1) // 2
            fl += 4 * HD * H * pairs
        by += B * N * H * (HD * 4 + 4)
        return {"bytes": by, "flops": fl}
    if c["kind"] == "verify":
        # a sequence that ends by a rejection needs both rows of that node, else the target's
        rows = 1 if c["given"] or c["N"] == 1 else 2
        return {"bytes": c["B"] * (rows * c["V"] * 4 + c["N"] * 16), "flops": 4 * c["B"] * c["V"]}
    if c["kind"] == "accept":
        row = 2 * c["Hkv"] * 68 + (128 if c["fp8"] else 68)
        moved = sum(sum(1 for i, p in enumerate(x) if p > i) for x in _paths(c))
        return {"bytes": moved * row * 2 + c["B"] * (c["N"] * 4 + 16), "flops": 0}
    lens = _fork_lens(c)
    rowb = (2 * c["Hkv"] + 1) * 68
    by = sum((lens[s] % PT) * rowb * 2 + (lens[s] // PT + 1) * 4 * 6 for s in _fork_rows(c))
    return {"bytes": by, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    if c["kind"] == "attn":
        return _exact_attn(c, seed)
    return None  # moved bytes, page ids and token ids: equal or wrong


def _exact_attn(c, seed):
    """Straight from the definition, in float64: one KV head of one sequence at a time, each cached
    row written out with its position, no page ranges left out."""
    B, N, H, Hkv = c["B"], c["N"], c["H"], c["Hkv"]
    G = H // Hkv
    if sum(_lens(c, N)) * N * H > 3e10:
        return None
    st = prepare(c, seed)
    out = torch.zeros((B, N, H, HD), dtype=torch.float64, device=DEV)
    lse = torch.full((B, N, H), -math.inf, dtype=torch.float64, device=DEV)
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64, device=DEV)
    mag = torch.tensor(GRID, dtype=torch.float64, device=DEV)
    trees = _trees(c)

    def values(pages, ids, h, L):
        p = pages[ids, h]
        b = p[:, :8192].reshape(-1, 64)[:L].long()
        s = p[:, 8192:].reshape(-1, 4)[:L].double()
        x = torch.empty((L, HD), dtype=torch.float64, device=DEV)
        x[:, 0::2] = mag[b % 8] * sign[(b // 8) % 2]
        x[:, 1::2] = mag[(b // 16) % 8] * sign[b // 128]
        return x * torch.pow(2.0, s - 127.0).repeat_interleave(32, dim=1)

    for s in range(B):
        L, n = st["lens"][s], st["counts"][s]
        base = L - n
        see = np.zeros((n, L), dtype=bool)
        depth = [0] * n
        for j in range(n):
            p = trees[s][j]
            depth[j] = 0 if p < 0 else depth[p] + 1
        for j in range(n):
            pos = base + depth[j]
            first = 0 if c["window"] == 0 else max(0, pos - c["window"] + 1)
            see[j, min(first, base):base] = True
            see[j, :min(base, c["sinks"] if c["window"] else 0)] = True
            a = j
            while a >= 0:
                at = base + depth[a]
                see[j, base + a] = c["window"] == 0 or at >= first or at < c["sinks"]
                a = trees[s][a]
        see = torch.from_numpy(see).to(DEV)
        ids = st["table"][s, :(L + PT - 1) // PT].long()
        for h in range(Hkv):
            k, v = values(st["k"], ids, h, L), values(st["v"], ids, h, L)
            for gq in range(G):
                x = st["q"][s, :n, h * G + gq].double() @ k.T * SCALE
                x = x.masked_fill(~see, -math.inf)
                z = torch.logsumexp(x, -1)
                some = see.any(-1)
                w = torch.exp(x - torch.where(some, z, torch.zeros_like(z))[:, None])
                out[s, :n, h * G + gq] = w @ v
                lse[s, :n, h * G + gq] = z
    return {"out": out, "lse": lse}
