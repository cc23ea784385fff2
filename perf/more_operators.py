"""The operators of a decode step over an 8-bit paged K/V cache: cases, inputs and plain forms.

New tokens' keys are turned by their positions and appended with their values to pages of E4M3
bytes, one power-of-two scale for each 32-token block and head (fp8_rope_append); the index keys
give every 128-token block a cheap score for each query (index_block_score, index_block_score_fp8);
the best blocks are chosen (block_topk); attention reads all pages (fp8_paged_decode) or the chosen
blocks (fp8_block_decode).

`own` chooses between the plain forms below and the package's calls.  K/V pages: uint8
[pages, heads, 16384], 128 token rows of 128 E4M3 bytes; scales uint8 [pages, heads, 4], e8m0.
Index pages: MXFP4 [pages, 8704] (128 rows of 64 bytes, two e2m1 codes each, low nibble first,
then 128 rows of 4 e8m0 scale bytes) or fp8 [pages, 16384].
"""
import math
import random

import torch

own = False

DEV = "cuda"
PT, HD, MX_PB, FP8_PB = 128, 128, 8704, 16384
SUB = 32                    # tokens that share a scale
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
SCALE = 1.0 / math.sqrt(HD)
F32, F64, BF16, E4M3, E8M0 = (torch.float32, torch.float64, torch.bfloat16, torch.float8_e4m3fn,
                              torch.float8_e8m0fnu)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's next token: the smallest write, latency
        _append("append_one_token", B=1, new=("fixed", 1, 1), ctx=("fixed", 776, 776), H=16, Hkv=1),
        # the next tokens of a decode batch, half of each head turned in neighbouring pairs
        _append("append_decode_batch", B=256, new=("fixed", 1, 1), ctx=("lognormal", 8192, 131071),
                H=64, Hkv=8, rot=64, inter=True),
        # prompts of odd lengths behind cached ones, fp32 projections, positions past a million in
        # a context that was stretched by 8, rows of padding behind the last sequence
        _append("append_prompts_ragged", B=5, new=("uniform", 600, 4096), ctx=("uniform", 0, 5000),
                H=40, Hkv=8, fp32=True, stretch=8.0, shift=1000003, pad=37),
        # block scores of the repository's serving batch: 256 ragged contexts, MXFP4 index keys
        _score("block_score_batch", B=256, q=1, lens=("lognormal", 8192, 131072)),
        # four tokens each of sixteen long contexts, fp8 index keys
        _score("block_score_long_fp8", B=16, q=4, lens=("fixed", 131072, 131072), fp8=True),
        # 16 blocks for each token of that batch
        _topk("block_topk_batch", B=256, q=1, lens=("lognormal", 8192, 131072), k=16, first=1, last=2),
        # eight contexts of up to eight million tokens, many blocks
        _topk("block_topk_longest", B=8, q=1, lens=("uniform", 4000000, 8388608), k=500, first=1,
              last=3),
        # one user's single token over a short context: the smallest read, latency
        _attn("decode_one_short", B=1, q=1, H=16, Hkv=1, lens=("fixed", 777, 777)),
        # the decode batch: 256 ragged contexts, the largest
        _attn("decode_batch_ragged", B=256, q=1, H=16, Hkv=1, lens=("lognormal", 8192, 131072)),
        # four tokens a sequence, grouped heads of odd width, some scales far apart
        _attn("decode_gqa_four", B=64, q=4, H=40, Hkv=8, lens=("uniform", 2048, 8192)),
        # one user's single token reads 16 of 1024 blocks
        _attn("blocks_one_long", B=1, q=1, H=16, Hkv=1, lens=("fixed", 131072, 131072), k=16),
        # a batch reads 16 blocks for each token, four KV heads
        _attn("blocks_batch_gqa", B=256, q=1, H=32, Hkv=4, lens=("lognormal", 8192, 65536), k=16),
    ]


def draw(rng):
    kind = rng.choice(["append", "append", "score", "topk", "attn", "attn", "blocks", "blocks"])
    Hkv = rng.choice([1, 1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16]) if Hkv > 1 else rng.choice([1, 4, 7, 16, 16, 16])
    if kind == "append":
        B = _log(rng, 1, 256)
        n = _log(rng, 1, max(1, min(4096, 12000 // B)))
        c = _append(None, B=B, new=("uniform", rng.randint(0 if B > 1 else 1, n), n),
                    ctx=("uniform", 0, _log(rng, 1, 8192)), H=G * Hkv, Hkv=Hkv,
                    rot=rng.choice([0, 16, 64, 96, 128, 128, 128]), inter=rng.random() < 0.5,
                    fp32=rng.random() < 0.4, stretch=rng.choice([1.0, 1.0, 8.0]),
                    shift=rng.choice([0, 0, 50000, 1000003]), pad=rng.choice([0, 0, 5]))
    elif kind == "score":
        B, q, fp8 = _log(rng, 1, 256), rng.randint(1, 8), rng.random() < 0.5
        hi = min(131072, max(q, 2500000 // B))
        c = _score(None, B=B, q=q, lens=("uniform", max(q, min(hi, _log(rng, 1, hi))), hi), fp8=fp8)
    elif kind == "topk":
        B, q = _log(rng, 1, 256), rng.randint(1, 8)
        hi = min(8388608, _log(rng, 1000, 60000000 // B))
        first, last = rng.choice([0, 1, 4]), rng.choice([0, 1, 3])
        c = _topk(None, B=B, q=q, lens=("uniform", q, hi), k=max(first + last, _log(rng, 1, 512)),
                  first=first, last=last)
    else:
        q = rng.choice([1, 1, 1, 2, 3, 4, 8])
        B = _log(rng, 1, 256)
        k = _log(rng, 1, 64) if kind == "blocks" else 0
        if k:  # at most 12000 blocks of one head are read
            B = max(1, min(B, 12000 // (k * Hkv * q)))
            hi = _log(rng, 1, min(65536, 1500000 // B // Hkv))
        else:  # at most 8000 pages of one head
            hi = _log(rng, 1, max(1, min(65536, 1000000 // (B * Hkv))))
        c = _attn(None, B=B, q=q, H=G * Hkv, Hkv=Hkv, lens=("uniform", rng.randint(0, hi), hi), k=k)
    c["shape_seed"] = rng.randrange(1 << 30)
    del c["name"]
    return c


def _log(rng, lo, hi):
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _spread(key, how):
    """A distribution of lengths: its kind, its least (lognormal: its median) and its largest."""
    return {key: how[0], key + "_lo": how[1], key + "_hi": how[2]}


def _append(name, B, new, ctx, H, Hkv, rot=128, inter=False, fp32=False, stretch=1.0, shift=0, pad=0):
    return {"name": name, "kind": "append", "B": B, **_spread("new", new), **_spread("ctx", ctx),
            "H": H, "Hkv": Hkv, "rot": rot, "inter": inter, "fp32": fp32, "stretch": stretch,
            "shift": shift, "pad": pad, "shape_seed": 1}


def _score(name, B, q, lens, fp8=False):
    return {"name": name, "kind": "score", "B": B, "q": q, **_spread("lens", lens), "fp8": fp8,
            "shape_seed": 2}


def _topk(name, B, q, lens, k, first, last):
    return {"name": name, "kind": "topk", "B": B, "q": q, **_spread("lens", lens), "k": k,
            "first": first, "last": last, "shape_seed": 3}


def _attn(name, B, q, H, Hkv, lens, k=0):
    """k > 0: over k listed blocks a token; 0: over the whole cache."""
    return {"name": name, "kind": "attn", "B": B, "q": q, "H": H, "Hkv": Hkv,
            **_spread("lens", lens), "k": k, "shape_seed": 4}


# ------------------------------------------------------------------ shapes (from the case alone)

def _sizes(c, key, salt):
    r = random.Random(c["shape_seed"] + salt)
    how, lo, hi = c[key], c[key + "_lo"], c[key + "_hi"]
    if how == "fixed":
        return [lo] * c["B"]
    if how == "lognormal":
        return [max(1, min(hi, int(lo * math.exp(r.gauss(0.0, 1.0))))) for _ in range(c["B"])]
    return [r.randint(lo, hi) for _ in range(c["B"])]


def _lens(c):
    return _sizes(c, "lens", 0)


def _append_lens(c):
    """(new tokens, cached tokens after the append) of each sequence."""
    new = _sizes(c, "new", 11)
    new[0] = max(1, new[0])
    return new, [n + o for n, o in zip(new, _sizes(c, "ctx", 12))]


def _lists(c):
    """Block lists of the tokens: the block of the token itself, its neighbours and others spread
    over the context, ascending, -1 padded."""
    r = random.Random(c["shape_seed"] + 13)
    out = []
    for L in _lens(c):
        for j in range(c["q"]):
            p = L - c["q"] + j
            n = p // PT + 1 if p >= 0 else 0
            near = [b for b in (n - 1, n - 2) if b >= 0][:c["k"]]
            rest = r.sample(range(max(0, n - 2)), min(c["k"] - len(near), max(0, n - 2)))
            x = sorted(near + rest)
            out.append(x + [-1] * (c["k"] - len(x)))
    return out


def _inv_freq(c):
    """fp32 [rot / 2] radians a position, base 10000, positions stretched by c["stretch"]."""
    f = [10000.0 ** (-2.0 * i / c["rot"]) / c["stretch"] for i in range(c["rot"] // 2)]
    return torch.tensor(f, dtype=F64).to(F32)


def _factor(c):
    """What turned dims are multiplied by: 1, and a little more in a stretched context."""
    return 1.0 if c["stretch"] == 1.0 else 0.1 * math.log(c["stretch"]) + 1.0


# ------------------------------------------------------------------ inputs

def _tables(c, lens, spare=2):
    """Page ids a random permutation of the pool; int32 block table, -1 past a sequence's pages."""
    n = [(L + PT - 1) // PT for L in lens]
    P = sum(n) + spare
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(c["shape_seed"] + 5))
    table = torch.full((len(lens), max(1, max(n))), -1, dtype=torch.int32)
    o = 0
    for s, k in enumerate(n):
        table[s, :k] = perm[o:o + k].to(torch.int32)
        o += k
    return table.to(DEV), P


def _page_list(lens):
    """Of every page in use: its sequence, and its number in the sequence (int64, on the device)."""
    n = torch.tensor([(L + PT - 1) // PT for L in lens])
    seq = torch.repeat_interleave(torch.arange(len(lens)), n)
    page = torch.arange(int(n.sum())) - (n.cumsum(0) - n)[seq]
    return seq.to(DEV), page.to(DEV)


def _fp8_pool(g, P, heads):
    """E4M3 rows of a normal distribution, largest values near the format's end."""
    pages = torch.empty((P, heads, FP8_PB), dtype=torch.uint8, device=DEV)
    step = max(1, 8192 // heads)
    for a in range(0, P, step):
        b = min(P, a + step)
        x = torch.randn((b - a, heads, FP8_PB), generator=g, device=DEV).mul_(110.0).clamp_(-448, 448)
        pages[a:b] = x.to(E4M3).view(torch.uint8)
    return pages


def _mx_pool(g, P):
    """MXFP4 rows of a normal distribution."""
    pages = torch.empty((P, MX_PB), dtype=torch.uint8, device=DEV)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for a in range(0, P, 4096):
        b = min(P, a + 4096)
        x = torch.randn((b - a, PT, 4, 32), generator=g, device=DEV)
        e = torch.frexp(x.abs().amax(-1)).exponent - 3
        y = torch.ldexp(x, -e.unsqueeze(-1))
        code = torch.bucketize(y.abs(), mids).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
        code = code.view(b - a, PT, 64, 2)
        pages[a:b, :PT * 64] = (code[..., 0] | (code[..., 1] << 4)).reshape(b - a, -1)
        pages[a:b, PT * 64:] = (e + 127).to(torch.uint8).reshape(b - a, -1)
    return pages


def _poison_tails(pages, table, lens, row_bytes, at=0):
    """Rows past a sequence's length hold what an empty cache holds: 0xFF."""
    t = [[s, L // PT, L % PT] for s, L in enumerate(lens) if L % PT]
    if not t:
        return
    t = torch.tensor(t, device=DEV)
    pid = table[t[:, 0], t[:, 1]].long()
    dead = torch.arange(PT, device=DEV)[None] >= t[:, 2][:, None]
    v = pages[pid]
    rows = v[..., at:at + PT * row_bytes].view(*v.shape[:-1], PT, row_bytes)
    if rows.dim() == 4:
        dead = dead[:, None].expand(-1, rows.shape[1], -1)
    rows[dead] = 255
    pages[pid] = v


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return {"append": _prepare_append, "score": _prepare_score, "topk": _prepare_topk,
            "attn": _prepare_attn}[c["kind"]](c, g)


def _prepare_append(c, g):
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    new, lens = _append_lens(c)
    table, P = _tables(c, lens)
    T = sum(new)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    cu = torch.tensor([0] + new).cumsum(0)
    pos = torch.tensor(lens)[seq] - torch.tensor(new)[seq] + torch.arange(T) - cu[seq]
    # the projections' output: q, k and v side by side, some values far out as in trained models
    x = torch.randn((T + c["pad"], (H + 2 * Hkv) * HD), generator=g, device=DEV)
    x.mul_(torch.exp(torch.randn((T + c["pad"], 1), generator=g, device=DEV)))
    x = x if c["fp32"] else x.to(BF16)
    q, k, v = (t.unflatten(-1, (-1, HD)) for t in x.split([H * HD, Hkv * HD, Hkv * HD], -1))
    inv = _inv_freq(c) if c["rot"] else None
    shifted = torch.zeros(T + c["pad"], dtype=torch.int64)
    shifted[:T] = pos + c["shift"]
    scales = torch.randint(117, 122, (2, P, Hkv, 4), generator=g, device=DEV, dtype=torch.uint8)
    # the first new token of each 32-token block: where a scale may grow
    first = (pos % SUB == 0) | (torch.arange(T) == cu[seq])
    st = {"case": c, "q": q, "k": k, "v": v, "table": table, "T": T,
          "cu": cu.to(torch.int32).to(DEV),
          "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
          "positions": shifted.to(DEV) if c["shift"] else None,
          "seq": seq.to(DEV), "pos": pos.to(DEV), "lead": first.nonzero()[:, 0].to(DEV),
          "inv": None if inv is None else inv.to(DEV),
          "kp": _fp8_pool(g, P, Hkv), "vp": _fp8_pool(g, P, Hkv), "ks": scales[0], "vs": scales[1],
          "q_out": torch.zeros((T + c["pad"], H, HD), dtype=BF16, device=DEV)}
    if own:
        import mxfp4_sparse_paged_gb300 as m
        st["phases"] = None if inv is None else m.rope_phases(st["inv"])
    return st


def _prepare_score(c, g):
    B, q = c["B"], c["q"]
    lens = [max(q, L) for L in _lens(c)]
    table, P = _tables(c, lens)
    if c["fp8"]:
        pages = _fp8_pool(g, P, 1)[:, 0]
        _poison_tails(pages, table, lens, 128)
    else:
        pages = _mx_pool(g, P)
        _poison_tails(pages, table, lens, 64)
        _poison_tails(pages, table, lens, 4, PT * 64)
    seq, page = _page_list(lens)
    return {"case": c, "pages": pages, "table": table,
            "iq": torch.randn((B * q, HD), generator=g, device=DEV).to(BF16),
            "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "seq": seq, "page": page,
            "scores": torch.zeros((B * q, table.shape[1]), dtype=F32, device=DEV)}


def _prepare_topk(c, g):
    B, q = c["B"], c["q"]
    lens = [max(q, L) for L in _lens(c)]
    W = (max(lens) + PT - 1) // PT
    # maxima of many scores: some blocks stand out, some tie (a shared prefix scores the same)
    x = torch.randn((B * q, W), generator=g, device=DEV).mul_(3.0).add_(8.0)
    x = torch.where(torch.rand((B * q, W), generator=g, device=DEV) < 0.2, x.round(), x)
    return {"case": c, "scores": x, "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "idx": torch.empty((B * q, c["k"]), dtype=torch.int32, device=DEV)}


def _prepare_attn(c, g):
    B, q, H, Hkv = c["B"], c["q"], c["H"], c["Hkv"]
    lens = _lens(c)
    table, P = _tables(c, lens)
    kp, vp = _fp8_pool(g, P, Hkv), _fp8_pool(g, P, Hkv)
    _poison_tails(kp, table, lens, HD)
    _poison_tails(vp, table, lens, HD)
    ks = torch.randint(119, 122, (P, Hkv, 4), generator=g, device=DEV, dtype=torch.uint8)
    vs = torch.randint(116, 123, (P, Hkv, 4), generator=g, device=DEV, dtype=torch.uint8)
    st = {"case": c, "kp": kp, "vp": vp, "ks": ks, "vs": vs, "table": table,
          # logits of standard deviation 2: some tokens stand out, as in a trained model
          "q": (2.0 * torch.randn((B * q, H, HD), generator=g, device=DEV)).to(BF16),
          "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
          "out": torch.empty((B * q, H, HD), dtype=BF16, device=DEV),
          "lse": torch.empty((B * q, H), dtype=F32, device=DEV)}
    if c["k"]:
        st["idx"] = torch.tensor(_lists(c), dtype=torch.int32, device=DEV)
    else:
        st["seq"], st["page"] = _page_list(lens)
    if own:
        import mxfp4_sparse_paged_gb300 as m
        n = (m.fp8_block_decode_workspace(B * q, c["k"], H, Hkv) if c["k"] else
             m.fp8_paged_decode_workspace(B * q, q, H, Hkv))
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    kind = st["case"]["kind"]
    if own:
        return {"append": _own_append, "score": _own_score, "topk": _own_topk,
                "attn": _own_attn}[kind](st)
    return {"append": _plain_append, "score": _plain_score, "topk": _plain_topk,
            "attn": _plain_attn}[kind](st)


def _own_append(st):
    import mxfp4_sparse_paged_gb300 as m
    c = st["case"]
    m.fp8_rope_append(st["q"], st["k"], st["v"], st["cu"], st["table"], st["seq_lens"], st["kp"],
                      st["vp"], st["ks"], st["vs"], st["q_out"], phases=st["phases"],
                      positions=st["positions"], interleaved=c["inter"], factor=_factor(c))
    return _append_out(st)


def _append_out(st):
    return {"q": st["q_out"], "k": st["kp"].view(E4M3), "v": st["vp"].view(E4M3),
            "k_scales": st["ks"].view(E8M0), "v_scales": st["vs"].view(E8M0)}


def _own_score(st):
    import mxfp4_sparse_paged_gb300 as m
    c = st["case"]
    if c["fp8"]:
        m.index_block_score_fp8(st["iq"], c["q"], st["pages"], st["table"], st["seq_lens"], 0.01,
                                st["scores"])
    else:
        m.index_block_score(st["iq"], c["q"], st["pages"], st["table"], st["seq_lens"],
                            st["scores"])
    return st["scores"]


def _own_topk(st):
    import mxfp4_sparse_paged_gb300 as m
    c = st["case"]
    m.block_topk(st["scores"], st["seq_lens"], c["q"], st["idx"], first=c["first"], last=c["last"])
    return st["idx"]


def _own_attn(st):
    import mxfp4_sparse_paged_gb300 as m
    c = st["case"]
    if c["k"]:
        m.fp8_block_decode(st["q"], c["q"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"],
                           st["seq_lens"], st["idx"], SCALE, st["out"], st["ws"], lse=st["lse"])
    else:
        m.fp8_paged_decode(st["q"], c["q"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"],
                           st["seq_lens"], SCALE, st["out"], st["ws"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------ plain forms

def _turned(x, pos, inv, rot, inter, factor):
    """Rows [T, heads, 128] turned by their positions, in 64 bits (angles of far positions)."""
    x = x.to(F64)
    if not rot:
        return x
    a = pos.to(F64)[:, None, None] * inv.to(F64)
    c, s = torch.cos(a) * factor, torch.sin(a) * factor
    h = rot // 2
    u, w = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :h], x[..., h:rot])
    lo, hi = u * c - w * s, w * c + u * s
    y = torch.stack((lo, hi), -1).flatten(-2) if inter else torch.cat((lo, hi), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _scale_exponent(amax):
    """The smallest E >= -127 with amax <= 448 * 2^E."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp_min(-127)


def _plain_store(st, rows, pages, scales):
    """New rows fp32 [T, heads, 128] into pages and scales, block by block."""
    T, (P, Hkv) = st["T"], pages.shape[:2]
    pid = st["table"][st["seq"], st["pos"] // PT].long()
    sub = st["pos"] % PT // SUB
    blk = (pid * 4 + sub)[:, None].expand(-1, Hkv)
    amax = torch.zeros((P * 4, Hkv), dtype=F32, device=DEV)
    amax.scatter_reduce_(0, blk, rows.abs().amax(-1), "amax")
    lead = st["lead"]
    lp, ls, at = pid[lead], sub[lead], st["pos"][lead] % SUB  # rows before `at` are there already
    old = scales.view(P, Hkv, 4)[lp, :, ls].to(torch.int32) - 127
    e = torch.maximum(_scale_exponent(amax[lp * 4 + ls]),
                      torch.where(at[:, None] > 0, old, torch.full_like(old, -127)))
    # [P, heads, 4, 32, 128]: the blocks' stored rows at the new scale
    view = pages.view(P, Hkv, 4, SUB, HD)
    x = view[lp, :, ls]
    y = torch.ldexp(x.view(E4M3).to(F32), (old - e)[..., None, None]).to(E4M3).view(torch.uint8)
    keep = (torch.arange(SUB, device=DEV)[None] < at[:, None])[:, None, :, None]
    grown = keep & (e > old)[..., None, None]
    view[lp, :, ls] = torch.where(grown, y, x)
    scales.view(P, Hkv, 4)[lp, :, ls] = (e + 127).to(torch.uint8)
    te = scales.view(P, Hkv, 4)[pid, :, sub].to(torch.int32) - 127
    code = torch.ldexp(rows, -te[..., None]).to(E4M3).view(torch.uint8)
    pages.view(P, Hkv, PT, HD)[pid, :, st["pos"] % PT] = code


def _plain_append(st):
    c, T = st["case"], st["T"]
    pos = st["pos"] if st["positions"] is None else st["positions"][:T]
    turn = (pos, st["inv"], c["rot"], c["inter"], _factor(c))
    st["q_out"][:T] = _turned(st["q"][:T], *turn).to(BF16)
    _plain_store(st, _turned(st["k"][:T], *turn).to(F32), st["kp"], st["ks"])
    _plain_store(st, st["v"][:T].to(F32), st["vp"], st["vs"])
    return _append_out(st)


def _mx_values(pages):
    """Bytes [..., 8704] of MXFP4 pages -> fp32 [..., 128 tokens, 128 dims]."""
    lut = torch.tensor(GRID + [-x for x in GRID], dtype=F32, device=pages.device)
    d = pages[..., :PT * 64].unflatten(-1, (PT, 64))
    x = lut[torch.stack((d & 15, d >> 4), -1).flatten(-2).int()]
    sc = pages[..., PT * 64:].unflatten(-1, (PT, 4)).to(torch.int32)
    f = torch.ldexp(torch.ones((), dtype=F32, device=pages.device), sc - 127)
    f = torch.where(sc == 255, torch.full_like(f, float("nan")), f)
    return (x.unflatten(-1, (4, 32)) * f.unsqueeze(-1)).flatten(-2)


def _plain_score(st):
    c, q = st["case"], st["case"]["q"]
    seq, page = st["seq"], st["page"]
    pages = st["pages"][st["table"][seq, page].long()]
    if c["fp8"]:
        x = pages.view(E4M3).to(F32).unflatten(-1, (PT, HD)) * 0.01
    else:
        x = _mx_values(pages)
    y = st["iq"].to(F32).view(-1, q, HD)[seq] @ x.transpose(1, 2)  # [pages, q, tokens]
    tok = page[:, None] * PT + torch.arange(PT, device=DEV)
    last = st["seq_lens"][seq].long()[:, None] - q + torch.arange(q, device=DEV)
    y = torch.where(tok[:, None] <= last[..., None], y, torch.full((), -math.inf, device=DEV))
    st["scores"].view(-1, q, st["scores"].shape[1])[seq, :, page] = y.amax(-1)
    return st["scores"]


def _plain_topk(st):
    c = st["case"]
    q, k = c["q"], c["k"]
    x = st["scores"]
    W = x.shape[1]
    last = st["seq_lens"].long()[:, None] - q + torch.arange(q, device=DEV)
    n = (last // PT + 1).view(-1, 1)
    b = torch.arange(W, device=DEV)
    always = (b < c["first"]) | (b >= n - c["last"])
    x = torch.where(always, torch.full((), math.inf, device=DEV), x)
    x = torch.where(b < n, x, torch.full((), -math.inf, device=DEV))
    at = x.sort(dim=-1, descending=True, stable=True).indices[:, :k]  # ties: the lower index first
    at = torch.where(torch.arange(at.shape[1], device=DEV) < n, at, torch.full_like(at, W))
    at = at.sort(-1).values
    st["idx"].fill_(-1)
    st["idx"][:, :at.shape[1]] = torch.where(at < W, at, torch.full_like(at, -1)).to(torch.int32)
    return st["idx"]


def _fp8_values(pages, scales):
    """E4M3 pages [n, heads, 16384] and scales [n, heads, 4] -> fp32 [n, heads, 128, 128]."""
    x = pages.view(E4M3).to(F32).unflatten(-1, (4, SUB * HD))
    return torch.ldexp(x, (scales.to(torch.int32) - 127).unsqueeze(-1)).unflatten(-1, (SUB, HD)).flatten(2, 3)


def _plain_attn(st):
    c = st["case"]
    B, q, H, Hkv, k = c["B"], c["q"], c["H"], c["Hkv"], c["k"]
    G = H // Hkv
    ninf = torch.full((), -math.inf, device=DEV)
    j = torch.arange(q, device=DEV)
    pos = st["seq_lens"].long()[:, None] - q + j  # [B, q]
    if k:  # a segment is a token, its rows the heads of a group
        N, R = B * q, G
        seg = torch.arange(N, device=DEV).repeat_interleave(k)
        page = st["idx"].flatten().long()
        pid = st["table"][seg // q, page.clamp_min(0)].long().clamp_min(0)
        limit = torch.where(page >= 0, pos.flatten()[seg], torch.full_like(page, -1))[:, None]
        page = page.clamp_min(0)
        rows = st["q"].view(N, Hkv, R, HD)
    else:  # a segment is a sequence, its rows the heads of a group for each of its tokens
        N, R = B, q * G
        seg, page = st["seq"], st["page"]
        pid = st["table"][seg, page].long()
        limit = pos[seg].repeat_interleave(G, 1)
        rows = st["q"].view(B, q, Hkv, G, HD).transpose(1, 2).reshape(B, Hkv, R, HD)
    tok = page[:, None] * PT + torch.arange(PT, device=DEV)
    see = tok[:, None] <= limit[..., None]  # [pages, rows, tokens]
    x = rows[seg].to(F32) @ _fp8_values(st["kp"][pid], st["ks"][pid]).transpose(2, 3) * SCALE
    x = torch.where(see[:, None], x, ninf)
    top = torch.full((N, Hkv, R), -math.inf, device=DEV)
    top.scatter_reduce_(0, seg[:, None, None].expand(-1, Hkv, R), x.amax(-1), "amax")
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(x - base[seg].unsqueeze(-1))
    z = torch.zeros((N, Hkv, R), device=DEV).index_add_(0, seg, e.sum(-1))
    v = _fp8_values(st["vp"][pid], st["vs"][pid])
    v = torch.where(see.any(1)[:, None, :, None], v, torch.zeros((), device=DEV))
    o = torch.zeros((N, Hkv, R, HD), device=DEV).index_add_(0, seg, e @ v)
    o = torch.where(z.unsqueeze(-1) > 0, o / z.unsqueeze(-1), torch.zeros_like(o))
    lse = torch.log(z) + base
    if not k:
        o = o.view(B, Hkv, q, G, HD).transpose(1, 2)
        lse = lse.view(B, Hkv, q, G).transpose(1, 2)
    return {"out": o.reshape(B * q, H, HD).to(BF16), "lse": lse.reshape(B * q, H)}


# ------------------------------------------------------------------ floors

def _npages(lens):
    return sum((L + PT - 1) // PT for L in lens)


def work(c):
    if c["kind"] == "append":
        new, _ = _append_lens(c)
        e = 4 if c["fp32"] else 2
        T, H, Hkv = sum(new), c["H"], c["Hkv"]
        return {"bytes": T * HD * ((H + 2 * Hkv) * e + H * 2 + 2 * Hkv), "flops": 6 * T * HD * (H + Hkv)}
    if c["kind"] == "score":
        lens = [max(c["q"], L) for L in _lens(c)]
        return {"bytes": sum(lens) * (128 if c["fp8"] else 68) + c["q"] * 4 * _npages(lens),
                "flops": 2 * HD * c["q"] * sum(lens)}
    if c["kind"] == "topk":
        return {"bytes": c["q"] * (4 * _npages([max(c["q"], L) for L in _lens(c)]) + 4 * c["B"] * c["k"]),
                "flops": 0}
    B, q, H, Hkv = c["B"], c["q"], c["H"], c["Hkv"]
    lens = _lens(c)
    if c["k"]:
        pos = [L - q + j for L in lens for j in range(q)]
        seen = sum(min(PT, p + 1 - b * PT) for x, p in zip(_lists(c), pos) for b in x if b >= 0)
        tok, pairs = seen, seen
    else:
        tok = sum(lens)
        pairs = sum(max(0, L - q + j + 1) for L in lens for j in range(q))
    return {"bytes": tok * Hkv * 2 * HD + 2 * tok * Hkv // SUB + B * q * H * (HD * 4 + 4),
            "flops": 4 * HD * H * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    if c["kind"] == "append":
        return _exact_append(c, seed)
    if c["kind"] == "score":
        return _exact_score(c, seed)
    if c["kind"] == "attn":
        return _exact_attn(c, seed)
    return None  # block numbers: equal or wrong


def _exact_append(c, seed):
    """The turned q as a product of complex numbers; the stored codes have no 64-bit value."""
    st = prepare(c, seed)
    T, rot = st["T"], c["rot"]
    y = st["q"].double().clone()
    if rot:
        p = (st["pos"] + c["shift"]).double()
        w = torch.polar(torch.full((T, rot // 2), _factor(c), dtype=F64, device=DEV),
                        p[:, None] * st["inv"].double()[None])[:, None]
        i = torch.arange(rot // 2, device=DEV)
        a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rot // 2)
        z = torch.complex(y[:T][..., a], y[:T][..., b]) * w
        y[:T, :, a], y[:T, :, b] = z.real, z.imag
    y[T:] = 0
    return {"q": y, "k": None, "v": None, "k_scales": None, "v_scales": None}


def _exact_score(c, seed):
    """One sequence at a time, every key written out."""
    st = prepare(c, seed)
    q = c["q"]
    out = torch.zeros(st["scores"].shape, dtype=F64, device=DEV)
    mag = torch.tensor(GRID, dtype=F64, device=DEV)
    for s, L in enumerate(st["seq_lens"].tolist()):
        n = (L + PT - 1) // PT
        p = st["pages"][st["table"][s, :n].long()]
        if c["fp8"]:
            x = p.view(E4M3).double().reshape(-1, HD)[:L] * 0.01
        else:
            d = p[:, :PT * 64].reshape(-1, 64)[:L].long()
            x = torch.empty((L, HD), dtype=F64, device=DEV)
            for half, nib in ((0, d % 16), (1, d // 16)):
                x[:, half::2] = mag[nib % 8] * (1.0 - 2.0 * (nib // 8))
            x = x * torch.pow(2.0, p[:, PT * 64:].reshape(-1, 4)[:L].double() - 127).repeat_interleave(32, 1)
        for j in range(q):
            y = torch.full((n * PT,), -math.inf, dtype=F64, device=DEV)
            m = L - q + j + 1
            y[:m] = x[:m] @ st["iq"][s * q + j].double()
            out[s * q + j, :n] = y.view(n, PT).max(1).values
    return out


def _exact_attn(c, seed):
    """One token of one sequence at a time, over the rows that it sees."""
    B, q, H, Hkv = c["B"], c["q"], c["H"], c["Hkv"]
    if sum(_lens(c)) * q * H > 2e9 or B * q * Hkv > 3000:
        return None
    st = prepare(c, seed)
    out = torch.zeros((B * q, H, HD), dtype=F64, device=DEV)
    lse = torch.full((B * q, H), -math.inf, dtype=F64, device=DEV)
    lists = _lists(c) if c["k"] else None

    def values(pool, scales, pid, rows):
        x = pool[pid].view(E4M3).double().reshape(len(pid), Hkv, PT, HD)
        f = torch.pow(2.0, scales[pid].double() - 127).repeat_interleave(SUB, dim=-1)
        return (x * f[..., None]).transpose(0, 1).reshape(Hkv, -1, HD)[:, rows]

    for s, L in enumerate(_lens(c)):
        for j in range(q):
            t, p = s * q + j, L - q + j
            blocks = [b for b in lists[t] if b >= 0] if c["k"] else list(range(p // PT + 1))
            if p < 0 or not blocks:
                continue
            at = torch.tensor(blocks, device=DEV)
            rows = ((at[:, None] * PT + torch.arange(PT, device=DEV)).flatten() <= p).nonzero()[:, 0]
            pid = st["table"][s, at].long()
            kk, vv = values(st["kp"], st["ks"], pid, rows), values(st["vp"], st["vs"], pid, rows)
            x = st["q"][t].double().view(Hkv, H // Hkv, HD) @ kk.transpose(1, 2) * SCALE
            out[t] = (torch.softmax(x, -1) @ vv).reshape(H, HD)
            lse[t] = torch.logsumexp(x, -1).reshape(H)
    return {"out": out, "lse": lse}
