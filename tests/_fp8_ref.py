"""Plain forms of the 8-bit cache's operators in 64 bits, on the CPU, written from the header."""
import math

import torch

E4M3 = torch.float8_e4m3fn
F64 = torch.float64


def values(pages, scales):
    """uint8 [P, H, 16384], [P, H, 4] -> float64 [P, H, 128, 128]."""
    P, H = pages.shape[:2]
    x = pages.contiguous().view(E4M3).to(F64).view(P, H, 4, 32 * 128)
    e = scales.to(F64)
    f = torch.where(e == 255, torch.full_like(e, math.nan), torch.pow(2.0, e - 127))
    return (x * f[..., None]).view(P, H, 128, 128)


def turned(x, pos, phases, interleaved, factor):
    """x [T, heads, 128] turned by int positions; angles from the integer phases, exactly reduced."""
    x = x.to(F64).clone()
    if phases is None:
        return x
    R = 2 * len(phases)
    for t, p in enumerate(pos):
        a = [((int(w) % (1 << 64)) * int(p) % (1 << 64)) / 2.0**64 * 2 * math.pi for w in phases]
        c = torch.tensor([math.cos(v) for v in a], dtype=F64) * factor
        s = torch.tensor([math.sin(v) for v in a], dtype=F64) * factor
        i = torch.arange(R // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        u, w = x[t][:, ia].clone(), x[t][:, ib].clone()
        x[t][:, ia], x[t][:, ib] = u * c - w * s, w * c + u * s
    return x


def exponent(amax):
    """The smallest E >= -127 with amax <= 448 * 2^E."""
    if amax == 0:
        return -127
    m, e = math.frexp(amax)
    return max(-127, e - 9 if m <= 0.875 else e - 8)


def attend(q, q_per_seq, k, v, table, lens, scale, blocks=None):
    """q [T, H, 128] over values k, v [P, Hkv, 128, 128]: (out, lse, sum of weight * |V|, sum of
    |q| |K|), float64.  blocks: lists of block numbers a token (None: all)."""
    T, H = q.shape[:2]
    Hkv = k.shape[1]
    G = H // Hkv
    out = torch.zeros((T, H, 128), dtype=F64)
    mag = torch.zeros((T, H, 128), dtype=F64)
    lse = torch.full((T, H), -math.inf, dtype=F64)
    big = torch.zeros((T, H), dtype=F64)
    for t in range(T):
        s, j = divmod(t, q_per_seq)
        p = lens[s] - q_per_seq + j
        if p < 0 or lens[s] > table.shape[1] * 128:
            continue
        todo = range(p // 128 + 1) if blocks is None else [b for b in blocks[t] if 0 <= b <= p // 128]
        rows = [(table[s][b], min(128, p + 1 - 128 * b)) for b in todo]
        rows = [(int(a), n) for a, n in rows if 0 <= a < k.shape[0]]
        if not rows:
            continue
        kk = torch.cat([k[a, :, :n] for a, n in rows], 1)
        vv = torch.cat([v[a, :, :n] for a, n in rows], 1)
        x = q[t].to(F64).view(Hkv, G, 128)
        l = x @ kk.transpose(1, 2) * scale
        w = torch.softmax(l, -1)
        out[t] = (w @ vv).view(H, 128)
        mag[t] = (w @ vv.abs()).view(H, 128)
        lse[t] = torch.logsumexp(l, -1).view(H)
        big[t] = (x.abs() @ kk.abs().transpose(1, 2)).amax(-1).view(H) * abs(scale)
    return out, lse, mag, big


def check_attention(out, lse, want):
    """bf16 out: half a step of bf16 (2^-8 of the value), weights rounded to 11 bits (2^-12 each, 2^-25 of the row's largest where f16 is subnormal,
    counted at 2^-11), and logits of fp32: 128 products summed in fp32 and one rounding of the
    exponent's argument, 2^-18 of sum |q||K| and of the logits' range, on each weight."""
    w, wl, mag, big = want
    out, lse = out.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isnan(out), torch.isnan(w)), "NaN pattern differs"
    dl = 2.0**-18 * (big + 1) + 2.0**-20 * wl.abs().nan_to_num(0, 0, 0)
    tol = 2.0**-8 * w.abs() + (2.0**-11 + 2 * dl[..., None]) * mag + 1e-30
    bad = (out - w).abs() > tol
    assert not bad.any(), (bad.nonzero()[:4], out[bad][:4], w[bad][:4], tol[bad][:4])
    fin = torch.isfinite(wl)
    assert torch.equal(torch.isfinite(lse), fin) and torch.equal(lse == -math.inf, wl == -math.inf)
    assert ((lse - wl).abs()[fin] <= dl[fin] + 1e-6).all(), (lse - wl).abs()[fin].max()


def topk(scores, lens, q, k, first, last):
    """Block lists by a full sort of (always, NaN, score, lower index)."""
    out = []
    for t in range(len(lens) * q):
        s, j = divmod(t, q)
        p = lens[s] - q + j
        n = p // 128 + 1 if p >= 0 else 0
        if n > scores.shape[1] or lens[s] < 0:
            n = 0
        x = scores[t].tolist()
        def order(b):
            if b < first or b >= n - last:
                return (0, 0.0, b)
            return (1, 0.0, b) if math.isnan(x[b]) else (2, -x[b], b)
        got = sorted(sorted(range(n), key=order)[:k])
        out.append(got + [-1] * (k - len(got)))
    return out
