"""Plain 64-bit implementations of a speculative decode step's operators (numpy, one
sequence and one node at a time, from include/mx4sp.h's formulas), and random inputs."""
import numpy as np

PT, HD, PB, FP8 = 128, 128, 8704, 16384
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def random_pages(rng, P, heads, lo=120, hi=128):
    """Pages of random codes, scale bytes in [lo, hi)."""
    pg = np.empty((P, heads, PB), np.uint8)
    pg[..., :8192] = rng.integers(0, 256, (P, heads, 8192), dtype=np.uint8)
    pg[..., 8192:] = rng.integers(lo, hi, (P, heads, 512), dtype=np.uint8)
    return pg


def block_table(rng, lens, spare=2):
    n = [(int(x) + PT - 1) // PT for x in lens]
    P = sum(n) + spare
    ids = rng.permutation(P).astype(np.int32)
    bt = np.full((len(lens), max(1, max(n))), -1, np.int32)
    o = 0
    for s, k in enumerate(n):
        bt[s, :k] = ids[o:o + k]
        o += k
    return bt, P


def rows_of(pages, table_row, head, L):
    """Values [L, 128] of one sequence's cached rows of one head."""
    out = np.zeros((L, HD))
    for a in range(0, L, PT):
        p = pages[table_row[a // PT], head]
        m = min(PT, L - a)
        c = p[:8192].reshape(PT, 64)[:m]
        x = np.stack((GRID[c & 15], GRID[c >> 4]), -1).reshape(m, HD)
        sc = p[8192:].reshape(PT, 4)[:m].astype(np.float64)
        f = np.where(sc == 255, np.nan, np.exp2(sc - 127))
        out[a:a + m] = x * np.repeat(f, 32, axis=1)
    return out


def random_tree(rng, N):
    return [-1] + [int(rng.integers(max(0, j - 6), j)) for j in range(1, N)]


def masks_of(parents):
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | (1 << j))
    return np.array(out, np.uint64)


def sees(L, n, mask, window, sinks):
    """Boolean [n, L]: what node j sees (mask: n Python ints)."""
    base = L - n
    bits = [int(m) & ((1 << n) - 1) for m in mask]
    d = [max(1, bin(b).count("1")) - 1 for b in bits]
    see = np.zeros((n, L), bool)
    for j in range(n):
        for i in range(base):
            see[j, i] = window == 0 or i > base + d[j] - window or i < sinks
        for i in range(n):
            see[j, base + i] = bool(bits[j] >> i & 1) and (
                window == 0 or d[i] > d[j] - window or base + d[i] < sinks)
    return see


def attend(q, kp, vp, bt, lens, n_nodes, mask, window, sinks, scale, rows=None):
    """(out, lse, tol_out, tol_lse), all [B, N, H(, 128)] float64.

    Tolerances, from the roundings that the operator states.  Logits: q goes into the
    tensor core as two E4M3 parts, off by at most 2^-22 of the largest element of its
    32-block; products and sums in fp32, 16 roundings of 2^-24 taken for the sum of the
    terms' magnitudes, doubled.  Output: one bf16 rounding (2^-8) of it and one of each
    weight, so of the weighted mean of |v|, and a logit error dl moves every weight by
    a factor e^dl, twice (its own and the sum's)."""
    B, N, H, _ = q.shape
    Hkv = kp.shape[1]
    G = H // Hkv
    out = np.zeros((B, N, H, HD))
    lse = np.full((B, N, H), -np.inf)
    t_out = np.zeros((B, N, H, HD))
    t_lse = np.zeros((B, N, H))
    for s in range(B):
        L, n = int(lens[s]), int(n_nodes[s])
        see = sees(L, n, mask[s], window, sinks)
        for h in range(Hkv):
            k, v = rows_of(kp, bt[s], h, L), rows_of(vp, bt[s], h, L)
            ka = np.abs(k).reshape(L, 4, 32).sum(-1)
            for j in range(n):
                at = see[j]
                if not at.any():
                    continue
                for g in range(G):
                    x = q[s, j, h * G + g].astype(np.float64)
                    l = scale * (k[at] @ x)
                    amax = np.abs(x).reshape(4, 32).max(-1)
                    dl = abs(scale) * (2.0 ** -22 * (ka[at] @ amax) +
                                       2.0 ** -19 * (np.abs(k[at]) @ np.abs(x)))
                    top = l.max()
                    w = np.exp(l - top)
                    z = w.sum()
                    o = (w @ v[at]) / z
                    A = (w @ np.abs(v[at])) / z
                    e = np.max(dl) + 2.0 ** -20
                    out[s, j, h * G + g] = o
                    lse[s, j, h * G + g] = np.log(z) + top
                    t_out[s, j, h * G + g] = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * e) * 1.02 * A
                    t_lse[s, j, h * G + g] = e + 2.0 ** -22 * (1 + abs(np.log(z) + top))
    return out, lse, t_out, t_lse


def verify(target, draft, tokens, parents, u, us, n_nodes):
    """(path, n_accepted, next_token) by the definition, float64."""
    B, N, V = target.shape
    path = np.full((B, N), -1, np.int32)
    acc = np.zeros(B, np.int32)
    nxt = np.full(B, -1, np.int32)
    for s in range(B):
        n = int(n_nodes[s])
        if n == 0:
            continue
        cur, got = 0, [0]
        W, T, shut = target[s, 0].astype(np.float64), 1.0, False
        for j in range(1, n):
            if parents[s, j] != cur or shut or not 0 <= tokens[s, j] < V:
                continue
            x = int(tokens[s, j])
            if draft is None:
                q = np.zeros(V)
                q[x] = 1.0
            else:
                q = draft[s, cur].astype(np.float64)
            if float(u[s, j]) * T * q[x] < W[x]:
                cur = j
                got.append(j)
                W, T = target[s, j].astype(np.float64), 1.0
            else:
                W = np.maximum(W - T * q, 0)
                T = W.sum()
                if T == 0:
                    W, shut = target[s, cur].astype(np.float64), True
        path[s, :len(got)] = got
        acc[s] = len(got)
        c = np.cumsum(W)
        if c[-1] > 0:
            nxt[s] = int(np.argmax(c > float(us[s]) * c[-1]))
    return path, acc, nxt


def row_parts(pool):
    """Writable views of a pool's rows: [..., 128, bytes] each."""
    if pool.shape[-1] == FP8:
        return [pool.reshape(*pool.shape[:-1], PT, 128)]
    return [pool[..., :8192].reshape(*pool.shape[:-1], PT, 64),
            pool[..., 8192:].reshape(*pool.shape[:-1], PT, 4)]


def join_parts(pool, parts):
    if len(parts) == 1:
        pool[...] = parts[0].reshape(pool.shape)
    else:
        pool[..., :8192] = parts[0].reshape(*pool.shape[:-1], 8192)
        pool[..., 8192:] = parts[1].reshape(*pool.shape[:-1], 512)


def accept(path, acc, lens, n_nodes, bt, pools):
    """New pools and lengths."""
    out = [p.copy() for p in pools]
    new = lens.copy()
    for x, pool in zip(out, pools):
        src, dst = row_parts(pool.copy()), [p.copy() for p in row_parts(x)]
        for s in range(len(lens)):
            base = int(lens[s]) - int(n_nodes[s])
            for i in range(int(acc[s])):
                a, b = base + int(path[s, i]), base + i
                for f, t in zip(src, dst):
                    t[bt[s, b // PT], ..., b % PT, :] = f[bt[s, a // PT], ..., a % PT, :]
        join_parts(x, dst)
    for s in range(len(lens)):
        new[s] = int(lens[s]) - int(n_nodes[s]) + int(acc[s])
    return out, new


def fork(rows, bt, lens, refs, fl, fc, pools):
    """(child tables, child lens, refs, free count, pools) after mx4_fork_pages."""
    refs, fc, pools = refs.copy(), int(fc), [p.copy() for p in pools]
    n, W = len(rows), bt.shape[1]
    child = np.full((n, W), -1, np.int32)
    cl = np.zeros(n, np.int32)
    for i, r in enumerate(rows):
        if not 0 <= r < len(bt):
            continue
        L = int(lens[r])
        full, rem = L // PT, L % PT
        if rem:
            if fc == 0:
                continue
            fc -= 1
            new = int(fl[fc])
            child[i, full] = new
            refs[new] = 1
            for p in pools:
                parts = [x.copy() for x in row_parts(p)]
                for x in parts:
                    x[new, ..., :rem, :] = x[bt[r, full], ..., :rem, :]
                join_parts(p, parts)
        child[i, :full] = bt[r, :full]
        for p in bt[r, :full]:
            refs[p] += 1
        cl[i] = L
    return child, cl, refs, fc, pools


def free(tables, lens, refs, fl, fc):
    refs, fl, fc = refs.copy(), fl.copy(), int(fc)
    gone = []
    for row, L in zip(tables, lens):
        for p in row[:(int(L) + PT - 1) // PT]:
            if refs[p] > 0:
                refs[p] -= 1
                if refs[p] == 0:
                    gone.append(int(p))
    for p in sorted(gone):
        fl[fc] = p
        fc += 1
    return refs, fl, fc
