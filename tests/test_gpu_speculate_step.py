"""SpeculativeStep and PageBook: several speculative steps in a row as a serving loop runs
them, against the plain implementations (decisions and cache bytes equal; the attention
within its tolerance), and a greedy loop that must give the tokens of one-at-a-time decoding."""
import numpy as np
import pytest
import torch

import _spec_ref as R
import mxfp4_sparse_paged_gb300 as m
from mxfp4_sparse_paged_gb300.speculate import PageBook, SpeculativeStep, tree_masks
from mxfp4_sparse_paged_gb300.step import PagedCaches

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda"


def test_tree_masks():
    rng = np.random.default_rng(1)
    p = np.array([R.random_tree(rng, 64) for _ in range(5)], np.int32)
    want = np.stack([R.masks_of(x) for x in p]).view(np.int64)
    assert np.array_equal(tree_masks(torch.from_numpy(p).to(DEV)).cpu().numpy(), want)


class Model:
    """A toy layer: embeddings to q, k, v and index rows, attention output to probabilities."""

    def __init__(self, V, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.E = r(V, 128)
        self.Wq, self.Wk, self.Wv, self.Wi = r(128, 16 * 128), r(128, 128), r(128, 128), r(128, 128)
        self.O = r(16 * 128, V)
        self.s = 128 ** -0.5

    def rows(self, tokens):
        x = self.E[tokens.long()]
        q = (x @ self.Wq * self.s).view(*tokens.shape, 16, 128).to(torch.bfloat16)
        return (q, (x @ self.Wk * self.s).unsqueeze(-2).contiguous(),
                (x @ self.Wv * self.s).unsqueeze(-2).contiguous(), (x @ self.Wi * self.s).contiguous())

    def probs(self, out, sharp=1.0):
        return torch.softmax(sharp * out.flatten(-2).float() @ self.O * 0.1, -1)


def prompts(model, lens, V, seed, spare, fp8=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = [(L + 200) // 128 + 1 for L in lens]
    P = sum(n) + spare
    ids = torch.randperm(P, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), max(n)), -1, dtype=torch.int32)
    o = 0
    caches = PagedCaches(P, device=DEV, fp8_index_scale=fp8)
    for s, L in enumerate(lens):
        table[s, :n[s]] = ids[o:o + n[s]].to(torch.int32)
        o += n[s]
    table = table.to(DEV)
    tokens = []
    for s, L in enumerate(lens):
        t = torch.randint(0, V, (L,), generator=g, device=DEV)
        _, k, v, ik = model.rows(t)
        pos = torch.arange(L, device=DEV)
        slots = table[s, pos // 128].long() * 128 + pos % 128
        caches.insert_rows(k, v, ik, slots)
        tokens.append(t.tolist())
    return caches, table, tokens


def test_steps_against_the_plain_implementations():
    V, N, lens = 40, 9, [5, 127, 300]
    model = Model(V, 1)
    caches, table, _ = prompts(model, lens, V, 2, 3, fp8=0.05)
    step = SpeculativeStep(caches, table, torch.tensor(lens, dtype=torch.int32, device=DEV), N)
    rng = np.random.default_rng(5)
    B, bt = len(lens), table.cpu().numpy()
    cur = np.array(lens, np.int32)
    root = torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)
    for it in range(4):
        parents = np.array([R.random_tree(rng, N) for _ in range(B)], np.int32)
        counts = rng.integers(1, N + 1, B).astype(np.int32)
        tokens = rng.integers(0, V, (B, N)).astype(np.int32)
        tk = torch.from_numpy(tokens).to(DEV)
        tk[:, 0] = root
        q, k, v, ik = model.rows(tk)
        pt = torch.from_numpy(parents).to(DEV)
        out = step.attend(q, k, v, ik, pt, torch.from_numpy(counts).to(DEV))
        kp, vp = caches.k_pages.cpu().numpy(), caches.v_pages.cpu().numpy()
        idx, f8 = caches.idx_pages.cpu().numpy(), caches.fp8_idx_pages.cpu().numpy()
        masks = np.stack([R.masks_of(p) for p in parents])
        want = R.attend(q.float().cpu().numpy(), kp, vp, bt, cur + counts, counts, masks, 0, 0,
                        step.scale)
        got = out.float().cpu().numpy()
        assert np.all(np.abs(got - want[0]) <= want[2])
        target = model.probs(out)
        draft = torch.softmax(torch.randn((B, N, V), device=DEV), -1) if it % 2 else None
        u = torch.rand((B, N), device=DEV)
        us = torch.rand((B,), device=DEV)
        path, acc, nxt = step.verify(target, draft, tk, pt, u, us)
        assert m.mx4_check_status() == 0
        ref = R.verify(target.cpu().numpy(), None if draft is None else draft.cpu().numpy(),
                       tk.cpu().numpy(), parents, u.cpu().numpy(), us.cpu().numpy(), counts)
        for g, w in zip((path, acc, nxt), ref):
            assert np.array_equal(g.cpu().numpy(), w)
        pools, new = R.accept(ref[0], ref[1], cur + counts, counts, bt, [kp, vp, idx, f8])
        for pool, w in zip((caches.k_pages, caches.v_pages, caches.idx_pages, caches.fp8_idx_pages), pools):
            assert np.array_equal(pool.cpu().numpy(), w)
        assert np.array_equal(step.seq_lens.cpu().numpy(), new)
        cur, root = new, nxt.clone()


def test_greedy_speculation_gives_the_greedy_tokens():
    # Targets as one-hot rows: a draft stands iff it is the target's own choice, so whatever
    # is drafted the tokens are those of decoding one at a time.  The two loops reach the same
    # attention by different tilings and orders, each within 2^-7 of the weighted mean of |v|:
    # a token is compared as long as its choice was clear, which a margin below decides.
    V, N, steps = 24, 6, 6
    model = Model(V, 3)
    lens = [37, 250]

    def onehot(p):
        return torch.nn.functional.one_hot(p.argmax(-1), V).float()

    def run(nodes, seed):
        caches, table, _ = prompts(model, lens, V, 4, 1)
        step = SpeculativeStep(caches, table, torch.tensor(lens, dtype=torch.int32, device=DEV), nodes)
        root = torch.tensor([5, 6], dtype=torch.int32, device=DEV)
        rng = np.random.default_rng(seed)
        out_tokens, margins = [[], []], [[], []]
        while min(map(len, out_tokens)) < 12:
            parents = np.array([R.random_tree(rng, nodes) for _ in lens], np.int32)
            tk = torch.from_numpy(rng.integers(0, V, (2, nodes)).astype(np.int32)).to(DEV)
            tk[:, 0] = root
            q, k, v, ik = model.rows(tk)
            pt = torch.from_numpy(parents).to(DEV)
            p = model.probs(step.attend(q, k, v, ik, pt), sharp=5.0)
            top = p.topk(2, -1).values
            path, acc, nxt = step.verify(onehot(p), None, tk, pt, torch.rand((2, nodes), device=DEV),
                                         torch.rand((2,), device=DEV))
            assert m.mx4_check_status() == 0
            for s in range(2):
                a = int(acc[s])
                nodes_in = path[s, :a].tolist()
                choice = [int(tk[s, j]) for j in nodes_in[1:]] + [int(nxt[s])]
                out_tokens[s] += choice
                margins[s] += [float(top[s, j, 0] / top[s, j, 1]) for j in nodes_in]
            root = nxt.clone()
        return out_tokens, margins

    one, mar = run(1, 0)
    for seed in (1, 2):
        many, _ = run(N, seed)
        for s in range(2):
            for a, b, mg in zip(one[s], many[s], mar[s]):
                if mg < 1.2:
                    break
                assert a == b


def test_page_book_forks_and_frees_as_beams_do():
    model = Model(16, 7)
    lens = [130, 256]
    caches, table, _ = prompts(model, lens, 16, 8, 20)
    book = PageBook(caches.num_pages, table)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    start = int(book.free_count)
    rows = torch.tensor([0, 0, 1, 0], dtype=torch.int32, device=DEV)
    tables, cl = book.fork(rows, table, sl, caches)
    assert m.mx4_check_status() == 0
    assert cl.tolist() == [130, 130, 256, 130] and int(book.free_count) == start - 3
    # a child attends like its parent
    q = torch.randn((1, 1, 16, 128), device=DEV).to(torch.bfloat16)
    outs = []
    for t, L in ((table[:1], sl[:1]), (tables[1:2], cl[1:2])):
        out = torch.empty_like(q)
        ws = torch.empty(m.tree_paged_decode_workspace(1, 1, 16, 1), dtype=torch.uint8, device=DEV)
        m.tree_paged_decode(q, caches.k_pages, caches.v_pages, t.contiguous(), L.contiguous(), 0.1, out, ws)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    book.free(tables, cl)
    book.free(table, torch.tensor([t * 128 for t in (table >= 0).sum(1).tolist()], dtype=torch.int32, device=DEV))
    assert m.mx4_check_status() == 0
    assert int(book.free_count) == caches.num_pages and not book.ref_counts.any()


def test_a_step_past_the_table_is_reported_and_leaves_the_lengths():
    # the first sequence's table ends one token on, the second's next page is none, the third has
    # room: the first two sit the step out, with a bad-slot bit and no other
    V, N, lens = 16, 3, [511, 128, 60]
    model = Model(V, 9)
    caches, table, _ = prompts(model, lens, V, 10, 3)
    table = table[:, :4].contiguous()
    table[1, 1:] = -1
    step = SpeculativeStep(caches, table, torch.tensor(lens, dtype=torch.int32, device=DEV), N)
    tk = torch.ones((3, N), dtype=torch.int32, device=DEV)
    pt = torch.tensor([[-1, 0, 1]] * 3, dtype=torch.int32, device=DEV)
    q, k, v, ik = model.rows(tk)
    out = step.attend(q, k, v, ik, pt)
    target = torch.full((3, N, V), 1.0 / V, device=DEV)
    path, acc, nxt = step.verify(target, None, tk, pt, torch.zeros((3, N), device=DEV),
                                 torch.zeros((3,), device=DEV))
    with pytest.raises(m.Mx4Error) as ei:
        m.mx4_check_status()
    assert ei.value.bits == 0x1
    assert step.seq_lens.tolist() == [511, 128, 63] and acc.tolist() == [0, 0, 3]
    assert nxt.tolist() == [-1, -1, 0] and not out[:2].any() and out[2].any()


def test_children_grow_over_page_borders_and_give_all_pages_back():
    # children of a partly filled page, of a full one and of one about to be full take pages as
    # they go, four steps of five nodes, each attending to its own rows; freed with their lengths
    V, N, lens = 16, 5, [126, 256, 250]
    model = Model(V, 11)
    caches, table, _ = prompts(model, lens, V, 12, 20)
    for s, L in enumerate(lens):  # no page ahead of the lengths
        table[s, (L + 127) // 128:] = -1
    book = PageBook(caches.num_pages, table)
    parents_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rows = torch.tensor([0, 1, 2, 0, 1], dtype=torch.int32, device=DEV)
    tables, cl = book.fork(rows, table, parents_lens, caches)
    step = SpeculativeStep(caches, tables, cl, N)
    rng = np.random.default_rng(3)
    cur = np.array(lens, np.int32)[rows.cpu().numpy()]
    for it in range(4):
        book.grow(tables, step.seq_lens, N)
        bt = tables.cpu().numpy()
        tk = torch.from_numpy(rng.integers(0, V, (5, N)).astype(np.int32)).to(DEV)
        q, k, v, ik = model.rows(tk)
        out = step.attend(q, k, v, ik)
        kp, vp = caches.k_pages.cpu().numpy(), caches.v_pages.cpu().numpy()
        chain = np.stack([R.masks_of(list(range(-1, N - 1)))] * 5)
        want = R.attend(q.float().cpu().numpy(), kp, vp, bt, cur + N, np.full(5, N), chain, 0, 0,
                        step.scale)
        assert np.all(np.abs(out.float().cpu().numpy() - want[0]) <= want[2])
        pt = torch.tensor([list(range(-1, N - 1))] * 5, dtype=torch.int32, device=DEV)
        target = torch.full((5, N, V), 1.0 / V, device=DEV)
        u = torch.zeros((5, N), device=DEV)  # all stand but, in one step, the first child's third
        if it == 1:
            u[0, 3] = 0.5
        step.verify(target, None, tk, pt, u, torch.rand((5,), device=DEV))
        assert m.mx4_check_status() == 0
        cur = cur + N
        if it == 1:
            cur[0] -= 2
        assert np.array_equal(step.seq_lens.cpu().numpy(), cur)
    assert all(len(set(bt[s][bt[s] >= 0])) == (cur[s] + 127) // 128 for s in range(5))
    book.free(tables, step.seq_lens)
    book.free(table, parents_lens)
    assert m.mx4_check_status() == 0
    assert int(book.free_count) == caches.num_pages and not book.ref_counts.any()
