"""Calls over many sequences on the GPU: append, tree attention, acceptance and adapters against their definitions
in float64, numbers in device memory that are out of range, a whole layer of several requests."""
import dataclasses
import os
import subprocess
import sys

import numpy as np
import pytest

import batch_reference as R
from quantized_transformer_prefill_q1_gb300 import pf, synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Step:
    """A batch over a cache with NaN in every slot that no sequence holds."""

    def __init__(self, kind, nq, nkv, hd, rows, start, paged=True, parents=None, norm=False, n_layers=2, layer=1, seed=0, spare=3):
        self.rng = rng = np.random.default_rng(seed)
        self.kind, self.dt, self.nq, self.nkv, self.hd, self.layer = kind, TYPES[kind], nq, nkv, hd, layer
        self.rows, self.start, self.norm = list(rows), list(start), norm
        self.begin = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.total = int(self.begin[-1])
        self.n_rows = self.total + spare
        self.max_seq = max(s + r for s, r in zip(start, rows)) + 5
        self.pages = -(-self.max_seq // 128)
        need = [-(-(s + r) // 128) for s, r in zip(start, rows)]
        self.pool = sum(need) + 2 if paged else 0
        shape = dataclasses.replace(synth.QWEN3_8B_LAYER, n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, kv_dtype=kind, qk_norm=norm)
        self.cfg = pf.make_config(shape, 256, n_layers=n_layers, max_seq=self.max_seq, kv_block_pool=self.pool)
        self.slots = self.pool * 128 if paged else self.max_seq
        self.parents = parents if parents is not None else [R.chain(n) for n in rows]
        self.parent_dev = None if parents is None else ints(np.concatenate([*parents, [7] * spare]))
        self.table = None
        if paged:
            order, at = rng.permutation(self.pool), 0
            self.table = np.full((len(rows), self.pages), -1, np.int32)
            for b, m in enumerate(need):
                self.table[b, :m] = order[at:at + m]
                at += m
        self.table_dev = ints(self.table) if paged else None
        self.begin_dev, self.start_dev = ints(self.begin), ints(self.start)
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.full((n_layers, nkv, self.slots, hd), float("nan"), dtype=self.dt, device="cuda") for _ in "kv")
        self.batch = self.make_batch()

    def make_batch(self, max_rows=None):
        return pf.Batch(self.begin_dev, n_rows=self.n_rows, max_rows=max_rows or max(1, *self.rows), start=self.start_dev,
                        parent=self.parent_dev, blocks=self.table_dev)

    def slot(self, b, p):
        p = np.asarray(p)
        return p if self.table is None else self.table[b][p // 128] * 128 + p % 128

    def fill(self, own_rows=True, heavy=1.0):
        """Cached positions (and the sequences' own rows) hold normal values."""
        for b, n in enumerate(self.rows):
            i = torch.from_numpy(np.asarray(self.slot(b, np.arange(self.start[b] + (n if own_rows else 0))), np.int64)).cuda()
            for c in (self.k, self.v):
                x = self.rng.standard_normal((c.shape[0], self.nkv, len(i), self.hd)) * (heavy if c is self.k else 1)
                c[:, :, i] = torch.from_numpy(x).cuda().to(self.dt)

    def held(self, c, b, layer=None):
        """Sequence b's values of positions 0 .. start + rows - 1, float64 [nkv, positions, hd]."""
        i = torch.from_numpy(np.asarray(self.slot(b, np.arange(self.start[b] + self.rows[b])), np.int64)).cuda()
        return c[self.layer if layer is None else layer][:, i].double().cpu().numpy()

    def scratch(self):
        return pf.attention_tree_scratch(self.cfg, len(self.rows), max(1, *self.rows))

    def q(self, scale=1.0):
        return torch.from_numpy(self.rng.standard_normal((self.n_rows, self.nq, self.hd)) * scale).cuda().to(self.dt)

    def attend(self, q, scratch=None):
        out = torch.full((self.n_rows, self.nq * self.hd), 7.0, dtype=torch.float16, device="cuda")
        pf.pf_op_attention_tree(self.cfg, self.batch, q, self.k, self.v, self.layer, out, self.scratch() if scratch is None else scratch,
                                self.status)
        return out

    def weights(self):
        """Rounding of the softmax weights: to the cache's type; for up to 8 query rows per kv head of a bf16 cache as
        two terms, where the second, at most half a step of the first, is rounded."""
        two = self.kind == "bf16" and max(1, *self.rows) * (self.nq // self.nkv) <= 8
        return R.half_step(self.kind) ** 2 if two else R.half_step(self.kind)

    def check_attention(self, q, out):
        got, qq = out.double().cpu().numpy().reshape(self.n_rows, self.nq, self.hd), q.double().cpu().numpy()
        for b, n in enumerate(self.rows):
            if n == 0:
                continue
            rows = slice(self.begin[b], self.begin[b + 1])
            ref, bound = R.attention(qq[rows], self.held(self.k, b), self.held(self.v, b), self.start[b], self.parents[b], self.weights())
            off = np.abs(got[rows] - ref)
            assert (off <= bound).all(), (b, n, self.start[b], float((off / bound).max()), np.argwhere(~(off <= bound))[:3])
        assert (got[self.total:] == 7).all()


def trees(rng, rows):
    return [R.random_tree(rng, n, roots=1 + (n > 5)) for n in rows]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nkv,hd,norm", [(32, 8, 128, True), (4, 2, 64, True), (1, 1, 128, False), (64, 1, 64, False), (64, 8, 128, True)])
@pytest.mark.parametrize("paged,tree", [(True, True), (True, False), (False, True)])
def test_append(kind, nq, nkv, hd, norm, paged, tree):
    rows, start = ([5, 0, 1, 40, 3, 130], [126, 9, 0, 250, 127, 1]) if paged else ([37], [11])
    rng = np.random.default_rng(hd + nq)
    s = Step(kind, nq, nkv, hd, rows, start, paged, trees(rng, rows) if tree else None, norm)
    width = (nq + 2 * nkv) * hd
    qkv = torch.from_numpy(rng.standard_normal((s.n_rows, width)) * 2).cuda().float()
    qn, kn = ((1 + 0.1 * rng.standard_normal((2, hd))).astype(np.float32) if norm else (None, None))
    qd, kd = (torch.from_numpy(x).cuda() if norm else None for x in (qn, kn))
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, hd, s.max_seq)).cuda()
    q = torch.full((s.n_rows, nq, hd), 7.0, dtype=s.dt, device="cuda")
    pf.pf_op_batch_append(s.cfg, s.batch, qkv, qd, kd, rope, s.layer, q, s.k, s.v, s.status)
    pf.pf_status_read(s.status)
    assert (q[s.total:] == 7).all()
    want_k, want_v = (torch.full_like(c, float("nan")) for c in (s.k, s.v))
    tiny = 2.0 ** -25 if kind == "f16" else 0.0
    for b, n in enumerate(rows):
        if n == 0:
            continue
        x = qkv[s.begin[b]:s.begin[b + 1]].cpu().numpy()
        pos = start[b] + R.depths(s.parents[b])
        rq, rk, rv, size = R.append(x, nq, nkv, hd, qn, kn, s.cfg.eps, s.cfg.rope_theta, pos)
        i = torch.from_numpy(np.asarray(s.slot(b, start[b] + np.arange(n)), np.int64)).cuda()
        got_q = q[s.begin[b]:s.begin[b + 1]].double().cpu().numpy()
        got_k = s.k[s.layer][:, i].double().cpu().numpy().transpose(1, 0, 2)
        # half a step of the type; f32: the norm (hd squares' sum, root, division, two products) and the rotation
        # (table, two products, their sum) within 16 roundings of the products' sizes
        for got, ref, sz in ((got_q, rq, size[:, :nq]), (got_k, rk, size[:, nq:])):
            off = np.abs(got - ref)
            bound = R.half_step(kind) * (np.abs(ref) + 16 * 2.0 ** -24 * sz) + 16 * 2.0 ** -24 * sz + tiny
            assert (off <= bound).all(), (b, float((off - bound).max()))
        want_k[s.layer][:, i] = s.k[s.layer][:, i]
        want_v[s.layer][:, i] = torch.from_numpy(rv.transpose(1, 0, 2)).cuda().float().to(s.dt)
    for got, want in ((s.k, want_k), (s.v, want_v)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_longest_chunks():
    """8,192 rows of one sequence beside others, appended and through adapters."""
    rng = np.random.default_rng(6)
    rows, start = [3, 8192, 0, 100], [1, 77, 5, 0]
    s = Step("bf16", 2, 1, 64, rows, start, True, n_layers=1, layer=0)
    qkv = torch.from_numpy(rng.standard_normal((s.n_rows, 4 * 64))).cuda().float()
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, 64, s.max_seq)).cuda()
    q = torch.full((s.n_rows, 2, 64), 7.0, dtype=s.dt, device="cuda")
    pf.pf_op_batch_append(s.cfg, s.batch, qkv, None, None, rope, 0, q, s.k, s.v, s.status)
    pf.pf_status_read(s.status)
    assert (q[s.total:] == 7).all()
    for b, n in enumerate(rows):
        pos = start[b] + np.arange(n)
        at = slice(s.begin[b], s.begin[b + 1])
        rq, rk, rv, size = R.append(qkv[at].cpu().numpy(), 2, 1, 64, None, None, s.cfg.eps, s.cfg.rope_theta, pos)
        i = torch.from_numpy(np.asarray(s.slot(b, pos), np.int64)).cuda()
        for got, ref, sz in ((q[at], rq, size[:, :2]), (s.k[0][:, i].transpose(0, 1), rk, size[:, 2:])):
            # half a step, and the rotation in f32 as in test_append
            off = np.abs(got.double().cpu().numpy() - ref)
            assert (off <= 2.0 ** -8 * (np.abs(ref) + 2.0 ** -20 * sz) + 2.0 ** -20 * sz).all()
        assert torch.equal(s.v[0][:, i], qkv[at, 3 * 64:].reshape(n, 1, 64).transpose(0, 1).to(s.dt))
    x = torch.from_numpy(rng.standard_normal((s.n_rows, 128))).cuda().half()
    a = torch.from_numpy(rng.standard_normal((1, 16, 128)) * 0.1).cuda().half()
    w = torch.from_numpy(rng.standard_normal((1, 256, 16)) * 0.1).cuda().half()
    y = qkv.clone()
    pf.pf_op_adapters(s.batch, x, y, y, ints([0, 0, 0, -1]), a, w, torch.ones(1, device="cuda"), s.status)
    pf.pf_status_read(s.status)
    last = int(s.begin[2])
    ref, bound = R.adapters(qkv[:last].cpu().numpy(), x[:last].cpu().numpy(), a[0].cpu().numpy(), w[0].cpu().numpy(), 1.0)
    assert (np.abs(y[:last].double().cpu().numpy() - ref) <= bound).all() and torch.equal(y[last:], qkv[last:])


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nkv,hd", [(32, 8, 128), (4, 2, 64), (8, 8, 64), (16, 1, 128), (64, 1, 64)])
@pytest.mark.parametrize("top", [1, 3, 16, 64])
def test_attention_ragged(kind, nq, nkv, hd, top):
    """Sequences of none to `top` rows, lengths that end on, before and behind pages and tiles."""
    rng = np.random.default_rng(top * 7 + hd + nq)
    start = [0, 1, 31, 127, 128, 129, 300, 511, 640]
    rows = [top, 1, max(1, top - 1), 1, top, 0, max(1, top // 2), top, 1]
    s = Step(kind, nq, nkv, hd, rows, start, True, trees(rng, rows), seed=top)
    s.fill()
    q = s.q()
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n,start,tree", [(1, 0, False), (1, 1000, False), (2, 2049, False), (26, 1021, True), (70, 130, False), (256, 100, True),
                                          (256, 0, False)])
def test_attention_linear(kind, n, start, tree):
    rng = np.random.default_rng(n + start)
    s = Step(kind, 8, 2, 128, [n], [start], False, [R.random_tree(rng, n)] if tree else None, seed=n)
    s.fill()
    q = s.q(2.0)
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("top", [1, 40])
def test_attention_large_scores(kind, top):
    """Scores of thousands: the running maximum rises and falls by hundreds; rows whose first tiles weigh nothing."""
    rng = np.random.default_rng(5)
    rows, start = [top, top, 1], [700, 5, 1500]
    s = Step(kind, 8, 2, 128, rows, start, True, trees(rng, rows), seed=3)
    s.fill(heavy=30.0)
    q = s.q(10.0)
    s.check_attention(q, s.attend(q))
    pf.pf_status_read(s.status)


@pytest.mark.parametrize("kind,nq,nkv,hd", [("bf16", 8, 2, 128), ("f16", 4, 2, 64)])
@pytest.mark.parametrize("top", [1, 4, 33, 64])
def test_attention_long_ragged(kind, nq, nkv, hd, top):
    """Many units a CTA, borders of ranges and tasks in every place: each ring goes round many times."""
    rng = np.random.default_rng(21)
    rows = [top - (i % 2) if top > 1 else 1 for i in range(40)]
    start = [int(x) for x in rng.integers(200, 9000, 40)]
    s = Step(kind, nq, nkv, hd, rows, start, True, trees(rng, rows), n_layers=1, layer=0)
    s.fill()
    q = s.q()
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)


def test_attention_deep_and_wide_trees():
    """A chain given by parents, a star, all nodes under the cache, two of them in one batch."""
    n = 256
    parents = [R.chain(n), np.array([-1] + [0] * (n - 1), np.int32), np.full(n, -1, np.int32), np.arange(n, dtype=np.int32) // 2 - 1 + (np.arange(n) == 1)]
    parents[3][0] = -1
    for p in parents:
        assert (p < np.arange(n)).all() and (p >= -1).all()
    s = Step("f16", 4, 2, 64, [n] * 4, [3, 0, 130, 77], True, parents)
    s.fill()
    q = s.q()
    s.check_attention(q, s.attend(q))
    pf.pf_status_read(s.status)


@pytest.mark.parametrize("top", [1, 64])
def test_attention_repeats_and_streams(top):
    """One scratch for call after call of other lengths, results equal bit for bit; a second stream; a captured call
    whose lengths and tree change between replays."""
    rng = np.random.default_rng(9)
    rows, start = [top, max(1, top - 3), 1, top], [900, 40, 513, 1]  # every position that a replay below reads
    s = Step("bf16", 32, 8, 128, rows, start, True, trees(rng, rows))
    s.fill()
    q, scratch = s.q(), s.scratch()
    first = s.attend(q, scratch)
    s.check_attention(q, first)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        again = s.attend(q, scratch)
    other.synchronize()
    assert torch.equal(first, again)
    out = torch.full_like(first, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pf.pf_op_attention_tree(s.cfg, s.batch, q, s.k, s.v, s.layer, out, scratch, s.status)
    graph.replay()
    assert torch.equal(out, first)
    # shorter rows and caches, other trees: the same addresses
    s.rows = [max(1, top // 2), 0, 1, top]
    s.start = [880, 41, 2, 1]
    s.begin = np.concatenate([[0], np.cumsum(s.rows)]).astype(np.int32)
    s.total = int(s.begin[-1])
    s.parents = trees(rng, s.rows)
    s.begin_dev.copy_(ints(s.begin))
    s.start_dev.copy_(ints(s.start))
    s.parent_dev[:s.total] = ints(np.concatenate(s.parents))
    out.fill_(7.0)
    graph.replay()
    s.check_attention(q, out)
    pf.pf_status_read(s.status)


@pytest.mark.parametrize("n_seq", [33, 200, 1024])
@pytest.mark.parametrize("top", [1, 20])
def test_attention_many_sequences(n_seq, top):
    """Hundreds of short tasks, several to a warp, with sequences of no rows between them."""
    rng = np.random.default_rng(n_seq)
    rows = [int(x) for x in rng.integers(0, top + 1, n_seq)]
    rows[0] = top
    start = [int(x) for x in rng.integers(0, 400, n_seq)]
    s = Step("bf16", 4, 2, 128, rows, start, True, trees(rng, rows), n_layers=1, layer=0)
    s.fill()
    q = s.q()
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)


@pytest.mark.parametrize("n_seq", [1, 3, 40])
@pytest.mark.parametrize("top", [1, 30])
def test_nothing_to_do(n_seq, top):
    """No sequence has a row: nothing is written, nothing recorded."""
    s = Step("f16", 8, 2, 64, [0] * n_seq, [5] * n_seq, True, [np.zeros(0, np.int32)] * n_seq)
    s.batch = s.make_batch(top)
    q = s.q()
    out = torch.full((s.n_rows, s.nq * s.hd), 7.0, dtype=torch.float16, device="cuda")
    pf.pf_op_attention_tree(s.cfg, s.batch, q, s.k, s.v, 1, out, pf.attention_tree_scratch(s.cfg, n_seq, top), s.status)
    rope = torch.zeros(s.max_seq, 32, 2, device="cuda")
    pf.pf_op_batch_append(s.cfg, s.batch, torch.zeros(s.n_rows, 12 * 64, device="cuda"), None, None, rope, 1, q, s.k, s.v, s.status)
    rows, seqs = (torch.full((m,), 9, dtype=torch.int32, device="cuda") for m in (s.n_rows, n_seq))
    path, count, after = rows.clone(), seqs.clone(), seqs.clone()
    pf.pf_op_tree_accept(s.cfg, s.batch, rows, rows, seqs, path, count, after, s.k, s.v, s.status)
    x, a = torch.ones(s.n_rows, 64, dtype=torch.float16, device="cuda"), torch.ones(1, 8, 64, dtype=torch.float16, device="cuda")
    y = torch.full((s.n_rows, 64), 7.0, device="cuda")
    pf.pf_op_adapters(s.batch, x, torch.zeros_like(y), y, torch.zeros_like(seqs), a, a.reshape(1, 64, 8), torch.ones(1, device="cuda"), s.status)
    pf.pf_status_read(s.status)
    assert (out == 7).all() and (y == 7).all() and (path == 9).all() and (count == 0).all() and (after == 9).all()
    assert torch.isnan(s.k).all() and torch.isnan(s.v).all()


@pytest.mark.parametrize("nq,nkv,hd", [(64, 1, 64), (16, 1, 128)])
def test_attention_many_row_blocks(nq, nkv, hd):
    """The most rows that a kv head can have: 256 nodes of all query heads, in blocks of 256."""
    rng = np.random.default_rng(3)
    rows, start = [256, 1, 250], [200, 0, 33]
    s = Step("bf16", nq, nkv, hd, rows, start, True, trees(rng, rows))
    s.fill()
    q = s.q()
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)


@pytest.mark.parametrize("n_seq", [1, 2])
@pytest.mark.parametrize("top", [1, 20, 200])
def test_attention_many_heads(n_seq, top):
    """More tasks of a sequence than SMs."""
    rng = np.random.default_rng(top)
    rows, start = [top, 3][:n_seq], [150, 700][:n_seq]
    s = Step("f16", 200, 200, 64, rows, start, True, trees(rng, rows), n_layers=1, layer=0)
    s.fill()
    q = s.q()
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)


@pytest.mark.parametrize("seed", range(10))
def test_attention_drawn(seed):
    rng = np.random.default_rng(100 + seed)
    nq, nkv, hd = [(32, 8, 128), (4, 2, 64), (8, 8, 64), (16, 1, 128), (32, 4, 128), (64, 8, 128)][rng.integers(6)]
    n_seq = int(np.exp(rng.uniform(0, np.log(70))))
    top = int(np.exp(rng.uniform(0, np.log(65))))
    rows = [int(x) for x in rng.integers(0 if n_seq > 1 else 1, top + 1, n_seq)]
    rows[0] = top
    start = [int(x) for x in rng.integers(0, max(2, int(np.exp(rng.uniform(0, np.log(40000 // n_seq))))), n_seq)]
    s = Step(["bf16", "f16"][seed % 2], nq, nkv, hd, rows, start, True, trees(rng, rows) if seed % 3 else None, seed=seed)
    s.fill()
    q = s.q()
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)


@pytest.mark.parametrize("nq,nkv", [(4, 2), (32, 8)])
def test_hidden_keys(nq, nkv):
    """NaN and infinities in the K of a node reach the rows that see it and no other."""
    n = 24 if nq == 32 else 4
    parent = np.arange(n, dtype=np.int32) // 2 - 1  # a binary tree with two roots
    s = Step("bf16", nq, nkv, 128, [n], [130], True, [parent])
    s.fill()
    q = s.q()
    want = s.attend(q)
    see = R.ancestors(parent)
    for j, bad in ((0, float("nan")), (n - 1, float("inf")), (n // 2, float("-inf"))):
        keep = s.k.clone()
        s.k[:, :, int(s.slot(0, 130 + j))] = bad
        got = s.attend(q)
        blind = torch.from_numpy(~see[:, j]).cuda()
        assert torch.equal(got[:n][blind], want[:n][blind]) and not torch.isfinite(got[:n][~blind]).all(1).any()
        s.k.copy_(keep)
    pf.pf_status_read(s.status)


def test_one_scratch_for_both_forms():
    """A scratch for the most rows serves calls of one row and of many in turn, and smaller batches."""
    rng = np.random.default_rng(8)
    big = Step("bf16", 32, 8, 128, [20, 3, 20, 1], [700, 0, 900, 40], True, trees(rng, [20, 3, 20, 1]))
    one = Step("bf16", 32, 8, 128, [1, 1, 1], [900, 2, 1500], True, trees(rng, [1, 1, 1]))
    scratch = pf.attention_tree_scratch(big.cfg, 4, 20)
    runs = []
    for s in (big, one):
        s.fill()
        runs.append((s, s.q()))
    first = [s.attend(q, scratch) for s, q in runs]
    for (s, q), out in zip(runs, first):
        s.check_attention(q, out)
    for _ in range(5):
        for (s, q), out in zip(runs, first):
            assert torch.equal(s.attend(q, scratch), out)
            pf.pf_status_read(s.status)


@pytest.mark.parametrize("top", [1, 30])
def test_two_streams_at_once(top):
    """Calls on two streams, each with a scratch of its own, and adapters beside them."""
    rng = np.random.default_rng(31)
    steps = []
    for seed in (1, 2):
        rows = [top, 1, top, top]
        s = Step("bf16", 32, 8, 128, rows, [3000 * seed, 50, 700, 5000], True, trees(rng, rows), seed=seed)
        s.fill()
        q = s.q()
        steps.append((s, q, s.attend(q), s.scratch(), torch.cuda.Stream()))
    batch = pf.Batch(ints([0, 70, 100]), n_rows=100, max_rows=70)
    x, base = torch.randn(100, 1024, device="cuda").half(), torch.randn(100, 512, device="cuda")
    a, b = torch.randn(2, 16, 1024, device="cuda").half() * 0.03, torch.randn(2, 512, 16, device="cuda").half()
    args = ints([1, 0]), a, b, torch.ones(2, device="cuda")
    plain = torch.empty_like(base)
    pf.pf_op_adapters(batch, x, base, plain, *args)
    torch.cuda.synchronize()
    outs = []
    for _ in range(15):
        for s, q, want, scratch, stream in steps:
            with torch.cuda.stream(stream):
                y = torch.empty_like(base)
                pf.pf_op_adapters(batch, x, base, y, *args)
                outs.append((s.attend(q, scratch), want))
                outs.append((y, plain))
    torch.cuda.synchronize()
    for s, *_ in steps:
        pf.pf_status_read(s.status)
    for i, (got, want) in enumerate(outs):
        assert torch.equal(got, want), i


def test_cache_past_32_bits():
    """A cache of more than 2^32 bytes: append, attention and acceptance in its last layer and last blocks."""
    rng = np.random.default_rng(12)
    nq, nkv, hd, layers = 32, 8, 128, 9
    rows, start = [26, 1, 40], [1000, 300, 127]
    s = Step("bf16", nq, nkv, hd, rows, start, True, trees(rng, rows), n_layers=1, layer=0)
    high = 1900
    assert layers * nkv * high * 128 * hd * 2 > 2 ** 32
    s.table[s.table >= 0] += high - s.pool  # the last blocks of a larger pool
    s.table_dev.copy_(ints(s.table))
    shape = dataclasses.replace(synth.QWEN3_8B_LAYER, n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, kv_dtype="bf16", qk_norm=False)
    s.cfg = pf.make_config(shape, 256, n_layers=layers, max_seq=s.max_seq, kv_block_pool=high)
    s.layer, s.slots = layers - 1, high * 128
    s.k, s.v = (torch.full((layers, nkv, s.slots, hd), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    s.fill(own_rows=False)
    before = s.k.clone()
    qkv = torch.randn(s.n_rows, (nq + 2 * nkv) * hd, device="cuda")
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, hd, s.max_seq)).cuda()
    q = torch.empty(s.n_rows, nq, hd, dtype=torch.bfloat16, device="cuda")
    pf.pf_op_batch_append(s.cfg, s.batch, qkv, None, None, rope, s.layer, q, s.k, s.v, s.status)
    pf.pf_status_read(s.status)
    changed = (s.k != before).any(-1)
    mine = sorted(int(s.slot(b, start[b] + i)) for b in range(3) for i in range(rows[b]))
    assert not changed[:-1].any() and changed[-1].any(0).nonzero().flatten().tolist() == mine
    v = qkv[:, (nq + nkv) * hd:].reshape(s.n_rows, nkv, hd)
    for b in range(3):
        i = torch.from_numpy(np.asarray(s.slot(b, start[b] + np.arange(rows[b])), np.int64)).cuda()
        assert torch.equal(s.v[-1][:, i], v[s.begin[b]:s.begin[b + 1]].transpose(0, 1).bfloat16())
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)
    tokens = ints(np.arange(s.n_rows))
    ids = np.full(s.n_rows, -5, np.int32)
    last = rows[0] - 1  # the way to the last node is accepted
    way = [i for i in range(rows[0]) if R.ancestors(s.parents[0])[last, i]]
    for i, j in zip(way, way[1:]):
        ids[i] = j
    path, count, after = (torch.full((m,), 9, dtype=torch.int32, device="cuda") for m in (s.n_rows, 3, 3))
    old = s.k[:, :, torch.from_numpy(np.asarray(s.slot(0, start[0] + np.array(way)), np.int64)).cuda()].clone()
    pf.pf_op_tree_accept(s.cfg, s.batch, tokens, ints(ids), ints([way[0], -7, -7]), path, count, after, s.k, s.v, s.status)
    pf.pf_status_read(s.status)
    assert path[:len(way)].tolist() == way and count.tolist() == [len(way), 0, 0]
    new = s.k[:, :, torch.from_numpy(np.asarray(s.slot(0, start[0] + np.arange(len(way))), np.int64)).cuda()]
    assert torch.equal(new, old)


def test_captured_append_accept_and_adapters():
    """The three other calls captured once and replayed with other rows, starts, trees, tokens and adapters."""
    rng = np.random.default_rng(40)
    rows, start = [30, 5, 12], [100, 0, 250]
    s = Step("f16", 8, 2, 64, rows, start, True, trees(rng, rows), n_layers=2)
    for c in (s.k, s.v):
        c.copy_(torch.from_numpy(rng.standard_normal(c.shape)).cuda())
    width = 12 * 64
    qkv = torch.from_numpy(rng.standard_normal((s.n_rows, width))).cuda().float()
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, 64, s.max_seq)).cuda()
    tokens, ids, root, which = ints(rng.integers(0, 3, s.n_rows)), ints(rng.integers(0, 3, s.n_rows)), ints(rng.integers(0, 3, 3)), ints([1, -1, 0])
    x = torch.from_numpy(rng.standard_normal((s.n_rows, 512))).cuda().half()
    a, b = torch.from_numpy(rng.standard_normal((2, 32, 512)) * 0.04).cuda().half(), torch.from_numpy(rng.standard_normal((2, width, 32))).cuda().half()
    scale = torch.tensor([1.0, 0.5], device="cuda")

    def step(o):
        pf.pf_op_adapters(s.batch, x, qkv, o["y"], which, a, b, scale, s.status)
        pf.pf_op_batch_append(s.cfg, s.batch, o["y"], None, None, rope, 1, o["q"], o["k"], o["v"], s.status)
        pf.pf_op_tree_accept(s.cfg, s.batch, tokens, ids, root, o["path"], o["count"], o["next"], o["k"], o["v"], s.status)

    def outputs():
        i32 = dict(dtype=torch.int32, device="cuda")
        return {"y": torch.full((s.n_rows, width), 7.0, device="cuda"), "q": torch.full((s.n_rows, 8, 64), 7.0, dtype=torch.float16, device="cuda"),
                "k": s.k.clone(), "v": s.v.clone(), "path": torch.full((s.n_rows,), 9, **i32), "count": torch.full((3,), 9, **i32),
                "next": torch.full((3,), 9, **i32)}

    step(outputs())
    o = outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o)
    for change in range(4):
        if change:
            s.rows = [int(r) for r in rng.integers(0, 31, 3)]
            s.begin = np.concatenate([[0], np.cumsum(s.rows)])
            if s.begin[-1] > s.n_rows:
                s.rows, s.begin = [10, 0, 3], np.array([0, 10, 10, 13])
            s.begin_dev.copy_(ints(s.begin))
            s.start_dev.copy_(ints([int(rng.integers(0, p + r - n + 1)) for p, r, n in zip(start, rows, [min(n, r) for n, r in zip(s.rows, rows)])]))
            s.parent_dev[:int(s.begin[-1])] = ints(np.concatenate(trees(rng, s.rows)))
            tokens.copy_(ints(rng.integers(0, 2, s.n_rows)))
            ids.copy_(ints(rng.integers(0, 2, s.n_rows)))
            which.copy_(ints(rng.integers(-1, 2, 3)))
        want = outputs()
        step(want)
        for name, t in outputs().items():
            o[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for name in o:
            assert torch.equal(o[name].contiguous().view(torch.uint8), want[name].contiguous().view(torch.uint8)), (change, name)


def test_first_calls_are_captured():
    """A process whose first calls of all are captured into a graph."""
    code = """
import numpy as np, torch, dataclasses
from quantized_transformer_prefill_q1_gb300 import pf, synth
shape = dataclasses.replace(synth.QWEN3_8B_LAYER, n_q_heads=8, n_kv_heads=2, head_dim=64, kv_dtype="f16")
cfg = pf.make_config(shape, 256, n_layers=1, max_seq=500, kv_block_pool=8)
i = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
torch.manual_seed(0)
b = pf.Batch(i([0, 9, 12]), n_rows=12, max_rows=9, start=i([300, 40]), blocks=i([[0, 1, 2, -1], [5, -1, -1, -1]]))
one = pf.Batch(i([0, 1, 2]), n_rows=12, max_rows=1, start=i([300, 40]), blocks=i([[0, 1, 2, -1], [5, -1, -1, -1]]))
k, v = (torch.randn(1, 2, 1024, 64, device="cuda").half() for _ in "kv")
q, x = torch.randn(12, 8, 64, device="cuda").half(), torch.randn(12, 256, device="cuda").half()
out, few = (torch.zeros(12, 512, dtype=torch.float16, device="cuda") for _ in "ab")
a, w, y = torch.randn(1, 16, 256, device="cuda").half(), torch.randn(1, 64, 16, device="cuda").half(), torch.zeros(12, 64, device="cuda")
scratch, base, which, scale = pf.attention_tree_scratch(cfg, 2, 9), torch.zeros(12, 64, device="cuda"), i([0, -1]), torch.ones(1, device="cuda")
def step():
    pf.pf_op_attention_tree(cfg, b, q, k, v, 0, out, scratch)
    pf.pf_op_attention_tree(cfg, one, q, k, v, 0, few, scratch)
    pf.pf_op_adapters(b, x, base, y, which, a, w, scale)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (out, few, y)]
for t in (out, few, y): t.zero_()
step()
assert all(torch.equal(s, t) and t.any() for s, t in zip(got, (out, few, y)))
print("alike")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "alike" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ acceptance
@pytest.mark.parametrize("kind,hd,paged", [("bf16", 128, True), ("f16", 64, True), ("f16", 128, False)])
@pytest.mark.parametrize("tree", [True, False])
def test_accept(kind, hd, paged, tree):
    rng = np.random.default_rng(hd)
    rows, start = ([1, 26, 0, 256, 61, 40], [5, 120, 3, 0, 127, 300]) if paged else ([33], [100])
    s = Step(kind, 4, 2, hd, rows, start, paged, trees(rng, rows) if tree else None, n_layers=3)
    for c in (s.k, s.v):
        c.copy_(torch.from_numpy(rng.standard_normal(c.shape)).cuda())
    before = s.k.clone(), s.v.clone()
    tokens = rng.integers(0, 4, s.n_rows).astype(np.int32)  # few tokens: several children fit
    ids = rng.integers(0, 4, s.n_rows).astype(np.int32)
    root = rng.integers(0, 4, len(rows)).astype(np.int32)
    for b, n in enumerate(rows):
        if n:
            root[b] = tokens[s.begin[b]]
        for i in range(n):  # most ids lead on
            kids = [j for j in range(n) if s.parents[b][j] == i]
            if kids and rng.random() < 0.95:
                ids[s.begin[b] + i] = tokens[s.begin[b] + kids[rng.integers(len(kids))]]
    path, count, after = (torch.full((m,), 99, dtype=torch.int32, device="cuda") for m in (s.n_rows, len(rows), len(rows)))
    pf.pf_op_tree_accept(s.cfg, s.batch, ints(tokens), ints(ids), ints(root), path, count, after, s.k, s.v, s.status)
    pf.pf_status_read(s.status)
    longest = 0
    for b, n in enumerate(rows):
        at = s.begin[b]
        want, follow = R.accept(s.parents[b], tokens[at:at + n], ids[at:at + n], root[b])
        assert path[at:at + n].tolist() == want + [-1] * (n - len(want))
        assert int(count[b]) == len(want) and int(after[b]) == follow
        longest = max(longest, len(want))
        if want:
            src = torch.from_numpy(np.asarray(s.slot(b, start[b] + np.array(want)), np.int64)).cuda()
            dst = torch.from_numpy(np.asarray(s.slot(b, start[b] + np.arange(len(want))), np.int64)).cuda()
            for old, now in zip(before, (s.k, s.v)):
                moved = old[:, :, src].clone()
                old[:, :, dst] = moved
    assert longest > 2  # the inputs lead on
    assert (path[s.total:] == 99).all()
    for old, now in zip(before, (s.k, s.v)):
        assert torch.equal(old, now)
    # without caches: the same answer, nothing moved
    p2, c2, a2 = (torch.full_like(t, 98) for t in (path, count, after))
    pf.pf_op_tree_accept(s.cfg, s.batch, ints(tokens), ints(ids), ints(root), p2, c2, a2, status=s.status)
    assert torch.equal(p2[:s.total], path[:s.total]) and torch.equal(c2, count) and torch.equal(a2, after)
    assert torch.equal(before[0], s.k)


# ------------------------------------------------------------------ adapters
@pytest.mark.parametrize("k,n,rank", [(256, 128, 8), (4096, 512, 16), (272, 1000, 24), (1040, 264, 64), (512, 2056, 128), (16, 8, 8)])
@pytest.mark.parametrize("top", [1, 5, 70, 300])
def test_adapters(k, n, rank, top):
    rng = np.random.default_rng(k + top)
    rows = [top, 0, 1, max(1, top - 1), top, max(1, top // 3), 2 if top > 1 else 1]
    which = np.array([1, 0, 2, -1, 1, 0, 3], np.int32)
    begin = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    total, n_rows = int(begin[-1]), int(begin[-1]) + 2
    batch = pf.Batch(ints(begin), n_rows=n_rows, max_rows=top if top > 1 else 1)
    x = torch.from_numpy(rng.standard_normal((n_rows, k + 8))).cuda().half()[:, :k]
    base = torch.from_numpy(rng.standard_normal((n_rows, n + 8))).cuda().float()[:, 4:n + 4]
    a = torch.from_numpy(rng.standard_normal((4, rank, k)) * k ** -0.5).cuda().half()
    b = torch.from_numpy(rng.standard_normal((4, n, rank)) * 0.1).cuda().half()
    scale = torch.tensor([0.5, 2.0, 1.25, 16.0], device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.full((n_rows, n), 7.0, device="cuda")
    pf.pf_op_adapters(batch, x, base, out, ints(which), a, b, scale, status)
    pf.pf_status_read(status)
    got = out.double().cpu().numpy()
    for i, w in enumerate(which):
        rs = slice(begin[i], begin[i + 1])
        bs = base[rs].cpu().numpy()
        if w < 0:
            assert np.array_equal(got[rs], bs.astype(np.float64))
            continue
        ref, bound = R.adapters(bs, x[rs].cpu().numpy(), a[w].cpu().numpy(), b[w].cpu().numpy(), float(scale[w]))
        off = np.abs(got[rs] - ref)
        assert (off <= bound).all(), (i, w, float((off / bound).max()))
    assert (got[total:] == 7).all()
    # in place over a block of wider rows: the same numbers, the columns beside it untouched
    wide = torch.full((n_rows, n + 24), 3.0, device="cuda")
    block = wide[:, 8:n + 8]
    block.copy_(base)
    pf.pf_op_adapters(batch, x, block, block, ints(which), a, b, scale, status)
    assert torch.equal(block[:total], out[:total]) and torch.equal(block[total:], base[total:])
    assert (wide[:, :8] == 3).all() and (wide[:, n + 8:] == 3).all()


@pytest.mark.parametrize("k,n,rank", [(512, 264, 16), (768, 520, 72), (1040, 128, 40)])
@pytest.mark.parametrize("n_seq,top", [(40, 45), (300, 3), (3, 200), (70, 17)])
def test_adapters_many_sequences(k, n, rank, n_seq, top):
    """Tiles of 16 and of 64 rows, with sequences of no rows and without an adapter between the others."""
    rng = np.random.default_rng(k + n_seq)
    rows = [int(x) for x in rng.integers(0, top + 1, n_seq)]
    rows[-1] = top
    which = rng.integers(-1, 5, n_seq).astype(np.int32)
    begin = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    total = int(begin[-1])
    batch = pf.Batch(ints(begin), n_rows=total + 1, max_rows=top)
    x = torch.from_numpy(rng.standard_normal((total + 1, k))).cuda().half()
    base = torch.from_numpy(rng.standard_normal((total + 1, n))).cuda().float()
    a = torch.from_numpy(rng.standard_normal((5, rank, k)) * k ** -0.5).cuda().half()
    b = torch.from_numpy(rng.standard_normal((5, n, rank)) * 0.1).cuda().half()
    scale = torch.tensor([0.5, 2.0, 1.25, 16.0, 0.0], device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.full((total + 1, n), 7.0, device="cuda")
    pf.pf_op_adapters(batch, x, base, out, ints(which), a, b, scale, status)
    pf.pf_status_read(status)
    got = out.double().cpu().numpy()
    for i, w in enumerate(which):
        rs = slice(begin[i], begin[i + 1])
        if w < 0:
            assert torch.equal(out[rs], base[rs])
            continue
        ref, bound = R.adapters(base[rs].cpu().numpy(), x[rs].cpu().numpy(), a[w].cpu().numpy(), b[w].cpu().numpy(), float(scale[w]))
        off = np.abs(got[rs] - ref)
        assert (off <= bound).all(), (i, w, float((off - bound).max()))
    assert (got[total] == 7).all()


def test_adapters_range():
    """Rows of 60,000s and of 1e-6: x A^T far beyond and below what an f16 holds."""
    rng = np.random.default_rng(2)
    k, n, rank = 2048, 256, 16
    x = torch.ones(3, k, dtype=torch.float16, device="cuda") * torch.tensor([[60000.0], [1.0], [6e-8]], device="cuda").half()
    a = torch.from_numpy(rng.standard_normal((1, rank, k)) * 8).cuda().half()
    b = torch.from_numpy(rng.standard_normal((1, n, rank))).cuda().half()
    scale, base = torch.ones(1, device="cuda"), torch.zeros(3, n, device="cuda")
    out = torch.empty_like(base)
    batch = pf.Batch(ints([0, 3]), n_rows=3, max_rows=3)
    pf.pf_op_adapters(batch, x, base, out, ints([0]), a, b, scale)
    ref, bound = R.adapters(base.cpu().numpy(), x.cpu().numpy(), a[0].cpu().numpy(), b[0].cpu().numpy(), 1.0)
    off = np.abs(out.double().cpu().numpy() - ref)
    assert (off <= bound).all(), float((off / bound).max())


# ------------------------------------------------------------------ numbers out of range
def status_of(f):
    with pytest.raises(pf.PfError) as e:
        f()
    return pf.STATUS[e.value.status]


@pytest.mark.parametrize("top", [2, 40])
def test_left_out_sequences(top):
    """A sequence with impossible rows or start is recorded and left out; the others are as without it."""
    rng = np.random.default_rng(4)
    rows, start = [top, 1, top], [130, 60, 20]
    for what, code in (("rows", "PF_ERR_SHAPE"), ("start", "PF_ERR_KV_CAPACITY"), ("negative", "PF_ERR_KV_CAPACITY"), ("far", "PF_ERR_KV_CAPACITY")):
        s = Step("f16", 8, 2, 128, rows, start, True, trees(rng, rows))
        s.fill()
        q = s.q()
        good = s.attend(q)
        kc = s.k.clone()
        if what == "rows":
            s.begin_dev.copy_(ints([0, top, top - 1, 2 * top + 1]))  # the second falls; the third overlaps it and has too many
        else:
            s.start_dev[1] = {"start": s.max_seq, "negative": -1, "far": 2 ** 31 - 1}[what]
        out = s.attend(q)
        torch.cuda.synchronize()
        assert status_of(lambda: pf.pf_status_read(s.status)) == code
        assert torch.equal(out[:top], good[:top])
        if what != "rows":
            assert (out[top] == 7).all() and torch.equal(out[top + 1:], good[top + 1:])
        else:
            assert (out[top:] == 7).all()
        # append and accept leave it out too
        qkv = torch.randn(s.n_rows, 12 * 128, device="cuda")
        rope = torch.from_numpy(pf.pf_rope_table_host(1e6, 128, s.max_seq)).cuda()
        q2 = torch.full_like(q, 7.0)
        pf.pf_op_batch_append(s.cfg, s.batch, qkv, None, None, rope, 0, q2, s.k, s.v, s.status)
        assert status_of(lambda: pf.pf_status_read(s.status)) == code
        assert (q2[top] == 7).all() and not (q2[:top] == 7).any()
        assert torch.equal(s.k[1].view(torch.int16), kc[1].view(torch.int16))
        path, count, after = (torch.full((m,), 99, dtype=torch.int32, device="cuda") for m in (s.n_rows, 3, 3))
        one = torch.ones(s.n_rows, dtype=torch.int32, device="cuda")
        pf.pf_op_tree_accept(s.cfg, s.batch, one, one, ints([1, 5, 1]), path, count, after, s.k, s.v, s.status)
        assert status_of(lambda: pf.pf_status_read(s.status)) == code
        assert count[1] == 0 and after[1] == 5 and path[top] == 99


@pytest.mark.parametrize("top", [2, 40])
def test_bad_parents_and_pages(top):
    rng = np.random.default_rng(4)
    rows, start = [top, 1, top], [130, 60, 20]
    s = Step("f16", 8, 2, 128, rows, start, True, trees(rng, rows))
    s.fill()
    q = s.q()
    # a parent that is no earlier node is the cache
    for bad in (top - 1, top, -2, 2 ** 31 - 1, -2 ** 31):
        p = [x.copy() for x in s.parents]
        p[0][top - 1] = -1
        s.parent_dev[:s.total] = ints(np.concatenate(p))
        want = s.attend(q)
        pf.pf_status_read(s.status)
        s.parent_dev[top - 1] = bad
        got = s.attend(q)
        assert status_of(lambda: pf.pf_status_read(s.status)) == "PF_ERR_INVALID_ARG"
        assert torch.equal(got, want)
    s.parent_dev[:s.total] = ints(np.concatenate(s.parents))
    # a page outside the pool: not written, read as any block, the other sequences unharmed
    want = s.attend(q)
    pf.pf_status_read(s.status)
    for bad in (-1, s.pool, 2 ** 31 - 1, -2 ** 31):
        s.table_dev[0, 1] = bad
        got = s.attend(q)
        assert status_of(lambda: pf.pf_status_read(s.status)) == "PF_ERR_KV_CAPACITY"
        assert torch.equal(got[top:], want[top:])
        before = s.k.clone()
        qkv = torch.randn(s.n_rows, 12 * 128, device="cuda")
        rope = torch.from_numpy(pf.pf_rope_table_host(1e6, 128, s.max_seq)).cuda()
        pf.pf_op_batch_append(s.cfg, s.batch, qkv, None, None, rope, 0, torch.empty_like(q), s.k, s.v, s.status)
        assert status_of(lambda: pf.pf_status_read(s.status)) == "PF_ERR_KV_CAPACITY"
        changed = (s.k.view(torch.int16) != before.view(torch.int16)).any(-1)
        mine = {int(s.slot(b, start[b] + i)) for b in (1, 2) for i in range(rows[b])}
        assert not changed[1].any() and {int(x) for x in changed[0].nonzero()[:, 1]} <= mine


def test_accept_with_a_bad_page():
    """Rows whose block is unknown stay where they are; the answer and the other rows are as with it."""
    s = Step("f16", 4, 2, 64, [4, 3], [126, 20], True, [np.array([-1, -1, 1, 2], np.int32), np.array([-1, -1, 1], np.int32)], n_layers=1, layer=0)
    for c in (s.k, s.v):
        c.copy_(torch.randn(c.shape, device="cuda"))
    tokens, ids = ints([9, 1, 2, 3, 9, 1, 2, 0, 0, 0]), ints([0, 2, 3, 4, 0, 2, 8, 0, 0, 0])
    before = s.k.clone()
    s.table_dev[0, 1] = s.pool  # positions 128 .. of the first: nodes 2 and 3
    path, count, after = (torch.full((m,), 99, dtype=torch.int32, device="cuda") for m in (s.n_rows, 2, 2))
    pf.pf_op_tree_accept(s.cfg, s.batch, tokens, ids, ints([1, 1]), path, count, after, s.k, s.v, s.status)
    assert status_of(lambda: pf.pf_status_read(s.status)) == "PF_ERR_KV_CAPACITY"
    assert path.tolist() == [1, 2, 3, -1, 1, 2, -1, 99, 99, 99] and count.tolist() == [3, 2] and after.tolist() == [4, 8]
    want = before.clone()
    want[:, :, int(s.slot(0, 126))] = before[:, :, int(s.slot(0, 127))]  # node 1 to place 0: both known
    for j in (0, 1):
        want[:, :, int(s.slot(1, 20 + j))] = before[:, :, int(s.slot(1, 21 + j))]
    assert torch.equal(s.k, want)


def test_binding_refusals():
    """Tensors of another type, place, width or layout, and scratches too small, are refused before a launch."""
    s = Step("f16", 4, 2, 64, [3, 1], [5, 200], True)
    s.fill()
    q, out, scratch = s.q(), torch.zeros(s.n_rows, 256, dtype=torch.float16, device="cuda"), s.scratch()

    def attend(q=q, k=s.k, v=s.v, out=out, scratch=scratch, batch=s.batch):
        pf.pf_op_attention_tree(s.cfg, batch, q, k, v, 1, out, scratch, s.status)

    attend()
    narrow = pf.Batch(s.begin_dev, n_rows=s.n_rows, max_rows=3, start=s.start_dev, blocks=s.table_dev[:, :1].contiguous())
    bare = pf.Batch(s.begin_dev, n_rows=s.n_rows, max_rows=3, start=s.start_dev)
    for kw in (dict(q=q.bfloat16()), dict(q=q[:2]), dict(q=q.cpu()), dict(q=None), dict(k=s.k.float()), dict(v=s.v[:1]), dict(out=out.float()),
               dict(out=out[:, ::2]), dict(out=q), dict(scratch=scratch.cpu()), dict(batch=narrow), dict(batch=bare)):
        assert status_of(lambda: attend(**kw)) == "PF_ERR_INVALID_ARG", kw.keys()
    assert status_of(lambda: attend(scratch=scratch[:64])) == "PF_ERR_WORKSPACE"
    for blocks in (s.table_dev.long(), s.table_dev[0], s.table_dev[:1], s.table_dev.cpu()):
        assert status_of(lambda: pf.Batch(s.begin_dev, n_rows=s.n_rows, max_rows=3, start=s.start_dev, blocks=blocks)) == "PF_ERR_INVALID_ARG"
    x, y = torch.zeros(s.n_rows, 64, dtype=torch.float16, device="cuda"), torch.zeros(s.n_rows, 32, device="cuda")
    a, b = torch.zeros(2, 8, 64, dtype=torch.float16, device="cuda"), torch.zeros(2, 32, 8, dtype=torch.float16, device="cuda")

    def adapters(x=x, base=y, out=torch.zeros_like(y), adapter=ints([0, 1]), a=a, b=b, scale=torch.ones(2, device="cuda")):
        pf.pf_op_adapters(s.batch, x, base, out, adapter, a, b, scale, s.status)

    adapters()
    for kw in (dict(x=x.float()), dict(x=x[:, :48]), dict(x=x[:2]), dict(x=x.t().contiguous().t()), dict(x=x.cpu()), dict(base=y.half()), dict(base=None),
               dict(out=y[:, :16]), dict(out=y[0]), dict(adapter=ints([0])), dict(adapter=ints([0, 1]).long()), dict(a=a[0]), dict(a=a[:1]), dict(a=a.float()),
               dict(b=b[:, :, :4]), dict(b=b.transpose(1, 2)), dict(scale=torch.ones(1, device="cuda")), dict(scale=None)):
        assert status_of(lambda: adapters(**kw)) == "PF_ERR_INVALID_ARG", kw.keys()
    assert status_of(lambda: adapters(base=y[:1].expand(s.n_rows, 32))) == "PF_ERR_SHAPE"  # one row for all: rows 0 apart
    wide = torch.zeros(s.n_rows, 48, device="cuda")
    assert status_of(lambda: adapters(base=wide[:, :32], out=wide.reshape(-1)[:s.n_rows * 32].reshape(s.n_rows, 32))) == "PF_ERR_SHAPE"
    pf.pf_status_read(s.status)


def test_bad_adapters():
    batch = pf.Batch(ints([0, 2, 3]), n_rows=3, max_rows=2)
    x, base = torch.randn(3, 64, device="cuda").half(), torch.randn(3, 32, device="cuda")
    a, b = torch.randn(2, 8, 64, device="cuda").half(), torch.randn(2, 32, 8, device="cuda").half()
    scale, status = torch.ones(2, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (2, -2, 2 ** 31 - 1, -2 ** 31):
        out = torch.full_like(base, 7.0)
        pf.pf_op_adapters(batch, x, base, out, ints([bad, 1]), a, b, scale, status)
        assert status_of(lambda: pf.pf_status_read(status)) == "PF_ERR_INVALID_ARG"
        assert torch.equal(out[:2], base[:2]) and not torch.equal(out[2], base[2])


# ------------------------------------------------------------------ together
def test_layer_of_several_requests():
    """What a layer's attention block does for five requests with trees and adapters: projection, adapters, append, attention,
    output projection with the residual and its adapters; then the accepted paths move up and the next step reads them."""
    rng = np.random.default_rng(17)
    shape = dataclasses.replace(synth.QWEN3_8B_LAYER, hidden=512, intermediate=512, n_q_heads=8, n_kv_heads=2, head_dim=64, kv_dtype="f16")
    nq, nkv, hd, h = 8, 2, 64, 512
    rows, start = [7, 1, 30, 12, 20], [0, 200, 127, 60, 310]
    s = Step("f16", nq, nkv, hd, rows, start, True, trees(rng, rows), norm=True, n_layers=1, layer=0, spare=0)
    s.fill(own_rows=False)
    width = (nq + 2 * nkv) * hd
    w = {name: synth.q1_weight(rng, n, k) for name, n, k in (("qkv", width, h), ("o", h, nq * hd))}
    dense = {}
    packed = {}
    for name, t in w.items():
        sign = np.unpackbits(t["bits"], axis=1, bitorder="little").astype(np.float64) * 2 - 1
        dense[name] = sign * np.repeat(t["scales"].astype(np.float64), 128, 1)
        packed[name] = torch.from_numpy(pf.pf_pack_weights_host(t)).cuda()
    x = torch.from_numpy(rng.standard_normal((s.total, h))).cuda().float()
    norm_w = torch.ones(h, device="cuda")
    qn, kn = (1 + 0.1 * rng.standard_normal((2, hd))).astype(np.float32)
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, hd, s.max_seq)).cuda()
    which = np.array([0, -1, 1, 0, 1], np.int32)
    ad = {name: (torch.from_numpy(rng.standard_normal((2, 16, k)) * k ** -0.5).cuda().half(), torch.from_numpy(rng.standard_normal((2, n, 16)) * 0.3).cuda().half())
          for name, n, k in (("q", nq * hd, h), ("v", nkv * hd, h), ("o", h, nq * hd))}
    scale = torch.tensor([1.0, 2.0], device="cuda")
    y, qkv = torch.empty(s.total, h, dtype=torch.float16, device="cuda"), torch.empty(s.total, width, device="cuda")
    q, attn = torch.empty(s.total, nq, hd, dtype=torch.float16, device="cuda"), torch.empty(s.total, nq * hd, dtype=torch.float16, device="cuda")
    out, qn_dev, kn_dev = x.clone(), torch.from_numpy(qn).cuda(), torch.from_numpy(kn).cuda()
    gs = pf.gemm_scratch(s.total, max(width, h))
    scratch, which_dev = s.scratch(), ints(which)

    def step():
        pf.pf_op_rmsnorm(x, norm_w, 1e-6, y)
        pf.pf_op_gemm(pf.W_Q1, pf.EPI_STORE_F32, y, packed["qkv"], s.total, width, h, qkv, gs, status=s.status)
        for name, lo, hi in (("q", 0, nq * hd), ("v", (nq + nkv) * hd, width)):
            pf.pf_op_adapters(s.batch, y, qkv[:, lo:hi], qkv[:, lo:hi], which_dev, *ad[name], scale, s.status)
        pf.pf_op_batch_append(s.cfg, s.batch, qkv, qn_dev, kn_dev, rope, 0, q, s.k, s.v, s.status)
        pf.pf_op_attention_tree(s.cfg, s.batch, q, s.k, s.v, 0, attn, scratch, s.status)
        pf.pf_op_gemm(pf.W_Q1, pf.EPI_RESID_ADD, attn, packed["o"], s.total, h, nq * hd, out, gs, status=s.status)
        pf.pf_op_adapters(s.batch, attn, out, out, which_dev, *ad["o"], scale, s.status)

    step()
    pf.pf_status_read(s.status)

    def lora(name, i, v):
        a, b = (t[i].double().cpu().numpy() for t in ad[name])
        return float(scale[i]) * (v @ a.T) @ b.T

    xn = x.double().cpu().numpy()
    ref = np.empty((s.total, h))
    kv = {}
    for b, n in enumerate(rows):
        xr = xn[s.begin[b]:s.begin[b + 1]]
        yr = xr / np.sqrt((xr * xr).mean(1, keepdims=True) + 1e-6)
        p = yr @ dense["qkv"].T
        if which[b] >= 0:
            p[:, :nq * hd] += lora("q", which[b], yr)
            p[:, (nq + nkv) * hd:] += lora("v", which[b], yr)
        rq, rk, rv, _ = R.append(p, nq, nkv, hd, qn, kn, s.cfg.eps, s.cfg.rope_theta, start[b] + R.depths(s.parents[b]))
        k, v = s.held(s.k, b), s.held(s.v, b)
        k[:, start[b]:], v[:, start[b]:] = rk.transpose(1, 0, 2), rv.transpose(1, 0, 2)
        kv[b] = k, v
        o = R.attention(rq, k, v, start[b], s.parents[b], R.half_step("f16"))[0].reshape(n, nq * hd)
        r = xr + o @ dense["o"].T
        ref[s.begin[b]:s.begin[b + 1]] = r + (lora("o", which[b], o) if which[b] >= 0 else 0)
    got = out.double().cpu().numpy()
    off = np.linalg.norm(got - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert off.max() < 5e-3, off  # f16 operands throughout: about ten roundings of 2^-11

    # the whole step captured and replayed
    out.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.copy_(x)
    graph.replay()
    pf.pf_status_read(s.status)
    got2 = out.double().cpu().numpy()
    assert (np.linalg.norm(got2 - ref, axis=1) / np.linalg.norm(ref, axis=1)).max() < 5e-3

    # acceptance, then one more token on the accepted positions
    tokens = rng.integers(0, 50, s.total).astype(np.int32)
    ids = rng.integers(0, 50, s.total).astype(np.int32)
    root = np.array([tokens[s.begin[b]] for b in range(5)], np.int32)
    for b, n in enumerate(rows):
        for i in range(n):
            kids = [j for j in range(n) if s.parents[b][j] == i]
            if kids:
                ids[s.begin[b] + i] = tokens[s.begin[b] + kids[-1]]
    path, count, after = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (s.total, 5, 5))
    pf.pf_op_tree_accept(s.cfg, s.batch, ints(tokens), ints(ids), ints(root), path, count, after, s.k, s.v, s.status)
    new_start = s.start_dev + count
    one = pf.Batch(ints(np.arange(6)), n_rows=5, max_rows=1, start=new_start - 1, blocks=s.table_dev)  # each path's last node again
    q1 = torch.stack([q[s.begin[b] + int(path[s.begin[b] + int(count[b]) - 1])] for b in range(5)])
    o1 = torch.empty(5, nq * hd, dtype=torch.float16, device="cuda")
    pf.pf_op_attention_tree(s.cfg, one, q1, s.k, s.v, 0, o1, pf.attention_tree_scratch(s.cfg, 5, 1), s.status)
    pf.pf_status_read(s.status)
    for b in range(5):
        node = int(path[s.begin[b] + int(count[b]) - 1])
        d = (o1[b].double() - attn[s.begin[b] + node].double()).abs().max()
        assert float(d) <= 2.0 ** -9 * float(attn[s.begin[b] + node].double().abs().max()), (b, float(d))
