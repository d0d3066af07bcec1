"""Calls over many sequences on the GPU where a value that is not finite, a small weight, a shared scratch or a replay
could go wrong without an error."""
import numpy as np
import pytest

import batch_reference as R
from quantized_transformer_prefill_q1_gb300 import pf
from test_gpu_batch import Step, ints, torch, trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nkv,hd", [(32, 8, 128), (8, 8, 64), (16, 1, 128)])
@pytest.mark.parametrize("rows", [[1], [26], [40], [1, 1, 1, 1], [26, 1, 40, 26], [200, 30, 1, 7]])
def test_nan_pages(kind, nq, nkv, hd, rows):
    """Cached K of NaN over so many pages that whole parts of a cut task see nothing else: every row of the sequence is NaN,
    the other sequences are as without it."""
    rng = np.random.default_rng(len(rows) + rows[0])
    s = Step(kind, nq, nkv, hd, rows, [8189, 7800, 8000, 7900][:len(rows)], True, trees(rng, rows), n_layers=1, layer=0)
    s.fill()
    q, scratch = s.q(), s.scratch()
    want = s.attend(q, scratch)
    for first, last in ((0, 50), (8, 60)):  # pages
        keep = s.k.clone()
        i = torch.from_numpy(np.asarray(s.slot(0, np.arange(128 * first, 128 * last)), np.int64)).cuda()
        s.k[:, :, i] = float("nan")
        got = s.attend(q, scratch)
        assert torch.isnan(got[:rows[0]]).all(), (first, last, int((~torch.isnan(got[:rows[0]])).sum()))
        assert torch.equal(got[rows[0]:], want[rows[0]:])
        s.k.copy_(keep)
    assert torch.equal(s.attend(q, scratch), want)
    pf.pf_status_read(s.status)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nkv,hd,n", [(8, 2, 128, 2), (8, 2, 128, 26), (8, 8, 64, 26), (16, 1, 128, 26)])
def test_nan_value_of_a_small_weight(kind, nq, nkv, hd, n):
    """A NaN in the V of a cached position reaches every row, also where its weight is e^-200 of the largest."""
    s = Step(kind, nq, nkv, hd, [n, 1], [130, 0], True, [R.chain(n), R.chain(1)], n_layers=1, layer=0)
    s.fill()
    first = torch.from_numpy(np.asarray(s.slot(0, np.arange(128)), np.int64)).cuda()
    s.k[0, :, :, 0] = 0
    s.k[0][:, first, 0] = 20.0
    q = s.q()
    q[:, :, 0] = 20.0 * hd ** 0.5
    want = s.attend(q)
    s.check_attention(q, want)
    s.v[0, :, int(s.slot(0, 128)), 5] = float("nan")
    got = s.attend(q).reshape(-1, nq, hd)
    assert torch.isnan(got[:n, :, 5]).all()
    got[:n, :, 5] = want.reshape(-1, nq, hd)[:n, :, 5]
    assert torch.equal(got.reshape(want.shape), want)
    pf.pf_status_read(s.status)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nkv,hd,n", [(8, 8, 64, 8), (32, 8, 128, 2), (8, 8, 64, 200), (32, 8, 128, 26), (4, 1, 128, 256)])
@pytest.mark.parametrize("others", [0, 3, 40])
def test_hidden_values(kind, nq, nkv, hd, n, others):
    """A NaN or an infinity in the V of a node: its column is NaN in every row of the sequence that does not see it, NaN or
    infinite in those that do, alone and beside other sequences; all else is as without it."""
    parent = np.full(n, -1, np.int32)
    parent[n // 2:] = n // 2 - 1  # half of them hang on one node
    see = R.ancestors(parent)
    rows, start = [n] + [1 + b % min(n, 3) for b in range(others)], [100] + [37 * b % 600 for b in range(others)]
    s = Step(kind, nq, nkv, hd, rows, start, True, [parent] + [R.chain(m) for m in rows[1:]], n_layers=1, layer=0)
    s.fill()
    q, scratch = s.q(), s.scratch()
    want = s.attend(q, scratch)
    s.check_attention(q, want)
    for j in (0, n // 2 - 1, n - 1):
        for bad in (float("nan"), float("inf"), float("-inf")):
            keep = s.v.clone()
            s.v[0, :, int(s.slot(0, 100 + j)), 3] = bad
            got = s.attend(q, scratch).reshape(-1, nq, hd)
            blind = torch.from_numpy(~see[:, j]).cuda()
            assert torch.isnan(got[:n][blind][:, :, 3]).all() and not torch.isfinite(got[:n, :, 3]).any(), (j, bad)
            got[:n, :, 3] = want.reshape(-1, nq, hd)[:n, :, 3]
            assert torch.equal(got.reshape(want.shape), want)
            s.v.copy_(keep)
    pf.pf_status_read(s.status)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("nq,nkv,hd,n", [(8, 8, 64, 1), (8, 2, 128, 2), (8, 8, 64, 26), (8, 2, 128, 40), (16, 1, 128, 30)])
@pytest.mark.parametrize("power", [12.3, 15.7, 20.4, 22.6, 24.3, 25.2, 26.4, 28.0])
def test_small_weights(kind, nq, nkv, hd, n, power):
    """Keys of weight 2^-power with values of one sign beside one key of weight 1 and value 0 in every 32: the small ones are all
    there is. A weight that an f16 holds is off by half a step or, below 2^-21 of the row's running maximum, by 2^-32 of it:
    the numbers are formed 2^7 larger, and the smallest step of an f16 is 2^-24."""
    rng = np.random.default_rng(n)
    s = Step(kind, nq, nkv, hd, [n, 1], [2000, 700], True, [R.random_tree(rng, n), R.chain(1)], n_layers=1, layer=0)
    s.fill()
    s.k.copy_(torch.nan_to_num(s.k) * 0)
    s.v.copy_(torch.from_numpy(rng.uniform(500, 1000, s.v.shape)).cuda())
    for b in range(2):
        p = np.arange(s.start[b] + s.rows[b])
        i = torch.from_numpy(np.asarray(s.slot(b, p), np.int64)).cuda()
        large = torch.from_numpy(p % 32 == 0).cuda()
        s.k[0][:, i, 0] = torch.where(large, 0.0, -power * float(np.log(2))).to(s.dt)
        s.v[0][:, i] = torch.where(large[:, None], torch.zeros((), dtype=s.dt, device="cuda"), s.v[0][:, i])
    q = torch.zeros(s.n_rows, nq, hd, dtype=s.dt, device="cuda")
    q[:, :, 0] = hd ** 0.5  # 8, or the type's nearest to 11.3
    out = s.attend(q)
    pf.pf_status_read(s.status)
    got, qq = out.double().cpu().numpy().reshape(-1, nq, hd), q.double().cpu().numpy()
    for b, m in enumerate(s.rows):
        at = slice(s.begin[b], s.begin[b + 1])
        k, v = s.held(s.k, b), s.held(s.v, b)
        ref, bound = R.attention(qq[at], k, v, s.start[b], s.parents[b], s.weights())
        if kind == "f16":  # a step of 2^-31 of the running maximum, which is at most the true one
            score = np.einsum("nh,hk->nhk", qq[at][:, :, 0], np.repeat(k[:, :, 0], nq // nkv, 0)) / np.sqrt(hd)
            see = np.ones((m, score.shape[2]), bool)
            see[:, s.start[b]:] = R.ancestors(s.parents[b])
            score = np.where(see[:, None], score, -np.inf)
            weight = np.exp(score - score.max(2, keepdims=True)).sum(2)
            values = np.einsum("nk,hkd->nhd", see, np.repeat(np.abs(v), nq // nkv, 0))
            bound = bound + 2.0 ** -32 * values / weight[:, :, None]
        off = np.abs(got[at] - ref)
        assert (off <= bound).all(), (b, float((off / bound).max()), float(got[at].max()), float(ref.max()))


def test_one_scratch_for_other_heads():
    """One scratch for calls with other numbers of kv heads, widths and types in turn, few rows and many, without a zero between."""
    rng = np.random.default_rng(5)
    steps = []
    for kind, nq, nkv, hd, rows, start in (("bf16", 2, 1, 64, [1], [9000]), ("f16", 64, 64, 64, [1] * 40, [200 + 7 * b for b in range(40)]),
                                           ("f16", 8, 2, 128, [30, 4], [3000, 900]), ("bf16", 32, 8, 128, [1, 2, 0, 1], [5000, 100, 3, 40]),
                                           ("bf16", 200, 200, 64, [1, 1], [150, 700])):
        s = Step(kind, nq, nkv, hd, rows, start, True, trees(rng, rows), n_layers=1, layer=0)
        s.fill()
        steps.append((s, s.q()))
    scratch = max((s.scratch() for s, _ in steps), key=len)
    for turn in range(3):
        for s, q in steps if turn < 2 else steps[::-1]:
            out = s.attend(q, scratch)
            pf.pf_status_read(s.status)
            s.check_attention(q, out)


def test_replays_against_the_definition():
    """Append, acceptance and adapters captured once and replayed with other rows, starts, trees, tokens, pages and adapters, all
    of them valid: each replay against float64."""
    rng = np.random.default_rng(41)
    nq, nkv, hd, k, width = 8, 2, 64, 512, 12 * 64
    most, room = [30, 9, 14], [400, 120, 300]  # rows, and positions that fit, of each sequence
    s = Step("f16", nq, nkv, hd, most, [r - m for r, m in zip(room, most)], True, trees(rng, most), norm=True)
    x = torch.from_numpy(rng.standard_normal((s.n_rows, k))).cuda().half()
    a, b = torch.from_numpy(rng.standard_normal((2, 32, k)) * 0.04).cuda().half(), torch.from_numpy(rng.standard_normal((2, width, 32))).cuda().half()
    scale = torch.tensor([1.0, 0.5], device="cuda")
    base = torch.empty(s.n_rows, width, device="cuda")
    qn, kn = (1 + 0.1 * rng.standard_normal((2, hd))).astype(np.float32)
    qn_dev, kn_dev = torch.from_numpy(qn).cuda(), torch.from_numpy(kn).cuda()
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, hd, s.max_seq)).cuda()
    tokens, ids, path, root, which, count, after = (ints(np.zeros(m)) for m in [s.n_rows] * 3 + [3] * 4)
    y, q = torch.empty_like(base), torch.empty(s.n_rows, nq, hd, dtype=torch.float16, device="cuda")
    held = {}

    def step():
        pf.pf_op_adapters(s.batch, x, base, y, which, a, b, scale, s.status)
        pf.pf_op_batch_append(s.cfg, s.batch, y, qn_dev, kn_dev, rope, s.layer, q, s.k, s.v, s.status)
        for name in "kv":  # what the acceptance moves, as it was before
            held[name].copy_(getattr(s, name))
        pf.pf_op_tree_accept(s.cfg, s.batch, tokens, ids, root, path, count, after, s.k, s.v, s.status)

    held.update(k=torch.empty_like(s.k), v=torch.empty_like(s.v))
    s.k.zero_()
    s.v.zero_()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    longest = 0
    for turn in range(6):
        s.rows = [int(rng.integers(0, m + 1)) for m in most]
        s.start = [int(rng.integers(0, r - n + 1)) for r, n in zip(room, s.rows)]
        s.begin = np.concatenate([[0], np.cumsum(s.rows)]).astype(np.int32)
        s.total = int(s.begin[-1])
        s.parents = trees(rng, s.rows)
        for row in s.table:  # the same pages in another order
            mine = row >= 0
            row[mine] = rng.permutation(row[mine])
        s.table_dev.copy_(ints(s.table))
        s.begin_dev.copy_(ints(s.begin))
        s.start_dev.copy_(ints(s.start))
        s.parent_dev[:s.total] = ints(np.concatenate(s.parents))
        t, i, r, w = (rng.integers(lo, hi, m).astype(np.int32) for lo, hi, m in ((0, 2, s.n_rows), (0, 2, s.n_rows), (0, 2, 3), (-1, 2, 3)))
        for to, of in ((tokens, t), (ids, i), (root, r), (which, w)):
            to.copy_(ints(of))
        base.copy_(torch.from_numpy(rng.standard_normal(base.shape)))
        for c, fill in ((y, 7), (q, 7), (path, 9), (count, 9), (after, 9), (s.k, 3), (s.v, 3)):
            c.fill_(fill)
        graph.replay()
        pf.pf_status_read(s.status)
        assert (y[s.total:] == 7).all() and (q[s.total:] == 7).all() and (path[s.total:] == 9).all()
        free = torch.ones(s.slots, dtype=torch.bool, device="cuda")
        moved = {name: held[name].clone() for name in "kv"}
        for n in range(3):
            at, rows = slice(s.begin[n], s.begin[n + 1]), s.rows[n]
            if w[n] < 0:
                assert torch.equal(y[at], base[at])
            else:
                ref, bound = R.adapters(*(z.cpu().numpy() for z in (base[at], x[at], a[w[n]], b[w[n]])), float(scale[w[n]]))
                assert (np.abs(y[at].double().cpu().numpy() - ref) <= bound).all(), (turn, n)
            slot = torch.from_numpy(np.asarray(s.slot(n, s.start[n] + np.arange(rows)), np.int64)).cuda()
            free[slot] = False
            if rows:
                rq, rk, rv, size = R.append(y[at].cpu().numpy(), nq, nkv, hd, qn, kn, s.cfg.eps, s.cfg.rope_theta, s.start[n] + R.depths(s.parents[n]))
                for got, ref, sz in ((q[at], rq, size[:, :nq]), (held["k"][s.layer][:, slot].transpose(0, 1), rk, size[:, nq:])):
                    # half a step of an f16 (2^-25 below its normal range), and the norm and rotation within 16 roundings in f32
                    off = np.abs(got.double().cpu().numpy() - ref)
                    assert (off <= 2.0 ** -11 * (np.abs(ref) + 2.0 ** -20 * sz) + 2.0 ** -20 * sz + 2.0 ** -25).all(), (turn, n)
                assert torch.equal(held["v"][s.layer][:, slot].transpose(0, 1), y[at, (nq + nkv) * hd:].reshape(rows, nkv, hd).half())
            want, follow = R.accept(s.parents[n], t[at], i[at], r[n])
            longest = max(longest, len(want))
            assert path[at].tolist() == want + [-1] * (rows - len(want)) and int(count[n]) == len(want) and int(after[n]) == follow
            for name in "kv":
                moved[name][:, :, slot[:len(want)]] = held[name][:, :, slot[want]]
        for name in "kv":
            assert torch.equal(getattr(s, name), moved[name]) and (held[name][:, :, free] == 3).all()
            assert (held[name][1 - s.layer] == 3).all()
    assert longest > 1


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nkv,hd,rows", [(32, 8, 128, [1, 2, 1, 1, 2]), (8, 2, 64, [20, 1, 33, 7, 12])])
def test_shared_pages(kind, nq, nkv, hd, rows):
    """Sequences that begin with the same pages, those of a prompt that they share: attention reads them, append and acceptance write
    the pages that each has for itself."""
    rng = np.random.default_rng(hd)
    s = Step(kind, nq, nkv, hd, rows, [300, 256, 511, 260, 700], True, trees(rng, rows), norm=False)
    s.table[1:, :2] = s.table[0, :2]  # positions 0 .. 255
    s.table_dev.copy_(ints(s.table))
    s.fill(own_rows=False)
    before = s.k.clone()
    qkv = torch.from_numpy(rng.standard_normal((s.n_rows, (nq + 2 * nkv) * hd))).cuda().float()
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, hd, s.max_seq)).cuda()
    q = torch.empty(s.n_rows, nq, hd, dtype=s.dt, device="cuda")
    pf.pf_op_batch_append(s.cfg, s.batch, qkv, None, None, rope, s.layer, q, s.k, s.v, s.status)
    out = s.attend(q)
    pf.pf_status_read(s.status)
    s.check_attention(q, out)
    shared = torch.from_numpy(np.asarray(s.slot(0, np.arange(256)), np.int64)).cuda()
    tokens = ints(np.arange(s.n_rows))
    way = [int(s.begin[b]) + next(i for i in range(n) if s.parents[b][i] < 0) for b, n in enumerate(rows)]
    path, count, after = (ints(np.zeros(m)) for m in (s.n_rows, len(rows), len(rows)))
    pf.pf_op_tree_accept(s.cfg, s.batch, tokens, ints(np.full(s.n_rows, -5)), ints(way), path, count, after, s.k, s.v, s.status)
    pf.pf_status_read(s.status)
    assert count.tolist() == [1] * len(rows)
    assert torch.equal(s.k[:, :, shared].view(torch.int16), before[:, :, shared].view(torch.int16))


@pytest.mark.parametrize("rows,rank", [([3, 1, 2], 16), ([100, 40, 70], 16), ([700, 300], 64), ([9, 300], 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_adapters_that_are_not_finite(rows, rank, bad):
    """One element of x, base, A or B that is not finite: the results that hold it in the definition are not finite, all others
    are right."""
    rng = np.random.default_rng(rank)
    k, n = 272, 136
    begin = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    x, base = rng.standard_normal((begin[-1], k)).astype(np.float16), rng.standard_normal((begin[-1], n)).astype(np.float32)
    a, b = (rng.standard_normal((2, rank, k)) * k ** -0.5).astype(np.float16), rng.standard_normal((2, n, rank)).astype(np.float16)
    batch, status, scale = pf.Batch(ints(begin), n_rows=int(begin[-1]), max_rows=max(rows)), torch.zeros(4, dtype=torch.int32, device="cuda"), [0.5, 2.0]
    for spoilt in range(4):
        t = [x.copy(), base.copy(), a.copy(), b.copy()]
        t[spoilt][tuple(int(rng.integers(m)) for m in t[spoilt].shape)] = bad
        dev = [torch.from_numpy(y).cuda() for y in t]
        out = torch.full((int(begin[-1]), n), 7.0, device="cuda")
        pf.pf_op_adapters(batch, dev[0], dev[1], out, ints(np.arange(len(rows)) % 2), dev[2], dev[3], torch.tensor(scale, device="cuda"), status)
        pf.pf_status_read(status)
        for i in range(len(rows)):
            at = slice(begin[i], begin[i + 1])
            got = out[at].cpu().numpy()
            with np.errstate(invalid="ignore"):
                ref, bound = R.adapters(t[1][at], t[0][at], t[2][i % 2], t[3][i % 2], scale[i % 2])
            fine = np.isfinite(ref)
            assert (np.isfinite(got) == fine).all() and (np.abs(got[fine] - ref[fine]) <= bound[fine]).all(), (spoilt, i)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("long", [0, 2, 4])
def test_a_long_sequence_in_a_call_of_its_own(kind, long):
    """Batches that point at entries of the same arrays: one sequence, those before it and those behind it."""
    rng = np.random.default_rng(long)
    rows = [1, 2, 1, 1, 2]
    rows[long] = 90
    s = Step(kind, 8, 2, 64, rows, [300, 5, 129, 0, 700], True, trees(rng, rows), n_layers=1, layer=0)
    s.fill(own_rows=False)
    whole = s.batch
    parts = [pf.Batch(s.begin_dev[i:j + 1], n_rows=s.n_rows, max_rows=max(rows[i:j]), start=s.start_dev[i:j], parent=s.parent_dev, blocks=s.table_dev[i:j])
             for i, j in ((0, long), (long, long + 1), (long + 1, 5)) if i < j]
    qkv = torch.from_numpy(rng.standard_normal((s.n_rows, 12 * 64))).cuda().float()
    rope = torch.from_numpy(pf.pf_rope_table_host(s.cfg.rope_theta, 64, s.max_seq)).cuda()
    x = torch.from_numpy(rng.standard_normal((s.n_rows, 256))).cuda().half()
    a, b = torch.from_numpy(rng.standard_normal((1, 16, 256)) / 16).cuda().half(), torch.from_numpy(rng.standard_normal((1, 512, 16))).cuda().half()
    which, one, scratch = ints(np.zeros(5)), torch.ones(1, device="cuda"), s.scratch()
    got = []
    for batches in ([whole], parts):
        q = torch.full((s.n_rows, 8, 64), 7.0, dtype=s.dt, device="cuda")
        out, y = torch.full((s.n_rows, 512), 7.0, dtype=torch.float16, device="cuda"), torch.full((s.n_rows, 512), 7.0, device="cuda")
        for batch in batches:
            pf.pf_op_batch_append(s.cfg, batch, qkv, None, None, rope, 0, q, s.k, s.v, s.status)
        for batch in batches:
            pf.pf_op_attention_tree(s.cfg, batch, q, s.k, s.v, 0, out, scratch, s.status)
            pf.pf_op_adapters(batch, x, qkv[:, :512], y, which[:batch.n_seq], a, b, one, s.status)
        pf.pf_status_read(s.status)
        s.check_attention(q, out)
        ref, bound = R.adapters(*(t[:s.total].cpu().numpy() for t in (qkv[:, :512], x)), a[0].cpu().numpy(), b[0].cpu().numpy(), 1.0)
        assert (np.abs(y[:s.total].cpu().numpy() - ref) <= bound).all() and (y[s.total:] == 7).all()
        got.append((q, s.k.clone(), s.v.clone()))
    for t, u in zip(*got):
        assert torch.equal(t.view(torch.int16), u.view(torch.int16))
