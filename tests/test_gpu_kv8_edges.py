"""The 8-bit cache's attention at the edges of what its calls allow: queries that are NaN, sessions whose clusters
are larger than the keys at hand."""
import dataclasses

import numpy as np
import pytest

import kv8_reference as R
import test_gpu_kv8 as T
from oracle import prefill_oracle as O
from quantized_transformer_prefill_q1_gb300 import pf, synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nkv,hd,start,m,nan_at", [
    # row sets of 64 tokens in CTA pairs, the earlier ones with fewer key tiles than the last
    (32, 8, 128, 0, 200, (0, 5, 31, 32, 63, 64, 150)),
    (16, 1, 128, 0, 300, (0, 1, 3, 4, 9, 17, 290)),
    # one CTA a row tile of 128 tokens
    (8, 8, 64, 0, 300, (0, 1, 64, 127, 128, 299)),
    (4, 2, 64, 100, 200, (0, 20, 63, 64, 199)),
    # the few-row form
    (8, 2, 128, 700, 4, (0, 2, 3)),
    (8, 1, 64, 5, 1, ()),
])
def test_a_nan_query_stays_in_its_own_row(nq, nkv, hd, start, m, nan_at):
    """A token's query of one head made NaN (of f16's largest pattern, whose pairs read as f32 are NaN too): that
    row is NaN, every other row keeps its bits."""
    c, val = T.random_cache("int8", nq, nkv, hd, start + m, True, seed=m)
    q = T.queries(c, m, nq, 1.0)
    want = T.attend(c, q, start, m)
    T.check_norms(c, val, q, want, start, m)
    nan = torch.tensor([0x7fff], dtype=torch.int16, device="cuda").view(torch.float16)
    for t in nan_at:
        h = t % nq
        bad = q.clone()
        bad[t, h] = nan
        got = T.attend(c, bad, start, m)[:m].view(m, nq, hd)
        assert bool(torch.isnan(got[t, h]).all()), t
        got[t, h] = want[:m].view(m, nq, hd)[t, h]
        assert torch.equal(got.view(m, -1), want[:m]), t
    pf.pf_status_read(c.status)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hd", [64, 128])
def test_session_with_room_for_far_more_keys(monkeypatch, kind, hd):
    """Chunks of several row tiles at the start of a long cache (the clusters are those of its length, most of
    their CTAs have no key tile yet), a short one, decoded tokens: logits within 2e-2 of the oracle with the same
    cache, as in the session tests of short caches."""
    s = dataclasses.replace(synth.TINY, n_layers=2, vocab=3000, max_seq=4500, n_q_heads=8, n_kv_heads=2, head_dim=hd, kv_dtype="f16")
    layers, extra = synth.model_inputs(s)
    toks = synth.tokens(700, s.vocab, seed=2)
    T.oracle_with_8_bits(monkeypatch, kind)
    dm = pf.DeviceModel(dataclasses.replace(s, kv_dtype=kind), layers, extra, max_chunk=280)
    sess = pf.Session(dm)
    om = O.OracleModel(s, layers, extra)
    logits = torch.empty(s.vocab, device="cuda")
    ids = torch.from_numpy(toks.astype(np.int32)).cuda()
    at = 0
    for m in (150, 9, 280, 1, 40, 1):
        _, want = om.forward_chunk(om.embed(toks[at:at + m]), at, True)
        if m == 1:
            sess.decode_step(ids[at:at + 1], logits)
        else:
            sess.prefill_chunk(toks[at:at + m], at, logits)
        sess.sync()
        at += m
        assert O.rel_l2(logits.cpu().numpy(), want) <= 2e-2, (at, m)
    assert sess.position == at


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("nq,nkv,hd,start,m", [(8, 2, 128, 500, 1), (8, 2, 128, 500, 4), (8, 2, 128, 500, 20), (8, 2, 128, 500, 100),
                                               (4, 4, 64, 300, 70), (16, 1, 128, 90, 60)])
def test_scores_of_hundreds_of_millions(kind, sign, nq, nkv, hd, start, m):
    """Queries and keys near f16's largest values, and all scores of either sign: the output is the value of the
    largest score (where no other one is within the scores' f32 error, 2 hd 2^-24 sum |q k| / sqrt(hd) each as in
    check_attention, plus the scale's and the sum's rounding, 2^-22 of the score). Its weight is rounded to f16 in
    the product and not in the sum, 2^-11, as is the output, 2^-11 and 2^-25; three f32 roundings more."""
    c = T.Cache(kind, nkv, hd, start + m, False, nq, seed=hd + m)
    k, v = c.rows(start + m, False), c.rows(start + m, False)
    k = np.clip(np.abs(k.astype(np.float64)) * 16000 + 8000, 0, 60000).astype(np.float16)
    c.store(k, v, 0)
    q = (sign * np.clip(np.abs(c.rng.standard_normal((m, nq, hd))) * 16000 + 8000, 0, 60000)).astype(np.float16)
    out = T.attend(c, torch.from_numpy(q).cuda(), start, m)[:m].cpu().numpy().astype(np.float64).reshape(m, nq, hd)
    assert np.isfinite(out).all()
    kd, vd = c.values("k", start + m), c.values("v", start + m)
    checked = 0
    for h in range(nq):
        s = q[:, h].astype(np.float64) @ kd[h // (nq // nkv)].T / np.sqrt(hd)  # all of one sign: |s| is the sum of |q k|
        s[np.arange(start + m)[None, :] > start + np.arange(m)[:, None]] = -np.inf
        order = np.argsort(s, 1)
        best, second = s[np.arange(m), order[:, -1]], s[np.arange(m), order[:, -2]]
        apart = best - second > 2 * (2 * hd * 2.0 ** -24 + 2.0 ** -22) * np.abs(second) + 200
        assert np.abs(best).min() > 1.5e9
        want = vd[h // (nq // nkv)][order[:, -1]]
        bound = (2 * 2.0 ** -11 + 2.0 ** -20) * np.abs(want) + 2.0 ** -25
        assert np.all((np.abs(out[:, h] - want) <= bound)[apart])
        checked += int(apart.sum())
    assert checked >= nq * m // 2


def given_cache(kind, nq, codes, scales, max_seq):
    """A linear cache of the given value codes [nkv, L, hd] (numbers of the 8-bit type) and scales [nkv, blocks], by w."""
    nkv, L, hd = codes["k"].shape
    c = T.Cache(kind, nkv, hd, max_seq, False, nq)
    for w in "kv":
        c.codes[w] = R.encode(kind, codes[w])
        c.scales[w] = scales[w].astype(np.float32)
        dev, s = pf.kv8_views(c.cfg, c.dev[w])
        dev.view(torch.uint8)[c.layer, :, :L] = torch.from_numpy(c.codes[w]).cuda()
        s[c.layer, :, :scales[w].shape[1]] = torch.from_numpy(c.scales[w]).cuda()
    return c


def check_scaled(c, q, out, start, m):
    """check_attention's bound elementwise, with its term for weights that are subnormal in f16 taken from what the
    weights are: probability times V scale, relative to the row's largest, 2^-25 of that for each code. A V
    scale below 2^-60 counts as that: codes up to 448 give at most 2^-51."""
    L, hd = start + m, c.hd
    k, v = c.values("k", L), c.values("v", L)
    qd = q.cpu().numpy().astype(np.float64)
    want, mag, _, big = R.attention(qd, k, v, start)
    got = out[:m].cpu().numpy().astype(np.float64).reshape(want.shape)
    s_err = (2 * hd + 8) * 2.0 ** -24 * big
    G = qd.shape[1] // c.nkv
    see = np.arange(L)[None, :] <= start + np.arange(m)[:, None]
    for h in range(qd.shape[1]):
        s = np.where(see, qd[:, h] @ k[h // G].T / np.sqrt(hd), -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        top = (p * np.repeat(c.scales["v"][h // G].astype(np.float64), R.BLOCK)[:L]).max(1)[:, None]
        codes = np.abs(R.decode(c.kind, c.codes["v"][h // G][:L])).sum(0)[None, :]
        bound = 2.0 ** -11 * np.abs(want[:, h]) + (2.0 ** -11 + 2 * np.expm1(s_err) + 2.0 ** -20) * mag[:, h]
        bound += 2.0 ** -25 * top * codes + 2.0 ** -24 + 2.0 ** -51
        assert np.all(np.abs(got[:, h] - want[:, h]) <= bound), h


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("m", [1, 3, 40, 300])
def test_value_scales_at_the_ends_of_their_range(kind, m):
    """Blocks of V at 2^16 (whose keys have weights of about 2^-23), 2^-40, 1, 0 and 2^-100: the small ones give
    nothing that an f16 holds."""
    nq, hd, start = 4, 64, 420
    L = start + m
    rng = np.random.default_rng(m)
    nblk = -(-L // R.BLOCK)
    blocks = np.arange(L) // R.BLOCK % 5
    k = rng.integers(-1, 2, (1, L, hd)).astype(np.float64)
    k[:, blocks == 0] = -4
    v = np.rint(rng.uniform(-14, 14, (1, L, hd))) * 8  # codes of both types
    scale = np.array([2.0 ** 16, 2.0 ** -40, 1.0, 0.0, 2.0 ** -100])[np.arange(nblk) % 5][None]
    c = given_cache(kind, nq, {"k": k, "v": v}, {"k": np.ones((1, nblk)), "v": scale}, L + 3)
    q = torch.from_numpy((0.5 + 0.02 * rng.standard_normal((m, nq, hd))).astype(np.float16)).cuda()
    check_scaled(c, q, T.attend(c, q, start, m), start, m)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("m", [1, 3, 40, 300])
def test_key_scales_at_the_ends_of_their_range(kind, m):
    """Blocks of K at 2^16 (queries are multiples of 2^-8, so that scores are of a few hundreds), 2^-40, 0 and 1."""
    nq, hd, start = 4, 64, 420
    L = start + m
    rng = np.random.default_rng(m)
    nblk = -(-L // R.BLOCK)
    k = rng.integers(-1, 2, (1, L, hd)) * (rng.random((1, L, hd)) < 0.2).astype(np.float64)
    v = np.rint(rng.uniform(-14, 14, (1, L, hd))) * 8
    scale = np.array([2.0 ** 16, 2.0 ** -40, 0.0, 1.0])[np.arange(nblk) % 4][None]
    c = given_cache(kind, nq, {"k": k, "v": v}, {"k": scale, "v": np.ones((1, nblk))}, L + 3)
    q = torch.from_numpy((rng.integers(-3, 4, (m, nq, hd)) * 2.0 ** -8).astype(np.float16)).cuda()
    check_scaled(c, q, T.attend(c, q, start, m), start, m)


@pytest.mark.parametrize("rows,at", [(1, 300), (50, 300), (3, 383), (200, 200), (130, 250)])
def test_store_through_a_bad_table_entry(rows, at):
    """A store whose positions reach a page outside the pool: the status is the store's own (nothing else has run),
    the positions of good pages are stored, every other byte stays."""
    for bad in (-1, 7, 1 << 30, -(1 << 31)):
        c = T.filled("int8", 2, 128, 600, True, 8)
        assert c.pool == 7
        t = c.table.copy()
        t[2] = bad  # positions 256 .. 383
        table = torch.from_numpy(t).cuda()
        before = {w: c.dev[w].clone() for w in "kv"}
        x = {w: c.rows(rows, False) for w in "kv"}
        d = {w: torch.from_numpy(x[w]).cuda() for w in "kv"}
        pf.pf_op_kv8_store(c.cfg, d["k"], d["v"], c.layer, at, rows, c.dev["k"], c.dev["v"], table, c.status)
        with pytest.raises(pf.PfError) as e:
            pf.pf_status_read(c.status)
        assert e.value.status == 6
        first = at // R.BLOCK * R.BLOCK  # a scale that grows takes its block's earlier codes along
        p = np.arange(first, at + rows)
        p = p[(p < 256) | (p >= 384)]
        blk = np.unique(p // R.BLOCK)
        slots = torch.from_numpy(c.slot_of(p)).cuda()
        sblk = torch.from_numpy(c.slot_of(blk * R.BLOCK) // R.BLOCK).cuda()
        for w in "kv":
            R.store(c.kind, c.codes[w], c.scales[w], x[w], at)
            want, scale = (t.clone() for t in pf.kv8_views(c.cfg, before[w]))
            want[c.layer].view(torch.uint8)[:, slots] = torch.from_numpy(c.codes[w][:, p]).cuda()
            scale[c.layer][:, sblk] = torch.from_numpy(c.scales[w][:, blk]).cuda()
            got, got_scale = pf.kv8_views(c.cfg, c.dev[w])
            assert torch.equal(got, want) and torch.equal(got_scale.view(torch.int32), scale.view(torch.int32))


def growing_rows(c, n):
    """Rows whose largest value grows by about 2^6 within every block of 32: every chunk raises its scale."""
    x = c.rng.standard_normal((n, c.nkv, c.hd)) * 2.0 ** (np.arange(n) % 32 / 5 - 3)[:, None, None]
    return x.astype(np.float16)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hd,paged", [(128, False), (64, True)])
def test_how_far_a_cut_prompt_is_from_one_chunk(kind, hd, paged):
    """The scales are the same. A code that later chunks of its block scale down is rounded once for each: by at
    most 1/2, then, in steps of the last scale, 1/4, 1/8, ... before it (each scale at most half of the next), less
    than 1 in all where one chunk rounds by 1/2: int8 codes differ by at most 1. So do e4m3's below 2^-6, whose steps
    are 2^-9; above, a power of two as the scale moves no rounding."""
    a, b = T.Cache(kind, 2, hd, 300, paged, seed=5), T.Cache(kind, 2, hd, 300, paged, seed=5)
    k, v = growing_rows(a, 300), growing_rows(a, 300)
    a.store(k, v, 0)
    at = 0
    for m in (3, 50, 1, 1, 17, 100, 5, 81, 1, 1, 40):
        b.store(k[at:at + m], v[at:at + m], at)
        at += m
    assert at == 300
    a.check(300), b.check(300)
    for w, x in (("k", k), ("v", v)):
        assert np.array_equal(a.scales[w], b.scales[w])
        one, cut = R.decode(kind, a.codes[w]), R.decode(kind, b.codes[w])
        step = 1.0 if kind == "int8" else 2.0 ** -9
        assert np.abs(one - cut).max() <= step
        if kind == "e4m3":
            assert np.array_equal(one[np.abs(one) > 2.0 ** -6], cut[np.abs(one) > 2.0 ** -6])
        s = np.repeat(b.scales[w].astype(np.float64), R.BLOCK, axis=1)[:, :300, None]
        err = np.abs(cut * s - x.astype(np.float64).transpose(1, 0, 2)) / s
        if kind == "int8":
            assert (one != cut).any()  # so it does differ
            assert err.max() < 1 and np.abs(one * s - x.astype(np.float64).transpose(1, 0, 2)).max() <= 0.5 * s.max()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_a_rejected_draft_leaves_its_scale(kind):
    """A draft of large rows is stored, all of it but the first token rejected, smaller rows stored in its place: the
    block keeps the draft's scale, until it is stored again from its first position."""
    c = T.Cache(kind, 2, 128, 128, True)
    small = [c.rows(32, False) for _ in range(2)]
    big = c.rows(5, False) * np.float16(64)
    c.store(small[0][:10], small[1][:10], 0)
    before = {w: c.scales[w][:, 0].copy() for w in "kv"}
    c.store(big, big, 10)
    c.store(small[0][11:20], small[1][11:20], 11)
    c.check(20)
    assert all((c.scales[w][:, 0] >= 32 * before[w]).all() for w in "kv")
    c.store(*(x[:20] for x in small), 0)
    c.check(20)
    assert all((c.scales[w][:, 0] <= 2 * before[w]).all() for w in "kv")


@pytest.mark.parametrize("kind,nq,nkv,hd,start,m", [("e4m3", 4, 2, 128, 0, 8192), ("int8", 4, 1, 128, 777, 5000),
                                                    ("int8", 2, 2, 64, 0, 8192), ("e4m3", 8, 1, 64, 100, 4100)])
def test_the_longest_chunks(kind, nq, nkv, hd, start, m):
    """As long as a session's chunk may be: row sets in several waves, of one to 64 key tiles."""
    c, val = T.random_cache(kind, nq, nkv, hd, start + m, True, seed=m)
    q = T.queries(c, m, nq, 1.0)
    out = T.attend(c, q, start, m)
    T.check_norms(c, val, q, out, start, m)
    assert bool((out[m:] == 3).all())
    pf.pf_status_read(c.status)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_offsets_past_32_bits(kind):
    """A layer of more than 2^32 bytes: the last positions stored, read back and attended to by both forms. The
    others hold zeros (score 0): the stored keys' scores of about 60 leave them a weight of 2^25 e^-60."""
    hd, nq, n = 128, 4, 100
    max_seq = (1 << 25) + 300
    c = T.Cache.__new__(T.Cache)
    c.kind, c.layer, c.nkv, c.hd, c.rng, c.table_dev = kind, 0, 1, hd, np.random.default_rng(1), None
    c.cfg = T.config(kind, nq, 1, hd, max_seq, 0, n_layers=1)
    c.status = torch.zeros(4, dtype=torch.int32, device="cuda")
    c.dev = {w: pf.kv8_cache(c.cfg) for w in "kv"}
    at = max_seq - n
    k, v = c.rows(n, False), c.rows(n, False)
    k[:, :, :8] = np.abs(k[:, :, :8]) + np.float16(8)
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    pf.pf_op_kv8_store(c.cfg, kd, vd, 0, at, n, c.dev["k"], c.dev["v"], None, c.status)
    val = {}
    for w in "kv":
        back = torch.empty(n, 1, hd, device="cuda")
        pf.pf_op_kv8_load(c.cfg, c.dev[w], 0, at, n, back, None, c.status)
        val[w] = back.double()[:, 0]
        codes, scales = np.zeros((1, 128, hd), np.uint8), np.zeros((1, 4), np.float32)
        lo = at % R.BLOCK
        scales[:, 0] = 2.0 ** -32  # the zeros before: a scale below any
        R.store(kind, codes, scales, k if w == "k" else v, lo)
        want = R.values(kind, codes, scales)[0, lo:lo + n]
        assert np.array_equal(back[:, 0].cpu().numpy().astype(np.float64), want)
        dev = pf.kv8_views(c.cfg, c.dev[w])[0]
        assert not bool(dev[0, 0, :1 << 20].view(torch.uint8).any()) and not bool(dev[0, 0, at - 1000:at].view(torch.uint8).any())
    for m in (1, 4, 40):
        q = torch.from_numpy((0.3 * c.rng.standard_normal((m, nq, hd))).astype(np.float16)).cuda()
        q[:, :, :8] = 10
        out = T.attend(c, q, max_seq - m, m)[:m].double().view(m, nq, hd)
        see = torch.arange(n, device="cuda")[None, :] <= n - m + torch.arange(m, device="cuda")[:, None]
        for h in range(nq):
            s = q[:, h].double() @ val["k"].T / hd ** 0.5
            assert float(s.min()) > 50
            p = torch.exp(s.masked_fill(~see, -float("inf")))
            want = p @ val["v"] / (p.sum(1, keepdim=True) + at)
            assert float((out[:, h] - want).norm() / want.norm()) <= 5e-4, (m, h)
    pf.pf_status_read(c.status)


def test_logits_rows_past_32_bits():
    """Rows whose distance is 2^30 + 8 values: the third starts behind 2^33 bytes."""
    ld, n = (1 << 30) + 8, 5000
    buf = torch.empty(3 * ld, device="cuda")
    x = buf.as_strided((3, n), (ld, 1))
    x.copy_(torch.randn(3, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)))
    lp, ids = torch.empty(3, device="cuda"), torch.empty(3, 4, dtype=torch.int32, device="cuda")
    tok = torch.tensor([1, 4999, 77], dtype=torch.int32, device="cuda")
    pf.pf_op_logprobs(x, 3, n, ld, tok, lp, None, 4, ids)
    ref = torch.log_softmax(x.double(), 1)
    assert float((lp.double() - ref.gather(1, tok.long()[:, None])[:, 0]).abs().max()) <= 2e-5
    assert torch.equal(ids.long(), ref.topk(4, 1).indices)
