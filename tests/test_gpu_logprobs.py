"""pf_op_logprobs against float64: ids exact (ties, infinities, NaN), log probabilities and entropies within
a derived bound, rows behind odd strides, every refusal's neighbour that is allowed."""
import math

import numpy as np
import pytest

from quantized_transformer_prefill_q1_gb300 import pf

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


def call(x, n, tokens, top, status=None, want=("lp", "ent", "tlp")):
    rows, ld = x.shape
    d = "cuda"
    lp = torch.full((rows + 1,), 7.0, device=d) if "lp" in want else None
    ent = torch.full((rows + 1,), 7.0, device=d) if "ent" in want else None
    ids = torch.full((rows + 1, max(top, 1)), 7, dtype=torch.int32, device=d) if top else None
    tlp = torch.full((rows + 1, max(top, 1)), 7.0, device=d) if top and "tlp" in want else None
    pf.pf_op_logprobs(x, rows, n, ld, tokens, lp, ent, top, ids, tlp, status)
    for t in (lp, ent, ids, tlp):  # nothing behind the last row
        assert t is None or bool((t[rows] == 7).all())
    return [None if t is None else t[:rows].cpu().numpy() for t in (lp, ent, ids, tlp)]


def reference(x, n, tokens, top):
    x = x[:, :n].cpu().numpy().astype(np.float64)
    rows = x.shape[0]
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        e = np.exp(x - m)
        # the maximum first (logits near 1e30 keep the rest), and the ones of the sum apart: in float64 too
        # log(1 + 1e-15) has no digits
        top_n = (x == m).sum(1, keepdims=True)
        d = x - m - np.log(top_n) - np.log1p(np.where((x == m) & (e == 1), 0.0, e).sum(1, keepdims=True) / top_n)
        p = e / e.sum(1, keepdims=True)
        ent = -np.where(p > 0, p * d, np.where(np.isnan(p), np.nan, 0.0)).sum(1)
        lp = d[np.arange(rows), tokens]
        ids, tlp = np.full((rows, top), -1), np.full((rows, top), np.nan)
        for r in range(rows):
            order = [i for i in np.argsort(-np.nan_to_num(x[r] + 0.0, nan=-np.inf), kind="stable") if x[r, i] == x[r, i]][:top]
            ids[r, :len(order)] = order
            tlp[r, :len(order)] = d[r, order]
    return lp, ent, ids, tlp


def check(x, n, top, tokens=None, seed=0):
    """Bound: x - m is exact to half an ulp (2^-24 |x - m|), so each exponential is off by that plus the
    approximation's 2^-21 |x - m| + 2^-21; a weighted sum of them inherits the weighted mean of those errors,
    at most 2^-20 (D + 1) with D the largest |x - m| that has weight (weights below e^-104 are 0 in f32), and a
    few hundred additions in f32 add at most 2^-16 of it in the worst case, 2^-20 in fact; the logarithm and
    the final differences round to half an ulp of their size."""
    rows = x.shape[0]
    if tokens is None:
        tokens = np.random.default_rng(seed).integers(0, n, rows)
    lp, ent, ids, tlp = call(x, n, torch.from_numpy(tokens.astype(np.int32)).cuda(), top)
    rlp, rent, rids, rtlp = reference(x, n, tokens, top)
    if top:
        assert np.array_equal(ids, rids)

    def near(got, want, what):
        fin = np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want)), what
        assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), what
        err = np.abs(got[fin] - want[fin])
        assert np.all(err <= 2.0 ** -23 * np.abs(want[fin]) + 2e-5), (what, float(err.max()) if err.size else 0)

    near(lp, rlp, "logprob")
    near(ent, rent, "entropy")
    if top:
        near(tlp, rtlp, "top_logprob")


def logits(rows, ld, seed, scale=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, ld, device="cuda", generator=g) * scale


@pytest.mark.parametrize("rows,n,ld", [(1, 1, 1), (1, 2, 5), (3, 31, 31), (2, 32, 33), (5, 33, 40), (4, 1000, 1003),
                                       (1, 5000, 5000), (7, 1023, 1024), (2, 4097, 4099), (9, 32768, 32768),
                                       (1, 151936, 151936), (20, 151936, 151936), (3, 100003, 100005), (70, 20011, 20012),
                                       (200, 7000, 7000), (400, 3001, 3003)])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_logprobs(rows, n, ld, top):
    check(logits(rows, ld, rows + n), n, top, seed=n)


@pytest.mark.parametrize("n", [40, 3000, 60001])
def test_ties(n):
    """Few distinct values, constant rows, -0 and +0: the lowest index first."""
    x = torch.zeros(6, n, device="cuda")
    x[1, ::2] = -0.0
    x[2] = logits(1, n, 1)[0].round() * 0.5
    x[3] = -1e30
    x[4, n // 2:] = 1.0
    x[5] = torch.arange(n, device="cuda") // 7
    check(x, n, 32)
    check(x, n, 1)


@pytest.mark.parametrize("n", [50, 2000, 70001])
def test_infinities_and_nan(n):
    x = logits(9, n, 3)
    x[0, 1:] = -math.inf                  # one token left: log probability 0, entropy 0
    x[1, ::3] = -math.inf
    x[2, 5:] = -math.inf                  # fewer finite values than alternatives
    x[3] = -math.inf                      # nothing left
    x[4, 7] = math.inf
    x[5, n - 1] = math.nan
    x[6] = math.nan
    x[7] = torch.finfo(torch.float32).min  # masked with the lowest value instead: uniform
    x[8, :] = torch.finfo(torch.float32).min
    x[8, 3] = 2.0
    check(x, n, 20, np.array([0, 1, 6, 4, 7, 2, 3, 9, 4]))


def test_large_spread_and_offset():
    x = logits(4, 9000, 5)
    x[0] += 1e6
    x[1] *= 1e4
    x[2] = torch.linspace(-200, 0, 9000, device="cuda")
    x[3] = -3e38
    x[3, 77] = 3e38
    rows = [2]
    check(x[rows].contiguous(), 9000, 10)
    # offsets of 1e6 and gaps of thousands: ids exact, results at the logits' own precision
    _, _, ids, tlp = call(x, 9000, torch.zeros(4, dtype=torch.int32, device="cuda"), 10)
    _, _, rids, rtlp = reference(x, 9000, np.zeros(4, int), 10)
    assert np.array_equal(ids, rids)
    with np.errstate(all="ignore"):
        beyond = np.isinf(rtlp.astype(np.float32))  # a gap of 6e38 is not an f32: it rounds to -inf
        assert beyond[3, 1:].all() and np.array_equal(tlp[beyond], rtlp.astype(np.float32)[beyond])
        assert np.all(np.abs(tlp - rtlp)[~beyond] <= (2.0 ** -22 * np.abs(rtlp) + 2e-5)[~beyond])


@pytest.mark.parametrize("gap", [4.0, 9.0, 16.0, 40.0])
def test_one_likely_token(gap):
    """A row of one likely token: ln S and the entropy are tiny and still right in their own size. The weights
    of the others are off by at most 2^-22 + gap' 2^-23 of themselves (gap' their distance, at most 60 here)
    and by as much again in their sum, the logarithm and the quotient by a few 2^-24."""
    x = logits(6, 30011, 12, 1.0)
    x[:, 777] = x.amax(1) + gap
    x[3, 778] = x[3, 777]  # two alike
    tok = torch.full((6,), 777, dtype=torch.int32, device="cuda")
    lp, ent, _, _ = call(x, 30011, tok, 3)
    rlp, rent, _, _ = reference(x, 30011, np.full(6, 777), 3)
    rel = 2 * (2.0 ** -22 + 60 * 2.0 ** -23)
    assert np.all(np.abs(lp - rlp) <= rel * np.abs(rlp) + 1e-37), (lp, rlp)
    assert np.all(np.abs(ent - rent) <= rel * np.abs(rent) + 1e-37), (ent, rent)


def test_tokens_outside_the_vocabulary():
    x = logits(3, 100, 8)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (-1, 97, 1 << 30):
        tok = torch.tensor([5, bad, 96], dtype=torch.int32, device="cuda")
        lp, ent, ids, tlp = call(x, 97, tok, 3, status)
        with pytest.raises(pf.PfError) as e:
            pf.pf_status_read(status)
        assert e.value.status == 5
        assert np.isnan(lp[1]) and np.isfinite(lp[[0, 2]]).all() and np.isfinite(ent).all()
    call(x, 97, tok, 3)  # without a status word: no record, no fault


@pytest.mark.parametrize("want", [("lp",), ("ent",), ("tlp",), ()])
def test_parts(want):
    """Any part alone gives what all together give."""
    x = logits(5, 4001, 9)
    tok = torch.tensor([0, 4000, 17, 3, 2], dtype=torch.int32, device="cuda")
    full = call(x, 4001, tok, 7)
    part = call(x, 4001, tok if "lp" in want else None, 7 if "tlp" in want or not want else 0, None, want)
    for f, p in zip(full, part):
        assert p is None or np.array_equal(f, p)


def test_graph_stream_and_repeat():
    x = logits(33, 50021, 10)
    tok = torch.arange(33, dtype=torch.int32, device="cuda") * 1500
    out = [torch.zeros(33, device="cuda"), torch.zeros(33, device="cuda"),
           torch.zeros(33, 9, dtype=torch.int32, device="cuda"), torch.zeros(33, 9, device="cuda")]

    def go():
        pf.pf_op_logprobs(x, 33, 50021, 50021, tok, out[0], out[1], 9, out[2], out[3])

    go()
    want = [t.clone() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    x2 = logits(33, 50021, 11)
    x.copy_(x2)  # new logits at the same address
    g.replay()
    torch.cuda.synchronize()
    lp = torch.log_softmax(x2.double(), 1)
    assert torch.equal(out[2][:, 0].long(), x2.argmax(1))
    assert float((out[3].double() - lp.gather(1, out[2].long())).abs().max()) <= 2e-5
