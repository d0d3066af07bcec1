"""8-bit KV cache on the GPU: store and read-back exact against the numpy definition; attention within
a derived bound of float64; sessions over an 8-bit cache against the oracle with the same quantisation."""
import dataclasses

import numpy as np
import pytest

import kv8_reference as R
from oracle import prefill_oracle as O
from quantized_transformer_prefill_q1_gb300 import pf, synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BASE = synth.QWEN3_8B_LAYER


def config(kind, nq, nkv, hd, max_seq, pool=0, n_layers=2):
    s = dataclasses.replace(BASE, kv_dtype=kind, n_q_heads=nq, n_kv_heads=nkv, head_dim=hd)
    return pf.make_config(s, 512, n_layers=n_layers, max_seq=max_seq, kv_block_pool=pool)


class Cache:
    """A K or V cache pair on the device and, per logical position, the definition's codes and scales."""

    def __init__(self, kind, nkv, hd, max_seq, paged, nq=None, layer=1, seed=0):
        self.rng = np.random.default_rng(seed)
        self.kind, self.layer, self.nkv, self.hd, self.max_seq = kind, layer, nkv, hd, max_seq
        pages = -(-max_seq // pf.KV_BLOCK)
        self.pool = pages + 2 if paged else 0
        self.table = self.rng.permutation(self.pool)[:pages].astype(np.int32) if paged else None
        self.table_dev = torch.from_numpy(self.table).cuda() if paged else None
        self.cfg = config(kind, nq or 2 * nkv, nkv, hd, max_seq, self.pool)
        self.slots = self.pool * pf.KV_BLOCK if paged else max_seq
        self.dev, self.codes, self.scales = {}, {}, {}
        for w in "kv":
            buf = pf.kv8_cache(self.cfg)
            # arbitrary bytes everywhere: NaN codes and NaN scales wherever nothing has been stored
            buf.copy_(torch.from_numpy(self.rng.integers(0, 256, buf.numel(), dtype=np.uint8)))
            pf.kv8_views(self.cfg, buf)[1].fill_(float("nan"))
            c = pf.kv8_views(self.cfg, buf)[0].view(torch.uint8)
            self.dev[w] = buf
            self.codes[w] = c[layer].cpu().numpy()[:, self.slot_of(np.arange(max_seq))].copy()
            self.scales[w] = np.full((nkv, -(-max_seq // R.BLOCK)), np.nan, np.float32)
        self.before = {w: self.dev[w].clone() for w in "kv"}
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")

    def slot_of(self, p):
        return p if self.table is None else self.table[p // pf.KV_BLOCK] * pf.KV_BLOCK + p % pf.KV_BLOCK

    def rows(self, m, spread=True):
        """f16 rows [m, nkv, hd]: normal, some blocks and channels far larger or smaller, some values zero."""
        x = self.rng.standard_normal((m, self.nkv, self.hd))
        if spread:
            x *= 2.0 ** self.rng.integers(-3, 4, (m, 1, 1))
            x[:, :, :: 17] *= 9
            x[self.rng.random(x.shape) < 0.02] = 0
        return x.astype(np.float16)

    def store(self, k, v, start, strided=False):
        m = k.shape[0]
        for w, x in (("k", k), ("v", v)):
            with np.errstate(all="ignore"):
                R.store(self.kind, self.codes[w], self.scales[w], x, start)
        kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
        if strided:  # [nkv][rows + 3][hd + 8], viewed token first
            def view(t):
                p = torch.full((self.nkv, m + 3, self.hd + 8), float("nan"), dtype=torch.float16, device="cuda")
                p[:, :m, :self.hd] = t.permute(1, 0, 2)
                return p[:, :m, :self.hd].permute(1, 0, 2)
            kd, vd = view(kd), view(vd)
        pf.pf_op_kv8_store(self.cfg, kd, vd, self.layer, start, m, self.dev["k"], self.dev["v"], self.table_dev, self.status)

    def check(self, end):
        """The device holds the definition's codes and scales below `end`, and nothing else changed."""
        pos = self.slot_of(np.arange(end))
        blk = pos[::R.BLOCK] // R.BLOCK
        for w in "kv":
            c, s = pf.kv8_views(self.cfg, self.dev[w])
            c = c.view(torch.uint8).cpu().numpy()
            s = s.cpu().numpy()
            assert np.array_equal(c[self.layer][:, pos], self.codes[w][:, :end]), w
            assert np.array_equal(s[self.layer][:, blk], self.scales[w][:, :len(blk)]), w
            c0, s0 = pf.kv8_views(self.cfg, self.before[w])
            c0, s0 = c0.view(torch.uint8).cpu().numpy().copy(), s0.cpu().numpy().copy()
            c0[self.layer][:, pos] = self.codes[w][:, :end]
            s0[self.layer][:, blk] = self.scales[w][:, :len(blk)]
            assert np.array_equal(c, c0) and np.array_equal(s, s0, equal_nan=True), w

    def values(self, w, end):
        return R.values(self.kind, self.codes[w][:, :end], self.scales[w][:, :-(-end // R.BLOCK)])


# ------------------------------------------------------------------ store
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hd,nkv,paged,strided", [(128, 8, False, False), (128, 1, True, True), (64, 2, True, False),
                                                  (64, 3, False, True)])
def test_store_exact(kind, hd, nkv, paged, strided):
    """A prompt, chunks that start and end inside blocks, single tokens: codes, scales and every other byte."""
    c = Cache(kind, nkv, hd, 300, paged, seed=hd + nkv)
    start = 0
    for m in (5, 1, 1, 30, 64, 27, 1, 100, 1, 70):
        c.store(c.rows(m), c.rows(m), start, strided)
        start += m
        c.check(start)
    assert start == 300
    pf.pf_status_read(c.status)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_store_scales(kind):
    """Scales that grow token by token through every exponent of f16, zero blocks, subnormals, the limits."""
    c = Cache(kind, 1, 64, 256, False)
    for t in range(41):  # 2^-24 .. 2^15 and the largest f16, past a block's end
        x = np.zeros((1, 1, 64), np.float16)
        x[0, 0, t % 64] = 65504 if t == 40 else 2.0 ** (t - 24)
        x[0, 0, (t + 1) % 64] = -x[0, 0, t % 64] / 3
        c.store(x, -x, t)
        c.check(t + 1)
    c.store(np.zeros((60, 1, 64), np.float16), -np.zeros((60, 1, 64), np.float16), 41)  # 64 .. 95: zeros alone
    c.check(101)
    ties = (np.arange(64) - 32).astype(np.float16) / 2 + np.float16(0.25)
    c.store(np.tile(ties, (20, 1, 1)), np.tile(ties[::-1], (20, 1, 1)), 101)
    c.check(121)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_store_again_after_rejected_tokens(kind):
    """Positions stored again (a rejected draft): the block keeps a scale that its old positions allow."""
    c = Cache(kind, 2, 128, 128, True)
    c.store(c.rows(40), c.rows(40), 0)
    c.store(c.rows(9) * np.float16(16), c.rows(9), 40)
    c.store(c.rows(3), c.rows(3), 42)
    # positions 45 .. 48 still hold the rejected draft
    c.check(49)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_store_nonfinite_is_recorded(kind):
    c = Cache(kind, 2, 64, 128, False)
    k, v = c.rows(40), c.rows(40)
    k[3, 0, 5], k[3, 1, 6], k[39, 0, 0], v[7, 1, 1] = np.nan, np.inf, -np.inf, np.nan
    k[32:, 1] = np.inf  # a block with no finite value but zero
    c.store(k, v, 0)
    c.check(40)
    with pytest.raises(pf.PfError) as e:
        pf.pf_status_read(c.status)
    assert e.value.status == 12


def test_e4m3_chunks_equal_one_shot():
    """Powers of two as scales: e4m3 codes do not depend on how the prompt was cut, but for values that the
    grown scale makes subnormal (below 2^-6 of the scale), which may round twice."""
    a, b = Cache("e4m3", 2, 128, 256, False, seed=5), Cache("e4m3", 2, 128, 256, False, seed=5)
    k, v = a.rows(256, False), a.rows(256, False)
    a.store(k, v, 0)
    s = 0
    for m in (3, 50, 1, 1, 120, 81):
        b.store(k[s:s + m], v[s:s + m], s)
        s += m
    for w in "kv":
        (ca, sa), (cb, sb) = pf.kv8_views(a.cfg, a.dev[w]), pf.kv8_views(b.cfg, b.dev[w])
        assert torch.equal(sa[1], sb[1])
        x, y = ca[1].float(), cb[1].float()
        assert torch.equal(x[x.abs() >= 2.0 ** -6], y[x.abs() >= 2.0 ** -6])
        assert float((x - y).abs().max()) <= 2.0 ** -9


# ------------------------------------------------------------------ read-back
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("paged", [False, True])
def test_load_exact(kind, paged):
    c = Cache(kind, 3, 64, 400, paged)
    c.store(c.rows(390), c.rows(390), 0)
    for start, m in ((0, 390), (0, 1), (127, 2), (200, 190), (389, 1)):
        for w in "kv":
            out = torch.full((m + 1, 3, 64), 7.0, device="cuda")
            pf.pf_op_kv8_load(c.cfg, c.dev[w], c.layer, start, m, out, c.table_dev)
            want = c.values(w, 390)[:, start:start + m].transpose(1, 0, 2)
            assert np.array_equal(out[:m].cpu().numpy().astype(np.float64), want)
            assert bool((out[m] == 7).all())


# ------------------------------------------------------------------ attention
def attend(c, q, start, m, scratch=None, out=None):
    nq = q.shape[1]
    if scratch is None:
        scratch = pf.attention_kv8_scratch(c.cfg, m)
    if out is None:
        out = torch.full((m + 1, nq * c.hd), 3.0, dtype=torch.float16, device="cuda")
    pf.pf_op_attention_kv8(c.cfg, q, c.dev["k"], c.dev["v"], c.layer, start, m, out, scratch, c.table_dev, c.status)
    return out


def check_attention(c, q, out, start, m):
    """Elementwise against float64. The output is rounded to f16 (2^-11 of it, 2^-25 when subnormal) and so is
    each probability, taken relative to a running maximum at most 2^8 below the true one (2^-11 of p, or 2^-25
    of the largest weight when subnormal: sum over L keys, divided by the denominator >= 1). A score is an f32
    sum of hd exact products, off by at most 2 hd 2^-24 sum |q k| / sqrt(hd) (each addition may truncate, as
    the tensor core's do) and by a few roundings of the scaling; the weights' relative error is that in the
    numerator and again in the denominator, and the approximate exponential adds 2^-21."""
    L = start + m
    k, v = c.values("k", L), c.values("v", L)
    qd = q.cpu().numpy().astype(np.float64)
    want, mag, den, big = R.attention(qd, k, v, start)
    got = out[:m].cpu().numpy().astype(np.float64).reshape(m, -1, c.hd)
    s_err = (2 * c.hd + 8) * 2.0 ** -24 * big
    vmax = np.abs(v).max()
    bound = 2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 2 * np.expm1(s_err) + 2.0 ** -20) * mag
    bound += L * 2.0 ** -25 * vmax / den[:, :, None] + 2.0 ** -24
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()), np.argwhere(bad)[:4].tolist())
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 5e-4, rel  # sqrt(2) 2^-12 if every error were a rounding; twice that with room for the sums
    if out.shape[0] > m:
        assert bool((out[m:] == 3).all())  # the row behind the last one


def filled(kind, nkv, hd, L, paged, nq, seed=0, spare=9, gain=1.0):
    c = Cache(kind, nkv, hd, L + spare, paged, nq, seed=seed)
    c.store(c.rows(L, False), c.rows(L), 0)
    return c


def queries(c, m, nq, gain):
    return torch.from_numpy((gain * c.rng.standard_normal((m, nq, c.hd))).astype(np.float16)).cuda()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("nq,nkv,hd", [(32, 8, 128), (4, 2, 64), (6, 6, 64), (16, 1, 128), (8, 1, 64), (64, 1, 128)])
@pytest.mark.parametrize("start,m", [(0, 1), (31, 1), (700, 1), (1023, 2), (0, 3), (95, 4), (1300, 7), (33, 16)])
def test_attention_few_tokens(kind, nq, nkv, hd, start, m):
    c = filled(kind, nkv, hd, start + m, (start + nq) % 2 == 0, nq, seed=start + m)
    q = queries(c, m, nq, 1.0)
    check_attention(c, q, attend(c, q, start, m), start, m)
    pf.pf_status_read(c.status)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("nq,nkv,hd,start,m", [(32, 8, 128, 0, 128), (32, 8, 128, 77, 100), (8, 8, 64, 1000, 77),
                                               (4, 2, 64, 0, 513), (16, 1, 128, 515, 33), (4, 4, 128, 640, 300),
                                               (64, 1, 64, 250, 9), (8, 2, 128, 2040, 130)])
def test_attention_chunks(kind, nq, nkv, hd, start, m):
    c = filled(kind, nkv, hd, start + m, start % 2 == 0, nq, seed=start + m)
    q = queries(c, m, nq, 1.0)
    check_attention(c, q, attend(c, q, start, m), start, m)
    pf.pf_status_read(c.status)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("m", [1, 4, 150])
def test_attention_peaked_and_rising(kind, m):
    """Large scores (the running maximum rises over and over), each later key block larger than the one before,
    and value blocks whose scales differ by 2^20."""
    nq, nkv, hd, start = 8, 2, 128, 600
    c = Cache(kind, nkv, hd, start + m + 3, True, nq, seed=m)
    k, v = c.rows(start + m, False), c.rows(start + m, False)
    k *= (1 + 6 * np.arange(start + m) / (start + m))[:, None, None].astype(np.float16)
    v[::64] *= np.float16(2.0 ** -10)
    v[64:96] *= np.float16(2.0 ** 10)
    c.store(k, v, 0)
    q = queries(c, m, nq, 1.5)
    check_attention(c, q, attend(c, q, start, m), start, m)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("m", [1, 60])
def test_attention_zero_values_and_queries(kind, m):
    """Blocks of zero keys and values (scale 2^-32), a row of zero queries: a plain mean of the values."""
    nq, nkv, hd, start = 4, 1, 64, 200
    c = Cache(kind, nkv, hd, start + m, False, nq, seed=m)
    k, v = c.rows(start + m, False), c.rows(start + m, False)
    k[32:64], v[96:128] = 0, 0
    c.store(k, v, 0)
    q = queries(c, m, nq, 1.0)
    q[0] = 0
    check_attention(c, q, attend(c, q, start, m), start, m)


def random_cache(kind, nq, nkv, hd, L, paged, seed):
    """A filled cache pair without the numpy mirror, and its values [L, nkv, hd] read back in float64."""
    c = Cache.__new__(Cache)
    rng = np.random.default_rng(seed)
    pages = -(-(L + 5) // pf.KV_BLOCK)
    c.pool = pages + 1 if paged else 0
    c.kind, c.layer, c.nkv, c.hd, c.rng = kind, 1, nkv, hd, rng
    c.table_dev = torch.from_numpy(rng.permutation(c.pool)[:pages].astype(np.int32)).cuda() if paged else None
    c.cfg = config(kind, nq, nkv, hd, L + 5, c.pool)
    c.status = torch.zeros(4, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    c.dev, val = {}, {}
    for w in "kv":
        c.dev[w] = pf.kv8_cache(c.cfg)
        c.dev[w].copy_(torch.randint(256, c.dev[w].shape, device="cuda", generator=g, dtype=torch.uint8))
    k, v = (torch.randn(L, nkv, hd, device="cuda", generator=g).half() for _ in range(2))
    for s in range(0, L, 8192):
        n = min(8192, L - s)
        pf.pf_op_kv8_store(c.cfg, k[s:s + n], v[s:s + n], 1, s, n, c.dev["k"], c.dev["v"], c.table_dev, c.status)
    for w in "kv":
        t = torch.empty(L, nkv, hd, device="cuda")
        pf.pf_op_kv8_load(c.cfg, c.dev[w], 1, 0, L, t, c.table_dev)
        val[w] = t.double()
    return c, val


def check_norms(c, val, q, out, start, m):
    """Per head within the norm bound of check_attention, against a float64 product on the GPU."""
    nq, L = q.shape[1], start + m
    G = nq // c.nkv
    out = out[:m].double().view(m, nq, c.hd)
    see = torch.arange(L, device="cuda")[None, :] <= start + torch.arange(m, device="cuda")[:, None]
    for h in range(nq):
        s = (q[:, h].double() @ val["k"][:L, h // G].T / c.hd ** 0.5).masked_fill(~see, -float("inf"))
        want = torch.softmax(s, 1) @ val["v"][:L, h // G]
        assert float((out[:, h] - want).norm() / want.norm()) <= 5e-4, h


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("m,start", [(1, 20011), (3, 20011), (40, 20011), (520, 1000), (512, 4095), (1, 60000)])
def test_attention_long_cache(kind, m, start):
    """Every form at full size: all splits of the few-row kernel, clusters with and without parts of the keys."""
    nq, nkv, hd = 32, 8, 128
    c, val = random_cache(kind, nq, nkv, hd, start + m, m % 2 == 1, 3)
    q = queries(c, m, nq, 1.0)
    check_norms(c, val, q, attend(c, q, start, m), start, m)
    pf.pf_status_read(c.status)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("nq,nkv,hd,m,start",
                         [(16, 2, 128, 5, 1500), (16, 2, 128, 16, 2030), (16, 1, 128, 3, 4000), (8, 2, 64, 40, 5000),
                          (16, 1, 64, 77, 1100), (32, 4, 128, 30, 3001), (64, 1, 128, 1, 2047), (64, 1, 64, 3, 9000),
                          (8, 8, 64, 100, 28), (32, 8, 128, 20, 107), (32, 8, 128, 20, 108), (32, 8, 128, 20, 109)])
def test_attention_wide_clusters(kind, nq, nkv, hd, m, start):
    """Few rows over many keys, whose tiles are cut over 9 to 16 CTAs or their pairs, down to one part a tile and
    uneven ones; and chunks that end just before, at and behind the first tile's end (one part, then two)."""
    for paged in (False, True):
        c, val = random_cache(kind, nq, nkv, hd, start + m, paged, seed=m + start)
        q = queries(c, m, nq, 1.0)
        out = attend(c, q, start, m)
        check_norms(c, val, q, out, start, m)
        assert torch.equal(attend(c, q, start, m)[:m], out[:m])
        pf.pf_status_read(c.status)


@pytest.mark.parametrize("seed", range(24))
def test_attention_drawn(seed):
    """Sizes over the whole range."""
    rng = np.random.default_rng(100 + seed)
    nq, nkv, hd = [(32, 8, 128), (4, 2, 64), (8, 8, 64), (16, 1, 128), (32, 4, 128), (2, 2, 64), (8, 8, 128), (64, 2, 64)][seed % 8]
    m = int(np.exp(rng.uniform(0, np.log(400))))
    start = int(np.exp(rng.uniform(0, np.log(9000)))) - 1
    c, val = random_cache("e4m3" if rng.random() < 0.5 else "int8", nq, nkv, hd, start + m, rng.random() < 0.5, seed)
    q = queries(c, m, nq, 1.5)
    out = attend(c, q, start, m)
    check_norms(c, val, q, out, start, m)
    assert bool((out[m:] == 3).all())
    pf.pf_status_read(c.status)


@pytest.mark.parametrize("ms", [(1, 1), (1, 300), (64, 64)])
def test_attention_on_two_streams_at_once(ms):
    """Calls that overlap, each with its own scratch, do not touch each other."""
    c, val = random_cache("e4m3", 8, 2, 128, 6000, True, 7)
    calls = []
    for i, m in enumerate(ms):
        q = queries(c, m, 8, 1.0)
        calls.append((q, 6000 - m, m, pf.attention_kv8_scratch(c.cfg, m), torch.zeros(m, 1024, dtype=torch.float16, device="cuda"),
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, start, m, scratch, out, st in calls:
            with torch.cuda.stream(st):
                attend(c, q, start, m, scratch, out)
    torch.cuda.synchronize()
    for q, start, m, scratch, out, _ in calls:
        check_norms(c, val, q, out, start, m)


def test_attention_repeats_and_shares_scratch():
    """Calls of other sizes on one scratch leave it ready for the next; the same call gives the same bits."""
    c = filled("e4m3", 2, 128, 900, True, 8, seed=1)
    scratch = pf.attention_kv8_scratch(c.cfg, 300)
    first = {}
    for _ in range(2):
        for m in (1, 300, 2, 64, 5, 1):
            q = torch.from_numpy(np.random.default_rng(m).standard_normal((m, 8, 128)).astype(np.float16)).cuda()
            out = attend(c, q, 900 - m, m, scratch)
            if m in first:
                assert torch.equal(out, first[m])
            else:
                first[m] = out
                check_attention(c, q, out, 900 - m, m)
    assert int(scratch[:4096].sum()) == 0


@pytest.mark.parametrize("m", [1, 200])
def test_attention_in_a_captured_graph_and_on_a_side_stream(m):
    c = filled("int8", 2, 128, 700, True, 8, seed=2)
    q = queries(c, m, 8, 1.0)
    want = attend(c, q, 700 - m, m)
    scratch, out = pf.attention_kv8_scratch(c.cfg, m), torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend(c, q, 700 - m, m, scratch, out)
    side.synchronize()
    assert torch.equal(out[:m], want[:m])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attend(c, q, 700 - m, m, scratch, out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:m], want[:m])


@pytest.mark.parametrize("m", [1, 100])
def test_bad_table_entries_are_recorded_not_followed(m):
    """Entries outside the pool (of a page in use): a status, no access outside the cache."""
    c = filled("e4m3", 2, 128, 600, True, 8)
    for bad in (-1, c.pool, 1 << 30, -(1 << 31)):
        t = c.table.copy()
        t[2] = bad
        table = torch.from_numpy(t).cuda()
        before = {w: c.dev[w].clone() for w in "kv"}
        q, out = queries(c, m, 8, 1.0), torch.zeros(m, 1024, dtype=torch.float16, device="cuda")
        pf.pf_op_attention_kv8(c.cfg, q, c.dev["k"], c.dev["v"], 1, 600 - m, m, out, pf.attention_kv8_scratch(c.cfg, m), table, c.status)
        with pytest.raises(pf.PfError) as e:
            pf.pf_status_read(c.status)
        assert e.value.status == 6
        x = torch.ones(m, 2, 128, dtype=torch.float16, device="cuda")
        pf.pf_op_kv8_store(c.cfg, x, x, 1, 300, min(m, 50), c.dev["k"], c.dev["v"], table, c.status) if m == 1 else None
        got = torch.empty(3, 2, 128, device="cuda")
        pf.pf_op_kv8_load(c.cfg, c.dev["k"], 1, 300, 3, got, table, c.status)
        with pytest.raises(pf.PfError) as e:
            pf.pf_status_read(c.status)
        assert e.value.status == 6
        assert all(torch.equal(before[w], c.dev[w]) for w in "kv")
    # an entry that no position of the call reaches is not looked at
    t = c.table.copy()
    t[4] = -1
    q = queries(c, 1, 8, 1.0)
    out = torch.empty(1, 1024, dtype=torch.float16, device="cuda")
    pf.pf_op_attention_kv8(c.cfg, q, c.dev["k"], c.dev["v"], 1, 500, 1, out, pf.attention_kv8_scratch(c.cfg, 1), torch.from_numpy(t).cuda(), c.status)
    pf.pf_status_read(c.status)


# ------------------------------------------------------------------ sessions
def oracle_with_8_bits(monkeypatch, kind):
    """The oracle's attention reads K and V as the 8-bit cache holds them: the rows it has just stored (f16
    values) are quantised in place, block by block, before the attention."""
    state, plain = {}, O.causal_gqa_attention

    def attention(q, k, v, start, window=None, sinks=0):
        for x in (k, v):
            key = x.__array_interface__["data"][0]
            nkv, n, hd = x.shape
            codes, scales = state.setdefault(key, (np.zeros(x.shape, np.uint8), np.zeros((nkv, -(-n // R.BLOCK)), np.float32)))
            m = q.shape[0]
            R.store(kind, codes, scales, x[:, start:start + m].transpose(1, 0, 2), start)
            x[:, :start + m] = R.values(kind, codes, scales)[:, :start + m]
        return plain(q, k, v, start, window, sinks)

    monkeypatch.setattr(O, "causal_gqa_attention", attention)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("paged", [False, True])
def test_session_over_an_8_bit_cache(monkeypatch, kind, paged):
    """A small stack in chunks and decoded tokens: hidden rows and logits within 2e-2 of the oracle with the
    same cache (f16 operands before the rounding to 8 bits: a code that falls on the other side of a rounding
    border moves one element by a step, which the bound covers as it does for the 16-bit caches)."""
    s = dataclasses.replace(synth.TINY, n_layers=2, vocab=5000, max_seq=400, kv_dtype="f16")
    layers, extra = synth.model_inputs(s)
    toks = synth.tokens(230, s.vocab, seed=1)
    oracle_with_8_bits(monkeypatch, kind)
    g = dataclasses.replace(s, kv_dtype=kind)
    dm = pf.DeviceModel(g, layers, extra, max_chunk=96, kv_block_pool=5 if paged else 0)
    sess = pf.Session(dm, block_table=[4, 0, 3, 1] if paged else None)
    om = O.OracleModel(s, layers, extra)
    logits = torch.empty(s.vocab, device="cuda")
    ids = torch.from_numpy(toks.astype(np.int32)).cuda()
    at = 0
    for m in (90, 7, 130, 1, 1, 1):
        want = None
        for o in range(0, m, 96):
            n = min(96, m - o)
            _, want = om.forward_chunk(om.embed(toks[at + o:at + o + n]), at + o, o + n == m)
        if m == 1:
            sess.decode_step(ids[at:at + 1], logits)
        else:
            sess.prefill_chunk(toks[at:at + m], at, logits)
        sess.sync()
        at += m
        assert O.rel_l2(logits.cpu().numpy(), want) <= 2e-2
    assert sess.position == 230


def test_score_over_an_8_bit_session_matches_verify_and_logprobs():
    """The whole path together: a prompt prefilled into an 8-bit cache, a chunk scored, against verify's logits."""
    s = dataclasses.replace(synth.TINY, n_layers=2, vocab=5000, max_seq=400, kv_dtype="e4m3")
    layers, extra = synth.model_inputs(s)
    toks = synth.tokens(200, s.vocab, seed=4)
    ids = torch.from_numpy(toks.astype(np.int32)).cuda()
    sess = pf.Session(pf.DeviceModel(s, layers, extra, max_chunk=128))
    sess.prefill_chunk(toks[:100], 0)
    m = 60
    logits = torch.empty(m, s.vocab, device="cuda")
    lp, ent, top_lp = torch.empty(m, device="cuda"), torch.empty(m, device="cuda"), torch.empty(m, 4, device="cuda")
    top = torch.empty(m, 4, dtype=torch.int32, device="cuda")
    sess.prefill_score(ids[100:160], ids[101:161], 100, logits, lp, ent, 4, top, top_lp)
    sess.sync()
    assert sess.position == 160
    ref = torch.log_softmax(logits.double(), 1)
    want = ref.gather(1, ids[101:161].long()[:, None])[:, 0]
    assert float((lp.double() - want).abs().max()) <= 1e-5 * float(want.abs().max())
    assert float((ent.double() + (ref.exp() * ref).sum(1)).abs().max()) <= 1e-4
    assert torch.equal(top[:, 0].long(), logits.argmax(1))
    assert torch.equal(top_lp[:, 0] >= top_lp[:, 1], torch.ones(m, dtype=torch.bool, device="cuda"))
    # verify on the same chunk gives the same logits up to the order of the GEMMs' additions
    sess.set_position(100)
    again, greedy = torch.empty_like(logits), torch.empty(m, dtype=torch.int32, device="cuda")
    sess.prefill_verify(ids[100:160], 100, again, greedy)
    sess.sync()
    assert float((again - logits).norm() / logits.norm()) <= 2e-3
    with pytest.raises(pf.PfError) as e:
        bad = ids[161:191].clone()
        bad[3] = s.vocab
        sess.prefill_score(ids[160:190], bad, 160, logits, lp)
        sess.sync()
    assert e.value.status == 5 and bool(torch.isnan(lp[3])) and not bool(torch.isnan(lp[:30]).all())
