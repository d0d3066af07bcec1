"""8-bit cache and log probabilities without a GPU: sizes, configuration checks, every refusal (before
any launch: the addresses below are never read), and the numpy definition against torch's casts."""
import ctypes
import dataclasses
import os

import numpy as np
import pytest

import kv8_reference as R
from quantized_transformer_prefill_q1_gb300 import pf, synth

P = 0x10000  # a 16-B aligned address that nothing may read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pf.LIB_PATH):
        from quantized_transformer_prefill_q1_gb300 import build
        build.build()
    return pf.lib()


def cfg8(kind="e4m3", **kw):
    s = dataclasses.replace(synth.QWEN3_8B_LAYER, kv_dtype=kind)
    return pf.make_config(s, 512, **kw)


def byref(c):
    return ctypes.byref(c)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_sizes(lib, kind):
    c = cfg8(kind, n_layers=3, max_seq=1001)
    codes = 3 * 8 * 1001 * 128
    assert lib.pf_kv8_scales_offset(byref(c)) == -(-codes // 256) * 256
    assert lib.pf_kv_bytes(byref(c)) == -(-codes // 256) * 256 + 3 * 8 * 32 * 4  # ceil(1001 / 32) = 32
    c = cfg8(kind, n_layers=3, max_seq=1001, kv_block_pool=11)
    assert lib.pf_kv_bytes(byref(c)) == 3 * 8 * 1408 * 128 + 3 * 8 * 44 * 4
    assert lib.pf_workspace_bytes(byref(c)) > 0
    sizes = [lib.pf_attention_kv8_scratch_bytes(byref(c), m) for m in (1, 2, 3, 4, 5, 8, 16, 17, 32, 33, 64, 100, 512, 1001)]
    assert sizes[0] >= 4096 and sizes == sorted(sizes)
    assert lib.pf_attention_kv8_scratch_bytes(byref(c), 0) == 0
    b16 = pf.make_config(synth.QWEN3_8B_LAYER, 512)
    assert lib.pf_kv8_scales_offset(byref(b16)) == 0 and lib.pf_attention_kv8_scratch_bytes(byref(b16), 1) == 0


def test_configuration_checks(lib):
    assert lib.pf_config_check(byref(cfg8())) == 0
    assert lib.pf_config_check(byref(cfg8(kv_block_pool=40))) == 0
    assert lib.pf_config_check(byref(cfg8(ring_capacity=256, sink_count=4))) == 8  # no ring
    assert lib.pf_config_check(byref(cfg8(max_seq=(1 << 30) + 1))) == 2
    c = cfg8()
    c.n_q_heads = c.n_kv_heads = 2048
    assert lib.pf_config_check(byref(c)) == 2
    c = cfg8()
    c.kv_dtype = 5
    assert lib.pf_config_check(byref(c)) == 1
    # the 16 / 32-bit single steps do not take an 8-bit configuration
    assert lib.pf_op_qk_norm_rope_kv(byref(cfg8()), P, P, P, P, 0, 0, 1, P, P, P, None) == 8
    assert lib.pf_op_attention(byref(cfg8()), P, P, P, 0, 0, 1, P, None) == 8
    assert lib.pf_op_attention_split(byref(cfg8()), P, P, P, 0, 0, 1, 2, P, 1 << 30, P, None) == 8
    assert lib.pf_attention_scratch_bytes(byref(cfg8()), 1, 2) == 0
    assert lib.pf_status_name(12) == b"PF_ERR_NONFINITE"


def test_store_refusals(lib):
    c, pg = cfg8(max_seq=1000), cfg8(max_seq=1000, kv_block_pool=9)

    def call(cfg=c, k=P, v=P, ts=1024, hs=128, layer=0, start=0, m=5, table=None, kc=P, vc=P):
        return lib.pf_op_kv8_store(byref(cfg), k, v, ts, hs, layer, start, m, table, kc, vc, None, None)

    b16 = pf.make_config(synth.QWEN3_8B_LAYER, 512)
    for st, kw in [(8, dict(cfg=b16)), (1, dict(table=P)), (1, dict(cfg=pg)), (3, dict(m=0)), (3, dict(m=-1)),
                   (2, dict(layer=1)), (2, dict(layer=-1)), (6, dict(start=-1)), (6, dict(start=996)),
                   (6, dict(start=0x7fffffff, m=0x7fffffff)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(kc=None)),
                   (1, dict(vc=None)), (1, dict(k=P + 2)), (1, dict(v=P + 8)), (1, dict(kc=P + 1)), (1, dict(ts=4)),
                   (1, dict(hs=-128))]:
        assert call(**kw) == st, kw
        assert lib.pf_last_error()


def test_load_refusals(lib):
    c = cfg8(max_seq=1000)

    def call(cfg=c, cache=P, layer=0, start=0, m=5, table=None, out=P):
        return lib.pf_op_kv8_load(byref(cfg), cache, layer, start, m, table, out, None, None)

    for st, kw in [(1, dict(cache=None)), (1, dict(out=None)), (1, dict(out=P + 4)), (1, dict(table=P)), (3, dict(m=0)),
                   (2, dict(layer=1)), (6, dict(start=996))]:
        assert call(**kw) == st, kw


def test_attention_refusals(lib):
    c, pg = cfg8(max_seq=1000), cfg8(max_seq=1000, kv_block_pool=9)
    need = lib.pf_attention_kv8_scratch_bytes(byref(c), 5)

    def call(cfg=c, q=P, kc=P, vc=P, layer=0, start=0, m=5, table=None, out=P, scratch=P, nbytes=need):
        return lib.pf_op_attention_kv8(byref(cfg), q, kc, vc, layer, start, m, table, out, scratch, nbytes, None, None)

    for st, kw in [(8, dict(cfg=pf.make_config(synth.QWEN3_8B_LAYER, 512))), (1, dict(table=P)), (1, dict(cfg=pg)),
                   (3, dict(m=0)), (2, dict(layer=1)), (6, dict(start=996)), (6, dict(start=-1)), (1, dict(q=None)),
                   (1, dict(out=None)), (1, dict(kc=None)), (1, dict(vc=None)), (1, dict(q=P + 2)), (1, dict(out=P + 8)),
                   (11, dict(scratch=None)), (11, dict(nbytes=need - 1)), (1, dict(scratch=P + 4))]:
        assert call(**kw) == st, kw


def test_logprobs_refusals(lib):
    def call(x=P, rows=2, n=10, ld=10, tok=P, lp=P, ent=P, top=3, ids=P, tlp=P):
        return lib.pf_op_logprobs(x, rows, n, ld, tok, lp, ent, top, ids, tlp, None, None)

    for st, kw in [(1, dict(x=None)), (1, dict(tok=None)), (2, dict(rows=0)), (2, dict(n=0)), (2, dict(ld=9)),
                   (2, dict(top=-1)), (2, dict(top=33)), (1, dict(ids=None)), (1, dict(top=0)), (1, dict(top=0, ids=None)),
                   (1, dict(lp=None, ent=None, top=0, ids=None, tlp=None))]:
        assert call(**kw) == st, kw
    assert lib.pf_prefill_score(None, P, P, 1, 0, P, P, P, 0, None, None, None) == 1


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 10)
    with pytest.raises(pf.PfError) as e:
        pf.pf_op_logprobs(x, 2, 10, 10, None, None, x[0, :2])
    assert e.value.status == 1
    c = cfg8(max_seq=64)
    k = torch.zeros(2, 8, 128, dtype=torch.float16)
    with pytest.raises(pf.PfError) as e:
        pf.pf_op_kv8_store(c, k, k, 0, 0, 2, None, None)
    assert e.value.status == 1


def test_reference_codes_match_torch_casts():
    """The definition's e4m3 rounding and values against torch's type, over every f16 bit pattern in range,
    and int8's against a brute search of the nearest code."""
    torch = pytest.importorskip("torch")
    x = np.arange(1 << 16, dtype=np.uint16).view(np.float16).astype(np.float64)
    x = x[np.isfinite(x) & (np.abs(x) <= 448)]
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = R.encode("e4m3", x)
    assert np.array_equal(got, want)
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(R.decode("e4m3", codes), t.astype(np.float64), equal_nan=True)
    y = np.linspace(-127, 127, 4001)
    grid = np.arange(-127, 128)
    near = np.abs(y[:, None] - grid[None, :]).min(1)
    assert np.allclose(np.abs(R.decode("int8", R.encode("int8", y)) - y), near)
    assert R.decode("int8", R.encode("int8", [0.5, 1.5, -2.5, 126.5])).tolist() == [0, 2, -2, 126]
    for kind in ("e4m3", "int8"):
        assert R.exponent(kind, 0.0) == -32
        assert R.exponent(kind, R.CMAX[kind]) == 0 and R.exponent(kind, R.CMAX[kind] * 1.001) == 1
