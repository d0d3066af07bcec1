"""The calls over many sequences without a GPU: sizes and every refusal before anything is launched."""
import ctypes
import dataclasses

import pytest

from quantized_transformer_prefill_q1_gb300 import pf, synth

P = 4096  # an aligned address that no refused call follows


@pytest.fixture(scope="module")
def lib():
    return pf.lib()


def config(kind="bf16", pool=0, **kw):
    names = {k: kw.pop(k) for k in list(kw) if k in ("n_q_heads", "n_kv_heads", "head_dim", "qk_norm")}
    s = dataclasses.replace(synth.QWEN3_8B_LAYER, kv_dtype=kind, **names)
    return pf.make_config(s, 256, n_layers=2, max_seq=kw.pop("max_seq", 1000), kv_block_pool=pool, **kw)


def batch(**kw):
    return pf.pf_batch(**{**dict(n_seq=1, n_rows=10, max_rows=10, row_begin_dev=P, start_dev=P, parent_dev=P, block_table_dev=None), **kw})


def name(st):
    return pf.STATUS[st]


def append(lib, c=None, b=None, qkv=P, qn=P, kn=P, rope=P, layer=1, q=P, kc=P, vc=P):
    c, b = c or config(), b if b is not None else batch()
    return name(lib.pf_op_batch_append(ctypes.byref(c), ctypes.byref(b) if b else None, qkv, qn, kn, rope, layer, q, kc, vc, None, None))


def attend(lib, c=None, b=None, q=P, kc=P, vc=P, layer=1, out=2 * P, scratch=P, nbytes=1 << 40):
    c, b = c or config(), b if b is not None else batch()
    return name(lib.pf_op_attention_tree(ctypes.byref(c), ctypes.byref(b) if b else None, q, kc, vc, layer, out, scratch, nbytes, None, None))


def accept(lib, c=None, b=None, tokens=P, ids=P, root=P, path=P, count=P, after=2 * P, kc=P, vc=P):
    c, b = c or config(), b if b is not None else batch()
    return name(lib.pf_op_tree_accept(ctypes.byref(c), ctypes.byref(b) if b else None, tokens, ids, root, path, count, after, kc, vc, None, None))


def adapters(lib, b=None, x=P, ldx=64, base=P, ldb=32, out=2 * P, ldo=32, k=64, n=32, rank=8, count=2, adapter=P, wa=P, wb=P, scale=P):
    b = b if b is not None else batch()
    return name(lib.pf_op_adapters(ctypes.byref(b) if b else None, x, ldx, base, ldb, out, ldo, k, n, rank, count, adapter, wa, wb, scale,
                                   None, None))


@pytest.mark.parametrize("call", [append, attend, accept])
def test_batch_refusals(lib, call):
    assert call(lib, b=False) == "PF_ERR_INVALID_ARG"
    for kw, want in ((dict(n_seq=0), "PF_ERR_SHAPE"), (dict(n_seq=1025), "PF_ERR_SHAPE"), (dict(n_rows=0), "PF_ERR_EMPTY_CHUNK"),
                     (dict(n_rows=-1), "PF_ERR_SHAPE"), (dict(max_rows=0), "PF_ERR_SHAPE"), (dict(max_rows=257), "PF_ERR_SHAPE"),
                     (dict(row_begin_dev=None), "PF_ERR_INVALID_ARG"), (dict(start_dev=None), "PF_ERR_INVALID_ARG"),
                     (dict(block_table_dev=P), "PF_ERR_INVALID_ARG"), (dict(n_seq=2), "PF_ERR_UNSUPPORTED"),
                     (dict(n_rows=2 ** 31 - 1), "PF_ERR_SHAPE")):
        assert call(lib, b=batch(**kw)) == want, kw
    paged = config(pool=20)
    assert call(lib, c=paged) == "PF_ERR_INVALID_ARG"  # no table
    for c, want in ((config("f32"), "PF_ERR_UNSUPPORTED"), (config("e4m3"), "PF_ERR_UNSUPPORTED"), (config("int8"), "PF_ERR_UNSUPPORTED"),
                    (config(ring_capacity=256, sink_count=4), "PF_ERR_UNSUPPORTED"), (config(max_seq=2 ** 27), "PF_ERR_SHAPE"),
                    (config(max_seq=0), "PF_ERR_SHAPE")):
        assert call(lib, c=c) == want
    if call is not accept:
        assert call(lib, layer=2) == "PF_ERR_SHAPE" and call(lib, layer=-1) == "PF_ERR_SHAPE"


def test_pointer_refusals(lib):
    for kw in ("qkv", "qn", "kn", "rope", "q", "kc", "vc"):
        assert append(lib, **{kw: None}) == "PF_ERR_INVALID_ARG", kw
        assert append(lib, **{kw: P + 4}) == "PF_ERR_INVALID_ARG", kw
    for kw in ("q", "kc", "vc", "out"):
        assert attend(lib, **{kw: None}) == "PF_ERR_INVALID_ARG", kw
        assert attend(lib, **{kw: P + 8}) == "PF_ERR_INVALID_ARG", kw
    assert attend(lib, out=P) == "PF_ERR_INVALID_ARG"  # q
    assert attend(lib, scratch=None) == "PF_ERR_WORKSPACE"
    assert attend(lib, scratch=P + 4) == "PF_ERR_INVALID_ARG"
    need = lib.pf_attention_tree_scratch_bytes(ctypes.byref(config()), 1, 10)
    assert need > 0 and attend(lib, nbytes=need - 1) == "PF_ERR_WORKSPACE"
    for kw in ("tokens", "ids", "root", "path", "count", "after", "kc", "vc"):
        assert accept(lib, **{kw: None}) == "PF_ERR_INVALID_ARG", kw
    assert accept(lib, kc=P + 8) == "PF_ERR_INVALID_ARG"
    assert accept(lib, after=P) == "PF_ERR_INVALID_ARG"  # the root ids


def test_adapter_refusals(lib):
    assert adapters(lib, b=False) == "PF_ERR_INVALID_ARG"
    for kw in ("x", "base", "out", "adapter", "wa", "wb", "scale"):
        assert adapters(lib, **{kw: None}) == "PF_ERR_INVALID_ARG", kw
    for kw in ("x", "base", "out", "wa", "wb"):
        assert adapters(lib, **{kw: P + 8}) == "PF_ERR_INVALID_ARG", kw
    for kw in (dict(rank=0), dict(rank=12), dict(rank=136), dict(k=0), dict(k=24), dict(n=0), dict(n=12), dict(count=0), dict(count=2 ** 28), dict(ldx=56), dict(ldx=68),
               dict(ldb=28), dict(ldb=34), dict(ldo=28), dict(ldo=33), dict(out=P, ldo=36), dict(b=batch(max_rows=8193)), dict(b=batch(n_seq=2000))):
        assert adapters(lib, **kw) == "PF_ERR_SHAPE", kw
    assert adapters(lib, b=batch(n_rows=0)) == "PF_ERR_EMPTY_CHUNK"


def test_attention_counts(lib):
    """The work of the longest sequences possible stays below 2^31 units."""
    big = config(pool=4, max_seq=2 ** 24)
    paged = dict(block_table_dev=P, n_rows=4000)
    assert attend(lib, c=big, b=batch(n_seq=511, **paged), nbytes=0) == "PF_ERR_WORKSPACE"  # 511 * 8 * (2^19 + 16)
    assert attend(lib, c=big, b=batch(n_seq=512, **paged), nbytes=0) == "PF_ERR_SHAPE"
    assert attend(lib, c=big, b=batch(n_seq=256, **{**paged, "max_rows": 65}), nbytes=0) == "PF_ERR_SHAPE"  # two blocks of 256 rows
    assert attend(lib, c=big, b=batch(n_seq=255, **{**paged, "max_rows": 65}), nbytes=0) == "PF_ERR_WORKSPACE"


def test_sizes(lib):
    c = ctypes.byref(config(pool=20))
    for n_seq, rows in ((0, 1), (1025, 1), (1, 0), (1, 257)):
        assert lib.pf_attention_tree_scratch_bytes(c, n_seq, rows) == 0
    last = 0
    for n_seq in (1, 2, 7, 48, 333, 1024):
        row = [lib.pf_attention_tree_scratch_bytes(c, n_seq, r) for r in (1, 2, 4, 5, 16, 33, 64, 65, 256)]
        assert row == sorted(row) and row[0] >= last > -1
        last = row[0]


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")

    def refused(f):
        with pytest.raises(pf.PfError) as e:
            f()
        assert e.value.status == 1
    t = torch.zeros(4, dtype=torch.int32)
    refused(lambda: pf.Batch(t, n_rows=3, max_rows=3))
    refused(lambda: pf.Batch(None, n_rows=3, max_rows=3))
    refused(lambda: pf.Batch(t.reshape(2, 2), n_rows=3, max_rows=3))
