"""What the binding's 8-bit and logits calls hand to the library for views of wider buffers, and which they
refuse: on host tensors, with the library's calls recorded."""
import dataclasses

import pytest

from quantized_transformer_prefill_q1_gb300 import pf, synth

torch = pytest.importorskip("torch")


class Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.startswith("pf_op_"):
            return lambda *a: self.calls.append((name, a)) or 0
        return getattr(self.real, name)


@pytest.fixture
def lib(monkeypatch):
    r = Recorder(pf.lib())
    monkeypatch.setattr(pf, "lib", lambda: r)
    monkeypatch.setattr(pf, "_here", lambda: -1)  # a host tensor's device
    monkeypatch.setattr(pf, "_torch", torch)
    return r


def refused(f):
    with pytest.raises(pf.PfError) as e:
        f()
    assert e.value.status == 1


def test_logits_as_a_view_of_wider_rows(lib):
    buf = torch.zeros(6, 40)
    tok, lp = torch.zeros(6, dtype=torch.int32), torch.zeros(6)

    def call(x, rows, n, ld):
        pf.pf_op_logprobs(x, rows, n, ld, tok, lp, stream=0)
        name, a = lib.calls.pop()
        assert name == "pf_op_logprobs" and a[1:4] == (rows, n, ld)
        return a[0]

    assert call(buf, 6, 33, 40) == buf.data_ptr()
    assert call(buf[:, :33], 6, 33, 40) == buf.data_ptr()
    assert call(buf[1:4, 5:38], 3, 33, 40) == buf.data_ptr() + 4 * 45
    assert call(buf[::2, :33], 3, 33, 80) == buf.data_ptr()
    assert call(buf[2:3, :33], 1, 33, 33) == buf.data_ptr() + 4 * 80  # one row: no next one
    assert call(buf[5], 1, 40, 40) == buf[5].data_ptr()
    assert call(buf[:, :1], 6, 1, 40) == buf.data_ptr()
    for x, rows, n, ld in [(buf[:, :33], 6, 34, 40),      # a wider row than the view has
                           (buf[:, :33], 7, 33, 40),      # more rows
                           (buf[:, :33], 6, 33, 33),      # another distance of the rows
                           (buf[:, ::2], 6, 20, 40),      # values apart
                           (buf.t()[:, :5], 40, 5, 40),
                           (buf[:, :33].double(), 6, 33, 33), (None, 6, 33, 40), (buf, 7, 40, 40)]:
        refused(lambda: pf.pf_op_logprobs(x, rows, n, ld, tok.repeat(7), lp.repeat(7), stream=0))
    assert not lib.calls


def test_strides_of_single_tokens_and_heads_do_not_count(lib):
    def call(nkv, k, v):
        cfg = pf.make_config(dataclasses.replace(synth.QWEN3_8B_LAYER, kv_dtype="int8", n_q_heads=8, n_kv_heads=nkv), 64, max_seq=64)
        cache = pf.kv8_cache(cfg, device="cpu")
        pf.pf_op_kv8_store(cfg, k, v, 0, 0, k.shape[0], cache, cache, stream=0)
        name, a = lib.calls.pop()
        assert name == "pf_op_kv8_store" and a[1:3] == (k.data_ptr(), v.data_ptr())
        return a[3:5]

    x = torch.zeros(9, 16, 128, dtype=torch.float16)  # 8 K heads, then 8 V heads
    odd = torch.zeros(9 * 2048 + 4, dtype=torch.float16)
    assert call(8, x[:, :8], x[:, 8:]) == (2048, 128)
    assert call(8, x[:1, :8], torch.zeros(1, 8, 128, dtype=torch.float16))[1] == 128  # token strides 2048 and 1024
    assert call(1, x[:, :1], odd.as_strided((9, 1, 128), (2048, 3, 1)))[0] == 2048     # head strides 128 and 3
    assert call(1, odd.as_strided((1, 1, 128), (5, 3, 1)), x[:1, :1]) == (0, 0)
    one = torch.zeros(9, 8, 128, dtype=torch.float16)
    for k, v in [(x[:, :8], one), (one, one.transpose(0, 1).contiguous().transpose(0, 1)), (x[:, :8], x[:, 8:, :64]),
                 (one.reshape(72, 128), one.reshape(72, 128)), (one.float(), one.float()),
                 (x.as_strided((9, 8, 128), (2048, 128, 0)), one), (one, x.as_strided((9, 8, 128), (1024, 128, 0)))]:
        refused(lambda: call(8, k, v))
    assert not lib.calls


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_views_give_what_the_buffers_give():
    buf = torch.randn(6, 4100, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    tok = torch.arange(6, dtype=torch.int32, device="cuda") * 600
    got = []
    for x in (buf, buf[:, :4001], buf[:6, :4100]):
        lp, ids = torch.empty(6, device="cuda"), torch.empty(6, 5, dtype=torch.int32, device="cuda")
        pf.pf_op_logprobs(x, 6, 4001, 4100, tok, lp, None, 5, ids)
        got.append((lp, ids))
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(g, got[0]))
    cfg = pf.make_config(dataclasses.replace(synth.QWEN3_8B_LAYER, kv_dtype="e4m3"), 64, max_seq=64)
    kv = torch.randn(9, 16, 128, device="cuda").half()
    caches = []
    for k, v in ((kv[4:5, :8], kv[4:5, 8:].contiguous()), (kv[4:5, :8].contiguous(), kv[4:5, 8:].contiguous())):
        caches.append((pf.kv8_cache(cfg), pf.kv8_cache(cfg)))
        pf.pf_op_kv8_store(cfg, k, v, 0, 0, 1, *caches[-1])
    assert all(torch.equal(a, b) for a, b in zip(*caches)) and bool(caches[0][0].any())
