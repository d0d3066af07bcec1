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


@pytest.mark.gpu
def test_views_give_what_the_buffers_give():
    buf = torch.randn(6, 4100, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    tok = torch.arange(6, dtype=torch.int32, device="cuda") * 600
    got = []
    for x in (buf, buf[:, :4001], buf[:6, :4100]):
        lp, ids = torch.empty(6, device="cuda"), torch.empty(6, 5, dtype=torch.int32, device="cuda")
        pf.pf_op_logprobs(x, 6, 4001, 4100, tok, lp, None, 5, ids)
        got.append((lp, ids))
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(g, got[0]))
