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
