"""Calls over many sequences without a GPU: what would reach a kernel that cannot take it is refused."""
import ctypes

import pytest

from quantized_transformer_prefill_q1_gb300 import pf
from test_batch_host import P, batch, config, lib  # noqa: F401


def refused(f, *args):
    return pf.STATUS[f(*args)]


@pytest.mark.parametrize("off", [1, 2, 3])
def test_words_off_their_alignment(lib, off):  # noqa: F811
    """Each array of 4-byte numbers, one after the other, at an address that is no multiple of 4."""
    linear, paged = ctypes.byref(config()), ctypes.byref(config(pool=20))

    def calls(b, **kw):
        w = {**dict.fromkeys(("status", "tokens", "ids", "root", "path", "count", "adapter", "scale"), P), "after": 2 * P, **kw}
        c = paged if b.block_table_dev else linear
        b = ctypes.byref(b)
        return {"append": (lib.pf_op_batch_append, c, b, P, P, P, P, 1, P, P, P, w["status"], None),
                "attention": (lib.pf_op_attention_tree, c, b, P, P, P, 1, 2 * P, P, 1 << 40, w["status"], None),
                "accept": (lib.pf_op_tree_accept, c, b, w["tokens"], w["ids"], w["root"], w["path"], w["count"], w["after"], P, P, w["status"], None),
                "adapters": (lib.pf_op_adapters, b, P, 64, P, 32, 2 * P, 32, 64, 32, 8, 2, w["adapter"], P, P, w["scale"], w["status"], None)}

    for field in ("row_begin_dev", "start_dev", "parent_dev", "block_table_dev"):
        for name, call in calls(batch(**{"n_seq": 1, field: P + off})).items():
            assert refused(*call) == "PF_ERR_INVALID_ARG" and b"4-B" in lib.pf_last_error(), (field, name)
    for name, words in (("append", ("status",)), ("attention", ("status",)), ("accept", ("tokens", "ids", "root", "path", "count", "after", "status")),
                        ("adapters", ("adapter", "scale", "status"))):
        for word in words:
            assert refused(*calls(batch(), **{word: P + off})[name]) == "PF_ERR_INVALID_ARG" and b"4-B" in lib.pf_last_error(), (name, word)


def test_adapters_of_the_widest_rows(lib):  # noqa: F811
    """K and N above 2^26, where a tile's elements or the columns rounded up would pass 32 bits."""
    def adapters(k, n):
        b = ctypes.byref(batch(n_rows=64, max_rows=64))
        return refused(lib.pf_op_adapters, b, P, k, P, n, 2 * P, n, k, n, 8, 1, P + 1, P, P, P, None, None)

    for k, n in ((2 ** 26 + 16, 32), (64, 2 ** 26 + 8), (2 ** 31 - 16, 32), (64, 2 ** 31 - 8), (64, 2 ** 27)):
        assert adapters(k, n) == "PF_ERR_SHAPE", (k, n)
    assert adapters(2 ** 26, 2 ** 26) == "PF_ERR_INVALID_ARG"  # the adapters' address, looked at later
