"""Argument checks of the weight gradient's weight and bias, without a GPU."""
from ctypes import byref

import pytest

from test_ops_refusals import L, P, WGRAD, call, ckpt, fields  # noqa: F401


@pytest.mark.parametrize("kw,word", [(dict(w_dtype=2), "type"), (dict(w_dtype=-1), "type"),
                                     (dict(w_dtype=1, weight=P + 1), "aligned"),
                                     (dict(w_dtype=1, bias=P + 1), "aligned"),
                                     (dict(w_dtype=0, weight=P + 2), "aligned")])
def test_weight_grad_refuses_weights(L, kw, word):  # noqa: F811
    a = fields(L.WeightGradArgs, WGRAD, **kw)
    a.saved = ckpt(L)
    rc, msg = call(L, "muon_weight_grad", byref(a), P, 1 << 40)
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg


def test_bf16_weights_need_a_workspace(L):  # noqa: F811
    import ctypes
    sizes = []
    for kw in (dict(), dict(weight=P), dict(weight=P + 2, w_dtype=1)):
        a = fields(L.WeightGradArgs, WGRAD, **kw)
        n = ctypes.c_size_t()
        assert L.lib().muon_weight_grad_workspace(byref(a), byref(n)) == 0
        sizes.append(n.value)
    assert sizes == [0, 0, 256]
