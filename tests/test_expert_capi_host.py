"""Host-side refusals of the router, expert-order and expert-product calls: they
return a status and a message without a GPU and without touching memory."""

import ctypes

import pytest

from tests.test_capi_host import capi  # noqa: F401

P = ctypes.c_void_p(256)  # never read: the calls are refused first


def calls(C):
    gate = C.moedx_gate(0, 1, 1, 0, 1.0, None)
    er = C.moedx_expert_rows(P, None, 8)
    g, e, n = ctypes.byref(gate), ctypes.byref(er), ctypes.c_size_t()
    return {
        "gate_topk": lambda: C.moedx_gate_topk(None, P, 0, 4, 2, g, P, P, None),
        "gate_topk_backward": lambda: C.moedx_gate_topk_backward(None, P, 0, 4, 2, g, P, P, P, None),
        "order_bytes": lambda: C.moedx_expert_order_workspace_bytes(None, 4, 2, ctypes.byref(n)),
        "order": lambda: C.moedx_expert_order(None, P, 4, 2, None, P, P, P, P, 4096, None),
        "sort": lambda: C.moedx_expert_sort(None, P, 0, 4, 2, 8, P, P, None),
        "unsort": lambda: C.moedx_expert_unsort(None, P, 0, 4, 2, 8, P, P, P, None),
        "unsort_backward": lambda: C.moedx_expert_unsort_backward(None, P, P, 0, 4, 2, 8, P, P, P, P,
                                                                  P, None),
        "linear": lambda: C.moedx_expert_linear(None, P, P, 0, 8, 8, e, 0, P, None, None),
        "linear_backward": lambda: C.moedx_expert_linear_backward(None, P, P, P, 0, 8, 8, e, P, P, 0,
                                                                  None),
        "swiglu_backward": lambda: C.moedx_expert_swiglu_backward(None, P, P, 0, 8, e, P, None),
    }


@pytest.mark.parametrize("name", ["gate_topk", "gate_topk_backward", "order_bytes", "order", "sort",
                                  "unsort", "unsort_backward", "linear", "linear_backward",
                                  "swiglu_backward"])
def test_null_ctx(capi, name):  # noqa: F811
    assert calls(capi)[name]() == capi.MOEDX_EINVAL
    assert capi.last_error()
