"""What moedx_expert_linear_int8 says when it refuses a call: its messages name the
caller's own sizes and the limit that was passed.  Refused calls touch nothing,
so the pointers here are never followed."""

import ctypes

import pytest

from tests.gpu_common import device, make_buffer

pytestmark = pytest.mark.gpu


@pytest.fixture
def linear():
    """The call over one expert's rows, with pointers that no call may follow."""
    from combine_get_dispatch_layout_amd import _capi as C
    device()
    buf = make_buffer(1, 1, 1, 1)

    def call(K, N, rows, swiglu=0):
        er = C.moedx_expert_rows(ctypes.c_void_p(4096), None, rows)
        p = [ctypes.c_void_p((1 << 44) + (k << 42)) for k in range(5)]
        rc = C.moedx_expert_linear_int8(buf.ctx, *p[:4], K, N, ctypes.byref(er), swiglu, p[4],
                                        C.MOEDX_BF16, None)
        return rc, C.last_error()

    call.ok, call.refused = C.MOEDX_OK, C.MOEDX_EINVAL
    return call


@pytest.mark.parametrize("K,N,swiglu", [(65536, 32768, 0), (65536, 16384, 1), (16, 1 << 20, 0),
                                        (2048, 1 << 20, 0), (131056, 16392, 0)])
def test_weights_past_2_gib(linear, K, N, swiglu):
    """An expert's N (2N gated) rows of K codes: K bytes each."""
    too_large = K * N * (2 if swiglu else 1) >= 1 << 31
    rc, said = linear(K, N, 0, swiglu)  # no rows: nothing is launched
    if not too_large:
        assert rc == linear.ok, said
        return
    assert rc == linear.refused
    assert f"N={N}, K={K}" in said and "2^31 bytes" in said, said
    # the next smaller product is taken
    assert linear(K, N - 8 if not swiglu else N - 16, 0, swiglu)[0] == linear.ok


def test_too_many_tiles(linear):
    """The limit is 2^23 tiles of 256 x 256, not the workgroups that the call would
    launch (512 at most)."""
    M = (1 << 31) - 1
    rc, said = linear(16, 8, M)
    assert rc == linear.refused
    assert f"rows={M}" in said and "2^23" in said and "256 x 256" in said, said
    assert "workgroups than a grid has" not in said, said
