"""Refusals on the host of the calls on rows grouped by owner (no GPU needed)."""
import ctypes

import pytest

P = 0x10000          # a pointer that is never followed


@pytest.fixture(scope="module")
def ep():
    from combine_layout_02_gb300 import build
    build.build()
    import combine_layout_02_gb300 as ep
    ep.lib()
    return ep


def test_selftest_of_the_products_waits(ep):
    launch, sh = ep.ep_launch(None, None, None, P), ep.ep_gemm_shape(10, 2, 64, 64)

    def call(shape=sh, product=0, rows=P, other=P, prefix=P, out=P, loads=64, ms=20, launch=launch):
        r = ctypes.byref
        return ep.lib().ep_selftest_gemm_timeout(r(shape), product, rows, other, prefix, out, loads, ms, r(launch))

    for bad in (dict(product=3), dict(product=-1), dict(loads=-64), dict(loads=32), dict(ms=0), dict(ms=10001),
                dict(launch=ep.ep_launch(None, None, None, None)), dict(shape=ep.ep_gemm_shape(10, 2, 60, 64)),
                dict(rows=None), dict(other=P + 8), dict(prefix=None), dict(out=None)):
        assert call(**bad) == ep.EP_ERR_INVALID_ARG, bad
