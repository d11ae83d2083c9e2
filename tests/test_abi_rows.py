"""Refusals of the operators on rows grouped by owner: every bad argument is rejected on the host
before any CUDA work (no GPU needed), and the workspace sizes."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ep():
    from combine_layout_02_gb300 import build
    build.build()
    import combine_layout_02_gb300 as ep
    ep.lib()
    return ep


P = 0x10000          # a pointer that is never followed


def refused(ep, name, shape, *args):
    r = ctypes.byref
    return getattr(ep.lib(), name)(r(shape), *[r(a) if isinstance(a, ctypes.Structure) else a for a in args])


def test_sort_refusals(ep):
    launch = ep.ep_launch(None, None, None, None)
    sh = ep.make_shape(1, 4000, 256, 16, 4)
    ok = ep.ep_sort(P, P, P, 16000)
    size = ep.ep_sort_workspace_size(sh)
    bad, unsup = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED

    def layout(shape=sh, idx=P, sort=ok, ws=P, n=size):
        return refused(ep, "ep_sort_layout", shape, idx, sort, ws, n, launch)

    assert layout(shape=ep.make_shape(2, 4000, 256, 16, 4)) == bad                  # one rank's rows
    assert layout(shape=ep.make_shape(1, 4000, 200, 16, 4)) == bad
    assert layout(shape=ep.make_shape(1, 4000, 256, 9000, 4)) == unsup
    assert layout(shape=ep.make_shape(1, 1 << 28, 256, 16, 8)) == unsup             # N*k beyond 2^30
    assert layout(idx=None) == bad and layout(ws=None) == bad and layout(ws=P + 8) == bad and layout(n=size - 1) == bad
    assert layout(sort=ep.ep_sort(None, P, P, 16000)) == bad
    assert layout(sort=ep.ep_sort(P, P, None, 16000)) == bad
    assert layout(sort=ep.ep_sort(P, P, P, -1)) == bad
    L = ep.lib()
    assert L.ep_sort_layout(ctypes.byref(sh), P, ctypes.byref(ok), P, size, None) == bad
    assert L.ep_sort_layout(ctypes.byref(sh), P, None, P, size, ctypes.byref(launch)) == bad

    def rows(x=P, dtype=ep.EP_BF16, sc=None, fmt=0, sort=ok, out=P, osc=None, shape=sh):
        return refused(ep, "ep_sort_rows", shape, x, dtype, sc, fmt, sort, out, osc, launch)

    assert rows(x=None) == bad and rows(out=None) == bad and rows(x=P + 8) == bad and rows(out=P + 2) == bad
    assert rows(dtype=2) == bad and rows(fmt=7) == bad and rows(fmt=-1) == bad
    assert rows(sc=P, osc=P) == bad                                                 # bf16 rows have no scales
    assert rows(dtype=ep.EP_FP8_E4M3, sc=P) == bad and rows(dtype=ep.EP_FP8_E4M3, osc=P) == bad
    assert rows(dtype=ep.EP_FP8_E4M3, sc=P + 1, osc=P) == bad
    assert rows(sort=ep.ep_sort(None, P, P, 16000)) == bad

    def back(y=P, w=P, sort=ok, out=P):
        return refused(ep, "ep_unsort_rows", sh, y, w, sort, out, launch)

    assert back(y=None) == bad and back(out=None) == bad and back(y=P + 4) == bad and back(out=P + 8) == bad
    assert back(sort=ep.ep_sort(None, P, P, 16000)) == bad

    def grad(dout=P, y=P, w=P, sort=ok, dy=P, dw=P):
        return refused(ep, "ep_unsort_rows_backward", sh, dout, y, w, sort, dy, dw, launch)

    assert grad(dout=None) == bad and grad(y=None) == bad and grad(dy=None, dw=None) == bad
    assert grad(dout=P + 8) == bad and grad(y=P + 8) == bad and grad(dy=P + 8) == bad


def test_expert_gemm_refusals(ep):
    launch = ep.ep_launch(None, None, None, None)
    bad, unsup = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    S = ep.ep_gemm_shape
    for name in ("ep_expert_gemm", "ep_expert_gemm_dgrad", "ep_expert_gemm_wgrad"):
        def call(shape=S(10, 2, 64, 64), a=P, b=P, prefix=P, out=P):
            return refused(ep, name, shape, a, b, prefix, out, launch)
        for s in (S(-1, 2, 64, 64), S(10, 0, 64, 64), S(10, 2, 60, 64), S(10, 2, 64, 0), S(10, 2, 64, 12)):
            assert call(shape=s) == bad
        for s in (S(10, 9000, 64, 64), S(10, 2, (1 << 20) + 8, 64), S(10, 2, 64, (1 << 20) + 8), S((1 << 30) + 1, 2, 64, 64)):
            assert call(shape=s) == unsup
        assert call(a=None) == bad and call(b=None) == bad and call(prefix=None) == bad and call(out=None) == bad
        assert call(a=P + 8) == bad and call(b=P + 2) == bad and call(out=P + 8) == bad and call(prefix=P + 2) == bad
        assert getattr(ep.lib(), name)(None, P, P, P, P, ctypes.byref(launch)) == bad
        assert getattr(ep.lib(), name)(ctypes.byref(S(10, 2, 64, 64)), P, P, P, P, None) == bad


def test_adapter_refusals(ep):
    launch = ep.ep_launch(None, None, None, None)
    bad, unsup = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED
    S = ep.ep_adapter_shape
    good = S(10, 64, 64, 3, 16)
    size = ep.ep_adapter_workspace_size(good)

    def call(shape=good, x=P, w=P, a=P, b=P, s=P, ids=P, y=P, ws=P, n=size):
        return refused(ep, "ep_adapter_gemm", shape, x, w, a, b, s, ids, y, ws, n, launch)

    for s in (S(-1, 64, 64, 3, 16), S(10, 60, 64, 3, 16), S(10, 64, 0, 3, 16), S(10, 64, 64, -1, 16), S(10, 64, 64, 3, 12),
              S(10, 64, 64, 3, 0)):
        assert call(shape=s) == bad and ep.ep_adapter_workspace_size(s) == 0
    for s in (S(10, 64, 64, 3, 264), S(10, 64, 64, 8193, 16), S(10, (1 << 20) + 8, 64, 3, 16), S((1 << 30) + 1, 64, 64, 3, 16)):
        assert call(shape=s) == unsup and ep.ep_adapter_workspace_size(s) == 0
    for name in ("x", "w", "a", "b", "s", "ids", "y", "ws"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: P + 2}) == bad, name
    assert call(n=size - 1) == bad


def test_workspace_sizes(ep):
    assert ep.ep_sort_workspace_size(ep.make_shape(1, 128, 256, 16, 4)) == 16            # one block, no scratch
    n, E = 20000 * 8, 32
    assert ep.ep_sort_workspace_size(ep.make_shape(1, 20000, 256, E, 8)) == (-(-n // 128) + 1) * E * 4
    assert ep.ep_sort_workspace_size(ep.make_shape(2, 128, 256, 16, 4)) == 0
