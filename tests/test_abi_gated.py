"""Refusals of the gated feed-forward block and of the checkpoints in 8 bits: every bad argument is rejected
on the host before any CUDA work (no GPU needed), and the workspace's size."""
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


def call(ep, name, *args):
    r = ctypes.byref
    return getattr(ep.lib(), name)(*[r(a) if isinstance(a, ctypes.Structure) else a for a in args])


def shapes(S, f):
    for s in (S(-1, 2, 64, 64), S(10, 0, 64, 64), S(10, 2, 60, 64), S(10, 2, 64, 0), S(10, 2, 64, 12)):
        yield s, "bad"
    for s in (S(10, 9000, 64, 64), S(10, 2, (1 << 20) + 8, 64), S(10, 2, 64, (1 << 20) + 8), S((1 << 30) + 1, 2, 64, 64)):
        yield s, "unsup"


def test_gated_refusals(ep):
    bad, unsup, S, C = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED, ep.ep_gemm_shape, ep.ep_checkpoint
    launch, q, b = ep.ep_launch(None, None, None, None), C(ep.EP_FP8_E4M3, P, P), C(ep.EP_BF16, P, None)

    def go(shape=S(10, 2, 64, 64), x=P, w=P, prefix=P, act=0, h=P, keep=q, launch=launch):
        return call(ep, "ep_expert_gated", shape, x, w, prefix, act, h, keep, launch)

    for s, status in shapes(S, go):
        assert go(shape=s) == {"bad": bad, "unsup": unsup}[status]
    assert go(shape=None) == bad and go(launch=None) == bad
    assert go(x=None) == bad and go(w=None) == bad and go(prefix=None) == bad and go(h=None, keep=None) == bad
    assert go(x=P + 8) == bad and go(w=P + 2) == bad and go(prefix=P + 2) == bad and go(h=P + 8) == bad
    assert go(act=2) == bad and go(act=-1) == bad
    for keep in (C(2, P, P), C(-1, P, P), C(ep.EP_FP8_E4M3, P, None), C(ep.EP_FP8_E4M3, None, P), C(ep.EP_BF16, None, None),
                 C(ep.EP_BF16, P, P), C(ep.EP_FP8_E4M3, P + 8, P), C(ep.EP_FP8_E4M3, P, P + 1), C(ep.EP_BF16, P + 4, None)):
        assert go(keep=keep) == bad

    def back(shape=S(10, 2, 64, 64), dy=P, w=P, prefix=P, act=1, kept=b, dgu=P, h=P, launch=launch):
        return call(ep, "ep_expert_gated_dgrad", shape, dy, w, prefix, act, kept, dgu, h, launch)

    for s, status in shapes(S, back):
        assert back(shape=s) == {"bad": bad, "unsup": unsup}[status]
    assert back(shape=None) == bad and back(launch=None) == bad and back(kept=None) == bad
    assert back(dy=None) == bad and back(w=None) == bad and back(prefix=None) == bad and back(dgu=None) == bad
    assert back(dy=P + 8) == bad and back(w=P + 2) == bad and back(prefix=P + 2) == bad and back(dgu=P + 8) == bad and back(h=P + 2) == bad
    assert back(act=7) == bad
    for kept in (C(2, P, P), C(ep.EP_FP8_E4M3, P, None), C(ep.EP_BF16, P, P), C(ep.EP_BF16, P + 2, None), C(ep.EP_FP8_E4M3, P, P + 1)):
        assert back(kept=kept) == bad


def test_checkpoint_refusals(ep):
    bad, unsup, C = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED, ep.ep_checkpoint
    launch, q = ep.ep_launch(None, None, None, None), C(ep.EP_FP8_E4M3, P, P)
    for name in ("ep_checkpoint_rows", "ep_restore_rows"):
        def go(rows=10, features=64, x=P, kept=q, launch=launch):
            a, b = (x, kept) if name == "ep_checkpoint_rows" else (kept, x)
            return call(ep, name, rows, features, a, b, launch)

        assert go(rows=-1) == bad and go(features=0) == bad and go(features=12) == bad and go(features=-8) == bad
        assert go(rows=(1 << 30) + 1) == unsup and go(features=(1 << 20) + 8) == unsup and go(rows=1 << 30, features=1 << 20) == unsup
        assert go(x=None) == bad and go(x=P + 8) == bad and go(kept=None) == bad and go(launch=None) == bad
        for kept in (C(ep.EP_BF16, P, None), C(ep.EP_BF16, P, P), C(9, P, P), C(ep.EP_FP8_E4M3, P, None), C(ep.EP_FP8_E4M3, None, P),
                     C(ep.EP_FP8_E4M3, P + 8, P)):
            assert go(kept=kept) == bad


def test_gradient_from_kept_rows_refusals(ep):
    bad, unsup, S, C = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED, ep.ep_gemm_shape, ep.ep_checkpoint
    launch, q, good = ep.ep_launch(None, None, None, None), C(ep.EP_FP8_E4M3, P, P), S(10, 2, 64, 64)
    size = ep.ep_wgrad_checkpoint_workspace_size(good)

    def go(shape=good, dy=P, x=q, prefix=P, dw=P, ws=P, n=size, launch=launch):
        return call(ep, "ep_expert_gemm_wgrad_checkpoint", shape, dy, x, prefix, dw, ws, n, launch)

    for s, status in shapes(S, go):
        assert go(shape=s, n=1 << 60) == {"bad": bad, "unsup": unsup}[status]
    assert go(shape=None) == bad and go(launch=None) == bad and go(x=None) == bad
    assert go(dy=None) == bad and go(prefix=None) == bad and go(dw=None) == bad and go(ws=None) == bad
    assert go(dy=P + 8) == bad and go(prefix=P + 2) == bad and go(dw=P + 2) == bad and go(ws=P + 8) == bad and go(n=size - 1) == bad
    for x in (C(ep.EP_BF16, P, None), C(ep.EP_FP8_E4M3, P, None), C(ep.EP_FP8_E4M3, None, P), C(ep.EP_FP8_E4M3, P + 8, P)):
        assert go(x=x) == bad
    assert go(shape=S(1 << 30, 1, 1 << 20, 8), n=1 << 60) == unsup
    assert size >= 16 and ep.ep_wgrad_checkpoint_workspace_size(S(0, 1, 8, 8)) == 16
    for s, _ in shapes(S, go):
        assert ep.ep_wgrad_checkpoint_workspace_size(s) == 0


def test_selftest_of_the_blocks_waits(ep):
    launch, sh, q = ep.ep_launch(None, None, None, P), ep.ep_gemm_shape(10, 2, 64, 64), ep.ep_checkpoint(ep.EP_FP8_E4M3, P, P)

    def go(shape=sh, product=0, rows=P, w=P, prefix=P, kept=q, out=P, loads=64, ms=20, launch=launch):
        return call(ep, "ep_selftest_gated_timeout", shape, product, rows, w, prefix, kept, out, loads, ms, launch)

    for bad in (dict(product=2), dict(product=-1), dict(loads=-64), dict(loads=32), dict(ms=0), dict(ms=10001), dict(launch=None),
                dict(launch=ep.ep_launch(None, None, None, None)), dict(shape=ep.ep_gemm_shape(10, 2, 60, 64)), dict(rows=None),
                dict(w=P + 8), dict(prefix=None), dict(product=1, out=None), dict(product=1, kept=None), dict(kept=None, out=None)):
        assert go(**bad) == ep.EP_ERR_INVALID_ARG, bad
