"""Refusals on the host of the calls on rows grouped by owner (no GPU needed)."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

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


def refuses(what, f, *args):
    """Before anything is launched: on the host, these tensors would be refused later for being there."""
    with pytest.raises(ValueError, match=f"^{what} has to be"):
        f(*args)


BF, F32, I64, I32, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.uint8


def t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


def test_placement_takes_int64_ids():
    from combine_layout_02_gb300.experts import ExpertSort
    refuses("topk_idx", ExpertSort, t(I32, 4, 2), 8, 256)
    refuses("topk_idx", ExpertSort, t(I64, 8), 8, 256)
    refuses("err", ExpertSort, t(I64, 4, 2), 8, 256, None, t(F32, 1))
    refuses("err", ExpertSort, t(I64, 4, 2), 8, 256, None, t(I32, 0))


def test_rows_have_the_placements_size_and_type():
    from combine_layout_02_gb300.experts import sort_rows, unsort_rows
    sort = SimpleNamespace(N=5, k=2, H=256, rows=7)
    # an e4m3 dispatch's rows are uint8 [N][H]: half the bytes that a bf16 row has
    for x in (t(U8, 5, 256), t(F32, 5, 256), t(BF, 5, 128), t(BF, 4, 256), t(BF, 6, 256), t(BF, 5 * 256), None):
        refuses("x", sort_rows, x, sort)
    for y in (t(F32, 7, 256), t(BF, 6, 256), t(BF, 7, 128), t(BF, 5, 256), None):
        refuses("y", unsort_rows, y, sort)
    for w in (t(BF, 5, 2), t(F32, 5, 3), t(F32, 7, 2), t(F32, 10)):
        refuses("weights", unsort_rows, t(BF, 7, 256), sort, w)


def test_product_operands_fit():
    from combine_layout_02_gb300.experts import expert_product
    x, w, p = t(BF, 9, 64), t(BF, 3, 128, 64), t(I32, 4)
    refuses("weight", expert_product, x, t(F32, 3, 128, 64), p)
    refuses("weight", expert_product, x, t(BF, 128, 64), p)
    refuses("x", expert_product, t(F32, 9, 64), w, p)
    refuses("x", expert_product, t(BF, 9, 128), w, p)
    refuses("expert_prefix", expert_product, x, w, t(I64, 4))
    refuses("expert_prefix", expert_product, x, w, t(I32, 3))
    refuses("err", expert_product, x, w, p, t(I64, 1))


def test_projection_operands_fit():
    from combine_layout_02_gb300.experts import adapter_projection
    good = dict(x=t(BF, 9, 64), weight=t(BF, 128, 64), a=t(BF, 3, 16, 64), b=t(BF, 3, 128, 16), scales=t(F32, 3),
                adapter_idx=t(I64, 9))
    bad = dict(x=[t(F32, 9, 64), t(BF, 9)], weight=[t(F32, 128, 64), t(BF, 128, 72), t(BF, 1, 128, 64)],
               a=[t(F32, 3, 16, 64), t(BF, 3, 16, 72), t(BF, 16, 64)],
               b=[t(F32, 3, 128, 16), t(BF, 2, 128, 16), t(BF, 3, 120, 16), t(BF, 3, 128, 8), None],
               scales=[t(BF, 3), t(F32, 2), None], adapter_idx=[t(I32, 9), t(I64, 8), t(I64, 9, 1)])
    for name, values in bad.items():
        for v in values:
            refuses(name, lambda: adapter_projection(**{**good, name: v}))
    refuses("adapter_idx", lambda: adapter_projection(good["x"], good["weight"], None, None, None, t(I32, 9)))


def test_layer_inputs_fit():
    from combine_layout_02_gb300.experts import MoELayer
    layer = MoELayer(SimpleNamespace(R=2, E=4, H=128, k=2), 16, device="cpu")
    x, idx, w = t(BF, 2, 5, 128), t(I64, 2, 5, 2), t(F32, 2, 5, 2)
    refuses("x", layer, x.float(), idx, w)
    refuses("x", layer, t(BF, 2, 5, 256), idx, w)
    refuses("topk_idx", layer, x, idx.int(), w)
    refuses("topk_idx", layer, x, t(I64, 2, 4, 2), w)
    refuses("topk_weights", layer, x, idx, w.bfloat16())
    refuses("topk_weights", layer, x, idx, t(F32, 2, 5, 3))
