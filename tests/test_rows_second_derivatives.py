"""The autograd functions' gradients are computed by library calls, which autograd does not see: a
second derivative has to raise instead of leaving its part out. (No GPU: the calls are replaced.)"""
from types import SimpleNamespace

import pytest
import torch

from combine_layout_02_gb300 import experts

N, K, H, E, F = 6, 2, 4, 3, 5


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """Plain forms of the calls, writing into their outputs; one entry per row, in order."""
    def put(out, value):
        if out is not None:
            out.copy_(value)

    def unsort_backward(sh, dout, y, w, sort, dy, dw, launch):
        put(dy, dout if w is None else dout * w[:, :1])
        put(dw, (dout * y).sum(1, keepdim=True).expand(N, K))

    plain = dict(
        make_launch=lambda **kw: None, ep_gemm_shape=lambda *a: None,
        ep_sort_rows=lambda sh, x, dt, xs, sort, out, osc, launch: put(out, x),
        ep_unsort_rows=lambda sh, y, w, sort, out, launch: put(out, y if w is None else y * w[:, :1]),
        ep_unsort_rows_backward=unsort_backward,
        ep_expert_gemm=lambda sh, x, w, p, y, launch: put(y, x @ w[0].t()),
        ep_expert_gemm_dgrad=lambda sh, dy, w, p, dx, launch: put(dx, dy @ w[0]),
        ep_expert_gemm_wgrad=lambda sh, dy, x, p, dw, launch: put(dw, (dy.t() @ x).expand(E, F, H)))
    for name, f in plain.items():
        monkeypatch.setattr(experts, name, f)


sort = SimpleNamespace(N=N, k=K, H=H, rows=N, shape=None, handle=None, launch=lambda: None)
regions = SimpleNamespace(row_offset=[0, N])
buf = SimpleNamespace(
    dispatch=lambda x, topk_idx=None, topk_weights=None, handle=None: (x.clone(), topk_idx, topk_weights, None, regions, None),
    combine=lambda y, handle, topk_weights=None: (y.clone(), topk_weights, None), _rows_tensor=lambda t, off: t)


def values(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(1)).requires_grad_(True)


def sort_rows():
    x = values(N, H)
    return experts._SortRows.apply(x, sort), x


def unsort_rows():
    y = values(N, H)
    return experts._UnsortRows.apply(y, values(N, K), sort), y


def product():
    x = values(N, H)
    return experts._ExpertProduct.apply(x, values(E, F, H), torch.tensor([0, N], dtype=torch.int32), None), x


def dispatch():
    x = values(N, H)
    return experts._Dispatch.apply(x, values(N, K), torch.zeros(N, K, dtype=torch.int64), buf, {})[0], x


def combine():
    y = values(N, H)
    return experts._Combine.apply(y, buf, regions), y


@pytest.mark.parametrize("make", [sort_rows, unsort_rows, product, dispatch, combine])
def test_first_derivatives_pass_and_second_ones_raise(make):
    out, x = make()
    grad, = torch.autograd.grad((out * out).sum(), x, create_graph=True)
    assert torch.isfinite(grad).all()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (out.sum() + (grad * grad).sum()).backward()
