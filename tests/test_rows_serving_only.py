"""The projection with adapters has no gradient: a backward pass that reaches it raises instead of
leaving its part out. (No GPU: the call is replaced.)"""
import pytest
import torch

from combine_layout_02_gb300 import experts

T, K, F, L, r = 5, 16, 8, 2, 8


@pytest.fixture(autouse=True)
def call(monkeypatch):
    def plain(sh, x, w, a, b, scales, idx, y, ws, launch):
        y.copy_(x @ w.t())

    monkeypatch.setattr(experts, "make_launch", lambda **kw: None)
    monkeypatch.setattr(experts, "ep_adapter_workspace_size", lambda shape: 64)
    monkeypatch.setattr(experts, "ep_adapter_gemm", plain)


def operands():
    bf = lambda *s: torch.ones(*s, dtype=torch.bfloat16)  # noqa: E731
    return dict(x=bf(T, K), weight=bf(F, K), a=bf(L, r, K), b=bf(L, F, r), scales=torch.ones(L),
                adapter_idx=torch.zeros(T, dtype=torch.int64))


@pytest.mark.parametrize("wants", ["x", "weight", "a", "b", "scales"])
def test_backward_raises(wants):
    d = operands()
    d[wants].requires_grad_(True)
    other = torch.ones(T, F, requires_grad=True)          # the rest of a model: its gradient alone would pass
    y = experts.adapter_projection(**d)
    assert bool((y == K).all())
    with pytest.raises(RuntimeError, match="has no gradient"):
        (y.float() * other).sum().backward()


def test_serving_is_as_before():
    d = operands()
    d["weight"].requires_grad_(True)
    with torch.no_grad():
        y = experts.adapter_projection(**d)
    assert not y.requires_grad and bool((y == K).all())
    y = experts.adapter_projection(**operands())
    assert not y.requires_grad and bool((y == K).all())
    y = experts.adapter_projection(operands()["x"], operands()["weight"], None, None, None, operands()["adapter_idx"])
    assert bool((y == K).all())
