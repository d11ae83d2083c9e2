"""The autograd functions on rows grouped by owner where there is little or nothing to do."""
import pytest
import torch

from combine_layout_02_gb300.api import Buffer
from combine_layout_02_gb300.experts import ExpertSort, MoELayer, expert_product, sort_rows, unsort_rows

pytestmark = pytest.mark.gpu


def bf16(*shape, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("N", [0, 1, 5, 700])
@pytest.mark.parametrize("weighted", [False, True])
def test_no_entry_placed(N, weighted):
    """Every entry masked: nothing sorted, zeros back, zero gradients."""
    E, H, k = 6, 256, 3
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sort = ExpertSort(torch.full((N, k), -1, device="cuda"), E, H, err=err)
    assert sort.rows == 0 and sort.handle.num_rows == 0
    x = bf16(N, H).requires_grad_(True)
    mats = bf16(E, H, H, seed=2).requires_grad_(True)
    w = torch.rand(N, k, device="cuda").requires_grad_(True) if weighted else None
    rows = sort_rows(x, sort)
    assert rows.shape == (0, H)
    out = unsort_rows(expert_product(rows, mats, sort.expert_prefix, err), sort, w)
    assert out.shape == (N, H) and bool((out == 0).all())
    out.backward(torch.ones_like(out))
    assert x.grad.shape == x.shape and bool((x.grad == 0).all())
    assert mats.grad.shape == mats.shape and bool((mats.grad == 0).all())
    if weighted:
        assert w.grad.shape == w.shape and bool((w.grad == 0).all())
    assert int(err.item()) == 0


def test_the_handle_holds_the_rows_there_are():
    """Masked entries leave fewer rows than entries; a later call is checked against those."""
    idx = torch.tensor([[0, -1, 1], [-1, -1, -1], [2, 2, -1]], device="cuda")
    sort = ExpertSort(idx, 3, 128)
    assert sort.rows == 4 and sort.handle.num_rows == 4
    x = bf16(3, 128)
    back = unsort_rows(sort_rows(x, sort), sort)
    assert torch.equal(back, (x.float() * (idx >= 0).sum(1, keepdim=True)).bfloat16())


def test_layer_without_any_routed_token():
    R, T, H, E, k = 2, 9, 128, 4, 2
    buf = Buffer(R, E, H, k)
    torch.manual_seed(3)
    layer = MoELayer(buf, 24)
    x = bf16(R, T, H).requires_grad_(True)
    w = torch.rand(R, T, k, device="cuda").requires_grad_(True)
    out = layer(x, torch.full((R, T, k), -1, device="cuda"), w)
    dout = bf16(R, T, H, seed=4)
    out.backward(dout)
    flat, m = dout.reshape(-1, H).double(), layer.shared.detach().double()
    torch.testing.assert_close(out.detach().double().reshape(-1, H), x.detach().double().reshape(-1, H) @ m.t(), rtol=0.01,
                               atol=0.01)
    torch.testing.assert_close(x.grad.double().reshape(-1, H), flat @ m, rtol=0.01, atol=0.01)
    assert bool((w.grad == 0).all())
    assert bool((layer.gate_up.grad == 0).all()) and bool((layer.down.grad == 0).all())
    assert buf.check_errors() == 0
