"""One row through the feed-forward block: where nothing is kept for a backward pass it takes a way of its own,
with the sums in another order; in training every kind of checkpoint has the same result."""
import pytest
import torch

from combine_layout_02_gb300.experts import expert_feed_forward
from kept_util import act
from rows_util import U16, U32, assert_within, sum_bound

pytestmark = pytest.mark.gpu

MODES = ("bf16", "e4m3", "recompute")
STEEP = 1.13          # the largest slope of silu (1.0998) and gelu (1.1290)


@pytest.mark.parametrize("E,expert,K,F,H", [(1, 0, 512, 264, 128), (3, 2, 4096, 1024, 264), (2, 0, 1000, 72, 4096)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_one_row(kind, E, expert, K, F, H):
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).bfloat16()  # noqa: E731
    x, gate_up, down = new(1, K), new(E, 2 * F, K, scale=1.5 * K ** -0.5), new(E, H, F, scale=F ** -0.5)
    dy = new(1, H)
    prefix = (torch.arange(E + 1, device="cuda") > expert).int()
    leaves = [t.requires_grad_(True) for t in (x, gate_up, down)]
    out = {}
    for mode in MODES:
        y = expert_feed_forward(*leaves, prefix, kind, mode)
        out[mode] = (y.detach(), *torch.autograd.grad(y, leaves, dy))
    # trained: the result does not depend on what is kept, and what is computed again is what was
    assert all(torch.equal(out[m][0], out["bf16"][0]) for m in MODES)
    assert all(torch.equal(a, b) for a, b in zip(out["bf16"], out["recompute"]))
    # served: the same formulas; both ways are within the bound of the fp32 sums, in whatever order
    with torch.no_grad():
        served = [expert_feed_forward(*leaves, prefix, kind, mode) for mode in MODES]
    assert all(torch.equal(s, served[0]) for s in served)
    x64, w, d = x.detach().double(), gate_up.detach()[expert].double(), down.detach()[expert].double()
    (a, b), off = (x64 @ w.t()).split(F, 1), sum_bound(K, x64.abs() @ w.abs().t(), 2 * U32)
    a_off, b_off = off.split(F, 1)
    v, _, v_off, _ = act(a, kind)
    v_off = v_off + STEEP * a_off
    h = v * b
    h_off = v.abs() * b_off + b.abs() * v_off + v_off * b_off + h.abs() * U32
    h_off = h_off + U16 * (h.abs() + h_off)          # h is rounded
    slack = h_off @ d.abs().t() + sum_bound(F, (h.abs() + h_off) @ d.abs().t(), 2 * U32)
    for y in (out["bf16"][0], served[0]):
        assert_within(y, h @ d.t(), slack, U16)
