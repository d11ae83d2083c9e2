"""Refusals on the host of the feed-forward block's and the checkpoints' functions, and that second
derivatives raise (no GPU needed: where a call is reached it is replaced)."""
from types import SimpleNamespace

import pytest
import torch

from combine_layout_02_gb300 import experts

BF, F32, I64, I32, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.uint8


def t(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


def refuses(what, f, *args, **named):
    with pytest.raises(ValueError, match=f"^{what} has to be"):
        f(*args, **named)


def test_block_operands_fit():
    good = dict(x=t(BF, 9, 64), gate_up=t(BF, 3, 80, 64), down=t(BF, 3, 64, 40), expert_prefix=t(I32, 4))
    bad = dict(x=[t(F32, 9, 64), t(BF, 9, 72), t(BF, 9)],
               gate_up=[t(F32, 3, 80, 64), t(BF, 80, 64), t(BF, 2, 80, 64), t(BF, 3, 40, 64), t(BF, 3, 88, 64)],
               down=[t(F32, 3, 64, 40), t(BF, 64, 40)], expert_prefix=[t(I64, 4), t(I32, 3), t(I32, 1, 4)])
    for name, values in bad.items():
        for v in values:
            refuses(name, experts.expert_feed_forward, **{**good, name: v})
    refuses("activation", experts.expert_feed_forward, **good, activation="relu")
    refuses("checkpoint", experts.expert_feed_forward, **good, checkpoint="fp8")
    refuses("checkpoint", experts.expert_feed_forward, **good, checkpoint=None)
    refuses("err", experts.expert_feed_forward, **good, err=t(F32, 1))


def test_widest_block_that_has_gradients():
    F = 1 << 19
    for features in (F, F + 8):
        x, gate_up, down, prefix = t(BF, 1, 8), t(BF, 1, 2 * features, 8), t(BF, 1, 8, features), t(I32, 2)
        for trained in (x, gate_up, down):
            wide = features > F and trained is not down
            trained.requires_grad_()
            with pytest.raises((ValueError, RuntimeError)) as refusal:          # none of these is on a GPU
                experts.expert_feed_forward(x, gate_up, down, prefix)
            assert str(refusal.value).startswith("gate_up has to be of 524288") == wide
            trained.requires_grad_(False)


def test_tensors_are_on_one_device():
    x, gate_up, down, prefix = t(BF, 9, 64), t(BF, 3, 80, 64), t(BF, 3, 64, 40), t(I32, 4)
    for f, args in ((experts.expert_feed_forward, (x.to("meta"), gate_up, down, prefix)),
                    (experts.expert_feed_forward, (x, gate_up, down.to("meta"), prefix)),
                    (experts.restore_rows, (t(U8, 4, 48), t(U8, 4, 3).to("meta"), 40))):
        with pytest.raises(ValueError, match="^all tensors have to be on the current device"):
            f(*args)


def test_kept_rows_fit():
    refuses("x", experts.checkpoint_rows, t(F32, 4, 64))
    refuses("x", experts.checkpoint_rows, t(BF, 64))
    refuses("values", experts.restore_rows, t(U8, 4, 40), t(U8, 4, 3), 40)
    refuses("values", experts.restore_rows, t(BF, 4, 48), t(U8, 4, 3), 40)
    refuses("scales", experts.restore_rows, t(U8, 4, 48), t(U8, 4, 2), 40)
    refuses("scales", experts.restore_rows, t(U8, 4, 48), t(U8, 5, 3), 40)
    refuses("scales", experts.restore_rows, t(U8, 4, 48), t(F32, 4, 3), 40)


def test_way_back_and_layer_modes():
    sort = SimpleNamespace(N=5, k=2, H=256, rows=7)
    refuses("checkpoint", experts.unsort_rows, t(BF, 7, 256), sort, None, "recompute")
    refuses("y", experts.unsort_rows, t(F32, 7, 256), sort, t(F32, 5, 2), "e4m3")
    refuses("weights", experts.unsort_rows, t(BF, 7, 256), sort, t(F32, 5, 3), "e4m3")
    buf = SimpleNamespace(R=2, E=4, H=128, k=2)
    refuses("checkpoint", experts.MoELayer, buf, 16, "cpu", checkpoint="fp8")
    refuses("activation", experts.MoELayer, buf, 16, "cpu", checkpoint="e4m3", activation="relu")
    refuses("activation", experts.MoELayer, buf, 16, "cpu", activation="gelu")          # the products alone: silu


N, K, E, F, H = 6, 4, 3, 5, 7


@pytest.fixture
def calls(monkeypatch):
    """Plain forms of the calls, writing into their outputs."""
    def put(out, value):
        if out is not None:
            out.copy_(torch.as_tensor(value))

    plain = dict(
        make_launch=lambda **kw: None, ep_gemm_shape=lambda *a: None, make_checkpoint=lambda *a: a,
        checkpoint_rows=lambda x: (x.detach().clone(), torch.zeros(len(x), 1)), restore_rows=lambda v, s, n: v.clone(),
        ep_checkpoint_rows=lambda *a: None, ep_wgrad_checkpoint_workspace_size=lambda sh: 16,
        ep_expert_gated=lambda sh, x, w, p, act, h, keep, launch: put(h, x @ w[0, :F].t()),
        ep_expert_gemm=lambda sh, x, w, p, y, launch: put(y, x @ w[0].t()),
        ep_expert_gated_dgrad=lambda *a: None,
        ep_expert_gemm_dgrad=lambda sh, dy, w, p, dx, launch: put(dx, 1.0),
        ep_expert_gemm_wgrad=lambda sh, dy, x, p, dw, launch: put(dw, 1.0),
        ep_expert_gemm_wgrad_checkpoint=lambda sh, dy, x, p, dw, ws, launch: put(dw, 1.0),
        ep_unsort_rows=lambda sh, y, w, sort, out, launch: put(out, y * w[:, :1]),
        ep_unsort_rows_backward=lambda sh, dout, y, w, sort, dy, dw, launch: (
            dw is not None and put(dw, (dout * y).sum(1, keepdim=True).expand(N, 2)), put(dy, dout * w[:, :1])))
    for name, f in plain.items():
        monkeypatch.setattr(experts, name, f)


def values(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(1)).requires_grad_(True)


@pytest.mark.parametrize("checkpoint", ["bf16", "e4m3", "recompute"])
def test_block_gradients_once(calls, checkpoint):
    x, gate_up, down = values(N, K), values(E, 2 * F, K), values(E, H, F)
    prefix = torch.tensor([0, N, N, N], dtype=torch.int32)
    y = experts._FeedForward.apply(x, gate_up, down, prefix, 0, checkpoint, None)
    grad, = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    assert torch.isfinite(grad).all()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (y.sum() + (grad * grad).sum()).backward()


@pytest.mark.parametrize("checkpoint", ["bf16", "e4m3", "recompute"])
@pytest.mark.parametrize("wanted", [(0,), (1,), (2,), (0, 2), (1, 2), (0, 1, 2)])
def test_block_gradients_where_wanted(calls, checkpoint, wanted):
    leaves = [values(N, K), values(E, 2 * F, K), values(E, H, F)]
    for i, v in enumerate(leaves):
        v.requires_grad_(i in wanted)
    y = experts._FeedForward.apply(*leaves, torch.tensor([0, N, N, N], dtype=torch.int32), 0, checkpoint, None)
    y.sum().backward()
    assert [v.grad is not None for v in leaves] == [i in wanted for i in range(3)]


def test_kept_way_back_gradients(calls):
    sort = SimpleNamespace(N=N, k=2, H=H, rows=N, shape=None, handle=None, launch=lambda: None)
    for y_wanted, w_wanted in ((True, True), (True, False), (False, True)):
        y, w = values(N, H), values(N, 2)
        y.requires_grad_(y_wanted), w.requires_grad_(w_wanted)
        out = experts._UnsortRowsKept.apply(y, w, sort)
        out.sum().backward()
        assert (y.grad is not None) == y_wanted and (w.grad is not None) == w_wanted
        if y_wanted:
            assert torch.equal(y.grad, w.detach()[:, :1].expand(N, H))
