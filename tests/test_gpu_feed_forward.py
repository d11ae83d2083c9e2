"""The gated feed-forward block as an autograd function and in the mixture-of-experts layer: forward and
every gradient against plain 64-bit forms with the same roundings and checkpoints."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from combine_layout_02_gb300.api import Buffer
from combine_layout_02_gb300.experts import (ExpertSort, MoELayer, check_errors, checkpoint_rows, expert_feed_forward, expert_product,
                                             restore_rows, sort_rows, unsort_rows)
from kept_util import act, quantised

pytestmark = pytest.mark.gpu

MODES = ("bf16", "e4m3", "recompute")


def through(t, value):
    """value forward, t's gradient."""
    return t + (value - t.detach())


def rounded(t):
    return through(t, t.detach().float().bfloat16().double())


def kept(t, mode):
    t = t.detach().float().bfloat16()
    return (quantised(t)[2].cuda() if mode == "e4m3" else t.double())


class Act(torch.autograd.Function):
    """act(g) u forward, with the derivatives at g and u as they were kept."""

    @staticmethod
    def forward(ctx, g, u, kind, mode):
        ctx.kind, ctx.parts = kind, (kept(g, mode), kept(u, mode))
        return act(g, kind)[0] * u

    @staticmethod
    def backward(ctx, dh):
        g, u = ctx.parts
        a, da = act(g, ctx.kind)[:2]
        return (dh * u * da).float().bfloat16().double(), (dh * a).float().bfloat16().double(), None, None


class Matrix(torch.autograd.Function):
    """x W^T, whose matrix gradient goes by x as it was kept."""

    @staticmethod
    def forward(ctx, x, w, there):
        ctx.save_for_backward(w, there)
        return x @ w.t()

    @staticmethod
    def backward(ctx, dy):
        w, there = ctx.saved_tensors
        return dy @ w, dy.t() @ there, None


def plain_block(x, gate_up, down, edge, kind, mode):
    out = []
    for e in range(len(edge) - 1):
        rows = x[edge[e]:edge[e + 1]]
        F = down.shape[2]
        g, u = Matrix.apply(rows, gate_up[e], kept(rows, mode)).split(F, 1)
        h = rounded(Act.apply(g, u, kind, mode))
        gk, uk = kept(g, mode), kept(u, mode)
        again = (act(gk, kind)[0] * uk).float().bfloat16().double()
        out.append(Matrix.apply(h, down[e], again))
    return torch.cat(out)


def close(got, want, what):
    """Both within a few bf16 roundings of sums of this size: 2-norm 1e-2 of the result (each rounding is
    2^-9 / sqrt(3) = 1.1e-3 of the value on average), and no value off by more than 5e-2 of the largest. (A
    sum that falls to the other side of an e4m3 step is rare: a rounding error of 2^-20 against steps
    of 2^-4.)"""
    got, want = got.detach().double(), want.detach().double()
    assert float((got - want).norm() / want.norm()) < 1e-2, what
    assert float((got - want).abs().max()) < 5e-2 * float(want.abs().max()), what


def block(counts, K, F, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    edge = [0]
    for n in counts:
        edge.append(edge[-1] + n)
    new = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).bfloat16().requires_grad_(True)  # noqa: E731
    x, gate_up, down = new(edge[-1], K), new(E, 2 * F, K, scale=1.5 * K ** -0.5), new(E, H, F, scale=F ** -0.5)
    dy = torch.randn(edge[-1], H, generator=g, device="cuda").bfloat16()
    return x, gate_up, down, torch.tensor(edge, dtype=torch.int32, device="cuda"), edge, dy


@pytest.mark.parametrize("counts,K,F,H", [([40, 0, 7, 90, 1], 72, 136, 200), ([300, 513], 256, 264, 136), ([3], 512, 1024, 512),
                                          ([1, 1, 0, 1], 128, 64, 128)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("mode", MODES)
def test_block_forward_and_gradients(mode, kind, counts, K, F, H):
    x, gate_up, down, prefix, edge, dy = block(counts, K, F, H, 1)
    y = expert_feed_forward(x, gate_up, down, prefix, kind, mode)
    got = torch.autograd.grad(y, (x, gate_up, down), dy)
    leaves = [t.detach().double().requires_grad_(True) for t in (x, gate_up, down)]
    want = plain_block(*leaves, edge, kind, mode)
    close(y, want, "y")
    for name, a, b in zip(("x", "gate_up", "down"), got, torch.autograd.grad(want, leaves, dy.double())):
        close(a, b, name)
    assert check_errors() == 0


def test_modes_agree():
    """Nothing of the result depends on what is kept; what is computed again is what bf16 keeps, bit for bit."""
    x, gate_up, down, prefix, _, dy = block([40, 0, 700], 192, 136, 264, 2)
    out = {}
    for mode in MODES:
        y = expert_feed_forward(x, gate_up, down, prefix, "silu", mode)
        out[mode] = (y.detach(), *torch.autograd.grad(y, (x, gate_up, down), dy))
    with torch.no_grad():
        y = expert_feed_forward(x, gate_up, down, prefix)
    assert all(torch.equal(y, out[m][0]) for m in MODES)
    assert all(torch.equal(a, b) for a, b in zip(out["bf16"], out["recompute"]))


def test_what_is_kept_between_the_passes():
    """Bytes that live from one pass to the other beside the inputs: 4F a row in bf16, K + 2F bytes and their
    scales in 8 bits, none with the projections run again."""
    x, gate_up, down, prefix, _, dy = block([2048, 2048], 1024, 512, 1024, 3)
    held = {}
    for mode in MODES:
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        y = expert_feed_forward(x, gate_up, down, prefix, "silu", mode)
        held[mode] = torch.cuda.memory_allocated() - before - y.numel() * 2
        y.backward(dy)
        del y
        x.grad = gate_up.grad = down.grad = None
    rows = 4096
    assert held == {"bf16": rows * 4 * 512, "e4m3": rows * (1024 + 2 * 512) * 17 // 16, "recompute": 0}


def test_serving_keeps_nothing():
    """Under torch.no_grad() with parameters that want gradients: two kernels, memory for h and y alone, and a
    single row takes the way of single rows."""
    x, gate_up, down, prefix, _, _ = block([2048, 2048], 1024, 512, 1024, 9)
    sort = ExpertSort(torch.arange(4096, device="cuda").remainder(2).view(-1, 1), 2, 1024)
    weights = torch.rand(4096, 1, device="cuda").requires_grad_(True)
    for mode in MODES:
        with torch.no_grad():
            torch.cuda.synchronize()
            torch.cuda.reset_peak_memory_stats()
            before, launched = torch.cuda.memory_allocated(), ep.ep_kernel_launch_count()
            y = expert_feed_forward(x, gate_up, down, prefix, "silu", mode)
            assert ep.ep_kernel_launch_count() - launched == 2
            assert torch.cuda.max_memory_allocated() - before == 4096 * (512 + 1024) * 2
            assert not y.requires_grad
            launched = ep.ep_kernel_launch_count()
            out = unsort_rows(y.requires_grad_(True), sort, weights, checkpoint="e4m3" if mode == "e4m3" else "bf16")
            assert ep.ep_kernel_launch_count() - launched == 1 and not out.requires_grad
    one = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    row = x.detach()[:1].contiguous()
    h = torch.empty(1, 512, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gated(ep.ep_gemm_shape(1, 2, 1024, 512), row, gate_up, one, ep.EP_ACT_SILU, h)
    with torch.no_grad():
        assert torch.equal(expert_feed_forward(row, gate_up, down, one), expert_product(h, down, one))


def test_block_without_rows():
    x, gate_up, down, prefix, _, dy = block([0, 0], 64, 48, 72, 4)
    for mode in MODES:
        y = expert_feed_forward(x, gate_up, down, prefix, "gelu", mode)
        assert y.shape == (0, 72)
        dx, dgate_up, ddown = torch.autograd.grad(y, (x, gate_up, down), dy)
        assert dx.shape == x.shape and not bool(dgate_up.any()) and not bool(ddown.any())


def test_block_on_another_stream_and_in_a_graph():
    """Captured with its backward pass, replayed on new rows, while an eager graph of other leaves lives."""
    x, gate_up, down, prefix, _, dy = block([33, 2, 130], 128, 72, 128, 5)
    eager = expert_feed_forward(x, gate_up, down, prefix, "silu", "e4m3")
    static = [t.detach().clone().requires_grad_(True) for t in (x, gate_up, down)]

    def step():
        y = expert_feed_forward(*static, prefix, "silu", "e4m3")
        return (y, *torch.autograd.grad(y, static, dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.detach().clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (6, 7):
        with torch.no_grad():
            static[0].copy_(block([33, 2, 130], 128, 72, 128, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        assert not torch.equal(got[0], first[0])
    want = torch.autograd.grad(eager, (x, gate_up, down), dy)
    for a, b in zip(want, first[1:]):
        assert torch.equal(a, b)
    assert torch.equal(eager, first[0])


# ------------------------------------------------------------------ in the layer

R, T, LH, LE, k, LF = 4, 37, 256, 16, 3, 136


def layer_inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, T, LH, generator=g, device="cuda").bfloat16()
    idx = torch.rand(R, T, LE, generator=g, device="cuda").argsort(-1)[..., :k].contiguous()
    idx[0, 3, 1] = -1
    idx[1, 5] = -1                       # a token without experts
    w = torch.softmax(torch.randn(R, T, k, generator=g, device="cuda"), -1)
    return g, x, idx, w


@pytest.mark.parametrize("kind,mode", [("silu", "bf16"), ("silu", "e4m3"), ("gelu", "e4m3"), ("gelu", "recompute")])
def test_layer_forward_and_gradients(kind, mode):
    g, x, idx, w = layer_inputs(1)
    buf = Buffer(R, LE, LH, k)
    torch.manual_seed(2)
    layer = MoELayer(buf, LF, checkpoint=mode, activation=kind)
    x.requires_grad_(True)
    w.requires_grad_(True)
    out = layer(x, idx, w)
    dout = torch.randn(out.shape, generator=g, device="cuda").bfloat16()
    out.backward(dout)
    assert buf.check_errors() == 0
    p = {n: t.detach().double().requires_grad_(True) for n, t in layer.named_parameters()}
    x64, w64 = x.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    flat = x64.reshape(-1, LH)
    want = torch.zeros_like(flat)
    for e in range(LE):
        at = (idx.reshape(-1, k) == e).nonzero()
        if len(at):
            rows = flat[at[:, 0]]
            y = rounded(plain_block(rows, p["gate_up"][e:e + 1], p["down"][e:e + 1], [0, len(at)], kind, mode))
            weight = w64.reshape(-1, k)[at[:, 0], at[:, 1]].unsqueeze(1)
            there = kept(y, "e4m3" if mode == "e4m3" else "bf16")
            # the weights' gradient goes by y as it was kept
            term = weight.detach() * y + (weight - weight.detach()) * there
            want = want.index_add(0, at[:, 0], term)
    want = (want + flat @ p["shared"].t()).view_as(x)
    want.backward(dout.double())
    close(out, want, "out")
    close(x.grad, x64.grad, "x")
    close(w.grad, w64.grad, "topk_weights")
    for n, t in layer.named_parameters():
        close(t.grad, p[n].grad, n)
    assert bool((w.grad[1, 5] == 0).all()) and float(w.grad[0, 3, 1]) == 0.0


def test_layer_serves_as_it_trains():
    _, x, idx, w = layer_inputs(3)
    buf = Buffer(R, LE, LH, k)
    torch.manual_seed(4)
    layer = MoELayer(buf, LF, checkpoint="e4m3")
    out = layer(x, idx, w)
    with torch.no_grad():
        assert torch.equal(layer(x, idx, w), out.detach())
    # within the roundings of h, silu and their product that the layer of single products has more
    torch.manual_seed(4)
    close(out, MoELayer(buf, LF)(x, idx, w), "product by product")


def test_way_back_keeps_eight_bits():
    g, x, idx, w = layer_inputs(5)
    sort = ExpertSort(idx.view(-1, k), LE, LH)
    y = torch.randn(sort.rows, LH, generator=g, device="cuda").bfloat16()
    dout = torch.randn(R * T, LH, generator=g, device="cuda").bfloat16()
    res = {}
    for mode, there in (("bf16", y), ("e4m3", restore_rows(*checkpoint_rows(y), LH))):
        a, b = there.clone().requires_grad_(True), w.reshape(-1, k).clone().requires_grad_(True)
        unsort_rows(a, sort, b).backward(dout)
        res[mode] = (a.grad, b.grad)
    a, b = y.clone().requires_grad_(True), w.reshape(-1, k).clone().requires_grad_(True)
    out = unsort_rows(a, sort, b, checkpoint="e4m3")
    assert torch.equal(out, unsort_rows(y, sort, b.detach()))
    out.backward(dout)
    assert torch.equal(a.grad, res["e4m3"][0]) and torch.equal(b.grad, res["e4m3"][1])
    assert torch.equal(res["bf16"][0], res["e4m3"][0])
    del out


def test_fused_block_against_the_products():
    """Where nothing is rounded away between them: whole numbers, gelu and silu apart, g as the products have it."""
    g = torch.Generator(device="cuda").manual_seed(8)
    E, K, F = 3, 64, 48
    edge = torch.tensor([0, 20, 20, 97], dtype=torch.int32, device="cuda")
    x = torch.randint(-3, 4, (97, K), generator=g, device="cuda").bfloat16()
    gate_up = torch.randint(-1, 2, (E, 2 * F, K), generator=g, device="cuda").bfloat16()
    both = expert_product(x, gate_up, edge)
    values = torch.empty(97, 2 * F, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gated(ep.ep_gemm_shape(97, E, K, F), x, gate_up, edge, ep.EP_ACT_SILU, None, ep.make_checkpoint(values))
    assert torch.equal(values, both)
    assert torch.equal(sort_rows(x.new_zeros(0, 128), ExpertSort(torch.zeros(0, 1, dtype=torch.int64, device="cuda"), E, 128)),
                       x.new_zeros(0, 128))
