"""The operators on rows grouped by owner together, as a mixture-of-experts layer over a Buffer:
dispatch, expert sort, products, way back, combine, the shared projection with adapters; forward
and every gradient against a plain 64-bit layer whose intermediate roundings are the same."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from combine_layout_02_gb300.api import Buffer
from combine_layout_02_gb300.experts import ExpertSort, MoELayer, adapter_projection, expert_product, sort_rows, unsort_rows

pytestmark = pytest.mark.gpu

R, T, H, E, k, F = 4, 37, 256, 16, 3, 136


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, T, H, generator=g, device="cuda").bfloat16()
    idx = torch.rand(R, T, E, generator=g, device="cuda").argsort(-1)[..., :k].contiguous()
    idx[0, 3, 1] = -1
    idx[1, 5] = -1                       # a token without experts
    w = torch.softmax(torch.randn(R, T, k, generator=g, device="cuda"), -1)
    return g, x, idx, w


def plain_layer(x, idx, w, layer, common):
    """The layer token by token in 64 bits, with a bf16 rounding where the layer has one (straight
    through for the gradient)."""
    def rounded(t):
        return t + (t.detach().float().bfloat16().double() - t.detach())
    flat = x.reshape(-1, H)
    out = torch.zeros_like(flat)
    for e in range(E):
        at = (idx.reshape(-1, k) == e).nonzero()
        if len(at) == 0:
            continue
        h = rounded(flat[at[:, 0]] @ layer["gate_up"][e].t())
        gate, up = h.chunk(2, 1)
        act = rounded(rounded(torch.nn.functional.silu(gate)) * up)
        y = rounded(act @ layer["down"][e].t())
        out = out.index_add(0, at[:, 0], w.reshape(-1, k)[at[:, 0], at[:, 1]].unsqueeze(1) * y)
    return (out + common(flat)).view_as(x)


def close(got, want, what):
    """Both within a few bf16 roundings of sums of this size: 2-norm 1e-2 of the result (each of the
    five roundings on the way is 2^-9 / sqrt(3) = 1.1e-3 of the value on average, as is every
    partial result that combine rounds), and no value off by more than 5e-2 of the largest."""
    got, want = got.detach().double(), want.detach().double()
    assert float((got - want).norm() / want.norm()) < 1e-2, what
    assert float((got - want).abs().max()) < 5e-2 * float(want.abs().max()), what


def test_layer_forward_and_gradients():
    g, x, idx, w = inputs(1)
    buf = Buffer(R, E, H, k)
    torch.manual_seed(2)
    layer = MoELayer(buf, F)
    x.requires_grad_(True)
    w.requires_grad_(True)
    out = layer(x, idx, w)
    dout = torch.randn(out.shape, generator=g, device="cuda").bfloat16()
    out.backward(dout)
    assert buf.check_errors() == 0
    p = {n: t.detach().double().requires_grad_(True) for n, t in layer.named_parameters()}
    x64, w64 = x.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    want = plain_layer(x64, idx, w64, p, lambda f: f @ p["shared"].t())
    want.backward(dout.double())
    close(out, want, "out")
    close(x.grad, x64.grad, "x")
    close(w.grad, w64.grad, "topk_weights")
    for n, t in layer.named_parameters():
        close(t.grad, p[n].grad, n)
    assert bool((w.grad[1, 5] == 0).all()) and float(w.grad[0, 3, 1]) == 0.0


def test_layer_with_adapters():
    g, x, idx, w = inputs(3)
    buf = Buffer(R, E, H, k)
    torch.manual_seed(4)
    layer = MoELayer(buf, F)
    L, r = 5, 16
    a = (torch.randn(L, r, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    b = (torch.randn(L, H, r, generator=g, device="cuda") * r ** -0.5).bfloat16()
    scales = torch.rand(L, generator=g, device="cuda") + 0.5
    who = torch.randint(-1, L, (R, T), generator=g, device="cuda")
    with torch.no_grad():
        out = layer(x, idx, w, adapters=(a, b, scales, who))

    def common(flat):
        y = flat @ layer.shared.detach().double().t()
        for i in range(L):
            t = (who.reshape(-1) == i).nonzero().reshape(-1)
            y[t] += scales[i].double() * ((flat[t] @ a[i].double().t()) @ b[i].double().t())
        return y

    p = {n: t.detach().double() for n, t in layer.named_parameters()}
    close(out, plain_layer(x.double(), idx, w.double(), p, common), "out")
    assert buf.check_errors() == 0


def test_functions_keep_their_dtypes_and_streams():
    _, x, idx, w = inputs(5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sort = ExpertSort(idx.view(-1, k), E, H)
        rows = sort_rows(x.view(-1, H), sort)
        back = unsort_rows(rows, sort)                       # every entry's row back: a count of copies
    torch.cuda.current_stream().wait_stream(side)
    n = (idx.view(-1, k) >= 0).sum(1, keepdim=True)
    assert rows.dtype == torch.bfloat16 and rows.shape == (int(n.sum()), H)
    assert torch.equal(back, (x.view(-1, H).float() * n).bfloat16())
    y = expert_product(rows, torch.zeros(E, 8, H, dtype=torch.bfloat16, device="cuda"), sort.expert_prefix)
    assert y.shape == (rows.shape[0], 8) and bool((y == 0).all())
    none = adapter_projection(x.view(-1, H), torch.zeros(8, H, dtype=torch.bfloat16, device="cuda"), None, None, None,
                              torch.full((R * T,), -1, device="cuda"))
    assert bool((none == 0).all())


def test_calls_replay_in_a_cuda_graph():
    """All of the operators captured once and replayed on new values."""
    g = torch.Generator(device="cuda").manual_seed(6)
    N, L, r = 90, 3, 16
    idx = torch.randint(-1, E, (N, k), generator=g, device="cuda")
    x = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    w = torch.rand(N, k, generator=g, device="cuda")
    mats = (torch.randn(E, F, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    a, b = torch.randn(L, r, H, generator=g, device="cuda").bfloat16(), torch.randn(L, H, r, generator=g, device="cuda").bfloat16()
    shared, scales = torch.randn(H, H, generator=g, device="cuda").bfloat16(), torch.ones(L, device="cuda")
    who = torch.randint(-1, L, (N,), generator=g, device="cuda")
    rows = N * k                                             # room for any routing: no read-back in the graph

    def step():
        sort = ExpertSort(idx, E, H, rows=rows)
        h = expert_product(sort_rows(x, sort), mats, sort.expert_prefix)
        dx = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_gemm_dgrad(ep.ep_gemm_shape(rows, E, H, F), h, mats, sort.expert_prefix, dx)
        dw = torch.empty_like(mats)
        ep.ep_expert_gemm_wgrad(ep.ep_gemm_shape(rows, E, H, F), h, sort_rows(x, sort), sort.expert_prefix, dw)
        return unsort_rows(dx, sort, w), dw, adapter_projection(x, shared, a, b, scales, who)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (7, 8):
        g.manual_seed(seed)
        idx.copy_(torch.randint(-1, E, (N, k), generator=g, device="cuda"))
        x.copy_(torch.randn(N, H, generator=g, device="cuda"))
        who.copy_(torch.randint(-1, L, (N,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for have, want in zip(got, step()):
            assert torch.equal(have, want)
