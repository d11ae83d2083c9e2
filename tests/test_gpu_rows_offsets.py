"""Rows, matrices and adapters that lie more than 2^31 elements into their buffers. Whole numbers,
so that sums are exact; what is looked at is the end of each buffer."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from combine_layout_02_gb300.buffers import SortBuffers
from rows_util import integers

pytestmark = pytest.mark.gpu

WIDE, MANY, LAST = 8192, (1 << 18) + 40, 40          # MANY rows of WIDE values are 2^31 and some


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def rounded(t):
    return t.float().bfloat16()


def placed(k=1):
    """The last rows in experts of their own: they come first and last among the sorted rows."""
    idx = torch.full((MANY, k), 1, dtype=torch.int64, device="cuda")
    idx[-LAST:] = torch.arange(LAST, device="cuda").unsqueeze(1) % 3
    idx[-1] = -1
    sh = ep.make_shape(1, MANY, WIDE, 3, k)
    s = SortBuffers(sh)
    ep.ep_sort_layout(sh, idx, s.handle(), s.workspace)
    return sh, s


def test_rows_into_expert_order_and_back():
    sh, s = placed()
    at = s.entry_rows[-LAST:-1, 0].long()
    assert int(at.max()) * WIDE > 1 << 31
    x, xs = zeros(MANY, WIDE), zeros(MANY, WIDE)
    x[-LAST:] = integers(gen(1), LAST, WIDE)
    ep.ep_sort_rows(sh, x, ep.EP_BF16, None, s.handle(), xs, None)
    assert torch.equal(xs[at], x[-LAST:-1]) and int(xs.count_nonzero()) == int(x[:-1].count_nonzero())
    w = torch.rand(MANY, 1, generator=gen(2), device="cuda")
    out = torch.empty_like(x)
    ep.ep_unsort_rows(sh, xs, w, s.handle(), out)
    assert torch.equal(out[-LAST:-1], rounded(w[-LAST:-1] * x[-LAST:-1].float())) and not bool(out[-1].any())
    dout, dy, dw = integers(gen(3), MANY, WIDE, most=1), torch.empty_like(x), torch.empty_like(w)
    ep.ep_unsort_rows_backward(sh, dout, xs, w, s.handle(), dy, dw)
    assert torch.equal(dy[at], rounded(w[-LAST:-1] * dout[-LAST:-1].float()))
    assert torch.equal(dw[-LAST:-1, 0], (dout[-LAST:-1].double() * x[-LAST:-1].double()).sum(1).float())
    assert float(dw[-1]) == 0.0


def test_quantised_rows_into_expert_order():
    sh, s = placed(2)
    at = s.entry_rows[-LAST:-1].long()
    x, sc = zeros(MANY, WIDE, dtype=torch.uint8), zeros(MANY, WIDE // 128, dtype=torch.float32)
    x[-LAST:] = torch.randint(0, 120, (LAST, WIDE), generator=gen(4), device="cuda").to(torch.uint8)
    sc[-LAST:] = torch.rand(LAST, WIDE // 128, generator=gen(5), device="cuda")
    xs, scs = zeros(2 * MANY, WIDE, dtype=torch.uint8), zeros(2 * MANY, WIDE // 128, dtype=torch.float32)
    ep.ep_sort_rows(sh, x, ep.EP_FP8_E4M3, sc, s.handle(), xs, scs)
    for j in range(2):
        assert torch.equal(xs[at[:, j]], x[-LAST:-1]) and torch.equal(scs[at[:, j]], sc[-LAST:-1])


def test_matrices_gradient_from_far_rows():
    K, F = WIDE, 64
    x, dy = zeros(MANY, K), zeros(MANY, F)
    x[-LAST:], dy[-LAST:] = integers(gen(6), LAST, K), integers(gen(7), LAST, F)
    for edge in (MANY - 33, MANY - 40, MANY - 16):          # tails of 33, 40 and 16 rows
        prefix = torch.tensor([0, edge, MANY], dtype=torch.int32, device="cuda")
        dw = torch.full((2, F, K), 7.0, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_gemm_wgrad(ep.ep_gemm_shape(MANY, 2, K, F), dy, x, prefix, dw)
        for e, rows in ((0, slice(MANY - LAST, edge)), (1, slice(edge, MANY))):
            assert torch.equal(dw[e], rounded(dy[rows].double().t() @ x[rows].double()))


@pytest.mark.parametrize("rows", [5, 300])
def test_products_with_far_matrices(rows):
    E, K, F = 33, WIDE, WIDE
    g = gen(8)
    w = zeros(E, F, K)
    w[-1] = integers(g, F, K, most=1)
    x, dy = integers(g, rows, K, most=1), integers(g, rows, F, most=1)
    prefix = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    prefix[-1] = rows
    sh = ep.ep_gemm_shape(rows, E, K, F)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    ep.ep_expert_gemm(sh, x, w, prefix, y)
    assert torch.equal(y, rounded(x.float() @ w[-1].float().t()))          # sums below 2^24: exact in fp32
    ep.ep_expert_gemm_dgrad(sh, dy, w, prefix, dx)
    assert torch.equal(dx, rounded(dy.float() @ w[-1].float()))
    w.fill_(7)
    ep.ep_expert_gemm_wgrad(sh, dy, x, prefix, w)
    assert torch.equal(w[-1], rounded(dy.float().t() @ x.float())) and not bool(w[:-1].any())


def adapters(x, w, a, b, s, ids):
    (T, K), F, (L, r) = x.shape, w.shape[0], a.shape[:2]
    sh = ep.ep_adapter_shape(T, K, F, L, r)
    ws = torch.empty(ep.ep_adapter_workspace_size(sh), dtype=torch.uint8, device="cuda")
    y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    ep.ep_adapter_gemm(sh, x, w, a, b, s, ids, y, ws)
    return y


def check(y, x, w, a, b, s, ids, rows):
    for t in rows:
        e, i = x[t].double(), int(ids[t])
        want = w.double() @ e
        if i >= 0:
            want += s[i].double() * (b[i].double() @ (a[i].double() @ e))
        assert torch.equal(y[t], rounded(want)), t


@pytest.mark.parametrize("K,F", [(WIDE, 64), (64, WIDE)])
@pytest.mark.parametrize("order", ["any", "sorted"])
def test_projection_of_far_rows(K, F, order):
    g = gen(9)
    x = integers(g, MANY, K, most=1) if K < F else zeros(MANY, K)
    x[-LAST:] = 0
    x[-LAST:, :64] = integers(g, LAST, 64, most=1)
    w, a, b = integers(g, F, K, most=1), integers(g, 3, 8, K, most=1), integers(g, 3, F, 8, most=1)
    ids = torch.randint(-1, 3, (MANY,), generator=g, device="cuda")
    if order == "sorted":
        ids = ids.sort().values
    s = torch.tensor([1.0, 2.0, 1.0], device="cuda")
    y = adapters(x, w, a, b, s, ids)
    check(y, x, w, a, b, s, ids, list(range(MANY - LAST, MANY)) + [0, MANY // 2])


@pytest.mark.parametrize("T", [3, 300])
def test_projection_with_far_adapters(T):
    L, K, F, r = 2100, 64, WIDE, 128                    # B has L * F * r > 2^31 values
    g = gen(10)
    b = zeros(L, F, r)
    b[-2:] = integers(g, 2, F, r, most=1)
    a, w, x = integers(g, L, r, K, most=1), integers(g, F, K, most=1), integers(g, T, K, most=1)
    ids = L - 1 - torch.arange(T, device="cuda") % 2
    s = torch.ones(L, device="cuda")
    check(adapters(x, w, a, b, s, ids), x, w, a, b, s, ids, range(0, T, max(1, T // 40)))
