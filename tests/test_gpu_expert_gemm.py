"""The experts' products and their gradients against plain forms in 64 bits: whole numbers
exactly, random numbers within the fp32 summation bound and one bf16 rounding."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from rows_util import U16, U32, assert_within, integers, sum_bound

pytestmark = pytest.mark.gpu

# rows per expert, in_features, out_features
CASES = {
    "one_value_tile": ([1], 8, 8),
    "one_row": ([1], 256, 128),
    "empty_between": ([0, 5, 0, 0, 3, 0], 64, 136),
    "odd": ([17, 1, 33, 130], 72, 200),
    "tile_edges": ([128, 127, 129, 256, 255, 257], 128, 256),
    "long_experts": ([1000, 24, 700], 192, 264),
    "deep": ([70, 9], 2056, 128),
    "wide": ([60, 300], 128, 2056),
    "many_experts": ([(7 * e) % 5 for e in range(300)], 64, 128),
    "one_each": ([1] * 32, 520, 392),
    "few_rows_deep": ([3, 0, 2, 5, 1, 0, 4, 1], 4096, 256),
    "many_rows_few_features": ([3000, 0, 1111, 1], 136, 200),
    "one_long_expert": ([4099], 264, 392),
    "decode": ([16, 30, 8, 15, 2, 40, 0, 9], 1024, 1024),
}


def data(counts, K, F, seed, make, before=0, after=0):
    """Rows of the experts, with `before` / `after` rows of no expert around them (NaN)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, rows = len(counts), sum(counts)
    prefix = torch.zeros(E + 1, dtype=torch.int32)
    prefix[1:] = torch.tensor(counts).cumsum(0)
    prefix = (prefix + before).int().cuda()
    full = lambda n: torch.full((before + rows + after, n), float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, dy = full(K), full(F)
    x[before:before + rows] = make(g, rows, K)
    dy[before:before + rows] = make(g, rows, F)
    return x, dy, make(g, E, F, K), prefix, before + rows + after


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


class Products:
    def __init__(self, x, dy, w, prefix, num_rows):
        E, F, K = w.shape
        self.sh = ep.ep_gemm_shape(num_rows, E, K, F)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        launch = ep.make_launch(error_flags=self.err)
        fill = lambda *shape: torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.y, self.dx, self.dw = fill(num_rows, F), fill(num_rows, K), fill(E, F, K)
        ep.ep_expert_gemm(self.sh, x, w, prefix, self.y, launch)
        ep.ep_expert_gemm_dgrad(self.sh, dy, w, prefix, self.dx, launch)
        ep.ep_expert_gemm_wgrad(self.sh, dy, x, prefix, self.dw, launch)
        torch.cuda.synchronize()


def plain(x, dy, w, edges, absolute=False):
    """(y, dx, dw) in 64 bits; rows of no expert 7."""
    f = (lambda t: t.double().abs()) if absolute else (lambda t: t.double())
    E, F, K = w.shape
    y = torch.full((len(x), F), 7.0, dtype=torch.float64, device="cuda")
    dx = torch.full((len(x), K), 7.0, dtype=torch.float64, device="cuda")
    dw = torch.zeros(E, F, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        at = slice(edges[e], edges[e + 1])
        y[at] = f(x[at]) @ f(w[e]).t()
        dx[at] = f(dy[at]) @ f(w[e])
        dw[e] = f(dy[at]).t() @ f(x[at])
    return y, dx, dw


@pytest.mark.parametrize("name", CASES)
def test_whole_numbers(name):
    counts, K, F = CASES[name]
    x, dy, w, prefix, n = data(counts, K, F, 1, integers, before=3, after=5)
    p = Products(x, dy, w, prefix, n)
    assert int(p.err.item()) == 0
    for got, want in zip((p.y, p.dx, p.dw), plain(x, dy, w, prefix.tolist())):
        assert torch.equal(got, want.to(torch.float32).to(torch.bfloat16))     # exact sums, rounded once


@pytest.mark.parametrize("counts,K,F", [([500, 77, 0, 1300], 1024, 640), ([5, 0, 61, 2], 7168, 256), ([2100], 512, 2048),
                                        ([900, 800, 3, 1000], 2048, 1280)])
def test_random_numbers(counts, K, F):
    x, dy, w, prefix, n = data(counts, K, F, 2, normal)
    p = Products(x, dy, w, prefix, n)
    want, mags = plain(x, dy, w, prefix.tolist()), plain(x, dy, w, prefix.tolist(), absolute=True)
    longest = max(counts)
    for got, e, m, terms in zip((p.y, p.dx, p.dw), want, mags, (K, F, longest)):
        assert_within(got, e, sum_bound(terms, m, 2 * U32), U16)
    q = Products(x, dy, w, prefix, n)
    assert torch.equal(p.y, q.y) and torch.equal(p.dx, q.dx) and torch.equal(p.dw, q.dw)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("counts", [[65, 30, 100], [3, 2, 4], [300, 200, 290]])
def test_one_experts_values_stay_its_own(bad, counts):
    K, F = 200, 136
    x, dy, w, prefix, n = data(counts, K, F, 3, integers)
    clean = plain(x, dy, w, prefix.tolist())
    at = slice(counts[0], counts[0] + counts[1])
    x[at], dy[at], w[1] = bad, bad, bad
    p = Products(x, dy, w, prefix, n)
    others = [i for i in range(n) if not at.start <= i < at.stop]
    assert torch.equal(p.y[others], clean[0][others].bfloat16()) and torch.equal(p.dx[others], clean[1][others].bfloat16())
    assert torch.equal(p.dw[[0, 2]], clean[2][[0, 2]].bfloat16())
    assert not bool(torch.isfinite(p.y[at]).any()) and not bool(torch.isfinite(p.dw[1]).any())


def test_an_infinite_value_reaches_its_own_row_only():
    counts, K, F = [20, 40], 128, 256
    x, dy, w, prefix, n = data(counts, K, F, 4, integers)
    w = w.abs() + 1
    x[25, 9] = float("inf")
    p = Products(x, dy, w, prefix, n)
    assert bool((p.y[25] == float("inf")).all())
    assert bool(torch.isfinite(p.y[[i for i in range(n) if i != 25]]).all())


def test_no_rows_at_all():
    w = torch.ones(3, 16, 24, dtype=torch.bfloat16, device="cuda")
    sh = ep.ep_gemm_shape(0, 3, 24, 16)
    prefix, dw = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full_like(w, 7.0)
    none = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gemm(sh, none, w, prefix, none)
    ep.ep_expert_gemm_dgrad(sh, none, w, prefix, none)
    ep.ep_expert_gemm_wgrad(sh, none, none, prefix, dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("prefix", [[0, 5, 40], [-3, 5, 20], [0, 9, 4], [50, 60, 70]])
def test_a_prefix_outside_the_rows_is_clipped_and_flagged(prefix):
    K, F, n = 64, 64, 20
    x, dy, w, _, _ = data([n], K, F, 5, integers)
    w = integers(torch.Generator(device="cuda").manual_seed(6), 2, F, K)
    p = Products(x, dy, w, torch.tensor(prefix, dtype=torch.int32, device="cuda"), n)
    assert int(p.err.item()) == ep.EP_DEVERR_RECV_OVERFLOW
    want = torch.full((n, F), 7.0, dtype=torch.float64, device="cuda")
    for e in range(2):
        b, t = min(max(prefix[e], 0), n), min(max(prefix[e + 1], 0), n)
        if t > b:
            want[b:t] = x[b:t].double() @ w[e].double().t()
    assert torch.equal(p.y, want.bfloat16())


def test_gradients_against_differences():
    """Whole numbers, every sum exact: a step in the rows and in the matrices changes the products
    by what the gradients say."""
    counts, K, F = [19, 0, 70, 33], 136, 72
    x, dy, w, prefix, n = data(counts, K, F, 7, lambda g, *s: integers(g, *s, most=1))
    g = torch.Generator(device="cuda").manual_seed(8)
    dxs, dws = integers(g, n, K, most=1), integers(g, len(counts), F, K, most=1)
    base, p = Products(x, dy, w, prefix, n).y.double(), Products(x, dy, w, prefix, n)
    d = dy.double()
    # |y| <= 136 * 2 < 256: exact in bf16, as are the gradients
    assert ((Products(x + dxs, dy, w, prefix, n).y.double() - base) * d).sum() == (p.dx.double() * dxs.double()).sum()
    assert ((Products(x, dy, w + dws, prefix, n).y.double() - base) * d).sum() == (p.dw.double() * dws.double()).sum()


def test_rows_beyond_32_bit_offsets():
    """The last expert's rows begin more than 2^31 elements into the row buffers."""
    K, F, n = 8192, 64, (1 << 18) + 40
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    x[-40:] = integers(g, 40, K, most=1)
    w = integers(g, 2, F, K, most=1)
    prefix = torch.tensor([0, n - 33, n], dtype=torch.int32, device="cuda")
    sh = ep.ep_gemm_shape(n, 2, K, F)
    y = torch.empty(n, F, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gemm(sh, x, w, prefix, y)
    assert torch.equal(y[-33:], (x[-33:].double() @ w[1].double().t()).float().bfloat16())
    assert torch.equal(y[-40:-33], (x[-40:-33].double() @ w[0].double().t()).float().bfloat16())
    dx = torch.empty_like(x)
    ep.ep_expert_gemm_dgrad(sh, y, w, prefix, dx)
    want = (y[-33:].double() @ w[1].double())
    mags = (y[-33:].double().abs() @ w[1].double().abs())
    assert_within(dx[-33:], want, sum_bound(F, mags, 2 * U32), U16)


def test_a_threads_first_call():
    """A thread that has made no CUDA call before (as autograd's has not)."""
    import threading
    x, dy, w, prefix, n = data([40, 30], 128, 64, 10, integers)
    want, got = Products(x, dy, w, prefix, n), []
    sh, y = ep.ep_gemm_shape(n, 2, 128, 64), torch.empty_like(dy)
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        try:
            ep.ep_expert_gemm(sh, x, w, prefix, y, ep.ep_launch(stream or None, None, None, None))
            got.append(None)
        except Exception as e:
            got.append(e)

    t = threading.Thread(target=call)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got == [None] and torch.equal(y, want.y)
