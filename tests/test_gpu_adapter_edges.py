"""The projection with adapters at the edges of its types, in every form it takes: few rows, many rows
by warp-level products of low's two bf16 terms, and many rows by fp32 multiply-adds."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from rows_util import U16, U32, assert_within, integers, sum_bound
from test_gpu_adapter import call, ids_of, make, normal, plain

pytestmark = pytest.mark.gpu

# rows, in_features, out_features, adapters, rank
FORMS = {
    "one": (1, 136, 264, 3, 16),
    "few": (40, 136, 264, 3, 16),
    "few_64": (90, 72, 136, 3, 64),
    "many_8": (700, 72, 264, 3, 8),
    "many_16": (700, 136, 264, 5, 16),
    "many_24": (1000, 72, 520, 40, 24),
    "many_64": (600, 264, 136, 3, 64),
    "many_72": (520, 72, 264, 4, 72),
    "many_short_runs": (2100, 72, 136, 700, 16),
    "plain": (2307, 2056, 4104, 7, 16),
    # contractions that several blocks share
    "one_shared": (1, 4096, 264, 3, 16),
    "few_shared": (40, 4104, 264, 3, 40),
    "hundred_shared": (100, 7168, 136, 30, 64),
    "many_shared": (300, 7168, 520, 3, 16),
    "many_64_shared": (520, 4096, 264, 4, 64),
}


def zeros(case, order, seed):
    """No projection, no adapters yet; every row's x is 1 in the first place and 0 elsewhere."""
    T, K, F, L, r = FORMS[case]
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    d = dict(x=bf(T, K), w=bf(F, K), a=bf(L, r, K), b=bf(L, F, r), s=torch.ones(L, device="cuda"), ids=ids_of(T, L, order, g))
    d["x"][:, 0] = 1
    d["ids"][0] = 0
    return d


@pytest.mark.parametrize("case", FORMS)
@pytest.mark.parametrize("order", ["any", "sorted"])
def test_low_at_the_end_of_fp32(case, order):
    """low values between bf16's and fp32's largest, scaled back by B: finite results. Everything
    but their one rounding, and where two bf16 terms stand for low its 2^-17, is exact."""
    d = zeros(case, order, 1)
    L, r = FORMS[case][3], FORMS[case][4]
    values = torch.tensor([3.39e38, 3.3961775e38, 3.397e38, 3.4e38, 3.4028234e38], device="cuda")
    d["s"] = values[torch.arange(L, device="cuda") % 5]
    rank = torch.arange(L, device="cuda") % r
    d["a"][torch.arange(L, device="cuda"), rank, 0] = torch.where(torch.arange(L, device="cuda") % 2 == 0, 1.0, -1.0).bfloat16()
    d["b"][torch.arange(L, device="cuda"), :, rank] = 2.0 ** -9
    got = call(d)
    y, delta = plain(d)
    assert bool(torch.isfinite(delta).all())
    assert_within(got, y + delta, 2.0 ** -17 * delta.abs(), U16)


@pytest.mark.parametrize("case", FORMS)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_low_not_finite(case, value):
    """An infinite low gives infinities of B's sign and NaN where B is zero; a NaN gives NaN."""
    d = zeros(case, "any", 2)
    F = FORMS[case][2]
    d["s"][0] = value
    d["a"][:, :, 0] = 1
    d["b"][:] = (torch.arange(F, device="cuda") % 3 - 1).bfloat16().view(1, F, 1)
    y, delta = plain(d)
    assert_within(call(d), y + delta, 0.0)


@pytest.mark.parametrize("case", FORMS)
def test_the_scale_is_of_the_whole_sum(case):
    """A x whose terms cancel over the contraction: times the scale they would be infinite, their sum is not."""
    d = zeros(case, "any", 3)
    K = FORMS[case][1]
    d["x"][:, K - 1] = 1
    d["s"][:] = 1e37
    d["a"][:, :, 0], d["a"][:, :, K - 1] = 100, -99
    d["b"][:, :, 0] = 2.0 ** -9
    y, delta = plain(d)
    assert bool(torch.isfinite(delta).all()) and bool((delta > 0).any())
    assert_within(call(d), y + delta, 2.0 ** -17 * delta.abs(), U16)


@pytest.mark.parametrize("case", FORMS)
@pytest.mark.parametrize("order", ["any", "sorted"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_b_not_finite(case, order, value):
    """An infinite value of B gives infinities of low's sign, NaN where low is zero, and leaves the features
    beside it alone."""
    d = zeros(case, order, 4)
    T, K, F, L, r = FORMS[case]
    g = torch.Generator(device="cuda").manual_seed(5)
    lows = torch.tensor([1.0, -2.0, 1.00390625, -1.01171875, 0.0, 1.0048828125, -3.0048828125], device="cuda")
    d["x"][:, 0] = 1
    d["x"][:, 1] = torch.randint(0, 7, (T,), generator=g, device="cuda").bfloat16()
    d["x"][:, 0] = lows[d["x"][:, 1].long()].bfloat16()
    d["x"][:, 1] = 0
    d["x"][:, 2] = (lows[torch.randint(0, 7, (T,), generator=g, device="cuda")] * 2.0 ** -11).bfloat16()
    d["a"][:, r - 1, 0], d["a"][:, r - 1, 2], d["a"][:, 0, 0] = 1, 1, 1
    d["b"][:, :, 0] = 1                                     # every feature: low of the first rank
    d["b"][0, 5, r - 1], d["b"][L - 1, F - 1, r - 1], d["b"][L // 2, 70, 0] = value, value, value
    y, delta = plain(d)
    _, mdelta = plain(d, absolute=True)
    got, slack = call(d), 2.0 ** -17 * torch.nan_to_num(mdelta, posinf=0.0)
    if case.startswith("many"):          # two terms of low: not finite, but NaN as well as an infinity
        bad = ~torch.isfinite(delta)
        assert torch.equal(~torch.isfinite(got), bad)
        got, delta = torch.where(bad, 0, got), torch.where(bad, 0, delta)
    assert_within(got, y + delta, slack, U16)


@pytest.mark.parametrize("T", [1, 32, 128, 129, 257, 70001])
def test_ids_without_any_adapter(T):
    """L = 0: the projection alone, every id but -1 flagged wherever it stands."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x, w = integers(g, T, 64), integers(g, 72, 64)
    d = dict(x=x, w=w, a=None, b=None, s=None, ids=torch.full((T,), -1, device="cuda"))
    want = (x.double() @ w.double().t()).float().bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(call(d, err=err), want) and int(err.item()) == 0
    for at in sorted({0, T // 2, T - 1}):
        d["ids"].fill_(-1)
        d["ids"][at] = 0
        err.zero_()
        assert torch.equal(call(d, err=err), want) and int(err.item()) == ep.EP_DEVERR_BAD_ADAPTER


# many rows of a short contraction, where what two bf16 terms leave of low shows beside the sums' bounds
SHORT = [(300, 8, 264, 3, 16), (700, 8, 264, 2, 64), (9001, 8, 136, 5, 8), (1000, 16, 520, 6, 24), (600, 24, 136, 300, 72),
         (2100, 32, 384, 40, 256), (513, 40, 776, 2, 32)]


@pytest.mark.parametrize("case", SHORT)
@pytest.mark.parametrize("order", ["any", "sorted", "one"])
def test_short_contractions(case, order):
    T, K, F, L, r = case
    d = make(case, order, 7, normal)
    (y, delta), (my, mdelta) = plain(d), plain(d, absolute=True)
    # as for longer ones (K products; the adapter's K products, scale and r products), and of low * B the part that
    # low's two terms leave: of a low in [1, 2) the first leaves less than 2^-8, whose unit in bf16 is 2^-16 or
    # smaller, and the second half a unit of that
    slack = sum_bound(K + 1, my, 2 * U32) + sum_bound(K + r + 3, mdelta, 2 * U32) + 2.0 ** -17 * mdelta
    got = call(d)
    assert_within(got, y + delta, slack, U16)
    assert torch.equal(got, call(d))
