"""The shared projection with each row's low-rank adapter against a plain form in 64 bits."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from rows_util import U16, U32, assert_within, integers, sum_bound

pytestmark = pytest.mark.gpu

# rows, in_features, out_features, adapters, rank
CASES = [(1, 8, 8, 1, 8), (1, 4096, 512, 8, 16), (2, 72, 200, 3, 24), (7, 520, 136, 2, 64), (16, 1024, 256, 16, 8),
         (33, 256, 392, 64, 16), (61, 2048, 640, 5, 32), (130, 640, 264, 4, 128), (257, 128, 256, 3, 256),
         (300, 384, 128, 300, 8), (1000, 512, 520, 6, 16), (700, 264, 776, 2, 64), (2100, 1024, 384, 40, 40),
         (9001, 64, 136, 5, 8), (8193, 72, 264, 700, 16), (200, 64, 72, 2000, 8), (100, 4096, 256, 3, 24), (65, 72, 4104, 30, 72)]


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def ids_of(T, L, order, g):
    ids = torch.randint(0, L, (T,), generator=g, device="cuda")
    if order == "sorted":
        ids = ids.sort().values
    if order == "one":
        ids = torch.full_like(ids, L - 1)
    ids[torch.rand(T, generator=g, device="cuda") < 0.15] = -1
    return ids


def make(case, order, seed, data):
    T, K, F, L, r = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    return dict(x=data(g, T, K), w=data(g, F, K), a=data(g, L, r, K), b=data(g, L, F, r),
                s=torch.randint(1, 4, (L,), generator=g, device="cuda").float(), ids=ids_of(T, L, order, g))


def call(d, launch=None, err=None):
    T, K = d["x"].shape
    F = d["w"].shape[0]
    L, r = (d["a"].shape[0], d["a"].shape[1]) if d["a"] is not None else (0, 8)
    sh = ep.ep_adapter_shape(T, K, F, L, r)
    ws = torch.empty(max(16, ep.ep_adapter_workspace_size(sh)), dtype=torch.uint8, device="cuda").fill_(0xFF)
    y = torch.full((T, F), 7.0, dtype=torch.bfloat16, device="cuda")
    launch = launch or ep.make_launch(error_flags=err)
    ep.ep_adapter_gemm(sh, d["x"], d["w"], d["a"], d["b"], d["s"], d["ids"], y, ws, launch)
    return y


def plain(d, absolute=False):
    f = (lambda t: t.double().abs()) if absolute else (lambda t: t.double())
    y = f(d["x"]) @ f(d["w"]).t()
    delta = torch.zeros_like(y)
    for i in range(0 if d["a"] is None else len(d["a"])):
        t = (d["ids"] == i).nonzero().reshape(-1)
        delta[t] = f(d["s"][i]) * ((f(d["x"][t]) @ f(d["a"][i]).t()) @ f(d["b"][i]).t())
    return y, delta


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("order", ["any", "sorted", "one"])
def test_random_numbers(case, order):
    T, K, F, L, r = case
    d = make(case, order, 1, normal)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(d, err=err)
    (y, delta), (my, mdelta) = plain(d), plain(d, absolute=True)
    # the projection: K products; the adapter: K products, the scale, r products; their sum
    slack = sum_bound(K + 1, my, 2 * U32) + sum_bound(K + r + 3, mdelta, 2 * U32)
    assert_within(got, y + delta, slack, U16)
    assert int(err.item()) == 0
    assert torch.equal(got, call(d))


# Many tiles of a long contraction with few ranks.
FEW_RANKS = [(2100, 1032, 4360, 5, 8), (2307, 2056, 4104, 40, 16)]


@pytest.mark.parametrize("case", FEW_RANKS)
@pytest.mark.parametrize("order", ["any", "sorted"])
def test_few_ranks_many_tiles(case, order):
    test_random_numbers(case, order)


@pytest.mark.parametrize("case", FEW_RANKS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_few_ranks_many_tiles_stay_their_own(case, bad):
    T, L = case[0], case[3]
    for order in ("any", "sorted"):
        d = make(case, order, 4, lambda g, *s: integers(g, *s, most=1))
        y, delta = plain(d)
        d["a"][1], d["b"][1], d["s"][1] = bad, bad, bad
        got, others = call(d), d["ids"] != 1
        assert torch.equal(got[others], (y + delta).float().bfloat16()[others])
        assert bool(torch.isnan(got[~others]).all())


@pytest.mark.parametrize("case", [(5, 72, 136, 3, 8), (61, 264, 392, 7, 16), (300, 136, 264, 4, 64), (90, 1024, 128, 2, 128)])
def test_whole_numbers(case):
    d = make(case, "any", 2, lambda g, *s: integers(g, *s, most=1))
    y, delta = plain(d)
    assert torch.equal(call(d), (y + delta).float().bfloat16())


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_one_adapters_values_stay_its_own(T, bad):
    case = (T, 136, 264, 3, 16)
    d = make(case, "any", 3, lambda g, *s: integers(g, *s, most=1))
    d["ids"][0], d["ids"][1], d["ids"][2] = 0, 1, -1
    y, delta = plain(d)
    d["a"][1], d["b"][1], d["s"][1] = bad, bad, bad
    got = call(d)
    others = d["ids"] != 1
    assert torch.equal(got[others], (y + delta)[others].float().bfloat16())
    assert not bool(torch.isfinite(got[~others]).any())


def test_no_adapters_and_no_rows():
    d = make((20, 64, 72, 2, 8), "any", 4, integers)
    y, _ = plain(d)
    want = y.float().bfloat16()
    d["ids"].fill_(-1)
    assert torch.equal(call(d), want)
    d["a"] = d["b"] = d["s"] = None
    assert torch.equal(call(d), want)
    d["x"], d["ids"] = d["x"][:0], d["ids"][:0]
    assert call(d).shape == (0, 72)


def test_ids_out_of_range_are_flagged_and_take_no_adapter():
    d = make((50, 64, 72, 3, 8), "any", 5, lambda g, *s: integers(g, *s, most=1))
    d["ids"][4], d["ids"][40], d["ids"][9] = 3, -2, 1 << 40
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(d, err=err)
    y, delta = plain(d)
    assert torch.equal(got, (y + delta).float().bfloat16())
    assert int(err.item()) == ep.EP_DEVERR_BAD_ADAPTER


def test_on_a_stream_with_events():
    d = make((200, 512, 256, 4, 16), "any", 6, normal)
    want, late = call(d), dict(d, x=torch.zeros_like(d["x"]))
    torch.cuda.synchronize()
    side, ready, done = torch.cuda.Stream(), torch.cuda.Event(), torch.cuda.Event()
    done.record()
    torch.cuda._sleep(2_000_000)
    late["x"].copy_(d["x"])                          # still to come when the call below is made
    ready.record()
    got = torch.empty_like(want)
    sh = ep.ep_adapter_shape(200, 512, 256, 4, 16)
    ws = torch.empty(ep.ep_adapter_workspace_size(sh), dtype=torch.uint8, device="cuda")
    ep.ep_adapter_gemm(sh, late["x"], d["w"], d["a"], d["b"], d["s"], d["ids"], got, ws,
                       ep.make_launch(side, wait_event=ready, record_event=done))
    torch.cuda.current_stream().wait_event(done)
    assert torch.equal(got, want)
