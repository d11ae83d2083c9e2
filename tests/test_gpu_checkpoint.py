"""Rows kept in 8 bits against a search over e4m3's values, byte by byte, and the matrices' gradient from kept
rows against 64 bits."""
import math

import pytest
import torch

import combine_layout_02_gb300 as ep
from combine_layout_02_gb300.experts import checkpoint_rows, restore_rows
from kept_util import GROUP, quantised, stands_for
from rows_util import U16, U32, assert_within, integers, sum_bound

pytestmark = pytest.mark.gpu


def wide_rows(rows, features, seed):
    """Values whose magnitudes go over many powers of two, within groups and between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, features, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-8, 4, (rows, features), generator=g, device="cuda").float())
    return (x * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g, device="cuda").float())).bfloat16()


@pytest.mark.parametrize("rows,features", [(1, 8), (1, 16), (2, 24), (7, 40), (3, 4104), (129, 200), (64, 512), (300, 136),
                                           (1, 7168), (1000, 16), (3, 1 << 17)])
def test_bytes_and_values(rows, features):
    x = wide_rows(rows, features, rows + features)
    x[0, :5] = torch.tensor([0.0, -0.0, 1.0, -1.0, 0.5], device="cuda")
    width = -(-features // GROUP) * GROUP
    values = torch.full((rows + 2, width), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 2, width // GROUP), 0xA5, dtype=torch.uint8, device="cuda")
    kept = ep.make_checkpoint(values[1:-1], scales[1:-1])
    ep.ep_checkpoint_rows(rows, features, x, kept)
    q, k, v = quantised(x)
    assert torch.equal(values[1:-1].cpu(), q) and torch.equal(scales[1:-1].cpu(), k)
    for t in (values, scales):
        assert bool((t[0] == 0xA5).all()) and bool((t[-1] == 0xA5).all())
    back = torch.full((rows + 2, features), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_restore_rows(rows, features, kept, back[1:-1])
    assert torch.equal(back[1:-1].cpu().double(), v)
    assert bool((back[0] == 7).all()) and bool((back[-1] == 7).all())
    # nearest of the type's values: 2^-4 relatively, half of 2^-9 of the group's power of two where they lie even
    step = torch.exp2(k.double() - 127).repeat_interleave(GROUP, 1)[:, :features] * 2.0 ** -10
    assert bool(((v - x.cpu().double()).abs() <= torch.maximum(x.cpu().double().abs() / 16, step)).all())


def test_every_value_of_a_binade():
    """Each bf16 value of two binades beside 448 (a power of two that stays) and alone (one of its own)."""
    v = torch.arange(256 * 2, dtype=torch.int32) + 0x4380                     # 256 up to below 1024
    v = (v << 16).view(torch.float32)
    x = torch.zeros(2 * len(v), 16)
    x[:len(v), 3] = v
    x[len(v):, 9], x[len(v):, 0] = v / 512, 448.0
    x = x.bfloat16().cuda()
    values, scales = checkpoint_rows(x)
    q, k, back = quantised(x)
    assert torch.equal(values.cpu(), q) and torch.equal(scales.cpu(), k)
    assert torch.equal(restore_rows(values, scales, 16).cpu().double(), back)


def test_zeros_infinities_nan_and_extremes():
    nan, inf = math.nan, math.inf
    rows = [[0.0] * 16, [-0.0] * 16, [nan] + [1.0] * 15, [nan] * 16, [nan, 3.0] * 8, [3.0, nan] * 8, [inf, 1.0, -2.0, 1e38, -3e38] + [0.0] * 11,
            [-inf] * 16, [nan, -inf] + [1e30] * 14, [3.3895e38, -3.2e38, 1.0] + [2.0 ** -126] * 13, [2.0 ** -126, 2.0 ** -130, 2.0 ** -133] + [0.0] * 13,
            [2.0 ** -110] * 8 + [-(2.0 ** -120)] * 8, [448.0, 449.0] + [1.0] * 14]
    x = torch.tensor(rows, dtype=torch.float32).bfloat16().cuda()
    values, scales = checkpoint_rows(x)
    q, k, v = quantised(x)
    nans = torch.isnan(x).cpu()
    assert torch.equal(scales.cpu()[~nans.all(1)], k[~nans.all(1)])          # (a group of NaN alone: any)
    assert torch.equal(values.cpu()[~nans], q[~nans]) and bool(((values.cpu()[nans] & 127) == 127).all())
    back = restore_rows(values, scales, 16).cpu().double()
    assert torch.equal(torch.isnan(back), nans)
    # exact but where a value is below bf16's least one
    assert torch.equal(back[~nans], v.float().bfloat16().double()[~nans])


def test_two_streams_and_a_replay():
    x = [wide_rows(200, 136, s) for s in (1, 2)]
    want = [quantised(t) for t in x]
    streams = [torch.cuda.Stream() for _ in x]
    got = []
    for s, t in zip(streams, x):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            kept = checkpoint_rows(t)
            got.append((*kept, restore_rows(*kept, 136)))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for g, w in zip(got, want):
        assert torch.equal(g[0].cpu(), w[0]) and torch.equal(g[1].cpu(), w[1]) and torch.equal(g[2].cpu().double(), w[2])
    still = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = checkpoint_rows(still)
        back = restore_rows(*kept, 136)
    still.copy_(x[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept[0].cpu(), want[1][0]) and torch.equal(back.cpu().double(), want[1][2])


def test_no_rows_and_refused_types():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    values, scales = checkpoint_rows(x)
    assert values.shape == (0, 64) and scales.shape == (0, 4) and restore_rows(values, scales, 64).shape == (0, 64)
    with pytest.raises(ValueError):
        checkpoint_rows(x.float())


def test_rows_beyond_two_to_the_32_bytes():
    rows, features = 300_007, 8184                       # 2.46e9 values; the last group of a row is half a one
    x = torch.zeros(rows, features, dtype=torch.bfloat16, device="cuda")
    tail = wide_rows(64, features, 3)
    x[-64:] = tail
    values, scales = checkpoint_rows(x)
    q, k, v = quantised(tail)
    assert torch.equal(values[-64:].cpu(), q) and torch.equal(scales[-64:].cpu(), k)
    assert not bool(values[:-64].any())
    del x
    assert torch.equal(restore_rows(values, scales, features)[-64:].cpu().double(), v)


# ------------------------------------------------------------------ the matrices' gradient from kept rows

CASES = {
    "one_row": ([1], 8, 8),
    "empty_between": ([0, 5, 0, 0, 3, 0], 64, 136),
    "odd": ([17, 1, 33, 130], 72, 200),
    "tile_edges": ([128, 127, 129, 256, 255, 257], 136, 256),
    "half_groups": ([63, 65, 64, 0, 200], 264, 392),
    "one_long_expert": ([4099], 264, 392),
    "many_experts": ([(7 * e) % 5 for e in range(300)], 64, 128),
    "wide": ([60, 300], 2056, 128),
    "train": ([500, 77, 0, 1300], 1024, 640),
}


def gradient(counts, K, F, seed, make, before=3, after=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, rows = len(counts), sum(counts)
    prefix = torch.zeros(E + 1, dtype=torch.int32)
    prefix[1:] = torch.tensor(counts).cumsum(0)
    prefix = (prefix + before).int().cuda()
    total = before + rows + after
    x, dy = (torch.full((total, n), math.nan, dtype=torch.bfloat16, device="cuda") for n in (K, F))
    x[before:before + rows] = make(g, rows, K)
    dy[before:before + rows] = make(g, rows, F)
    values, scales = checkpoint_rows(x)
    sh = ep.ep_gemm_shape(total, E, K, F)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = torch.full((E, F, K), 7.0, dtype=torch.bfloat16, device="cuda")
    workspace = torch.empty(max(16, ep.ep_wgrad_checkpoint_workspace_size(sh)), dtype=torch.uint8, device="cuda")
    ep.ep_expert_gemm_wgrad_checkpoint(sh, dy, ep.make_checkpoint(values, scales), prefix, dw, workspace,
                                       ep.make_launch(error_flags=err))
    kept = stands_for(values, scales, K)
    want, magnitude = torch.zeros(E, F, K, dtype=torch.float64, device="cuda"), torch.zeros(E, F, K, dtype=torch.float64, device="cuda")
    edge = prefix.tolist()
    for e in range(E):
        at = slice(edge[e], edge[e + 1])
        want[e] = dy[at].double().t() @ kept[at]
        magnitude[e] = dy[at].double().abs().t() @ kept[at].abs()
    assert int(err.item()) == 0
    return dw, want, magnitude, max(counts)


@pytest.mark.parametrize("name", CASES)
def test_gradient_whole_numbers(name):
    counts, K, F = CASES[name]
    dw, want, _, _ = gradient(counts, K, F, 1, integers)               # up to 3: exact in e4m3
    assert torch.equal(dw, want.to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("name", CASES)
def test_gradient_random_numbers(name):
    counts, K, F = CASES[name]
    dw, want, magnitude, most = gradient(counts, K, F, 2, lambda g, *s: torch.randn(*s, generator=g, device="cuda").bfloat16())
    assert_within(dw, want, sum_bound(most, magnitude, 2 * U32), U16)


def test_gradient_repeats_bit_for_bit():
    once = gradient([500, 77, 0, 1300], 1024, 640, 5, lambda g, *s: torch.randn(*s, generator=g, device="cuda").bfloat16())[0]
    again = gradient([500, 77, 0, 1300], 1024, 640, 5, lambda g, *s: torch.randn(*s, generator=g, device="cuda").bfloat16())[0]
    assert torch.equal(once, again)


def test_gradient_without_rows():
    sh = ep.ep_gemm_shape(0, 3, 64, 32)
    dw = torch.full((3, 32, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 64, dtype=torch.uint8, device="cuda")
    workspace = torch.empty(16, dtype=torch.uint8, device="cuda")
    ep.ep_expert_gemm_wgrad_checkpoint(sh, None, ep.make_checkpoint(none, none[:, :4].contiguous()),
                                       torch.zeros(4, dtype=torch.int32, device="cuda"), dw, workspace)
    assert not bool(dw.any())
