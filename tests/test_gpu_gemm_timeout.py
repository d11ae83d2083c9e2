"""The products' waits give up after their time limit: an operand that does not arrive leaves its
tile unwritten in every CTA that shares it, sets EP_DEVERR_TIMEOUT, and the context stays usable."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from rows_util import integers

pytestmark = pytest.mark.gpu

FORWARD, DGRAD, WGRAD = 0, 1, 2
CALLS = (ep.ep_expert_gemm, ep.ep_expert_gemm_dgrad, ep.ep_expert_gemm_wgrad)

# product, rows per expert, in_features, out_features, contracted values that arrive
CASES = {
    "pairs": (FORWARD, [300, 200], 512, 520, 128),
    "pairs_nothing": (FORWARD, [300, 200], 512, 520, 0),
    "pairs_last_step": (FORWARD, [700], 520, 264, 512),
    "pairs_many_tiles": (FORWARD, [9000, 9000], 256, 1024, 192),
    "narrow": (FORWARD, [3, 0, 5], 256, 136, 128),
    "cluster_last_part": (FORWARD, [3, 5, 2], 4096, 256, 64 * 60),
    "cluster_first_part_alone": (FORWARD, [3, 5, 2], 4096, 256, 64 * 8),
    "wide_cluster": (FORWARD, [200], 8192, 256, 64 * 100),
    "dgrad_pairs": (DGRAD, [300, 200], 520, 512, 128),
    "dgrad_cluster": (DGRAD, [3, 5, 2], 256, 4096, 64 * 60),
    "wgrad_pairs": (WGRAD, [200, 300], 264, 520, 128),
    "wgrad_tail": (WGRAD, [70, 100], 264, 520, 64),
    "wgrad_cluster": (WGRAD, [2050], 128, 136, 64 * 20),
    "wgrad_cluster_tail": (WGRAD, [2050], 128, 136, 64 * 32),
}


def make(case):
    product, counts, K, F, _ = CASES[case]
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, E = sum(counts), len(counts)
    x, dy, w = integers(g, rows, K), integers(g, rows, F), integers(g, E, F, K)
    prefix = torch.tensor([0] + counts).cumsum(0).int().cuda()
    a, b, shape = [(x, w, (rows, F)), (dy, w, (rows, K)), (dy, x, (E, F, K))][product]
    return product, ep.ep_gemm_shape(rows, E, K, F), a, b, prefix, shape


def run(call, shape):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(shape, 7.5, dtype=torch.bfloat16, device="cuda")
    call(out, ep.make_launch(error_flags=err))
    torch.cuda.synchronize()
    return out, int(err.item())


@pytest.mark.parametrize("case", CASES)
def test_tiles_without_their_operands_are_not_written(case):
    product, sh, a, b, prefix, shape = make(case)
    loads, test = CASES[case][4], ep.ep_selftest_gemm_timeout
    want, flags = run(lambda out, la: CALLS[product](sh, a, b, prefix, out, la), shape)
    assert flags == 0 and not bool((want == 7.5).all())
    out, flags = run(lambda out, la: test(sh, product, a, b, prefix, out, loads, 20, la), shape)
    assert flags == ep.EP_DEVERR_TIMEOUT
    assert bool((out == 7.5).all())
    # with operands that do arrive it is the product, and the product right after is itself
    out, flags = run(lambda out, la: test(sh, product, a, b, prefix, out, 1 << 20, 2000, la), shape)
    assert flags == 0 and torch.equal(out, want)
    out, flags = run(lambda out, la: CALLS[product](sh, a, b, prefix, out, la), shape)
    assert flags == 0 and torch.equal(out, want)


# One tile's products take longer than the limit of a wait, but nothing is missing: rows of one expert
# beside many empty ones (pairs), of one expert (a cluster), with and without a tail. (The limit is first
# looked at after many tries, about 0.1 s.)
LONG = [([0] * 30 + [64_000_000] + [0] * 41, 8, 8), ([0] * 30 + [60_000_037, 1_000_001] + [0] * 41, 16, 8),
        ([400_000_001], 8, 8)]


@pytest.mark.parametrize("counts,K,F", LONG)
def test_long_products_are_not_given_up(counts, K, F):
    rows, E = sum(counts), len(counts)
    x = torch.ones(rows, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(rows, F, dtype=torch.bfloat16, device="cuda")
    dy[::9973] = 1
    prefix = torch.tensor([0] + counts).cumsum(0).int().cuda()
    want = torch.stack([torch.full((F, K), float(dy[a:b, 0].float().sum()), device="cuda")
                        for a, b in zip(prefix.tolist()[:-1], prefix.tolist()[1:])]).bfloat16()
    sh = ep.ep_gemm_shape(rows, E, K, F)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

    def call(out, launch):
        start.record()
        ep.ep_selftest_gemm_timeout(sh, WGRAD, dy, x, prefix, out, 1 << 30, 1, launch)
        stop.record()

    out, flags = run(call, (E, F, K))
    assert start.elapsed_time(stop) > 120                 # ms: longer than it takes to give up
    assert flags == 0 and torch.equal(out, want)
