"""The gated block's waits give up after their time limit: an operand that does not arrive leaves its tile
unwritten in every CTA that shares it, what is kept included, sets EP_DEVERR_TIMEOUT, and the context
stays usable. (Nothing faults or hangs: the self-test withholds loads, and the waits have limits.)"""
import pytest
import torch

import combine_layout_02_gb300 as ep
from kept_util import GROUP
from rows_util import integers

pytestmark = pytest.mark.gpu

# product (0 forward, 1 way back), rows per expert, contracted features, the others, contracted values that arrive
CASES = {
    "pairs": (0, [1300, 1200], 2048, 520, 1024),
    "pairs_nothing": (0, [1300, 1200], 2048, 520, 0),
    "pairs_short": (0, [9000, 9000], 256, 1032, 192),
    "narrow": (0, [300, 200], 512, 264, 128),
    "one_row": (0, [1], 512, 264, 128),
    "cluster_last_part": (0, [3, 5, 2], 4096, 136, 64 * 60),
    "cluster_first_part_alone": (0, [3, 5, 2], 4096, 136, 64 * 8),
    "wide_cluster": (0, [200], 8192, 128, 64 * 100),
    "back_pairs": (1, [1300, 1200], 2048, 1040, 1024),
    "back_narrow": (1, [300, 200], 512, 520, 128),
    "back_cluster": (1, [3, 5, 2], 4096, 264, 64 * 60),
    "back_wide_cluster": (1, [200], 8192, 264, 64 * 100),
}


@pytest.mark.parametrize("keep", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_tiles_without_their_operands_are_not_written(case, keep):
    product, counts, C, F, loads = CASES[case]
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, E = sum(counts), len(counts)
    prefix = torch.tensor([0] + counts).cumsum(0).int().cuda()
    x = integers(g, rows, C)
    w = integers(g, E, 2 * F, C) if product == 0 else integers(g, E, C, F)
    shape = ep.ep_gemm_shape(rows, E, C, F) if product == 0 else ep.ep_gemm_shape(rows, E, F, C)
    width = -(-F // GROUP) * GROUP
    made = torch.randint(1, 100, (rows, 2 * width), generator=g, device="cuda", dtype=torch.uint8)

    def run(call):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((rows, F if product == 0 else 2 * F), 7.5, dtype=torch.bfloat16, device="cuda")
        if keep == "bf16":
            values, scales = made[:, :2 * F].to(torch.bfloat16).contiguous(), None
        else:
            values, scales = made.clone(), torch.full((rows, width // GROUP, 2), 120, dtype=torch.uint8, device="cuda")
        call(out, ep.make_checkpoint(values, scales), ep.make_launch(error_flags=err))
        torch.cuda.synchronize()
        return [out, values] + ([] if scales is None else [scales]), int(err.item())

    def plain(out, checkpoint, launch):
        if product == 0:
            ep.ep_expert_gated(shape, x, w, prefix, ep.EP_ACT_SILU, out, checkpoint, launch)
        else:
            ep.ep_expert_gated_dgrad(shape, x, w, prefix, ep.EP_ACT_SILU, checkpoint, out, None, launch)

    def test(arrive, ms):
        return lambda out, checkpoint, launch: ep.ep_selftest_gated_timeout(shape, product, x, w, prefix, checkpoint, out, arrive, ms, launch)

    want, flags = run(plain)
    assert flags == 0 and not bool((want[0] == 7.5).all())
    untouched, _ = run(lambda *a: None)
    got, flags = run(test(loads, 20))
    assert flags == ep.EP_DEVERR_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(got, untouched))
    # with operands that do arrive it is the call, and the call right after is itself
    for call in (test(1 << 20, 2000), plain):
        got, flags = run(call)
        assert flags == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
