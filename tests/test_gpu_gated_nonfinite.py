"""The gated feed-forward block with infinities and NaN in single rows: what is kept of them, and that the other
rows come out as they would without them, bit for bit."""
import math

import pytest
import torch

import combine_layout_02_gb300 as ep
from kept_util import GROUP, quantised

pytestmark = pytest.mark.gpu

ACTS = {"silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU_TANH}

# rows per expert, in_features, out_features of h: pairs, narrow tiles, a contraction split over a cluster;
# features that are odd multiples of 8 and multiples of 16
CASES = {
    "pairs": ([7000, 0, 5130], 1160, 264),
    "pairs_short": ([3000, 1111], 136, 1032),
    "narrow": ([40, 0, 200, 30], 64, 136),
    "cluster": ([3, 7, 2], 4096, 264),
    "cluster_whole_groups": ([9, 5], 4096, 128),
}
BEFORE, AFTER = 2, 3          # rows of no expert around them


class Rows:
    def __init__(self, counts, K, F, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.E, self.K, self.F, self.n = len(counts), K, F, BEFORE + sum(counts) + AFTER
        self.prefix = (torch.tensor([0] + counts).cumsum(0) + BEFORE).int().cuda()
        self.x, self.dy = new(self.n, K), new(self.n, K)
        self.gate_up, self.down = (new(self.E, 2 * F, K) * 1.5 * K ** -0.5).bfloat16(), (new(self.E, K, F) * F ** -0.5).bfloat16()
        for w in (self.gate_up, self.down):          # (0 times an infinity is a NaN all the same, but says less)
            w[w == 0] = 2.0 ** -7
        # a NaN, an infinity, both, a row of NaN: the first expert's second and third row, the last's two last
        self.bad = [BEFORE + 1, BEFORE + 2, self.n - AFTER - 2, self.n - AFTER - 1]
        self.good = torch.ones(self.n, dtype=torch.bool, device="cuda")
        self.good[self.bad] = False
        self.mine = slice(BEFORE, self.n - AFTER)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.launch = ep.make_launch(error_flags=self.err)

    def spoil(self, t):
        """t with its bad rows."""
        t = t.clone()
        t[self.bad[0], t.shape[1] // 3] = math.nan
        t[self.bad[1], 5] = math.inf
        t[self.bad[2], 0], t[self.bad[2], -1] = -math.inf, math.nan
        t[self.bad[3]] = math.nan
        return t

    def buffers(self, keep):
        width = -(-self.F // GROUP) * GROUP
        if keep == "bf16":
            return torch.full((self.n, 2 * self.F), 7.0, dtype=torch.bfloat16, device="cuda"), None
        return (torch.full((self.n, 2 * width), 0xA5, dtype=torch.uint8, device="cuda"),
                torch.full((self.n, width // GROUP, 2), 0xA5, dtype=torch.uint8, device="cuda"))

    def forward(self, x, kind, keep):
        h = torch.full((self.n, self.F), 7.0, dtype=torch.bfloat16, device="cuda")
        values, scales = self.buffers(keep)
        ep.ep_expert_gated(ep.ep_gemm_shape(self.n, self.E, self.K, self.F), x, self.gate_up, self.prefix, ACTS[kind], h,
                           ep.make_checkpoint(values, scales), self.launch)
        return h, values, scales

    def backward(self, dy, values, scales, kind):
        dgu = torch.full((self.n, 2 * self.F), 7.0, dtype=torch.bfloat16, device="cuda")
        h = torch.full((self.n, self.F), 7.0, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_gated_dgrad(ep.ep_gemm_shape(self.n, self.E, self.F, self.K), dy, self.down, self.prefix, ACTS[kind],
                                 ep.make_checkpoint(values, scales), dgu, h, self.launch)
        return dgu, h

    def outside(self, *outputs):
        for t in outputs:
            if t is not None:
                rest = torch.cat([t[:self.mine.start], t[self.mine.stop:]])
                assert bool((rest == (0xA5 if t.dtype == torch.uint8 else 7)).all())
        assert int(self.err.item()) == 0


@pytest.mark.parametrize("name", CASES)
def test_padding_is_zeros(name):
    """Features beyond the last are zeros in a checkpoint whatever the row holds."""
    b = Rows(*CASES[name])
    _, values, _ = b.forward(b.spoil(b.x), "silu", "e4m3")
    for part in values.chunk(2, 1):
        assert not bool(part[b.mine, b.F:].any())


@pytest.mark.parametrize("name", CASES)
def test_kept_bytes(name):
    """What is kept in 8 bits is the checkpoint of the bf16 values, byte for byte: NaN is left out of its
    group's scale, also where the group has nothing else."""
    b = Rows(*CASES[name])
    x = b.spoil(b.x)
    _, values, scales = b.forward(x, "silu", "e4m3")
    _, halves, _ = b.forward(x, "silu", "bf16")
    nan = torch.isnan(halves[b.bad])
    assert bool(nan[3].all()) and bool(torch.isinf(halves[b.bad[1]]).any())
    for side in range(2):
        q, k, _ = quantised(halves[b.mine].chunk(2, 1)[side])
        assert torch.equal(scales[b.mine, :, side].cpu(), k)
        assert torch.equal(values[b.mine].chunk(2, 1)[side][:, :b.F].cpu(), q[:, :b.F])


def same(a, b):
    """Bit for bit (NaN included)."""
    as_bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t  # noqa: E731
    return torch.equal(as_bits(a), as_bits(b))


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("name", CASES)
def test_bad_rows_stay_alone_forward(name, kind, keep):
    """A row with a NaN or an infinity has no finite value of h (every weight is other than 0), and what is
    kept of it is NaN or an infinity; all other rows are as they are without it."""
    b = Rows(*CASES[name])
    got, want = b.forward(b.spoil(b.x), kind, keep), b.forward(b.x, kind, keep)
    for a, w in zip(got, want):
        assert a is None or same(a[b.good], w[b.good])
    assert not bool(torch.isfinite(got[0][b.bad]).any()) and bool(torch.isfinite(want[0][b.mine]).all())
    if keep == "bf16":
        assert not bool(torch.isfinite(got[1][b.bad]).any())
    b.outside(*got)


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("name", CASES)
def test_bad_rows_stay_alone_backward(name, kind, keep):
    """Of dy: the row's dg and du have no finite value but where their factor is 0, h is as without. Of g
    and u as they were kept: their own features of dg, du and h alone (bf16; in 8 bits an infinity
    sets the scale of its group)."""
    b = Rows(*CASES[name])
    _, values, scales = b.forward(b.x, kind, keep)
    want = b.backward(b.dy, values, scales, kind)
    assert all(bool(torch.isfinite(t[b.mine]).all()) for t in want)
    dgu, h = b.backward(b.spoil(b.dy), values, scales, kind)
    assert same(dgu[b.good], want[0][b.good]) and same(h, want[1])
    # dh is NaN or an infinity, and so is its product with any factor: 0 times an infinity is NaN
    assert not bool(torch.isfinite(dgu[b.bad]).any())
    b.outside(dgu, h)
    # one feature of g in a row, one of u in another
    for side, row in enumerate(b.bad[:2]):
        for bad in (math.nan, math.inf, -math.inf):
            f = b.F - 3
            v, s = values.clone(), scales if scales is None else scales.clone()
            if keep == "bf16":
                v[row, side * b.F + f] = bad
                group = [f]
            else:
                wide = v.shape[1] // 2
                if math.isnan(bad):
                    v[row, side * wide + f] = 0x7F
                    group = [f]
                else:          # 448 * 2^120
                    v[row, side * wide + f] = 0x7E if bad > 0 else 0xFE
                    s[row, f // GROUP, side] = 247
                    group = list(range(f // GROUP * GROUP, min(b.F, (f // GROUP + 1) * GROUP)))
            dgu, h = b.backward(b.dy, v, s, kind)
            hit = torch.zeros(b.F, dtype=torch.bool, device="cuda")
            hit[group] = True
            rest = torch.ones(b.n, dtype=torch.bool, device="cuda")
            rest[row] = False
            assert same(dgu[rest], want[0][rest]) and same(h[rest], want[1][rest])
            assert same(dgu[row].view(2, -1)[:, ~hit], want[0][row].view(2, -1)[:, ~hit]) and same(h[row, ~hit], want[1][row, ~hit])
            if math.isnan(bad):          # act(g) u, dh u act'(g) and, of g, dh act(g) (of u: du does not have it)
                assert bool(torch.isnan(h[row, f])) and bool(torch.isnan(dgu[row, f]))
                assert bool(torch.isnan(dgu[row, b.F + f])) == (side == 0)
            elif side == 1:          # u: h and dg are infinite (or NaN where act is 0), du has none of it
                assert not bool(torch.isfinite(h[row, f]))
                assert keep == "e4m3" or same(dgu[row, b.F + f], want[0][row, b.F + f])
            b.outside(dgu, h)
