"""The gated feed-forward block's kernels against plain forms in 64 bits: forward with and without a
checkpoint, the way back from both kinds of checkpoint. Bounds: the fp32 sums' (rows_util), those of exp
and division (kept_util), carried through the formulas, and one rounding to bf16."""
import math

import pytest
import torch

import combine_layout_02_gb300 as ep
from kept_util import GROUP, act, quantised, stands_for
from rows_util import U16, U32, assert_within, integers, sum_bound

pytestmark = pytest.mark.gpu

ACTS = {"silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU_TANH}
STEEP = 1.13          # the largest slope of silu (1.0998) and gelu (1.1290)

# rows per expert, in_features, out_features (of h)
CASES = {
    "least": ([1], 8, 8),
    "one_row": ([1], 256, 128),
    "empty_between": ([0, 5, 0, 0, 3, 0], 64, 136),
    "odd": ([17, 1, 33, 130], 72, 200),
    "tile_edges": ([128, 127, 129, 256, 255, 257], 128, 256),
    "half_groups": ([300, 24, 700], 192, 264),
    "deep_few": ([70, 9], 2056, 128),
    "wide": ([60, 300], 128, 1032),
    "many_experts": ([(7 * e) % 5 for e in range(300)], 64, 72),
    "one_each": ([1] * 32, 520, 392),
    "few_rows_split": ([3, 0, 2, 5, 1, 0, 4, 1], 4096, 256),
    "many_rows_few_features": ([3000, 0, 1111, 1], 136, 104),
    "one_long_expert": ([4099], 264, 392),
    "one_deep": ([200], 4160, 264),
    "wide_and_narrow": ([97, 0, 160, 31], 1096, 520),
    "decode": ([16, 30, 8, 15, 2, 40, 0, 9], 1024, 1024),
}


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def by_row(scales):
    """[rows][groups][2] -> each side's [rows][groups]."""
    return [scales[:, :, side].contiguous() for side in range(2)]


class Block:
    """Rows of the experts with some of no expert around them: NaN where inputs, 7 where outputs."""

    def __init__(self, counts, K, F, seed, make=normal, scale=None, before=3, after=5, H=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.K, self.F, self.H = len(counts), K, F, H or K
        prefix = torch.zeros(self.E + 1, dtype=torch.int32)
        prefix[1:] = torch.tensor(counts).cumsum(0)
        self.prefix = (prefix + before).int().cuda()
        self.edge = self.prefix.tolist()
        self.n = before + sum(counts) + after
        self.mine = slice(before, before + sum(counts))
        rows = lambda n: torch.full((self.n, n), math.nan, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.dy = rows(K), rows(self.H)
        self.x[self.mine], self.dy[self.mine] = make(g, sum(counts), K), make(g, sum(counts), self.H)
        one = make is normal
        self.gate_up = (make(g, self.E, 2 * F, K) * (1.5 * K ** -0.5 if one else 1)).bfloat16()
        self.down = (make(g, self.E, self.H, F) * (F ** -0.5 if one else 1)).bfloat16()
        self.shape, self.down_shape = ep.ep_gemm_shape(self.n, self.E, K, F), ep.ep_gemm_shape(self.n, self.E, F, self.H)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.launch = ep.make_launch(error_flags=self.err)

    def buffers(self, keep):
        """(values, scales, checkpoint)"""
        if keep is None:
            return None, None, None
        if keep == "bf16":
            values, scales = torch.full((self.n, 2 * self.F), 7.0, dtype=torch.bfloat16, device="cuda"), None
        else:
            width = -(-self.F // GROUP) * GROUP
            values = torch.full((self.n, 2 * width), 0xA5, dtype=torch.uint8, device="cuda")
            scales = torch.full((self.n, width // GROUP, 2), 0xA5, dtype=torch.uint8, device="cuda")
        return values, scales, ep.make_checkpoint(values, scales)

    def parts(self, values, scales):
        """g and u as kept, in 64 bits."""
        if scales is None:
            return values.double().chunk(2, 1)
        return [stands_for(v.contiguous(), s.contiguous(), self.F) for v, s in zip(values.chunk(2, 1), by_row(scales))]

    def forward(self, kind, keep=None, with_h=True):
        h = torch.full((self.n, self.F), 7.0, dtype=torch.bfloat16, device="cuda") if with_h else None
        values, scales, checkpoint = self.buffers(keep)
        ep.ep_expert_gated(self.shape, self.x, self.gate_up, self.prefix, ACTS[kind], h, checkpoint, self.launch)
        return h, values, scales

    def sums(self):
        """g, u and the bounds of their fp32 sums, rows of no expert 0."""
        new = lambda: torch.zeros(self.n, 2 * self.F, dtype=torch.float64, device="cuda")  # noqa: E731
        s, m = new(), new()
        for e in range(self.E):
            at = slice(self.edge[e], self.edge[e + 1])
            x, w = self.x[at].double(), self.gate_up[e].double()
            s[at], m[at] = x @ w.t(), x.abs() @ w.abs().t()
        return s.chunk(2, 1), [sum_bound(self.K, t, 2 * U32) for t in m.chunk(2, 1)]

    def outside(self, *outputs):
        """Rows of no expert are as they were."""
        for t in outputs:
            if t is not None:
                rest = torch.cat([t[:self.mine.start], t[self.mine.stop:]])
                assert bool((rest == (0xA5 if t.dtype == torch.uint8 else 7)).all())


def product_bound(a, a_off, b, b_off):
    return a.abs() * b_off + b.abs() * a_off + a_off * b_off


@pytest.mark.parametrize("kind,keep", [("silu", None), ("gelu", "e4m3"), ("silu", "bf16")])
@pytest.mark.parametrize("name", CASES)
def test_forward(name, kind, keep):
    b = Block(*CASES[name], seed=1)
    h, values, scales = b.forward(kind, keep)
    (g, u), (g_off, u_off) = b.sums()
    a, _, a_off, _ = act(g, kind)
    at = b.mine
    assert_within(h[at], (a * u)[at], (product_bound(a, a_off + STEEP * g_off, u, u_off) + (a * u).abs() * U32)[at], U16)
    if keep is not None:
        for got, want, off in zip(b.parts(values, scales), (g, u), (g_off, u_off)):
            slack = off + U16 * (want.abs() + off)
            if keep == "e4m3":          # half a step: 2^-4 relatively, or 2^-10 of a power of two <= amax / 224
                wide = torch.nn.functional.pad((want.abs() + slack)[at], (0, -b.F % GROUP)).unflatten(1, (-1, GROUP)).amax(2)
                even = (wide / 224 * 2.0 ** -10).clamp(min=2.0 ** -136).repeat_interleave(GROUP, 1)[:, :b.F]
                slack[at] += torch.maximum((want.abs() + slack)[at] / 16, even)
            assert_within(got[at], want[at], slack[at])
    b.outside(h, values, scales)
    assert int(b.err.item()) == 0


@pytest.mark.parametrize("name", CASES)
def test_kept_bytes_of_whole_numbers(name):
    """Sums that fp32 holds exactly: the checkpoint is that of their bf16 roundings, byte for byte, the
    padding of half groups included; and it does not depend on whether h is asked for."""
    b = Block(*CASES[name], seed=2, make=integers)
    h, values, scales = b.forward("silu", "e4m3", with_h=False)
    sums, _ = b.sums()
    for side, (v, s) in enumerate(zip(values.chunk(2, 1), by_row(scales))):
        q, k, _ = quantised(sums[side][b.mine].float().bfloat16())
        assert torch.equal(v[b.mine].cpu(), q) and torch.equal(s[b.mine].cpu(), k)
    _, halves, _ = b.forward("silu", "bf16")
    assert torch.equal(halves[b.mine], torch.cat([t[b.mine] for t in sums], 1).float().bfloat16())
    again = b.forward("gelu", "e4m3")
    assert torch.equal(again[1], values) and torch.equal(again[2], scales)
    b.outside(values, scales, halves)


@pytest.mark.parametrize("E,expert,K,F", [(1, 0, 8, 8), (1, 0, 256, 128), (5, 3, 520, 1000), (300, 299, 64, 72), (2, 0, 4096, 264),
                                          (3, 2, 4104, 136), (1, 0, 7168, 136), (1, 0, 16384, 64), (2, 1, 9000, 72), (4000, 2222, 264, 40)])
@pytest.mark.parametrize("kind", ACTS)
def test_one_row(kind, E, expert, K, F):
    """A single token, which goes another way: sums of even and of odd values, of lanes and of warps."""
    counts = [0] * E
    counts[expert] = 1
    b = Block(counts, K, F, seed=12, before=0, after=0)
    h, _, _ = b.forward(kind)
    (g, u), (g_off, u_off) = b.sums()
    a, _, a_off, _ = act(g, kind)
    assert_within(h, a * u, product_bound(a, a_off + STEEP * g_off, u, u_off) + (a * u).abs() * U32, U16)
    assert int(b.err.item()) == 0
    assert torch.equal(b.forward(kind)[0], h)
    b.prefix[:] = 0                                  # a row of no expert
    assert bool((b.forward(kind)[0] == 7).all()) and int(b.err.item()) == 0
    b.prefix[1:] = 3                                 # beyond the rows: clipped, flagged
    b.forward(kind)
    assert int(b.err.item()) == ep.EP_DEVERR_RECV_OVERFLOW


def backward(b, kind, keep, with_h=True, seed=9):
    g = torch.Generator(device="cuda").manual_seed(seed)
    values, scales, checkpoint = b.buffers(keep)
    made = (torch.randn(b.n, 2 * b.F, generator=g, device="cuda") * 1.5).bfloat16()
    if keep == "bf16":
        values.copy_(made)
    else:
        for side, part in enumerate(made.chunk(2, 1)):
            q, k, _ = quantised(part)
            wide = q.shape[1]
            values[:, side * wide:(side + 1) * wide], scales[:, :, side] = q.cuda(), k.cuda()
    for t in (values, scales):          # rows of no expert: not read
        if t is not None:
            t[:b.mine.start], t[b.mine.stop:] = (math.nan, math.nan) if t.dtype == torch.bfloat16 else (0x7F, 0x7F)
    dgu = torch.full((b.n, 2 * b.F), 7.0, dtype=torch.bfloat16, device="cuda")
    h = torch.full((b.n, b.F), 7.0, dtype=torch.bfloat16, device="cuda") if with_h else None
    ep.ep_expert_gated_dgrad(b.down_shape, b.dy, b.down, b.prefix, ACTS[kind], checkpoint, dgu, h, b.launch)
    return dgu, h, b.parts(values, scales)


@pytest.mark.parametrize("kind,keep", [("silu", "e4m3"), ("gelu", "bf16"), ("gelu", "e4m3")])
@pytest.mark.parametrize("name", CASES)
def test_backward(name, kind, keep):
    counts, K, F = CASES[name]
    b = Block(counts, K, F, seed=3)
    dgu, h, (g, u) = backward(b, kind, keep)
    dh, off = (torch.zeros(b.n, F, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(b.E):
        at = slice(b.edge[e], b.edge[e + 1])
        dh[at] = b.dy[at].double() @ b.down[e].double()
        off[at] = sum_bound(b.H, b.dy[at].double().abs() @ b.down[e].double().abs(), 2 * U32)
    at = b.mine
    g, u, dh, off = g[at], u[at], dh[at], off[at]
    a, da, a_off, da_off = act(g, kind)
    one = 4 * U32          # two or three more products
    dg = dh * u * da
    assert_within(dgu[at, :F], dg, u.abs() * product_bound(dh, off, da, da_off) + dg.abs() * one, U16)
    assert_within(dgu[at, F:], dh * a, product_bound(dh, off, a, a_off) + (dh * a).abs() * one, U16)
    assert_within(h[at], a * u, u.abs() * a_off + (a * u).abs() * one, U16)
    b.outside(dgu, h)
    assert int(b.err.item()) == 0
    assert torch.equal(backward(b, kind, keep, with_h=False)[0], dgu)


def test_the_way_back_is_the_forward_passes_derivative():
    """Central differences of sum(dy * (Wd h)) along random directions of g and u, in 64 bits at the kept values."""
    b = Block([40, 7, 90], 128, 200, seed=4)
    for kind in ACTS:
        dgu, _, (g, u) = backward(b, kind, "bf16")
        at = b.mine
        g, u = g[at], u[at]
        dh = torch.cat([b.dy[b.edge[e]:b.edge[e + 1]].double() @ b.down[e].double() for e in range(b.E)])
        gen = torch.Generator(device="cuda").manual_seed(5)
        vg, vu = (torch.randn(g.shape, generator=gen, device="cuda", dtype=torch.float64) for _ in range(2))
        step = 1e-4          # error of the difference ~ step^2, of the division ~ 1e-16 / step
        loss = lambda t: (dh * act(g + t * vg, kind)[0] * (u + t * vu)).sum(1)  # noqa: E731
        want = (loss(step) - loss(-step)) / (2 * step)
        got = dgu[at].double()
        terms = torch.cat([got[:, :b.F] * vg, got[:, b.F:] * vu], 1)
        # each value is rounded to bf16 (2^-8); the fp32 sums of 128 terms and the difference are far below 1e-4
        slack = terms.abs().sum(1) * (U16 * 1.01) + 1e-4 * (dh.abs() * (u.abs() + g.abs() + 1)).sum(1)
        assert bool(((terms.sum(1) - want).abs() <= slack).all())


@pytest.mark.parametrize("name", ["odd", "few_rows_split", "one_long_expert"])
def test_repeats_bit_for_bit(name):
    b = Block(*CASES[name], seed=6)
    once, again = b.forward("silu", "e4m3"), b.forward("silu", "e4m3")
    assert all(torch.equal(p, q) for p, q in zip(once, again))
    assert torch.equal(backward(b, "silu", "e4m3")[0], backward(b, "silu", "e4m3")[0])


@pytest.mark.parametrize("counts", [[40, 200, 30], [3, 2, 4]])
@pytest.mark.parametrize("kind", ACTS)
def test_large_and_infinite_sums(kind, counts):
    """An infinite or NaN row reaches its own outputs alone; large sums stay finite where the formula is."""
    b = Block(counts, 64, 48, seed=7)
    start = b.mine.start
    b.x[start + 1, 0] = math.inf
    b.x[start + 2, 3] = math.nan
    b.x[start + 4] *= 2.0 ** 40
    h, values, scales = b.forward(kind, "e4m3")
    (g, u), _ = b.sums()
    want = (act(g, kind)[0] * u)[b.mine]
    fine = torch.ones(len(want), dtype=torch.bool, device="cuda")
    fine[1:3] = False
    assert bool(torch.isfinite(h[b.mine][fine]).all())
    assert not bool(torch.isfinite(h[b.mine][~fine]).any(1).all())
    big = want[4].abs() > 2.0 ** 50
    assert bool(big.any()) and bool(((h[b.mine][4].double() - want[4])[big].abs() <= want[4][big].abs() * 2.0 ** -6).all())
    dgu, again, _ = backward(b, kind, "bf16")
    assert bool(torch.isfinite(dgu[b.mine]).all()) and bool(torch.isfinite(again[b.mine]).all())


def test_slopes_far_out():
    """Large |g|: the slope is 0 or 1, and nothing is NaN."""
    for kind in ACTS:
        b = Block([9, 300], 64, 64, seed=8)
        values, _, checkpoint = b.buffers("bf16")
        ends = torch.tensor([-3e38, -1e20, -1e4, -200.0, -90.0, -30.0, 30.0, 90.0, 200.0, 1e4, 1e20, 3e38], device="cuda").bfloat16()
        values[:, :64] = ends.repeat(6)[:64]
        values[:, 64:] = 1.0
        dgu, h = torch.empty_like(values), torch.empty(b.n, 64, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_gated_dgrad(b.down_shape, b.dy, b.down, b.prefix, ACTS[kind], checkpoint, dgu, h, b.launch)
        dh = torch.cat([b.dy[b.edge[e]:b.edge[e + 1]].double() @ b.down[e].double() for e in range(2)])
        up = (values[b.mine, :64].double() > 0).double()
        # e^-30 * 30 is 3e-12; the fp32 sum of 64 terms and one rounding
        off = sum_bound(64, torch.cat([b.dy[b.edge[e]:b.edge[e + 1]].double().abs() @ b.down[e].double().abs() for e in range(2)]), 2 * U32)
        assert_within(dgu[b.mine, :64], dh * up, off + 1e-10 * dh.abs(), U16)
        assert_within(h[b.mine], values[b.mine, :64].double() * up, 1e-10, U16)


def test_prefix_beyond_the_rows_is_flagged():
    b = Block([20, 30], 64, 64, seed=10)
    b.prefix[-1] = b.n + 9
    h, _, _ = b.forward("silu")
    assert int(b.err.item()) & ep.EP_DEVERR_RECV_OVERFLOW


def test_calls_on_two_streams_and_replayed():
    """The same buffers' shapes on two streams at once, and captured: nothing of the calls is shared."""
    blocks = [Block([40, 0, 7, 90, 1], 264, 136, seed=s) for s in (20, 21)]
    one = Block([1], 520, 72, seed=22, before=0, after=0)
    want = [b.forward("silu", "e4m3") for b in blocks] + [one.forward("gelu")]
    streams = [torch.cuda.Stream() for _ in blocks]
    got = []
    for s, b in zip(streams, blocks):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            b.launch = ep.make_launch(error_flags=b.err)
            got.append([b.forward("silu", "e4m3") for _ in range(5)][-1])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for a, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for b in (*blocks, one):
            b.launch = ep.make_launch(error_flags=b.err)
        out = [b.forward("silu", "e4m3") for b in blocks] + [one.forward("gelu")]
    for _ in range(2):
        for t in out:
            t[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(out, want):
            assert all(torch.equal(x, y) for x, y in zip(a, w) if x is not None)


@pytest.mark.parametrize("counts,K,F", [([3], 1 << 20, 8), ([1, 2], 8, 1 << 20), ([1 if e % 80 == 3 else 0 for e in range(8192)], 64, 16),
                                        ([70] * 3, 8, 1 << 16), ([5, 300], 1 << 16, 8)])
def test_largest_sizes(counts, K, F):
    """Features and experts at their limits, both ways, keeping 8 bits (the way back with as many features out)."""
    b = Block(counts, K, F, seed=30)
    h, values, scales = b.forward("silu", "e4m3")
    (g, u), (g_off, u_off) = b.sums()
    a, _, a_off, _ = act(g, "silu")
    at = b.mine
    assert_within(h[at], (a * u)[at], (product_bound(a, a_off + STEEP * g_off, u, u_off) + (a * u).abs() * U32)[at], U16)
    dgu, _, (g, u) = backward(b, "silu", "e4m3", with_h=False)
    dh, off = (torch.zeros(b.n, F, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(b.E):
        rows = slice(b.edge[e], b.edge[e + 1])
        if rows.start < rows.stop:
            dh[rows] = b.dy[rows].double() @ b.down[e].double()
            off[rows] = sum_bound(b.H, b.dy[rows].double().abs() @ b.down[e].double().abs(), 2 * U32)
    a, da, a_off, da_off = act(g, "silu")
    assert_within(dgu[at, :F], (dh * u * da)[at], (u.abs() * product_bound(dh, off, da, da_off) + (dh * u * da).abs() * 4 * U32)[at], U16)
    assert_within(dgu[at, F:], (dh * a)[at], (product_bound(dh, off, a, a_off) + (dh * a).abs() * 4 * U32)[at], U16)
    b.outside(h, values, scales, dgu)
    assert int(b.err.item()) == 0


def test_no_rows():
    sh = ep.ep_gemm_shape(0, 3, 64, 32)
    prefix = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gated(sh, None, None, prefix, ep.EP_ACT_SILU, None, None)
    ep.ep_expert_gated(sh, None, None, prefix, ep.EP_ACT_SILU, None, ep.make_checkpoint(none))
    ep.ep_expert_gated_dgrad(sh, None, None, prefix, ep.EP_ACT_SILU, ep.make_checkpoint(none), None, None)
    torch.cuda.synchronize()


def test_many_rows_beyond_two_to_the_31_values():
    """dgu and the checkpoint pass 2^31 values: the last rows are theirs."""
    n, K, F = 1_100_003, 64, 1000
    b = Block([n], K, F, seed=11, before=0, after=0)
    h, values, scales = b.forward("silu", "e4m3")
    last = slice(n - 200, n)
    w = b.gate_up[0].double()
    g, u = (b.x[last].double() @ w.t()).chunk(2, 1)
    off = sum_bound(K, b.x[last].double().abs() @ w.abs().t(), 2 * U32)
    a, _, a_off, _ = act(g, "silu")
    assert_within(h[last], a * u, product_bound(a, a_off + STEEP * off[:, :F], u, off[:, F:]) + (a * u).abs() * U32, U16)
    dgu = torch.empty(n, 2 * F, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gated_dgrad(b.down_shape, b.dy, b.down, b.prefix, ep.EP_ACT_SILU, ep.make_checkpoint(values, scales), dgu, None, b.launch)
    g, u = (stands_for(v[last].contiguous(), s[last].contiguous(), F) for v, s in zip(values.chunk(2, 1), by_row(scales)))
    dh = b.dy[last].double() @ b.down[0].double()
    off = sum_bound(K, b.dy[last].double().abs() @ b.down[0].double().abs(), 2 * U32)
    a, _, a_off, _ = act(g, "silu")
    assert_within(dgu[last, F:], dh * a, product_bound(dh, off, a, a_off) + (dh * a).abs() * 4 * U32, U16)
    assert int(b.err.item()) == 0
