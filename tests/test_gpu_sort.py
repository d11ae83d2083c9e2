"""Rows into expert order and back (ep_sort_layout, ep_sort_rows, ep_unsort_rows,
ep_unsort_rows_backward) against plain forms in 64 bits: the placement and the moved bytes
exactly, the sums within the fp32 summation bound and one bf16 rounding."""
import pytest
import torch

import combine_layout_02_gb300 as ep
from combine_layout_02_gb300.buffers import SortBuffers
from rows_util import U16, U32, assert_within, integers, placement, sum_bound

pytestmark = pytest.mark.gpu

# N, E, k, share of entries that are local, how they fall
CASES = [
    (1, 1, 1, 1.0), (1, 8, 8, 0.0), (2, 3, 2, 0.5), (31, 8, 2, 0.7), (33, 32, 8, 0.3), (128, 32, 8, 0.125),
    (1000, 256, 8, 0.5), (1024, 128, 8, 1.0), (1025, 7, 8, 1.0), (1500, 33, 32, 0.9), (5000, 1, 3, 0.9),
    (4099, 300, 6, 0.6), (40000, 128, 6, 1.0), (900, 8192, 4, 1.0), (5000, 8192, 4, 0.8), (700, 2049, 8, 1.0),
]


def routing(N, E, k, share, seed, distinct=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if distinct:
        idx = torch.rand(N, E, generator=g, device="cuda").argsort(1)[:, :k]
    else:
        # skewed, with repeats inside a row
        idx = (torch.rand(N, k, generator=g, device="cuda").pow(1.7) * E).long().clamp(max=E - 1)
    keep = torch.rand(N, k, generator=g, device="cuda") < share
    return torch.where(keep, idx, torch.full_like(idx, -1)).contiguous(), g


class Sorted:
    def __init__(self, idx, E, H=128, rows=None):
        N, k = idx.shape
        self.idx, self.err = idx, torch.zeros(1, dtype=torch.int32, device="cuda")
        self.sh = ep.make_shape(1, N, H, E, k)
        self.sb = SortBuffers(self.sh, rows)
        for t in self.sb.tensors():
            t.fill_(77)
        self.launch = ep.make_launch(error_flags=self.err)
        ep.ep_sort_layout(self.sh, idx, self.sb.handle(), self.sb.workspace, self.launch)

    def flags(self):
        torch.cuda.synchronize()
        return int(self.err.item())


@pytest.mark.parametrize("N,E,k,share", CASES)
def test_placement(N, E, k, share):
    idx, _ = routing(N, E, k, share, N + E)
    s = Sorted(idx, E)
    rows_of, entries, prefix = placement(idx.cpu(), E)
    assert s.sb.entry_rows.reshape(-1).tolist() == rows_of
    assert s.sb.expert_prefix.tolist() == prefix
    assert s.sb.row_entries.tolist()[:len(entries)] == entries
    assert bool((s.sb.row_entries[len(entries):] == 77).all())
    assert s.flags() == 0


def test_placement_of_no_rows():
    sh = ep.make_shape(1, 0, 128, 5, 2)
    sb = SortBuffers(sh)
    sb.expert_prefix.fill_(9)
    ep.ep_sort_layout(sh, torch.empty(0, 2, dtype=torch.int64, device="cuda"), sb.handle(), sb.workspace)
    out = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    ep.ep_sort_rows(sh, out, ep.EP_BF16, None, sb.handle(), out, None)
    ep.ep_unsort_rows(sh, out, None, sb.handle(), out)
    ep.ep_unsort_rows_backward(sh, out, out, None, sb.handle(), out, torch.empty(0, 2, device="cuda"))
    assert sb.expert_prefix.tolist() == [0] * 6


@pytest.mark.parametrize("N", [40, 3000])
def test_ids_out_of_range_are_flagged_and_masked(N):
    idx, _ = routing(N, 9, 4, 0.8, 5)
    idx[3, 1], idx[N - 1, 3], idx[7, 0] = 9, -2, 1 << 40
    s = Sorted(idx, 9)
    rows_of, _, prefix = placement(idx.cpu(), 9)
    assert s.sb.entry_rows.reshape(-1).tolist() == rows_of
    assert s.sb.expert_prefix.tolist() == prefix
    assert s.flags() == ep.EP_DEVERR_BAD_EXPERT


@pytest.mark.parametrize("N", [50, 3000])
def test_rows_beyond_the_buffers_are_skipped_and_flagged(N):
    idx, g = routing(N, 6, 4, 0.9, 6)
    rows_of, _, prefix = placement(idx.cpu(), 6)
    room = prefix[-1] - 17
    s = Sorted(idx, 6, rows=room)
    assert s.flags() == ep.EP_DEVERR_RECV_OVERFLOW
    assert s.sb.entry_rows.reshape(-1).tolist() == [r if r < room else -1 for r in rows_of]
    assert s.sb.expert_prefix.tolist() == prefix
    # a placement made for more rows than the buffers now hold: skipped and flagged, not written
    full = Sorted(idx, 6)
    x = integers(g, N, 128)
    out = torch.full((prefix[-1], 128), 5.0, dtype=torch.bfloat16, device="cuda")
    h = full.sb.handle()
    h.num_rows = room
    ep.ep_sort_rows(full.sh, x, ep.EP_BF16, None, h, out, None, full.launch)
    assert full.flags() == ep.EP_DEVERR_RECV_OVERFLOW
    assert bool((out[room:] == 5.0).all())


# Where one block's sort ends, and around the 32 and 256 entries that a warp takes at a time.
@pytest.mark.parametrize("N,E,k", [(640, 17, 8), (5121, 64, 1), (8191, 5, 1), (8193, 65, 1), (255, 3, 1), (257, 8, 1), (2050, 8192, 2)])
def test_placement_around_the_steps(N, E, k):
    test_placement(N, E, k, 0.9)


# Just below and at 48 KB of dynamic shared memory, which static shared memory adds to.
@pytest.mark.parametrize("N,E,k", [(300, 372, 4), (300, 384, 4), (3000, 1365, 4), (3000, 1536, 4)])
def test_placement_with_tables_of_48_kilobytes(N, E, k):
    test_placement(N, E, k, 0.9)


@pytest.mark.parametrize("H", [5888, 6016, 6144])
def test_rows_of_which_a_block_holds_48_kilobytes(H):
    test_bf16_rows_move_bit_for_bit(526, H, 16, 2, 1.0)
    test_e4m3_rows_move_with_their_scales(526, 2 * H, 16, 2, 1.0, False)


@pytest.mark.parametrize("N,H,E,k,share", [(1, 128, 4, 2, 1.0), (33, 7168, 32, 8, 0.125), (517, 384, 16, 3, 0.5),
                                           (64, 25728, 8, 2, 0.6), (3000, 256, 128, 6, 1.0)])
def test_bf16_rows_move_bit_for_bit(N, H, E, k, share):
    idx, g = routing(N, E, k, share, 7)
    s = Sorted(idx, E, H)
    _, entries, _ = placement(idx.cpu(), E)
    bits = torch.randint(-32768, 32768, (N, H), generator=g, device="cuda").to(torch.int16)    # NaN and infinities too
    out = torch.full((N * k, H), 1234, dtype=torch.int16, device="cuda")
    ep.ep_sort_rows(s.sh, bits, ep.EP_BF16, None, s.sb.handle(), out, None, s.launch)
    assert s.flags() == 0
    at = torch.tensor(entries, dtype=torch.long, device="cuda") // k
    assert torch.equal(out[:len(entries)], bits[at])
    assert bool((out[len(entries):] == 1234).all())


@pytest.mark.parametrize("N,H,E,k,share", [(1, 128, 4, 2, 1.0), (65, 7168, 32, 8, 0.25), (300, 640, 16, 3, 0.5), (9, 52224, 4, 2, 1.0)])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_e4m3_rows_move_with_their_scales(N, H, E, k, share, ue8m0):
    idx, g = routing(N, E, k, share, 8)
    s = Sorted(idx, E, H)
    _, entries, _ = placement(idx.cpu(), E)
    q = torch.randint(0, 256, (N, H), generator=g, device="cuda", dtype=torch.uint8)
    if ue8m0:
        sc = torch.randint(0, 256, (N, H // 128), generator=g, device="cuda", dtype=torch.uint8)
    else:
        sc = torch.rand(N, H // 128, generator=g, device="cuda")
    out, out_sc = torch.empty(N * k, H, dtype=torch.uint8, device="cuda"), torch.empty(N * k, H // 128, dtype=sc.dtype, device="cuda")
    fmt = ep.EP_FP8_SCALE_UE8M0 if ue8m0 else ep.EP_FP8_SCALE_FP32
    ep.ep_sort_rows(s.sh, q, ep.EP_FP8_E4M3, sc, s.sb.handle(), out, out_sc, s.launch, scale_format=fmt)
    at = torch.tensor(entries, dtype=torch.long, device="cuda") // k
    assert torch.equal(out[:len(entries)], q[at]) and torch.equal(out_sc[:len(entries)], sc[at])
    assert s.flags() == 0


def plain_unsort(y, entry_rows, w):
    """(sum, sum of magnitudes) in 64 bits."""
    at = entry_rows.long()
    got = torch.where((at >= 0)[..., None], y.double()[at.clamp(min=0)], torch.zeros((), dtype=torch.float64, device=y.device))
    c = torch.ones_like(at, dtype=torch.float64) if w is None else w.double()
    got = torch.where((at >= 0)[..., None], got * c[..., None], torch.zeros_like(got))
    return got.sum(1), got.abs().sum(1)


FORMS = [(1, 128, 1, 1, 1.0), (70, 256, 8, 4, 0.5), (70, 1024, 8, 5, 0.5), (65, 2048, 16, 2, 0.8), (129, 7168, 32, 8, 0.2),
         (40, 1152, 64, 32, 0.9), (50, 4096, 16, 6, 1.0)]


@pytest.mark.parametrize("N,H,E,k,share", FORMS)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("shift", [0, 8])           # y on a 16-byte boundary that is not a 32-byte one
def test_back_to_rows(N, H, E, k, share, weighted, shift):
    idx, g = routing(N, E, k, share, 9)
    if N > 10:
        idx[4] = -1                                  # a row that no expert takes
    s = Sorted(idx, E, H)
    total = int((idx >= 0).sum())
    store = torch.full((N * k * H + shift,), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = store[shift:].view(N * k, H)
    y[:total] = torch.randn(total, H, generator=g, device="cuda")     # the rows that follow stay NaN
    w = torch.randn(N, k, generator=g, device="cuda")
    w[idx < 0] = float("nan")                        # masked entries' weights are not used
    out = torch.full((N, H), 3.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_unsort_rows(s.sh, y, w if weighted else None, s.sb.handle(), out, s.launch)
    assert s.flags() == 0
    exact, mags = plain_unsort(y, s.sb.entry_rows, torch.nan_to_num(w) if weighted else None)
    assert_within(out, exact, sum_bound(k + 1, mags), U16)
    again = torch.empty_like(out)
    ep.ep_unsort_rows(s.sh, y, w if weighted else None, s.sb.handle(), again, s.launch)
    assert torch.equal(out, again)


@pytest.mark.parametrize("N,H,E,k,share", FORMS + [(1, 7168, 8, 8, 1.0), (3, 25728, 8, 3, 1.0)])
def test_gradient_of_the_way_back(N, H, E, k, share):
    idx, g = routing(N, E, k, share, 10)
    if N > 10:
        idx[4] = -1
    s = Sorted(idx, E, H)
    total = int((idx >= 0).sum())
    y = torch.full((N * k, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    y[:total] = torch.randn(total, H, generator=g, device="cuda")
    dout = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, k, generator=g, device="cuda")
    dy = torch.full((N * k, H), 3.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((N, k), 3.0, device="cuda")
    ep.ep_unsort_rows_backward(s.sh, dout, y, w, s.sb.handle(), dy, dw, s.launch)
    assert s.flags() == 0
    at = s.sb.entry_rows.long()
    there = at >= 0
    e_dy = torch.full((N * k, H), 3.0, dtype=torch.float64, device="cuda")
    full = w.double()[..., None] * dout.double()[:, None, :]
    e_dy[at[there]] = full[there]
    assert_within(dy, e_dy, U32 * e_dy.abs(), U16)
    prod = torch.where(there[..., None], y.double()[at.clamp(min=0)] * dout.double()[:, None, :], torch.zeros((), dtype=torch.float64, device="cuda"))
    assert_within(dw, prod.sum(-1), sum_bound(H, prod.abs().sum(-1)))
    # one output at a time, without weights, and in place
    dw2 = torch.empty_like(dw)
    ep.ep_unsort_rows_backward(s.sh, dout, y, w, s.sb.handle(), None, dw2, s.launch)
    assert torch.equal(dw, dw2)
    dy2 = torch.full_like(dy, 3.0)
    ep.ep_unsort_rows_backward(s.sh, dout, None, w, s.sb.handle(), dy2, None, s.launch)
    assert torch.equal(dy, dy2)
    ones = torch.full_like(dy, 3.0)
    ep.ep_unsort_rows_backward(s.sh, dout, None, None, s.sb.handle(), ones, None, s.launch)
    assert torch.equal(ones[at[there]], dout[:, None, :].expand(N, k, H)[there])
    dw3, y3 = torch.empty_like(dw), y.clone()
    ep.ep_unsort_rows_backward(s.sh, dout, y3, w, s.sb.handle(), y3, dw3, s.launch)
    assert torch.equal(dw, dw3) and torch.equal(y3[at[there]], dy[at[there]])


def test_gradients_against_differences():
    """Whole numbers, so that every sum is exact: a step in y, in the weights and in the rows
    changes the outputs by what the gradients say."""
    N, H, E, k = 37, 384, 8, 3
    idx, g = routing(N, E, k, 0.8, 11)
    s = Sorted(idx, E, H)
    total, h = int((idx >= 0).sum()), s.sb.handle()
    y, step = integers(g, N * k, H), integers(g, N * k, H, most=1)
    w, wstep = integers(g, N, k).float(), integers(g, N, k, most=1).float()
    dout = integers(g, N, H, most=2)

    def back(y_, w_):
        out = torch.empty(N, H, dtype=torch.bfloat16, device="cuda")
        ep.ep_unsort_rows(s.sh, y_, w_, h, out)
        return out.double()

    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    ep.ep_unsort_rows_backward(s.sh, dout, y, w, h, dy, dw)
    d = dout.double()
    assert ((back(y + step, w) - back(y, w)) * d).sum() == (dy[:total].double() * step[:total].double()).sum()
    assert ((back(y, w + wstep) - back(y, w)) * d).sum() == (dw.double() * wstep.double()).sum()
    # the rows' gradient: sort_rows is linear, its gradient the unweighted way back
    x, xstep, dxs = integers(g, N, H), integers(g, N, H, most=1), integers(g, N * k, H, most=2)

    def there(x_):
        out = torch.zeros(N * k, H, dtype=torch.bfloat16, device="cuda")
        ep.ep_sort_rows(s.sh, x_, ep.EP_BF16, None, h, out, None)
        return out.double()

    dx = torch.empty(N, H, dtype=torch.bfloat16, device="cuda")
    ep.ep_unsort_rows(s.sh, dxs, None, h, dx)
    assert ((there(x + xstep) - there(x)) * dxs.double()).sum() == (dx.double() * xstep.double()).sum()


def test_on_a_stream_with_events():
    N, H, E, k = 600, 512, 16, 4
    idx, g = routing(N, E, k, 0.7, 12)
    x = integers(g, N, H)
    s = Sorted(idx, E, H)
    want = torch.zeros(N * k, H, dtype=torch.bfloat16, device="cuda")
    ep.ep_sort_rows(s.sh, x, ep.EP_BF16, None, s.sb.handle(), want, None)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), torch.zeros_like(want)
    ready, done = torch.cuda.Event(), torch.cuda.Event()
    late = torch.zeros_like(x)
    sb = SortBuffers(s.sh)
    torch.cuda._sleep(2_000_000)
    late.copy_(x)                                    # still to come when the calls below are made
    ready.record()
    done.record()
    ep.ep_sort_layout(s.sh, idx, sb.handle(), sb.workspace, ep.make_launch(side, wait_event=ready))
    ep.ep_sort_rows(s.sh, late, ep.EP_BF16, None, sb.handle(), got, None, ep.make_launch(side, record_event=done))
    torch.cuda.current_stream().wait_event(done)
    assert torch.equal(got, want)
