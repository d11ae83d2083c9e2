"""Plain 64-bit forms of the operators on rows grouped by owner, and the error bounds of their
tests. No library code.

u = 2^-8 is the unit roundoff of bf16 and 2^-24 of binary32. A sum of n products in fp32, taken
in any order, is off by at most n 2^-24 / (1 - n 2^-24) times the sum of the magnitudes (Higham,
"Accuracy and Stability of Numerical Algorithms", 2nd ed., section 4.2); where tensor cores may
truncate instead of rounding, each step counts twice (2^-23). The one rounding to bf16 adds at
most 2^-8 of the value that is rounded."""
from __future__ import annotations

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -126


def placement(idx: torch.Tensor, E: int):
    """idx [N][k] -> (entry_rows, row_entries, prefix) as lists, entry by entry."""
    flat = idx.reshape(-1).tolist()
    rows_of, entries, prefix = [-1] * len(flat), [], [0]
    by = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            by[e].append(i)
    for e in range(E):
        for i in by[e]:
            rows_of[i] = len(entries)
            entries.append(i)
        prefix.append(len(entries))
    return rows_of, entries, prefix


def sum_bound(n, magnitude, step=U32):
    g = n * step
    return g / (1 - g) * magnitude


def assert_within(got, exact, slack, rounding=0.0):
    """|got - exact| <= slack + rounding * (|exact| + slack), in 64 bits; NaN and infinities in
    the same places."""
    got, exact = got.double(), exact.double()
    assert got.shape == exact.shape
    fine = torch.isfinite(exact)
    assert torch.equal(torch.isnan(got), torch.isnan(exact))
    assert torch.equal(got[~fine & ~torch.isnan(exact)], exact[~fine & ~torch.isnan(exact)])
    slack = torch.as_tensor(slack, dtype=torch.float64, device=got.device).expand_as(exact)
    bad = fine & ((got - exact).abs() > slack + rounding * (exact.abs() + slack) + TINY)
    if bool(bad.any()):
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} values off; first at {at}: "
                             f"{float(got[at])} against {float(exact[at])}, allowed {float(slack[at])}")


def integers(g, *shape, most=3):
    """Small whole numbers in bf16: their products' sums are exact in fp32."""
    return torch.randint(-most, most + 1, shape, generator=g, device=g.device).to(torch.bfloat16)
