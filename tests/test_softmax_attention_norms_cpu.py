"""The norm-wise limits of attention_norms: a kernel's roundings stay inside them, mistakes do not.  No GPU is used."""
import pytest
import torch

import attention_norms as norms

BF16 = torch.bfloat16
# T, S, H, Hk, D, causal
CASES = [(400, 513, 8, 2, 128, False), (1100, 1100, 4, 1, 64, True), (257, 257, 6, 2, 80, True)]


def operands(case):
    T, S, H, Hk, D, causal = case
    gen = torch.Generator().manual_seed(T)
    q, do = (torch.randn(T, H, D, generator=gen).to(BF16) for _ in range(2))
    k, v = (torch.randn(S, Hk, D, generator=gen).to(BF16) for _ in range(2))
    return q, k, v, do, causal


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_roundings_stay_inside(case):
    args = operands(case)
    want, got = norms.attention64(*args), norms.attention64(*args, rounding=BF16)
    for n in want:
        assert norms.off(got[n], want[n]) <= norms.LIMIT[BF16], n


@pytest.mark.parametrize("spoil,shows", [(("delta", 0.0), ("dq", "dk")), (("delta", 0.75), ("dq", "dk")), (("delta", 0.9), ("dq", "dk")),
                                         (("delta", 1.25), ("dq", "dk")), (("tile", 0), ("dq",)), (("tile", 1), ("dq",)),
                                         (("p", 0), ("dv",))])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_mistakes_do_not(case, spoil, shows):
    args = operands(case)
    want, got = norms.attention64(*args), norms.attention64(*args, spoil=spoil, rounding=BF16)
    for n in shows:
        assert norms.off(got[n], want[n]) > 1.25 * norms.LIMIT[BF16], n


def test_gradients_against_differences():
    gen = torch.Generator().manual_seed(1)
    q, do = (torch.randn(7, 4, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(9, 2, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    got = norms.attention64(q, k, v, do, True)
    for i, n in enumerate(("dq", "dk", "dv")):
        step = torch.randn([q, k, v][i].shape, generator=gen, dtype=torch.float64)
        ends = []
        for h in (1e-5, -1e-5):
            x = [q, k, v]
            x[i] = x[i] + h * step
            ends.append(float((norms.attention64(*x, do, True)["o"] * do).sum()))
        slope = (ends[0] - ends[1]) / 2e-5
        assert abs(float((got[n] * step).sum()) - slope) < 1e-7 * max(1.0, abs(slope))
