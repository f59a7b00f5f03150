"""GPU tests of how many digits the linear losses keep: soft caps of every size,
long rows, confident tokens, and the workspace's exact size.

Tolerances are those of test_gpu_losses.py but for the cap's share, which is
relative here (u = 2^-24): for |x| < c/2 the series is off by 1.5 u (first
omitted term), its rounded argument and Horner steps by 2 u and the last product
by 1 u; past it c - 2c / (1 + e) has e off by (4 + 8 |x|/c) u, at |x| = c/2
worth 0.85 of that, 3 u of the reciprocal's term times (1 - t)/t = 1.2, and one
rounding, 12 u in all, falling with |x|.  So a capped logit is off by less than
2^-20 of itself, whatever the cap.
"""
import numpy as np
import pytest
import torch

from oracle import losses
from tests.gpu_util import to_f64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_collective_gb300 as fcc  # noqa: E402
from tests.test_gpu_losses import Case, check, within  # noqa: E402


class Relative(Case):
    """The cap's error is relative to the logit."""

    def logit_err(self):
        X, W = self.f64()
        return (self.D * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T)
                + 2.0 ** -20 * np.abs(losses.logits(X, W, self.cap)))


@pytest.mark.parametrize("K,smoothing", [(0, 0.0), (0, 0.1), (5, 0.0)])
@pytest.mark.parametrize("cap", [0.25, 5.0, 30.0, 1e3, 1e4, 1e6, 1e30])
def test_a_soft_cap_of_any_size_keeps_the_digits(cap, K, smoothing):
    for T in (40, 130):
        check(Relative(1, T, 600, 16, K=K, cap=cap, smoothing=smoothing))


@pytest.mark.parametrize("cap", [2.0, 30.0])
def test_capped_logits_that_are_not_finite(cap):
    """An infinite product is the cap itself; a NaN shows in its own row only."""
    T, V, D = 40, 300, 16
    c = Relative(1, T, V, D, cap=cap)
    c.labels[5] = 11
    c.X[5] = 0
    c.X[5, 3] = float("inf")   # (the row's logits: +-cap)
    c.W[:, 3] = torch.where(c.W[:, 3] == 0, 0.5, c.W[:, 3].float()).bfloat16()
    c.X[7, 2] = float("nan")
    c.dev()
    loss, lse = c.forward()
    sign = torch.sign(c.W[:, 3].double())
    want = torch.logsumexp(cap * sign, 0)
    # (+-cap exactly; the sum and the logarithm as in the header of test_gpu_losses.py)
    assert abs(float(lse[0][5]) - float(want)) <= 2.0 ** -20 * (2 + abs(float(want)))
    gap = float(want) - cap * float(sign[11])
    assert abs(float(loss[0][5]) - gap) <= 2.0 ** -19 * (2 + abs(float(want)) + cap)
    assert torch.isnan(lse[0][7])
    rest = [t for t in range(T) if t != 7]
    assert torch.isfinite(lse[0][rest]).all() and torch.isfinite(loss[0][rest]).all()
