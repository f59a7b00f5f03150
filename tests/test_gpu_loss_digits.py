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


def _confident(T, D, l, second, sparse, seed):
    """X, W, labels: token t's product with its label 2t is about l, with 2t + 1 `second` times
    that, with all others near 0.  Dense: every term of the label's product is positive;
    sparse: only one is not zero."""
    g = torch.Generator().manual_seed(seed)
    V = 2 * T + 40
    if sparse:
        W, X = torch.zeros(V, D), torch.zeros(T, D)
        at = (torch.arange(T) * 37) % D
        X[torch.arange(T), at] = 5.0
        W[2 * torch.arange(T), at] = l / 5.0
    else:
        W = torch.randn(V, D, generator=g) / D ** 0.5
        X = W[0:2 * T:2] * (l / (W[0:2 * T:2] ** 2).sum(1, keepdim=True))
    W[1:2 * T:2] = W[0:2 * T:2] * second
    return X.bfloat16(), W.bfloat16(), 2 * torch.arange(T, dtype=torch.int32), V


@pytest.mark.parametrize("K,cap", [(0, 0.0), (1, 0.0), (0, 40.0)])
@pytest.mark.parametrize("T", [1, 5, 100])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("D,l,rest", [(4096, 22.0, 1e-3), (8192, 25.0, 1e-3), (8192, 25.0, 1e-4)])
def test_a_confident_tokens_gradient_keeps_its_digits(D, l, rest, sparse, T, K, cap):
    """dl at a label of probability p is p - 1, so that an error e of its logit against lse
    is an error e / (1 - p) of dl.  The label's logit is summed in f32 by 256 threads
    (D / 2048 vectors of 8, four sums each: D / 1024 additions, then 2 + 5 + 3, and a cap's
    2^-20 of it): off by (10 + D / 1024) 2^-24 of sum |x w|; lse by 2^-20 (2 + |lse|).
    The bound of the other columns is the header's."""
    uncap = (lambda a: cap * np.arctanh(a / cap)) if cap else (lambda a: a)
    second = uncap(l + np.log(rest)) / uncap(l)
    X, W, y, V = _confident(T, D, uncap(l), second, sparse, 7 * T + D)
    Xd, Wd, yn = X.double().numpy(), W.double().numpy(), y.numpy()
    x, w = X.cuda(), W.cuda()
    up = torch.ones(T, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dX, dW = torch.empty_like(x), torch.empty_like(w)
    if K:
        i, q = y[:, None].contiguous().cuda(), torch.zeros(T, 1, device="cuda")
        fcc.fcc_linear_distill(1, [x], [w], i, q, T, V, D, 1, [loss], [lse], softcap=cap)
        fcc.fcc_linear_distill_grad(1, [x], [w], i, q, [lse], up, T, V, D, 1, [dX], [dW], softcap=cap)
    else:
        fcc.fcc_linear_xent(1, [x], [w], y.cuda(), T, V, D, [loss], [lse], softcap=cap)
        fcc.fcc_linear_xent_grad(1, [x], [w], y.cuda(), [lse], up, T, V, D, [dX], [dW], softcap=cap)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    d = losses.xent_dlogits(Xd, Wd, yn, np.ones(T), softcap=cap)
    rl, rs = losses.xent(Xd, Wd, yn, softcap=cap)
    lg = losses.logits(Xd, Wd, cap)
    p = np.exp(lg - rs[:, None])
    rows = np.arange(T)
    assert (1 - p[rows, yn] < 10 * rest).all() and (1 - p[rows, yn] > 1e-5).all()
    mags = np.abs(Xd) @ np.abs(Wd).T
    err = D * 2.0 ** -23 * mags
    err[rows, yn] = (10 + D / 1024) * 2.0 ** -24 * mags[rows, yn]
    err += 2.0 ** -20 * np.abs(lg) * (cap > 0)
    tl = 2.0 ** -20 * (2 + np.abs(rs)) + (p * err).sum(1)
    ed = p * (err + tl[:, None] + 2.0 ** -20)
    if cap:  # (the factor 1 - (l / cap)^2 and its own error)
        f = 1 - (lg / cap) ** 2
        raw_d = np.abs(d / f)
        ed = ed * f + raw_d * (2 * np.abs(lg) / cap ** 2 * err + 2.0 ** -22)
    ed = ed + np.abs(d) * (2.0 ** -16 if T <= 64 else 2.0 ** -8)
    gX, gW = losses.gradients(d, Xd, Wd)
    tW = ed.T @ np.abs(Xd) + T * 2.0 ** -23 * (np.abs(d).T @ np.abs(Xd))
    tX = ed @ np.abs(Wd) + V * 2.0 ** -23 * (np.abs(d) @ np.abs(Wd))
    at = yn  # the labels' rows of dW: dl at the label times the token's X
    within(dW[at], gW[at], (tW + 2.0 ** -8 * (np.abs(gW) + tW))[at], "dW at the labels")
    within(dX, gX, tX + 2.0 ** -8 * (np.abs(gX) + tX), "dX")


@pytest.mark.parametrize("D", [1024, 8192, 1 << 17, 1 << 20])
def test_rows_that_nothing_is_cut_off_from(D):
    """Logits of a single product each, which the tensor core's sum holds exactly: what the
    forward pass multiplies back, 1.6e-8 for every 16 of D up to 131072, is then the
    error itself and bounds it (and 2^-20 (2 + |lse|) for lse's own rounding)."""
    T, V = 8, 24
    X, W = torch.zeros(T, D), torch.zeros(V, D)
    at = (torch.arange(T) * 1037) % D
    X[torch.arange(T), at] = 2.0
    W[torch.arange(T), at] = 100.0 + torch.arange(T)   # (the largest logits: word t for token t)
    X, W = X.bfloat16(), W.bfloat16()
    y = torch.arange(T, dtype=torch.int32) + T         # (labels elsewhere)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fcc.fcc_linear_xent(1, [X.cuda()], [W.cuda()], y.cuda(), T, V, D, [loss], [lse])
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    rl, rs = losses.xent(X.double().numpy(), W.double().numpy(), y.numpy())
    tol = (1.6e-8 * (min(D, 1 << 17) / 16) * rs + 2.0 ** -20 * (2 + rs))
    within(lse, rs, tol, "lse")
    within(loss, rl, tol, "loss")


@pytest.mark.parametrize("q", [(0.5, 0.05, 0.45), (0.05, 0.5, 0.45), (0.3, 0.02, 0.02, 0.3, 0.03, 0.33),
                               (0.2,) * 5])
def test_an_index_given_often_is_in_the_sum_once(q):
    """Heavy entries of one index with light ones between them: the sum takes the logit that
    is known by itself once.  Its f32 sum over 32 lanes of D / 8 products has at most D / 128
    + 7 additions, each off by 2^-24 of sum |x w|."""
    T, D, K = 6, 8192, len(q) + 2
    X, W, y, V = _confident(T, D, 25.0, 0.7, False, 3)
    idx = torch.stack([torch.cat([y[t:t + 1].repeat(len(q)), torch.tensor([(t + 5) % V, -1])])
                       for t in range(T)]).int()
    te = torch.log(torch.tensor([[*q, 0.01, 1.0]])).repeat(T, 1)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fcc.fcc_linear_distill(1, [X.cuda()], [W.cuda()], idx.cuda(), te.cuda(), T, V, D, K, [loss], [lse])
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    Xd, Wd = X.double().numpy(), W.double().numpy()
    rl, rs = losses.distill(Xd, Wd, idx.numpy(), te.numpy())
    mags = np.abs(Xd) @ np.abs(Wd).T
    p = np.exp(losses.logits(Xd, Wd) - rs[:, None])
    err = D * 2.0 ** -23 * mags
    err[np.arange(T), y.numpy()] *= (D / 128 + 7) / (2 * D)
    tl = (p * err).sum(1) + 2.0 ** -20 * (2 + rs)
    within(lse, rs, tl, "lse")

