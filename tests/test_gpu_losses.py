"""GPU parity: the vocabulary-parallel losses and their gradients against the
fp64 oracle, through the C ABI.

Tolerances (u16 = 2^-8, bf16's rounding; u32 = 2^-24):
  logits    a sum of D products in f32: at most D 2^-23 sum |x w| (the tensor
            cores may cut a sum off rather than round it), plus 2^-21 cap
            where it is capped (tanhf and two products);
  lse       the logits' error / tau, plus 2^-20 (2 + |lse|) for the base-2
            maximum, the approximate exponentials (2^-22 each, relative), the
            sums and the logarithm;
  loss      tau^2 (twice those, plus 2^-20 (the logits' size + |lse| + log V)),
            and 2 z |lse| times lse's error;
  gradients elementwise: each dl is off by 2^-8 |dl| (bf16) and by
            a p (lse's + the logits' error + 2^-20) (+ 2^-20 |w| at a target);
            through the product with |W| or |X|, whose own sums are off by
            n 2^-23 of the sum of magnitudes; then 2^-8 |result|.
"""
import numpy as np
import pytest
import torch

from oracle import losses
from tests.gpu_util import bits, to_f64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_collective_gb300 as fcc  # noqa: E402

IGNORE = -100


class Case:
    """Inputs on the device and in fp64, and the oracle's answers with their tolerances."""

    def __init__(self, R, T, V, D, K=0, smoothing=0.0, z=0.0, cap=0.0, tau=1.0, seed=0, scale=1.5):
        g = torch.Generator().manual_seed(1000 * seed + 7 * T + V + D + K)
        self.R, self.T, self.V, self.D, self.K = R, T, V, D, K
        self.smoothing, self.z, self.cap, self.tau = smoothing, z, cap, tau
        X = torch.randn(T, D, generator=g).bfloat16()
        W = (torch.randn(V, D, generator=g) * scale / D ** 0.5).bfloat16()
        self.labels = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
        for t, y in ((0, V - 1), (1, 0), (2, V // R - 1), (3, V // R % V), (4, min(V - 1, 255)),
                     (5, min(V - 1, 256)), (6, IGNORE), (8, IGNORE)):
            if t < T and T > 1:
                self.labels[t] = y
        self.idx = self.te = None
        if K:
            self.idx = torch.stack([torch.randperm(V, generator=g)[:K] if V >= K else
                                    torch.randint(0, V, (K,), generator=g) for _ in range(T)]).int()
            self.te = torch.randn(T, K, generator=g) * 2
            if T > 4:
                self.idx[1] = -1                            # nothing
                self.idx[2, K // 2:] = -1                   # half
                self.te[3, : K - 1] = -float("inf")         # one entry left
                self.te[4] = torch.finfo(torch.float32).min  # all at the type's lowest value
                self.idx[0, 0] = V - 1
        self.dloss = torch.randn(T, generator=g)
        self.X, self.W = X, W
        self.dev()

    def dev(self):
        self.dX_in = [self.X.cuda() for _ in range(self.R)]
        self.dW_in = [w.contiguous() for w in self.W.cuda().split(self.V // self.R)]
        self.y = self.labels.cuda()
        self.di = self.idx.cuda() if self.K else None
        self.dt = self.te.cuda() if self.K else None
        self.g = self.dloss.cuda()

    def forward(self, opts=None, stream=None, check=True):
        R, T = self.R, self.T
        loss = [torch.full((T,), float("nan"), device="cuda") for _ in range(R)]
        lse = [torch.full((T,), float("nan"), device="cuda") for _ in range(R)]
        if self.K:
            fcc.fcc_linear_distill(R, self.dX_in, self.dW_in, self.di, self.dt, T, self.V, self.D,
                                   self.K, loss, lse, temperature=self.tau, softcap=self.cap,
                                   opts=opts, stream=stream)
        else:
            fcc.fcc_linear_xent(R, self.dX_in, self.dW_in, self.y, T, self.V, self.D, loss, lse,
                                ignore_index=IGNORE, smoothing=self.smoothing, z_weight=self.z,
                                softcap=self.cap, opts=opts, stream=stream)
        if check:
            assert fcc.fcc_stream_status(stream) == fcc.FCC_OK
        return loss, lse

    def backward(self, lse, opts=None, stream=None, dx=True, dw=True, check=True):
        R, T, nan = self.R, self.T, float("nan")
        dX = [torch.full((T, self.D), nan, device="cuda", dtype=torch.bfloat16)
              for _ in range(R)] if dx else None
        dW = [torch.full((self.V // R, self.D), nan, device="cuda", dtype=torch.bfloat16)
              for _ in range(R)] if dw else None
        if self.K:
            fcc.fcc_linear_distill_grad(R, self.dX_in, self.dW_in, self.di, self.dt, lse, self.g, T,
                                        self.V, self.D, self.K, dX, dW, temperature=self.tau,
                                        softcap=self.cap, opts=opts, stream=stream)
        else:
            fcc.fcc_linear_xent_grad(R, self.dX_in, self.dW_in, self.y, lse, self.g, T, self.V,
                                     self.D, dX, dW, ignore_index=IGNORE, smoothing=self.smoothing,
                                     z_weight=self.z, softcap=self.cap, opts=opts, stream=stream)
        if check:
            assert fcc.fcc_stream_status(stream) == fcc.FCC_OK
        return dX, dW

    # ---------------------------------------------------------------- oracle
    def f64(self):
        return self.X.double().numpy(), self.W.double().numpy()

    def logit_err(self):
        X, W = self.f64()
        e = self.D * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T)
        return e + 2.0 ** -21 * self.cap

    def oracle_forward(self):
        X, W = self.f64()
        if self.K:
            loss, lse = losses.distill(X, W, self.idx.numpy(), self.te.numpy(), self.tau, self.cap)
        else:
            loss, lse = losses.xent(X, W, self.labels.numpy(), IGNORE, self.smoothing, self.z,
                                    self.cap)
        el = self.logit_err().max(axis=1) / self.tau
        top = np.abs(losses.logits(X, W, self.cap)).max(axis=1) / self.tau
        tl = el + 2.0 ** -20 * (2 + np.abs(lse))
        to = self.tau ** 2 * (2 * (el + tl) + 2.0 ** -20 * (top + np.abs(lse) + np.log(self.V) + 1))
        return loss, lse, to + 2 * self.z * np.abs(lse) * tl, tl

    def oracle_backward(self):
        X, W = self.f64()
        live = np.ones(self.T, bool)
        if self.K:
            d = losses.distill_dlogits(X, W, self.idx.numpy(), self.te.numpy(), self.dloss.numpy().astype(float),
                                       self.tau, self.cap)
            live = np.array([bool(r) for r in losses.teacher_probs(
                self.idx.numpy(), self.te.numpy(), self.V, self.tau)])
        else:
            y = self.labels.numpy()
            d = losses.xent_dlogits(X, W, y, self.dloss.numpy().astype(float), IGNORE, self.smoothing,
                                    self.z, self.cap)
            live = (y >= 0) & (y < self.V)
        _, lse, _, tl = self.oracle_forward()
        l = losses.logits(X, W, self.cap) / self.tau
        a = np.abs(self.dloss.numpy().astype(float)) * self.tau * (1 + 2 * self.z * np.abs(lse)) * live
        p = np.exp(l - lse[:, None])
        ed = 2.0 ** -8 * np.abs(d) + a[:, None] * (p * (tl[:, None] + self.logit_err() / self.tau
                                                        + 2.0 ** -20) + 2.0 ** -20 * (p > 0))
        dX, dW = losses.gradients(d, X, W)
        tX = ed @ np.abs(W) + self.V * 2.0 ** -23 * (np.abs(d) @ np.abs(W))
        tW = ed.T @ np.abs(X) + self.T * 2.0 ** -23 * (np.abs(d).T @ np.abs(X))
        return dX, dW, tX + 2.0 ** -8 * (np.abs(dX) + tX), tW + 2.0 ** -8 * (np.abs(dW) + tW)


def within(got, ref, tol, what):
    got = to_f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][:3]} for {ref[bad][:3]}, tolerance {tol[bad][:3]}")


def check(c, opts=None):
    loss, lse = c.forward(opts)
    rl, rs, tol_l, tol_s = c.oracle_forward()
    for r in range(c.R):
        within(lse[r], rs, tol_s, f"lse {r}")
        within(loss[r], rl, tol_l, f"loss {r}")
    dX, dW = c.backward(lse, opts)
    gX, gW, tX, tW = c.oracle_backward()
    n = c.V // c.R
    for r in range(c.R):
        within(dX[r], gX, tX, f"dX {r}")
        within(dW[r], gW[r * n:(r + 1) * n], tW[r * n:(r + 1) * n], f"dW {r}")


SHAPES = [  # R, T, V, D
    (1, 1, 1, 8), (1, 1, 300, 64), (1, 2, 255, 72), (1, 9, 256, 8), (1, 127, 257, 128),
    (1, 128, 1009, 200), (1, 129, 513, 64), (2, 33, 514, 264), (3, 17, 999, 136), (4, 70, 1028, 56),
    (8, 5, 8, 16), (8, 200, 2056, 96), (1, 300, 700, 520), (2, 257, 1024, 256),
]


@pytest.mark.parametrize("R,T,V,D", SHAPES)
def test_xent(R, T, V, D):
    check(Case(R, T, V, D))


@pytest.mark.parametrize("R,T,V,D,K", [(*s, k) for s, k in zip(
    SHAPES, [1, 2, 31, 32, 33, 128, 256, 7, 64, 100, 3, 5, 255, 20])])
@pytest.mark.parametrize("tau,cap", [(1.0, 0.0), (2.5, 5.0)])
def test_distill(R, T, V, D, K, tau, cap):
    check(Case(R, T, V, D, K=K, tau=tau, cap=cap))


@pytest.mark.parametrize("smoothing,z,cap", [(0.1, 0.0, 0.0), (0.0, 1e-2, 0.0), (0.0, 0.0, 4.0),
                                             (0.3, 1e-3, 30.0)])
@pytest.mark.parametrize("R,T,V,D", [(1, 40, 777, 96), (2, 140, 1100, 64)])
def test_xent_terms(R, T, V, D, smoothing, z, cap):
    check(Case(R, T, V, D, smoothing=smoothing, z=z, cap=cap))


@pytest.mark.parametrize("pair", [1, 2])
@pytest.mark.parametrize("chunks", [1, 2, 3])
def test_tile_shapes_and_pieces(pair, chunks):
    for K in (0, 12):
        check(Case(2, 300, 2 * 777, 328, K=K), fcc.make_opts(cta_pair=pair, chunks=chunks))
    check(Case(1, 20, 513, 64, smoothing=0.1), fcc.make_opts(cta_pair=pair, chunks=chunks, max_ctas=3))


@pytest.mark.parametrize("max_ctas", [1, 2, 5, 8, 11, 40])
@pytest.mark.parametrize("chunks", [1, 3])
def test_every_way_to_share_the_tiles(max_ctas, chunks):
    """Few CTAs: whole rounds of dX tiles, shared ones with and without helpers,
    last pieces shorter than the plan."""
    o = fcc.make_opts(max_ctas=max_ctas, chunks=chunks)
    for case in (Case(2, 300, 2 * 650, 648), Case(1, 100, 1500, 1160, K=6), Case(1, 20, 900, 520)):
        check(case, o)


def test_few_tokens_keep_the_gradients_exact():
    """Up to 64 tokens dl is two bf16 numbers: dW is one rounding (2^-8) off, not two."""
    for T in (1, 2, 31, 32, 33, 63, 64):
        for K in (0, 3):
            c = Case(1, T, 400, 64, K=K)
            _, lse = c.forward()
            dX, dW = c.backward(lse)
            gX, gW, tX, tW = c.oracle_backward()
            # what is left of tX, tW without dl's rounding: below 2^-14 of the sums of magnitudes
            X, W = c.f64()
            l = losses.logits(X, W)
            p = np.exp(l - losses.logsumexp(l)[:, None])
            a = np.abs(c.dloss.numpy().astype(float))[:, None] * (p + 2.0 ** -10)
            within(dX[0], gX, 2.0 ** -8 * np.abs(gX) + 2.0 ** -12 * (a @ np.abs(W)), f"dX {T} {K}")
            within(dW[0], gW, 2.0 ** -8 * np.abs(gW) + 2.0 ** -12 * (a.T @ np.abs(X)), f"dW {T} {K}")


@pytest.mark.parametrize("D", [64, 1024, 8192])
def test_losses_hold_their_digits_over_long_rows(D):
    """A label that stands out, and sums of up to 8192 terms that agree in sign:
    the loss is off by less than 4e-6 (2^-18) of lse and logit; the tensor
    cores alone, which cut off, would be off by 1.6e-8 per 16 terms, 8e-5 here."""
    g = torch.Generator().manual_seed(D)
    T, V = 200, 700
    W = (torch.randn(V, D, generator=g) * 1.3 / D ** 0.5).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    X = (torch.randn(T, D, generator=g) + 6 * W[y.long()].float()).bfloat16()
    idx = y[:, None].contiguous()
    rl, rs = losses.xent(X.double().numpy(), W.double().numpy(), y.numpy())
    x, w = X.cuda(), W.cuda()
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fcc.fcc_linear_xent(1, [x], [w], y.cuda(), T, V, D, [loss], [lse])
    kd, ks = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fcc.fcc_linear_distill(1, [x], [w], idx.cuda(), torch.zeros(T, 1, device="cuda"), T, V, D, 1, [kd], [ks])
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    for got in (loss, kd):
        assert np.abs(to_f64(got) - rl).max() <= 2.0 ** -18 * (np.abs(rs).max() + 1)
    for got in (lse, ks):
        assert np.abs(to_f64(got) - rs).max() <= 2.0 ** -18 * (np.abs(rs).max() + 1)


def test_a_suspended_wait_runs_out():
    fcc.fcc_test_suspended_wait_timeout(2_000_000)  # 2 ms on a barrier nothing completes
    assert fcc.fcc_stream_status() == fcc.FCC_ERR_TIMEOUT
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    check(Case(1, 30, 300, 64))


def test_the_example_trains():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "train_head.py"), "--steps", "12"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "cross entropy" in r.stdout and "distillation" in r.stdout


@pytest.mark.parametrize("K", [0, 9])
def test_rows_without_targets(K):
    """All rows ignored: losses and gradients are exact zeros, whatever dloss holds."""
    c = Case(2, 37, 600, 64, K=K)
    if K:
        c.idx.fill_(-1)
    else:
        c.labels.fill_(IGNORE)
    c.dloss.fill_(float("nan"))
    c.dev()
    loss, lse = c.forward()
    _, rs, _, tol = c.oracle_forward()
    dX, dW = c.backward(lse)
    for r in range(2):
        within(lse[r], rs, tol, "lse")
        for x in (loss[r], dX[r], dW[r]):
            assert torch.count_nonzero(x) == 0 and not torch.isnan(x).any()


def test_bad_targets_are_reported_and_ignored():
    c = Case(1, 20, 300, 64)
    c.labels[3], c.labels[7] = 300, -5
    c.dev()
    loss, lse = c.forward(check=False)
    assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID
    dX, dW = c.backward(lse, check=False)
    assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID
    rl, _, tol, _ = c.oracle_forward()
    within(loss[0], rl, tol, "loss")
    gX, gW, tX, tW = c.oracle_backward()
    within(dX[0], gX, tX, "dX")
    within(dW[0], gW, tW, "dW")
    c = Case(1, 20, 300, 64, K=5)
    c.idx[6, 2], c.idx[9, 0] = 300, 2 ** 31 - 1
    c.dev()
    loss, lse = c.forward(check=False)
    assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID
    rl, _, tol, _ = c.oracle_forward()
    within(loss[0], rl, tol, "loss")
    assert fcc.fcc_stream_status() == fcc.FCC_OK


def test_an_index_given_twice_counts_twice():
    c = Case(1, 12, 280, 64, K=6)
    c.idx[:, 3] = c.idx[:, 0]
    c.idx[5:, 4] = c.idx[5:, 0]
    c.dev()
    check(c)


def test_ignore_index_may_be_a_vocabulary_index():
    c = Case(1, 30, 270, 64)
    c.labels[::3] = 0
    c.dev()
    loss = torch.empty(30, device="cuda")
    lse = torch.empty(30, device="cuda")
    fcc.fcc_linear_xent(1, c.dX_in, c.dW_in, c.y, 30, 270, 64, [loss], [lse], ignore_index=0)
    dX = torch.empty(30, 64, device="cuda", dtype=torch.bfloat16)
    fcc.fcc_linear_xent_grad(1, c.dX_in, c.dW_in, c.y, [lse], c.g, 30, 270, 64, [dX], None,
                             ignore_index=0)
    fcc.fcc_stream_status()  # (label -100 is out of range here)
    dead = c.y == 0
    assert torch.count_nonzero(loss[dead]) == 0 and torch.count_nonzero(dX[dead]) == 0
    assert (loss[c.y > 0] != 0).all()


@pytest.mark.parametrize("K", [0, 4])
def test_one_sided_gradients_are_the_same(K):
    c = Case(2, 150, 700, 96, K=K)
    _, lse = c.forward()
    dX, dW = c.backward(lse)
    only_x, none_w = c.backward(lse, dw=False)
    none_x, only_w = c.backward(lse, dx=False)
    assert none_w is None and none_x is None
    for r in range(2):
        assert np.array_equal(bits(dX[r]), bits(only_x[r]))
        assert np.array_equal(bits(dW[r]), bits(only_w[r]))


@pytest.mark.parametrize("K", [0, 40])
def test_repeatable_on_other_streams_and_in_a_graph(K):
    c = Case(2, 200, 1500, 264, K=K, smoothing=0.0 if K else 0.1)
    loss, lse = c.forward()
    dX, dW = c.backward(lse)
    want = [bits(x) for x in (*loss, *lse, *dX, *dW)]
    size = max(fcc.fcc_linear_loss_workspace_size(2, 200, 1500, 264, K, g) for g in (False, True))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    o = fcc.make_opts(workspace=ws, workspace_bytes=size)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        ws.fill_(0xFF)
        l2, s2 = c.forward(o, st)
        x2, w2 = c.backward(s2, o, st)
    st.synchronize()
    for a, b in zip(want, (*l2, *s2, *x2, *w2)):
        assert np.array_equal(a, bits(b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = torch.cuda.current_stream()
        l3, s3 = c.forward(o, cap, check=False)
        x3, w3 = c.backward(s3, o, cap, check=False)
    for _ in range(2):
        for x in (*l3, *s3, *x3, *w3):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (*l3, *s3, *x3, *w3)):
            assert np.array_equal(a, bits(b))
    # a workspace one byte short is refused
    for call in (lambda q: c.forward(q, check=False), lambda q: c.backward(lse, q, check=False)):
        with pytest.raises(fcc.FccError) as e:
            call(fcc.make_opts(workspace=ws, workspace_bytes=200))
        assert e.value.status == fcc.FCC_ERR_WORKSPACE


def test_outputs_end_where_they_should():
    """Guard words on both sides of every output stay untouched."""
    R, T, V, D = 2, 45, 2 * 301, 72
    c = Case(R, T, V, D)

    def guarded(n, dtype):
        t = torch.full((n + 64,), 7.0, device="cuda", dtype=dtype)
        return t, t[32:32 + n]

    loss, lse = ([guarded(T, torch.float32) for _ in range(R)] for _ in range(2))
    dX = [guarded(T * D, torch.bfloat16) for _ in range(R)]
    dW = [guarded(V // R * D, torch.bfloat16) for _ in range(R)]
    fcc.fcc_linear_xent(R, c.dX_in, c.dW_in, c.y, T, V, D, [x for _, x in loss], [x for _, x in lse])
    fcc.fcc_linear_xent_grad(R, c.dX_in, c.dW_in, c.y, [x for _, x in lse], c.g, T, V, D,
                             [x for _, x in dX], [x for _, x in dW])
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    for whole, part in (*loss, *lse, *dX, *dW):
        assert (whole[:32] == 7).all() and (whole[-32:] == 7).all()
        assert not (part == 7).all()


def test_large_logits_and_non_finite_ones():
    """Logits of +-1e4 neither overflow nor lose the loss; NaN and infinite ones show."""
    c = Case(1, 40, 600, 64, scale=2e3)
    check(c)
    c = Case(1, 6, 300, 64)
    c.X[2, 5] = float("nan")
    c.W[7] = float("inf")   # (a logit of +-inf or NaN in every row)
    c.dev()
    loss, lse = c.forward()
    assert not torch.isfinite(loss[0][c.y >= 0]).any()
    c = Case(1, 6, 300, 64)
    c.X[2, 5] = float("nan")
    c.dev()
    loss, lse = c.forward()
    assert torch.isnan(lse[0][2]) and torch.isfinite(lse[0][[0, 1, 3, 4, 5]]).all()
    dX, dW = c.backward(lse)
    assert torch.isnan(dX[0][2]).all() and torch.isfinite(dX[0][[0, 1, 3, 4, 5]]).all()


@pytest.mark.parametrize("K,tau,cap", [(0, 1.0, 0.0), (0, 1.0, 6.0), (8, 2.0, 0.0)])
def test_gradient_against_differences(K, tau, cap):
    """The kernels' own loss at X + h and X - h (both exact in bf16) against dX."""
    T, V, D = 16, 500, 64
    c = Case(1, T, V, D, K=K, tau=tau, cap=cap)
    c.dloss.fill_(1.0)
    c.X = (torch.round(c.X * 16) / 16).clamp(-3, 3).bfloat16()  # k/16, |k| <= 48
    h = 2.0 ** -6
    u = torch.where(torch.rand(T, D, generator=torch.Generator().manual_seed(5)) < 0.5, -h, h)
    X0 = c.X
    c.dev()
    _, lse = c.forward()
    dX, _ = c.backward(lse)
    _, _, tX, _ = c.oracle_backward()
    got = []
    tol = np.zeros(T)
    for sign in (1, -1):
        c.X = (X0.float() + sign * u).bfloat16()
        assert torch.equal(c.X.float(), X0.float() + sign * u)
        c.dev()
        got.append(to_f64(c.forward()[0][0]))
        tol += c.oracle_forward()[2]
    un = u.double().numpy()
    along = (to_f64(dX[0]) * un).sum(1)
    # third derivative of a log-sum-exp along a line: at most 2 (max |dl|)^3, the cap's adds as much
    dl = np.abs(un @ c.W.double().numpy().T).max(1) / tau
    curve = tau ** 2 * (2 + 8 * (cap > 0)) * dl ** 3 / 6 * 2
    tol = tol / 2 + (tX * np.abs(un)).sum(1) + curve
    assert (np.abs((got[0] - got[1]) / 2 - along) <= tol).all()
    assert np.max(np.abs(along) / tol) > 4  # (the steps of some tokens stand out of the tolerance)


def test_offsets_past_32_bits():
    """dl of 2.4e9 elements in one piece; partials and outputs checked on sampled rows."""
    T, V, D = 40000, 60000, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(T, D, device="cuda", generator=g).bfloat16()
    W = (torch.randn(V, D, device="cuda", generator=g) / 8).bfloat16()
    y = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    dl = torch.full((T,), 1.0, device="cuda")
    o = fcc.make_opts(chunks=1)
    size = fcc.fcc_linear_loss_workspace_size(1, T, V, D, 0, True, o)
    assert size > 2 ** 32
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    o = fcc.make_opts(chunks=1, workspace=ws, workspace_bytes=size)
    fcc.fcc_linear_xent(1, [X], [W], y, T, V, D, [loss], [lse])
    fcc.fcc_linear_xent_grad(1, [X], [W], y, [lse], dl, T, V, D, [dX], [dW], opts=o)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    rows = torch.tensor([0, 1, 19999, T - 2, T - 1], device="cuda")
    l = X[rows].double() @ W.double().T
    ref = torch.logsumexp(l, 1)
    # |logits| < 10: the header's bounds come to less than 2e-4
    assert (lse[rows].double() - ref).abs().max() < 2e-4
    at = l.gather(1, y[rows].long()[:, None])[:, 0]
    assert (loss[rows].double() - (ref - at)).abs().max() < 4e-4
    d = torch.softmax(l, 1)
    d.scatter_add_(1, y[rows].long()[:, None], -torch.ones(len(rows), 1, device="cuda").double())
    want = d @ W.double()
    # each dl is off by 2^-8 (and 1e-3 for the statistics), the sum by V 2^-23, the result by 2^-8
    tol = (2.0 ** -8 + 1e-3 + V * 2.0 ** -23) * (d.abs() @ W.double().abs()) * 1.01 + 2.0 ** -8 * want.abs()
    assert ((dX[rows].double() - want).abs() <= tol).all()
    cols = torch.tensor([0, 255, 256, V - 2, V - 1], device="cuda")
    d = torch.exp(X.double() @ W[cols].double().T - lse.double()[:, None])
    d -= (y[:, None] == cols[None]).double()
    want = d.T @ X.double()
    tol = (2.0 ** -8 + 1e-3 + T * 2.0 ** -23) * (d.abs().T @ X.double().abs()) * 1.01 + 2.0 ** -8 * want.abs()
    assert ((dW[cols].double() - want).abs() <= tol).all()
