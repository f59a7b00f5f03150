"""CPU checks of the vocabulary-parallel losses: the fp64 oracle against finite
differences and limiting cases, and the entry points' refusals and sizes."""
import ctypes

import numpy as np
import pytest

from oracle import losses


@pytest.fixture(scope="module")
def fcc():
    import __graft_entry__
    __graft_entry__.build()
    import gemm_collective_gb300 as m
    return m


def _case(seed, T=4, V=11, D=6, K=3):
    g = np.random.default_rng(seed)
    X, W = g.standard_normal((T, D)), g.standard_normal((V, D))
    labels = g.integers(0, V, T)
    labels[1] = -100
    idx = np.stack([g.permutation(V)[:K] for _ in range(T)])
    idx[2, 1:] = -1
    idx[3] = -1
    return X, W, labels, idx, g.standard_normal((T, K)) * 2, 0.5 + g.random(T)


@pytest.mark.parametrize("softcap", [0.0, 3.0])
@pytest.mark.parametrize("smoothing,z,tau", [(0.0, 0.0, 1.0), (0.1, 0.01, 2.0), (0.3, 0.0, 0.7)])
def test_oracle_gradients_match_differences(softcap, smoothing, z, tau):
    X, W, y, idx, te, g = _case(3)
    kinds = [(lambda a, b: losses.xent(a, b, y, -100, smoothing, z, softcap)[0],
              losses.xent_dlogits(X, W, y, g, -100, smoothing, z, softcap)),
             (lambda a, b: losses.distill(a, b, idx, te, tau, softcap)[0],
              losses.distill_dlogits(X, W, idx, te, g, tau, softcap))]
    h = 1e-5
    for f, d in kinds:
        dX, dW = losses.gradients(d, X, W)
        for A, dA, which in ((X, dX, 0), (W, dW, 1)):
            for i in np.ndindex(A.shape):
                up, dn = A.copy(), A.copy()
                up[i] += h
                dn[i] -= h
                a = (g * f(*((up, W) if which == 0 else (X, up)))).sum()
                b = (g * f(*((dn, W) if which == 0 else (X, dn)))).sum()
                # third derivatives of these losses are below 1e3 here: h^2 1e3 / 6
                assert abs((a - b) / (2 * h) - dA[i]) < 1e-7 + 1e-9 / h


def test_oracle_limits():
    X, W, y, idx, te, g = _case(5)
    loss, lse = losses.xent(X, W, y)
    p = np.exp(losses.logits(X, W) - lse[:, None])
    assert np.allclose(p.sum(1), 1)
    assert loss[1] == 0 and np.allclose(loss[0], -np.log(p[0, y[0]]))
    # one teacher entry is a label; a large cap is none
    one = np.where(y < 0, -1, y)[:, None]
    assert np.allclose(losses.distill(X, W, one, np.zeros((4, 1)))[0], loss)
    assert np.allclose(losses.xent(X, W, y, softcap=1e6)[0], loss)
    # a teacher that is the student has no loss and no gradient
    full = np.tile(np.arange(11), (4, 1))
    same = losses.logits(X, W)
    assert np.allclose(losses.distill(X, W, full, same, 2.0)[0], 0)
    assert np.allclose(losses.distill_dlogits(X, W, full, same, g, 2.0), 0)
    # -inf, negative and far indices are no entries; an index given twice counts twice
    bad = np.array([[1, 5, -1, 99]] * 4)
    tl = np.array([[0.5, -np.inf, 3.0, 3.0]] * 4)
    assert losses.teacher_probs(bad, tl, 11, 1.0) == [[(1, 1.0)]] * 4
    twice = losses.distill_dlogits(X, W, np.array([[2, 2]] * 4), np.zeros((4, 2)), g)
    assert np.allclose(twice, losses.distill_dlogits(X, W, np.array([[2]] * 4), np.zeros((4, 1)), g))
    # every rank's rows of dW are the whole head's rows
    d = losses.xent_dlogits(X, W, y, g)
    dX, dW = losses.gradients(d, X, W)
    parts = [losses.gradients(d[:, s], X, W[s]) for s in (slice(0, 5), slice(5, 11))]
    assert np.allclose(parts[0][0] + parts[1][0], dX)
    assert np.allclose(np.concatenate([q[1] for q in parts]), dW)


P = ctypes.c_void_p
F = ctypes.c_float


def _arr(*a):
    return (P * len(a))(*a)


def _xent(f, **k):
    two = _arr(16, 32)
    a = dict(R=2, X=two, W=two, y=P(16), T=4, V=10, D=16, loss=two, lse=two, ig=-100, s=0.0, z=0.0,
             cap=0.0, dt=0, o=None)
    a.update(k)
    return f.raw_status("fcc_linear_xent", a["R"], a["X"], a["W"], a["y"], ctypes.c_int64(a["T"]),
                        ctypes.c_int64(a["V"]), ctypes.c_int64(a["D"]), a["loss"], a["lse"],
                        ctypes.c_int32(a["ig"]), F(a["s"]), F(a["z"]), F(a["cap"]), a["dt"], a["o"],
                        None)


def _xent_grad(f, **k):
    two = _arr(16, 32)
    a = dict(R=2, X=two, W=two, y=P(16), lse=two, g=P(16), T=4, V=10, D=16, dX=two, dW=two, ig=-100,
             s=0.0, z=0.0, cap=0.0, dt=0, od=0, o=None)
    a.update(k)
    return f.raw_status("fcc_linear_xent_grad", a["R"], a["X"], a["W"], a["y"], a["lse"], a["g"],
                        ctypes.c_int64(a["T"]), ctypes.c_int64(a["V"]), ctypes.c_int64(a["D"]),
                        a["dX"], a["dW"], ctypes.c_int32(a["ig"]), F(a["s"]), F(a["z"]), F(a["cap"]),
                        a["dt"], a["od"], a["o"], None)


def _distill(f, **k):
    two = _arr(16, 32)
    a = dict(R=2, X=two, W=two, i=P(16), te=P(16), T=4, V=10, D=16, K=3, loss=two, lse=two, tau=1.0,
             cap=0.0, dt=0, o=None)
    a.update(k)
    return f.raw_status("fcc_linear_distill", a["R"], a["X"], a["W"], a["i"], a["te"],
                        ctypes.c_int64(a["T"]), ctypes.c_int64(a["V"]), ctypes.c_int64(a["D"]),
                        a["K"], a["loss"], a["lse"], F(a["tau"]), F(a["cap"]), a["dt"], a["o"], None)


def _distill_grad(f, **k):
    two = _arr(16, 32)
    a = dict(R=2, X=two, W=two, i=P(16), te=P(16), lse=two, g=P(16), T=4, V=10, D=16, K=3, dX=two,
             dW=two, tau=1.0, cap=0.0, dt=0, od=0, o=None)
    a.update(k)
    return f.raw_status("fcc_linear_distill_grad", a["R"], a["X"], a["W"], a["i"], a["te"], a["lse"],
                        a["g"], ctypes.c_int64(a["T"]), ctypes.c_int64(a["V"]),
                        ctypes.c_int64(a["D"]), a["K"], a["dX"], a["dW"], F(a["tau"]), F(a["cap"]),
                        a["dt"], a["od"], a["o"], None)


def test_refusals_without_a_device(fcc):
    bad, null = _arr(16, 36), _arr(16, 0)
    odd = _arr(16, 34)
    nan, inf = float("nan"), float("inf")
    every = [dict(R=0), dict(R=9), dict(T=0), dict(T=-1), dict(V=0), dict(V=11), dict(D=12),
             dict(D=0), dict(T=1 << 29), dict(V=1 << 31), dict(D=1 << 25), dict(X=bad), dict(W=bad),
             dict(X=null), dict(W=null), dict(X=None), dict(W=None), dict(cap=-1.0), dict(cap=nan),
             dict(cap=inf), dict(dt=7), dict(dt=-1)]
    opts = [dict(o=ctypes.byref(fcc.make_opts(algo=99))), dict(o=ctypes.byref(fcc.make_opts(algo=-1))),
            dict(o=ctypes.byref(fcc.make_opts(cta_pair=3))),
            dict(o=ctypes.byref(fcc.make_opts(chunks=-1)))]
    xent = [dict(y=P(0)), dict(y=P(18)), dict(s=1.0), dict(s=-0.1), dict(s=nan), dict(z=-1.0),
            dict(z=nan), dict(z=inf)]
    teach = [dict(i=P(0)), dict(te=P(0)), dict(i=P(18)), dict(te=P(18)), dict(K=0), dict(K=-1),
             dict(K=257), dict(tau=0.0), dict(tau=-1.0), dict(tau=nan), dict(tau=inf)]
    fwd = [dict(loss=None), dict(lse=None), dict(loss=null), dict(lse=null), dict(lse=odd),
           dict(loss=odd)]
    grad = [dict(lse=None), dict(lse=null), dict(g=P(0)), dict(g=P(18)), dict(dX=None, dW=None),
            dict(dX=bad), dict(dW=bad), dict(dX=null), dict(dW=null), dict(od=5)]
    for call, own in ((_xent, xent + fwd), (_xent_grad, xent + grad), (_distill, teach + fwd),
                      (_distill_grad, teach + grad)):
        for k in every + opts + own:
            assert call(fcc, **k) == fcc.FCC_ERR_INVALID, (call.__name__, k)
        # valid, but not built: other input types, other forms; f16 or f32 gradients
        for k in [dict(dt=fcc.FCC_F16), dict(dt=fcc.FCC_F32),
                  *(dict(o=ctypes.byref(fcc.make_opts(algo=a)))
                    for a in (fcc.FCC_ALGO_UNFUSED, fcc.FCC_ALGO_INTERDECOM, fcc.FCC_ALGO_CE))]:
            assert call(fcc, **k) == fcc.FCC_ERR_UNSUPPORTED, (call.__name__, k)
    for call in (_xent_grad, _distill_grad):
        for od in (fcc.FCC_F16, fcc.FCC_F32):
            assert call(fcc, od=od) == fcc.FCC_ERR_UNSUPPORTED
    with pytest.raises(fcc.FccError):
        fcc.fcc_linear_xent(1, [16], [16], 16, 0, 8, 8, [16], [16])


def test_workspace_sizes(fcc):
    size = fcc.fcc_linear_loss_workspace_size
    assert size(0, 4, 8, 8) == 0 and size(9, 4, 8, 8) == 0 and size(1, 0, 8, 8) == 0
    assert size(1, 4, 8, 8, 257) == 0
    # forward: far less than the logits; backward: at least a piece of dl and dX's f32 sums
    T, V, D = 4096, 131072, 4096
    assert 0 < size(8, T, V, D) < T * V * 2 // 16
    g = size(8, T, V, D, grad=True)
    # and blocks for shared dX tiles (at most two of 128 KiB per SM)
    assert 2 * T * D <= g <= (512 << 20) + 4 * T * D + (2 * 256 * 128 << 10) + (1 << 20)
    # the caller's pieces
    more = size(8, T, V, D, grad=True, opts=fcc.make_opts(chunks=16))
    assert more < g
    assert size(1, 1, 1, 8, 1, True) > 0
