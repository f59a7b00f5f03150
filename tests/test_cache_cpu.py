"""CPU checks of the paged cache: the fp64 oracle against torch's own conversions
and a dense softmax, and the entry points' refusals and sizes."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as oc


@pytest.fixture(scope="module")
def fcc():
    import __graft_entry__
    __graft_entry__.build()
    import gemm_collective_gb300 as m
    return m


def test_oracle_codes_are_e4m3():
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oc.e4m3_values(), ref, equal_nan=True)
    # every value between two codes' middles, and every middle itself (ties)
    pos = oc.e4m3_values()[:127]
    mid = (pos[:-1] + pos[1:]) / 2
    x = np.concatenate([pos, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e3)])
    x = np.concatenate([x, -x])
    rows = np.stack([x, np.full_like(x, 448)], 1)  # (the second value fixes the power at 2^0)
    codes, power = oc.quantise(rows)
    assert (power == 127).all()
    f32 = torch.from_numpy(x)  # (float64 to e4m3 rounds once)
    want = f32.to(torch.float8_e4m3fn).double().numpy()
    via32 = f32.float().double().numpy() == x
    assert np.array_equal(oc.values(codes, power)[via32, 0], want[via32])


def test_oracle_powers():
    for a, k in [(448.0, 0), (449.0, 1), (224.0, -1), (0.0, -64), (2.0 ** -80, -64), (1.75, -8), (1.76, -7),
                 (3.0e38, 120)]:
        codes, power = oc.quantise(np.array([[a, 0.0]]))
        assert power[0] == k + 127, (a, power)
    codes, power = oc.quantise(np.array([[np.inf, 1.0, np.nan, -2.0]]))
    v = oc.values(codes, power)[0]
    assert power[0] == 127 - 7 and np.isnan(v[0]) and np.isnan(v[2]) and v[1] == 1 and v[3] == -2


def test_oracle_attention_is_a_masked_softmax():
    g = np.random.default_rng(0)
    n, L, H, G, d = 5, 23, 2, 3, 8
    Q, K, V = g.standard_normal((n, H * G, d)), g.standard_normal((L, H, d)), g.standard_normal((L, H, d))
    for window in (0, 1, 4, 100):
        O, lse, A = oc.attention(Q, K, V, L, 0.3, window)
        s = 0.3 * np.einsum("ihd,jhd->ihj", Q, np.repeat(K, G, 1))
        p, j = np.arange(L - n, L)[:, None], np.arange(L)[None]
        seen = (j <= p) & ((j > p - window) if window else True)
        s = np.where(seen[:, None], s, -np.inf)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        assert np.allclose(O, np.einsum("ihj,jhd->ihd", w, np.repeat(V, G, 1)))
        assert np.allclose(A, np.einsum("ihj,jhd->ihd", w, np.abs(np.repeat(V, G, 1))))
        assert np.allclose(lse, np.log(np.exp(s).sum(-1)))
    # what no row sees may hold anything
    K2, V2 = K.copy(), V.copy()
    K2[:L - n - 3] = np.nan
    V2[:L - n - 3] = np.inf
    assert np.array_equal(oc.attention(Q, K2, V2, L, 0.3, 4)[0], oc.attention(Q, K, V, L, 0.3, 4)[0])
    O, lse, _ = oc.attention(Q, K, V, n - 1, 0.3)
    assert (O == 0).all() and (lse == -np.inf).all()


def test_oracle_pages():
    g = np.random.default_rng(1)
    pool = g.standard_normal((5, 2, 4, 3))
    rows = oc.rows_of(pool, np.array([3, 0, 4]), 2, 9)
    assert rows.shape == (7, 2, 3)
    assert np.array_equal(rows[0], pool[3, :, 2]) and np.array_equal(rows[6], pool[4, :, 0])


P, F = ctypes.c_void_p, ctypes.c_float
I64 = ctypes.c_int64


def _arr(*a):
    return (P * len(a))(*a)


def _cache(f, **k):
    two = [16, 32]
    a = dict(K=two, V=two, pages=9, page_size=16, H=2, d=128, dtype=f.FCC_BF16, K_exp=None, V_exp=None)
    a.update(k)
    return f.make_cache(a["K"], a["V"], a["pages"], a["page_size"], a["H"], a["d"], a["dtype"], a["K_exp"], a["V_exp"])


def _batch(f, **k):
    a = dict(start=16, len=16, table=16, T=4, B=3, max_pages=5)
    a.update(k)
    return f.make_batch(a["start"], a["len"], a["table"], a["T"], a["B"], a["max_pages"])


def _calls(f, R=2, cache=None, batch=None, o=None, x=None, y=None, ld=0, t=0, u=0, Hq=4, lse=None, scale=0.0, window=0,
           which=("append", "gather", "attention")):
    two = _arr(16, 32)
    c = ctypes.byref(cache if cache is not None else _cache(f))
    b = ctypes.byref(batch if batch is not None else _batch(f))
    x, y = (two if v is None else v for v in (x, y))
    out = []
    if "append" in which:
        out.append(f.raw_status("fcc_cache_append", R, x, y, I64(ld), c, b, t, o, None))
    if "gather" in which:
        out.append(f.raw_status("fcc_cache_gather", R, c, b, x, y, I64(ld), t, o, None))
    if "attention" in which:
        out.append(f.raw_status("fcc_paged_attention", R, x, I64(ld), c, b, Hq, y, I64(ld), lse, F(scale), I64(window), t, u,
                                o, None))
    return out


def test_refusals(fcc):
    bad, null = _arr(16, 33), _arr(16, 0)
    n0 = fcc.fcc_launch_count()

    def refused(want, **k):
        got = _calls(fcc, **k)
        assert got and all(g == want for g in got), (k, got)

    inv, uns = fcc.FCC_ERR_INVALID, fcc.FCC_ERR_UNSUPPORTED
    for R in (0, -1, 9):
        refused(inv, R=R)
    for v in (bad, null):
        refused(inv, x=v)
        refused(inv, y=v)
    for k in [dict(K=[16, 33]), dict(V=[0, 16]), dict(pages=0), dict(pages=1 << 31), dict(page_size=0), dict(page_size=24),
              dict(page_size=1 << 17), dict(H=0), dict(H=1025), dict(d=0), dict(dtype=7), dict(dtype=fcc.FCC_E4M3),
              dict(dtype=fcc.FCC_E4M3, K_exp=[16, 32]), dict(dtype=fcc.FCC_E4M3, K_exp=[16, 32], V_exp=[16, 24])]:
        refused(inv, cache=_cache(fcc, **k), Hq=k.get("H", 2) * 2)
    for k in [dict(start=0), dict(start=18), dict(len=0), dict(table=0), dict(table=33), dict(T=0), dict(T=1 << 31), dict(B=0),
              dict(B=65537), dict(max_pages=0), dict(max_pages=1 << 31)]:
        refused(inv, batch=_batch(fcc, **k))
    for ld in (-8, 128, 264 + 1, 1 << 31):
        refused(inv, ld=ld)
    refused(inv, ld=500, which=("append", "gather"))   # not a multiple of 8
    for t in (-1, 3, 7):
        refused(inv, t=t)
    for t in (fcc.FCC_F16, fcc.FCC_F32):
        refused(uns, t=t)
        refused(uns, u=t, which=("attention",))
    for d in (32, 96, 256):
        refused(uns, cache=_cache(fcc, d=d))
    for dt in (fcc.FCC_F16, fcc.FCC_F32):
        refused(uns, cache=_cache(fcc, dtype=dt))
    refused(uns, o=ctypes.byref(fcc.make_opts(algo=fcc.FCC_ALGO_UNFUSED)))
    for k in [dict(Hq=0), dict(Hq=3), dict(Hq=1026), dict(u=9), dict(scale=-1.0), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(window=-1), dict(lse=bad), dict(lse=null), dict(ld=300)]:
        refused(inv, which=("attention",), **k)
    two = _arr(16, 32)
    c, b = ctypes.byref(_cache(fcc)), ctypes.byref(_batch(fcc))
    assert fcc.raw_status("fcc_cache_append", 2, None, two, I64(0), c, b, 0, None, None) == inv
    assert fcc.raw_status("fcc_cache_append", 2, two, two, I64(0), None, b, 0, None, None) == inv
    assert fcc.raw_status("fcc_cache_gather", 2, c, None, two, two, I64(0), 0, None, None) == inv
    assert fcc.raw_status("fcc_paged_attention", 2, two, I64(0), c, b, 4, None, I64(0), None, F(0), I64(0), 0, 0, None, None) == inv
    assert fcc.fcc_launch_count() == n0
    with pytest.raises(fcc.FccError):  # a cache described for fewer ranks than the call's
        fcc.fcc_cache_append(3, [16] * 3, [16] * 3, _cache(fcc), _batch(fcc))


def test_scales_whose_exponents_overflow_are_refused(fcc):
    # scale * log2(e) is what a score is multiplied by; FLT_MAX / log2(e) is 2.3587e38
    for scale in (2.36e38, 3.4e38):
        assert _calls(fcc, scale=scale, which=("attention",)) == [fcc.FCC_ERR_INVALID]


def test_batches_of_other_types_and_sizes_are_refused(fcc):
    start, length, table = (torch.zeros(n, dtype=torch.int32) for n in (4, 3, 15))
    good = dict(start=start, len=length, table=table.view(3, 5))
    assert _batch(fcc, **good).table == table.data_ptr()
    _batch(fcc, start=torch.zeros(9, dtype=torch.int32), len=table[3:], table=torch.zeros(7, 5, dtype=torch.int32))  # larger ones
    _batch(fcc, **dict(good, table=table))
    for k in [dict(start=start.long()), dict(len=length.float()), dict(table=table.view(3, 5).long()),
              dict(start=start[:3]), dict(len=length[:2]), dict(table=table[:14]), dict(table=table[:10].view(2, 5)),
              dict(table=table.view(5, 3)), dict(table=torch.zeros(3, 8, dtype=torch.int32)[:, :5]),
              dict(table=table.view(5, 3).t()), dict(start=torch.zeros(8, dtype=torch.int32)[::2])]:
        with pytest.raises(fcc.FccError) as e:
            _batch(fcc, **dict(good, **k))
        assert e.value.status == fcc.FCC_ERR_INVALID, k
    one = torch.zeros(4, 8, dtype=torch.int32)
    fcc.make_batch(start, length, one[1:2, :5], 4, 1, 5)    # a single row of a wider table


def test_a_cache_counts_the_ranks_of_the_arrays_that_it_uses(fcc):
    two = [16, 32]
    assert fcc.make_cache(two, two, 9, 16, 2, 128, fcc.FCC_BF16, [16], []).ranks == 2
    assert fcc.make_cache(two, [16], 9, 16, 2, 128).ranks == 1
    assert fcc.make_cache(two, two, 9, 16, 2, 128, fcc.FCC_E4M3, two, [16]).ranks == 1
