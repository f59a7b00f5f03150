"""The paged cache on the GPU against the fp64 oracle.

Tolerances of the attention's outputs, derived here and used throughout:
 * a score is a sum of d products in f32: off by at most e_s = 2^-16 scale sum|q k|
   (128 additions that may each cut off up to 2^-23 of the sum of magnitudes), and its
   exponential by e = e_s + 2^-17 relatively (the exponent's own rounding, 2^-24 of
   at most 64, and the exponential instruction);
 * the probabilities enter the product in 16 bits: 2^-8 of each (bf16), so an output
   is off by (2^-8 + 2 e) sum softmax |v|, and its own rounding by 2^-8 of itself;
   second-order terms are below a hundredth of that, 1.02 covers them;
 * e4m3 with few rows: probabilities below 2^-38 of the largest become zero, which
   2^-8 of the sum covers for any length;
 * lse: e, and the sum's additions, at most one rounding of 2^-24 for each position.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_collective_gb300 as fcc  # noqa: E402
from tests.gpu_util import bits, to_f64  # noqa: E402


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype).cuda()


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda().bfloat16()


class Step:
    """Sequences (n new rows, L positions each) over a paged cache that holds seeded values."""

    def __init__(self, seqs, H=2, d=128, P=16, dtype="bf16", R=1, seed=0, lead=0, behind=0, spare=3, scale_v=1.0):
        g = self.g = np.random.default_rng(seed)
        self.seqs, self.H, self.d, self.P, self.R, self.e4m3 = seqs, H, d, P, R, dtype == "e4m3"
        n = [a for a, _ in seqs]
        self.start_np = lead + np.concatenate([[0], np.cumsum(n)])
        self.T = int(self.start_np[-1]) + behind
        own = [max(0, -(-L // P)) for _, L in seqs]
        self.max_pages = max(1, max(own)) + 1
        self.pages = sum(own) + spare
        perm = g.permutation(self.pages)
        self.table_np = np.full((len(seqs), self.max_pages), -1)
        at = 0
        for b, k in enumerate(own):
            self.table_np[b, :k] = perm[at:at + k]
            at += k
        self.start, self.len, self.table = dev(self.start_np), dev([L for _, L in seqs]), dev(self.table_np)
        shape = (R, self.pages, H, P, d)
        x = [g.standard_normal(shape, dtype=np.float32), g.standard_normal(shape, dtype=np.float32) * scale_v]
        self.exps = [None, None]
        if self.e4m3:
            self.codes, self.exps = map(list, zip(*[oc.quantise(v) for v in x]))
            for v, e in zip(x, self.exps):  # (a power of its own for each row, some far from the others)
                e[:] = np.clip(e.astype(int) + g.integers(-3, 4, e.shape), 1, 254)
            self.vals = [oc.values(c, e) for c, e in zip(self.codes, self.exps)]
        else:
            self.pools = [torch.from_numpy(v).bfloat16() for v in x]
            self.vals = [p.double().numpy() for p in self.pools]
        self.spoil = np.ones((self.pages, P), bool)  # rows that no sequence has
        for b, (_, L) in enumerate(seqs):
            for j in range(L):
                self.spoil[self.table_np[b, j // P], j % P] = False
        self.upload()

    def upload(self):
        """What no sequence owns holds NaN."""
        self.dev = []
        for i in range(2):
            if self.e4m3:
                c, e = self.codes[i].copy(), self.exps[i].copy()
                c.transpose(0, 1, 3, 2, 4)[:, self.spoil] = 0x7F
                self.dev.append([torch.from_numpy(c[r]).cuda() for r in range(self.R)])
                self.dev.append([torch.from_numpy(e[r]).cuda() for r in range(self.R)])
            else:
                p = self.pools[i].clone()
                p.permute(0, 1, 3, 2, 4)[:, torch.from_numpy(self.spoil)] = float("nan")
                self.dev += [[p[r].cuda() for r in range(self.R)], None]
        self.K, self.Ke, self.V, self.Ve = self.dev

    def cache(self):
        return fcc.make_cache(self.K, self.V, self.pages, self.P, self.H, self.d, fcc.FCC_E4M3 if self.e4m3 else fcc.FCC_BF16,
                              self.Ke, self.Ve)

    def batch(self, T=None):
        return fcc.make_batch(self.start, self.len, self.table, T or self.T, len(self.seqs), self.max_pages)

    def held(self, which, r, b, first, last):
        return oc.rows_of(self.vals[which][r], self.table_np[b], first, last)


def attend(s, G, Q, scale=0.0, window=0, opts=None, lse=True, ldo=0, stream=None):
    Hq = s.H * G
    O = [torch.full((s.T, ldo // s.d if ldo else Hq, s.d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(s.R)]
    z = [torch.full((s.T, Hq), 7.0, device="cuda") for _ in range(s.R)] if lse else None
    fcc.fcc_paged_attention(s.R, Q, s.cache(), s.batch(), Hq, O, z, scale=scale, window=window, opts=opts, ldo=ldo,
                            ldq=Q[0].stride(0), stream=stream)
    return O, z


def check(s, G, Q, O, lse, scale, window=0, spread=1.0):
    """Every sequence's rows against the oracle, and all other rows untouched."""
    Hq = s.H * G
    for r in range(s.R):
        o, q = to_f64(O[r]), to_f64(Q[r])
        z = lse[r].double().cpu().numpy() if lse is not None else None
        covered = np.zeros(s.T, bool)
        for b, (n, L) in enumerate(s.seqs):
            rows = slice(int(s.start_np[b]), int(s.start_np[b]) + n)
            covered[rows] = True
            if n == 0:
                continue
            lo = max(0, L - n - window + 1) if window else 0
            keys, vals = np.full((max(L, 0), s.H, s.d), np.nan), np.full((max(L, 0), s.H, s.d), np.nan)
            if L >= n:
                keys[lo:], vals[lo:] = s.held(0, r, b, lo, L), s.held(1, r, b, lo, L)
            ref, zr, A = oc.attention(q[rows], keys, vals, L, scale, window)
            e_s = 2.0 ** -16 * scale * (np.abs(q[rows]).max(axis=(1, 2)) * np.nanmax(np.abs(keys).sum(-1), initial=0.0))[:, None]
            e = e_s + 2.0 ** -17
            tol = 1.02 * (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * A) * spread
            got = o[rows]
            assert np.isfinite(got).all(), (r, b)
            bad = np.abs(got - ref) > tol
            assert not bad.any(), (r, b, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], bad.mean())
            if z is not None:
                none = np.isneginf(zr)
                assert np.array_equal(np.isneginf(z[rows]), none), (r, b)
                dz = np.abs(np.where(none, 0, z[rows]) - np.where(none, 0, zr))
                tz = e + L * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(none, 0, zr))
                assert (dz <= tz).all(), (r, b, (dz - tz).max(), dz.max())
        assert (o[~covered] == 7).all()
        if z is not None:
            assert (z[~covered] == 7).all()


def queries(s, G, seed=1, amp=1.0, ldq=0):
    g = np.random.default_rng(seed)
    Hq = s.H * G
    wide = ldq // s.d if ldq else Hq
    return [bf16(g.standard_normal((s.T, wide, s.d)) * amp)[:, :Hq] for _ in range(s.R)]


ONE = [[(1, 1)], [(1, 2), (1, 16), (1, 17), (1, 129), (1, 300)], [(1, 1000)], [(1, 40)] * 7 + [(0, 90), (0, 0), (1, 700)]]
MANY = [[(2, 2)], [(5, 37), (1, 9), (3, 260)], [(33, 33)], [(130, 400), (1, 77), (0, 5), (17, 17)], [(300, 300)]]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,P", [(128, 16), (64, 32), (128, 1), (64, 128)])
@pytest.mark.parametrize("seqs", range(len(ONE) + len(MANY)))
def test_attention(dtype, d, P, seqs):
    case = (ONE + MANY)[seqs]
    for H, G, R in [(2, 4, 1), (1, 7, 2), (3, 1, 1), (1, 16, 1)]:
        s = Step(case, H=H, d=d, P=P, dtype=dtype, R=R, seed=seqs, lead=seqs % 3, behind=2)
        Q = queries(s, G, amp=1.5)
        O, lse = attend(s, G, Q)
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        check(s, G, Q, O, lse, 1 / np.sqrt(d))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8])
def test_ragged_steps_in_every_form(dtype, G):
    """6.25 rows to a sequence for each head of a group: by items of 8 and of 16 rows, and by tiles of 128, each
    with a sequence of many rows among ones of few."""
    s = Step([(1, 300), (21, 400), (1, 1), (2, 130)], H=2, dtype=dtype, seed=G, lead=1)
    Q = queries(s, G)
    for window in (0, 77):
        O, lse = attend(s, G, Q, window=window)
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        check(s, G, Q, O, lse, 1 / np.sqrt(128), window)
        again, z = attend(s, G, Q, window=window)
        assert torch.equal(O[0], again[0]) and torch.equal(lse[0], z[0])  # a fixed order of summation


@pytest.mark.parametrize("B,n,G", [(700, 1, 2), (1100, 3, 12)])
def test_many_sequences(B, n, G):
    """More sequences than a block of threads counts one by one, some without rows."""
    seqs = [(0 if b % 7 == 3 else n, n + b % 23) for b in range(B)]
    s = Step(seqs, H=1, d=64, P=8, dtype="bf16", seed=1)
    Q = queries(s, G)
    O, lse = attend(s, G, Q)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    check(s, G, Q, O, lse, 1 / 8)


@pytest.mark.parametrize("case,G", [([(1, 200), (1, 70)], 4), ([(9, 200)], 3), ([(150, 300), (40, 40)], 2)])
@pytest.mark.parametrize("step", [10, 16, 40])
def test_powers_of_neighbours_far_apart(case, G, step):
    """e4m3 rows whose powers of two differ by 2^step from one position to the next: the small ones keep their digits."""
    s = Step(case, H=2, dtype="e4m3", seed=step)
    for which in (0, 1):
        e = s.exps[which].astype(int)
        e[:, :, :, 1::3] -= step
        e[:, :, :, 2::3] = 63  # 2^-64, the least that append writes
        s.exps[which] = np.clip(e, 63, 247).astype(np.uint8)
        s.vals[which] = oc.values(s.codes[which], s.exps[which])
    s.upload()
    Q = queries(s, G, amp=3.0)
    O, lse = attend(s, G, Q, window=2)  # (few positions to a row: some rows see only small ones)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    check(s, G, Q, O, lse, 1 / np.sqrt(128), 2)
    O, lse = attend(s, G, Q)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    check(s, G, Q, O, lse, 1 / np.sqrt(128))


def test_eight_ranks():
    s = Step([(1, 150), (3, 40)], H=1, d=64, P=4, dtype="e4m3", R=8)
    for G in (2, 30):
        Q = queries(s, G)
        O, lse = attend(s, G, Q)
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        check(s, G, Q, O, lse, 1 / 8)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 100, 128, 129, 1000000])
def test_window(dtype, window):
    for case, G in [([(1, 300), (1, 17), (1, 1)], 4), ([(40, 300), (1, 290), (140, 140)], 3)]:
        s = Step(case, dtype=dtype, seed=window % 97)
        Q = queries(s, G)
        O, lse = attend(s, G, Q, window=window, scale=0.2)
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        check(s, G, Q, O, lse, 0.2, window)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("case,G", [([(1, 2000), (1, 5)], 8), ([(200, 900)], 4)])
def test_sharp_and_rising_scores(dtype, case, G):
    """Scores of hundreds, and a maximum that grows from position to position."""
    s = Step(case, H=1, dtype=dtype, seed=3)
    ramp = np.linspace(0.01, 3, s.P * s.pages).reshape(s.pages, 1, s.P, 1)
    order = np.argsort(s.table_np[0, :-(-case[0][1] // s.P)])
    inv = np.arange(s.pages)
    inv[s.table_np[0, :len(order)]] = np.arange(len(order))
    if s.e4m3:
        s.codes[0], s.exps[0] = oc.quantise(np.abs(s.vals[0]) * ramp[inv][None])
        s.vals[0] = oc.values(s.codes[0], s.exps[0])
    else:
        s.pools[0] = torch.from_numpy(np.abs(s.vals[0]) * ramp[inv][None]).bfloat16()
        s.vals[0] = s.pools[0].double().numpy()
    s.upload()
    for sign in (1.0, -1.0):
        Q = [q.abs() * sign for q in queries(s, G, amp=2.0)]
        O, lse = attend(s, G, Q, scale=0.5)
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        check(s, G, Q, O, lse, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("case,G,window", [([(1, 300)], 4, 100), ([(6, 300)], 8, 100), ([(6, 300)], 2, 0), ([(150, 300)], 4, 0),
                                           ([(150, 300)], 4, 60)])
def test_unseen_positions_may_hold_anything(dtype, case, G, window):
    """Infinities and NaN in keys and values: rows that do not see the position are what they are without it."""
    s = Step(case, H=1, dtype=dtype, seed=5)
    Q = queries(s, G)
    n, L = case[0]
    clean, z0 = attend(s, G, Q, window=window)
    check(s, G, Q, clean, z0, 1 / np.sqrt(128), window)
    for j in [L - n // 2, L - n - 70]:
        page, row = s.table_np[0, j // s.P], j % s.P
        for which in (0, 1):
            bad = Step(case, H=1, dtype=dtype, seed=5)
            if bad.e4m3:
                bad.codes[which][0, page, 0, row] = 0x7F
            else:
                bad.pools[which][0, page, 0, row, ::3] = float("inf")
                bad.pools[which][0, page, 0, row, 1::3] = float("nan")
            bad.upload()
            O, z = attend(bad, G, Q, window=window)
            assert fcc.fcc_stream_status() == fcc.FCC_OK
            p = np.arange(L - n, L)
            sees = torch.from_numpy((p >= j) & ((p < j + window) if window else True)).cuda()
            assert not bool(O[0][sees].isfinite().all(dim=-1).any())
            assert bool(torch.equal(O[0][~sees].isnan(), torch.zeros_like(O[0][~sees], dtype=torch.bool)))
            got, want = to_f64(O[0][~sees]), to_f64(clean[0][~sees])
            assert np.abs(got - want).max(initial=0) <= 2.0 ** -6 * np.abs(want).max(initial=1), (j, which)
            assert torch.allclose(z[0][~sees], z0[0][~sees], rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("case,G", [([(1, 200), (1, 90)], 4), ([(70, 200), (3, 90)], 4)])
def test_rows_with_infinite_or_nan_queries_stay_alone(case, G):
    for dtype in ("bf16", "e4m3"):
        s = Step(case, dtype=dtype)
        Q = queries(s, G)
        O0, _ = attend(s, G, Q)
        Q2 = [Q[0].clone()]
        Q2[0][0, 1] = float("nan")
        Q2[0][0, 3, 5] = float("inf")
        O, _ = attend(s, G, Q2)
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        assert bool(O[0][0, 1].isnan().all())
        keep = torch.ones(s.T, s.H * G, dtype=torch.bool, device="cuda")
        keep[0, 1] = keep[0, 3] = False
        assert torch.equal(O[0][keep], O0[0][keep])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_sequences_that_are_not_valid(dtype):
    for G, more in [(4, 0), (4, 60)]:
        # the second sequence has fewer positions than rows, the third a page outside the pool, the fourth too few pages
        s = Step([(1 + more, 100), (2 + more, 1), (1 + more, 90), (1, 50)], dtype=dtype)
        Q = queries(s, G)
        s.table[2, 1] = s.pages
        O, lse = attend(s, G, Q)
        assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID and fcc.fcc_stream_status() == fcc.FCC_OK
        a = slice(int(s.start_np[1]), int(s.start_np[2]))
        assert bool((O[0][a] == 0).all()) and bool((lse[0][a] == -torch.inf).all())
        # the positions of the bad page are left out: what is left is finite
        assert bool(O[0].isfinite().all())
        keep = s.seqs
        s.seqs = [keep[0], (0, 0), (0, 0), keep[3]]
        o, z = [O[0].clone()], [lse[0].clone()]
        b = slice(int(s.start_np[1]), int(s.start_np[3]))
        o[0][b], z[0][b] = 7.0, 7.0
        check(s, G, Q, o, z, 1 / np.sqrt(128))
        s.seqs = keep
        # rows outside the token arrays: nothing of them is touched
        t = Step([(1 + more, 100), (2 + more, 60)], dtype=dtype)
        Q = queries(t, G)
        for start in ([0, 1 + more, t.T + 5], [0, 5 + more, 2], [-3, 1 + more, t.T]):
            t.start = dev(start)
            attend(t, G, Q)
            assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID, start
        # a table that is narrower than the positions need
        t = Step([(1 + more, 100)], dtype=dtype)
        Q = queries(t, G)
        t.table, t.max_pages = t.table[:, :4].contiguous(), 4
        O, lse = attend(t, G, Q)
        assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID
        assert bool(O[0].isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("more", [0, 3, 60])
def test_lengths_far_past_the_table(dtype, more):
    """All that the table's pages hold is seen (no time is spent on the rest), with a window nothing."""
    for window in (0, 100):
        s = Step([(1 + more, 80), (2 + more, 160), (1 + more, 70)], dtype=dtype, P=16)
        s.table, s.max_pages = s.table[:, :10].contiguous(), 10   # the second sequence's 160 positions, exactly
        s.len = dev([80, 2**31 - 1, 70])
        Q = queries(s, 4)
        O, lse = attend(s, 4, Q, window=window)
        assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID and fcc.fcc_stream_status() == fcc.FCC_OK
        a, b = int(s.start_np[1]), int(s.start_np[2])
        if window:
            assert bool((O[0][a:b] == 0).all()) and bool((lse[0][a:b] == -torch.inf).all())
            O[0][a:b], lse[0][a:b] = 7.0, 7.0
            s.seqs[1] = (0, 0)
        else:                                             # each of its rows is the newest of 160 positions
            s.seqs = [s.seqs[0]] + [(1, 160)] * (b - a) + [s.seqs[2]]
            s.start_np = np.concatenate([[0], np.arange(a, b + 1), [s.T]])
            s.table_np = s.table_np[[0] + [1] * (b - a) + [2]]
        check(s, 4, Q, O, lse, 128 ** -0.5, window)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("case,G", [([(1, 300), (1, 50)], 4), ([(100, 300), (1, 50)], 4)])
def test_strides_streams_lse_and_repeats(dtype, case, G):
    s = Step(case, dtype=dtype, R=2, behind=3)
    Hq = s.H * G
    Q = queries(s, G, ldq=(Hq + 5) * s.d)
    assert Q[0].stride(0) == (Hq + 5) * s.d
    O, lse = attend(s, G, Q, ldo=(Hq + 2) * s.d)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    assert all(bool((o[:, Hq:] == 7).all()) for o in O)
    check(s, G, Q, [o[:, :Hq] for o in O], lse, 1 / np.sqrt(128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = fcc.fcc_paged_attention_workspace_size(s.R, s.T, len(case), Hq, s.H, s.d)
    for size in (n, n + 1000):
        ws = torch.full((max(size, 16) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            O2, none = attend(s, G, [q.contiguous() for q in Q], lse=False, stream=side,
                              opts=fcc.make_opts(workspace=ws, workspace_bytes=size))
        assert fcc.fcc_stream_status(side) == fcc.FCC_OK and none is None
        assert bool((ws[max(size, 16):] == 0xFF).all())
        assert all(torch.equal(a[:, :Hq], b) for a, b in zip(O, O2))
    if n:
        with pytest.raises(fcc.FccError) as e:
            attend(s, G, Q, opts=fcc.make_opts(workspace=ws, workspace_bytes=n - 1))
        assert e.value.status == fcc.FCC_ERR_WORKSPACE
    torch.cuda.synchronize()


@pytest.mark.parametrize("ctas", [1, 3, 40])
def test_any_number_of_ctas(ctas):
    for case, G in [([(1, 3000), (1, 1), (1, 700)], 4), ([(60, 900), (1, 30)], 4)]:
        for dtype in ("bf16", "e4m3"):
            s = Step(case, dtype=dtype, seed=ctas)
            Q = queries(s, G)
            O, lse = attend(s, G, Q, opts=fcc.make_opts(max_ctas=ctas))
            assert fcc.fcc_stream_status() == fcc.FCC_OK
            check(s, G, Q, O, lse, 1 / np.sqrt(128))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,P", [(128, 16), (64, 1), (128, 64), (64, 16)])
@pytest.mark.parametrize("H", [1, 3, 8])
def test_append_and_gather(dtype, d, P, H):
    g = np.random.default_rng(H)
    s = Step([(1, 1), (0, 20), (37, 50), (5, 5), (1, 200)], H=H, d=d, P=P, dtype=dtype, R=2, lead=2, behind=1)
    before = [[x.clone() for x in xs] if xs else None for xs in s.dev]
    x = g.standard_normal((2, 2, s.T, H, d)) * np.exp2(g.integers(-30, 20, (2, 2, s.T, H, 1)))
    x[0, 0, 3] = 0
    x[1, 1, 4, 0, :] = 2.0 ** -70  # below what the least power keeps apart
    x[0, 1, 6, 0, 0] = 448 * 2.0 ** 9
    wide = torch.zeros(2, s.T, 3 * H * d + 8, device="cuda", dtype=torch.bfloat16)  # part of a fused projection
    ld = wide.shape[2]
    for r in range(2):
        wide[r, :, H * d:3 * H * d] = bf16(x[:, r].transpose(1, 0, 2, 3).reshape(s.T, 2 * H * d))
    k, v = [wide[r, :, H * d:] for r in range(2)], [wide[r, :, 2 * H * d:] for r in range(2)]
    fcc.fcc_cache_append(2, k, v, s.cache(), s.batch(), ld=ld)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    back = [[torch.full((s.T, H, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)] for _ in range(2)]
    fcc.fcc_cache_gather(2, s.cache(), s.batch(), *back)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    touched = np.zeros((s.pages, P), bool)
    owner = np.zeros(s.T, bool)
    for b, (n, L) in enumerate(s.seqs):
        for i in range(n):
            j, t = L - n + i, int(s.start_np[b]) + i
            owner[t] = True
            page, row = s.table_np[b, j // P], j % P
            touched[page, row] = True
            for r in range(2):
                for which, src in ((0, k), (1, v)):
                    new = to_f64(src[r][t, :H * d]).reshape(H, d)
                    pool, exps = s.dev[2 * which][r], s.dev[2 * which + 1]
                    if s.e4m3:
                        codes, power = oc.quantise(new)
                        got = pool[page, :, row].cpu().numpy()
                        # (a negative number that becomes zero may keep its sign)
                        assert np.array_equal(oc.values(got, power), oc.values(codes, power)), (b, i)
                        assert np.array_equal(exps[r][page, :, row].cpu().numpy(), power)
                        new = oc.values(codes, power)
                    else:
                        assert np.array_equal(to_f64(pool[page, :, row]), new)
                    assert np.array_equal(to_f64(back[which][r][t]), new), (b, i)
    for a, c in zip(before, s.dev):  # every other place is what it was
        for r in range(2) if a else ():
            same = (bits(a[r]) == bits(c[r]))
            same = same.transpose(0, 2, 1, 3).all(axis=(2, 3)) if same.ndim == 4 else same.transpose(0, 2, 1).all(axis=2)
            assert same[~touched].all()
    for which in range(2):
        assert all(bool((x[torch.from_numpy(~owner).cuda()] == 7).all()) for x in back[which])


def test_rows_of_sequences_far_apart_in_the_list():
    """Neighbouring rows with many sequences without rows between them, and rows that begin in the middle of a group."""
    seqs = [(2, 5)] + [(0, 7)] * 70 + [(3, 9)] + [(0, 0)] * 40 + [(1, 1)] * 33 + [(25, 31)]
    s = Step(seqs, H=3, d=64, P=4, dtype="bf16", lead=3, behind=9)
    x = torch.randn(2, s.T, 3, 64, device="cuda").bfloat16()
    fcc.fcc_cache_append(1, [x[0]], [x[1]], s.cache(), s.batch())
    out = torch.full_like(x, 7.0)
    fcc.fcc_cache_gather(1, s.cache(), s.batch(), [out[0]], [out[1]])
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    assert torch.equal(out[:, 3:-9], x[:, 3:-9]) and bool((out[:, :3] == 7).all()) and bool((out[:, -9:] == 7).all())
    for b in (0, 71, 112, 144, 145):
        n, L = seqs[b]
        for which, pool in ((0, s.K[0]), (1, s.V[0])):
            got = oc.rows_of(to_f64(pool), s.table_np[b], L - n, L)
            assert np.array_equal(got, to_f64(x[which, int(s.start_np[b]):int(s.start_np[b]) + n])), b


def test_append_of_numbers_that_are_not_finite():
    s = Step([(2, 20)], H=2, dtype="e4m3")
    x = torch.ones(2, 2, 128, device="cuda", dtype=torch.bfloat16)
    x[0, 0, :3] = torch.tensor([float("inf"), float("nan"), -float("inf")], device="cuda")
    fcc.fcc_cache_append(1, [x], [x], s.cache(), s.batch())
    out = [torch.empty_like(x) for _ in range(2)]
    fcc.fcc_cache_gather(1, s.cache(), s.batch(), [out[0]], [out[1]])
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    for o in out:
        assert bool(o[0, 0, :3].isnan().all()) and bool((o[0, 0, 3:] == 1).all()) and bool((o[0, 1] == 1).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_and_gather_with_bad_sequences(dtype):
    s = Step([(2, 30), (3, 2), (1, 40), (1, 9)], dtype=dtype)
    s.table[2, 2] = -5
    before = [[x.clone() for x in xs] if xs else None for xs in s.dev]
    x = torch.ones(s.T, 2, 128, device="cuda", dtype=torch.bfloat16)
    out = [torch.full_like(x, 7.0) for _ in range(2)]
    for call in (lambda: fcc.fcc_cache_append(1, [x], [x], s.cache(), s.batch()),
                 lambda: fcc.fcc_cache_gather(1, s.cache(), s.batch(), [out[0]], [out[1]])):
        call()
        assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID and fcc.fcc_stream_status() == fcc.FCC_OK
    for o in out:
        assert bool((o[:2] == 1).all()) and bool((o[2:6] == 7).all()) and bool((o[6:] == 1).all())
    changed = [int((bits(a[0]) != bits(c[0])).any(axis=-1).sum()) for a, c in zip(before[::2], s.dev[::2])]
    assert all(0 < c <= 6 for c in changed)  # three rows of two heads
    for start in ([0, 2, 1, 6, 90], [0, 2, 5, 6, 8], [-1, 2, 5, 6, 7]):
        s.start = dev(start)
        fcc.fcc_cache_append(1, [x], [x], s.cache(), s.batch())
        assert fcc.fcc_stream_status() == fcc.FCC_ERR_INVALID


def test_places_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 values, used at its end."""
    P, H, d, pages = 64, 8, 128, 1 << 15  # 2^31 values
    for dtype in (torch.bfloat16, torch.uint8):
        e4m3 = dtype == torch.uint8
        K, V = (torch.empty(pages + 40, H, P, d, dtype=dtype, device="cuda") for _ in range(2))
        exps = [torch.empty(pages + 40, H, P, dtype=torch.uint8, device="cuda") for _ in range(2)] if e4m3 else [None, None]
        cache = fcc.make_cache([K], [V], pages + 40, P, H, d, fcc.FCC_E4M3 if e4m3 else fcc.FCC_BF16,
                               [exps[0]] if e4m3 else None, [exps[1]] if e4m3 else None)
        for n in (300, 1):
            table = dev([[pages + 39, 3, pages + 38, pages // 2 + 1, pages]])
            start, L = dev([0, n]), dev([300])
            x = torch.randn(2, 300, H, d, device="cuda").bfloat16()
            fcc.fcc_cache_append(1, [x[0]], [x[1]], cache, fcc.make_batch(dev([0, 300]), L, table, 300, 1, 5))
            out = torch.empty_like(x)
            fcc.fcc_cache_gather(1, cache, fcc.make_batch(dev([0, 300]), L, table, 300, 1, 5), [out[0]], [out[1]])
            if not e4m3:
                assert torch.equal(out, x)
            q = torch.randn(n, 2 * H, d, device="cuda").bfloat16()
            O = torch.empty_like(q)
            fcc.fcc_paged_attention(1, [q], cache, fcc.make_batch(start, L, table, n, 1, 5), 2 * H, [O])
            assert fcc.fcc_stream_status() == fcc.FCC_OK
            ref, _, A = oc.attention(to_f64(q), to_f64(out[0]), to_f64(out[1]), 300, 1 / np.sqrt(d))
            # e = 2^-16 scale sum|q k| + 2^-17 is below 2^-10 here (|q|, |k| < 5.5 over 128 products, scale 1/11.3)
            assert (np.abs(to_f64(O) - ref) <= 1.02 * (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -6) * A)).all()
        del K, V, exps, cache


def test_replayed_graphs_read_the_step_anew():
    """Two graphs with a workspace each; lengths, tables and contents change between replays."""
    G, cases = 4, [[(1, 700), (1, 30)], [(1, 40), (1, 333)], [(1, 2), (1, 1)]]
    steps = [Step(c, dtype="bf16", seed=i, spare=80 - sum(-(-L // 16) for _, L in c)) for i, c in enumerate(cases)]
    assert len({s.pages for s in steps}) == 1
    live = Step(cases[0], dtype="bf16", spare=steps[0].pages - sum(-(-L // 16) for _, L in cases[0]))
    wide = max(s.max_pages for s in steps)
    table = torch.zeros((2, wide), dtype=torch.int32, device="cuda")
    live.table, live.max_pages = table, wide
    length = live.len
    Q = queries(live, G)[0].clone()
    n = fcc.fcc_paged_attention_workspace_size(1, live.T, 2, 8, 2, 128)
    graphs = []
    side = torch.cuda.Stream()
    for _ in range(2):
        ws, O, z = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), torch.zeros_like(Q), torch.zeros(2, 8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        cache, batch, o = live.cache(), live.batch(), fcc.make_opts(workspace=ws, workspace_bytes=max(n, 16))
        fcc.fcc_paged_attention(1, [Q], cache, batch, 8, [O], [z], opts=o)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            fcc.fcc_paged_attention(1, [Q], cache, batch, 8, [O], [z], opts=o, stream=torch.cuda.current_stream())
        graphs.append((graph, ws, O, z))
    for i in (1, 2, 0, 1):
        s = steps[i]
        length.copy_(dev([L for _, L in s.seqs]))
        table.fill_(-1)
        table[:, :s.table_np.shape[1]] = dev(s.table_np)
        live.K[0].copy_(s.K[0]), live.V[0].copy_(s.V[0])
        Q.copy_(queries(s, G, seed=50 + i)[0])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for st, (graph, _, _, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        for _, _, O, z in graphs:
            check(s, G, [Q], [O], [z], 1 / np.sqrt(128))
        assert torch.equal(graphs[0][2], graphs[1][2])


def test_a_captured_call_brings_its_workspace():
    s = Step([(1, 100)])
    Q = queries(s, 4)
    O = torch.zeros_like(Q[0])
    cache, batch = s.cache(), s.batch()
    fcc.fcc_paged_attention(1, Q, cache, batch, 8, [O])
    if not fcc.fcc_paged_attention_workspace_size(1, s.T, 1, 8, 2, 128):
        pytest.skip("no workspace")
    torch.cuda.synchronize()
    graph, seen = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        try:
            fcc.fcc_paged_attention(1, Q, cache, batch, 8, [O], stream=torch.cuda.current_stream())
        except fcc.FccError as e:
            seen.append(e.status)
        O.zero_()
    assert seen == [fcc.FCC_ERR_WORKSPACE]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_decode_step_of_two_ranks(dtype):
    """Append, attention and the output projection, as a serving loop runs them, for a prompt and then token by token."""
    R, H, G, d, P, B, N = 2, 2, 3, 64, 16, 3, 256
    Hq = H * G
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()

    e4m3 = dtype == "e4m3"
    pages, wide = 40, 12
    K, V = ([torch.zeros(pages, H, P, d, device="cuda", dtype=torch.uint8 if e4m3 else torch.bfloat16) for _ in range(R)] for _ in range(2))
    exps = [[torch.zeros(pages, H, P, device="cuda", dtype=torch.uint8) for _ in range(R)] if e4m3 else None for _ in range(2)]
    cache = fcc.make_cache(K, V, pages, P, H, d, fcc.FCC_E4M3 if e4m3 else fcc.FCC_BF16, *exps)
    table_np = np.random.default_rng(0).permutation(pages)[:B * wide].reshape(B, wide)
    table = dev(table_np)
    W = [rand(Hq * d, N) for _ in range(R)]
    lens = np.array([70, 1, 33])
    steps = [lens.copy()] + [np.ones(B, int)] * 4
    total = np.zeros(B, int)
    history = [[[[] for _ in range(B)] for _ in range(R)] for _ in range(2)]
    for n in steps:
        total = total + n
        T = int(n.sum())
        start = np.concatenate([[0], np.cumsum(n)])
        batch = fcc.make_batch(s0 := dev(start), l0 := dev(total), table, T, B, wide)
        qkv = [rand(T, Hq + 2 * H, d) for _ in range(R)]
        ld = (Hq + 2 * H) * d
        k, v = [x[:, Hq:] for x in qkv], [x[:, Hq + H:] for x in qkv]
        O = [torch.empty(T, Hq, d, device="cuda", dtype=torch.bfloat16) for _ in range(R)]
        y = [torch.empty(T, N, device="cuda") for _ in range(R)]
        fcc.fcc_cache_append(R, k, v, cache, batch, ld=ld)
        fcc.fcc_paged_attention(R, qkv, cache, batch, Hq, O, ldq=ld)
        project = fcc.fcc_gemv_ar if T <= 16 else fcc.fcc_gemm_ar
        project(R, O, W, y, T, N, Hq * d, fcc.FCC_BF16, fcc.FCC_F32)
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        want = np.zeros((T, N))
        slack = np.zeros((T, N))
        for r in range(R):
            ref, A = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
            for b in range(B):
                rows = slice(start[b], start[b + 1])
                for which, x in ((0, k), (1, v)):
                    new = to_f64(x[r][rows, :H])
                    history[which][r][b].append(oc.values(*oc.quantise(new)) if e4m3 else new)
                ref[rows], _, A[rows] = oc.attention(to_f64(qkv[r][rows, :Hq]), np.concatenate(history[0][r][b]),
                                                     np.concatenate(history[1][r][b]), int(total[b]), 1 / np.sqrt(d))
            w = to_f64(W[r])
            want += ref.reshape(T, -1) @ w
            # (scores: |q|, |k| < 5 over 64 products, scale 1/8: e < 2^-8.6 / 2^16 * ... < 2^-10)
            slack += (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * A).reshape(T, -1) @ np.abs(w)
        for r in range(R):
            assert (np.abs(to_f64(y[r]) - want) <= 1.02 * slack + 1e-4 * slack.max()).all()
        del s0, l0
