"""The paged attention's tiles on contents that they cannot give by themselves: values that are not finite, and e4m3
rows whose powers of two are far apart.  Such rows are marked and computed again behind the tiles.

Tolerances: those of the attention (see test_gpu_cache.py), which hold for either way.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_collective_gb300 as fcc  # noqa: E402
from tests.gpu_util import to_f64  # noqa: E402
from tests.test_gpu_cache import Step, attend, check, dev, queries  # noqa: E402


def attend_again(s, G, Q, scale=0.0, window=0, **opts):
    """attend() in tiles with a workspace of its own; also whether rows were computed again (the plan's fourth word)."""
    n = fcc.fcc_paged_attention_workspace_size(s.R, s.T, len(s.seqs), s.H * G, s.H, s.d)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    O, z = attend(s, G, Q, scale, window, opts=fcc.make_opts(workspace=ws, workspace_bytes=n, **opts))
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    return O, z, int(ws[12:16].view(torch.int32))


def set_powers(s, which, e):
    s.exps[which] = np.clip(e, 63, 247).astype(np.uint8)
    s.vals[which] = oc.values(s.codes[which], s.exps[which])


def test_powers_far_apart_in_long_sequences_stay_within_the_wait_limit():
    """Each block of 20000 positions holds powers too far apart, and every CTA has several items: no warp of the tiles
    may wait for rows that take long (20 ms here; by one warp, a row of 20000 positions takes 16)."""
    s = Step([(40, 20000), (70, 300), (36, 6000)], H=2, d=64, dtype="e4m3", seed=11)
    for which in (0, 1):
        e = s.exps[which].astype(int)
        e[:, :, :, 3::16] -= 40
        set_powers(s, which, e)
    s.upload()
    Q = queries(s, 4)
    for ctas in (3, 0):
        O, lse, again = attend_again(s, 4, Q, max_ctas=ctas, timeout_ns=20_000_000)
        assert again == 1
        check(s, 4, Q, O, lse, 1 / 8)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_value_that_is_not_finite_costs_other_rows_nothing(dtype):
    """NaN in one value that every row of a long sequence sees: their outputs are NaN, all others' what they are."""
    s = Step([(50, 20000), (40, 600), (33, 33)], H=2, d=64, dtype=dtype, seed=12)
    page, row = s.table_np[0, 100 // s.P], 100 % s.P
    if s.e4m3:
        s.codes[1][0, page, 1, row, 7] = 0x7F
    else:
        s.pools[1][0, page, 1, row, 7] = float("nan")
    s.upload()
    G = 4
    Q = queries(s, G)
    O, lse, again = attend_again(s, G, Q, max_ctas=2, timeout_ns=20_000_000)
    assert again == 1
    hit = O[0][:50, G:].clone()
    assert bool(hit[..., 7].isnan().all()) and bool(hit[..., :7].isfinite().all()) and bool(hit[..., 8:].isfinite().all())
    O[0][:50, G:, 7] = 0   # (column 7 of the second head is NaN and checked: the oracle's value is set to match)
    if s.e4m3:
        s.vals[1][0, page, 1, row, 7] = 0.0
    s.vals[1][0, :, 1, :, 7] = 0.0
    O[0][50:, G:, 7] = 0   # (nor is that column compared in the other sequences, whose values were set to 0 with it)
    check(s, G, Q, O, lse, 1 / 8)


@pytest.mark.parametrize("G", [1, 3, 7])
@pytest.mark.parametrize("R", [1, 2])
def test_marked_rows_anywhere_in_a_step(G, R):
    """Sequences whose rows begin anywhere in a word of marks, some with powers far apart, on every rank."""
    s = Step([(50, 90), (7, 300), (0, 5), (0, 0), (133, 133), (90, 120), (1, 40), (129, 700)], H=2, d=128, P=16, dtype="e4m3", R=R,
             seed=G, lead=1, behind=2)
    for which in (0, 1):
        e = s.exps[which].astype(int)
        for b in (1, 4, 7):
            for page in s.table_np[b]:
                if page >= 0:
                    e[:, page, b % 2, 5] -= 40
        set_powers(s, which, e)
    s.upload()
    Q = queries(s, G)
    O, lse, again = attend_again(s, G, Q)
    assert again == 1
    check(s, G, Q, O, lse, 1 / np.sqrt(128))
    O2, lse2, _ = attend_again(s, G, Q)
    assert all(torch.equal(a, b) for a, b in zip(O + lse, O2 + lse2))   # a fixed order of summation
    O3, lse3, _ = attend_again(s, G, Q, max_ctas=5)
    check(s, G, Q, O3, lse3, 1 / np.sqrt(128))


def test_marks_of_the_call_before_are_gone():
    """The same workspace for a step with marked rows and one without, as a captured step is replayed."""
    s = Step([(60, 200), (20, 333)], H=1, dtype="bf16", seed=3)
    Q = queries(s, 4)
    clean, z0, again = attend_again(s, 4, Q)
    assert again == 0
    n = fcc.fcc_paged_attention_workspace_size(1, s.T, 2, 4, 1, 128)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    o = fcc.make_opts(workspace=ws, workspace_bytes=n)
    page, row = s.table_np[0, 0], 3
    keep = s.V[0][page, 0, row].clone()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    O, z = torch.zeros_like(Q[0]), torch.zeros(s.T, 4, device="cuda")
    cache, batch = s.cache(), s.batch()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        fcc.fcc_paged_attention(1, Q, cache, batch, 4, [O], [z], opts=o, stream=torch.cuda.current_stream())
    for bad in (False, True, False, True):
        s.V[0][page, 0, row] = float("inf") if bad else keep
        O.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert fcc.fcc_stream_status() == fcc.FCC_OK
        assert int(ws[12:16].view(torch.int32)) == int(bad)
        if bad:
            # (inf times positive weights; the second sequence does not see it)
            assert bool((to_f64(O[:60]) == np.inf).all()) and torch.equal(O[60:], clean[0][60:])
        else:
            assert torch.equal(O, clean[0]) and torch.equal(z, z0[0])


@pytest.mark.parametrize("L", [257, 289, 352, 400, 384])
@pytest.mark.parametrize("powers", [(113, 113), (129, 113), (113, 90), (240, 190)])
def test_positions_that_are_not_there_have_no_power(powers, L):
    """A last block that ends inside or before a group of 32 positions, behind blocks with larger powers: what is not
    there must not take a power from the block before (an infinity times zero), which would mark every row."""
    s = Step([(64, L), (33, L - 31)], H=1, d=64, dtype="e4m3", seed=L)
    for which in (0, 1):
        e = np.full_like(s.exps[which], powers[0] if which else 120).astype(int)
        for b, (_, n) in enumerate(s.seqs):
            for j in range(n // 128 * 128, n):
                e[:, s.table_np[b, j // s.P], :, j % s.P] = powers[1] if which else 120
        set_powers(s, which, e)
    s.upload()
    Q = queries(s, 4)
    for ctas in (1, 0):
        O, lse, again = attend_again(s, 4, Q, max_ctas=ctas)
        check(s, 4, Q, O, lse, 1 / 8)
        assert again == 0, ctas


@pytest.mark.parametrize("L", [40, 168, 300, 384])
@pytest.mark.parametrize("scale", [0.0, 1e-20, 3.0])
def test_rows_of_small_queries(L, scale):
    """Queries of zero and of 2^-8 to 2^-30, and a scale that makes everything small: a masked score is -inf times a
    factor that must not round to zero, above all where a block ends before its last group of 32 positions."""
    s = Step([(40, L)], H=1, d=128, dtype="e4m3", seed=L)
    Q = queries(s, 4)
    Q[0][0] = 0
    Q[0][17, 2] = 0
    Q[0][5:9] *= 2.0 ** -8
    Q[0][9] *= 2.0 ** -30
    O, lse, again = attend_again(s, 4, Q, scale=scale)
    check(s, 4, Q, O, lse, scale or 128 ** -0.5)
    assert again == 0
    Q[0][11] *= 2.0 ** -110       # (these may be computed again)
    Q[0][13, 1] *= 2.0 ** -130
    O, lse, _ = attend_again(s, 4, Q, scale=scale)
    check(s, 4, Q, O, lse, scale or 128 ** -0.5)


@pytest.mark.parametrize("case,G", [([(1, 70)], 8), ([(2, 70)], 8), ([(80, 149)], 4)])
@pytest.mark.parametrize("bits", [10.3, 26.4764])
def test_small_probabilities_keep_their_digits(case, G, bits):
    """e4m3, by items of 8 and 16 rows and by tiles: one position, whose values are zero, has 2^bits times the weight
    of each other.  The output is the others'.  The largest probability is 2^8 at least, so that theirs
    are 2^-18.5 at least, and f16 rounds them by 2^-25 at most: 2^-6.5 of themselves in the worst case.  These are
    46.00 steps of 2^-24, off by less than 2^-10 (with a largest of 2^6 they were 11.50 steps, off by 2^-4.5)."""
    s = Step(case, H=1, d=128, dtype="e4m3", seed=int(bits))
    for which in (0, 1):
        set_powers(s, which, np.full_like(s.exps[which], 119).astype(int))
    page, row = s.table_np[0, 0], 3
    s.codes[0][:] = 0
    s.codes[0][0, page, 0, row, 0] = 0x38                     # 1.0: the only key that is not zero
    s.codes[1][(s.codes[1] & 0x7F) == 0] |= 1
    s.codes[1][0, page, 0, row] = 0
    for which in (0, 1):
        s.vals[which] = oc.values(s.codes[which], s.exps[which])
    s.upload()
    Q = [torch.zeros(s.T, G, 128, device="cuda", dtype=torch.bfloat16)]
    Q[0][..., 0] = 1.0
    scale = float(np.float32(bits * np.log(2) * 2.0 ** 8))    # (the key is 2^-8)
    O, lse = attend(s, G, Q, scale=scale)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    check(s, G, Q, O, lse, scale)


@pytest.mark.parametrize("apart", [16, 20, 22])
def test_powers_up_to_22_apart_are_a_tiles_own(apart):
    """Values (and keys) that append makes quiet beside their neighbours, one position in eight and each its own way."""
    s = Step([(60, 700), (33, 95)], H=2, d=128, dtype="e4m3", seed=apart)
    for which in (0, 1):
        e = np.full_like(s.exps[which], 140).astype(int)
        quiet = s.g.random(e.shape) < 1 / 8
        e[quiet] -= s.g.integers(0, apart + 1, e.shape)[quiet]
        if which == 0:
            e -= 22
        # (a column in which the loudest position holds zero shows the others' P, which f16 may have cut short)
        s.codes[which][(s.codes[which] & 0x7F) == 0] |= 1
        set_powers(s, which, e)
    s.upload()
    Q = queries(s, 4)
    for window in (0, 3):
        O, lse, again = attend_again(s, 4, Q, window=window)
        check(s, 4, Q, O, lse, 128 ** -0.5, window)
        assert again == 0


def test_a_cache_with_quiet_rows_as_append_writes_it():
    """Value rows 2^-20 of the others in one place of a hundred (and rows of zeros) are ordinary contents."""
    H, d, P, L, n, G = 2, 128, 16, 1500, 100, 4
    s = Step([(n, L)], H=H, d=d, P=P, dtype="e4m3", seed=2)
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(L, H, d, device="cuda", generator=g) for _ in range(2))
    v *= torch.where(torch.rand(L, H, 1, device="cuda", generator=g) < 0.01, 2.0 ** -20, 1.0)
    v[5] = 0
    k[300] = 0
    k, v = k.bfloat16(), v.bfloat16()
    fcc.fcc_cache_append(1, [k], [v], s.cache(), fcc.make_batch(dev([0, L]), dev([L]), s.table, L, 1, s.max_pages))
    for which, x in ((0, k), (1, v)):
        codes, power = oc.quantise(to_f64(x))
        for j in range(L):
            page, row = s.table_np[0, j // P], j % P
            s.codes[which][0, page, :, row], s.exps[which][0, page, :, row] = codes[j], power[j]
        s.vals[which] = oc.values(s.codes[which], s.exps[which])
    Q = queries(s, G)
    O, lse, again = attend_again(s, G, Q)
    check(s, G, Q, O, lse, 1 / np.sqrt(d))
    assert again == 0


def test_the_longest_token_arrays():
    """T = 2^31 - 1, where the last group of rows ends at the largest int.  Only a sequence's own rows are touched,
    which begin the arrays here."""
    s = Step([(5, 9), (2, 40)], H=1, d=64, dtype="bf16", seed=1)
    T = s.T
    out = [torch.full((T, 1, 64), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    fcc.fcc_cache_gather(1, s.cache(), s.batch(2 ** 31 - 1), [out[0]], [out[1]])
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    for which in range(2):
        for b, (n, L) in enumerate(s.seqs):
            a = int(s.start_np[b])
            assert np.array_equal(to_f64(out[which][a:a + n]), s.held(which, 0, b, L - n, L))


@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("e4m3", 1)])
def test_marked_rows_with_strides_windows_and_no_lse(dtype, P):
    """Rows that are computed again are stored where the tiles' are: rows of O apart, no lse, a window, a second rank."""
    s = Step([(70, 300), (50, 180)], H=2, d=64, P=P, dtype=dtype, R=2, seed=P, lead=3, behind=2)
    for b, j in ((0, 200), (1, 100)):
        page, row = s.table_np[b, j // P], j % P
        if s.e4m3:
            for which in (0, 1):
                e = s.exps[which].astype(int)
                e[:, page, :, row] -= 40
                set_powers(s, which, e)
        else:
            s.pools[1][:, page, :, row] = float("nan")        # (only each sequence's first row, at 230 and 130, sees it)
    s.upload()
    G, window = 4, 31 if dtype == "bf16" else 150
    Hq = s.H * G
    Q = queries(s, G, ldq=(Hq + 3) * 64)
    n = fcc.fcc_paged_attention_workspace_size(2, s.T, 2, Hq, 2, 64)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    O, none = attend(s, G, Q, window=window, lse=False, ldo=(Hq + 2) * 64, opts=fcc.make_opts(workspace=ws, workspace_bytes=n))
    assert fcc.fcc_stream_status() == fcc.FCC_OK and none is None
    assert int(ws[12:16].view(torch.int32)) == 1 and bool((ws[n:] == 0xFF).all())
    assert all(bool((o[:, Hq:] == 7).all()) for o in O)
    if dtype == "bf16":
        for o in O:
            for t in s.start_np[:2]:
                assert bool(o[t, :Hq].isnan().all())
                o[t, :Hq] = 7.0
        s.start_np, s.seqs = s.start_np[:2] + 1, [(n - 1, L) for n, L in s.seqs]   # the others
    check(s, G, Q, [o[:, :Hq] for o in O], None, 1 / 8, window)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_step_in_two_calls(dtype):
    """Sequences of one row and a chunk behind them, each by a call of its own over its part of the arrays."""
    s = Step([(1, 100), (1, 30), (1, 1), (1, 200), (0, 50), (60, 300)], dtype=dtype, seed=6)
    G = 4
    Q = queries(s, G)
    O, lse = [torch.full_like(Q[0], 7.0)], [torch.full((s.T, s.H * G), 7.0, device="cuda")]
    few = fcc.make_batch(s.start, s.len, s.table, 4, 5, s.max_pages)
    many = fcc.make_batch(s.start[5:], s.len[5:], s.table[5:], s.T, 1, s.max_pages)
    for batch in (few, many):
        fcc.fcc_paged_attention(1, Q, s.cache(), batch, s.H * G, O, lse)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    check(s, G, Q, O, lse, 128 ** -0.5)


@pytest.mark.parametrize("case,G", [([(1, 200)], 8), ([(2, 200)], 8), ([(80, 279)], 4)])
def test_zeros_beside_values_2_to_the_120_above(case, G):
    """The widest range of powers that a row may see: 70 positions of zeros (byte 63) before values of byte 183.  The
    zeros' weights count in the sum: p 2^-b is 2^8 2^-120 2^64 for them and 2^8 2^-56 for the others."""
    s = Step(case, H=1, d=64, dtype="e4m3", seed=20)
    e = np.full_like(s.exps[1], 183).astype(int)
    for j in range(70):
        page, row = s.table_np[0, j // s.P], j % s.P
        e[:, page, :, row] = 63
        s.codes[1][:, page, :, row] = 0
    set_powers(s, 0, np.full_like(s.exps[0], 119).astype(int))
    set_powers(s, 1, e)
    s.upload()
    Q = queries(s, G)
    O, lse = attend(s, G, Q)
    assert fcc.fcc_stream_status() == fcc.FCC_OK
    check(s, G, Q, O, lse, 1 / 8)
