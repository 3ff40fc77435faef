"""The paged cache on the GPU against the fp64 oracle: appending (bf16 and e4m3), reading
back, decoding, and a run of them together with the block-sparse call.

Tolerances of a decode (derived, u = 2^-24): a logit is a sum of d products of two 16-bit or
8-bit values, exact as products, summed in fp32 in any order and possibly truncated, then
scaled: |dl| <= (d + 8) * 2u * scale * sum|q_c k_c|. A weight e^(l - m) carries the errors of
two logits, of the exponential (2^-21 with its argument's rounding, which is relative to the
logit's size) and, in the product with v, what its 16-bit pieces drop: half a step of the
last piece, 2^-11 of the weight for one f16 piece (e4m3 rows, bf16 output), 2^-16 for two
bf16 pieces (bf16 rows, bf16 output), 2^-22 and 2^-24 for the two f16 or three bf16 pieces of
an fp32 output. The output is a convex mix of the v, so its error is at most twice the
weights' relative error times max|v|, plus the sums' own n*u rounding (taken as 2^-18 for the
lengths used here) and, for bf16 outputs, half a step 2^-8 relative to the value. The sum of
weights, and so the lse, has the whole fp32 weights."""
import numpy as np
import pytest
import torch

from free_block_sparse_kv_b200 import attention as A
from free_block_sparse_kv_b200 import paged_cache as P
from free_block_sparse_kv_b200 import sparse_attn as C
from free_block_sparse_kv_b200 import workloads as W
from oracle import paged_cache as O

pytestmark = pytest.mark.gpu

E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    C.load_library()


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _np(x):
    return x.detach().double().cpu().numpy()


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(BF16).cuda()


def _filled(rng, num_pages, H, page, d, dtype):
    """A pool with every byte set: a cache of random rows."""
    c = P.allocate_cache(num_pages, H, page, d, dtype)
    for name in ("k", "v"):
        x = rng.standard_normal((num_pages, H, page, d)) * np.exp2(
            rng.integers(-3, 4, (num_pages, H, page, 1)))
        if dtype == BF16:
            getattr(c, name).copy_(torch.from_numpy(x.astype(np.float32)))
        else:
            code, s = O.quantise(x)
            getattr(c, name).copy_(torch.from_numpy(code.astype(np.float32)).to(E4M3))
            getattr(c, name + "_scale").copy_(
                torch.from_numpy(s.astype(np.float32)).to(torch.float8_e8m0fnu))
    return c


def _table(rng, need, page, num_pages, spare=0):
    """Distinct random pages for every sequence, -1 where it needs none."""
    used = [-(-n // page) for n in need]
    perm = rng.permutation(num_pages)
    assert sum(used) <= num_pages
    t = np.full((len(need), max(1, max(used)) + spare), -1)
    at = 0
    for b, u in enumerate(used):
        t[b, :u] = perm[at:at + u]
        at += u
    return t


def _raw(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)


def _snapshot(c):
    return [None if x is None else _raw(x).clone() for x in (c.k, c.v, c.k_scale, c.v_scale)]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,H,T,d,page,major", [
    (1, 1, 1, 128, 16, False), (3, 5, 1, 64, 32, False), (2, 3, 37, 128, 64, True),
    (4, 2, 130, 64, 16, True), (2, 7, 65, 128, 256, False), (5, 40, 3, 128, 128, True)])
def test_append(B, H, T, d, page, major, dtype):
    rng = np.random.default_rng(B * 100 + T)
    start = [int(x) for x in rng.integers(0, 3 * page, B)]
    count = [T if b == 0 else int(rng.integers(0, T + 1)) for b in range(B)]
    table = _table(rng, [s + n for s, n in zip(start, count)], page, 4 + sum(
        -(-(s + n) // page) for s, n in zip(start, count)), spare=1)
    num = int(table.max()) + 3
    c = _filled(rng, num, H, page, d, dtype)
    shape = (B, T, H, d) if major else (B, H, T, d)
    k, v = _bf16(rng, *shape, scale=3.0), _bf16(rng, *shape, scale=0.02)
    k.view(-1)[::7] *= 16
    if major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    want = []
    for x, pages, scales in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        p, s = _np(pages), None if scales is None else _np(scales)
        O.append(p, s, _np(x), table, start, count, page)
        want += [p, s]
    flag = _ints([0])
    P.cache_append(c, k, v, _ints(table), _ints(start), _ints(count), err_flag=flag)
    P.check(flag)
    # every value of the pool: the new rows as the oracle stores them, the others as they were
    for got, w in zip((c.k, c.k_scale, c.v, c.v_scale), want):
        if w is not None:
            assert np.array_equal(_np(got), w)


def test_append_without_counts_and_out_of_place_rows():
    """count None appends T rows of every sequence; rows without a page are left out and
    reported, everything else is written and nothing else is touched."""
    rng = np.random.default_rng(5)
    B, H, T, d, page = 4, 2, 20, 64, 16
    c = _filled(rng, 9, H, page, d, E4M3)
    k, v = _bf16(rng, B, H, T, d), _bf16(rng, B, H, T, d)
    table = np.array([[0, 1, 2], [3, 9, 4], [5, 6, -1], [7, 8, 8]])
    start = [3, 5, 20, 40]       # 1: page 9 is past the pool; 2: page -1; 3: past the table
    wk, wv = (_np(x) for x in (c.k, c.v))
    sk, sv = (_np(x) for x in (c.k_scale, c.v_scale))
    for p, s, x in ((wk, sk, k), (wv, sv, v)):
        for b, live in enumerate([range(20), list(range(11)), list(range(12)), list(range(8))]):
            if b == 1:
                live = [t for t in range(20) if (5 + t) // page != 1]
            for t in live:
                pg, row = table[b][(start[b] + t) // page], (start[b] + t) % page
                p[pg, :, row], s[pg, :, row] = O.quantise(_np(x)[b, :, t])
    flag = _ints([0])
    P.cache_append(c, k, v, _ints(table), _ints(start), err_flag=flag)
    with pytest.raises(C.SparseAttnError) as e:
        P.check(flag)
    assert e.value.code == C.SA_ERR_INDEX
    for got, w in ((c.k, wk), (c.v, wv), (c.k_scale, sk), (c.v_scale, sv)):
        assert np.array_equal(_np(got), w)
    before = _snapshot(c)
    for st, n in (([-1] * B, [T] * B), ([0] * B, [-3] * B)):
        flag.zero_()
        P.cache_append(c, k, v, _ints(table), _ints(st), _ints(n), err_flag=flag)
        assert int(flag.item()) == C.SA_FLAG_INDEX
    assert all(torch.equal(a, b) for a, b in zip(before, _snapshot(c)))


def test_append_extreme_rows():
    """Zeros, subnormals, the largest values, infinities and NaN."""
    d, page = 64, 16
    x = np.zeros((1, 1, 12, d), np.float32)
    x[0, 0, 1] = 2.0 ** -133
    x[0, 0, 2, 5] = 3.0e38
    x[0, 0, 3, :3] = [np.inf, 1.0, -2.0]
    x[0, 0, 4, :3] = [np.nan, -np.inf, 0.0]
    x[0, 0, 5] = np.linspace(-448, 448, d)
    x[0, 0, 6, :2] = [1.75 * 256, 1.0]
    x[0, 0, 7, :2] = [1.7578125 * 256, 1.0]
    x[0, 0, 8] = np.float32(2.0) ** np.arange(-60, 4)
    x[0, 0, 9, 0] = -0.0
    x[0, 0, 10] = 2.0 ** -120
    x[0, 0, 11, :2] = [2.0 ** 127, -2.0 ** 100]
    k = torch.from_numpy(x).to(BF16).cuda()
    c = P.allocate_cache(1, 1, page, d, E4M3)
    for y in (c.k, c.v, c.k_scale, c.v_scale):
        y.view(torch.uint8).fill_(1)
    P.cache_append(c, k, -k, _ints([[0]]), _ints([2]))
    code, s = O.quantise(_np(k)[0, 0])
    assert np.array_equal(_np(c.k)[0, 0, 2:14], code, equal_nan=True)
    assert np.array_equal(_np(c.v)[0, 0, 2:14], -code, equal_nan=True)
    assert np.array_equal(_np(c.k_scale)[0, 0, 2:14], s)
    out = torch.zeros(2, 1, 1, 16, d, dtype=BF16, device="cuda")
    P.cache_read(c, _ints([[0]]), _ints([14]), out[0], out[1], first=_ints([2]))
    want = torch.from_numpy(code * s[:, None]).to(BF16).double().numpy()
    assert np.array_equal(_np(out[0])[0, 0, 2:14], want, equal_nan=True)
    assert not _np(out[:, 0, 0, :2]).any() and not _np(out[:, 0, 0, 14:]).any()


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,H,N,d,page,major", [
    (1, 1, 1, 64, 16, False), (3, 2, 200, 128, 64, True), (4, 3, 77, 64, 32, False),
    (2, 5, 600, 128, 256, True), (2, 40, 33, 128, 16, False)])
def test_read(B, H, N, d, page, major, dtype):
    rng = np.random.default_rng(N)
    lens = [N] + [int(x) for x in rng.integers(0, N + 1, B - 1)]
    first = [0 if b % 2 == 0 else min(lens[b], 5 + page // 2) for b in range(B)]
    num = sum(-(-n // page) for n in lens) + 2
    table = _table(rng, lens, page, num)
    c = _filled(rng, num, H, page, d, dtype)
    mk = lambda: torch.full((B, N, H, d) if major else (B, H, N, d), 7.0, dtype=BF16, device="cuda")
    k, v = mk(), mk()
    kk, vv = (k.transpose(1, 2), v.transpose(1, 2)) if major else (k, v)
    flag = _ints([0])
    P.cache_read(c, _ints(table), _ints(lens), kk, vv, first=_ints(first), err_flag=flag)
    P.check(flag)
    for got, pages, scales in ((kk, c.k, c.k_scale), (vv, c.v, c.v_scale)):
        want = np.full((B, H, N, d), 7.0)
        for b in range(B):
            for h in range(H):
                want[b, h, first[b]:lens[b]] = O.rows(
                    _np(pages), None if scales is None else _np(scales), table[b], lens[b], h,
                    page)[first[b]:]
        assert np.array_equal(_np(got), want)
    if first[-1] == 0 or B == 1:
        k2, v2 = torch.zeros_like(kk), torch.zeros_like(vv)
        P.cache_read(c, _ints(table), _ints(lens), k2, v2)
        assert torch.equal(k2[0, :, :lens[0]], kk[0, :, :lens[0]])


def test_read_out_of_range_is_reported():
    rng = np.random.default_rng(8)
    H, d, page, N = 2, 64, 16, 40
    c = _filled(rng, 4, H, page, d, BF16)
    k, v = (torch.full((3, H, N, d), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    # 0: a page past the pool in the middle; 1: longer than the table; 2: negative length
    table, lens = [[0, 4, 1], [2, 3, 0], [1, 1, 1]], [40, 60, -2]
    flag = _ints([0])
    P.cache_read(c, _ints(table), _ints(lens), k, v, err_flag=flag)
    assert int(flag.item()) == C.SA_FLAG_INDEX
    for got, pages in ((k, _np(c.k)), (v, _np(c.v))):
        got = _np(got)
        assert np.array_equal(got[0, :, :16], pages[0]) and np.array_equal(got[0, :, 32:], pages[1][:, :8])
        assert (got[0, :, 16:32] == 7).all() and (got[2] == 7).all()
        assert np.array_equal(got[1], np.concatenate([pages[2], pages[3], pages[0][:, :8]], 1))


# ------------------------------------------------------------------ decode
DROP = {(E4M3, BF16): 2.0 ** -11, (E4M3, F32): 2.0 ** -22, (BF16, BF16): 2.0 ** -16,
        (BF16, F32): 2.0 ** -24}


def _bounds(rows_dtype, out_dtype, d, scale, want, lse, vmax, qk):
    w = 2 * (d + 8) * 2.0 ** -23 * abs(scale) * qk + 2.0 ** -20 * (1 + abs(scale) * qk)
    tol = (2 * (w + DROP[rows_dtype, out_dtype]) + 2.0 ** -18)[..., None] * vmax[..., None]
    if out_dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    return tol, w + 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def _check(got, lse_got, out_dtype, d, scale, q, c, table, lens, page, kept=None):
    ks, vs = (None if x is None else _np(x) for x in (c.k_scale, c.v_scale))
    want, lse, vmax, qk = O.decode(_np(q), _np(c.k), _np(c.v), ks, vs, table, lens, page, scale, kept)
    tol, ltol = _bounds(c.k.dtype, out_dtype, d, scale, want, lse, vmax, qk)
    err = np.abs(_np(got) - want)
    assert (err <= tol).all(), (err - tol).max()
    empty = np.isneginf(lse)
    lg = _np(lse_got)
    assert np.array_equal(np.isneginf(lg), empty)
    assert (np.abs(lg[~empty] - lse[~empty]) <= ltol[~empty]).all()
    assert not _np(got)[empty].any()


CASES = [  # B, Hq, H, T, d, page, lens
    (1, 1, 1, 1, 64, 16, [1]),
    (1, 2, 2, 1, 128, 16, [17]),
    (3, 4, 2, 1, 128, 64, [0, 63, 65]),
    (4, 6, 2, 1, 64, 32, [1, 300, 0, 129]),
    (2, 8, 1, 1, 128, 128, [1000, 127]),
    (1, 40, 40, 1, 128, 128, [515]),
    (2, 10, 2, 2, 64, 16, [1, 257]),
    (3, 8, 4, 4, 128, 16, [2, 4, 131]),
    (2, 9, 3, 7, 128, 32, [3, 400]),
    (2, 32, 2, 2, 128, 64, [777, 16]),
    (1, 35, 1, 1, 64, 64, [321]),
    (2, 20, 1, 16, 128, 16, [9, 200]),
    (17, 2, 1, 1, 64, 256, list(range(0, 17 * 31, 31))),
    (1, 16, 16, 1, 128, 64, [1560]),
    (1, 4, 1, 3, 128, 16, [9001]),
    # more sequences than a warp scans by itself, many of one step, some of none
    (300, 2, 1, 1, 64, 16, [(7 * b) % 90 if b % 5 else 0 for b in range(300)]),
    (600, 1, 1, 2, 128, 16, [1 + (b * b) % 37 for b in range(600)]),
    # segments of one step and of many in turn, so that shares hold several and parts of others
    (40, 16, 4, 1, 128, 16, [3 if b % 3 else 2000 for b in range(40)]),
    (24, 36, 2, 1, 64, 32, [33 * b + 1 for b in range(24)]),
    (5, 40, 1, 1, 128, 64, [4100, 1, 0, 2222, 640]),
]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode(case, out_dtype, dtype):
    B, Hq, H, T, d, page, lens = CASES[case]
    rng = np.random.default_rng(case)
    num = sum(-(-n // page) for n in lens) + 1
    table = _table(rng, lens, page, num, spare=case % 3)
    c = _filled(rng, num, H, page, d, dtype)
    q = _bf16(rng, B, Hq, T, d) if case % 2 else _bf16(rng, B, T, Hq, d).transpose(1, 2)
    flag = _ints([0])
    out, lse = P.decode(q, c, _ints(table), _ints(lens), out_dtype=out_dtype, return_lse=True,
                        err_flag=flag)
    P.check(flag)
    assert out.dtype == out_dtype
    _check(out, lse, out_dtype, d, 1 / np.sqrt(d), q, c, table, lens, page)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,Hq,H,T,d,page,lens,cap", [
    (2, 4, 4, 1, 128, 64, [1000, 130], 5), (3, 8, 2, 1, 64, 16, [0, 200, 333], 9),
    (2, 6, 1, 3, 128, 32, [500, 2], 4), (1, 8, 8, 1, 128, 128, [5000], 40)])
def test_decode_kept_pages(B, Hq, H, T, d, page, lens, cap, dtype):
    """Lists of different lengths per kv head (empty ones among them), entries past the
    length or outside the table, the last partial page kept or not."""
    rng = np.random.default_rng(cap)
    num = sum(-(-n // page) for n in lens) + 1
    table = _table(rng, lens, page, num, spare=2)
    width = table.shape[1]
    c = _filled(rng, num, H, page, d, dtype)
    q = _bf16(rng, B, Hq, T, d)
    idx, cnt = np.full((B, H, cap), 12345), np.zeros((B, H), int)
    kept = [[[] for _ in range(H)] for _ in range(B)]
    for b in range(B):
        n = -(-lens[b] // page)
        for h in range(H):
            m = min(cap, int(rng.integers(0, n + 1))) if (b + h) % 4 else 0
            pages = sorted(rng.choice(n, m, replace=False).tolist()) if m else []
            if b == 0 and h == 0 and n:
                pages = [n - 1]
            kept[b][h] = pages
            row = pages + [width + 7, -2, n][: cap - len(pages)]      # ignored or past the length
            idx[b, h, :len(row)], cnt[b, h] = row, len(row)
    out, lse = P.decode(q, c, _ints(table), _ints(lens), _ints(idx), _ints(cnt), return_lse=True)
    _check(out, lse, F32, d, 1 / np.sqrt(d), q, c, table, lens, page, kept)
    full = [[list(range(-(-lens[b] // page)))[:cap] for _ in range(H)] for b in range(B)]
    for b in range(B):
        for h in range(H):
            idx[b, h, :len(full[b][h])], cnt[b, h] = full[b][h], cap + 3    # clamped to cap
            idx[b, h, len(full[b][h]):] = -1
    out, lse = P.decode(q, c, _ints(table), _ints(lens), _ints(idx)[:, :, None],
                        _ints(cnt)[:, :, None], scale=-0.3, out_dtype=BF16, return_lse=True)
    _check(out, lse, BF16, d, -0.3, q, c, table, lens, page, full)


def test_decode_kept_lists_of_many_heads():
    """More (sequence, head) lists than a warp scans by itself."""
    rng = np.random.default_rng(41)
    B, H, d, page = 45, 8, 64, 16
    lens = [(37 * b) % 150 for b in range(B)]
    num = sum(-(-n // page) for n in lens) + 1
    table = _table(rng, lens, page, num)
    c = _filled(rng, num, H, page, d, E4M3)
    q = _bf16(rng, B, 2 * H, 1, d)
    kept = [[sorted(rng.choice(-(-n // page), rng.integers(0, -(-n // page) + 1), replace=False).tolist())
             for _ in range(H)] for n in lens]
    idx, cnt = np.zeros((B, H, 10), int), np.zeros((B, H), int)
    for b in range(B):
        for h in range(H):
            idx[b, h, :len(kept[b][h])], cnt[b, h] = kept[b][h], len(kept[b][h])
    out, lse = P.decode(q, c, _ints(table), _ints(lens), _ints(idx), _ints(cnt), return_lse=True)
    _check(out, lse, F32, d, 1 / np.sqrt(d), q, c, table, lens, page, kept)


def test_decode_zero_rows_beside_small_values():
    """Rows of zeros (stored with scale 1) do not drown values of 1e-9 in 8 bits: the output
    is compared on the values' own scale."""
    rng = np.random.default_rng(43)
    H, d, page, n = 2, 128, 32, 300
    k, v = _bf16(rng, 1, H, n, d), _bf16(rng, 1, H, n, d, scale=1e-9)
    v[:, :, ::3] = 0
    v[:, 1, :, :] = 0          # and a head with nothing else
    c = P.allocate_cache(10, H, page, d, E4M3)
    table = [list(range(10))]
    P.cache_append(c, k, v, _ints(table), _ints([0]))
    q = _bf16(rng, 1, 4 * H, 1, d)
    for dt in (F32, BF16):
        out, lse = P.decode(q, c, _ints(table), _ints([n]), out_dtype=dt, return_lse=True)
        _check(out, lse, dt, d, 1 / np.sqrt(d), q, c, table, [n], page)
        assert not out[:, 4:].any() and out[:, :4].any()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("T,G", [(1, 2), (5, 3), (16, 1)])
def test_decode_ignores_what_a_row_does_not_attend(T, G, dtype):
    """NaN and infinities in unused pages, behind the last row, and in the K and V of new
    tokens that earlier rows do not see."""
    rng = np.random.default_rng(T)
    B, H, d, page, lens = 2, 2, 128, 16, [100, 37]
    num = 14
    table = _table(rng, lens, page, num, spare=1)
    c = _filled(rng, num, H, page, d, dtype)
    q = _bf16(rng, B, H * G, T, d)
    tab, ln = _ints(table), _ints(lens)
    clean, clean_lse = P.decode(q, c, tab, ln, return_lse=True)
    bad = torch.tensor(float("nan"), device="cuda")
    used = np.zeros((num, page), bool)
    for b in range(B):
        pos = np.arange(lens[b])
        used[table[b][pos // page], pos % page] = True
    hole = torch.from_numpy(~used).cuda()
    for name in ("k", "v"):
        x = getattr(c, name).float()
        x = torch.where(hole[:, None, :, None], bad, x)
        for b in range(B):       # the last token: only row T - 1 attends it
            pos = lens[b] - 1
            x[table[b][pos // page], :, pos % page, ::3] = float("nan")
            if dtype == BF16:
                x[table[b][pos // page], :, pos % page, 1::3] = float("inf")
        getattr(c, name).copy_(x.to(dtype))
        if dtype == E4M3:
            s = getattr(c, name + "_scale").view(torch.uint8)
            s.masked_fill_(hole[:, None, :].expand_as(s), 255)
    out, lse = P.decode(q, c, tab, ln, return_lse=True)
    assert not torch.isfinite(out[:, :, T - 1]).all(-1).any()
    assert torch.equal(out[:, :, :T - 1], clean[:, :, :T - 1])
    assert torch.equal(lse[:, :, :T - 1], clean_lse[:, :, :T - 1])


def test_decode_out_of_range_pages_and_lengths():
    rng = np.random.default_rng(11)
    H, d, page = 2, 64, 16
    c = _filled(rng, 6, H, page, d, BF16)
    q = _bf16(rng, 3, 4, 1, d)
    table = [[0, 6, 1], [2, 3, 4], [5, 5, 5]]
    lens = [45, 1000, -1]        # 0: a bad page in the middle; 1: past the table; 2: negative
    flag = _ints([0])
    out, lse = P.decode(q, c, _ints(table), _ints(lens), return_lse=True, err_flag=flag)
    with pytest.raises(C.SparseAttnError) as e:
        P.check(flag)
    assert e.value.code == C.SA_ERR_INDEX
    # what is left: pages 0 and 2 of the first sequence, the whole table row of the second
    kept = [[[0, 2]] * H, [[0, 1, 2]] * H, [[]] * H]
    _check(out, lse, F32, d, 1 / np.sqrt(d), q, c, [[0, 0, 1], [2, 3, 4], [5, 5, 5]], [45, 48, 0],
           page, kept)
    # an empty table and an empty pool: nothing is attended, nothing is read
    none = P.allocate_cache(0, H, page, d)
    out, lse = P.decode(q, none, _ints(np.zeros((3, 0))), _ints([0, 0, 0]), return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    flag.zero_()
    out, lse = P.decode(q, none, _ints(np.zeros((3, 2))), _ints([5, 0, 32]), return_lse=True,
                        err_flag=flag)
    assert not out.any() and torch.isneginf(lse).all() and int(flag.item()) == C.SA_FLAG_INDEX
    empty = P.decode(q[:0], c, _ints(np.zeros((0, 3))), _ints([]))
    assert empty.shape == (0, 4, 1, d)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_decode_extreme_values(dtype):
    """Logits of +-10^4 (weights that underflow), one dominant key, values of very
    different sizes between rows, and a zero scale (equal weights)."""
    rng = np.random.default_rng(13)
    B, H, d, page, lens = 2, 2, 128, 32, [700, 33]
    num = 25
    table = _table(rng, lens, page, num)
    c = P.allocate_cache(num, H, page, d, dtype)
    T = num * page
    k = _bf16(rng, 1, H, T, d, scale=20)
    v = _bf16(rng, 1, H, T, d)
    v *= torch.exp2(torch.from_numpy(rng.integers(-20, 20, (1, H, T, 1)).astype(np.float32))).cuda()
    k[:, :, ::50] *= 8
    P.cache_append(c, k, v.to(BF16), _ints([list(range(num))]), _ints([0]))
    q = _bf16(rng, B, 2 * H, 1, d, scale=5)
    for scale in (1 / np.sqrt(d), 0.0, 1e-4):
        out, lse = P.decode(q, c, _ints(table), _ints(lens), scale=scale, return_lse=True)
        _check(out, lse, F32, d, scale, q, c, table, lens, page)


def test_decode_far_pages_of_a_large_pool():
    """Element offsets past 2^32 (bf16) and byte offsets past 2^32 (e4m3)."""
    H, page, d = 64, 256, 128
    for dtype, num in ((BF16, 2100), (E4M3, 2100)):
        rng = np.random.default_rng(17)
        assert num * H * page * d > 1 << 32
        c = P.allocate_cache(num, H, page, d, dtype)
        table, lens = [[num - 1, 3]], [300]
        x = _bf16(rng, 2, 1, H, 300, d)
        flag = _ints([0])
        P.cache_append(c, x[0], x[1], _ints(table), _ints([0]), err_flag=flag)
        q = _bf16(rng, 1, H, 1, d)
        out, lse = P.decode(q, c, _ints(table), _ints(lens), return_lse=True, err_flag=flag)
        back = torch.empty(2, 1, H, 300, d, dtype=BF16, device="cuda")
        P.cache_read(c, _ints(table), _ints(lens), back[0], back[1], err_flag=flag)
        P.check(flag)
        near = P.allocate_cache(2, H, page, d, dtype)
        P.cache_append(near, x[0], x[1], _ints([[1, 0]]), _ints([0]))
        assert torch.equal(out, P.decode(q, near, _ints([[1, 0]]), _ints(lens)))
        if dtype == BF16:
            assert torch.equal(back, x)
        _check(out, lse, F32, d, 1 / np.sqrt(d), q, near, [[1, 0]], lens, page)
        del c


# ------------------------------------------------------------------ streams, graphs, arguments
@pytest.mark.parametrize("lens,num", [([4000, 65, 2111], 110), ([30000, 65, 9111], 640)])
def test_repeats_streams_and_graphs(lens, num):
    """The same bits from call to call, on another stream, and from two captured graphs that
    replay at the same time on new data: sizes that run as clusters (no scratch) and on the
    line of all steps (scratch of each call)."""
    rng = np.random.default_rng(19)
    B, Hq, H, d, page = 3, 8, 2, 128, 64
    need = C.sparse_attn_decode_work_bytes(B, Hq, H, 1, d, C.SA_CACHE_E4M3, page, -(-lens[0] // page))
    assert (need > 0) == (lens[0] > 4000)
    table, ln = _ints(_table(rng, lens, page, num)), _ints(lens)
    c = _filled(rng, num, H, page, d, E4M3)
    q = [_bf16(rng, B, Hq, 1, d) for _ in range(4)]
    want = [P.decode(x, c, table, ln, return_lse=True) for x in q]
    for x, (o, l) in zip(q, want):
        o2, l2 = P.decode(x, c, table, ln, return_lse=True)
        assert torch.equal(o, o2) and torch.equal(l, l2)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [P.decode(x, c, table, ln, stream=side[i % 2]) for i, x in enumerate(q)]
    raw = P.decode(q[0], c, table, ln, stream=side[0].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w[0]) for g, w in zip(got, want)) and torch.equal(raw, want[0][0])
    ins = [q[0].clone(), q[1].clone()]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(P.decode(ins[i], c, table, ln))
        graphs.append(g)
    for i in range(2):
        ins[i].copy_(q[2 + i])
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[2][0]) and torch.equal(outs[1], want[3][0])


def test_append_and_read_in_a_graph_on_a_stream():
    rng = np.random.default_rng(23)
    B, H, T, d, page = 2, 3, 1, 64, 16
    c = _filled(rng, 6, H, page, d, E4M3)
    k, v = _bf16(rng, B, H, T, d), _bf16(rng, B, H, T, d)
    table, start, lens = _ints([[0, 1], [2, 3]]), _ints([14, 3]), _ints([15, 4])
    back = torch.zeros(2, B, H, 32, d, dtype=BF16, device="cuda")
    q = _bf16(rng, B, H, 1, d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.cache_append(c, k, v, table, start)
        P.cache_read(c, table, lens, back[0], back[1], first=start)
        out = P.decode(q, c, table, lens)
        start.add_(1)
        lens.add_(1)
    rows = []
    for step in range(4):        # across a page border of the first sequence
        k.copy_(_bf16(rng, B, H, T, d))
        v.copy_(_bf16(rng, B, H, T, d))
        g.replay()
        rows.append((k.clone(), v.clone()))
        torch.cuda.synchronize()
        _check(out, P.decode(q, c, table, _ints([15 + step, 4 + step]), return_lse=True)[1], F32, d,
               1 / np.sqrt(d), q, c, [[0, 1], [2, 3]], [15 + step, 4 + step], page)
    for step, (kk, vv) in enumerate(rows):
        for b, s in ((0, 14), (1, 3)):
            for x, got in ((kk, back[0]), (vv, back[1])):
                code, sc = O.quantise(_np(x)[b, :, 0])
                assert np.array_equal(_np(got)[b, :, s + step], code * sc[:, None])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,Hq,H,T,d,page,lens", [
    (2, 3, 1, 1, 64, 16, [1, 77]), (1, 8, 8, 5, 128, 64, [129]), (3, 40, 2, 2, 128, 16, [0, 31, 333]),
    (40, 16, 4, 1, 128, 16, [3 if b % 3 else 2000 for b in range(40)])])
def test_every_write_stays_in_its_buffer(B, Hq, H, T, d, page, lens, dtype):
    """Pools, outputs and scratch (of exactly the stated size) between canary regions."""
    from tests.test_gpu_canary import Guarded
    rng = np.random.default_rng(B + T)
    num = sum(-(-n // page) for n in lens) + 1
    table = _table(rng, lens, page, num)
    tab, ln = _ints(table), _ints(lens)
    g = dict(k=Guarded((num, H, page, d), dtype), v=Guarded((num, H, page, d), dtype))
    if dtype == E4M3:
        g.update(ks=Guarded((num, H, page), torch.float8_e8m0fnu), vs=Guarded((num, H, page), torch.float8_e8m0fnu))
    c = P.PagedCache(g["k"].t, g["v"].t, *(g[n].t for n in ("ks", "vs") if n in g))
    N = max(lens)
    k, v = _bf16(rng, B, H, N, d), _bf16(rng, B, H, N, d)
    P.cache_append(c, k, v, tab, _ints([0] * B), ln)
    g.update(k_out=Guarded((B, H, N, d), BF16), v_out=Guarded((B, H, N, d), BF16))
    P.cache_read(c, tab, ln, g["k_out"].t, g["v_out"].t)
    q = _bf16(rng, B, Hq, T, d)
    for odt, code in ((F32, C.SA_OUT_F32), (BF16, C.SA_OUT_BF16)):
        dt = C.SA_CACHE_BF16 if dtype == BF16 else C.SA_CACHE_E4M3
        need = C.sparse_attn_decode_work_bytes(B, Hq, H, T, d, dt, page, table.shape[1], -1, code)
        g.update(work=Guarded((need,), torch.uint8), out=Guarded((B, Hq, T, d), odt),
                 lse=Guarded((B, Hq, T), F32))
        C.sparse_attn_decode(q, q.stride()[:3], B, Hq, H, T, d, c.k, c.v, c.k_scale, c.v_scale, dt, num,
                             page, tab, table.shape[1], table.shape[1], ln, None, None, 0, d ** -0.5,
                             g["work"].t if need else None, g["out"].t, code, g["lse"].t)
        torch.cuda.synchronize()
        for name, x in g.items():
            assert x.intact(), name
        _check(g["out"].t, g["lse"].t, odt, d, 1 / np.sqrt(d), q, c, table, lens, page)


def test_python_checks():
    c = P.allocate_cache(4, 2, 16, 64, E4M3)
    q = torch.zeros(1, 4, 1, 64, dtype=BF16, device="cuda")
    t, n = _ints([[0, 1]]), _ints([3])
    bad = [lambda: P.decode(q.half(), c, t, n), lambda: P.decode(q, c, t.long(), n),
           lambda: P.decode(q, c, t, n.cpu()), lambda: P.decode(q, c, t, _ints([3, 4])),
           lambda: P.decode(q[..., :32], c, t, n), lambda: P.decode(q[0], c, t, n),
           lambda: P.decode(q, c, t, n, kv_idx=_ints([[[0]]])),
           lambda: P.decode(q, c, t, n, _ints([[[0]]]), _ints([[1]])),
           lambda: P.decode(q, c, t, n, out=torch.zeros(1, 4, 2, 64, device="cuda")),
           lambda: P.decode(q, c, t, n, out_dtype=torch.float16),
           lambda: P.decode(q, P.PagedCache(c.k, c.v), t, n),
           lambda: P.decode(q, P.PagedCache(c.k, c.v[:2], c.k_scale, c.v_scale), t, n),
           lambda: P.decode(q.transpose(2, 3), c, t, n),
           lambda: P.cache_append(c, q, q, t, n),
           lambda: P.cache_read(c, t, n, q[:, :2].expand(1, 2, 8, 64), q[:, :2])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    with pytest.raises(C.SparseAttnError):
        P.decode(torch.zeros(1, 3, 1, 64, dtype=BF16, device="cuda"), c, t, n)
    with pytest.raises(C.SparseAttnError):     # rows that do not start on 16 bytes
        P.decode(torch.zeros(1 * 4 * 64 + 4, dtype=BF16, device="cuda")[4:].view(1, 4, 1, 64), c, t, n)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_a_run_of_them_with_the_block_sparse_call(dtype):
    """A rollout: a prompt is appended and read back for the block-sparse call, which gives
    what it gives on the rows themselves; then tokens are appended one by one, each routed to
    a part of the pages by the framework's own pooling and routing, and decoded."""
    rng = np.random.default_rng(29)
    B, H, d, page, N0, steps = 2, 4, 128, 64, 500, 14
    cap = N0 + steps
    num = B * (-(-cap // page)) + 1
    table = _table(rng, [cap] * B, page, num)
    tab = _ints(table)
    c = P.allocate_cache(num, H, page, d, dtype)
    k, v = _bf16(rng, B, N0, H, d).transpose(1, 2), _bf16(rng, B, N0, H, d).transpose(1, 2)
    flag = _ints([0])
    P.cache_append(c, k, v, tab, _ints([0] * B), err_flag=flag)
    kc, vc = (torch.zeros(B, H, cap, d, dtype=BF16, device="cuda") for _ in range(2))
    P.cache_read(c, tab, _ints([N0] * B), kc, vc, err_flag=flag)
    if dtype == BF16:
        assert torch.equal(kc[:, :, :N0], k) and torch.equal(vc[:, :, :N0], v)
    else:
        for got, x in ((kc, k), (vc, v)):
            code, s = O.quantise(_np(x))
            assert np.array_equal(_np(got)[:, :, :N0], code * s[..., None])
    q = _bf16(rng, B, H, 130, d)
    p = A.Problem(B, H, 130, N0, d, page, 1)
    op = A.BlockSparseAttention(p, "topk", rho=(1, 2))
    kn, vn = kc[:, :, :N0].contiguous(), vc[:, :, :N0].contiguous()
    sparse = op(q, kn, vn)
    op.check()
    # every page kept and order 0: the block-sparse call of one query block is the decode
    dense = A.BlockSparseAttention(A.Problem(B, H, 1, N0, d, page, 0), "topk", rho=(1, 1))
    one = dense(q[:, :, :1].contiguous(), kn, vn)
    got = P.decode(q[:, :, :1], c, tab, _ints([N0] * B))
    assert (one - got).abs().max() <= 1e-2      # the block-sparse call's own bar
    assert sparse.isfinite().all()
    lens = N0
    for step in range(steps):
        kt, vt, qt = (_bf16(rng, B, H, 1, d) for _ in range(3))
        P.cache_append(c, kt, vt, tab, _ints([lens] * B), err_flag=flag)
        P.cache_read(c, tab, _ints([lens + 1] * B), kc, vc, first=_ints([lens] * B), err_flag=flag)
        lens += 1
        pr = A.Problem(B, H, 1, lens, d, page, 0)
        kn, vn = kc[:, :, :lens].contiguous(), vc[:, :, :lens].contiguous()
        t = A.allocate_tables(pr, "cuda")
        A.pool(qt, kn, vn, pr, t)
        keep = -(-pr.nkb // 3)
        idx, cnt = A.allocate_lists(pr, keep, "cuda")
        A.route(pr, t, idx, cnt, "topk", rho=(1, 3))
        out, lse = P.decode(qt, c, tab, _ints([lens] * B), idx, cnt, return_lse=True, err_flag=flag)
        P.check(flag)
        kept = [[idx[b, h, 0, :keep].tolist() for h in range(H)] for b in range(B)]
        assert (cnt == keep).all()
        _check(out, lse, F32, d, 1 / np.sqrt(d), qt, c, table, [lens] * B, page, kept)
