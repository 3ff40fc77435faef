"""Decode and read calls at the edges of what they accept, and every form of the decode on the
line of steps, against the fp64 oracle (tolerances as in test_gpu_paged_cache.py)."""
import numpy as np
import pytest
import torch

from free_block_sparse_kv_b200 import paged_cache as P
from free_block_sparse_kv_b200 import sparse_attn as C
from oracle import paged_cache as O
from tests.test_gpu_paged_cache import (BF16, E4M3, F32, _bf16, _bounds, _check, _filled, _ints, _np,
                                        _table)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    C.load_library()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_lists_without_room(dtype):
    """kv_idx [B,H,0]: every list is empty, every output 0 with lse -inf."""
    rng = np.random.default_rng(1)
    B, H, d, page = 3, 2, 64, 16
    c = _filled(rng, 6, H, page, d, dtype)
    q = _bf16(rng, B, 2 * H, 2, d)
    table, lens = _ints([[0, 1], [2, 3], [4, 5]]), _ints([32, 0, 17])
    for cnt in (0, 5):                               # clamped to the room
        for idx, n in ((torch.zeros(B, H, 0, dtype=torch.int32, device="cuda"), _ints(np.full((B, H), cnt))),
                       (torch.zeros(B, H, 1, 0, dtype=torch.int32, device="cuda"), _ints(np.full((B, H, 1), cnt)))):
            out, lse = P.decode(q, c, table, lens, idx, n, return_lse=True,
                                out=torch.full((B, 2 * H, 2, d), 7.0, device="cuda"))
            assert not out.any() and torch.isneginf(lse).all()


def test_read_into_far_more_rows_than_there_are():
    """N is the destination's room, not what is read: up to 2^31 - 1."""
    rng = np.random.default_rng(2)
    H, d, page, n = 2, 64, 16, 21
    for dtype in (BF16, E4M3):
        c = _filled(rng, 2, H, page, d, dtype)
        table, lens = _ints([[1, 0]]), _ints([n])
        want = torch.zeros(2, 1, H, n, d, dtype=BF16, device="cuda")
        P.cache_read(c, table, lens, want[0], want[1])
        got = torch.zeros_like(want)
        C.sparse_attn_cache_read(c.k, c.v, c.k_scale, c.v_scale,
                                 C.SA_CACHE_BF16 if dtype == BF16 else C.SA_CACHE_E4M3, 2, page, table, 2,
                                 2, None, lens, 1, H, (1 << 31) - 1, d, got[0], got[1],
                                 (0, n * d, d), (0, n * d, d), None,
                                 torch.cuda.current_stream().cuda_stream)
        assert torch.equal(got, want)


def test_calls_from_several_threads():
    """Decodes of different shapes from eight host threads at once, each on a stream of its own,
    give what they give one after the other."""
    import threading
    rng = np.random.default_rng(5)
    page, d, jobs = 32, 64, []
    for i in range(8):
        B, H, G, dtype = 1 + i % 3, 2, (1, 10, 20)[i % 3], (BF16, E4M3)[i % 2]
        lens = [int(x) for x in rng.integers(1, 3000, B)]
        num = sum(-(-n // page) for n in lens)
        table = _ints(_table(rng, lens, page, num, spare=3000 * (i // 4)))
        jobs.append((_bf16(rng, B, G * H, 1, d), _filled(rng, num, H, page, d, dtype), table, _ints(lens)))
    want = [P.decode(*j, return_lse=True) for j in jobs]
    torch.cuda.synchronize()
    P._work_bytes.cache_clear()
    got, go = [None] * 8, threading.Barrier(8)

    def work(i):
        stream = torch.cuda.Stream()
        go.wait(timeout=60)
        for _ in range(20):
            got[i] = P.decode(*jobs[i], return_lse=True, stream=stream)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    for (o, l), (o2, l2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(l, l2)


# ------------------------------------------------------------------ every form on the line of steps
LINE = [  # B, Hq, H, T, d, page, lens: 9-16, 17-32 and more rows of a kv head
    (70, 36, 3, 1, 128, 32, [1 + (37 * b * b) % 700 for b in range(70)]),
    (90, 16, 1, 1, 64, 16, [(b * 53) % 1900 if b % 7 else 0 for b in range(90)]),
    (40, 60, 3, 1, 128, 16, [1 + (61 * b * b) % 900 for b in range(40)]),
    (80, 4, 1, 5, 64, 64, [(29 * b) % 1500 + (b % 3) for b in range(80)]),
    (40, 40, 1, 1, 128, 64, [5 + (41 * b * b) % 1100 for b in range(40)]),
    (12, 16, 2, 16, 64, 32, [16 * b + 3 if b % 4 else 2500 + b for b in range(12)]),
    (33, 9, 9, 11, 128, 128, [(b * 97) % 1300 for b in range(33)]),
    # more sequences than a warp scans by itself, 20 rows each
    (300, 20, 1, 1, 64, 16, [(11 * b) % 200 for b in range(300)]),
    # several short segments to a warp's share
    (1500, 20, 2, 1, 128, 16, [(7 * b) % 61 for b in range(1500)]),
    (1200, 40, 2, 1, 128, 16, [(11 * b) % 67 for b in range(1200)]),
    (700, 40, 1, 2, 64, 32, [(13 * b) % 230 for b in range(700)]),
    # a few long segments: whole CTAs for each, CTAs left over
    (1, 3, 3, 1, 128, 64, [40001]),
    (5, 4, 1, 3, 128, 64, [20000, 20011, 19990, 0, 20003]),
    (3, 24, 3, 2, 64, 128, [21000, 21004, 20998]),
    (2, 20, 2, 4, 128, 32, [9003, 9100]),
]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("case", range(len(LINE)))
def test_line(case, dtype):
    """Shares that hold parts of several segments, whole CTAs for a few long ones, row groups
    that read the same keys. A table wider than the lengths keeps the call off the clusters."""
    B, Hq, H, T, d, page, lens = LINE[case]
    rng = np.random.default_rng(100 + case)
    num = sum(-(-n // page) for n in lens) + 1
    table = _table(rng, lens, page, num, spare=60000 // page)
    code = C.SA_CACHE_BF16 if dtype == BF16 else C.SA_CACHE_E4M3
    c = _filled(rng, num, H, page, d, dtype)
    q = _bf16(rng, B, Hq, T, d)
    ks, vs = (None if x is None else _np(x) for x in (c.k_scale, c.v_scale))
    scale = 1 / np.sqrt(d)
    want, lse, vmax, qk = O.decode(_np(q), _np(c.k), _np(c.v), ks, vs, table, lens, page, scale)
    empty = np.isneginf(lse)
    for out_dtype, odt in ((F32, C.SA_OUT_F32), (BF16, C.SA_OUT_BF16)):
        assert C.sparse_attn_decode_work_bytes(B, Hq, H, T, d, code, page, table.shape[1], -1, odt) > 0
        flag = _ints([0])
        out, got_lse = P.decode(q, c, _ints(table), _ints(lens), out_dtype=out_dtype, return_lse=True,
                                err_flag=flag)
        P.check(flag)
        tol, ltol = _bounds(dtype, out_dtype, d, scale, want, lse, vmax, qk)
        assert (np.abs(_np(out) - want) <= tol).all()
        assert np.array_equal(np.isneginf(_np(got_lse)), empty) and not _np(out)[empty].any()
        assert (np.abs(_np(got_lse)[~empty] - lse[~empty]) <= ltol[~empty]).all()
        assert torch.equal(out, P.decode(q, c, _ints(table), _ints(lens), out_dtype=out_dtype))


@pytest.mark.parametrize("out_dtype,Hq,H,T,d,n,spare", [
    (BF16, 9, 9, 1, 128, 3001, 90000), (BF16, 20, 10, 1, 64, 2500, 90000), (BF16, 14, 14, 3, 128, 17, 90000),
    (BF16, 16, 16, 1, 128, 30001, 100), (F32, 24, 24, 1, 128, 1501, 90000), (F32, 28, 14, 4, 64, 2000, 90000),
    (BF16, 288, 32, 1, 128, 700, 60000), (F32, 34, 34, 11, 64, 650, 60000), (BF16, 66, 33, 12, 128, 333, 60000)])
def test_heads_of_one_sequence_in_clusters(out_dtype, Hq, H, T, d, n, spare):
    """bf16 rows of one sequence whose heads hold most SMs: a cluster each, at any length. (More
    than 31 clusters of four CTAs need not fit at once, which the device says: 34 did not, and
    run on the line.)"""
    rng = np.random.default_rng(H)
    page, lens = 64, [n]
    num = -(-n // page) + 1
    table = _table(rng, lens, page, num, spare=spare // page)
    odt = C.SA_OUT_F32 if out_dtype == F32 else C.SA_OUT_BF16
    if H <= 31:
        assert C.sparse_attn_decode_work_bytes(1, Hq, H, T, d, C.SA_CACHE_BF16, page, table.shape[1], -1, odt) == 0
    c = _filled(rng, num, H, page, d, BF16)
    q = _bf16(rng, 1, Hq, T, d)
    out, lse = P.decode(q, c, _ints(table), _ints(lens), out_dtype=out_dtype, return_lse=True)
    _check(out, lse, out_dtype, d, 1 / np.sqrt(d), q, c, table, lens, page)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,Hq,H,T,d,page,lens,cap", [
    (30, 24, 2, 1, 128, 32, [(b * 71) % 1400 for b in range(30)], 30),
    (20, 60, 3, 1, 64, 16, [(b * 113) % 1500 for b in range(20)], 90),
    (24, 12, 2, 6, 128, 64, [(b * 89) % 1300 for b in range(24)], 20)])
def test_line_kept_pages(B, Hq, H, T, d, page, lens, cap, dtype):
    rng = np.random.default_rng(cap)
    num = sum(-(-n // page) for n in lens) + 1
    table = _table(rng, lens, page, num, spare=3)
    c = _filled(rng, num, H, page, d, dtype)
    q = _bf16(rng, B, Hq, T, d)
    wide = cap + 40000 // page                       # lists with much room: off the clusters
    idx, cnt = np.full((B, H, wide), -1), np.zeros((B, H), int)
    kept = [[[] for _ in range(H)] for _ in range(B)]
    for b in range(B):
        pages = -(-lens[b] // page)
        for h in range(H):
            m = int(rng.integers(0, min(cap, pages) + 1))
            kept[b][h] = sorted(rng.choice(pages, m, replace=False).tolist()) if m else []
            idx[b, h, :m], cnt[b, h] = kept[b][h], m
    code = C.SA_CACHE_BF16 if dtype == BF16 else C.SA_CACHE_E4M3
    assert C.sparse_attn_decode_work_bytes(B, Hq, H, T, d, code, page, table.shape[1], wide) > 0
    out, lse = P.decode(q, c, _ints(table), _ints(lens), _ints(idx), _ints(cnt), return_lse=True)
    _check(out, lse, F32, d, 1 / np.sqrt(d), q, c, table, lens, page, kept)
