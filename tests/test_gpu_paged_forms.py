"""Decode and read calls at the edges of what they accept, and every form of the decode on the
line of steps, against the fp64 oracle (tolerances as in test_gpu_paged_cache.py)."""
import numpy as np
import pytest
import torch

from free_block_sparse_kv_b200 import paged_cache as P
from free_block_sparse_kv_b200 import sparse_attn as C
from tests.test_gpu_paged_cache import BF16, E4M3, F32, _bf16, _check, _filled, _ints, _table

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
