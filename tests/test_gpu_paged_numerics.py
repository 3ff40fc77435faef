"""Decode over a paged cache where numbers are hard: values of very different sizes, long sums,
logits far from zero. Each tolerance is derived where it is used (u = 2^-24)."""
import numpy as np
import pytest
import torch

from free_block_sparse_kv_b200 import paged_cache as P
from free_block_sparse_kv_b200 import sparse_attn as C
from oracle import paged_cache as O
from tests.test_gpu_paged_cache import BF16, DROP, E4M3, F32, _bf16, _bounds, _check, _ints, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    C.load_library()


def _cache(k, v, page, dtype):
    """The rows k, v [1,H,n,d] in the pages of one sequence, and its table."""
    _, H, n, d = k.shape
    num = -(-n // page)
    c = P.allocate_cache(num, H, page, d, dtype)
    table = [list(range(num))[::-1]]
    P.cache_append(c, k, v, _ints(table), _ints([0]))
    return c, table


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("n,page", [(40, 16), (3000, 64)])
def test_values_near_the_smallest(n, page, out_dtype):
    """Values of 2^-112 and 2^-118 (8-bit rows hold them with scales down to 2^-126) are
    attended like any others: compared on their own scale. What fp32 itself drops there is
    2^-149, 2^-31 of the smaller ones."""
    rng = np.random.default_rng(n)
    H, d = 2, 128
    k, v = _bf16(rng, 1, H, n, d), _bf16(rng, 1, H, n, d)
    v = (v.float() * torch.tensor([2.0 ** -112, 2.0 ** -118], device="cuda").view(1, 2, 1, 1)).to(BF16)
    q = _bf16(rng, 1, 2 * H, 1, d)
    for dtype in (E4M3, BF16):
        c, table = _cache(k, v, page, dtype)
        out, lse = P.decode(q, c, _ints(table), _ints([n]), out_dtype=out_dtype, return_lse=True)
        _check(out, lse, out_dtype, d, 1 / np.sqrt(d), q, c, table, [n], page)
        assert out.any(-1).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n,Hq", [(200, 1), (9001, 12), (300, 20)])
def test_values_near_the_largest(n, Hq, dtype):
    """V of 3e38 at keys that outweigh what came before them by up to 2^4: the product of a
    weight and a value must not overflow where their share of the output does not."""
    rng = np.random.default_rng(3)
    d, page = 128, 32
    k = torch.zeros(1, 1, n, d, dtype=BF16, device="cuda")
    v = _bf16(rng, 1, 1, n, d)
    q = torch.zeros(1, Hq, 1, d, dtype=BF16, device="cuda")
    q[..., 0] = 1
    for i, bits in ((n // 2, 1.0), (n - 20, 3.5)):
        k[0, 0, i, 0] = bits * np.log(2)
        v[0, 0, i] = 0
        v[0, 0, i, ::5] = 3.0e38 * (1 if i % 2 else -1)
    c, table = _cache(k, v, page, dtype)
    out, lse = P.decode(q, c, _ints(table), _ints([n]), scale=1.0, return_lse=True)
    assert out.isfinite().all()
    _check(out, lse, F32, d, 1.0, q, c, table, [n], page)


@pytest.mark.parametrize("B,G,T,H,pages", [(8, 1, 1, 4, 3200), (8, 16, 1, 4, 3200), (4, 8, 4, 2, 9000)])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_long_sums(B, G, T, H, pages, dtype):
    """Hundreds of steps a warp over columns of V that each hold one value: the output is that
    value. A step's products are a short chain on the tensor cores (their sums lose at most
    2^-23 each, all to one side: 4 in a row at most), and the steps are added to nearest: S of
    them into a sum that grows evenly are off by u sqrt(S / 9) in the mean square, the sum of
    weights as much; six times that. The pieces of a weight keep 2^-22 of it."""
    rng = np.random.default_rng(G + T)
    d, page, num = 128, 256, 24
    n = pages * page
    c = P.allocate_cache(num, H, page, d, dtype)
    k = _bf16(rng, 1, H, num * page, d)
    col = _bf16(rng, 1, H, 1, d).abs() + 0.5        # of one exponent's size: 8 bits keep 4 of them
    col = col.to(E4M3).to(BF16)
    rows = list(range(num))
    P.cache_append(c, k, col.expand(1, H, num * page, d), _ints([rows]), _ints([0]))
    table = _ints(rng.integers(0, num, (B, pages)))  # pages that are only read may be shared
    q = _bf16(rng, B, G * H, T, d)
    out, lse = P.decode(q, c, table, _ints([n] * B), return_lse=True)
    want = torch.empty(1, H, num * page, d, dtype=BF16, device="cuda")
    P.cache_read(c, _ints([rows]), _ints([num * page]), torch.empty_like(want), want)
    want = want[:, :, :1].double().repeat_interleave(G, 1)
    # steps of a warp: the line has at least 8 warps on each of at least 132 SMs
    steps = B * H * -(-G * T // 32) * n * d * (1 if dtype == E4M3 else 2) / 4096 / (132 * 8)
    tol = 2.0 ** -22 + 4 * 2.0 ** -23 + 6 * 2.0 ** -24 * np.sqrt(2 * steps / 9)
    assert steps > 500
    err = ((out.double() - want) / want).abs().max().item()
    assert err <= tol, (err, tol)


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n,page,T,G", [(50, 16, 1, 1), (700, 64, 1, 12), (5000, 32, 3, 9), (9000, 128, 1, 2)])
def test_an_outlier_in_one_column(n, page, T, G, dtype, out_dtype):
    """One V row holds an outlier in column 0, 2^3 to 2^100 times the other rows, and zeros
    beside it: the other columns are a mix of the other rows, at their own size. Their error is
    that of the weights (the same derivation as for whole rows) times the column's largest
    value; what 16-bit pieces drop of a weight relates to the weight at its row's own scale."""
    H, d = 1, 128
    scale = 1 / np.sqrt(d)
    for place, ratio in ((0, 3), (n // 2, 8), (n - T - 1, 20), (n // 3, 36), (n // 2, 100)):
        rng = np.random.default_rng(ratio)
        k, v = _bf16(rng, 1, H, n, d, scale=0.3), _bf16(rng, 1, H, n, d)
        v[:, :, place] = 0
        v[:, :, place, 0] = 2.0 ** ratio
        q = _bf16(rng, 1, G * H, T, d)
        c, table = _cache(k, v, page, dtype)
        out, lse = P.decode(q, c, _ints(table), _ints([n]), out_dtype=out_dtype, return_lse=True)
        ks, vs = (None if x is None else _np(x) for x in (c.k_scale, c.v_scale))
        want, wlse, _, qk = O.decode(_np(q), _np(c.k), _np(c.v), ks, vs, table, [n], page, scale)
        vmax = np.ones_like(qk)
        tol, _ = _bounds(dtype, F32, d, scale, want, wlse, vmax, qk)     # relative to |v|
        if out_dtype == BF16:
            tol = tol + 2 * DROP[dtype, BF16]
        held = O.rows(_np(c.v), vs, table[0], n, 0, page)
        top = np.abs(held).max(0)
        tol = tol * top
        if out_dtype == BF16:
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        err = np.abs(_np(out) - want)
        assert (err <= tol).all(), (ratio, (err / tol).max((0, 1, 2))[:4], (err / tol)[..., 1:].max())


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("Hq", [2, 14, 40])
def test_one_key_gives_its_value(Hq, dtype):
    """A row that attends one key gets that key's V, at sizes from 2^-100 to 2^100: the weight's
    pieces keep 2^-22 of it, and weight, reciprocal and their products round a few times (8u)."""
    rng = np.random.default_rng(Hq)
    B, H, d, page = 64, 2, 128, 16
    c = P.allocate_cache(B, H, page, d, dtype)
    q, k = _bf16(rng, B, Hq, 1, d), _bf16(rng, B, H, 1, d)
    size = torch.exp2(torch.linspace(-100, 100, B, device="cuda").round()).view(B, 1, 1, 1)
    v = (_bf16(rng, B, H, 1, d).float() * size).to(BF16)
    table, lens = _ints(np.arange(B)[:, None]), _ints([1] * B)
    P.cache_append(c, k, v, table, _ints([0] * B))
    back = torch.empty(2, B, H, 1, d, dtype=BF16, device="cuda")
    P.cache_read(c, table, lens, back[0], back[1])
    out, _ = P.decode(q, c, table, lens, return_lse=True)
    want = back[1].double().repeat_interleave(Hq // H, 1)
    assert ((out.double() - want).abs() <= (2.0 ** -22 + 8 * 2.0 ** -24) * want.abs()).all()


@pytest.mark.parametrize("T,G", [(2, 1), (7, 2), (16, 2)])
def test_scales_of_unseen_tokens(T, G):
    """8-bit rows: whatever a new token's scales are (NaN, the largest, the smallest) and its codes
    (zeros, NaN), rows that do not attend it keep their bits."""
    from tests.test_gpu_paged_cache import _filled, _table
    rng = np.random.default_rng(T)
    B, H, d, page, lens = 3, 2, 64, 16, [90, 16, T]
    num = sum(-(-n // page) for n in lens) + 1
    table = _table(rng, lens, page, num)
    c = _filled(rng, num, H, page, d, E4M3)
    q = _bf16(rng, B, G * H, T, d)
    tab, ln = _ints(table), _ints(lens)
    for odt in (F32, BF16):
        clean, clean_lse = P.decode(q, c, tab, ln, out_dtype=odt, return_lse=True)
        for byte, code in ((255, None), (254, None), (0, None), (127, None), (127, 0), (255, 0x7F), (100, 0xFF)):
            held = [x.view(torch.uint8).clone() for x in (c.k_scale, c.v_scale, c.k, c.v)]
            for b in range(B):
                pos = lens[b] - 1
                for x in (c.k_scale, c.v_scale):
                    x.view(torch.uint8)[table[b][pos // page], :, pos % page] = byte
                for x in (c.k, c.v) if code is not None else ():
                    x.view(torch.uint8)[table[b][pos // page], :, pos % page] = code
            out, lse = P.decode(q, c, tab, ln, out_dtype=odt, return_lse=True)
            assert torch.equal(out[:, :, :T - 1], clean[:, :, :T - 1])
            assert torch.equal(lse[:, :, :T - 1], clean_lse[:, :, :T - 1])
            assert (byte != 255) or out[:, :, T - 1].isnan().all()
            for x, y in zip((c.k_scale, c.v_scale, c.k, c.v), held):
                x.view(torch.uint8).copy_(y)
