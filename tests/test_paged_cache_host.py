"""The paged cache without a GPU: the oracle's 8-bit row format pinned against torch's e4m3
type and its own definition, the oracle's decode against closed forms, and the refusals of
the three entry points (all found on the host)."""
import ctypes

import numpy as np
import pytest
import torch

from free_block_sparse_kv_b200 import build
from free_block_sparse_kv_b200 import paged_cache as P
from free_block_sparse_kv_b200 import sparse_attn as C
from oracle import paged_cache as O


@pytest.fixture(scope="module")
def lib():
    build.build()
    return C.load_library()


def test_e4m3_values_and_rounding_match_torch():
    codes = np.arange(256)
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_value(codes), want, equal_nan=True)
    rng = np.random.default_rng(1)
    grid = np.sort(want[np.isfinite(want)])
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 1e-2, 4000), grid,
                        (grid[1:] + grid[:-1]) / 2]).astype(np.float32)   # ties among them
    got = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_round(y), got)


def test_row_scale_is_the_smallest_power_of_two():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((500, 64)) * np.exp2(rng.integers(-100, 100, (500, 1)))
    x[0] = 0
    x[1, 0] = 448.0 * 2.0 ** 5
    x[1, 1:] = 1
    x[2] = np.nextafter(448.0, 449)
    x[3, 0] = np.inf
    x[4] = 2.0 ** -133
    s = O.row_scale(x)
    a = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
    assert s[0] == 1 and s[1] == 32 and s[2] == 2 and s[4] == 2.0 ** -126
    big = a > 448 * 2.0 ** -126
    assert (a[big] <= 448 * s[big]).all() and (a[big] > 448 * s[big] / 2).all()
    code, s = O.quantise(x[5:])
    err = np.abs(code * s[:, None] - x[5:])
    # half a step: 2^-4 of a normal value, 2^-10 of the scale below
    assert (err <= np.maximum(np.abs(x[5:]) * 2.0 ** -4, s[:, None] * 2.0 ** -10)).all()


def test_oracle_decode_closed_forms():
    rng = np.random.default_rng(3)
    P_, H, page, d = 5, 2, 16, 64
    k, v = rng.standard_normal((2, P_, H, page, d))
    table = [[3, 1, 4], [0, 2, -1]]
    q = rng.standard_normal((2, 4, 2, d))
    out, lse, _, _ = O.decode(q, k, v, None, None, table, [1, 0], page, 0.1)
    # one cached token, two new ones: row 0 attends nothing, row 1 the token itself
    assert not out[0, :, 0].any() and np.isneginf(lse[0, :, 0]).all()
    assert np.allclose(out[0, 2, 1], v[3, 1, 0])
    assert np.allclose(lse[0, 2, 1], 0.1 * q[0, 2, 1] @ k[3, 1, 0])
    assert not out[1].any() and np.isneginf(lse[1]).all()
    # equal logits: the mean of the values
    out, lse, _, _ = O.decode(q * 0, k, v, None, None, table, [37, 20], page, 0.1)
    want = np.concatenate([v[3, 1], v[1, 1], v[4, 1, :5]]).mean(0)
    assert np.allclose(out[0, 3, 1], want) and np.allclose(lse[0, 3, 1], np.log(37))
    # kept pages partition the keys: partial results merge by their lse
    full, l0, _, _ = O.decode(q, k, v, None, None, table, [37, 20], page, 0.1)
    parts = [O.decode(q, k, v, None, None, table, [37, 20], page, 0.1, kept=[[[a]] * H] * 2)[:2]
             for a in range(3)]
    w = np.stack([np.exp(l - l0) for _, l in parts])
    assert np.allclose(w.sum(0), 1) and np.allclose(sum(x[..., None] * o for x, (o, _) in
                                                        zip(w, parts)), full)


def test_refusals(lib):
    buf = (ctypes.c_char * 4096)()
    base = ctypes.addressof(buf)
    p = base + (-base) % 16
    st = (4096, 128, 128)

    def app(k=p, v=p, ks=st, vs=st, B=1, H=1, T=4, d=128, table=p, w=4, ts=4, start=p, count=p,
            kp=p, vp=p + 16, sk=p, sv=p + 16, dt=1, n=4, page=16, flag=None):
        C.sparse_attn_cache_append(k, v, ks, vs, B, H, T, d, table, w, ts, start, count, kp, vp, sk,
                                   sv, dt, n, page, flag, 0)

    def read(kp=p, vp=p + 16, sk=p, sv=p + 16, dt=1, n=4, page=16, table=p, w=4, ts=4, first=p,
             lens=p, B=1, H=1, N=64, d=128, k=p, v=p + 16, ks=st, vs=st, flag=None):
        C.sparse_attn_cache_read(kp, vp, sk, sv, dt, n, page, table, w, ts, first, lens, B, H, N, d,
                                 k, v, ks, vs, flag, 0)

    def dec(q=p, qs=st, B=1, Hq=2, H=1, T=1, d=128, kp=p, vp=p + 16, sk=p, sv=p + 16, dt=1, n=4,
            page=16, table=p, w=4, ts=4, lens=p, idx=None, cnt=None, cap=0, scale=0.1, work=p,
            out=p, odt=0, lse=None, flag=None):
        C.sparse_attn_decode(q, qs, B, Hq, H, T, d, kp, vp, sk, sv, dt, n, page, table, w, ts, lens,
                             idx, cnt, cap, scale, work, out, odt, lse, flag, 0)

    common = [dict(d=96), dict(B=-1), dict(H=-1), dict(B=300, H=300), dict(dt=2), dict(page=48),
              dict(page=8), dict(page=512), dict(n=-1), dict(w=-1), dict(w=1 << 28, page=16),
              dict(B=2, ts=3), dict(kp=None), dict(vp=p + 8), dict(vp=p), dict(sk=None),
              dict(sv=p + 1), dict(sv=p), dict(table=None), dict(table=p + 2), dict(flag=p + 2)]
    rows = [dict(k=None), dict(v=p + 8), dict(ks=(4, 128, 128)), dict(vs=(4096, 128, -128))]
    cases = [(app, kw) for kw in common + rows + [
        dict(T=-1), dict(start=None), dict(start=p + 2), dict(count=p + 1),
        dict(H=65535, T=1 << 20)]]
    cases += [(read, kw) for kw in common + rows + [dict(N=-1), dict(lens=None), dict(lens=p + 2),
                                                    dict(first=p + 2), dict(v=p)]]
    cases += [(dec, kw) for kw in common if kw != dict(H=-1)]
    cases += [(dec, kw) for kw in [
        dict(T=0), dict(T=17), dict(Hq=3, H=2), dict(Hq=-1), dict(H=0), dict(B=1 << 15, Hq=1 << 16),
        dict(q=None), dict(q=p + 8), dict(qs=(0, 0, 4)), dict(out=None), dict(out=p + 8),
        dict(odt=2), dict(lens=None), dict(lens=p + 2), dict(scale=float("inf")),
        dict(scale=float("nan")), dict(idx=p), dict(cnt=p), dict(idx=p, cnt=p, cap=-1),
        dict(idx=p, cnt=p, cap=1 << 27),
        dict(idx=p + 2, cnt=p, cap=1), dict(idx=p, cnt=p + 2, cap=1), dict(lse=p + 2)]]
    for fn, kw in cases:
        with pytest.raises(C.SparseAttnError) as e:
            fn(**kw)
        assert e.value.code == C.SA_ERR_INVALID, (fn.__name__, kw, str(e.value))
    for kw in (dict(T=0), dict(d=80), dict(Hq=3, Hkv=2), dict(dt=2), dict(page=24), dict(width=-1),
               dict(width=1 << 28), dict(cap=-2), dict(cap=1 << 28), dict(odt=3)):
        a = dict(B=1, Hq=2, Hkv=1, T=1, d=128, dt=1, page=16, width=4, cap=-1, odt=0) | kw
        with pytest.raises(C.SparseAttnError) as e:
            C.sparse_attn_decode_work_bytes(*a.values())
        assert e.value.code == C.SA_ERR_INVALID
    assert C.sparse_attn_decode_work_bytes(0, 2, 1, 1, 128, 1, 16, 4) == 0
    # empty calls look at no buffer
    app(B=0, k=None, v=None, kp=None, table=None, start=None)
    app(T=0, k=None, v=None, kp=None, table=None, start=None)
    read(N=0, k=None, v=None, kp=None, table=None, lens=None)
    dec(B=0, q=None, out=None, lens=None, kp=None, table=None)
    dec(Hq=0, H=0, q=None, out=None, lens=None, kp=None, table=None)


def test_python_refusals_and_allocation():
    c = P.allocate_cache(3, 2, page=16, d=64, dtype=torch.float8_e4m3fn, device="cpu")
    assert c.k.shape == (3, 2, 16, 64) and c.k_scale.dtype == torch.float8_e8m0fnu
    assert P.allocate_cache(3, 2, device="cpu").k_scale is None
    with pytest.raises(ValueError):
        P.allocate_cache(3, 2, dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError):
        P.allocate_cache(3, 2, page=48, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: P.cache_append(c, x, x, i[None], i), lambda: P.decode(x, c, i[None], i),
                 lambda: P.cache_read(c, i[None], i, x, x.clone())):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    # rows that share memory are no destination
    y = torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16)
    P._apart("k", y)
    P._apart("k", y.transpose(1, 2).contiguous().transpose(1, 2))
    P._apart("k", y[:, :, ::2])
    for bad in (y[:1].expand(2, 3, 8, 64), y[:, :, :1].expand(2, 3, 8, 64),
                torch.as_strided(y, (2, 3, 8, 64), (512, 512, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            P._apart("k", bad)
