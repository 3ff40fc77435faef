"""Host side of the paged cache and of what shares its error flag (no GPU needed)."""
import pytest
import torch

from free_block_sparse_kv_b200 import attention as A
from free_block_sparse_kv_b200 import paged_cache as P
from free_block_sparse_kv_b200 import sparse_attn as C


@pytest.mark.parametrize("flag,code", [
    (C.SA_FLAG_RANGE, C.SA_ERR_RANGE), (C.SA_FLAG_INDEX, C.SA_ERR_INDEX), (1, C.SA_ERR_TIMEOUT),
    (1 << 14, C.SA_ERR_TIMEOUT), (C.SA_FLAG_INDEX | 2, C.SA_ERR_INDEX),
    (C.SA_FLAG_INDEX | C.SA_FLAG_RANGE, C.SA_ERR_RANGE)])
def test_flag_of_the_block_sparse_call(flag, code):
    """One flag passed through append, read, pool and forward: a bad page number is no timeout."""
    op = A.BlockSparseAttention.__new__(A.BlockSparseAttention)
    op.err_flag = torch.tensor([flag], dtype=torch.int32)
    with pytest.raises(C.SparseAttnError) as e:
        op.check()
    assert e.value.code == code
    if flag & C.SA_FLAG_INDEX:
        with pytest.raises(C.SparseAttnError) as e:
            P.check(op.err_flag)
        assert e.value.code == C.SA_ERR_INDEX
    op.err_flag.zero_()
    op.check()
    P.check(op.err_flag)


def test_destinations_whose_rows_do_not_overlap():
    """Every second row (or head) of a buffer with an odd number of them is a destination; the
    exact check is against the addresses themselves."""
    def overlaps(x):
        b, h, t = torch.meshgrid(*(torch.arange(n) for n in x.shape[:3]), indexing="ij")
        sb, sh, st, _ = x.stride()
        at = (b * sb + h * sh + t * st).reshape(-1).sort().values
        return bool((at.diff() < x.shape[3]).any())

    y = torch.zeros(3, 5, 7, 64, dtype=torch.bfloat16)
    fine = [y[:, :, ::2], y[:, ::2], y[::2, ::2, ::2], y[:, :, ::3], y.transpose(1, 2)[:, ::2],
            torch.zeros(2, 7, 3, 5, 64, dtype=torch.bfloat16)[:, :, 1].transpose(1, 2),
            y[:1, :, 1::2],
            y[:, :, :0], y[:0], y[:, :, 3:4]]
    for x in fine:
        assert not overlaps(x)
        P._apart("k", x)
    bad = [y[:1].expand(2, 5, 7, 64), torch.as_strided(y, (2, 3, 8, 64), (64, 512, 64, 1)),
           torch.as_strided(y, (1, 3, 4, 64), (0, 192, 64, 1)), torch.as_strided(y, (1, 1, 4, 64), (0, 0, 56, 1))]
    for x in bad:
        assert overlaps(x)
        with pytest.raises(ValueError, match="overlap"):
            P._apart("k", x)


def test_addresses_of_integer_types():
    """Every entry point takes device addresses as integers, subclasses of int among them."""
    class Address(int):
        pass

    t = torch.zeros(3)
    assert C._ptr(Address(64)) == 64 and C._ptr(64) == 64 and C._ptr(None) is None
    assert C._ptr(t) == t.data_ptr()
    C.sparse_attn_cache_append(Address(0), Address(0), (0, 0, 0), (0, 0, 0), 0, 1, 1, 64, Address(0), 1, 1,
                               Address(0), None, Address(0), Address(0), None, None, C.SA_CACHE_BF16, 1, 16,
                               None, Address(0))
