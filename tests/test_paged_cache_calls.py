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
