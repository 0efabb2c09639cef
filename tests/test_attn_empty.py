"""A batch without sequences in the attention-layer calls (no GPU needed, nothing is launched): the C ABI
takes what the binding passes for empty tensors, whose address is NULL."""
import pytest
import torch

import test_attn_oracle as R

K = R.K


@pytest.mark.parametrize("call", [R.write, R.read, R.attn])
def test_no_sequences_is_a_no_op(call):
    for width in (0, 16):
        assert call(kc=R.cache(table=None, width=width), N=0, T=0) == K.KDA_OK and R.err() == ""
    assert call(kc=R.cache(table=None), N=1, T=0) == K.KDA_ERR_ARG and "table" in R.err()
    assert call(kc=R.cache(width=0), N=1, T=0) == K.KDA_ERR_ARG and "width" in R.err()
    assert call(kc=R.cache(table=None), N=0, T=1) == K.KDA_ERR_ARG


def test_empty_tensors_have_no_address():
    assert torch.zeros((0, 5), dtype=torch.int32).data_ptr() == 0
    form = R.K.KVCache(torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2, 16, 64), dtype=torch.uint8),
                       torch.ones(3, 2), torch.ones(3, 2), torch.zeros((0, 5), dtype=torch.int32)).form()
    assert K._cache_sizes(form, 0, 2, 64, -1) == (3, 16, 5)
