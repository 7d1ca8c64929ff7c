"""Host-side answers of the attention calls that reach no kernel (no GPU needed)."""
import ctypes

import pytest
import torch

from exact_certified_top_b200 import binding
from test_attention_abi import FAKE, SMALL, _cache, _call, _evict, _rows


@pytest.fixture(scope="module")
def lib():
    return binding.load()


@pytest.mark.parametrize("K", [(1 << 30) + 1, (1 << 31) - 1])
def test_lists_longer_than_a_call_takes_have_no_workspace_size(lib, K):
    """As the call itself answers; the parts' 32-bit lengths would overflow."""
    at = binding.Attention(**SMALL)
    with pytest.raises(binding.DosaError) as e:
        at.attend_workspace_size([[0, 0, 30], [2, 40, 0]], K=K)
    assert e.value.code == 1
    assert _call(lib, "attend", at, sel=FAKE, K=K) == 1
    assert at.attend_workspace_size([[0, 0, 30], [2, 40, 0]], K=1 << 30) > 0
