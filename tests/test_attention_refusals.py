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


def test_evictions_that_keep_nothing_are_checked_like_others(lib):
    """A result of no columns needs no address, and wrong spans stay wrong."""
    at = binding.Attention(**SMALL)
    nothing = [[0, 40, 0, 0], [40, 0, 3, 0]]
    assert _evict(lib, at, nothing, kept=None, ld=0) == 0
    assert _evict(lib, at, nothing, kept=FAKE, ld=0) == 0
    assert _evict(lib, at, [[0, 40, 0, 20]], kept=None, ld=0) == 1
    assert _evict(lib, at, nothing, kept=None, ld=0, first=1) == 1     # more than keep
    for spans in ([[0, 65, 0, 0]], [[-1, 4, 0, 0]], [[0, -4, 0, 0]], [[0, 4, 0, -2]], [[0, 4, 65, 0]]):
        assert _evict(lib, at, spans, kept=None, ld=0) == 1, spans
    assert _evict(lib, at, nothing, kept=None, ld=4) == 1
    assert _evict(lib, at, nothing, kept=None, ld=-1) == 1


@pytest.fixture
def host_as_device(monkeypatch):
    """Host tensors pass for the current device's: what is refused is refused
    before anything would be launched."""
    monkeypatch.setattr(binding.torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(binding, "_stream", lambda dev=None: None)


def test_the_binding_checks_evictions_that_keep_nothing(host_as_device):
    at = binding.Attention(Hq=8, Hkv=2)
    src, dst = (binding.Cache4.empty(2, 64, device="cpu") for _ in range(2))
    assert at.evict(src, dst, [[0, 40, 0, 0]]).shape == (1, 0)
    for spans, first in (([[0, 65, 0, 0]], 0), ([[0, 40, 0, 0]], 1), ([[0, 4, 0, -2]], 0)):
        with pytest.raises(binding.DosaError) as e:
            at.evict(src, dst, spans, first=first)
        assert e.value.code == 1


@pytest.mark.parametrize("op", ["prompt", "attend"])
def test_workspaces_with_gaps_are_refused(host_as_device, op):
    """The call takes a workspace as one run of bytes: those between a view's
    elements, and behind the last, are someone else's."""
    at = binding.Attention(Hq=8, Hkv=2)
    so = [[0, 0, 29], [1, 30, 0]]
    q, k = torch.zeros((1, 8, 128), dtype=torch.bfloat16), torch.zeros((30, 2, 128), dtype=torch.bfloat16)
    cache = binding.Cache4.empty(2, 30, device="cpu")
    call = (lambda ws: at.prompt(q, k, k, so, workspace=ws)) if op == "prompt" else \
        (lambda ws: at.attend(cache, q, so, workspace=ws))
    size = at.prompt_workspace_size(so) if op == "prompt" else at.attend_workspace_size(so)
    room = torch.zeros(4 * size, dtype=torch.uint8)
    for ws in (room[::2], room.view(4, size)[:, :size // 2], room.view(-1, 2)[:, 0]):
        with pytest.raises(ValueError, match="contiguous"):
            call(ws)
    with pytest.raises(binding.DosaError) as e:            # bytes count, not elements
        call(torch.zeros(size // 4 - 1, dtype=torch.float32))
    assert e.value.code in (1, 3)


def test_recorded_weights_of_rows_that_out_replaces_are_refused(lib):
    """Over every key the weights read the query rows again behind the result."""
    at = binding.Attention(**SMALL)
    assert _call(lib, "attend", at, add=1) == 1                        # out is q
    assert _call(lib, "attend", at, add=1, out=_rows(ptr=FAKE + (1 << 20)), ws=None) == 1
    assert _call(lib, "attend", at, add=1, out=_rows(ptr=FAKE + (1 << 20)), n=100) == 3
    none = [[0, 0, 0], [0, 40, 0]]
    assert _call(lib, "attend", at, none, add=1) == 0                  # no rows to replace
