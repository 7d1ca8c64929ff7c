"""The attention operators at the ends of what they are given: units one behind
another, infinite scores, weights far below a row's largest, value groups of very
different sizes, quotients next to a half.  Bounds: attn_ref."""
import math

import pytest
import torch

import attn_ref as ref
from exact_certified_top_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prompt_many_short_units_behind_one_another(dtype):
    """Units of one key tile, some with one tile of rows and some with two, dozens
    per CTA, alone and from two streams at once."""
    t, Hq, Hkv = ref.DTYPES[dtype], 16, 16
    seqs = [((7 * i) % 130 + 1, (7 * i) % 130 + 1 + (3 * i) % 60) for i in range(400)] + [(256, 300)] * 40
    so = ref.offsets(seqs)
    at = binding.Attention(dtype, Hq=Hq, Hkv=Hkv)
    jobs = []
    for j in range(2):
        q = ref.vectors(int(so[-1, 0]), Hq, 3 * j + 1, t)
        k = ref.vectors(int(so[-1, 1]), Hkv, 3 * j + 2, t)
        v = ref.vectors(int(so[-1, 1]), Hkv, 3 * j + 3, t)
        ws = torch.zeros(at.prompt_workspace_size(so), dtype=torch.uint8, device="cuda")
        jobs.append((q, k, v, ws, torch.cuda.Stream()))
    want = []
    for q, k, v, ws, _ in jobs:
        out, lse = at.prompt(q, k, v, so, lse=True, workspace=ws)
        binding.check_device(ws)
        ref.prompt_expected(q, k, v, seqs, so).check(out, lse, t, ref.half_step(t))
        want.append((out, lse))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for j, (q, k, v, ws, stream) in enumerate(jobs):
            with torch.cuda.stream(stream):
                got[j].append(at.prompt(q, k, v, so, lse=True, workspace=ws))
    torch.cuda.synchronize()
    for j, (_, _, _, ws, stream) in enumerate(jobs):
        with torch.cuda.stream(stream):
            binding.check_device(ws)
        for out, lse in got[j]:
            assert torch.equal(out, want[j][0]) and torch.equal(lse, want[j][1])
