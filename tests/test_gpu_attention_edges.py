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


@pytest.mark.parametrize("at_key", [3, 4, 10, 12, 29, 32 + 5, 64 + 4, 96 + 16])
@pytest.mark.parametrize("seqs", [[(150, 150)], [(6, 9000)]], ids=["whole", "split"])
@pytest.mark.parametrize("how", ["key", "overflow"])
def test_prompt_a_score_of_plus_infinity_is_not_dropped(how, seqs, at_key):
    """inf - inf has no weight: the rows that see the key are NaN, whichever
    column it is in (softmax of +infinity), and say so in their lse."""
    t, (rows, s) = torch.bfloat16, seqs[0]
    so = ref.offsets(seqs)
    q, k, v = ref.vectors(rows, 4, 1, t), ref.vectors(s, 1, 2, t), ref.vectors(s, 1, 3, t)
    at_key += s - rows if rows < 10 and at_key < 4 else 0      # seen by some rows only
    if how == "key":
        q[..., 0], k[at_key, 0, 0] = 1.0, math.inf
    else:
        q[..., 0], k[..., 0], k[at_key, 0, 0] = 2.0 ** 100, 0.0, 2.0 ** 100
    out, lse = binding.Attention("bf16", Hq=4, Hkv=1).prompt(q, k, v, so, lse=True)
    first = max(0, at_key - (s - rows))
    assert torch.isnan(out[first:]).all() and torch.isnan(lse[first:]).all()
    if how == "key" and first > 0:                             # the rows before it are as ever
        k[at_key, 0, 0] = 0.0
        e = ref.prompt_expected(q, k, v, seqs, so)
        for f in ("out", "A", "lse", "dx"):
            setattr(e, f, getattr(e, f)[:first])
        e.check(out[:first], lse[:first], t, ref.half_step(t))


@pytest.mark.parametrize("Hq,selected", [(8, False), (8, True), (16, False), (32, False)])
def test_attend_a_score_of_plus_infinity_is_not_dropped(Hq, selected):
    """Scores that overflow fp32 upwards, in rows with ordinary ones beside them."""
    s, t = 300, torch.bfloat16
    so = ref.offsets([(1, s)])
    cache = binding.Cache4.empty(1, s)
    kv = ref.vectors(s, 1, 2, t)
    kv[..., 0] = 0.0
    kv[77, 0, 0] = 2.0 ** 15
    at = binding.Attention("bf16", Hq=Hq, Hkv=1)
    at.append(cache, kv, ref.vectors(s, 1, 3, t), ref.offsets([(s, s)]))
    q = ref.vectors(1, Hq, 1, t)
    q[..., 0] = 2.0 ** 127
    sel = torch.arange(s, dtype=torch.int32, device="cuda")[None] if selected else None
    out, lse = at.attend(cache, q, so, sel_idx=sel, lse=True)
    assert torch.isnan(out).all() and not (lse == -math.inf).any()
