"""The attention operators at the ends of what they are given: units one behind
another, infinite scores, weights far below a row's largest, value groups of very
different sizes, quotients next to a half.  Bounds: attn_ref."""
import math
from fractions import Fraction

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


def _cache_of(k, v):
    """A cache whose slots hold rows k, v [n, Hkv, D]."""
    cache = binding.Cache4.empty(k.shape[1], k.shape[0])
    for kind, x in (("k", k), ("v", v)):
        codes, params = ref.quantise(x, kind)
        getattr(cache, kind + "_codes").copy_(codes)
        getattr(cache, kind + "_params").copy_(params)
    return cache


def _largest_weight(cache, q, e):
    """[rows, Hq, 1]: each row's largest weight (of every key the last row sees)."""
    G = q.shape[1] // cache.Hkv
    sc, mn = ref.unpack(cache.k_codes, cache.k_params, "k")
    x = torch.einsum("rhgd,hnd->rhgn", q.double().unflatten(1, (cache.Hkv, G)), sc + mn)
    top = x.amax(-1).flatten(1) / math.sqrt(ref.D)
    return torch.exp(top - e.lse).clamp(max=1.0)[..., None]


def _check_attend(cache, q, dtype, sel=None, weights=False):
    """Against the definition.  Weights enter the value product rounded to fp16 with
    the row's largest at 2^12 or more: 2^-11 each, or half a step of 2^-24 below
    2^-14, i.e. 2^-37 of the largest weight, times |min|.  Times the scale the same,
    the scale of its group's largest being 1/2 or more and codes up to 15: 2^-36 of
    the largest weight times 15 scales."""
    s = cache.capacity
    Hq, Hkv, rows = q.shape[1], cache.Hkv, q.shape[0]
    so = ref.offsets([(rows, s)])
    at = binding.Attention(dtype, Hq=Hq, Hkv=Hkv)
    out, lse = at.attend(cache, q, so, sel_idx=sel, lse=True, weights=weights)
    e, w, wt = ref.cache_expected(cache, q, [(rows, s)], so, sel)
    n = s if sel is None else sel.shape[1]
    part = cache.v_params.double().abs().amax(1)                       # [Hkv, 4, 2]
    far = n * 2.0 ** -36 * (15 * part[..., 0] + part[..., 1])
    far = far.repeat_interleave(32, 1).repeat_interleave(Hq // Hkv, 0) * _largest_weight(cache, q, e)
    u = ref.half_step(ref.DTYPES[dtype])
    tol = u * e.out.abs() + (2.0 ** -11 + 2 * e.dx[..., None] + 2.0 ** -18) * e.A + far
    tol = tol + torch.finfo(ref.DTYPES[dtype]).smallest_normal * 2 * u
    err = (out.double() - e.out).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse.double() - e.lse).abs() <= e.dx + 2.0 ** -20 * (1 + e.lse.abs())).all()
    if weights:
        assert ((cache.weight.double() - w).abs() <= wt + 2.0 ** -23 * w * (Hq + 8)).all()
    return out, e


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,rows,selected", [(8, 1, False), (8, 1, True), (16, 1, False), (16, 1, True),
                                              (32, 1, False), (8, 4, False), (32, 1, True)])
@pytest.mark.parametrize("gap", [20.5, 24.5, 25.9, 30.6])
def test_attend_many_keys_far_below_the_maximum_add_up(dtype, Hq, rows, selected, gap):
    """One key in 16 at the maximum with values of zero, so that every warp has some;
    the others 2^-gap below carry the values."""
    t, n = ref.DTYPES[dtype], 4096
    q = torch.zeros((rows, Hq, ref.D), dtype=t, device="cuda")
    q[..., 0] = 8.0
    k = torch.zeros((n, 1, ref.D), device="cuda")
    k[::16, :, 0] = gap * math.log(2) * math.sqrt(ref.D) / 8
    v = ref.vectors(n, 1, 3, torch.float32).abs() * 4 + 1
    v[::16] = 0
    cache = _cache_of(k, v)
    sel = torch.arange(n, dtype=torch.int32, device="cuda").expand(rows, n).contiguous() if selected else None
    out, e = _check_attend(cache, q, dtype, sel, weights=True)
    if gap < 26 and dtype == "bf16":       # (fp16's own steps are 2^-24)
        u = ref.half_step(t)
        assert ((out.double() - e.out).abs() <= (u + 2.0 ** -9) * e.out.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,rows", [(8, 1), (16, 1), (8, 4)])
@pytest.mark.parametrize("spread", [10, 22, 28])
def test_attend_value_groups_of_very_different_sizes(dtype, Hq, rows, spread):
    """Each group of a token's dimensions 2^spread / 3 times smaller than the last."""
    t, n = ref.DTYPES[dtype], 900
    q, k = ref.vectors(rows, Hq, 1, t), ref.vectors(n, 1, 2, t)
    v = ref.vectors(n, 1, 3, torch.float32) * 500
    v = v * torch.exp2(-spread / 3 * torch.arange(4, device="cuda").repeat_interleave(32))
    for x in (v, v.flip(-1), v[:1].expand(n, 1, ref.D)):   # (equal scales round alike)
        _check_attend(_cache_of(k, x), q, dtype)


@pytest.mark.parametrize("G", [8, 16])
def test_attend_an_infinite_scale_does_not_hide_the_finite_ones(G):
    """A token that only the last row sees has an infinite value scale; the scales
    beside it, 2^16 times the first ones, must reach the other rows whole.  So many
    heads that the keys are not split: token 256 is the first warp's again."""
    t, n, rows, Hkv = torch.bfloat16, 272, 2, 256
    q, k = ref.vectors(rows, G * Hkv, 1, t), ref.vectors(n, Hkv, 2, t)
    v = ref.vectors(n, Hkv, 3, torch.float32) * 0.01
    v[256:] *= 2.0 ** 16
    cache = _cache_of(k, v)
    at, so = binding.Attention("bf16", Hq=G * Hkv, Hkv=Hkv), ref.offsets([(rows, n)])
    want = at.attend(cache, q, so)
    cache.v_params[:, n - 1, :, 0] = math.inf
    out = at.attend(cache, q, so)
    assert torch.isfinite(want).all() and torch.equal(out[0], want[0])
    assert not torch.isfinite(out[1]).any()


def test_profile_counts_every_kernel_of_the_attention_calls():
    """Split calls record their joining kernel; a selection with weights of one and
    of several rows, and an eviction, each of theirs."""
    t, Hq, Hkv, n = torch.bfloat16, 8, 1, 9000
    at = binding.Attention("bf16", Hq=Hq, Hkv=Hkv)
    q, k, v = ref.vectors(2, Hq, 1, t), ref.vectors(n, Hkv, 2, t), ref.vectors(n, Hkv, 3, t)
    cache = binding.Cache4.empty(Hkv, n)
    dst = binding.Cache4.empty(Hkv, 64)
    whole, short = ref.offsets([(n, n)]), ref.offsets([(1, 5)])
    one, two = ref.offsets([(1, n)]), ref.offsets([(2, n)])
    sel = torch.arange(2048, dtype=torch.int32, device="cuda").expand(2, 2048).contiguous()
    calls = [
        (lambda: at.prompt(q, k, v, short), "prompt", 1),
        (lambda: at.prompt(q, k, v, one), "prompt", 2),
        (lambda: at.append(cache, k, v, whole), "cache", 1),
        (lambda: at.attend(cache, q, short), "attend", 1),
        (lambda: at.attend(cache, q, one), "attend", 2),
        (lambda: at.attend(cache, q, two, weights=True), "attend", 3),
        (lambda: at.attend(cache, q, one, sel_idx=sel[:1], weights=True), "attend", 3),
        (lambda: at.attend(cache, q, two, sel_idx=sel, weights=True), "attend", 4),
        (lambda: at.evict(cache, dst, [[0, n, 0, 64]]), "evict", 2),
    ]
    try:
        binding.profile_enable(True)
        for i, (call, kind, kernels) in enumerate(calls):
            binding.profile_reset()
            call()
            torch.cuda.synchronize()
            got = {name: c for name, (c, _) in binding.profile_read().items() if c}
            assert got == {kind: kernels}, (i, got)
    finally:
        binding.profile_enable(False)


def _near_halves(dtype, n, seed):
    """[n, 32] groups whose elements lie next to, or on, the half-integer multiples
    of their scale: lo and hi random, the others the 16-bit numbers around
    min + (i + 1/2) scale."""
    t = ref.DTYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    lo = -(torch.rand(n, generator=g) * 8 + 0.1)
    hi = torch.rand(n, generator=g) * 8 + 0.1
    few = torch.arange(n) % 3 == 0                    # few bits: many exact multiples
    unit = torch.exp2(torch.randint(-3, 3, (n,), generator=g).float())
    odd = 2 * torch.randint(0, 15, (n,), generator=g) + 1
    k = torch.tensor([1.0, 3.0, 5.0, 7.0])[torch.randint(0, 4, (n,), generator=g)] * unit
    lo, hi = torch.where(few, -odd / 2 * k, lo), torch.where(few, (15 - odd / 2) * k, hi)
    lo, hi = lo.to(t), hi.to(t)
    scale = ((hi.float() - lo.float()) / torch.full((n,), 15.0)).half().double()
    mn = lo.half().double()
    x = torch.empty((n, 32), dtype=t)
    x[:, 0], x[:, 1] = lo, hi
    for i in range(15):
        at = mn + (i + 0.5) * scale
        x[:, 2 + 2 * i] = at.to(t)
        x[:, 3 + 2 * i] = (at + torch.where(torch.rand(n, generator=g) < 0.5, 1.0, -1.0) *
                           torch.exp2(-torch.randint(8, 100, (n,), generator=g).double())).to(t)
    tiny = torch.exp2(-torch.randint(9, 100 if dtype == "bf16" else 24, (n, 32), generator=g).double())
    tiny = tiny * (1 + torch.rand((n, 32), generator=g).double()) * torch.where(
        torch.rand((n, 32), generator=g) < 0.5, 1.0, -1.0)
    swap = (torch.rand((n, 32), generator=g) < 0.3) & (torch.arange(32) >= 2)
    x = torch.where(swap, tiny.to(t), x)
    small = torch.arange(n) % 5 == 4                  # minima small against the maximum
    x[small, 0] = -tiny[small, 0].abs().to(t)
    x[small, 1:] = x[small, 1:].abs()
    return torch.minimum(torch.maximum(x, x[:, :1]), x[:, 1:2].abs())


def _codes(x):
    """The definition in exact arithmetic: (codes, scale, min) of one group."""
    lo, hi = min(x), max(x)
    f32 = torch.tensor([hi, lo], dtype=torch.float32)
    scale = ((f32[0] - f32[1]) / torch.tensor(15.0)).half().item()
    mn = torch.tensor(lo).half().item()
    if scale == 0:
        return [0] * len(x), scale, mn
    q = [round((Fraction(v) - Fraction(mn)) / Fraction(scale)) for v in x]   # (ties to even)
    return [min(15, max(0, c)) for c in q], scale, mn


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_rounds_the_exact_quotient(dtype):
    t, n = ref.DTYPES[dtype], 2048
    x = _near_halves(dtype, n, 3)
    # a quotient of 3.4999999995 that is 3.5 in fp32, and one on either side of 14.5
    x[0] = torch.tensor([-3.5, 11.5] + [-1e-9, 1e-9, 0.0] * 10, dtype=t)
    x[1] = torch.tensor([-14.5, 0.5] + [-2.0 ** -23, 2.0 ** -23, 0.0] * 10, dtype=t)
    rows = x.view(n // 4, 1, ref.D).cuda()
    cache = binding.Cache4.empty(1, n // 4)
    at = binding.Attention(dtype, Hq=1, Hkv=1)
    at.append(cache, rows, rows.clone(), ref.offsets([(n // 4, n // 4)]))
    want = [_codes(r) for r in x.double().tolist()]
    codes = torch.tensor([w[0] for w in want])
    params = torch.tensor([w[1:] for w in want], dtype=torch.float16)
    plain = ref.quantise(rows, "k")[0]
    for kind in "kv":
        got = getattr(cache, kind + "_codes")[0].cpu()
        nib = torch.stack((got & 15, got >> 4), -1).flatten(-2).long()
        nib = nib[:, torch.argsort(ref.order(kind))].reshape(n, 32)
        assert torch.equal(getattr(cache, kind + "_params")[0].cpu().view(n, 2), params)
        assert torch.equal(nib, codes), int((nib != codes).sum())
    # the fp32 quotient's rounding would differ in some of these groups
    assert not torch.equal(plain, cache.k_codes)


@pytest.mark.parametrize("rows,n", [(300, 300), (4, 9000), (1, 5)], ids=["whole", "split", "short"])
def test_prompt_means_of_the_largest_values_stay_finite(rows, n):
    """A mean is no larger than its largest value: rounding the weights up must not
    push it over fp16's end; a visible infinity still does.  (Weights and result
    round by 2^-11 each, so the mean may be that much smaller.)"""
    t, Hq = torch.float16, 8
    so = ref.offsets([(rows, n)])
    far = torch.finfo(t).max
    sign = torch.where(torch.arange(ref.D, device="cuda") % 3 == 0, -far, far).to(t)
    k, v = ref.vectors(n, 1, 2, t), sign.expand(n, 1, ref.D).contiguous()
    at = binding.Attention("fp16", Hq=Hq, Hkv=1)
    near = lambda x: (x.double() / sign[:x.shape[-1]].double() - 1).abs() <= 2.0 ** -10 + 2.0 ** -17
    for seed in range(8):
        q = ref.vectors(rows, Hq, seed, t)
        out = at.prompt(q, k, v, so)
        assert near(out).all(), (seed, int(torch.isinf(out).sum()))
    # from key 64 on weights of 1 + 2^-11 and a little of the maximum at hand: every one
    # rounds up to 1 + 2^-10
    q, k2 = torch.zeros_like(q), torch.zeros_like(k)
    q[..., 0], k2[64:, 0, 0] = 1.0, math.log(1 + 1.02 * 2.0 ** -11) * math.sqrt(ref.D)
    out = at.prompt(q, k2, v, so)
    assert near(out).all(), int(torch.isinf(out).sum())
    first = min(2, n - rows)
    v[first, 0, 3], v[first, 0, 4] = math.inf, -math.inf
    out = at.prompt(q, k, v, so)[max(0, first - (n - rows)):]
    assert (out[..., 3] == math.inf).all()                 # (with -far beside it, in fp32)
    assert (out[..., 4] == -math.inf).all()
    assert near(out)[..., 5:].all()
