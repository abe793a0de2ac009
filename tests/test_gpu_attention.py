"""GPU parity of the attention calls against the fp64 oracle.

Bounds, per element, with h the half step of the output type (finfo.eps / 2)
and u = 2^-24:

* norm and rotation: h |y| for the one rounding, plus fp32 arithmetic: the
  mean of D squares, its root and two products are good to (D/2 + 8) u, the
  angle to 2^-25 turns and sincospif to two ulp, so the sine and cosine to
  2^-21; both act on |a| + |b|.
* attention: a score sums D products in fp32 (relative to sum_d |q_d k_d| at
  most (D + 2) u, ds); the exponential of a difference of two scores is off
  by at most 2 ds + 2^-20 |s - m| u-scale terms and the function's own 2^-21,
  together e_p = 2 ds + 2^-18; a weight is rounded to the operand type (h,
  and for fp16 at most 2^-25 of the largest where it is subnormal); the sums
  over n keys lose at most (n + 64) u; the result is rounded once (h).
  |out - ref| <= h |ref| + (h + 2 e_p + (n + 64) u) sum p|v| + tiny.
* lse: ds + 2^-18 + 4 u |lse| + (n + 64) u.
"""

import numpy as np
import pytest
import torch

import lut_binary_gemv_b200 as fb
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -100}   # half a step of subnormals, with margin for fp16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    off = np.abs(got - ref)
    bad = ~((off <= bound) | (got == ref) | np.isnan(ref))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bound; worst {np.nanmax(off - bound):.3e} over"


# ---- norm and rotation -------------------------------------------------------


def rope_case(T, Hq, Hkv, D, rot, norm, neighbours, t_in, t_out, page_size, seed=0, fused=True, first=0):
    g = gen(seed)
    qkv = normal(g, T, Hq + 2 * Hkv, D, dtype=t_in)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, 5000, (T,), generator=g, device=DEV, dtype=torch.int32) + first
    wq, wk = (1 + 0.2 * torch.randn(2, D, generator=g, device=DEV)) if norm else (None, None)
    freq = fb.rope_frequencies(rot) if rot else None
    cache = slots = None
    if page_size:
        pages = (T + page_size - 1) // page_size + 3
        cache = tuple(normal(g, pages, Hkv, page_size, D, dtype=t_out) for _ in range(2))
        slots = torch.randperm(pages * page_size, generator=g, device=DEV)[:T].to(torch.int32)
    return q, k, v, pos, freq, wq, wk, cache, slots


def rope_reference(x, w, pos, freq, neighbours, eps):
    D = x.shape[-1]
    y = A.norm(f64(x), None if w is None else f64(w), eps)
    mag = np.abs(y)
    if freq is None:
        return y, mag * (D / 2 + 8) * U
    r = A.rotate(y, pos.cpu().numpy(), f64(freq), neighbours)
    half = freq.numel()
    pair = np.abs(y[..., :2 * half]).reshape(*y.shape[:-1], *((half, 2) if neighbours else (2, half)))
    both = pair.sum(-1 if neighbours else -2, keepdims=True)
    mag[..., :2 * half] = np.broadcast_to(both, pair.shape).reshape(*y.shape[:-1], 2 * half)
    return r, mag * (2.0 ** -21 + (D / 2 + 8) * U)


def check_rows(got, ref, arith, what):
    h = HALF[got.dtype]
    assert_within(f64(got), ref, h * np.abs(ref) + (1 + h) * arith + TINY[got.dtype], what)


ROPE = [
    # T, Hq, Hkv, D, rot, norm, neighbours, t_in, t_out, page_size
    (1, 32, 32, 128, 128, True, False, torch.float32, torch.bfloat16, 64),
    (1, 1, 1, 16, 16, True, True, torch.float16, torch.float16, 1),
    (7, 8, 2, 64, 32, False, True, torch.float32, torch.float16, 16),
    (33, 5, 1, 128, 64, True, False, torch.bfloat16, torch.float16, 8),
    (130, 64, 8, 128, 128, True, True, torch.bfloat16, torch.bfloat16, 32),
    (65, 6, 3, 256, 256, True, False, torch.float16, torch.bfloat16, 128),
    (19, 4, 4, 80, 48, True, False, torch.float32, torch.bfloat16, 4),
    (12, 3, 1, 96, 0, True, False, torch.float16, torch.float16, 2),
    (700, 10, 2, 64, 64, False, False, torch.bfloat16, torch.bfloat16, 0),
]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("fused", [True, False])
def test_rope(case, fused):
    T, Hq, Hkv, D, rot, norm, neighbours, t_in, t_out, page_size = case
    q, k, v, pos, freq, wq, wk, cache, slots = rope_case(*case, seed=T, fused=fused)
    before = None if cache is None else [c.clone() for c in cache]
    qo, ko, vo = fb.fb_qk_norm_rope(q, k, v, pos, freq, wq, wk, 1e-5, neighbours, cache, slots, out_dtype=t_out)
    check_rows(qo, *rope_reference(q, wq, pos, freq, neighbours, 1e-5), "q")
    kr, ka = rope_reference(k, wk, pos, freq, neighbours, 1e-5)
    if cache is None:
        check_rows(ko, kr, ka, "k")
        assert torch.equal(vo, v.to(t_out))
        return
    assert ko is None and vo is None
    rows = [c.transpose(1, 2).reshape(-1, Hkv, D) for c in cache]
    at = slots.long()
    check_rows(rows[0][at], kr, ka, "cached k")
    assert torch.equal(rows[1][at], v.to(t_out))
    rest = torch.ones(len(rows[0]), dtype=torch.bool, device=DEV)
    rest[at] = False
    for c, b in zip(rows, before):
        assert torch.equal(c[rest], b.transpose(1, 2).reshape(-1, Hkv, D)[rest])


def test_rope_far_and_negative_positions():
    q, k, v, pos, freq, *_ = rope_case(64, 2, 1, 128, 128, False, False, torch.float32, torch.bfloat16, 0, seed=2)
    pos = torch.linspace(-2 ** 31, 2 ** 31 - 1, 64, dtype=torch.float64, device=DEV).to(torch.int32)
    qo, ko, _ = fb.fb_qk_norm_rope(q, k, v, pos, freq, out_dtype=torch.bfloat16)
    # the oracle's own angle, pos * freq in fp64, is good to 2^31 * 2^-53 radians: nothing beside 2^-21
    check_rows(qo, *rope_reference(q, None, pos, freq, False, 1e-6), "q")
    check_rows(ko, *rope_reference(k, None, pos, freq, False, 1e-6), "k")


def test_rope_in_place_and_beside_the_cache():
    case = rope_case(21, 8, 2, 128, 128, True, False, torch.bfloat16, torch.bfloat16, 16, seed=9)
    q, k, v, pos, freq, wq, wk, cache, slots = case
    qr, kr, vr = fb.fb_qk_norm_rope(q, k, v, pos, freq, wq, wk)
    fb.fb_qk_norm_rope(q, k, v, pos, freq, wq, wk, cache=cache, slots=slots, q_out=q, k_out=k, v_out=v)
    assert torch.equal(q, qr) and torch.equal(k, kr) and torch.equal(v, vr)
    rows = cache[0].transpose(1, 2).reshape(-1, 2, 128)
    assert torch.equal(rows[slots.long()], kr)


def test_rope_outputs_between_the_rows_of_the_inputs():
    # q, k, v and all outputs in one buffer: rows side by side, and in place beside strangers
    q, k, v, pos, freq, wq, wk, *_ = rope_case(37, 4, 2, 64, 64, True, False, torch.bfloat16, torch.bfloat16, 0, seed=10)
    want = fb.fb_qk_norm_rope(q, k, v, pos, freq, wq, wk)
    buf = torch.full((37, 18, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    buf[:, 1:9] = torch.cat([q, k, v], 1)
    parts = lambda at: (buf[:, at:at + 4], buf[:, at + 4:at + 6], buf[:, at + 6:at + 8])  # noqa: E731
    got = fb.fb_qk_norm_rope(*parts(1), pos, freq, wq, wk, q_out=parts(9)[0], k_out=parts(9)[1], v_out=parts(9)[2])
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and torch.equal(buf[:, 1:9], torch.cat([q, k, v], 1))
    assert bool((buf[:, [0, 17]] == 3.0).all())
    got = fb.fb_qk_norm_rope(*parts(1), pos, freq, wq, wk, q_out=parts(1)[0], k_out=parts(1)[1], v_out=parts(1)[2])
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and bool((buf[:, [0, 17]] == 3.0).all())
    one = q[:1].clone()
    fb.fb_qk_norm_rope(one, k[:1], v[:1], pos[:1], freq, wq, wk, q_out=one)
    assert torch.equal(one, want[0][:1])
    wide = torch.zeros(37, 5, 64, dtype=torch.bfloat16, device=DEV)
    wide[:, :4] = q
    with pytest.raises(fb.FbError, match="INVALID_VALUE"):   # rows of another pitch over the input's
        fb.fb_qk_norm_rope(wide[:, :4], k, v, pos, freq, wq, wk, q_out=wide.view(-1)[:37 * 256].view(37, 4, 64))


def test_rope_skips_slots_outside_the_cache():
    q, k, v, pos, freq, wq, wk, cache, slots = rope_case(9, 4, 2, 64, 64, True, False, torch.float16, torch.float16,
                                                         4, seed=5)
    total = cache[0].shape[0] * 4
    buf = torch.zeros(2, total + 64, 2, 64, dtype=torch.float16, device=DEV)   # room on both sides of the cache
    cache = tuple(b[32:32 + total].view(total // 4, 2, 4, 64) for b in buf)
    bad = torch.tensor([-1, -2 ** 31, total, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    slots = torch.cat([slots[:5], bad])
    fb.fb_qk_norm_rope(q, k, v, pos, freq, wq, wk, cache=cache, slots=slots)
    written = (buf != 0).flatten(2).any(-1)
    assert written[:, 32:32 + total].reshape(2, -1).any(1).all()
    assert not written[:, :32].any() and not written[:, 32 + total:].any()
    assert int((cache[1].transpose(1, 2).reshape(total, -1) != 0).any(-1).sum()) == 5


def test_rope_special_values_stay_in_their_head():
    q, k, v, pos, freq, wq, wk, *_ = rope_case(4, 4, 2, 64, 64, True, False, torch.float32, torch.bfloat16, 0, seed=6)
    ref = [t.clone() for t in fb.fb_qk_norm_rope(q, k, v, pos, freq, wq, wk)]
    q[1, 2, 5], k[2, 0, 0], v[3, 1, 7] = float("nan"), float("inf"), float("-inf")
    got = fb.fb_qk_norm_rope(q, k, v, pos, freq, wq, wk)
    for r, g, at in zip(ref, got, [(1, 2), (2, 0), (3, 1)]):
        same = torch.ones(r.shape[:2], dtype=torch.bool, device=DEV)
        same[at] = False
        assert torch.equal(r[same], g[same]) and not torch.isfinite(g[at]).all()


# ---- attention -----------------------------------------------------------------


def check_attention(out, lse, refs, D, dtype, what):
    """refs: (token rows, head, (out, lse, sum p|v|, max sum|qk|), keys a row)."""
    h = HALF[dtype]
    o, l = f64(out), None if lse is None else f64(lse)
    for rows, head, (ro, rl, wabs, sabs), n in refs:
        ds = sabs * (D + 2) * U
        e_p = 2 * ds + 2.0 ** -18
        sums = (n + 64) * U
        extra = 2.0 ** -25 * n if dtype == torch.float16 else 0.0
        bound = h * np.abs(ro) + ((h + 2 * e_p + sums)[:, None] * wabs) + (extra[:, None] if np.ndim(extra) else extra) \
            + TINY[dtype]
        assert_within(o[rows, head], ro, bound, f"{what}: out, head {head}")
        if l is not None:
            rl_abs = np.where(np.isfinite(rl), np.abs(rl), 0)
            assert_within(l[rows, head], rl, ds + 2.0 ** -18 + 4 * U * rl_abs + sums, f"{what}: lse, head {head}")


def prompt_refs(q, k, v, cu, scale, heads=None):
    Hq, Hkv = q.shape[1], k.shape[1]
    qn, kn, vn = f64(q), f64(k), f64(v)
    refs = []
    for a, b in zip(cu[:-1], cu[1:]):
        if b <= a:
            continue
        seen = np.tril(np.ones((b - a, b - a), bool))
        for h in range(Hq) if heads is None else heads:
            hk = h // (Hq // Hkv)
            refs.append((slice(a, b), h, A.attend(qn[a:b, h], kn[a:b, hk], vn[a:b, hk], seen, scale),
                         np.arange(1, b - a + 1)))
    return refs


def prompt_inputs(lens, Hq, Hkv, D, dtype, tail=0, seed=0, fused=False):
    g = gen(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    T = int(cu[-1]) + tail
    if fused:
        qkv = normal(g, T, Hq + 2 * Hkv, D, dtype=dtype)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = normal(g, T, Hq, D, dtype=dtype), normal(g, T, Hkv, D, dtype=dtype), normal(g, T, Hkv, D, dtype=dtype)
    return q, k, v, cu.tolist(), torch.tensor(cu, dtype=torch.int32, device=DEV)


PROMPTS = [
    # lens, Hq, Hkv, D, dtype, tail, fused
    ([1], 1, 1, 64, torch.float16, 0, False),
    ([2], 4, 2, 128, torch.bfloat16, 0, False),
    ([127, 128, 129], 2, 1, 128, torch.bfloat16, 0, True),
    ([255, 256, 257], 2, 2, 64, torch.float16, 3, False),
    ([0, 5, 0, 0, 64, 1, 0], 5, 1, 128, torch.float16, 7, True),
    ([383, 1, 385, 640], 8, 2, 64, torch.bfloat16, 0, False),
    ([1000, 33], 6, 2, 128, torch.float16, 130, False),
    ([1] * 70 + [3, 300], 3, 3, 128, torch.bfloat16, 1, True),
]


# with few items (split over their keys) and with as many as go round the SMs
@pytest.mark.parametrize("times", [1, 300])
@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1]}/{c[2]}-{c[3]}-{str(c[4])[6:]}")
def test_prompt(case, times):
    lens, Hq, Hkv, D, dtype, tail, fused = case
    group, Hkv = Hq // Hkv, Hkv * -(-times // Hq)
    Hq = Hkv * group
    q, k, v, cu, cud = prompt_inputs(lens, Hq, Hkv, D, dtype, tail, seed=sum(lens), fused=fused)
    out = torch.full((q.shape[0], Hq, D), 7.5, dtype=dtype, device=DEV)
    lse = torch.full((q.shape[0], Hq), -3.25, device=DEV)
    scale = 0.9 * D ** -0.5
    assert fb.fb_attn_prompt(q, k, v, cud, scale, out, lse) is out
    heads = None if times == 1 else [0, Hq // 2, Hq - 1]
    check_attention(out, lse, prompt_refs(q, k, v, cu, scale, heads), D, dtype, "prompt")
    assert (out[cu[-1]:] == 7.5).all() and (lse[cu[-1]:] == -3.25).all()
    again = fb.fb_attn_prompt(q, k, v, cud, scale)
    assert torch.equal(again[:cu[-1]], out[:cu[-1]])                    # deterministic; lse not needed
    assert fb.fb_attn_errors() == 0


def test_prompt_longer_one_head():
    q, k, v, cu, cud = prompt_inputs([2500], 2, 1, 128, torch.bfloat16, seed=11)
    q *= 4                                                               # peaked rows, moving maxima
    lse = torch.empty(2500, 2, device=DEV)
    out = fb.fb_attn_prompt(q, k, v, cud, lse=lse)
    check_attention(out, lse, prompt_refs(q, k, v, cu, 128 ** -0.5, heads=[1]), 128, torch.bfloat16, "long")


@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_rising_scores(D, H):
    # every key scores above all earlier ones by 3 (base e): the running maximum moves at every key
    n = 700
    q = torch.zeros(n, H, D, dtype=torch.float16, device=DEV)
    k = torch.zeros(n, 1, D, dtype=torch.float16, device=DEV)
    q[..., 0] = 1.0
    k[..., 0] = (torch.arange(n, device=DEV) * 3.0)[:, None].half()
    v = normal(gen(1), n, 1, D, dtype=torch.float16)
    cud = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lse = torch.empty(n, H, device=DEV)
    out = fb.fb_attn_prompt(q, k, v, cud, 1.0, lse=lse)
    check_attention(out, lse, prompt_refs(q, k, v, [0, n], 1.0, heads=[H - 1]), D, torch.float16, "rising")
    out = fb.fb_attn_prompt(q, k.flip(0).contiguous(), v, cud, 1.0, lse=lse)
    check_attention(out, lse, prompt_refs(q, k.flip(0), v, [0, n], 1.0, heads=[0]), D, torch.float16, "falling")


@pytest.mark.parametrize("Hkv", [2, 160])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_prompt_special_values_reach_only_rows_that_see_them(value, Hkv):
    lens, Hq, D = [200, 61, 300], 2 * Hkv, 128
    q, k, v, cu, cud = prompt_inputs(lens, Hq, Hkv, D, torch.bfloat16, tail=9, seed=8)
    ref = fb.fb_attn_prompt(q, k, v, cud)
    at = 230                                             # in the second sequence
    v2 = v.clone()
    v2[at, 0, 17] = value
    v2[-1] = value                                       # a padding row
    got = fb.fb_attn_prompt(q, k, v2, cud)
    hit = torch.zeros(q.shape[0], Hq, D, dtype=torch.bool, device=DEV)
    hit[at:261, :2, 17] = True
    assert torch.equal(got[:561][~hit[:561]], ref[:561][~hit[:561]])
    bad = got[hit]
    assert bool((torch.isnan(bad) if value != value else bad == value).all())
    k2 = k.clone()
    k2[at, 1, 3] = float("nan")
    k2[-1] = value
    got = fb.fb_attn_prompt(q, k2, v, cud)
    hit[:] = False
    hit[at:261, 2:4] = True
    assert torch.equal(got[:561][~hit[:561]], ref[:561][~hit[:561]]) and bool(torch.isnan(got[hit]).all())


LOW = -30000.0   # a key of it against 1 scores below -3700: no weight, as one of minus infinity


@pytest.mark.parametrize("H", [1, 200])
@pytest.mark.parametrize("key", [0, 130])
@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_prompt_infinite_scores(D, dtype, key, H):
    n = 300
    q, k, v, cu, cud = prompt_inputs([n], H, 1, D, dtype, seed=18)
    q[..., 0] = torch.tensor([1.0, -1.0, 0.0], device=DEV)[torch.arange(n, device=DEV) % 3, None]
    k[key, 0, 0] = LOW
    low, k[key, 0, 0] = k.clone(), float("-inf")
    lses = [torch.empty(n, H, device=DEV) for _ in range(2)]
    want, got = (fb.fb_attn_prompt(q, x, v, cud, lse=y) for x, y in zip((low, k), lses))
    i = torch.arange(n, device=DEV)
    nan = (i >= key) & (i % 3 > 0)                       # plus infinity, and zero times infinity
    same = ~nan & (i > 0) if key == 0 else ~nan
    assert torch.equal(got[same], want[same]) and torch.equal(lses[1][same], lses[0][same])
    assert bool(torch.isnan(got[nan]).all()) and bool(torch.isnan(lses[1][nan]).all())
    if key == 0:                                         # nothing but minus infinity
        assert not got[0].any() and bool((lses[1][0] == -float("inf")).all())


def test_prompt_clamps_offsets_outside_the_tokens():
    q, k, v, cu, cud = prompt_inputs([40, 60], 2, 1, 64, torch.float16, seed=4)
    ref = fb.fb_attn_prompt(q, k, v, cud)
    wild = torch.tensor([-5, 40, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    assert torch.equal(fb.fb_attn_prompt(q, k, v, wild), ref)


def test_prompt_that_starts_behind_the_first_token():
    q, k, v, cu, cud = prompt_inputs([60, 9], 2, 2, 128, torch.float16, seed=14)
    out = torch.full_like(q, 3.0)
    fb.fb_attn_prompt(q, k, v, torch.tensor([11, 60], dtype=torch.int32, device=DEV), out=out)
    check_attention(out, None, prompt_refs(q, k, v, [11, 60], 128 ** -0.5), 128, torch.float16, "late")
    assert bool((out[:11] == 3.0).all()) and bool((out[60:] == 3.0).all())


def test_prompt_many_short_sequences_and_heads():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 300).tolist()
    q, k, v, cu, cud = prompt_inputs(lens, 40, 8, 64, torch.bfloat16, seed=15)
    lse = torch.empty(q.shape[0], 40, device=DEV)
    out = fb.fb_attn_prompt(q, k, v, cud, lse=lse)
    check_attention(out, lse, prompt_refs(q, k, v, cu, 64 ** -0.5, heads=[0, 17, 39]), 64, torch.bfloat16, "short")


def test_prompts_on_two_streams_at_once():
    cases = [prompt_inputs([1500], 8, 2, 128, torch.bfloat16, seed=s) for s in (16, 17)]
    refs = [fb.fb_attn_prompt(q, k, v, cud) for q, k, v, _, cud in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for _ in range(3):
        for (q, k, v, _, cud), s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append(fb.fb_attn_prompt(q, k, v, cud))
    torch.cuda.synchronize()
    assert all(torch.equal(o, refs[i % 2]) for i, o in enumerate(outs)) and fb.fb_attn_errors() == 0


def test_prompt_side_stream_and_graph():
    q, k, v, cu, cud = prompt_inputs([300, 50], 4, 2, 128, torch.bfloat16, seed=3)
    ref = fb.fb_attn_prompt(q, k, v, cud)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = fb.fb_attn_prompt(q, k, v, cud, flags=fb.FB_GEMV_PDL)
    side.synchronize()
    assert torch.equal(a, ref)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.fb_attn_prompt(q, k, v, cud, out=out)
    q.copy_(q.flip(0))
    cud.copy_(torch.tensor([0, 20, 350], dtype=torch.int32, device=DEV))   # the graph reads the new sequences
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fb.fb_attn_prompt(q, k, v, cud))


# Every 16th key is a sink: it outscores the others by 2^octaves and its value is zero, so the output is made of the
# others' small weights.  The bound is of each weight: `w` of its size, and for fp16 half a step of its subnormals,
# 2^-25, against a largest weight of at least 2^7: 2^-32 of a sink's.


SINKS = [3.0, 18.3, 20.6, 22.4, 24.6, 25.5]


def check_sinks(out, refs, octaves, most, D, dtype, w, what):
    for rows, head, (ro, rl, wabs, sabs), n in refs:
        e_p = 2 * sabs * (D + 2) * U + 2.0 ** -18
        largest = 1.0 if octaves is None else np.exp(octaves * np.log(2) - rl)       # of the row's weights, at most
        floor = 2.0 ** -32 * n * most * largest * (dtype == torch.float16)
        bound = HALF[dtype] * np.abs(ro) + (w + 2 * e_p + (n + 64) * U)[:, None] * wabs + floor[:, None] + TINY[dtype]
        assert_within(f64(out)[rows, head], ro, bound, f"{what}: head {head}")


def sinks_in(k, v, octaves, g):
    """k, v [keys, heads, D]: scores 0 but for every 16th key, for queries that are the first unit vector."""
    k.zero_()
    k[::16, :, 0] = octaves * np.log(2)
    v.copy_(256 * (1 + torch.rand(v.shape, generator=g, device=DEV)))
    v[::16] = 0
    return float(k[0, 0, 0]) / np.log(2)


@pytest.mark.parametrize("octaves", SINKS)
@pytest.mark.parametrize("H", [2, 320])
@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.float16), (64, torch.bfloat16)])
def test_prompt_small_weights_beside_sinks(D, dtype, H, octaves):
    n = 700
    q, k, v = (torch.zeros(n, h, D, dtype=dtype, device=DEV) for h in (H, 1, 1))
    q[..., 0] = 1
    octaves = sinks_in(k, v, octaves, gen(51))
    out = fb.fb_attn_prompt(q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV), 1.0)
    check_sinks(out, prompt_refs(q, k, v, [0, n], 1.0, heads=[H - 1]), octaves, 512, D, dtype, HALF[dtype], "prompt")


# ---- trees over a paged cache ----------------------------------------------------


def tree_inputs(lens, drafts, Hq, Hkv, D, page_size, dtype, seed=0, garbage=float("nan")):
    """A cache whose rows behind the sequences hold garbage, a shuffled page table with -1 behind them."""
    g = gen(seed)
    rng = np.random.default_rng(seed)
    need = [-(-(a + b) // page_size) for a, b in zip(lens, drafts)]
    pages = sum(need) + 3
    order = rng.permutation(pages)
    table = np.full((len(lens), max(need) + 2), -1, np.int32)
    k, v = (normal(g, pages, Hkv, page_size, D, dtype=dtype) for _ in range(2))
    used = torch.zeros(pages, page_size, dtype=torch.bool)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
        for p in range(lens[s] + drafts[s]):
            used[int(table[s, p // page_size]), p % page_size] = True
    hide = ~used[:, None, :, None].to(DEV).expand_as(k)
    k[hide] = garbage
    v[hide] = garbage
    T = sum(drafts)
    q = normal(g, T, Hq, D, dtype=dtype)
    cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    masks = []
    for m in drafts:
        seen = []
        for j in range(m):
            parent = rng.integers(-1, j)
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        masks += seen
    return dict(q=q, k=k, v=v, table=table, lens=lens, drafts=drafts, cu=cu, masks=masks, D=D, Hq=Hq, Hkv=Hkv,
                page_size=page_size, dtype=dtype)


def tree_call(c, masks="own", scale=None, **kw):
    table = torch.tensor(c["table"], device=DEV)
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    cu = torch.tensor(c["cu"], device=DEV)
    masks = c["masks"] if masks == "own" else masks
    if masks is not None:
        masks = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)
    lse = torch.empty(c["q"].shape[0], c["Hq"], device=DEV)
    out = fb.fb_attn_tree(c["q"], (c["k"], c["v"]), table, lens, cu, max(c["drafts"]), masks, scale, lse=lse, **kw)
    return out, lse


def tree_refs(c, masks, scale, heads=None, seqs=None):
    qn, kn, vn = f64(c["q"]), f64(c["k"]), f64(c["v"])
    refs, P = [], c["page_size"]
    for s, (a, m) in enumerate(zip(c["lens"], c["drafts"])):
        if m == 0 or (seqs is not None and s not in seqs):
            continue
        p = np.arange(a + m)
        pages, rows = c["table"][s][p // P], p % P
        seen = np.ones((m, a + m), bool)
        for i in range(m):
            for j in range(m):
                seen[i, a + j] = j <= i if masks is None else bool(masks[c["cu"][s] + i] >> j & 1)
        for h in range(c["Hq"]) if heads is None else heads:
            hk = h // (c["Hq"] // c["Hkv"])
            refs.append((slice(int(c["cu"][s]), int(c["cu"][s]) + m), h,
                         A.attend(qn[c["cu"][s]:c["cu"][s] + m, h], kn[pages, hk, rows], vn[pages, hk, rows], seen,
                                  scale), seen.sum(1)))
    return refs


TREES = [
    # lens, drafts, Hq, Hkv, D, page_size, dtype
    ([0], [1], 1, 1, 64, 16, torch.float16),
    ([37], [1], 32, 32, 128, 64, torch.bfloat16),
    ([1, 0, 63, 64, 65, 700], [1] * 6, 8, 1, 128, 16, torch.bfloat16),
    ([500, 3, 129], [5, 0, 17], 10, 2, 64, 8, torch.float16),
    ([100, 257, 0], [64, 33, 64], 4, 4, 128, 1, torch.float16),
    ([300, 1, 511], [64, 2, 63], 16, 2, 128, 128, torch.bfloat16),
    ([1000, 77], [3, 16], 24, 1, 64, 32, torch.bfloat16),
    ([200] * 40, [1] * 40, 6, 2, 128, 4, torch.float16),
    ([6000], [2], 16, 2, 128, 64, torch.bfloat16),
    ([9, 2000, 31], [31, 7, 1], 40, 8, 64, 1024, torch.float16),
    # more than 32 rows a key head
    ([700, 5, 1300, 127], [64, 40, 9, 1], 16, 2, 128, 8, torch.bfloat16),
    ([129, 0], [64, 3], 64, 1, 64, 64, torch.float16),
    ([0, 2500, 128], [33, 64, 50], 8, 8, 128, 16, torch.float16),
    ([9000], [64], 8, 1, 128, 256, torch.bfloat16),
    ([300, 64], [7, 64], 128, 1, 64, 128, torch.bfloat16),
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: f"{len(c[0])}x{max(c[0])}+{max(c[1])}-{c[2]}/{c[3]}-{c[4]}-p{c[5]}-{str(c[6])[6:]}")
@pytest.mark.parametrize("chain", [False, True])
def test_tree(case, chain):
    c = tree_inputs(*case, seed=len(case[0]) + case[2])
    masks = None if chain else c["masks"]
    scale = 1.1 * c["D"] ** -0.5
    out, lse = tree_call(c, masks, scale)
    check_attention(out, lse, tree_refs(c, masks, scale), c["D"], c["dtype"], "tree")
    o2, l2 = tree_call(c, masks, scale, flags=fb.FB_GEMV_PDL)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert fb.fb_attn_errors() == 0


# up to 16 rows a key head (weights good to 2^-16), up to 32, more by each path
@pytest.mark.parametrize("octaves", SINKS)
@pytest.mark.parametrize("Hq,drafts,page_size,dtype", [
    (1, 12, 16, torch.float16), (2, 7, 4, torch.float16), (1, 16, 64, torch.bfloat16), (4, 8, 64, torch.float16),
    (4, 20, 4, torch.float16), (8, 20, 16, torch.float16)])
def test_tree_small_weights_beside_sinks(Hq, drafts, page_size, dtype, octaves):
    D = 64
    c = tree_inputs([1600, 30], [drafts, 1], Hq, 1, D, page_size, dtype, seed=52)
    c["q"].zero_()
    c["q"][..., 0] = 1
    for s, (a, m) in enumerate(zip(c["lens"], c["drafts"])):
        p = np.arange(a + m)
        k, v = (torch.empty(a + m, 1, D, dtype=dtype, device=DEV) for _ in range(2))
        octaves = sinks_in(k, v, octaves, gen(53 + s))
        pages, rows = torch.tensor(c["table"][s][p // page_size], device=DEV).long(), torch.tensor(p % page_size, device=DEV)
        c["k"][pages, 0, rows], c["v"][pages, 0, rows] = k[:, 0], v[:, 0]
    out, _ = tree_call(c, None, 1.0)
    check_sinks(out, tree_refs(c, None, 1.0, heads=[Hq - 1]), octaves, 512, D, dtype,
                2.0 ** -16 if Hq * drafts <= 16 else HALF[dtype], "tree")


@pytest.mark.parametrize("case", [t for t in TREES if t[2] // t[3] * max(t[1]) <= 16] +
                         [([5000, 64, 1], [8, 1, 3], 4, 2, 128, 32, torch.bfloat16)],
                         ids=lambda c: f"{len(c[0])}x{max(c[0])}+{max(c[1])}-{c[2]}/{c[3]}-{c[4]}-p{c[5]}-{str(c[6])[6:]}")
def test_tree_weights_of_up_to_16_rows_lose_no_more_than_they_may(case):
    c = tree_inputs(*case, seed=45)
    out, _ = tree_call(c)
    refs = tree_refs(c, c["masks"], c["D"] ** -0.5)
    check_sinks(out, refs, None, 8.0, c["D"], c["dtype"], 2.0 ** -16, "few rows")    # no normal value reaches 8


def test_tree_single_tokens_without_offsets():
    c = tree_inputs([70, 5], [1, 1], 4, 2, 64, 16, torch.float16, seed=1)
    a, _ = tree_call(c, None)
    b = fb.fb_attn_tree(c["q"], (c["k"], c["v"]), torch.tensor(c["table"], device=DEV),
                        torch.tensor(c["lens"], dtype=torch.int32, device=DEV))
    assert torch.equal(a, b)


def test_tree_masks_that_leave_nothing_or_holes():
    c = tree_inputs([0, 40], [6, 6], 4, 2, 128, 16, torch.bfloat16, seed=2)
    masks = [0, 1, 0, 0b100000, ~0 & (2 ** 64 - 1), 2, 0, 0, 0b111, 1 << 63, 0b101010, 0b1]
    seen = [m & 0b111111 for m in masks]                                  # bits behind the drafts are ignored
    out, lse = tree_call(c, masks)
    check_attention(out, lse, tree_refs(c, seen, 128 ** -0.5), 128, torch.bfloat16, "holes")
    for row in (0, 2):
        assert not out[row].any() and bool((lse[row] == -float("inf")).all())


@pytest.mark.parametrize("garbage", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,D,page_size,dtype", [(1, 64, 16, torch.float16), (1, 128, 16, torch.bfloat16),
                                                  (20, 64, 64, torch.bfloat16), (20, 128, 4, torch.float16)])
def test_tree_values_behind_the_keys_reach_no_row(Hq, D, page_size, dtype, garbage):
    # every place of the last key within a tile and within a warp's keys, the values behind it not finite
    c = tree_inputs(list(range(130)), [1] * 130, Hq, 1, D, page_size, dtype, seed=41, garbage=garbage)
    out, lse = tree_call(c, None)
    check_attention(out, lse, tree_refs(c, None, D ** -0.5, heads=[0, Hq - 1]), D, dtype, "behind")
    for _ in range(20):
        again, _ = tree_call(c, None)
        assert torch.equal(again, out)


@pytest.mark.parametrize("key", [100, 1999, 2002])
@pytest.mark.parametrize("Hq,drafts,page_size", [(1, 8, 16), (1, 8, 4), (4, 8, 16), (4, 8, 4), (8, 8, 16), (8, 8, 4)])
def test_tree_infinite_scores(Hq, drafts, page_size, key):
    # committed or drafted; the second sequence's only key scores minus infinity, or plus, in every head
    c = tree_inputs([2000, 0, 0], [drafts, 1, 1], Hq, 1, 64, page_size, torch.bfloat16, seed=19)
    c["q"][:drafts:2, :, 0], c["q"][1:drafts:2, :, 0], c["q"][drafts:, :, 0] = 1, -1, 1
    places = [(0, key, -1), (1, 0, -1), (2, 0, 1)]
    k = [(int(c["table"][s, p // page_size]), 0, p % page_size, 0) for s, p, _ in places]
    for at in k:
        c["k"][at] = LOW
    want, want_lse = tree_call(c)
    for at, (_, _, sign) in zip(k, places):
        c["k"][at] = sign * float("inf")
    got, lse = tree_call(c)
    for i in range(drafts):
        if i % 2 == 0 or (key >= 2000 and not c["masks"][i] >> (key - 2000) & 1):
            assert torch.equal(got[i], want[i]) and torch.equal(lse[i], want_lse[i])
        else:
            assert bool(torch.isnan(got[i]).all()) and bool(torch.isnan(lse[i]).all())
    assert not got[drafts].any() and bool((lse[drafts] == -float("inf")).all())
    assert bool(torch.isnan(got[drafts + 1]).all()) and bool(torch.isnan(lse[drafts + 1]).all())


# up to 16 rows a key head, up to 32, more by each path
@pytest.mark.parametrize("Hq,page_size", [(2, 16), (2, 4), (8, 16), (8, 4)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_tree_special_values_reach_only_rows_that_see_them(value, Hq, page_size):
    c = tree_inputs([50], [20], Hq, 2, 128, page_size, torch.bfloat16, seed=5)
    ref, _ = tree_call(c)
    j = 7
    p = 50 + j
    page, row = int(c["table"][0, p // page_size]), p % page_size
    c["v"][page, 1, row, 5] = value
    got, _ = tree_call(c)
    hit = torch.zeros(20, Hq, 128, dtype=torch.bool, device=DEV)
    for i in range(20):
        if c["masks"][i] >> j & 1:
            hit[i, Hq // 2:, 5] = True
    assert torch.equal(got[~hit], ref[~hit])
    assert bool((torch.isnan(got[hit]) if value != value else got[hit] == value).all())


# one item of several pieces, the drafts on both sides of a tile's end; up to 16 rows a key head, up to 32, more
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("j", [3, 8])
@pytest.mark.parametrize("Hq,page_size", [(1, 16), (1, 4), (2, 64), (2, 4), (8, 16), (8, 4)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_tree_special_values_in_cut_items(dtype, Hq, page_size, j, value):
    c = tree_inputs([4090, 70], [12, 1], Hq, 1, 64, page_size, dtype, seed=43)
    ref, ref_lse = tree_call(c)
    check_attention(ref, ref_lse, tree_refs(c, c["masks"], 64 ** -0.5, heads=[Hq - 1]), 64, dtype, "cut")
    p = 4090 + j
    c["v"][int(c["table"][0, p // page_size]), 0, p % page_size, 5] = value
    got, lse = tree_call(c)
    hit = torch.zeros(13, Hq, 64, dtype=torch.bool, device=DEV)
    for i in range(12):
        hit[i, :, 5] = bool(c["masks"][i] >> j & 1)
    assert torch.equal(got[~hit], ref[~hit]) and torch.equal(lse, ref_lse)
    assert bool((torch.isnan(got[hit]) if value != value else got[hit] == value).all())


# heads that no tensor-core tile holds: the two-by-two warps, over pages of both forms
@pytest.mark.parametrize("Hq,Hkv,D,page_size,dtype", [
    (256, 1, 64, 16, torch.float16), (256, 1, 128, 64, torch.bfloat16), (160, 1, 128, 8, torch.bfloat16),
    (1024, 4, 64, 32, torch.float16)])
def test_tree_groups_of_more_than_128_heads(Hq, Hkv, D, page_size, dtype):
    c = tree_inputs([70, 0, 900, 33], [2, 1, 3, 0], Hq, Hkv, D, page_size, dtype, seed=44)
    out, lse = tree_call(c)
    heads = [0, 63, 64, 129, Hq - 1]
    check_attention(out, lse, tree_refs(c, c["masks"], D ** -0.5, heads=heads), D, dtype, "wide groups")
    again, _ = tree_call(c, flags=fb.FB_GEMV_PDL)
    assert torch.equal(again, out) and fb.fb_attn_errors() == 0
    p = 900                                                               # the third sequence's first drafted token
    c["v"][int(c["table"][2, p // page_size]), 0, p % page_size, 5] = float("nan")
    got, _ = tree_call(c)
    hit = torch.zeros_like(out, dtype=torch.bool)
    for i in range(3):
        hit[3 + i, :Hq // Hkv, 5] = bool(c["masks"][3 + i] & 1)
    assert torch.equal(got[~hit], out[~hit]) and bool(torch.isnan(got[hit]).all())


@pytest.mark.parametrize("where", ["page", "negative", "width"])
@pytest.mark.parametrize("Hq,page_size", [(8, 16), (8, 8), (64, 16), (64, 4)])
def test_tree_bad_pages_give_nan_and_an_error_bit(where, Hq, page_size):
    c = tree_inputs([300, 20, 45], [2, 1, 1], Hq, 2, 64, page_size, torch.float16, seed=6)
    ref, _ = tree_call(c)
    assert fb.fb_attn_errors() == 0
    if where == "width":
        c["table"] = np.ascontiguousarray(c["table"][:, :192 // page_size])   # 192 positions of 302
    else:
        c["table"][0, 3] = c["k"].shape[0] if where == "page" else -7
    out, lse = tree_call(c, None)
    assert fb.fb_attn_errors(clear=False) == 1 and fb.fb_attn_errors() == 1 and fb.fb_attn_errors() == 0
    assert bool(torch.isnan(out[:2]).all()) and bool(torch.isnan(lse[:2]).all())
    assert bool(torch.isfinite(out[2:]).all())
    assert torch.equal(out[2:], ref[2:])


def test_tree_bad_page_among_the_drafts_reaches_only_rows_that_see_it():
    c = tree_inputs([64], [20], 8, 2, 128, 8, torch.bfloat16, seed=12)
    ref, _ = tree_call(c)
    c["table"][0, 9] = -5                                                 # drafted tokens 8 to 15
    got, lse = tree_call(c)
    assert fb.fb_attn_errors() == 1
    for i in range(20):
        if c["masks"][i] >> 8 & 0xFF:
            assert bool(torch.isnan(got[i]).all()) and bool(torch.isnan(lse[i]).all())
        else:
            assert torch.equal(got[i], ref[i])


@pytest.mark.parametrize("Hq", [4, 64])
def test_tree_lengths_beyond_every_bound(Hq):
    c = tree_inputs([100, 30, 7], [1, 2, 1], Hq, 2, 64, 16, torch.bfloat16, seed=13)
    ref, _ = tree_call(c)
    c["lens"] = [2 ** 31 - 1, 30, -4]
    out, _ = tree_call(c)
    assert fb.fb_attn_errors() == 1
    assert bool(torch.isnan(out[0]).all()) and torch.equal(out[1:3], ref[1:3])
    c["lens"] = [100, 30, 0]                                              # a negative length is none
    again, _ = tree_call(c)
    assert torch.equal(again[3], out[3]) and fb.fb_attn_errors() == 0


@pytest.mark.parametrize("page_size,Hq,drafts", [(64, 8, 1), (4, 8, 1), (64, 8, 20)])
def test_tree_and_rope_in_a_cache_past_32_bits(page_size, Hq, drafts):
    # 2.4e9 elements of keys and as many of values; the sequence lies in the last pages
    Hkv, D = 8, 128
    pages = 2_400_000_000 // (Hkv * page_size * D)
    if torch.cuda.mem_get_info()[0] < 14 * 10 ** 9:
        pytest.skip("needs 14 GB")
    g = gen(31)
    k, v = (torch.empty(pages, Hkv, page_size, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    T = 70 + drafts
    need = -(-T // page_size)
    table = torch.arange(pages - need, pages, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    at = torch.arange(T, device=DEV)
    slots = (table[0, at // page_size].long() * page_size + at % page_size).to(torch.int32)
    q, kk, vv = (normal(g, T, H, D, dtype=torch.bfloat16) for H in (Hkv, Hkv, Hkv))
    qr, kr, _ = fb.fb_qk_norm_rope(q, kk, vv, at.to(torch.int32), fb.rope_frequencies(D))
    fb.fb_qk_norm_rope(q, kk, vv, at.to(torch.int32), fb.rope_frequencies(D), cache=(k, v), slots=slots)
    cu = torch.tensor([0, drafts], dtype=torch.int32, device=DEV)
    lens = torch.tensor([70], dtype=torch.int32, device=DEV)
    out = fb.fb_attn_tree(qr[70:], (k, v), table, lens, cu, drafts)
    want = fb.fb_attn_prompt(qr, kr, vv, torch.tensor([0, T], dtype=torch.int32, device=DEV))[70:]
    assert fb.fb_attn_errors() == 0
    assert (out.float() - want.float()).abs().max() <= 4 * HALF[torch.bfloat16] * vv.abs().max()


def test_tree_counts_above_max_draft():
    c = tree_inputs([33, 10], [4, 2], 4, 2, 64, 16, torch.float16, seed=7)
    out = torch.full((6, 4, 64), 9.0, dtype=torch.float16, device=DEV)
    ref, _ = tree_call(c, None)
    fb.fb_attn_errors()
    c["drafts"] = [3, 2]                                                  # max_draft = 3
    tree_call(c, None, out=out)
    assert fb.fb_attn_errors() == 1
    assert torch.equal(out[:3], ref[:3]) and bool((out[3] == 9.0).all()) and torch.equal(out[4:], ref[4:])


def test_tree_rows_of_no_sequence_and_strided_rows():
    c = tree_inputs([90, 20], [3, 2], 4, 2, 128, 16, torch.bfloat16, seed=8)
    ref, rl = tree_call(c)
    wide = torch.full((9, 4 * 128 + 64), 5.0, dtype=torch.bfloat16, device=DEV)
    wide[2:7, :512] = c["q"].reshape(5, 512)
    q = wide[:, :512].view(9, 4, 128)
    buf = torch.full((9, 4 * 128 + 8), -2.0, dtype=torch.bfloat16, device=DEV)
    out = buf[:, :512].view(9, 4, 128)
    lse = torch.full((9, 4), 11.0, device=DEV)
    cu = torch.tensor([2, 5, 7], dtype=torch.int32, device=DEV)
    masks = torch.tensor([0, 0] + c["masks"] + [0, 0], dtype=torch.int64, device=DEV)
    table = torch.tensor(np.pad(c["table"], ((0, 0), (0, 3)), constant_values=1 << 30), device=DEV)
    table = table[:, :c["table"].shape[1]]
    fb.fb_attn_tree(q, (c["k"], c["v"]), table, torch.tensor([90, 20], dtype=torch.int32, device=DEV), cu, 3, masks,
                    out=out, lse=lse)
    assert torch.equal(out[2:7], ref) and torch.equal(lse[2:7], rl)
    assert bool((buf[:, 512:] == -2.0).all()) and bool((out[:2] == -2.0).all()) and bool((out[7:] == -2.0).all())
    assert bool((lse[:2] == 11.0).all()) and bool((lse[7:] == 11.0).all())


@pytest.mark.parametrize("drafts", [1, 30])
def test_tree_graphs_with_a_workspace_each(drafts):
    c = tree_inputs([4000, 900], [drafts, drafts], 16, 2, 128, 64, torch.bfloat16, seed=9)
    cu = torch.tensor(c["cu"], device=DEV)
    table, lens = torch.tensor(c["table"], device=DEV), torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    ref = fb.fb_attn_tree(c["q"], (c["k"], c["v"]), table, lens, cu, drafts)
    outs = [torch.empty_like(ref) for _ in range(2)]
    wss = [torch.full((fb.fb_attn_tree_workspace_bytes(16, (c["k"], c["v"]), drafts, table.shape[1]),), 255, dtype=torch.uint8, device=DEV)
           for _ in range(2)]
    graphs = []
    for o, w in zip(outs, wss):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fb.fb_attn_tree(c["q"], (c["k"], c["v"]), table, lens, cu, drafts, out=o, ws=w)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    lens.copy_(torch.tensor([1234, 8], dtype=torch.int32, device=DEV))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], fb.fb_attn_tree(c["q"], (c["k"], c["v"]), table, lens, cu, drafts))


def test_prompt_and_tree_agree_on_a_chain():
    # the last 30 tokens of a prompt, as a drafted chain behind its first 170
    q, k, v, cu, cud = prompt_inputs([200], 8, 2, 128, torch.float16, seed=21)
    whole = fb.fb_attn_prompt(q, k, v, cud)
    pages = torch.zeros(2, 13, 2, 16, 128, dtype=torch.float16, device=DEV)
    for src, dst in zip((k, v), pages):
        dst.transpose(1, 2).reshape(-1, 2, 128)
        dst.copy_(torch.cat([src, src.new_zeros(8, 2, 128)]).view(13, 16, 2, 128).transpose(1, 2))
    table = torch.arange(13, dtype=torch.int32, device=DEV)[None]
    out = fb.fb_attn_tree(q[170:], (pages[0], pages[1]), table, torch.tensor([170], dtype=torch.int32, device=DEV),
                          torch.tensor([0, 30], dtype=torch.int32, device=DEV), 30)
    assert (out - whole[170:]).abs().max() <= 4 * HALF[torch.float16] * v.abs().max()
