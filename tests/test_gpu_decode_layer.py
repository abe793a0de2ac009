"""A decoder layer's attention from end to end, as a decode loop uses it: the
grouped q/k/v GEMV, the norm and rotation into the paged cache, the prompt's
attention, drafted trees over the cache, the o GEMV."""

import numpy as np
import pytest
import torch

import lut_binary_gemv_b200 as fb
import workloads as wl
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def test_layer_prompt_then_drafts():
    Hq, Hkv, D, width, P = 4, 2, 64, 256, 16
    dims = dict(K=2, nS=32, Ks=1, x_dtype="f16")
    wq = fb.Weights.from_problem(wl.make_problem(Hq * D, width, seed=1, **dims))
    wk = fb.Weights.from_problem(wl.make_problem(Hkv * D, width, seed=2, **dims))
    wv = fb.Weights.from_problem(wl.make_problem(Hkv * D, width, seed=3, **dims))
    wo = fb.Weights.from_problem(wl.make_problem(width, Hq * D, seed=4, **dims))
    g = torch.Generator(device=DEV).manual_seed(5)
    n_prompt, n_draft = 50, 5
    x = torch.randn(n_prompt + n_draft, width, generator=g, device=DEV).half()
    freq, nw = fb.rope_frequencies(D), 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    cache = tuple(torch.zeros(6, Hkv, P, D, dtype=torch.float16, device=DEV) for _ in range(2))
    table = torch.tensor([[4, 0, 5, 2]], dtype=torch.int32, device=DEV)
    at = torch.arange(n_prompt + n_draft, device=DEV)
    slots = (table[0, at // P] * P + at % P).to(torch.int32)
    depth = torch.tensor([0, 1, 1, 2, 2], device=DEV)                     # two branches behind the first draft
    masks = [0b1, 0b11, 0b101, 0b1011, 0b10101]
    pos = torch.cat([torch.arange(n_prompt, device=DEV), n_prompt + depth]).to(torch.int32)

    # the prompt: its projections in passes of up to 64 tokens
    q, k, v = (fb.fb_gemv_batched(w, x[:n_prompt]).view(n_prompt, -1, D) for w in (wq, wk, wv))
    qr, kr, vr = fb.fb_qk_norm_rope(q, k, v, pos[:n_prompt], freq, nw, nw, cache=cache, slots=slots[:n_prompt],
                                    k_out=torch.empty(n_prompt, Hkv, D, dtype=torch.float16, device=DEV),
                                    v_out=torch.empty(n_prompt, Hkv, D, dtype=torch.float16, device=DEV))
    cu = torch.tensor([0, n_prompt], dtype=torch.int32, device=DEV)
    prompt = fb.fb_attn_prompt(qr, kr, vr, cu)

    # the drafts: one grouped call a token, then all of them at once
    heads = [torch.stack(t) for t in zip(*(fb.fb_gemv_grouped([wq, wk, wv], xi) for xi in x[n_prompt:]))]
    qd, kd, vd = (t.view(n_draft, -1, D) for t in heads)
    qr2, _, _ = fb.fb_qk_norm_rope(qd, kd, vd, pos[n_prompt:], freq, nw, nw, cache=cache, slots=slots[n_prompt:])
    lens = torch.tensor([n_prompt], dtype=torch.int32, device=DEV)
    tree = fb.fb_attn_tree(qr2, cache, table, lens, torch.tensor([0, n_draft], dtype=torch.int32, device=DEV), n_draft,
                           torch.tensor(masks, dtype=torch.int64, device=DEV))
    y = fb.fb_gemv_batched(wo, tree.view(n_draft, Hq * D))
    last = fb.fb_gemv(wo, prompt[-1].reshape(-1))
    assert fb.fb_attn_errors() == 0

    # the same layer in fp64 from the projections on; fp16 queries, keys, values, weights and outputs each round
    # by 2^-11 relative, scores are below 8 * sqrt(8) in size (normed heads), so a weight moves by at most
    # 2 * 8 * 2^-10 relative: 0.02 of the largest value bounds the attention's error with room
    def turned(t, p):
        return A.rotate(A.norm(f64(t), f64(nw), 1e-6), p.cpu().numpy(), f64(freq), False)
    Q = np.concatenate([turned(q, pos[:n_prompt]), turned(qd, pos[n_prompt:])])
    K = np.concatenate([turned(k, pos[:n_prompt]), turned(kd, pos[n_prompt:])])
    V = np.concatenate([f64(v), f64(vd)])
    seen = np.tril(np.ones((n_prompt + n_draft,) * 2, bool))
    for i, m in enumerate(masks):
        for j in range(n_draft):
            seen[n_prompt + i, n_prompt + j] = bool(m >> j & 1)
    for h in range(Hq):
        ref, *_ = A.attend(Q[:, h], K[:, h // 2], V[:, h // 2], seen, D ** -0.5)
        got = np.concatenate([f64(prompt[:, h]), f64(tree[:, h])])
        assert np.abs(got - ref).max() <= 0.02 * np.abs(V[:, h // 2]).max()
    assert torch.equal(y[0], fb.fb_gemv_batched(wo, tree[:1].reshape(1, -1))[0])
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(last).all())
    rows = cache[1].transpose(1, 2).reshape(-1, Hkv, D)[slots.long()]
    assert torch.equal(rows, torch.cat([v, vd]).half())


def test_decode_step_as_one_graph():
    Hq, Hkv, D, width, P = 8, 2, 128, 1024, 16
    dims = dict(K=2, nS=0, x_dtype="f16")
    ws = [fb.Weights.from_problem(wl.make_problem(m, width, seed=s, **dims))
          for s, m in enumerate((Hq * D, Hkv * D, Hkv * D))]
    wo = fb.Weights.from_problem(wl.make_problem(width, Hq * D, seed=9, **dims))
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(width, generator=g, device=DEV).half()
    cache = tuple(torch.randn(20, Hkv, P, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    table = torch.randperm(20, generator=g, device=DEV).to(torch.int32)[None]
    lens = torch.tensor([77], dtype=torch.int32, device=DEV)
    pos, slots = lens.clone(), torch.empty(1, dtype=torch.int32, device=DEV)
    freq, y = fb.rope_frequencies(D), torch.empty(width, device=DEV)
    pdl = fb.FB_GEMV_PDL

    def step(flags):
        q, k, v = fb.fb_gemv_grouped(ws, x, flags=flags)
        qr, _, _ = fb.fb_qk_norm_rope(q.view(1, Hq, D), k.view(1, Hkv, D), v.view(1, Hkv, D), pos, freq, cache=cache,
                                      slots=slots, flags=flags)
        o = fb.fb_attn_tree(qr, cache, table, lens, flags=flags)
        return fb.fb_gemv(wo, o.view(-1), y, flags=flags)

    def at(n):
        lens.fill_(n), pos.fill_(n)
        slots.copy_(table[0, n // P:n // P + 1] * P + n % P)

    at(77)
    step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pdl)
    for n in (77, 78, 95, 96, 300):
        at(n)
        want = step(0).clone()
        y.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert fb.fb_attn_errors() == 0
