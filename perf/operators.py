"""Measured cases of the attention operators that stand beside the GEMV in a
decoder layer: the norm and rotation of projected heads, the attention of
packed prompts, and the attention of tokens and drafted trees over a paged
cache.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the library's calls; both take what `prepare` returns.

A case is a dict of plain values.  Ragged lengths are texts ("5,0,731").
"""

import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _numbers(text):
    return [int(s) for s in str(text).split(",")]


# ---- cases ------------------------------------------------------------------


def listed():
    return [
        # one decode step's token of a 4096-wide layer: fp32 heads straight from the grouped q/k/v GEMV
        {"name": "rotate_token", "op": "rotate", "T": 1, "Hq": 32, "Hkv": 32, "D": 128, "rot": 128, "norm": True,
         "pairs": "halves", "fused": False, "t_in": "f32", "t": "bf16", "pages": 64, "page_size": 64, "first": 2047},
        # a batched pass of 63 tokens with a partial rotation of neighbouring pairs, far positions, no norm
        {"name": "rotate_batch", "op": "rotate", "T": 63, "Hq": 64, "Hkv": 8, "D": 64, "rot": 32, "norm": False,
         "pairs": "neighbours", "fused": False, "t_in": "f16", "t": "f16", "pages": 37, "page_size": 16, "first": 1000003},
        # a long prompt of an 8192-wide layer with grouped heads, q/k/v as slices of one fused projection
        {"name": "rotate_prompt", "op": "rotate", "T": 16384, "Hq": 64, "Hkv": 8, "D": 128, "rot": 128, "norm": True,
         "pairs": "halves", "fused": True, "t_in": "bf16", "t": "bf16", "pages": 300, "page_size": 64, "first": 0},
        # one short prompt
        {"name": "prompt_short", "op": "prompt", "lens": "77", "tail": 0, "Hq": 32, "Hkv": 32, "D": 128, "t": "f16"},
        # a packed batch of prompts of a 4096-wide layer, one of them empty, padding rows behind the last
        {"name": "prompt_packed", "op": "prompt", "lens": "1,511,0,128,2900,1057,1300,2000,259", "tail": 36, "Hq": 32,
         "Hkv": 32, "D": 128, "t": "bf16"},
        # heads of 64 with groups of 8, sixteen short prompts
        {"name": "prompt_heads64", "op": "prompt",
         "lens": "700,901,333,64,1200,1025,87,510,777,1500,45,640,999,210,1111,1898", "tail": 0, "Hq": 32, "Hkv": 4,
         "D": 64, "t": "f16"},
        # one long prompt
        {"name": "prompt_long", "op": "prompt", "lens": "16384", "tail": 0, "Hq": 32, "Hkv": 8, "D": 128, "t": "bf16"},
        # one token of a short conversation: latency
        {"name": "token_short", "op": "tree", "lens": "333", "drafts": "1", "chain": True, "holes": False, "Hq": 32,
         "Hkv": 32, "D": 128, "t": "bf16", "page_size": 64},
        # one token each of 32 conversations of very different lengths, groups of 8
        {"name": "token_batch", "op": "tree",
         "lens": "131,8000,2047,517,3999,64,1,7203,255,4096,6011,900,12000,333,2500,5000,"
                 "4500,48,1023,7777,300,9100,2222,610,15000,80,3333,1500,6500,410,2750,5900",
         "drafts": ",".join(["1"] * 32), "chain": True, "holes": False, "Hq": 64, "Hkv": 8, "D": 128, "t": "bf16",
         "page_size": 64},
        # one token over a long cache: the long axis has to be split
        {"name": "token_long", "op": "tree", "lens": "131071", "drafts": "1", "chain": True, "holes": False, "Hq": 64,
         "Hkv": 8, "D": 128, "t": "bf16", "page_size": 64},
        # drafted trees of a few tokens each over small pages, every head with its own keys
        {"name": "tree_drafts", "op": "tree", "lens": "1500,40,2777,0,913,2048,600,3500",
         "drafts": "16,24,7,12,31,1,20,9", "chain": False, "holes": False, "Hq": 32, "Hkv": 32, "D": 128, "t": "f16",
         "page_size": 16},
        # full trees of 64 with groups of 8: 512 rows for each pair of keys and values
        {"name": "tree_wide", "op": "tree", "lens": "8192,5000,7001,6100", "drafts": "64,64,64,63", "chain": False,
         "holes": True, "Hq": 64, "Hkv": 8, "D": 128, "t": "bf16", "page_size": 128},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "prompt", "tree"])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    group = rng.choice([1, 2, 4, 5, 8] if Hkv <= 8 else [1])
    D = rng.choice([64, 128])
    t = rng.choice(["f16", "bf16"])
    case = {"op": op, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "t": t}
    if op == "rotate":
        T = _spread(rng, 1, 12000)
        page_size = rng.choice([1, 16, 64, 128])
        case |= {"T": T, "rot": rng.choice([D, D // 2, 16]), "norm": rng.random() < 0.7,
                 "pairs": rng.choice(["halves", "neighbours"]), "fused": rng.random() < 0.5,
                 "t_in": rng.choice(["f32", t]), "pages": (T + page_size - 1) // page_size + rng.randrange(1, 9),
                 "page_size": page_size, "first": rng.choice([0, _spread(rng, 1, 1000000)])}
    elif op == "prompt":
        n = rng.randrange(1, 13)
        lens = [0 if rng.random() < 0.1 else _spread(rng, 1, 16384) for _ in range(n)]
        while sum(v * v for v in lens) * Hkv * group > 8 * 10**9:   # stays below the longest listed prompt
            lens[lens.index(max(lens))] //= 2
        if not any(lens):
            lens[0] = 1
        case |= {"lens": ",".join(map(str, lens)), "tail": rng.choice([0, 0, rng.randrange(1, 40)])}
    else:
        n = _spread(rng, 1, 48)
        chain = rng.random() < 0.4
        most = 64 if n <= 8 else 16
        cap = min(60000, 2 * 10**9 // (n * Hkv * D * 4))
        lens = [0 if rng.random() < 0.05 else _spread(rng, 1, min(cap, 20000 if n > 2 else cap)) for _ in range(n)]
        drafts = [1 if chain else _spread(rng, 1, most) for _ in range(n)]
        case |= {"lens": ",".join(map(str, lens)), "drafts": ",".join(map(str, drafts)), "chain": chain,
                 "holes": (not chain) and rng.random() < 0.5, "page_size": rng.choice([8, 16, 64, 128, 256])}
    return case


def work(case):
    D, Hq, Hkv, t = case["D"], case["Hq"], case["Hkv"], 2
    if case["op"] == "rotate":
        T, heads = case["T"], Hq + 2 * Hkv
        t_in = 4 if case["t_in"] == "f32" else 2
        norm = 2 * D * 4 if case["norm"] else 0
        # the heads in and out, one position and one slot a token, the frequencies, the norms' weights;
        # three operations an element of a norm, three an element of a rotation, on q and k
        return {"bytes": T * heads * D * (t_in + t) + 8 * T + 4 * case["rot"] + norm,
                "flops": T * (Hq + Hkv) * ((3 * D if case["norm"] else 0) + 3 * case["rot"])}
    if case["op"] == "prompt":
        lens = _numbers(case["lens"])
        T = sum(lens)
        return {"bytes": T * D * t * 2 * (Hq + Hkv) + 4 * T * Hq + 4 * (len(lens) + 1),
                "flops": sum(2 * D * Hq * n * (n + 1) for n in lens)}
    lens, drafts = _numbers(case["lens"]), _numbers(case["drafts"])
    keys = sum(a + b for a, b in zip(lens, drafts))
    T = sum(drafts)
    return {"bytes": keys * Hkv * D * t * 2 + T * Hq * D * t * 2 + 4 * T * Hq + 8 * T
            + 4 * sum(-(-(a + b) // case["page_size"]) for a, b in zip(lens, drafts)),
            "flops": sum(4 * D * Hq * b * (a + (b + 1) / 2) for a, b in zip(lens, drafts))}


# ---- inputs -----------------------------------------------------------------


def _heads(g, T, H, D, dtype):
    """Rows of normal values whose channels differ in size, as projections' do."""
    size = torch.exp(0.4 * torch.randn(H, D, generator=g, device="cuda"))
    size /= size.square().mean().sqrt()
    return (torch.randn(T, H, D, generator=g, device="cuda") * size).to(dtype)


def _tree_masks(drafts, chain, holes, g):
    """One 64-bit mask a drafted token: bit j is set where it sees drafted token j of its sequence."""
    pick = torch.rand(sum(drafts), 2, generator=g, device="cuda").cpu().tolist()
    masks, at = [], 0
    for m in drafts:
        seen = []
        for j in range(m):
            u, hole = pick[at]
            at += 1
            parent = j - 1 if chain else int(u * (j + 1)) - 1
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << j))
            if holes and hole < 0.1:
                masks.append(0)           # a padded draft: it sees the committed keys alone
            else:
                masks.append(seen[j])
    return torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in masks], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    D, Hq, Hkv, dtype = case["D"], case["Hq"], case["Hkv"], _TYPES[case["t"]]
    st = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "rotate":
        T, rot, t_in = case["T"], case["rot"], _TYPES[case["t_in"]]
        qkv = _heads(g, T, Hq + 2 * Hkv, D, t_in)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not case["fused"]:
            st["q"], st["k"], st["v"] = st["q"].contiguous(), st["k"].contiguous(), st["v"].contiguous()
        st["pos"] = torch.arange(T, device="cuda", dtype=torch.int32) + case["first"]
        st["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        weight = lambda: 1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")  # noqa: E731
        st["wq"], st["wk"] = (weight(), weight()) if case["norm"] else (None, None)
        st["eps"] = 1e-6
        pages, size = case["pages"], case["page_size"]
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        st["slots"] = (order[t // size] * size + t % size).to(torch.int32)
        k, v = (torch.zeros(pages, Hkv, size, D, dtype=dtype, device="cuda") for _ in range(2))
        st["q_out"] = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    elif case["op"] == "prompt":
        lens = _numbers(case["lens"])
        T = sum(lens) + case["tail"]
        st["q"], st["k"], st["v"] = (_heads(g, T, H, D, dtype) for H in (Hq, Hkv, Hkv))
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        st["ends"] = ends
        st["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        st["out"] = torch.zeros(T, Hq, D, dtype=dtype, device="cuda")
        st["lse"] = torch.zeros(T, Hq, dtype=torch.float32, device="cuda")
    else:
        lens, drafts = _numbers(case["lens"]), _numbers(case["drafts"])
        size, n, T = case["page_size"], len(lens), sum(drafts)
        need = [-(-(a + b) // size) for a, b in zip(lens, drafts)]
        pages = sum(need)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((n, max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = order[at:at + m]
            at += m
        k, v = (_heads(g, pages * size, Hkv, D, dtype).view(pages, size, Hkv, D).transpose(1, 2).contiguous()
                for _ in range(2))
        st["q"] = _heads(g, T, Hq, D, dtype)
        starts = [0]
        for m in drafts:
            starts.append(starts[-1] + m)
        st["table"], st["cu"] = table, torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["most"] = max(drafts)
        st["longest"] = max(a + b for a, b in zip(lens, drafts))
        st["mask"] = None if case["chain"] else _tree_masks(drafts, False, case["holes"], g)
        st["out"] = torch.zeros(T, Hq, D, dtype=dtype, device="cuda")
        st["lse"] = torch.zeros(T, Hq, dtype=torch.float32, device="cuda")
    if case["op"] != "prompt":
        st["k_pages"], st["v_pages"] = k, v
    return st


# ---- one pass ---------------------------------------------------------------


def run(st):
    if own:
        return _library(st)
    return {"rotate": _plain_rotate, "prompt": _plain_prompt, "tree": _plain_tree}[st["case"]["op"]](st)


def _library(st):
    import lut_binary_gemv_b200 as fb
    op = st["case"]["op"]
    if op == "rotate":
        fb.fb_qk_norm_rope(st["q"], st["k"], st["v"], st["pos"], st["inv_freq"], q_weight=st["wq"], k_weight=st["wk"],
                           eps=st["eps"], interleaved=st["case"]["pairs"] == "neighbours", cache=(st["k_pages"], st["v_pages"]),
                           slots=st["slots"], q_out=st["q_out"])
        return [st["q_out"], st["k_pages"], st["v_pages"]]
    if op == "prompt":
        fb.fb_attn_prompt(st["q"], st["k"], st["v"], st["cu"], scale=st["scale"], out=st["out"], lse=st["lse"])
    else:
        fb.fb_attn_tree(st["q"], (st["k_pages"], st["v_pages"]), st["table"], st["lens"], cu_draft=st["cu"], max_draft=st["most"],
                        mask=st["mask"], scale=st["scale"], out=st["out"], lse=st["lse"])
    return [st["out"], st["lse"]]


def _plain_rotate(st):
    case = st["case"]
    rot, dtype = case["rot"], st["q_out"].dtype
    turn = torch.remainder(st["pos"].double()[:, None] * st["inv_freq"], 2 * math.pi).float()   # far positions: 64 bits
    cos, sin = torch.cos(turn)[:, None], torch.sin(turn)[:, None]

    def rotated(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w
        y = x.clone()
        if case["pairs"] == "halves":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        return y.to(dtype)

    st["q_out"].copy_(rotated(st["q"], st["wq"]))
    page, at = st["slots"].long() // case["page_size"], st["slots"].long() % case["page_size"]
    st["k_pages"][page, :, at] = rotated(st["k"], st["wk"])
    st["v_pages"][page, :, at] = st["v"].to(dtype)
    return [st["q_out"], st["k_pages"], st["v_pages"]]


def _weighted(scores, v):
    """softmax(scores) @ v and the logarithm of the softmax's sum, in place on the scores; where a row has no
    finite score, zeros and minus infinity."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights, v) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (torch.log(total) + top).squeeze(-1)


def _plain_prompt(st):
    Hq, Hkv, D = st["case"]["Hq"], st["case"]["Hkv"], st["case"]["D"]
    group = Hq // Hkv
    for a, b in zip(st["ends"][:-1], st["ends"][1:]):     # the packed sequences
        if a == b:
            continue
        n = b - a
        q = st["q"][a:b].float().view(n, Hkv, group, D).permute(1, 2, 0, 3).reshape(Hkv, group * n, D)
        k, v = st["k"][a:b].float().transpose(0, 1), st["v"][a:b].float().transpose(0, 1)
        scores = torch.matmul(q * st["scale"], k.transpose(1, 2)).view(Hkv, group, n, n)
        i = torch.arange(n, device="cuda")
        scores.masked_fill_(i[None, :] > i[:, None], -math.inf)
        out, lse = _weighted(scores.view(Hkv, group * n, n), v)
        st["out"][a:b] = out.view(Hq, n, D).transpose(0, 1).to(st["out"].dtype)
        st["lse"][a:b] = lse.view(Hq, n).transpose(0, 1)
    return [st["out"], st["lse"]]


def _plain_tree(st):
    case = st["case"]
    Hq, Hkv, D, size = case["Hq"], case["Hkv"], case["D"], case["page_size"]
    group, n, most, longest = Hq // Hkv, st["lens"].numel(), st["most"], st["longest"]
    pages = st["table"].clamp(min=0).long()
    key = torch.arange(longest, device="cuda")
    where = pages[:, key // size] * size + key % size                                  # [n, longest]
    k, v = (x.transpose(1, 2).reshape(-1, Hkv, D)[where].float().transpose(1, 2) for x in (st["k_pages"], st["v_pages"]))
    counts = st["cu"][1:] - st["cu"][:-1]
    draft = torch.arange(most, device="cuda")
    there = draft < counts[:, None]                                                     # [n, most]
    token = torch.where(there, st["cu"][:-1, None] + draft, 0).long()
    q = st["q"][token].float().view(n, most, Hkv, group, D).permute(0, 2, 1, 3, 4).reshape(n, Hkv, most * group, D)
    scores = torch.matmul(q * st["scale"], k.transpose(2, 3)).view(n, Hkv, most, group, longest)
    j = key - st["lens"][:, None]                                                       # the drafted token a key is
    if st["mask"] is None:
        seen = j[:, None] <= draft[:, None]
    else:
        bit = (st["mask"][token][:, :, None] >> j.clamp(0, 63)[:, None]) & 1
        seen = (j[:, None] < 0) | ((bit == 1) & (j < counts[:, None])[:, None])
    scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    # a value that no row sees may be anything, so it is cleared before it meets a weight of zero
    v = v.masked_fill_(~seen.any(1)[:, None, :, None], 0.0)
    out, lse = _weighted(scores.view(n, Hkv, most * group, longest), v)
    out = out.view(n, Hkv, most, group, D).permute(0, 2, 1, 3, 4).reshape(n, most, Hq, D)
    lse = lse.view(n, Hkv, most, group).permute(0, 2, 1, 3).reshape(n, most, Hq)
    st["out"][token[there]] = out[there].to(st["out"].dtype)
    st["lse"][token[there]] = lse[there]
    return [st["out"], st["lse"]]


# ---- the definition in 64 bits ----------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    group = Hq // Hkv
    if case["op"] == "rotate":
        rot = case["rot"]
        angle = st["pos"].double().outer(st["inv_freq"])
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]                      # cos + i sin

        def rotated(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + st["eps"]) * w.double()
            head, rest = x[..., :rot], x[..., rot:]
            shape = (2, rot // 2) if case["pairs"] == "halves" else (rot // 2, 2)
            pairs = head.reshape(*head.shape[:-1], *shape)
            if case["pairs"] == "halves":
                pairs = pairs.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            if case["pairs"] == "halves":
                z = z.transpose(-1, -2)
            return torch.cat([z.reshape(head.shape), rest], -1)

        pages, size = case["pages"], case["page_size"]
        rows = [torch.zeros(pages * size, Hkv, D, dtype=torch.float64, device="cuda") for _ in range(2)]
        rows[0].index_copy_(0, st["slots"].long(), rotated(st["k"], st["wk"]))
        rows[1].index_copy_(0, st["slots"].long(), st["v"].double())
        k, v = (r.view(pages, size, Hkv, D).transpose(1, 2).contiguous() for r in rows)
        return [rotated(st["q"], st["wq"]), k, v]
    T = st["q"].shape[0]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")

    def attend(rows, head, q, k, v, seen):
        s = (q.double() @ k.double().T) / math.sqrt(D)
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
        out[rows, head], lse[rows, head] = p @ v.double(), z

    if case["op"] == "prompt":
        for a, b in zip(st["ends"][:-1], st["ends"][1:]):
            for h in range(Hq if b > a else 0):
                seen = torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").tril()
                attend(slice(a, b), h, st["q"][a:b, h], st["k"][a:b, h // group], st["v"][a:b, h // group], seen)
        return [out, lse]
    lens, drafts = _numbers(case["lens"]), _numbers(case["drafts"])
    masks = None if st["mask"] is None else st["mask"].cpu().tolist()
    at = 0
    for i, (a, m) in enumerate(zip(lens, drafts)):
        used = st["table"][i, :-(-(a + m) // case["page_size"])].long()
        k, v = (x[used].transpose(1, 2).reshape(-1, Hkv, D)[:a + m] for x in (st["k_pages"], st["v_pages"]))
        seen = torch.ones(m, a + m, dtype=torch.bool)
        for r in range(m):
            for j in range(m):
                seen[r, a + j] = j <= r if masks is None else bool(masks[at + r] >> j & 1)
        seen = seen.cuda()
        for h in range(Hq):
            attend(slice(at, at + m), h, st["q"][at:at + m, h], k[:, h // group], v[:, h // group], seen)
        at += m
    return [out, lse]
