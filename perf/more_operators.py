"""The attention half of a block around the ternary linear layer, as cases to be measured.

Three operators, in the order in which a block runs them:

  int8       int8_linear: the product of rotated int8 activations with a weight that
             is held in 8 bits (the projections that are not ternary), one scale for
             each token and one for each channel.
  rope       qk_norm_rope: RMSNorm of every query and key head of the projection's
             output and the position rotation, keys and values into the pages of a
             cache.
  attention  window_attention: causal attention over those pages with a sliding
             window and a few first tokens that stay visible, for prompts, chunks,
             drafted tokens and single tokens.

`run` computes a case in elementary torch operations, or, with `own` set, by the
calls a user makes of the library.
"""
import math
import random

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one new token of one request through a fused query/key/value projection
        {"name": "int8 1 token", "op": "int8", "M": 1, "K": 5120, "N": 7168, "dtype": "bfloat16", "bias": False},
        # 24 streams' new tokens through the output head, logits in fp32
        {"name": "int8 24 tokens wide", "op": "int8", "M": 24, "K": 5120, "N": 65536, "dtype": "float32", "bias": False},
        # a ragged chunk through a small layer of odd sizes with a bias
        {"name": "int8 333 tokens odd", "op": "int8", "M": 333, "K": 2064, "N": 4001, "dtype": "float32", "bias": True},
        # long prompts batched, the widest projection
        {"name": "int8 4096 tokens", "op": "int8", "M": 4096, "K": 5120, "N": 17408, "dtype": "bfloat16", "bias": False},
        # one new token between its projection and the attention
        {"name": "rope 1 token", "op": "rope", "M": 1, "n_q": 40, "n_kv": 8, "D": 128, "rot": 128, "dtype": "bfloat16",
         "norm": True, "interleaved": False, "page": 64},
        # 24 streams, wide heads of which a quarter is rotated, an fp32 projection
        {"name": "rope 24 tokens partial", "op": "rope", "M": 24, "n_q": 20, "n_kv": 4, "D": 256, "rot": 64, "dtype": "float32",
         "norm": True, "interleaved": False, "page": 16},
        # long prompts batched
        {"name": "rope 8192 tokens", "op": "rope", "M": 8192, "n_q": 40, "n_kv": 8, "D": 128, "rot": 128, "dtype": "bfloat16",
         "norm": True, "interleaved": False, "page": 64},
        # one new token of one request over a middling context
        {"name": "attention 1 token", "op": "attention", "kind": "decode", "B": 1, "q": 1, "kv": 5000, "n_q": 40, "n_kv": 8, "D": 128,
         "page": 64, "window": 0, "sinks": 0, "mix": 1},
        # 24 streams' new tokens over long contexts of uneven length
        {"name": "attention 24 tokens", "op": "attention", "kind": "decode", "B": 24, "q": 1, "kv": 16384, "n_q": 20, "n_kv": 4, "D": 256,
         "page": 64, "window": 0, "sinks": 0, "mix": 2},
        # a few drafted tokens of eight streams to be verified, a window over long contexts
        {"name": "attention drafts", "op": "attention", "kind": "drafts", "B": 8, "q": 8, "kv": 6000, "n_q": 16, "n_kv": 2, "D": 64,
         "page": 16, "window": 1024, "sinks": 4, "mix": 3},
        # uneven chunks of five prompts, part of each prompt in the cache before
        {"name": "attention ragged chunks", "op": "attention", "kind": "chunks", "B": 5, "q": 1000, "kv": 4000, "n_q": 20, "n_kv": 4, "D": 256,
         "page": 16, "window": 1000, "sinks": 5, "mix": 4},
        # one long prompt
        {"name": "attention 8192 tokens", "op": "attention", "kind": "prompts", "B": 1, "q": 8192, "kv": 8192, "n_q": 40, "n_kv": 8, "D": 128,
         "page": 64, "window": 4096, "sinks": 4, "mix": 5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["int8", "rope", "attention"])
    if op == "int8":
        K = 1024 * _log(rng, 1, 17) if rng.random() < 0.5 else 16 * _log(rng, 2, 1088)
        N = _log(rng, 16, 65536)
        M = _log(rng, 1, min(8192, max(1, 4096 * 5120 * 17408 // (K * N))))
        return {"op": op, "M": M, "K": K, "N": N, "dtype": rng.choice(["float32", "bfloat16"]), "bias": rng.random() < 0.3}
    D = rng.choice([64, 128, 256])
    n_kv, group = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        M = _log(rng, 1, 8192 * 48 * 128 // (n_kv * (group + 2) * D) if n_kv * (group + 2) * D > 6144 else 8192)
        return {"op": op, "M": M, "n_q": n_kv * group, "n_kv": n_kv, "D": D, "rot": rng.choice([D, D // 2, D // 4]),
                "dtype": rng.choice(["float32", "bfloat16"]), "norm": rng.random() < 0.75, "interleaved": rng.random() < 0.3, "page": page}
    kind = rng.choice(["decode", "decode", "drafts", "chunks", "prompts", "mixed"])
    B = _log(rng, 1, {"decode": 48, "drafts": 24, "chunks": 6, "prompts": 4, "mixed": 12}[kind])
    heads = n_kv * group
    if kind in ("decode", "drafts"):
        kv, q = _log(rng, 1, min(32768, 24 * 16384 * 1024 // (B * n_kv * D))), 1 if kind == "decode" else rng.randint(2, 12)
        kv = max(kv, q)
    else:
        # padded scores of the plain form, and products, of at most the largest listed case's
        kv = _log(rng, 16, min(8192, math.isqrt(12 * 8192 * 8192 * 128 // (B * heads * D))))
        q = kv if kind == "prompts" else max(1, kv * rng.randint(1, 3) // 4)
    window = rng.choice([0, _log(rng, 1, 4096)])
    return {"op": op, "kind": kind, "B": B, "q": q, "kv": kv, "n_q": heads, "n_kv": n_kv, "D": D, "page": page,
            "window": window, "sinks": rng.choice([0, 1, 4, 16]) if window else 0, "mix": rng.randrange(1 << 30)}


def _lengths(case):
    """New tokens and context length of every sequence of an attention case."""
    rng = random.Random(case["mix"])
    out = []
    for b in range(case["B"]):
        kv = case["kv"] if b == 0 else rng.randint(max(1, case["kv"] // 8), case["kv"])
        q = case["q"] if b == 0 else rng.randint(1, case["q"])
        if case["kind"] == "mixed" and b % 2:  # every other sequence decodes
            q = 1
        q = min(q, kv)
        out.append((kv if case["kind"] == "prompts" else q, kv))
    return out


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _pages(g, count, spare=3):
    """A cache's pages in the order in which a server hands them out after a while: any."""
    return torch.randperm(count + spare, generator=g, device="cuda")[:count].to(torch.int32), count + spare


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, bf = case["op"], torch.bfloat16
    s = {"case": case}
    if op == "int8":
        M, K, N = case["M"], case["K"], case["N"]
        # activations as the rotation leaves them: near normal, the row's largest at 127
        x = _randn(g, M, K)
        top = x.abs().amax(1, keepdim=True)
        s["x_i8"] = torch.round(x * (127.0 / top)).to(torch.int8)
        s["a_scale"] = (top[:, 0] * (0.5 + torch.rand(M, generator=g, device="cuda")) / 127.0)
        w = _randn(g, N, K)
        top = w.abs().amax(1, keepdim=True)
        s["w_i8"] = torch.round(w * (127.0 / top)).to(torch.int8)
        s["w_scale"] = top[:, 0] * (0.5 + torch.rand(N, generator=g, device="cuda")) / (127.0 * math.sqrt(K))
        s["bias"] = 0.1 * _randn(g, N) if case["bias"] else None
        return s
    n_q, n_kv, D, page = case["n_q"], case["n_kv"], case["D"], case["page"]
    if op == "rope":
        M, rot = case["M"], case["rot"]
        s["qkv"] = (_randn(g, M, (n_q + 2 * n_kv) * D) * (0.2 + 2.0 * torch.rand(M, 1, generator=g, device="cuda"))).to(getattr(torch, case["dtype"]))
        for name in ("q_weight", "k_weight"):
            s[name] = (1.0 + 0.2 * _randn(g, D)).to(bf) if case["norm"] else None
        n_pos = 32768
        # the angles of far positions in 64 bits
        inverse = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inverse
        s["cos_sin"] = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
        if M <= 64:  # streams that decode, each at a place of its own
            s["positions"] = torch.randint(0, n_pos, (M,), generator=g, device="cuda").to(torch.int32)
            pages, n_pages = _pages(g, M)
            s["slots"] = pages * page + s["positions"] % page
        else:  # prompts, one after the other
            cut = M // 3
            i = torch.arange(M, device="cuda")
            s["positions"] = torch.where(i < cut, i, i - cut).to(torch.int32)
            pages, n_pages = _pages(g, (cut + page - 1) // page + (M - cut + page - 1) // page)
            place = torch.where(i < cut, i, i - cut + (cut + page - 1) // page * page)
            s["slots"] = (pages[place // page] * page + (place % page).to(torch.int32))
        s["k_cache"] = _randn(g, n_pages, n_kv, page, D).to(bf)
        s["v_cache"] = _randn(g, n_pages, n_kv, page, D).to(bf)
        return s
    lengths = _lengths(case)
    B = len(lengths)
    need = [(kv + page - 1) // page for _, kv in lengths]
    pages, n_pages = _pages(g, sum(need))
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    table = table.cuda()
    s["page_table"] = torch.where(table >= 0, pages[table.long().clamp(min=0)], -1).to(torch.int32)
    starts = [0]
    for q, _ in lengths:
        starts.append(starts[-1] + q)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32).cuda()
    s["kv_len"] = torch.tensor([kv for _, kv in lengths], dtype=torch.int32).cuda()
    s["longest"] = (max(q for q, _ in lengths), max(kv for _, kv in lengths))
    # normed queries and keys of a common direction; the first tokens draw attention, as they do in earnest
    common = _randn(g, n_kv, 1, D)
    s["q"] = (_randn(g, starts[-1], n_kv, n_q // n_kv, D) + 0.5 * common).to(bf).view(starts[-1], n_q, D)
    s["k_cache"] = _randn(g, n_pages, n_kv, page, D).to(bf)
    s["v_cache"] = _randn(g, n_pages, n_kv, page, D).to(bf)
    first = s["page_table"][:, 0].long()
    s["k_cache"][first, :, 0:2] = (s["k_cache"][first, :, 0:2].float() + 0.6 * common).to(bf)
    return s


def _own_int8(s):
    import ternary_weight_linear_block_amd as twl
    return twl.int8_linear(s["x_i8"], s["a_scale"], s["w_i8"], s["w_scale"], bias=s["bias"], out_dtype=getattr(torch, s["case"]["dtype"]))


def _plain_int8(s):
    y = (s["x_i8"].float() @ s["w_i8"].float().t()) * s["a_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(getattr(torch, s["case"]["dtype"]))


def _own_rope(s):
    import ternary_weight_linear_block_amd as twl
    c = s["case"]
    q, k_cache, v_cache = twl.qk_norm_rope(
        s["qkv"], s["positions"], s["cos_sin"], c["n_q"], c["n_kv"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
        interleaved=c["interleaved"], slots=s["slots"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    return {"q": q, "k_cache": k_cache, "v_cache": v_cache}


def _plain_rope(s):
    c = s["case"]
    n_q, n_kv, D, rot, M = c["n_q"], c["n_kv"], c["D"], c["rot"], c["M"]
    x = s["qkv"].float().view(M, n_q + 2 * n_kv, D)
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., : rot // 2], cs[..., rot // 2:]

    def turned(t, weight):
        if weight is not None:
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * weight.float()
        if c["interleaved"]:
            a, b = t[..., 0:rot:2], t[..., 1:rot:2]
            front = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = t[..., : rot // 2], t[..., rot // 2: rot]
            front = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((front, t[..., rot:]), -1).to(torch.bfloat16)

    page, where = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    s["k_cache"][page, :, where] = turned(x[:, n_q: n_q + n_kv], s["k_weight"])
    s["v_cache"][page, :, where] = x[:, n_q + n_kv:].to(torch.bfloat16)
    return {"q": turned(x[:, :n_q], s["q_weight"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import ternary_weight_linear_block_amd as twl
    c = s["case"]
    return twl.window_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_start"], s["kv_len"],
                                window=c["window"], sinks=c["sinks"])


def _plain_attention(s):
    # sequences padded to the longest
    c = s["case"]
    n_q, n_kv, D, page = c["n_q"], c["n_kv"], c["D"], c["page"]
    (Lq, Lk), B, group = s["longest"], c["B"], n_q // n_kv
    dev = s["q"].device
    j, i = torch.arange(Lk, device=dev), torch.arange(Lq, device=dev)
    pages = s["page_table"].long()[:, j // page].clamp(min=0)
    k = s["k_cache"][pages, :, j % page].permute(0, 2, 3, 1).float()      # [B, n_kv, D, Lk]
    v = s["v_cache"][pages, :, j % page].permute(0, 2, 1, 3).float()      # [B, n_kv, Lk, D]
    start, kv = s["q_start"].long(), s["kv_len"].long()
    n = start[1:] - start[:-1]
    t = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][t].float().view(B, Lq, n_kv, group, D).permute(0, 2, 3, 1, 4).reshape(B, n_kv, group * Lq, D)
    p = (kv - n)[:, None] + i
    seen = (j <= p[:, :, None]) & (j < kv[:, None, None])
    if c["window"]:
        seen &= (p[:, :, None] - j < c["window"]) | (j < c["sinks"])
    x = (q @ k).mul_(1.0 / math.sqrt(D)).view(B, n_kv, group, Lq, Lk)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(-1)
    out = (x.view(B, n_kv, group * Lq, Lk) @ v).view(B, n_kv, group, Lq, D) / total.clamp(min=1e-30)[..., None]
    rows = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(start, rows, right=True) - 1
    return out.permute(0, 3, 1, 2, 4)[b, rows - start[b]].reshape(-1, n_q, D).to(torch.bfloat16)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"int8": _own_int8, "rope": _own_rope, "attention": _own_attention}[op](state)
    return {"int8": _plain_int8, "rope": _plain_rope, "attention": _plain_attention}[op](state)


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "int8":
        # each output channel's own sum; the products are whole numbers
        x, out = s["x_i8"].double(), []
        for w, scale in zip(s["w_i8"].split(8192), s["w_scale"].split(8192)):
            out.append(torch.mm(x, w.double().t()) * torch.outer(s["a_scale"].double(), scale.double()))
        y = torch.cat(out, 1)
        return y if s["bias"] is None else y + s["bias"].double()
    n_q, n_kv, D, page = case["n_q"], case["n_kv"], case["D"], case["page"]
    if case["op"] == "rope":
        M, half = case["M"], case["rot"] // 2
        q, k, v = s["qkv"].double().split([n_q * D, n_kv * D, n_kv * D], 1)
        table = s["cos_sin"].double().index_select(0, s["positions"].long())
        turn = torch.complex(table[:, :half], table[:, half:])[:, None]

        def heads(x, n, weight):
            x = x.reshape(M, n, D)
            if weight is not None:
                x = x / ((x * x).sum(2, keepdim=True) / D + EPS).sqrt() * weight.double()
            pairs = x[..., : 2 * half].reshape(M, n, half, 2) if case["interleaved"] else x[..., : 2 * half].reshape(M, n, 2, half).transpose(2, 3)
            z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn)
            z = z if case["interleaved"] else z.transpose(2, 3)
            return torch.cat((z.reshape(M, n, 2 * half), x[..., 2 * half:]), 2)

        caches = []
        for cache, new in ((s["k_cache"], heads(k, n_kv, s["k_weight"])), (s["v_cache"], v.reshape(M, n_kv, D))):
            flat = cache.double().transpose(1, 2).reshape(-1, n_kv, D)
            flat[s["slots"].long()] = new
            caches.append(flat.reshape(-1, page, n_kv, D).transpose(1, 2).contiguous())
        return {"q": heads(q, n_q, s["q_weight"]), "k_cache": caches[0], "v_cache": caches[1]}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, kv) in enumerate(_lengths(case)):
        used = s["page_table"][b, : (kv + page - 1) // page].long()
        for h in range(n_kv):
            k = s["k_cache"][used, h].reshape(-1, D)[:kv].double()
            v = s["v_cache"][used, h].reshape(-1, D)[:kv].double()
            for at in range(0, n, 1024):
                m = min(1024, n - at)
                query = s["q"][row + at: row + at + m, h * (n_q // n_kv): (h + 1) * (n_q // n_kv)].double()
                behind = (kv - n + at + torch.arange(m, device="cuda"))[:, None] - torch.arange(kv, device="cuda")[None, :]
                hidden = behind < 0
                if case["window"]:
                    hidden |= (behind >= case["window"]) & (torch.arange(kv, device="cuda") >= case["sinks"])[None, :]
                score = torch.matmul(query.transpose(0, 1), k.t()) / math.sqrt(D)
                weight = torch.softmax(torch.where(hidden, -math.inf, score), -1)
                out[row + at: row + at + m, h * (n_q // n_kv): (h + 1) * (n_q // n_kv)] = torch.matmul(weight, v).transpose(0, 1)
        row += n
    return out


def work(case):
    op = case["op"]
    size = 4 if case.get("dtype") == "float32" else 2
    if op == "int8":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * (K + 4) + N * (K + 4 + 4 * case["bias"]) + size * M * N, "flops": 2 * M * N * K}
    n_q, n_kv, D = case["n_q"], case["n_kv"], case["D"]
    if op == "rope":
        return {"bytes": case["M"] * ((n_q + 2 * n_kv) * D * (size + 2) + 4 * case["rot"] + 8), "flops": case["M"] * (n_q + n_kv) * D * 8}
    tokens = pairs = keys = 0
    w, sinks = case["window"], case["sinks"]
    for n, kv in _lengths(case):
        first = kv - n  # the first new token's position
        tokens += n
        if w:
            pairs += sum(min(p + 1, w) + min(sinks, max(0, p + 1 - w)) for p in range(first, kv))
            keys += min(kv, n + w - 1 + min(sinks, max(0, first + 1 - w)))
        else:
            pairs += n * first + n * (n + 1) // 2
            keys += kv
    return {"bytes": 4 * tokens * n_q * D + 4 * keys * n_kv * D, "flops": 4 * pairs * n_q * D}
