"""The block operators around the ternary linear layer, as cases to be measured.

Three operators, all at the layer's own boundary (bf16 activations in, rotated
int8 activations or projection outputs out):

  norm    norm_rotate_quant_act: RMSNorm of a block's output, gate, residual
          scale and residual add, RMSNorm before the next block, then the signed
          block-1024 Hadamard rotation and the per-token int8 quantisation.
  lora    lora_add: y + scale[id] * (x A[id]^T) B[id]^T, one adapter (or none)
          for each token, beside the shared projection that made y.
  gated   ternary_gated_linear: SiLU(gate) * up of the two ternary projections
          of one quantised input.

`run` computes a case in elementary torch operations, or, with `own` set, by the
calls a user makes of the library.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK, GROUP = 1024, 128


def listed():
    return [
        # one new token of one request, between two blocks that norm their output
        {"name": "norm 1 token", "op": "norm", "M": 1, "K": 5120, "residual": True, "post": True, "gate": "none", "normed": False},
        # a decode step of 24 streams, a learned scale for each channel on the branch
        {"name": "norm 24 tokens gate", "op": "norm", "M": 24, "K": 5120, "residual": True, "post": False, "gate": "channel", "normed": True},
        # a ragged prompt before the down projection of the wide layer: the norm alone
        {"name": "norm 333 tokens wide", "op": "norm", "M": 333, "K": 17408, "residual": False, "post": False, "gate": "none", "normed": False},
        # long prompts batched, everything on: gate for each token, both norms
        {"name": "norm 8192 tokens full", "op": "norm", "M": 8192, "K": 5120, "residual": True, "post": True, "gate": "token", "normed": True},
        # one request's new token with its adapter on an attention projection
        {"name": "lora 1 token", "op": "lora", "M": 1, "K": 5120, "N": 5120, "R": 16, "adapters": 8, "dtype": "float32", "order": "mixed"},
        # 24 streams, most with an adapter of their own, beside the gate projection
        {"name": "lora 24 tokens", "op": "lora", "M": 24, "K": 5120, "N": 17408, "R": 16, "adapters": 32, "dtype": "bfloat16", "order": "mixed"},
        # a prefill step of several requests, beside the down projection
        {"name": "lora 500 tokens down", "op": "lora", "M": 500, "K": 17408, "N": 5120, "R": 64, "adapters": 8, "dtype": "float32", "order": "segments"},
        # long prompts batched, beside the gate projection
        {"name": "lora 4096 tokens", "op": "lora", "M": 4096, "K": 5120, "N": 17408, "R": 64, "adapters": 16, "dtype": "bfloat16", "order": "segments"},
        # one new token through the gate and up projections
        {"name": "gated 1 token", "op": "gated", "M": 1, "K": 5120, "N": 17408, "dtype": "bfloat16"},
        # 24 streams' new tokens
        {"name": "gated 24 tokens", "op": "gated", "M": 24, "K": 5120, "N": 17408, "dtype": "bfloat16"},
        # a small layer of odd width on a ragged chunk
        {"name": "gated 77 tokens odd", "op": "gated", "M": 77, "K": 2048, "N": 4001, "dtype": "float32"},
        # a prefill step
        {"name": "gated 2048 tokens", "op": "gated", "M": 2048, "K": 5120, "N": 17408, "dtype": "bfloat16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "lora", "gated"])
    if op == "norm":
        K = BLOCK * _log(rng, 1, 17)
        M = _log(rng, 1, min(8192, 8192 * 5120 // K))
        return {"op": op, "M": M, "K": K, "residual": rng.random() < 0.7, "post": rng.random() < 0.5,
                "gate": rng.choice(["none", "channel", "token"]), "normed": rng.random() < 0.5}
    K = BLOCK * _log(rng, 1, 17)
    N = _log(rng, 64, 17408)
    if op == "lora":
        M = _log(rng, 1, min(4096, 4096 * 5120 // K))
        return {"op": op, "M": M, "K": K, "N": N, "R": rng.choice([8, 16, 24, 32, 64, 128]),
                "adapters": _log(rng, 1, 48), "dtype": rng.choice(["float32", "bfloat16"]),
                "order": "mixed" if M <= 64 or rng.random() < 0.2 else "segments"}
    M = _log(rng, 1, min(2048, 2048 * 5120 // K))
    return {"op": op, "M": M, "K": K, "N": N, "dtype": rng.choice(["float32", "bfloat16"])}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    bf = torch.bfloat16
    s = {"case": case}
    if op == "norm":
        # a residual stream with a few large channels, a block's output, norm
        # weights around one
        big = 1.0 + 7.0 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        s["x"] = (_randn(g, M, K) * (0.5 if case["residual"] else 1.0) * big).to(bf)
        s["residual"] = (2.0 * _randn(g, M, K) * big).to(bf) if case["residual"] else None
        s["post_weight"] = (1.0 + 0.2 * _randn(g, K)).to(bf) if case["post"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: (0.5 + 0.2 * _randn(g, K)).to(bf),
                     "token": lambda: torch.sigmoid(_randn(g, M, K)).to(bf)}[case["gate"]]()
        s["branch_scale"] = 0.75 if case["residual"] else 1.0
        s["weight"] = (1.0 + 0.2 * _randn(g, K)).to(bf)
        s["sign"] = (2 * torch.randint(0, 2, (K,), generator=g, device="cuda") - 1).to(torch.int8)
        i = torch.arange(BLOCK, device="cuda")
        bits = i[:, None] & i[None, :]
        for h in (8, 4, 2, 1):
            bits = bits ^ (bits >> h)
        s["hadamard"] = (1 - 2 * (bits & 1)).to(torch.float32)  # the rotation as a matrix, for the plain form
        return s
    N = case["N"]
    if op == "lora":
        n, R = case["adapters"], case["R"]
        s["x"] = _randn(g, M, K).to(bf)
        s["y"] = _randn(g, M, N).to(getattr(torch, case["dtype"]))
        s["a"] = (_randn(g, n, R, K) / math.sqrt(K)).to(bf)
        s["b"] = (_randn(g, n, N, R) * (0.3 / math.sqrt(R))).to(bf)
        s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        if case["order"] == "mixed":
            ids = torch.randint(0, n, (M,), generator=g, device="cuda")
        else:  # requests one after the other, of uneven lengths, an adapter each
            parts = max(1, min(M, n + n // 2))
            cuts = torch.randint(0, M, (parts - 1,), generator=g, device="cuda").sort().values
            which = torch.randint(0, n, (parts,), generator=g, device="cuda")
            ids = which[torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)]
        if M > 1:  # one request in nine has no adapter
            ids = torch.where(ids % 9 == 8, -1, ids)
        s["ids"] = ids.to(torch.int32)
        return s
    # gated: int8 activations and their scales as the rotation leaves them, codes
    # with two fifths of zeros, fp16 group scales
    s["x_i8"] = (_randn(g, M, K) * 30.0).round().clamp(-127, 127).to(torch.int8)
    s["a_scale"] = 0.02 + 0.01 * torch.rand(M, generator=g, device="cuda")
    u = torch.rand(2, N, K, generator=g, device="cuda")
    code = (u > 0.7).to(torch.int8) - (u < 0.3).to(torch.int8)
    del u
    scale = ((0.5 + torch.rand(2, N, K // GROUP, generator=g, device="cuda")) * (2.0 / math.sqrt(K))).to(torch.float16)
    if own:
        # the load-time layout that a user's program keeps
        import ternary_weight_linear_block_amd as twl
        s["weights"] = twl.pack_ternary_gated(code[0], scale[0], code[1], scale[1])
    else:
        # the same weights as int8 code * q and a scale for each row
        smax = scale.float().abs().amax(-1)
        q = torch.round(127.0 * scale.float() / smax[..., None])
        s["w"] = (code.view(2, N, K // GROUP, GROUP) * q[..., None]).to(torch.int8).view(2, N, K)
        s["smax"] = smax
    return s


def _own_norm(s):
    import ternary_weight_linear_block_amd as twl
    x_i8, a_scale, h, normed = twl.norm_rotate_quant_act(
        s["x"], s["weight"], s["sign"], eps=EPS, residual=s["residual"], post_weight=s["post_weight"], gate=s["gate"],
        branch_scale=s["branch_scale"], return_normed=s["case"]["normed"])
    # the int8 activations as the values they stand for
    values = torch.empty(x_i8.shape, dtype=torch.bfloat16, device=x_i8.device)
    torch.mul(x_i8, a_scale[:, None], out=values)
    return {"values": values, "a_scale": a_scale, "h": h, "normed": normed}


def _plain_norm(s):
    # in 64 bits up to the two bf16 roundings: a value next to a border of the
    # rounding would fall on either side of it otherwise
    bf = torch.bfloat16
    t = s["x"].double()
    h = None
    if s["post_weight"] is not None:
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * s["post_weight"].double()
    if s["gate"] is not None:
        t = t * s["gate"].double()
    if s["branch_scale"] != 1.0:
        t = t * s["branch_scale"]
    if s["residual"] is not None:
        t = t + s["residual"].double()
    if s["residual"] is not None or s["post_weight"] is not None or s["gate"] is not None:
        h = t.to(bf)
        t = h.double()
    normed = (t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()).to(bf)
    M, K = normed.shape
    r = (normed.float() * s["sign"].float()).view(M * (K // BLOCK), BLOCK) @ s["hadamard"]
    r = r.view(M, K) / 32.0
    a_scale = r.abs().amax(-1) / 127.0
    step = torch.where(a_scale > 0, a_scale, 1.0)[:, None]
    values = (torch.round(r / step).clamp(-127, 127) * a_scale[:, None]).to(bf)
    return {"values": values, "a_scale": a_scale, "h": h, "normed": normed if s["case"]["normed"] else None}


def _own_lora(s):
    import ternary_weight_linear_block_amd as twl
    return twl.lora_add(s["y"], s["x"], s["ids"], s["a"], s["b"], s["scale"])


def _plain_lora(s):
    # every adapter on every token, then the token's own kept
    n, R, K = s["a"].shape
    M = s["x"].shape[0]
    v = s["x"].float() @ s["a"].float().view(n * R, K).t()
    keep = s["ids"][:, None] == torch.arange(n, device="cuda")[None, :]
    v = torch.where(keep[:, :, None], v.view(M, n, R) * s["scale"][None, :, None], 0.0)
    b = s["b"].float().permute(0, 2, 1).reshape(n * R, -1)
    return (s["y"].float() + v.view(M, n * R) @ b).to(s["y"].dtype)


def _own_gated(s):
    import ternary_weight_linear_block_amd as twl
    packed, q, smax = s["weights"]
    return twl.ternary_gated_linear(s["x_i8"], s["a_scale"], packed, q, smax, out_dtype=getattr(torch, s["case"]["dtype"]))


def _plain_gated(s):
    x = s["x_i8"].float()
    gate = (x @ s["w"][0].float().t()) * s["a_scale"][:, None] * (s["smax"][0] / 127.0)
    up = (x @ s["w"][1].float().t()) * s["a_scale"][:, None] * (s["smax"][1] / 127.0)
    return (gate / (1.0 + torch.exp(-gate)) * up).to(getattr(torch, s["case"]["dtype"]))


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "lora": _own_lora, "gated": _own_gated}[op](state)
    return {"norm": _plain_norm, "lora": _plain_lora, "gated": _plain_gated}[op](state)


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        def rms(t, w):
            return t / torch.sqrt((t * t).sum(1, keepdim=True) / K + EPS) * w.double()[None, :]

        branch = s["x"].double()
        if case["post"]:
            branch = rms(branch, s["post_weight"])
        if case["gate"] != "none":
            branch = branch * s["gate"].double()
        branch = branch * s["branch_scale"]
        h = branch + s["residual"].double() if case["residual"] else branch
        has_h = case["residual"] or case["post"] or case["gate"] != "none"
        # h and the normed activation are bf16 by definition
        h = h.to(torch.bfloat16).double()
        normed = rms(h, s["weight"]).to(torch.bfloat16).double()
        r = (normed * s["sign"].double()).view(M, K // BLOCK, BLOCK)
        width = 1
        while width < BLOCK:  # the Hadamard transform by its recursion
            pairs = r.view(M, K // BLOCK, BLOCK // (2 * width), 2, width)
            r = torch.stack((pairs[..., 0, :] + pairs[..., 1, :], pairs[..., 0, :] - pairs[..., 1, :]), -2)
            width *= 2
        r = r.reshape(M, K) / 32.0
        a_scale = r.abs().max(1).values / 127.0
        values = torch.round(r / torch.clamp(a_scale, min=1e-300)[:, None]) * a_scale[:, None]
        return {"values": values, "a_scale": a_scale, "h": h if has_h else None, "normed": normed if case["normed"] else None}
    if case["op"] == "lora":
        out = s["y"].double()
        for i in range(case["adapters"]):
            rows = (s["ids"] == i).nonzero()[:, 0]
            v = s["x"][rows].double() @ s["a"][i].double().t()
            out[rows] += s["scale"][i].double() * (v @ s["b"][i].double().t())
        return out
    if own:
        return None
    x = s["x_i8"].double() * s["a_scale"].double()[:, None]
    gate, up = (x @ s["w"][i].double().t() * (s["smax"][i].double() / 127.0) for i in (0, 1))
    return gate * torch.sigmoid(gate) * up


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "norm":
        has_h = case["residual"] or case["post"] or case["gate"] != "none"
        wide = 1 + case["residual"] + (case["gate"] == "token") + has_h + case["normed"]
        table = 1 + case["post"] + (case["gate"] == "channel")
        return {"bytes": M * K * (2 * wide + 1) + 4 * M + K * (2 * table + 1), "flops": M * K * 24}
    N = case["N"]
    if op == "lora":
        R, used = case["R"], min(M, case["adapters"])
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": 2 * M * K + 2 * size * M * N + 2 * used * R * (K + N) + 4 * M, "flops": 2 * M * R * (K + N)}
    size = 4 if case["dtype"] == "float32" else 2
    return {"bytes": 2 * N * (K // 4 + K // GROUP + 4) + M * (K + 4) + size * M * N, "flops": 4 * M * N * K}
