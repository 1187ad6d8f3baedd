"""Measured cases of the layer's 8-bit and per-head-decay operators.

Four operators around and beside the KDA core (head size 128, hidden size 7168,
2, 12 or 96 heads, as in the package's workloads):

* quant_rows   -- h = x + residual, RMSNorm(h) * w, rows quantised to int8 with
                  one fp32 scale a row (or plain rows quantised, without norm);
* linear_i8    -- y = (x_i8 . w_i8^T) * x_scale[row] * w_scale[column], bf16;
* la_step      -- linear attention with a decay a head, one token a sequence,
                  states in a slot pool updated in place;
* la_prefill   -- the same attention over prompts packed one after the other,
                  the last state of each stored in its slot.

`run` computes them in elementary torch operations, or, where `own` is true,
through the package's entry points.
"""
import math

import torch

own = False

HEAD = 128
HIDDEN = 7168
EPS = 1e-6
DEV = "cuda"


def listed():
    return [
        # the norm in front of in_proj for one token of one request: latency
        {"name": "quant_norm_1x7168", "op": "quant_rows", "rows": 1, "cols": 7168, "norm": True, "residual": True},
        # the same norm over a long prompt's rows (an odd count): bandwidth
        {"name": "quant_norm_8191x7168", "op": "quant_rows", "rows": 8191, "cols": 7168, "norm": True,
         "residual": True},
        # the 96-head core's output rows, quantised for o_proj: no norm, no residual
        {"name": "quant_core_1024x12288", "op": "quant_rows", "rows": 1024, "cols": 12288, "norm": False,
         "residual": False},
        # in_proj of a 12-head slice for one token: the weight's bytes
        {"name": "i8_in_proj_1", "op": "linear_i8", "rows": 1, "K": 7168, "N": 6284},
        # o_proj of a 12-head slice for a decode batch
        {"name": "i8_o_proj_64", "op": "linear_i8", "rows": 64, "K": 1536, "N": 7168},
        # in_proj for a large decode batch
        {"name": "i8_in_proj_512", "op": "linear_i8", "rows": 512, "K": 7168, "N": 6284},
        # in_proj over a long prompt's rows (an odd count): tensor rate
        {"name": "i8_in_proj_4111", "op": "linear_i8", "rows": 4111, "K": 7168, "N": 6284},
        # one token of one request on two heads: latency
        {"name": "la_step_1x2", "op": "la_step", "rows": 1, "heads": 2, "qk_heads": 2, "pool": 4, "bf16_state": False,
         "token_decay": False},
        # a large decode batch: the states' bytes
        {"name": "la_step_512x12", "op": "la_step", "rows": 512, "heads": 12, "qk_heads": 12, "pool": 1024,
         "bf16_state": False, "token_decay": False},
        # a short prompt on two heads: latency
        {"name": "la_prefill_37x2", "op": "la_prefill", "rows": 37, "seqs": 1, "heads": 2, "qk_heads": 2, "pool": 4,
         "bf16_state": False, "token_decay": False, "resume": False},
        # one long prompt on a 12-head slice
        {"name": "la_prefill_8192x12", "op": "la_prefill", "rows": 8192, "seqs": 1, "heads": 12, "qk_heads": 12,
         "pool": 8, "bf16_state": False, "token_decay": False, "resume": False},
        # ragged prompts, some continuing from stored states, decays from the tokens, heads sharing q and k
        {"name": "la_prefill_ragged_5000x12", "op": "la_prefill", "rows": 5000, "seqs": 16, "heads": 12,
         "qk_heads": 4, "pool": 64, "bf16_state": True, "token_decay": True, "resume": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    heads = rng.choice([1, 2, 3, 5, 8, 12, 16, 24, 40, 96])
    shared = rng.choice([d for d in range(1, heads + 1) if heads % d == 0]) if rng.random() < 0.3 else heads
    return heads, shared


def draw(rng):
    op = rng.choice(["quant_rows", "linear_i8", "la_step", "la_prefill"])
    if op == "quant_rows":
        cols = 16 * _log(rng, 8, 768)
        rows = min(_log(rng, 1, 8192), 8191 * 7168 // cols)
        return {"op": op, "rows": rows, "cols": cols, "norm": rng.random() < 0.7, "residual": rng.random() < 0.6}
    if op == "linear_i8":
        K, N = 16 * _log(rng, 16, 768), _log(rng, 64, 16384)
        rows = max(1, min(_log(rng, 1, 4111), 4111 * 7168 * 6284 // (K * N)))
        return {"op": op, "rows": rows, "K": K, "N": N}
    heads, shared = _heads(rng)
    if op == "la_step":
        rows = min(_log(rng, 1, 512), 6144 // heads)
        return {"op": op, "rows": rows, "heads": heads, "qk_heads": shared, "pool": rows + rng.randrange(1, 9),
                "bf16_state": rng.random() < 0.4, "token_decay": rng.random() < 0.5}
    rows = min(_log(rng, 1, 16384), 8192 * 12 // heads)
    seqs = min(_log(rng, 1, 32), rows)
    return {"op": op, "rows": rows, "seqs": seqs, "heads": heads, "qk_heads": shared,
            "pool": seqs + rng.randrange(1, 9), "bf16_state": rng.random() < 0.4, "token_decay": rng.random() < 0.5,
            "resume": rng.random() < 0.5}


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _int8_rows(x):
    """Rows of x in int8 with one scale a row."""
    top = x.abs().amax(dim=1, keepdim=True)
    return (x * (127.0 / top)).round().to(torch.int8), (top[:, 0] / 127.0).contiguous()


def _lengths(rows, seqs, gen):
    """`seqs` ragged lengths of at least one token that add up to `rows`."""
    share = torch.rand(seqs, generator=gen, device=DEV).add_(0.05).double().cpu()
    cuts = (share.cumsum(0) / share.sum() * (rows - seqs)).round().long()
    ends = [int(c) + i + 1 for i, c in enumerate(cuts)]
    ends[-1] = rows
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "quant_rows":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _normal(gen, rows, cols).bfloat16()
        s["residual"] = (4.0 * _normal(gen, rows, cols)).bfloat16() if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * _normal(gen, cols)).bfloat16() if case["norm"] else None
        s["out"] = torch.empty(rows, cols, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(rows, dtype=torch.float32, device=DEV)
        return s
    if case["op"] == "linear_i8":
        rows, K, N = case["rows"], case["K"], case["N"]
        s["x"], s["x_scales"] = _int8_rows(_normal(gen, rows, K))
        s["w"], s["w_scales"] = _int8_rows(0.02 * _normal(gen, N, K))
        s["out"] = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
        return s
    rows, H, Hk = case["rows"], case["heads"], case["qk_heads"]
    # q | k | v as columns of one projected row, as in_proj writes them
    packed = _normal(gen, rows, (2 * Hk + H) * HEAD).bfloat16()
    s["q"] = packed[:, : Hk * HEAD].view(rows, Hk, HEAD)
    s["k"] = packed[:, Hk * HEAD: 2 * Hk * HEAD].view(rows, Hk, HEAD)
    s["v"] = packed[:, 2 * Hk * HEAD:].view(rows, H, HEAD)
    if case["token_decay"]:
        s["g"] = -torch.nn.functional.softplus(_normal(gen, rows, H) - 2.0)
    else:
        s["g"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)
    state = 0.5 * _normal(gen, case["pool"], H, HEAD, HEAD)
    s["state"] = state.bfloat16() if case["bf16_state"] else state
    s["out"] = torch.empty(rows, H, HEAD, dtype=torch.bfloat16, device=DEV)
    order = torch.randperm(case["pool"], generator=gen, device=DEV)
    if case["op"] == "la_step":
        s["slots"] = order[:rows].to(torch.int32).contiguous()
        return s
    seqs = case["seqs"]
    lens = _lengths(rows, seqs, gen)
    ends = torch.tensor([0] + lens, device=DEV).cumsum(0)
    s["cu_seqlens"] = ends.to(torch.int32)
    s["max_len"] = max(lens)
    s["slots"] = order[:seqs].to(torch.int32).contiguous()
    s["has_state"] = (torch.arange(seqs, device=DEV) % 3 != 1).to(torch.int32) if case["resume"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms


def _plain_quant_rows(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).bfloat16()
        s["residual"].copy_(h)
        h = h.float()
    if s["weight"] is not None:
        p = h * s["weight"].float()
        inv = torch.rsqrt(h.double().square().mean(dim=1) + EPS)
    else:
        p, inv = h, torch.ones(h.shape[0], dtype=torch.float64, device=h.device)
    # 127 p / max |p| may lie next to a half: in 64 bits
    top = p.abs().amax(dim=1).double()
    q = torch.where(top[:, None] > 0, 127.0 * p.double() / top[:, None], 0.0).round().to(torch.int8)
    return q, (inv * top / 127.0).float(), s["residual"]


def _plain_linear_i8(s):
    y = s["x"].float() @ s["w"].float().t()
    return (y * s["x_scales"][:, None] * s["w_scales"][None, :]).bfloat16()


def _plain_la_step(s):
    H = s["v"].shape[1]
    share = H // s["q"].shape[1]
    q = s["q"].float().repeat_interleave(share, dim=1)
    k = s["k"].float().repeat_interleave(share, dim=1)
    at = s["slots"].long()
    S = s["state"][at].float() * torch.exp(s["g"].expand(at.shape[0], H))[:, :, None, None]
    S = S + s["v"].float()[:, :, :, None] * k[:, :, None, :]
    s["state"][at] = S.to(s["state"].dtype)
    out = (S * q[:, :, None, :]).sum(-1) * HEAD ** -0.5
    return out.bfloat16(), s["state"]


CHUNK = 64


def _plain_la_prefill(s):
    rows, H, _ = s["v"].shape
    share = H // s["q"].shape[1]
    cu = s["cu_seqlens"].long()
    seqs, chunks = cu.shape[0] - 1, -(-s["max_len"] // CHUNK)
    # [seqs, heads, chunks, 64, 128], rows behind a sequence's end as zeros
    pos = torch.arange(chunks * CHUNK, device=DEV)
    at = (cu[:-1, None] + pos).clamp(max=rows - 1)
    live = pos < (cu[1:] - cu[:-1])[:, None]

    def split(x):
        x = x.float()[at] * live[:, :, None, None]
        return x.repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2).reshape(seqs, H, chunks, CHUNK, -1)

    q, k, v = split(s["q"]), split(s["k"]), split(s["v"])
    G = split(s["g"].expand(rows, H)[:, :, None])[..., 0].cumsum(-1)  # log decay from the chunk's start
    total = G[..., -1]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    inner = torch.where(low, torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, 0.0)), 0.0)
    inner = (q @ k.transpose(-1, -2)) * inner @ v
    local = v.transpose(-1, -2) @ (k * torch.exp(total[..., None] - G)[..., None])  # [.., chunks, v, k]
    # the state before each chunk, and behind the last: the chunks' own, decayed, and the first
    P = torch.nn.functional.pad(total.double().cumsum(-1), (1, 0))
    before = torch.ones(chunks + 1, chunks, dtype=torch.bool, device=DEV).tril(-1)
    D = torch.where(before, torch.exp((P[..., :, None] - P[..., None, 1:]).masked_fill(~before, 0.0)), 0.0).float()
    slots = s["slots"].long()
    first = s["state"][slots].float()
    first = first * s["has_state"][:, None, None, None] if s["has_state"] is not None else torch.zeros_like(first)
    states = (D @ local.reshape(seqs, H, chunks, -1)).reshape(seqs, H, chunks + 1, HEAD, HEAD)
    states = states + torch.exp(P).float()[..., None, None] * first[:, :, None]
    out = inner + torch.exp(G)[..., None] * (q @ states[:, :, :-1].transpose(-1, -2))
    out = out.reshape(seqs, H, chunks * CHUNK, HEAD).transpose(1, 2)[live] * HEAD ** -0.5
    s["state"][slots] = states[:, :, -1].to(s["state"].dtype)
    return out.bfloat16(), s["state"]


# ---------------------------------------------------------------------------
# the package's entry points


def _own_quant_rows(s):
    import linear_attention_decode_03_gb300 as kda

    q, scales = kda.quant_rows(s["x"], residual=s["residual"], norm_weight=s["weight"], eps=EPS, out=s["out"],
                               scales=s["scales"])
    return q, scales, s["residual"]


def _own_linear_i8(s):
    import linear_attention_decode_03_gb300 as kda

    return kda.linear_i8(s["x"], s["x_scales"], s["w"], s["w_scales"], out=s["out"])


def _own_la_step(s):
    import linear_attention_decode_03_gb300 as kda

    out = kda.la_step(s["q"], s["k"], s["v"], s["g"], state=s["state"], slots=s["slots"], out=s["out"])
    return out, s["state"]


def _own_la_prefill(s):
    import linear_attention_decode_03_gb300 as kda

    out = kda.la_prefill(s["q"], s["k"], s["v"], s["g"], state=s["state"], slots=s["slots"],
                         cu_seqlens=s["cu_seqlens"], max_len=s["max_len"], has_state=s["has_state"], out=s["out"])
    return out, s["state"]


_PLAIN = {"quant_rows": _plain_quant_rows, "linear_i8": _plain_linear_i8, "la_step": _plain_la_step,
          "la_prefill": _plain_la_prefill}
_OWN = {"quant_rows": _own_quant_rows, "linear_i8": _own_linear_i8, "la_step": _own_la_step,
        "la_prefill": _own_la_prefill}


def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def work(case):
    if case["op"] == "quant_rows":
        rows, cols = case["rows"], case["cols"]
        b = rows * cols * (2 + 1 + (4 if case["residual"] else 0)) + 4 * rows + (2 * cols if case["norm"] else 0)
        return {"bytes": b, "flops": 6 * rows * cols}
    if case["op"] == "linear_i8":
        rows, K, N = case["rows"], case["K"], case["N"]
        return {"bytes": rows * K + N * K + 2 * rows * N + 4 * (rows + N), "flops": 2 * rows * K * N}
    rows, H, Hk = case["rows"], case["heads"], case["qk_heads"]
    block = HEAD * HEAD * (2 if case["bf16_state"] else 4)
    b = rows * 2 * HEAD * (2 * Hk + 2 * H) + 4 * (rows * H if case["token_decay"] else H)
    if case["op"] == "la_step":
        return {"bytes": b + 2 * rows * H * block, "flops": 5 * HEAD * HEAD * rows * H}
    seqs = case["seqs"]
    read = sum(i % 3 != 1 for i in range(seqs)) if case["resume"] else 0
    return {"bytes": b + (seqs + read) * H * block, "flops": 4 * HEAD * HEAD * rows * H}


def exact(case, seed):
    """The definitions, token by token and in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "quant_rows":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).bfloat16().double()
        w = s["weight"].double() if s["weight"] is not None else torch.ones((), dtype=torch.float64, device=DEV)
        y = h * w
        if s["weight"] is not None:
            y = y / ((h * h).sum(1, keepdim=True) / case["cols"] + EPS).sqrt()
        # whole numbers are compared with the plain form's alone
        return None, y.abs().amax(1) / 127.0, h if s["residual"] is not None else None
    if case["op"] == "linear_i8":
        return torch.einsum("mk,nk->mn", s["x"].double() * s["x_scales"].double()[:, None],
                            s["w"].double() * s["w_scales"].double()[:, None])
    H, Hk = case["heads"], case["qk_heads"]
    of = torch.arange(H, device=DEV) // (H // Hk)  # the q / k head that serves each head
    d = s["g"].double().exp().expand(case["rows"], H)
    q, k, v = s["q"].double() * HEAD ** -0.5, s["k"].double(), s["v"].double()
    pool = s["state"].double()
    if case["op"] == "la_step":
        lens = [1] * case["rows"]
        starts = torch.arange(case["rows"], device=DEV)
        S = pool[s["slots"].long()]
    else:
        cu = s["cu_seqlens"].tolist()
        lens = [b - a for a, b in zip(cu, cu[1:])]
        starts = s["cu_seqlens"][:-1].long()
        S = pool[s["slots"].long()]
        if s["has_state"] is None:
            S = S * 0.0
        else:
            S = S * s["has_state"].double()[:, None, None, None]
    out = torch.zeros(case["rows"], H, HEAD, dtype=torch.float64, device=DEV)
    # longest sequences first, so that those with a token t are a prefix
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    index = torch.tensor(order, device=DEV)
    starts, S = starts[index], S[index].contiguous()
    longest, alive = lens[order[0]], len(lens)
    for t in range(longest):
        while lens[order[alive - 1]] <= t:
            alive -= 1
        r = starts[:alive] + t
        A = S[:alive]
        A *= d[r][:, :, None, None]
        A += v[r][:, :, :, None] * k[r][:, of][:, :, None, :]
        out[r] = torch.matmul(A, q[r][:, of][:, :, :, None])[..., 0]
    pool[s["slots"].long()[index]] = S
    return out, pool
