"""Plain 64-bit forms of the operators of include/kda_ops.h, on the CPU, and
the error bounds that go with them.  Nothing here uses the library."""
from __future__ import annotations

import torch

HEAD = 128
# the largest relative error of one rounding
U32, UBF16 = 2.0 ** -24, 2.0 ** -8
CHUNK = 128  # tokens la_prefill works on at a time


def bf16(x):
    return x.to(torch.bfloat16)


def quant_rows(x, residual, weight, eps):
    """(q int64, scales, h bf16): exact whole numbers (ties to even).

    h, w are bf16, so 254 |p| and (2 m + 1) top are exact in 64 bits."""
    h = x.double()
    if residual is not None:
        h = bf16(h + residual.double()).double()  # bf16 + bf16 is exact in 64 bits but for far exponents, where
        # the smaller cannot move the rounding
    p = h * weight.double() if weight is not None else h
    top = p.abs().amax(dim=1)
    n = 1.0 / torch.sqrt((h * h).mean(dim=1) + eps) if weight is not None else torch.ones_like(top)
    bad = ~torch.isfinite(top)
    safe = torch.where((top > 0) & ~bad, top, 1.0)[:, None]
    a = torch.where(bad[:, None], 0.0, p.abs())
    m = torch.floor(127.0 * a / safe)
    # floor(127 a / top) may be one off where the quotient lies next to a whole number
    m = m - (m * safe > 127.0 * a).double() + ((m + 1) * safe <= 127.0 * a).double()
    lhs, rhs = 254.0 * a, (2.0 * m + 1.0) * safe
    up = (lhs > rhs) | ((lhs == rhs) & (m % 2 == 1))
    q = torch.where(p < 0, -(m + up.double()), m + up.double()).to(torch.int64)
    q[bad] = 0
    scales = torch.where(bad, float("nan"), torch.where(top > 0, n * top / 127.0, 0.0))  # a row of zeros: 0
    return q, scales, h.to(torch.bfloat16)


def scale_bound(cols):
    """Relative error of a row's scale: the sum of squares adds each thread's
    values in a chain (at most 64 of them) and then over 32 lanes and 32
    warps (10 levels), each square fused; the root halves it; the mean, eps, root,
    quotient and two products add 8."""
    return (0.5 * (64 + 10) + 8) * U32


def linear_i8(x, sx, w, sw):
    return (x.double() @ w.double().t()) * sx.double()[:, None] * sw.double()[None, :]


def linear_i8_bound(x, sx, w, sw, ref):
    """One rounding to bf16 and three in 32 bits (the sum's own to fp32, two scales); the partial
    sums are whole numbers, exact up to 2^24, beyond that each of at most K / 8 additions
    of the tensor pipe and 16 of the split may be off by a step."""
    total = x.double().abs() @ w.double().abs().t()
    steps = torch.where(total < 2.0 ** 24, 0.0, (x.shape[1] / 8 + 16) * 2.0 * U32)
    return ref.abs() * (UBF16 + 4 * U32) + total * steps * (sx.double().abs()[:, None] * sw.double().abs()[None, :])


def attention(q, k, v, g, scale, starts):
    """Token by token.  q, k [T, Hk, 128], v [T, H, 128], g [T, H], starts [H, 128, 128];
    returns out [T, H, 128], the last state, and for both a magnitude: the sums with every
    product's absolute value (out: of the state's magnitude with |q|)."""
    T, H, _ = v.shape
    share = H // q.shape[1]
    q = q.double().repeat_interleave(share, 1)
    k = k.double().repeat_interleave(share, 1)
    v, d = v.double(), g.double().exp()
    S, M = starts.double().clone(), starts.double().abs()
    out, mag, states = torch.zeros(T, H, HEAD, dtype=torch.float64), torch.zeros(T, H, HEAD, dtype=torch.float64), []
    for t in range(T):
        S = S * d[t][:, None, None] + v[t][:, :, None] * k[t][:, None, :]
        M = M * d[t][:, None, None] + (v[t][:, :, None] * k[t][:, None, :]).abs()
        out[t] = scale * (S * q[t][:, None, :]).sum(-1)
        mag[t] = abs(scale) * (M * q[t].abs()[:, None, :]).sum(-1)
        states.append(S)
    return out, S, mag, M, states


def step_bounds(out, S, mag, M, bf16_state):
    """la_step: the decay (expf within 2 steps, so 4 U32), its product, the fused sum: 6 U32 of
    the magnitudes; the output adds at most 8 terms in a chain and 5 levels, the scale, and
    one rounding to bf16.  A bf16 pool rounds the stored state once."""
    return (out.abs() * UBF16 * (1 + 2.0 ** -8) + 24 * U32 * mag,
            M * 8 * U32 + (S.abs() * UBF16 if bf16_state else 0.0))


def prefill_bounds(q, k, v, g, scale, out, S, mag, M, states, starts, bf16_state):
    """la_prefill works on chunks of CHUNK tokens (from the sequence's start): inside one the
    scores (q . k_j) e^{..}, and towards one the state before it, are rounded to bf16 once
    each, so an output is off by at most UBF16 times sum_j |score_j| |v_j| and sum_k |q_k| |S_k| of the state
    before its chunk; its own rounding is one more.  Keys times their decay enter
    the state as two bf16 parts (what the two leave out is at most UBF16^2 of each
    product), and sums and decays in 32 bits: at most 300 roundings of the magnitudes
    over a chunk, and 4 for each chunk after it."""
    T, H, _ = v.shape
    share = H // q.shape[1]
    qd, kd = q.double().repeat_interleave(share, 1), k.double().repeat_interleave(share, 1)
    extra = torch.zeros_like(out)
    G = g.double().cumsum(0)
    for c in range(0, T, CHUNK):
        e = min(T, c + CHUNK)
        before = states[c - 1] if c else starts.double()
        base = G[c - 1] if c else torch.zeros(H, dtype=torch.float64)
        part = torch.einsum("thk,hvk->thv", qd[c:e].abs(), before.abs()) * (G[c:e] - base).exp()[:, :, None]
        P = torch.einsum("ihk,jhk->hij", qd[c:e], kd[c:e])
        diff = (G[c:e, None] - G[None, c:e]).permute(2, 0, 1)
        P = torch.where(torch.ones(e - c, e - c, dtype=torch.bool).tril(), P.abs() * diff.clamp(max=0).exp(), 0.0)
        extra[c:e] = (part + torch.einsum("hij,jhv->ihv", P, v[c:e].double().abs())) * abs(scale)
    fine = (300 + 4 * (T / CHUNK + 1)) * U32
    return (UBF16 * (out.abs() + extra) * (1 + 2.0 ** -6) + (UBF16 ** 2 + fine) * mag,
            (UBF16 ** 2 + fine) * M + (S.abs() * UBF16 if bf16_state else 0.0))
