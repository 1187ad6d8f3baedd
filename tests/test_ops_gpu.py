"""quant_rows, linear_i8, la_step and la_prefill against their plain 64-bit
forms (tests/ops_reference.py), with the bounds derived there."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_attention_decode_03_gb300 as kda
from tests import ops_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _close(got, want, bound, what):
    diff = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all(), what
    over = diff - bound
    assert (over <= 0).all(), f"{what}: off by {diff.flatten()[over.argmax()]:.3g}, allowed {bound.flatten()[over.argmax()]:.3g}"


# ---------------------------------------------------------------------------
# quant_rows


def _quant(x, residual, weight, eps=1e-6, **kw):
    xd = x.to(DEV)
    rd = residual.to(DEV) if residual is not None else None
    q, s = kda.quant_rows(xd, residual=rd, norm_weight=weight.to(DEV) if weight is not None else None, eps=eps, **kw)
    assert torch.equal(xd.cpu().view(torch.int16), x.view(torch.int16))
    wq, ws, wh = R.quant_rows(x, residual, weight, eps)
    assert torch.equal(q.cpu().long(), wq)
    bad = torch.isnan(ws)
    assert torch.equal(torch.isnan(s.cpu()), bad)
    assert ((s.cpu().double() - ws).abs()[~bad] <= (R.scale_bound(x.shape[1]) * ws)[~bad] + 2.0 ** -149).all()
    if residual is not None:
        assert torch.equal(rd.cpu().view(torch.int16)[~bad], wh.view(torch.int16)[~bad])
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (5, 1536), (2, 4096), (3, 4112), (7, 7168), (2, 12288),
                                       (1, 16400), (2, 32768)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("res", [True, False])
def test_quant_rows(rows, cols, norm, res):
    r = _gen(rows * cols + 2 * norm + res)
    x = torch.randn(rows, cols, generator=r).bfloat16()
    residual = (3 * torch.randn(rows, cols, generator=r)).bfloat16() if res else None
    weight = (1 + 0.2 * torch.randn(cols, generator=r)).bfloat16() if norm else None
    _quant(x, residual, weight)


def test_quant_rows_many_rows_on_and_next_to_halves():
    # few distinct magnitudes: ties and quotients one bit off a half are common
    r = _gen(5)
    x = (torch.randint(-254, 255, (700, 512), generator=r).float() / 2).bfloat16()
    x[:, 0] = torch.tensor([127.0, 254.0, 63.5, 253.0])[torch.randint(0, 4, (700,), generator=r)].bfloat16()
    _quant(x, None, None)
    w = (torch.randint(1, 255, (512,), generator=r).float() / 128).bfloat16()
    _quant(x, None, w)
    _quant(x, x.flip(0), w)


def test_quant_rows_strides():
    r = _gen(6)
    wide = torch.randn(9, 400, generator=r).bfloat16().to(DEV)
    res = torch.randn(9, 320, generator=r).bfloat16().to(DEV)
    keep = res.clone()
    out = torch.full((9, 288), 77, dtype=torch.int8, device=DEV)
    x, rv = wide[:, 16:272], res[:, 8:264]
    q, s = kda.quant_rows(x, residual=rv, out=out[:, 8:264])
    wq, ws, wh = R.quant_rows(x.cpu(), keep[:, 8:264].cpu(), None, 0.0)
    assert torch.equal(q.cpu().long(), wq) and torch.equal(rv.cpu(), wh)
    assert (out[:, :8] == 77).all() and (out[:, 264:] == 77).all()
    assert torch.equal(res[:, :8], keep[:, :8]) and torch.equal(res[:, 264:], keep[:, 264:])
    # the residual may be x itself
    y = torch.randn(3, 64, generator=r).bfloat16()
    yd = y.to(DEV)
    q, s = kda.quant_rows(yd, residual=yd)
    assert torch.equal(yd.cpu(), (2 * y.float()).bfloat16())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_quant_rows_not_finite(value):
    r = _gen(7)
    x = torch.randn(4, 256, generator=r).bfloat16()
    x[1, 200] = value
    for w in (None, torch.zeros(256).bfloat16(), torch.ones(256).bfloat16()):
        _quant(x, None, w)
    big = torch.full((2, 256), 3.3e38).bfloat16()  # the sum with the residual overflows in row 0
    res = torch.zeros(2, 256).bfloat16()
    res[0] = 3.3e38
    _quant(big, res, None)


@pytest.mark.parametrize("size", [1e-40, 1e-38, 1e-30, 1e-20, 1e18, 1e25, 3e37])
def test_quant_rows_far_magnitudes(size):
    r = _gen(8)
    x = (torch.rand(3, 512, generator=r) * size).bfloat16()
    x[2, :] = 0
    w = (0.5 + torch.rand(512, generator=r)).bfloat16()
    _quant(x, None, w)
    _quant(x, None, w, eps=0.0 if size > 1e-15 else 1e-6)
    q, s = kda.quant_rows(x.to(DEV))
    wq, ws, _ = R.quant_rows(x, None, None, 0.0)
    assert torch.equal(q.cpu().long(), wq)
    # a scale below fp32's normal range is rounded to its steps
    assert ((s.cpu().double() - ws).abs() <= R.scale_bound(512) * ws + 2 * 2.0 ** -149).all()


@pytest.mark.parametrize("h,w,eps", [
    (1e-25, 1.0, 0.0), (1e-38, 1.0, 0.0), (1e-25, 1e10, 0.0), (1e-25, 1e10, 1e-30), (1e-12, 1.0, 1e-25),  # squares too small
    (1e-38, 1e-37, 0.0), (1e-30, 1e-20, 1e-6), (1e-38, 1e-38, 1e-4),  # products too small
    (1e30, 1e30, 1e-6), (1e37, 1e5, 1e-6), (1e2, 1e37, 1e-6), (2e38, 1.0, 1e-6)])  # products or squares too large
def test_quant_rows_products_out_of_range(h, w, eps):
    r = _gen(10)
    x = (torch.randint(-254, 255, (20, 512), generator=r) / 254 * h).bfloat16()
    x[:, 0] = torch.tensor(h).bfloat16()
    weight = (torch.ones(512) * w).bfloat16()
    cases = [weight, (weight * (0.5 + 0.5 * torch.rand(512, generator=r))).bfloat16()]
    cases.append(cases[1].clone())
    cases[2][1::2] = 0  # zeros next to a large or a scaled factor
    for c in cases:
        wq, ws, _ = R.quant_rows(x, None, c, eps)
        q, s = kda.quant_rows(x.to(DEV), norm_weight=c.to(DEV), eps=eps)
        assert torch.equal(q.cpu().long(), wq)
        # a scale below fp32's normal range is rounded to its steps, at most twice
        assert ((s.cpu().double() - ws).abs() <= R.scale_bound(512) * ws + 2 * 2.0 ** -149).all()


def test_quant_rows_zeros_next_to_the_largest():
    big = torch.tensor(3.3e38).bfloat16()
    x, w = torch.zeros(3, 64).bfloat16(), torch.zeros(64).bfloat16()
    x[1, 3], x[2] = big, 1e-35
    w[5], w[8] = big, 1e-20
    q, s = kda.quant_rows(x.to(DEV), norm_weight=w.to(DEV))
    wq, ws, _ = R.quant_rows(x, None, w, 1e-6)
    assert torch.equal(q.cpu().long(), wq) and (s[:2] == 0).all()
    assert abs(float(s[2]) - float(ws[2])) <= R.scale_bound(64) * float(ws[2])


@pytest.mark.parametrize("size", [1e36, 3e36, 1e38, 3.3e38])
def test_quant_rows_largest_on_halves(size):
    r = _gen(12)
    x = torch.randint(-254, 255, (200, 512), generator=r).float() * 2.0 ** 111
    x[:, 0] = 254 * 2.0 ** 111
    k = 2.0 ** int(torch.tensor(size).log2().floor() - 119)
    _quant((x * k).bfloat16(), None, None)


def test_quant_rows_more_rows_than_ctas():
    # CTAs take rows in turn: the first, ordinary ones, rows that need the careful way, rows that do not, mixed
    r = _gen(9)
    x = torch.randn(2500, 256, generator=r)
    x[::7] *= 1e-38
    x[1::11] *= 1e25
    x[5::13] = 0
    x = x.bfloat16()
    x[3::401, 17] = float("nan")
    x[4::403, 250] = float("inf")
    w = (1 + 0.2 * torch.randn(256, generator=r)).bfloat16()
    _quant(x, None, None)
    _quant(x, None, w)
    res = torch.randn(2500, 256, generator=r).bfloat16()
    _quant(x, res, w)
    w[9] = float("nan")
    _quant(x[:700], None, w)
    w[9] = float("inf")
    _quant(x[:700], res[:700], w)


def test_quant_rows_none():
    q, s = kda.quant_rows(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,)


# ---------------------------------------------------------------------------
# linear_i8


def _i8(rows, K, N, seed, lo=-127, hi=127, xpad=0, ypad=0):
    r = _gen(seed)
    x = torch.randint(lo, hi + 1, (rows, K + xpad), generator=r).to(torch.int8)[:, :K]
    w = torch.randint(lo, hi + 1, (N, K), generator=r).to(torch.int8)
    sx, sw = torch.rand(rows, generator=r) + 0.01, (torch.rand(N, generator=r) + 0.01) / 64
    whole = torch.full((rows, N + ypad), 7.0, dtype=torch.bfloat16, device=DEV)
    xd = torch.empty((rows, K + xpad), dtype=torch.int8, device=DEV)[:, :K]
    xd.copy_(x)
    y = kda.linear_i8(xd, sx.to(DEV), w.to(DEV), sw.to(DEV), out=whole[:, :N])
    assert kda.kda_linear_i8_check() == 0
    ref = R.linear_i8(x, sx, w, sw)
    _close(y, ref, R.linear_i8_bound(x, sx, w, sw, ref), (rows, K, N))
    assert (whole[:, N:] == 7.0).all()


@pytest.mark.parametrize("rows,K,N", [
    (1, 16, 1), (1, 7168, 1154), (2, 48, 77), (3, 1536, 300), (7, 208, 515), (8, 4096, 256), (9, 272, 129),
    (15, 7168, 100), (16, 1024, 640), (17, 1024, 640), (31, 272, 777), (33, 1536, 512), (64, 1536, 1154), (65, 64, 384),
    (100, 784, 203), (128, 512, 256), (129, 528, 257), (200, 2048, 999), (256, 1536, 384), (300, 272, 640),
    (513, 144, 1030),
    (18, 256, 500), (32, 512, 3000), (27, 1536, 7168), (161, 256, 40), (176, 1040, 300), (340, 400, 260),
    (1000, 272, 700)])
def test_linear_i8(rows, K, N):
    _i8(rows, K, N, seed=rows * 31 + N, xpad=16 * (rows % 3), ypad=rows % 5)


@pytest.mark.parametrize("rows", [1, 5, 16, 40, 64, 128, 160, 512])
def test_linear_i8_layer_shapes(rows):
    _i8(rows, 7168, 1154, seed=rows)      # the 2-head in_proj
    _i8(rows, 1536, 7168, seed=rows + 1)  # the 12-head o_proj


@pytest.mark.parametrize("rows", [2, 40, 200])
def test_linear_i8_largest_values(rows):
    _i8(rows, 12288, 130, seed=1, lo=127, hi=127)    # every product 127 * 127: sums beyond 2^24
    _i8(rows, 1040, 130, seed=2, lo=-128, hi=-128)   # -128 is a value as well
    _i8(rows, 528, 130, seed=3, lo=-128, hi=127)


def test_linear_i8_scales_carry_through():
    x = torch.ones(3, 64, dtype=torch.int8, device=DEV)
    w = torch.ones(20, 64, dtype=torch.int8, device=DEV)
    sx = torch.tensor([1.0, float("nan"), 0.0], device=DEV)
    sw = torch.ones(20, device=DEV)
    y = kda.linear_i8(x, sx, w, sw).float().cpu()
    assert (y[0] == 64).all() and torch.isnan(y[1]).all() and (y[2] == 0).all()


def test_linear_i8_refusals():
    x = torch.zeros(4, 40, dtype=torch.int8, device=DEV)
    w = torch.zeros(8, 40, dtype=torch.int8, device=DEV)
    s4, s8 = torch.ones(4, device=DEV), torch.ones(8, device=DEV)
    with pytest.raises(kda.KdaError):
        kda.linear_i8(x, s4, w, s8)  # K = 40
    x, w = x[:, :32].contiguous(), w[:, :32].contiguous()
    for args in ((x, s8, w, s8), (x, s4, w, s4), (x, s4, w[:, :16], s8), (x.float(), s4, w, s8),
                 (x, s4.double(), w, s8), (x, s4, w.cpu(), s8)):
        with pytest.raises((ValueError, TypeError)):
            kda.linear_i8(*args)
    with pytest.raises((ValueError, TypeError)):
        kda.linear_i8(x, s4, w, s8, out=torch.empty(4, 8, device=DEV))


# ---------------------------------------------------------------------------
# la_step, la_prefill


def _attn(rows, heads, qk_heads, seed, token_decay, pad=0, slow=False):
    """q, k, v as columns of one packed row, and g."""
    r = _gen(seed)
    wide = (2 * qk_heads + heads) * 128 + pad
    packed = torch.randn(rows, wide, generator=r).bfloat16()
    cut = [0, qk_heads * 128, 2 * qk_heads * 128, wide - pad]
    parts = [packed[:, a:b].view(rows, -1, 128) for a, b in zip(cut, cut[1:])]
    if token_decay:
        g = -torch.nn.functional.softplus(torch.randn(rows, heads, generator=r) - (6.0 if slow else 1.0))
    else:
        g = -torch.exp2(-8.0 * torch.arange(1, heads + 1) / heads)
    gpu = packed.to(DEV)
    dev = [gpu[:, a:b].view(rows, -1, 128) for a, b in zip(cut, cut[1:])]
    return parts, dev, g, r


def _pool(pool, heads, bf16_state, r):
    state = 0.5 * torch.randn(pool, heads, 128, 128, generator=r)
    return state.bfloat16() if bf16_state else state


@pytest.mark.parametrize("bf16_state", [False, True])
@pytest.mark.parametrize("rows,heads,qk_heads,token_decay", [(1, 2, 2, False), (1, 1, 1, True), (5, 3, 1, True),
                                                             (7, 12, 12, False), (3, 12, 4, True), (33, 2, 1, False)])
def test_la_step(rows, heads, qk_heads, token_decay, bf16_state):
    (q, k, v), (qd, kd, vd), g, r = _attn(rows, heads, qk_heads, rows + heads, token_decay, pad=16)
    state = _pool(rows + 3, heads, bf16_state, r)
    slots = torch.randperm(rows + 3, generator=r)[:rows].to(torch.int32)
    sd = state.to(DEV)
    out = kda.la_step(qd, kd, vd, g.to(DEV), state=sd, slots=slots.to(DEV), scale=0.3)
    assert kda.kda_la_check() == 0
    got = sd.cpu()
    gg = g.expand(rows, heads)
    for b in range(rows):
        s = int(slots[b])
        o, S, mag, M, _ = R.attention(q[b:b + 1], k[b:b + 1], v[b:b + 1], gg[b:b + 1], 0.3, state[s])
        bo, bs = R.step_bounds(o, S, mag, M, bf16_state)
        _close(out[b:b + 1], o, bo, f"row {b}")
        _close(got[s], S, bs, f"state of row {b}")
    rest = [i for i in range(rows + 3) if i not in slots.tolist()]
    assert torch.equal(got[rest], state[rest])


def test_la_step_padding_and_bad_slots():
    rows, heads = 5, 3
    _, (qd, kd, vd), g, r = _attn(rows, heads, heads, 3, False)
    state = _pool(4, heads, False, r).to(DEV)
    before = state.clone()
    slots = torch.tensor([2, -1, 4, -2, 0, 9], dtype=torch.int32, device=DEV)  # longer than the batch
    out = torch.full((rows, heads, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    kda.la_step(qd, kd, vd, g.to(DEV), state=state, slots=slots, out=out)
    assert kda.kda_la_check() == kda.KDA_ERR_SLOT
    assert kda.kda_la_check() == 0
    assert (out[1] == 0).all() and (out[2] == 5).all() and (out[3] == 5).all()
    assert torch.equal(state[[1, 3]], before[[1, 3]]) and not torch.equal(state[[0, 2]], before[[0, 2]])


def test_la_step_decay_limits():
    heads = 3
    (q, k, v), (qd, kd, vd), _, r = _attn(2, heads, heads, 4, False)
    state = _pool(2, heads, False, r)
    g = torch.tensor([-float("inf"), 0.0, -200.0])
    sd = state.to(DEV)
    kda.la_step(qd, kd, vd, g.to(DEV), state=sd, slots=torch.tensor([0, 1], dtype=torch.int32, device=DEV))
    new = (v.float()[:, :, :, None] * k.float()[:, :, None, :])
    got = sd.cpu()
    assert torch.equal(got[:, 0], new[:, 0]) and torch.equal(got[:, 2], new[:, 2])
    assert torch.allclose(got[:, 1], state[:, 1] + new[:, 1], rtol=0, atol=2.0 ** -22 * 32)


def _prefill(lens, heads, qk_heads, seed, token_decay, bf16_state, resume, tail=0, pad=8, max_len=None, slow=False,
             scale=None):
    rows = sum(lens) + tail
    (q, k, v), (qd, kd, vd), g, r = _attn(max(rows, 1), heads, qk_heads, seed, token_decay, pad=pad, slow=slow)
    if rows == 0:
        q, k, v, qd, kd, vd = (t[:0] for t in (q, k, v, qd, kd, vd))
        g = g[:0] if token_decay else g
    seqs = len(lens)
    state = _pool(seqs + 2, heads, bf16_state, r)
    slots = torch.randperm(seqs + 2, generator=r)[:seqs].to(torch.int32)
    has = torch.tensor([i % 3 != 1 for i in range(seqs)], dtype=torch.int32) if resume else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    sd = state.to(DEV)
    out = torch.full((rows, heads, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    kda.la_prefill(qd, kd, vd, g.to(DEV), state=sd, slots=slots.to(DEV), cu_seqlens=cu.to(DEV),
                   max_len=max(lens) if max_len is None else max_len, has_state=has.to(DEV) if resume else None,
                   out=out, scale=scale)
    assert kda.kda_la_check() == 0
    got = sd.cpu()
    gg = g.expand(rows, heads)
    scale = 128 ** -0.5 if scale is None else scale
    for i in range(seqs):
        a, b, s = int(cu[i]), int(cu[i + 1]), int(slots[i])
        start = state[s].float() if resume and has[i] else torch.zeros(heads, 128, 128)
        o, S, mag, M, states = R.attention(q[a:b], k[a:b], v[a:b], gg[a:b], scale, start)
        bo, bs = R.prefill_bounds(q[a:b], k[a:b], v[a:b], gg[a:b], scale, o, S, mag, M, states, start, bf16_state)
        _close(out[a:b], o, bo, f"out of sequence {i}, {b - a} tokens")
        _close(got[s], S, bs, f"state of sequence {i}, {b - a} tokens")
    assert (out[rows - tail:] == 5).all()
    rest = [i for i in range(seqs + 2) if i not in slots.tolist()]
    assert torch.equal(got[rest], state[rest])


@pytest.mark.parametrize("bf16_state", [False, True])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 256, 257, 300])
def test_la_prefill_one_sequence(length, bf16_state):
    _prefill([length], 2, 2, length, length % 2 == 0, bf16_state, resume=length % 3 == 0)


@pytest.mark.parametrize("lens", [[5, 130, 0, 1, 64, 257], [128, 128, 128], [1] * 20, [0, 0], [400, 3]])
@pytest.mark.parametrize("resume", [False, True])
def test_la_prefill_packed(lens, resume):
    _prefill(lens, 3, 1, sum(lens) + 1, True, False, resume, tail=4, max_len=max(lens) + 50)
    _prefill(lens, 2, 2, sum(lens) + 2, False, True, resume, max_len=5000)


@pytest.mark.parametrize("bf16_state", [False, True])
def test_la_prefill_long(bf16_state):
    # enough tokens for several segments of the long axis
    _prefill([2100], 1, 1, 11, True, bf16_state, resume=True, slow=True)
    _prefill([1030, 1500], 2, 1, 12, False, bf16_state, resume=True)


@pytest.mark.parametrize("bf16_state", [False, True])
@pytest.mark.parametrize("lens", [[40, 0, 1700, 128, 1, 300, 129, 900], [1400, 5], [3, 257, 1400]])
def test_la_prefill_long_among_short(lens, bf16_state):
    # some sequences are cut into segments, the others run by themselves in the same call
    assert kda.la_prefill_workspace(sum(lens) + 3, 2, len(lens), max(lens)) > 0
    _prefill(lens, 2, 1, 40 + len(lens), True, bf16_state, resume=True, tail=3)
    _prefill(lens, 2, 2, 50 + len(lens), False, bf16_state, resume=False, tail=3, max_len=4000)


@pytest.mark.parametrize("length", [0, 5, 128, 400])
def test_la_prefill_one_short_sequence_before_many_rows(length):
    assert kda.la_prefill_workspace(length + 3000, 2, 1, 3000) > 0
    for resume in (False, True):
        _prefill([length], 2, 2, 60 + length, True, False, resume, tail=3000, max_len=3000)


def test_la_prefill_long_padding_and_bad_values():
    heads, lens = 2, [1500, 40, 1300, 30, 1400, 20]
    rows = sum(lens)
    _, dev, g, r = _attn(rows, heads, heads, 24, False)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    state = _pool(4, heads, False, r).to(DEV)

    def go(cu, slots, max_len=1500):
        sd = state.clone()
        out = torch.full((rows, heads, 128), 5.0, dtype=torch.bfloat16, device=DEV)
        kda.la_prefill(*dev, g.to(DEV), state=sd, slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
                       cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_len=max_len, out=out,
                       has_state=torch.ones(6, dtype=torch.int32, device=DEV))
        return out, sd, kda.kda_la_check()

    assert kda.la_prefill_workspace(rows, heads, 6, 1500) > 0
    want, sw, flags = go(cu, [0, -1, -1, 1, -1, 2])
    assert flags == 0 and (want[1500:2840] == 0).all() and torch.equal(sw[3], state[3])
    out, sd, flags = go(cu, [0, -1, -1, 1, 9, 2])
    assert flags == kda.KDA_ERR_SLOT
    assert (out[2870:4270] == 5).all() and torch.equal(sd, sw)
    out[2870:4270] = 0
    assert torch.equal(out, want)
    # the third sequence is longer than max_len allows the first to be; an end before a beginning
    out, sd, flags = go(cu, [0, -1, -1, 1, -1, 2], 1350)
    assert flags == kda.KDA_ERR_SEQ and (out[:1500] == 5).all() and torch.equal(sd[[1, 2, 3]], sw[[1, 2, 3]])
    bad = cu.copy()
    bad[4] = 2800
    out, sd, flags = go(bad, [0, -1, -1, 1, -1, 2])
    assert flags == kda.KDA_ERR_SEQ and torch.equal(out[:1500], want[:1500])
    assert torch.equal(sd[[0, 2]], sw[[0, 2]]) and torch.equal(sd[[1, 3]], state[[1, 3]])


def test_la_prefill_decay_limits():
    # tokens that drop the state, tokens that keep all of it, decays below fp32's range
    lens, heads = [150, 40], 3
    rows = sum(lens)
    (q, k, v), (qd, kd, vd), _, r = _attn(rows, heads, heads, 21, False)
    g = torch.zeros(rows, heads)
    g[::7, 0] = -float("inf")
    g[::5, 1] = -150.0
    g[:, 2] = -1e-3
    state = _pool(2, heads, False, r)
    sd, cu = state.to(DEV), torch.tensor([0, 150, 190], dtype=torch.int32)
    out = kda.la_prefill(qd, kd, vd, g.to(DEV), state=sd, slots=torch.tensor([1, 0], dtype=torch.int32, device=DEV),
                         cu_seqlens=cu.to(DEV), max_len=150, has_state=torch.ones(2, dtype=torch.int32, device=DEV))
    for i, s in enumerate((1, 0)):
        a, b = int(cu[i]), int(cu[i + 1])
        args = (q[a:b], k[a:b], v[a:b], g[a:b].clamp(min=-150.0), 128 ** -0.5)
        o, S, mag, M, states = R.attention(*args[:3], g[a:b], args[4], state[s])
        bo, bs = R.prefill_bounds(*args, o, S, mag, M, states, state[s], False)
        # sums of logs that pass 104 * 128 keep 2^-11 of a step: a decay may be off by that much
        _close(out[a:b], o, bo + 2.0 ** -10 * mag, f"out {i}")
        _close(sd.cpu()[s], S, bs, f"state {i}")


def test_la_prefill_neighbours_stay_apart():
    """NaN in one sequence, in the rows behind the last one and in unused slots reaches nobody else."""
    lens, heads, tail = [100, 30, 140], 2, 9
    rows = sum(lens) + tail
    (q, k, v), dev, g, r = _attn(rows, heads, heads, 22, False)
    for t in dev:
        t[100:130] = float("nan")
        t[270:] = float("inf")
    state = _pool(4, heads, False, r)
    state[3] = float("nan")
    sd, cu = state.to(DEV), torch.tensor([0, 100, 130, 270], dtype=torch.int32)
    slots = torch.tensor([0, 1, 2], dtype=torch.int32)
    out = kda.la_prefill(*dev, g.to(DEV), state=sd, slots=slots.to(DEV), cu_seqlens=cu.to(DEV), max_len=140)
    assert torch.isnan(out[100:130]).all() and torch.isnan(sd[1]).all()
    gg = g.expand(rows, heads)
    for i in (0, 2):
        a, b = int(cu[i]), int(cu[i + 1])
        zero = torch.zeros(heads, 128, 128)
        o, S, mag, M, states = R.attention(q[a:b], k[a:b], v[a:b], gg[a:b], 128 ** -0.5, zero)
        bo, bs = R.prefill_bounds(q[a:b], k[a:b], v[a:b], gg[a:b], 128 ** -0.5, o, S, mag, M, states, zero, False)
        _close(out[a:b], o, bo, f"out {i}")
        _close(sd.cpu()[i], S, bs, f"state {i}")


def test_la_prefill_padding_and_bad_values():
    heads = 2
    lens = [20, 10, 30, 5, 7, 6]
    rows = sum(lens)
    _, dev, g, r = _attn(rows, heads, heads, 23, False)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    state = _pool(4, heads, False, r).to(DEV)

    def go(cu, slots, max_len):
        sd = state.clone()
        out = torch.full((rows, heads, 128), 5.0, dtype=torch.bfloat16, device=DEV)
        kda.la_prefill(*dev, g.to(DEV), state=sd, slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
                       cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), max_len=max_len, out=out)
        return out, sd, kda.kda_la_check()

    out, sd, flags = go(cu, [0, -1, 4, 1, -7, 2], 30)
    assert flags == kda.KDA_ERR_SLOT
    assert (out[20:30] == 0).all() and (out[30:60] == 5).all() and (out[65:72] == 5).all()
    assert torch.equal(sd[3], state[3])
    good = {0: (0, 20), 1: (60, 65), 2: (72, 78)}
    # the others are what they are by themselves
    alone, sa, _ = go(cu, [0, -1, -1, 1, -1, 2], 30)
    for s, (a, b) in good.items():
        assert torch.equal(out[a:b], alone[a:b]) and torch.equal(sd[s], sa[s])
    # a sequence longer than max_len, one that ends before it begins, one that ends behind the rows
    out, sd, flags = go(cu, [0, -1, -1, 1, -1, 2], 25)
    assert flags == 0 or flags == kda.KDA_ERR_SEQ
    bad = cu.copy()
    bad[2] = 15
    bad[6] = rows + 1
    out, sd, flags = go(bad, [0, 1, -1, -1, -1, 2], 50)
    assert flags == kda.KDA_ERR_SEQ
    assert torch.equal(sd[[1, 2, 3]], state[[1, 2, 3]]) and torch.equal(out[:20], alone[:20])
    out, sd, flags = go(cu, [0, 1, 2, 3, -1, -1], 19)
    assert flags == kda.KDA_ERR_SEQ  # 20 and 30 tokens
    assert torch.equal(sd[[0, 2]], state[[0, 2]]) and (out[:20] == 5).all() and (out[30:60] == 5).all()


def test_prefill_then_steps_then_prefill():
    """A prompt, single tokens and a second chunk continue one another: as one long sequence."""
    heads, lens = 2, [90, 141, 33]
    T = sum(lens) + 3
    (q, k, v), (qd, kd, vd), g, r = _attn(T, heads, heads, 31, True)
    state = torch.full((3, heads, 128, 128), float("nan"), device=DEV)  # a new sequence does not read its slot
    slots = torch.tensor([1], dtype=torch.int32, device=DEV)
    gd = g.to(DEV)
    outs, at = [], 0
    for i, n in enumerate(lens):
        e = at + n
        outs.append(kda.la_prefill(qd[at:e], kd[at:e], vd[at:e], gd[at:e], state=state, slots=slots,
                                   cu_seqlens=torch.tensor([0, n], dtype=torch.int32, device=DEV), max_len=n,
                                   has_state=torch.ones(1, dtype=torch.int32, device=DEV) if i else None))
        outs.append(kda.la_step(qd[e:e + 1], kd[e:e + 1], vd[e:e + 1], gd[e:e + 1], state=state, slots=slots))
        at = e + 1
    zero = torch.zeros(heads, 128, 128)
    o, S, mag, M, states = R.attention(q, k, v, g, 128 ** -0.5, zero)
    # chunks begin where each call does: the bound of the sum over both ways to cut
    at, bound = 0, torch.zeros_like(o)
    for n in lens:
        start = states[at - 1] if at else zero
        for a, b in ((at, at + n), (at + n, at + n + 1)):
            bo, bs = R.prefill_bounds(q[a:b], k[a:b], v[a:b], g[a:b], 128 ** -0.5, o[a:b], S, mag[a:b], M,
                                      states[a:b], states[a - 1] if a else zero, False)
            bound[a:b] = bo
        at += n + 1
    fine = 6 * (R.UBF16 ** 2 + 400 * R.U32)  # six calls, each within its own share of the magnitudes
    _close(torch.cat(outs), o, bound + fine * mag, "out")
    _close(state[1], S, fine * M, "state")
    assert torch.isnan(state[[0, 2]]).all()
