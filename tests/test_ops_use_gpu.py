"""The operators as a layer uses them: one after the other (prompt, then
tokens; around the KDA core), on other streams, in captured graphs, two calls
at once, the same call twice, buffers whose offsets pass 32 bits."""
from __future__ import annotations

import dataclasses

import numpy as np
import pytest
import torch

import linear_attention_decode_03_gb300 as kda
from tests import gpu_harness as G
from tests import ops_reference as R
from tests.helpers import case

pytestmark = pytest.mark.gpu
DEV = "cuda"
HIDDEN, HEADS = 512, 2
DIM = HEADS * 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def _close(got, want, bound, what):
    diff = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all() and (diff <= bound).all(), f"{what}: off by up to {diff.max():.3g}"


class Layer:
    """Norm, 8-bit in_proj, linear attention, 8-bit o_proj, with its weights quantised by quant_rows."""

    def __init__(self, seed=1):
        r = torch.Generator().manual_seed(seed)
        self.norm = (1 + 0.1 * torch.randn(HIDDEN, generator=r)).bfloat16().to(DEV)
        self.w_in, self.s_in = kda.quant_rows((0.05 * torch.randn(3 * DIM, HIDDEN, generator=r)).bfloat16().to(DEV))
        self.w_o, self.s_o = kda.quant_rows((0.05 * torch.randn(HIDDEN, DIM, generator=r)).bfloat16().to(DEV))
        self.g = torch.tensor([-0.3, -0.02], device=DEV)

    def __call__(self, x, residual, state, slots, prompt=None, keep=None):
        """prompt: (cu_seqlens, max_len, has_state), or None for a token a sequence."""
        q8, sq = kda.quant_rows(x, residual=residual, norm_weight=self.norm)
        proj = kda.linear_i8(q8, sq, self.w_in, self.s_in)
        q, k, v = (proj[:, i * DIM:(i + 1) * DIM].view(-1, HEADS, 128) for i in range(3))
        if prompt is None:
            core = kda.la_step(q, k, v, self.g, state=state, slots=slots)
        else:
            cu, max_len, has = prompt
            core = kda.la_prefill(q, k, v, self.g, state=state, slots=slots, cu_seqlens=cu, max_len=max_len,
                                  has_state=has)
        c8, sc = kda.quant_rows(core.view(-1, DIM))
        y = kda.linear_i8(c8, sc, self.w_o, self.s_o)
        if keep is not None:
            keep.update(q8=q8, sq=sq, proj=proj, core=core, c8=c8, sc=sc)
        return y


def _inputs(rows, seed):
    r = torch.Generator().manual_seed(seed)
    return torch.randn(rows, HIDDEN, generator=r).bfloat16(), torch.randn(rows, HIDDEN, generator=r).bfloat16()


def test_layer_stage_by_stage():
    """Prompts, then two rounds of single tokens: each stage against its 64-bit form on what the stage before gave."""
    layer = Layer()
    lens = [140, 33, 270]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    state = torch.zeros(5, HEADS, 128, 128, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    before = torch.zeros(5, HEADS, 128, 128)
    for turn in range(3):
        rows = sum(lens) if turn == 0 else 3
        x, res = _inputs(rows, 10 + turn)
        rd, st = res.to(DEV), {}
        prompt = (torch.from_numpy(cu).to(DEV), max(lens), None) if turn == 0 else None
        y = layer(x.to(DEV), rd, state, slots, prompt, keep=st)
        c = {n: t.cpu() for n, t in st.items()}
        wq, ws, wh = R.quant_rows(x, res, layer.norm.cpu(), 1e-6)
        assert torch.equal(c["q8"].long(), wq) and torch.equal(rd.cpu(), wh)
        _close(st["sq"], ws, R.scale_bound(HIDDEN) * ws, "scales")
        args = (c["q8"], c["sq"], layer.w_in.cpu(), layer.s_in.cpu())
        ref = R.linear_i8(*args)
        _close(st["proj"], ref, R.linear_i8_bound(*args, ref), "in_proj")
        q, k, v = (c["proj"][:, i * DIM:(i + 1) * DIM].view(-1, HEADS, 128) for i in range(3))
        g = layer.g.cpu().expand(rows, HEADS)
        scale = 128 ** -0.5
        after = state.cpu()
        for i, s in enumerate(slots.tolist()):
            a, b = (int(cu[i]), int(cu[i + 1])) if turn == 0 else (i, i + 1)
            o, S, mag, M, states = R.attention(q[a:b], k[a:b], v[a:b], g[a:b], scale, before[s])
            if turn == 0:
                bo, bs = R.prefill_bounds(q[a:b], k[a:b], v[a:b], g[a:b], scale, o, S, mag, M, states, before[s], False)
            else:
                bo, bs = R.step_bounds(o, S, mag, M, False)
            _close(st["core"][a:b], o, bo, f"core {turn} {i}")
            _close(after[s], S, bs, f"state {turn} {i}")
        wq, ws, _ = R.quant_rows(c["core"].view(-1, DIM), None, None, 0.0)
        assert torch.equal(c["c8"].long(), wq)
        args = (c["c8"], c["sc"], layer.w_o.cpu(), layer.s_o.cpu())
        ref = R.linear_i8(*args)
        _close(y, ref, R.linear_i8_bound(*args, ref), "o_proj")
        before = after
    assert kda.kda_la_check() == 0 and kda.kda_linear_i8_check() == 0


def test_around_the_kda_core():
    """quant_rows -> linear_i8 writes the packed projection row that the KDA step reads: the step on it equals the
    oracle's on the same bits."""
    si = case(heads=2, requests=4, L=1, pool=8, seed=401)
    pitch = si.projected.shape[1]
    x, res = _inputs(4, 20)
    r = torch.Generator().manual_seed(21)
    w, sw = kda.quant_rows((0.05 * torch.randn(pitch, HIDDEN, generator=r)).bfloat16().to(DEV))
    q8, sq = kda.quant_rows(x.to(DEV), residual=res.to(DEV), norm_weight=torch.ones(HIDDEN).bfloat16().to(DEV))
    proj = kda.linear_i8(q8, sq, w, sw)
    si = dataclasses.replace(si, projected=G.torch_bf16_to_np(proj))
    ds = G.DeviceStep(si)
    ds.projected = proj
    assert ds.run() == 0
    out_ref, rows, used, pool_ref, conv_ref, err = G.oracle_requests(si, np.arange(4))
    assert err == 0
    G.assert_out_close(G.torch_bf16_to_np(ds.out), out_ref)
    c8, sc = kda.quant_rows(ds.out)
    w_o, s_o = kda.quant_rows((0.05 * torch.randn(HIDDEN, ds.out.shape[1], generator=r)).bfloat16().to(DEV))
    y = kda.linear_i8(c8, sc, w_o, s_o)
    args = (c8.cpu(), sc.cpu(), w_o.cpu(), s_o.cpu())
    ref = R.linear_i8(*args)
    _close(y, ref, R.linear_i8_bound(*args, ref), "o_proj")
    ds.close()


def _long_call(seed, tokens=2500, heads=3):
    """A prompt call that is cut into segments: fresh inputs, state and outputs."""
    r = torch.Generator(device=DEV).manual_seed(seed)
    q, k, v = (torch.randn(tokens, heads, 128, generator=r, device=DEV).bfloat16() for _ in range(3))
    return dict(q=q, k=k, v=v, g=torch.full((heads,), -0.01, device=DEV),
                state=torch.randn(2, heads, 128, 128, generator=r, device=DEV),
                slots=torch.tensor([1], dtype=torch.int32, device=DEV),
                cu_seqlens=torch.tensor([0, tokens], dtype=torch.int32, device=DEV), max_len=tokens,
                has_state=torch.ones(1, dtype=torch.int32, device=DEV))


def test_same_bits_every_time():
    layer = Layer()
    x, res = _inputs(300, 30)
    runs = []
    for _ in range(2):
        state = torch.zeros(2, HEADS, 128, 128, device=DEV)
        y = layer(x.to(DEV), res.to(DEV), state, torch.tensor([1], dtype=torch.int32, device=DEV),
                  (torch.tensor([0, 300], dtype=torch.int32, device=DEV), 300, None))
        c = _long_call(31)
        runs.append((y, state, kda.la_prefill(**c), c["state"]))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert kda.la_prefill_workspace(2500, 3, 1, 2500) > 0  # the long call has segments


def test_two_calls_at_once():
    """Prompts and products on two streams, both at a time: what each gives by itself."""
    calls = [_long_call(40), _long_call(41)]
    want = []
    for c in calls:
        c2 = {**c, "state": c["state"].clone()}
        want.append((kda.la_prefill(**c2), c2["state"]))
    r = torch.Generator(device=DEV).manual_seed(42)
    x = torch.randint(-127, 128, (200, 2048), generator=r, device=DEV).to(torch.int8)
    w = torch.randint(-127, 128, (3000, 2048), generator=r, device=DEV).to(torch.int8)
    sx, sw = torch.ones(200, device=DEV), torch.full((3000,), 1e-4, device=DEV)
    y_want = kda.linear_i8(x, sx, w, sw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(3):
        outs = []
        for c, s in zip(calls, streams):
            c2 = {**c, "state": c["state"].clone()}
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                outs.append((kda.la_prefill(**c2), c2["state"], kda.linear_i8(x, sx, w, sw)))
        torch.cuda.synchronize()
        got.append(outs)
    for outs in got:
        for (o, st, y), (wo, ws) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(st, ws) and torch.equal(y, y_want)
    assert kda.kda_la_check() == 0 and kda.kda_linear_i8_check() == 0


def test_an_explicit_stream():
    """stream= : the call runs there, behind what is there, and its own workspace belongs to that stream."""
    c = _long_call(50)
    c2 = {**c, "state": c["state"].clone()}
    want = kda.la_prefill(**c2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(want)
    q = torch.zeros_like(c["q"])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        q.copy_(c["q"])  # behind the sleep: a call on another stream would read zeros
    got = kda.la_prefill(**{**c, "q": q}, out=out, stream=s.cuda_stream)
    junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(8)]  # would land in a freed workspace
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(c["state"], c2["state"])
    del junk


def test_results_of_an_explicit_stream():
    """stream= without out: the results are that stream's memory, not blocks that the current stream has freed with
    writes still to come."""
    r = torch.Generator().manual_seed(70)
    x = torch.randn(64, 1024, generator=r).bfloat16().to(DEV)
    w = torch.randint(-127, 128, (512, 1024), generator=r).to(torch.int8).to(DEV)
    sw = torch.rand(512, generator=r).to(DEV)
    q8, sx = kda.quant_rows(x)
    y = kda.linear_i8(q8, sx, w, sw)
    qkv = torch.randn(3, 64, 2, 128, generator=r).bfloat16().to(DEV)
    g = -torch.rand(2, generator=r).to(DEV)
    slots = torch.arange(64, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 64], dtype=torch.int32, device=DEV)

    def state():
        return torch.zeros(64, 2, 128, 128, device=DEV)

    calls = [lambda s: kda.quant_rows(x, stream=s), lambda s: (kda.linear_i8(q8, sx, w, sw, stream=s),),
             lambda s: (kda.la_step(*qkv, g, state=states[0], slots=slots, stream=s),),
             lambda s: (kda.la_prefill(*qkv, g, state=states[1], slots=slots, cu_seqlens=cu, max_len=64, stream=s),)]
    states = [state(), state()]
    want = [[t.clone() for t in c(None)] for c in calls]
    assert torch.equal(want[0][0], q8) and torch.equal(want[1][0], y)
    side = torch.cuda.Stream()
    for s in (side.cuda_stream, 0):
        states = [state(), state()]
        torch.cuda.synchronize()
        for call, expect in zip(calls, want):
            kept = [torch.empty_like(t) for t in expect]  # a block of each size that the call would be given
            torch.cuda.synchronize()
            with torch.cuda.stream(torch.cuda.default_stream()):
                torch.cuda._sleep(10_000_000)
            for t in kept:
                t.view(torch.uint8).fill_(99)
            del kept, t
            got = call(s)
            torch.cuda.synchronize()
            for a, b in zip(got, expect):
                assert torch.equal(a, b)


def test_captured_and_replayed():
    """The layer in a CUDA graph, replayed on new inputs, equals the calls made one by one; two graphs with
    segments each have a workspace of their own."""
    layer = Layer()
    slots = torch.tensor([1], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 200], dtype=torch.int32, device=DEV)
    x, res = (t.to(DEV) for t in _inputs(200, 60))
    tok, tok_res = (t.to(DEV) for t in _inputs(1, 61))
    state = torch.zeros(2, HEADS, 128, 128, device=DEV)
    calls = [_long_call(62), _long_call(63)]
    layer(x, res.clone(), state, slots, (cu, 200, None))  # warm: first-use lookups are no part of a capture
    kda.la_prefill(**{**calls[0], "state": calls[0]["state"].clone()})
    torch.cuda.synchronize()
    first = [c["state"].clone() for c in calls]
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = layer(x, res, state, slots, (cu, 200, None))
            y1 = layer(tok, tok_res, state, slots)
            o = kda.la_prefill(**c)
        graphs.append(g)
        outs.append((y, y1, o))
    for seed in (64, 65):
        for g, c, (y, y1, o), st0 in zip(graphs, calls, outs, first):
            nx, nres = _inputs(200, seed)
            nt, ntr = _inputs(1, seed + 100)
            for dst, src in ((x, nx), (res, nres), (tok, nt), (tok_res, ntr)):
                dst.copy_(src)
            c["state"].copy_(st0)
            state.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            st2 = torch.full_like(state, float("nan"))
            c2 = {**c, "state": st0.clone()}
            assert torch.equal(y, layer(nx.to(DEV), nres.to(DEV), st2, slots, (cu, 200, None)))
            assert torch.equal(y1, layer(nt.to(DEV), ntr.to(DEV), st2, slots))
            assert torch.equal(state[1], st2[1]) and torch.isnan(state[0]).all()
            assert torch.equal(o, kda.la_prefill(**c2)) and torch.equal(c["state"], c2["state"])
    for g in graphs:  # back to back, nothing waited for between them
        g.replay()
    torch.cuda.synchronize()
    assert kda.kda_la_check() == 0 and kda.kda_linear_i8_check() == 0


def test_one_after_the_other_without_a_pause(monkeypatch):
    """Calls whose CTAs may be placed while the call before them ends: prompts, tokens and copies on the same buffers,
    all queued at once, give what they give with a wait behind every call."""
    from linear_attention_decode_03_gb300 import ops

    layer = Layer()
    real = ops._call

    def waiting(name, device, stream, *args):
        real(name, device, stream, *args)
        torch.cuda.synchronize()

    rows, turns = (1, 40, 300), 12
    sources = [[tuple(t.to(DEV) for t in _inputs(n, 80 + i)) for n in rows] for i in range(turns)]
    long = [_long_call(130), _long_call(131)]
    slots = torch.tensor([1], dtype=torch.int32, device=DEV)
    ends = {n: torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in rows}
    results = []
    for call in (real, waiting):
        monkeypatch.setattr(ops, "_call", call)
        x, res = (torch.zeros(max(rows), HIDDEN, device=DEV).bfloat16() for _ in range(2))
        state = torch.zeros(2, HEADS, 128, 128, device=DEV)
        big = torch.empty_like(long[0]["v"])
        st = long[0]["state"].clone()
        got = []
        torch.cuda.synchronize()
        for i in range(turns):
            for n, (sx, sr) in zip(rows, sources[i]):
                x[:n].copy_(sx)
                res[:n].copy_(sr)
                y = layer(x[:n], res[:n], state, slots, None if n == 1 else (ends[n], n, slots))
                x[:n].fill_(float("nan"))
                got += [y, res[:n].clone()]
                res[:n].fill_(float("nan"))
            kda.la_prefill(**{**long[i % 2], "state": st}, out=big)
            q8, s8 = kda.quant_rows(big.view(-1, 384))
            big.fill_(float("nan"))
            got += [q8, s8, st.clone(), state.clone()]
        torch.cuda.synchronize()
        results.append(got)
    for a, b in zip(*results):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_captured_in_branches():
    """Calls as a graph's first nodes, behind copies, on two branches and where they meet."""
    layer = Layer()
    x, res = (t.to(DEV) for t in _inputs(70, 140))
    src = [t.clone() for t in (x, res)]
    c = _long_call(141)
    first = c["state"].clone()
    tok = {n: c[n][:1] for n in "qkv"}
    state = torch.zeros(1, 3, 128, 128, device=DEV)
    slots = torch.zeros(1, dtype=torch.int32, device=DEV)

    def both(side):
        main = torch.cuda.current_stream()
        q0, s0 = kda.quant_rows(src[0], norm_weight=layer.norm)  # nothing before it
        side.wait_stream(main)
        with torch.cuda.stream(side):
            o1 = kda.la_step(**tok, g=c["g"], state=state, slots=slots)
            o2 = kda.la_prefill(**c)
        x.copy_(src[0])
        res.copy_(src[1])
        q8, sq = kda.quant_rows(x, residual=res, norm_weight=layer.norm)
        main.wait_stream(side)
        y = kda.linear_i8(q8, sq, layer.w_in, layer.s_in)  # behind both
        z, sz = kda.quant_rows(o2.view(-1, 384))
        o3 = kda.la_step(**tok, g=c["g"], state=state, slots=slots)
        return q0, s0, o1, o2, y, z, sz, o3

    side = torch.cuda.Stream()
    want = [t.clone() for t in both(side)]
    torch.cuda.synchronize()
    last, token = c["state"].clone(), state.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both(side)
    for _ in range(3):
        c["state"].copy_(first)
        state.zero_()
        x.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(c["state"], last) and torch.equal(state, token)
    assert kda.kda_la_check() == 0 and kda.kda_linear_i8_check() == 0


def test_offsets_past_32_bits():
    """A pool of more than 2^31 values, its last slot; rows and weights of more than 2^31 bytes."""
    heads, pool = 96, 1500
    assert pool * heads * 128 * 128 > 2 ** 31
    state = torch.zeros(pool, heads, 128, 128, dtype=torch.bfloat16, device=DEV)
    r = torch.Generator(device=DEV).manual_seed(70)
    q, k, v = (torch.randn(3, h, 128, generator=r, device=DEV).bfloat16() for h in (1, 1, heads))
    g = torch.full((heads,), -0.1, device=DEV)
    slots = torch.tensor([pool - 1], dtype=torch.int32, device=DEV)
    kda.la_prefill(q[:2], k[:2], v[:2], g, state=state, slots=slots, max_len=2,
                   cu_seqlens=torch.tensor([0, 2], dtype=torch.int32, device=DEV))
    kda.la_step(q[2:], k[2:], v[2:], g, state=state, slots=slots)
    small = torch.zeros(1, heads, 128, 128, dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    kda.la_prefill(q[:2], k[:2], v[:2], g, state=small, slots=zero, max_len=2,
                   cu_seqlens=torch.tensor([0, 2], dtype=torch.int32, device=DEV))
    kda.la_step(q[2:], k[2:], v[2:], g, state=small, slots=zero)
    assert torch.equal(state[-1], small[0]) and not state[:-1].any()
    assert kda.kda_la_check() == 0
    del state
    rows, cols = 70000, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-2:] = torch.randn(2, cols, generator=r, device=DEV).bfloat16()
    q8, s = kda.quant_rows(x)
    wq, ws, _ = R.quant_rows(x[-2:].cpu(), None, None, 0.0)
    assert torch.equal(q8[-2:].cpu().long(), wq) and not s[:-2].any()
    # the same bytes as a weight, and as the rows
    for n in (1, 40):
        xi = torch.randint(-127, 128, (n, cols), generator=r, device=DEV).to(torch.int8)
        y = kda.linear_i8(xi, torch.ones(n, device=DEV), q8, torch.full((rows,), 2.0 ** -20, device=DEV))
        args = (xi.cpu(), torch.ones(n), q8[-2:].cpu(), torch.full((2,), 2.0 ** -20))
        ref = R.linear_i8(*args)
        _close(y[:, -2:], ref, R.linear_i8_bound(*args, ref), "last columns")
        assert not y[:, :-2].any()
    y = kda.linear_i8(q8, torch.full((rows,), 2.0 ** -20, device=DEV), xi, torch.ones(40, device=DEV))
    args = (q8[-2:].cpu(), torch.full((2,), 2.0 ** -20), xi.cpu(), torch.ones(40))
    ref = R.linear_i8(*args)
    _close(y[-2:], ref, R.linear_i8_bound(*args, ref), "last rows")
    assert not y[:-2].any() and kda.kda_linear_i8_check() == 0


def test_separate_strided_tensors():
    """q, k, v and out of different strides, g of a row stride of its own, a decay a head given as an expanded
    matrix, heads shared by three."""
    r = torch.Generator().manual_seed(80)
    rows, heads = 150, 3
    q = torch.randn(rows, 4, 128, generator=r).bfloat16().to(DEV)[:, 2:3]
    k = torch.randn(rows, 1, 136, generator=r).bfloat16().to(DEV)[:, :, :128]
    v = torch.randn(rows, 5, 128, generator=r).bfloat16().to(DEV)[:, 1:4]
    g = -torch.rand(rows, 7, generator=r).to(DEV)[:, 2:5]
    whole = torch.full((rows, 6, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    out = whole[:, 2:5]
    cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(q, k, v, g, out=None):
        state = torch.zeros(1, heads, 128, 128, device=DEV)
        o = kda.la_prefill(q, k, v, g, state=state, slots=zero, cu_seqlens=cu, max_len=rows, out=out)
        o1 = kda.la_step(q[:1], k[:1], v[:1], g[:1], state=state, slots=zero)
        return o.clone(), o1, state

    a = run(q, k, v, g, out)
    b = run(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous())
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    assert (whole[:, :2] == 3).all() and (whole[:, 5:] == 3).all()
    one = torch.tensor([-0.5, -0.1, -0.01], device=DEV)
    state = [torch.zeros(1, heads, 128, 128, device=DEV) for _ in range(2)]
    o = [kda.la_prefill(q, k, v, gg, state=s, slots=zero, cu_seqlens=cu, max_len=rows)
         for gg, s in ((one, state[0]), (one.expand(rows, heads), state[1]))]
    assert torch.equal(o[0], o[1]) and torch.equal(state[0], state[1])


def test_refusals_of_the_binding():
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(2, device=DEV)
    state = torch.zeros(3, 2, 128, 128, device=DEV)
    slots = torch.zeros(4, dtype=torch.int32, device=DEV)
    good = dict(q=q, k=q, v=q, g=g, state=state, slots=slots)
    bad = [dict(k=q[:, :1]), dict(v=q[:3]), dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(g=g[:1]),
           dict(g=g.double()), dict(g=torch.zeros(3, 2, device=DEV)), dict(state=state.half()), dict(state=state[:, :1]),
           dict(state=state.transpose(2, 3)), dict(slots=slots.long()), dict(slots=slots[::2]), dict(state=state[0]),
           dict(v=torch.zeros(4, 3, 128, dtype=torch.bfloat16, device=DEV)), dict(k=q.cpu()), dict(state=None),
           dict(out=torch.zeros(4, 2, 128, device=DEV)), dict(out=q[:, :1])]
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for change in bad + [dict(slots=slots[:3])]:
        with pytest.raises((TypeError, ValueError)):
            kda.la_step(**{**good, **change})
    for change in bad + [dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[:0]), dict(has_state=slots[:2]), dict(max_len=-1),
                         dict(slots=slots[:0]), dict(workspace=torch.zeros(4, device=DEV))]:
        with pytest.raises((TypeError, ValueError)):
            kda.la_prefill(**{**good, "cu_seqlens": cu, "max_len": 4, **change})
    long = _long_call(90)
    with pytest.raises(ValueError):  # a workspace that is too small
        kda.la_prefill(**long, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(residual=x[:2]), dict(residual=x.float()), dict(norm_weight=x[0, :32]), dict(out=x),
               dict(scales=torch.zeros(2, device=DEV)), dict(residual=x.t()), dict(norm_weight=x[0].float())):
        with pytest.raises((TypeError, ValueError)):
            kda.quant_rows(x, **kw)
    with pytest.raises(kda.KdaError):
        kda.quant_rows(x[:, :40])  # not a multiple of 16 columns
    with pytest.raises(kda.KdaError):
        kda.quant_rows(x, residual=x[:1].expand(3, 64))  # rows that share their memory cannot all be written
    # pinned host memory where tensor maps address this GPU's own
    host = torch.zeros(1 << 16, dtype=torch.uint8).pin_memory().data_ptr()
    lib = kda.load_library()
    assert lib.kda_linear_i8(host, 32, 64, g.data_ptr(), q.data_ptr(), g.data_ptr(), 8, 64, q.data_ptr(), 8, None) == -1
    assert lib.kda_la_prefill(host, 256, q.data_ptr(), 256, q.data_ptr(), 256, 4, 2, 2, g.data_ptr(), 0, 1.0,
                              cu.data_ptr(), 1, 4, None, state.data_ptr(), 0, 3, slots.data_ptr(), q.data_ptr(), 256,
                              None, 0, None) == -1
