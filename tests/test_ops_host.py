"""The operators of include/kda_ops.h without a GPU: the header's functions are
exported, invalid arguments are rejected before any CUDA call, the binding's
names resolve, and the 64-bit forms the GPU tests compare with are pinned."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import linear_attention_decode_03_gb300 as kda
from tests import ops_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 12  # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    kda.build()
    return kda.load_library()


def test_header_and_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kda_ops.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?(?:long long|int)\s+(kda_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(["kda_quant_rows", "kda_linear_i8", "kda_linear_i8_check", "kda_la_step",
                            "kda_la_prefill", "kda_la_prefill_workspace", "kda_la_check"])
    raw = ctypes.CDLL(kda.LIB_PATH)
    for name in names:
        assert hasattr(raw, name), name
    for name in ("quant_rows", "linear_i8", "la_step", "la_prefill", "la_prefill_workspace", "kda_la_check"):
        assert callable(getattr(kda, name)) and name in kda.__all__


QUANT = dict(x=P, rows=4, ldx=64, cols=64, res=None, ldr=0, w=None, eps=1e-6, q=P, ldq=64, scales=P, stream=None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(cols=8), dict(cols=56), dict(cols=32784, ldx=32784, ldq=32784), dict(x=None),
    dict(q=None), dict(scales=None), dict(ldx=56), dict(ldx=68), dict(ldq=56), dict(ldq=68), dict(x=P + 2),
    dict(q=P + 4), dict(scales=P + 2), dict(res=P, ldr=56), dict(res=P, ldr=66), dict(res=P + 8, ldr=64),
    dict(w=P + 8), dict(w=P, eps=-1e-6), dict(w=P, eps=float("nan")), dict(rows=1 << 31)])
def test_quant_rows_refusals(lib, change):
    assert lib.kda_quant_rows(*{**QUANT, **change}.values()) == -1


I8 = dict(x=P, rows=4, ldx=64, sx=P, w=P, sw=P, N=8, K=64, y=P, ldy=8, stream=None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(N=0), dict(K=0), dict(K=8), dict(K=56), dict(x=None), dict(sx=None), dict(w=None),
    dict(sw=None), dict(y=None), dict(ldx=48), dict(ldx=72), dict(ldy=7), dict(x=P + 8), dict(w=P + 8),
    dict(y=P + 1), dict(sx=P + 2), dict(sw=P + 1), dict(K=1 << 32, ldx=1 << 32), dict(N=1 << 32, ldy=1 << 32),
    dict(rows=1 << 32)])
def test_linear_i8_refusals(lib, change):
    assert lib.kda_linear_i8(*{**I8, **change}.values()) == -1


STEP = dict(q=P, ldq=256, k=P, ldk=256, v=P, ldv=512, rows=2, heads=4, qk_heads=2, g=P, ldg=0, scale=1.0, state=P,
            dtype=0, pool=4, slots=P, out=P, ldo=512, stream=None)
COMMON = [
    dict(rows=-1), dict(heads=0), dict(heads=65536, qk_heads=1), dict(qk_heads=0), dict(qk_heads=3), dict(q=None),
    dict(k=None), dict(v=None), dict(g=None), dict(state=None), dict(slots=None), dict(out=None), dict(pool=0),
    dict(pool=1 << 31), dict(dtype=2), dict(dtype=-1), dict(ldq=128), dict(ldk=248), dict(ldv=504), dict(ldo=504),
    dict(ldq=260), dict(ldk=257), dict(ldv=516), dict(ldo=514), dict(ldg=3), dict(ldg=-4), dict(q=P + 8),
    dict(k=P + 2), dict(v=P + 4), dict(out=P + 8), dict(state=P + 8), dict(g=P + 2), dict(slots=P + 2)]


@pytest.mark.parametrize("change", COMMON + [dict(rows=1 << 31)])
def test_la_step_refusals(lib, change):
    assert lib.kda_la_step(*{**STEP, **change}.values()) == -1


PREFILL = dict(q=P, ldq=256, k=P, ldk=256, v=P, ldv=512, rows=2, heads=4, qk_heads=2, g=P, ldg=0, scale=1.0, cu=P,
               seqs=1, max_len=2, has_state=None, state=P, dtype=0, pool=4, slots=P, out=P, ldo=512, ws=P,
               ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change", COMMON + [
    dict(rows=1 << 31), dict(cu=None), dict(cu=P + 2), dict(seqs=-1), dict(max_len=-1), dict(has_state=P + 2),
    dict(seqs=1 << 31)])
def test_la_prefill_refusals(lib, change):
    assert lib.kda_la_prefill(*{**PREFILL, **change}.values()) == -1


def test_nothing_to_do(lib):
    # the sizes are checked first; with nothing to do the pointers are not looked at
    assert lib.kda_quant_rows(*{**QUANT, "rows": 0, "x": None, "q": None, "scales": None}.values()) == 0
    assert lib.kda_linear_i8(*{**I8, "rows": 0, "x": None, "y": None}.values()) == 0
    assert lib.kda_la_step(*{**STEP, "rows": 0, "q": None, "out": None}.values()) == 0
    assert lib.kda_la_prefill(*{**PREFILL, "seqs": 0, "q": None, "cu": None}.values()) == 0
    assert lib.kda_linear_i8_check(None, None) == -1
    assert lib.kda_la_check(None, None) == -1
    for sizes in ((-1, 2, 1, 1), (8, 0, 1, 8), (8, 2, -1, 8), (8, 2, 1, -1), (1 << 31, 2, 1, 8)):
        assert lib.kda_la_prefill_workspace(*sizes) == 0


def test_binding_wants_cuda_tensors():
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    i8, f = torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2)
    qkv, g = torch.zeros(2, 1, 128, dtype=torch.bfloat16), torch.zeros(1)
    state, slots = torch.zeros(2, 1, 128, 128), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        kda.quant_rows(x)
    with pytest.raises(TypeError):
        kda.linear_i8(i8, f, i8, f)
    with pytest.raises(TypeError):
        kda.la_step(qkv, qkv, qkv, g, state=state, slots=slots)
    with pytest.raises(TypeError):
        kda.la_prefill(qkv, qkv, qkv, g, state=state, slots=slots, cu_seqlens=slots, max_len=2)


def test_reference_quantisation_decides_halves():
    # 127 p / top next to and on halves: top = 2, p = (2 m + 1) / 127 is no bf16; build exact ties with top = 254
    x = torch.tensor([[254.0, 1.0, 3.0, -1.0, -3.0, 5.0, 0.0, -254.0]]).bfloat16()
    q, s, _ = R.quant_rows(x, None, None, 0.0)
    assert q.tolist() == [[127, 0, 2, 0, -2, 2, 0, -127]]  # 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    assert s.item() == 2.0
    r = torch.Generator().manual_seed(1)
    x = torch.randn(64, 256, generator=r).bfloat16()
    q, s, _ = R.quant_rows(x, None, None, 0.0)
    assert ((q * s[:, None] - x.double()).abs() <= 0.5 * s[:, None] * (1 + 1e-12)).all()


def test_reference_attention_closed_forms():
    r = torch.Generator().manual_seed(2)
    T, H = 5, 2
    q, k, v = (torch.randn(T, h, 128, generator=r).bfloat16() for h in (1, 1, H))
    S0 = torch.randn(H, 128, 128, generator=r)
    # a decay of zero keeps the last token alone; no decay sums all of them
    out, S, _, _, _ = R.attention(q, k, v, torch.full((T, H), -float("inf")), 1.0, S0)
    want = v[-1].double()[:, :, None] * k[-1].double()[:, None, :]
    assert torch.equal(S, want) and torch.allclose(out[-1], (want * q[-1].double()[:, None, :]).sum(-1))
    out, S, _, _, _ = R.attention(q, k, v, torch.zeros(T, H), 0.5, S0)
    want = S0.double() + torch.einsum("thv,tk->hvk", v.double(), k.double()[:, 0])
    assert torch.allclose(S, want) and torch.allclose(out[-1], 0.5 * torch.einsum("hvk,k->hv", want, q[-1, 0].double()))
