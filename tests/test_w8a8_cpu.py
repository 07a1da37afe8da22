"""W8A8 calls that the library refuses, on the host before anything is
enqueued (made-up addresses), and the workspace query."""
import ctypes as C

import pytest

from rank_error_correction_b200 import build, glowq

ARG, SHAPE, ALIGN = 1, 2, 3

@pytest.fixture(scope="module")
def L():
    build.build()
    return glowq.lib()

def _mods(n=1, O=128, q=0x10000, s=0x2000, A=0x3000, Y=0x4000, ldY=128):
    arr = (glowq._Int8Module * n)()
    for m in arr:
        m.codes, m.scales, m.A, m.out_features, m.Y, m.ldY = q, s, A, O, Y, ldY
    return arr

def _group(L, mods=None, m=1, d=256, B=0x5000, r=16, X=0x6000, T=4, R=0x7000, ws=0x8000, n=1 << 30):
    return L.glowq_group_forward_w8a8(_mods() if mods is None else mods, m, d, B, r, X, T, R, ws, n, None)

def test_refusals(L):
    assert _group(L, T=0) == 0                                   # an empty batch is a no-op
    assert _group(L, T=-1) == ARG
    assert _group(L, m=0) == ARG
    assert _group(L, _mods(9), m=9) == ARG
    assert _group(L, d=200) == SHAPE
    assert _group(L, d=131072 + 128) == SHAPE                    # 127^2 d would pass 2^31
    assert _group(L, r=12) == SHAPE
    assert _group(L, r=264) == SHAPE
    assert _group(L, _mods(O=100)) == SHAPE
    assert _group(L, _mods(O=0)) == SHAPE
    assert _group(L, _mods(q=None)) == ARG
    assert _group(L, _mods(s=None)) == ARG
    assert _group(L, _mods(Y=None)) == ARG
    assert _group(L, _mods(q=0x10008)) == ALIGN
    assert _group(L, _mods(s=0x2002)) == ALIGN
    assert _group(L, _mods(A=0x3008)) == ALIGN
    assert _group(L, _mods(Y=0x4002)) == ALIGN
    assert _group(L, _mods(ldY=120)) == ALIGN
    assert _group(L, _mods(ldY=132)) == ALIGN
    assert _group(L, B=None) == ARG
    assert _group(L, X=None) == ARG
    assert _group(L, X=0x6008) == ALIGN
    assert _group(L, R=None) == ARG
    assert _group(L, R=0x7004) == ALIGN
    assert _group(L, ws=None) == ARG
    assert _group(L, ws=0x8004) == ALIGN
    need = glowq.w8a8_workspace_bytes(4, 256, 16, [128])
    assert _group(L, n=need - 1) == ARG
    assert L.glowq_solo_forward_w8a8(_mods(), 256, 0x5000, 16, 0x6000, 4, None, 0, None) == ARG
    assert L.glowq_pack_int8(0x1000, 16, 200, 0x2000, 0x3000, None) == SHAPE
    assert L.glowq_pack_int8(0x1000, -1, 256, 0x2000, 0x3000, None) == ARG
    assert L.glowq_pack_int8(None, 16, 256, 0x2000, 0x3000, None) == ARG
    assert L.glowq_pack_int8(0x1008, 16, 256, 0x2000, 0x3000, None) == ALIGN
    assert L.glowq_pack_int8(None, 0, 256, None, None, None) == 0
    assert L.glowq_dequant_int8(0x1000, 0x2002, 16, 256, 0x3000, None) == ALIGN
    assert L.glowq_dequant_int8(0x1000, None, 16, 256, 0x3000, None) == ARG
    assert L.glowq_quantize_act_int8(0x1000, 4, 250, 0x2000, 0x3000, None) == SHAPE
    assert L.glowq_quantize_act_int8(0x1000, 0, 256, None, None, None) == 0
    assert L.glowq_quantize_act_int8(0x1000, 4, 256, 0x2004, 0x3000, None) == ALIGN

def test_workspace(L):
    f = glowq.w8a8_workspace_bytes
    assert f(0, 256, 16, [128]) == 0 and f(4, 200, 16, [128]) == 0 and f(4, 256, 12, [128]) == 0
    assert f(4, 256, 16, []) == 0 and f(4, 256, 16, [100]) == 0 and f(4, 1 << 18, 16, [128]) == 0
    for T in (1, 8, 9, 16, 17, 64, 65, 300, 4096):
        for d, r, outs in ((128, 0, [16]), (4096, 64, [4096] * 3), (14336, 256, [4096])):
            n = f(T, d, r, outs)
    
    assert L.glowq_w8a8_workspace_bytes(4, 256, 16, None, 1) == 0
    assert L.glowq_w8a8_workspace_bytes(4, 256, 16, (C.c_int64 * 9)(*[128] * 9), 9) == 0

def test_binding_refuses_what_is_not_on_a_gpu():
    import torch
    with pytest.raises(ValueError, match="CUDA"):
        glowq.pack_int8(torch.zeros(16, 128))
    with pytest.raises(ValueError, match="CUDA"):
        glowq.Int8ForwardPlan([], None, torch.zeros(1, 128, dtype=torch.float16))


@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 64, 65, 300, 4096])
@pytest.mark.parametrize("d,r,outs", [(128, 0, [16]), (4096, 64, [4096] * 3), (14336, 256, [4096])])
def test_workspace_holds_what_a_call_keeps_there(L, T, d, r, outs):
    """The head, the codes, a scale per token and a solo module's R at least, and beside them the sums of split tiles: of 74
    CTA pairs and fewer tiles than pairs, cut into shares of 8 k-blocks or more, there are 296 segments of two times 128
    rows x 256 tokens at most."""
    n = glowq.w8a8_workspace_bytes(T, d, r, outs)
    least = 65536 + T * d + 4 * T + 2 * T * r
    assert least <= n <= least + 16 * d + 4096 + 296 * 2 * 128 * 256 * 4
    assert n >= glowq.w8a8_workspace_bytes(T, d, 0, outs)
    assert glowq.w8a8_workspace_bytes(T, d, r, outs + [16]) > 65536


def test_a_product_of_no_tokens_needs_no_arrays(L):
    assert _group(L, _mods(Y=None), T=0, X=None, R=None, ws=None, n=0) == 0
    assert _group(L, _mods(Y=None, q=None), T=0) == ARG
    assert _group(L, _mods(Y=None, ldY=120), T=0) == ALIGN
    assert L.glowq_solo_forward_w8a8(_mods(Y=None), 256, 0x5000, 16, None, 0, None, 0, None) == 0
