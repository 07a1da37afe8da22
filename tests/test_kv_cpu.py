"""Key/value cache and attention calls that the library refuses, on the host
before anything is enqueued (made-up addresses), and the workspace query."""
import ctypes as C

import pytest

from rank_error_correction_b200 import build, glowq

ARG, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    build.build()
    return glowq.lib()


def _cache(**kw):
    v = dict(k_codes=0x1000, v_codes=0x2000, k_scales=0x3000, v_scales=0x4000, k_tail=0x5000, v_tail=0x6000, pages=10,
             slots=4, kv_heads=2, head_dim=128)
    v.update(kw)
    return C.byref(glowq._KVCache(**v))


def _batch(**kw):
    v = dict(q_start=0x7000, kv_len=0x7100, page_table=0x7200, slot=0x7300, n_seq=2, max_pages=8, rows=4, max_new=3)
    v.update(kw)
    return C.byref(glowq._KVBatch(**v))


def _append(L, c=None, b=None, Q=0x8000, ldQ=512, hq=4, K=0x9000, ldK=256, V=0xa000, ldV=256, rope=0xb000, n=100,
            Qo=0xc000, ldO=512):
    return L.glowq_kv_append(c or _cache(), b or _batch(), Q, ldQ, hq, K, ldK, V, ldV, rope, n, Qo, ldO, None)


def _read(L, c=None, b=None, first=0x8000, count=5, K=0x9000, V=0xa000):
    return L.glowq_kv_read(c or _cache(), b or _batch(), first, count, K, V, None)


def _attend(L, c=None, b=None, Q=0x8000, ldQ=512, hq=4, scale=0.1, Y=0x9000, ldY=512, ws=0xa000, n=1 << 30):
    return L.glowq_kv_attention(c or _cache(), b or _batch(), Q, ldQ, hq, scale, Y, ldY, ws, n, None)


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_caches_and_batches(L, call):
    for kw, code in [(dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE), (dict(kv_heads=0), ARG),
                     (dict(pages=-1), ARG), (dict(slots=-1), ARG), (dict(k_codes=None), ARG), (dict(v_scales=None), ARG),
                     (dict(v_tail=None), ARG), (dict(k_codes=0x1008), ALIGN), (dict(v_tail=0x6004), ALIGN),
                     (dict(k_scales=0x3002), ALIGN), (dict(kv_heads=1 << 17), SHAPE), (dict(pages=1 << 40), SHAPE)]:
        assert call(L, c=_cache(**kw)) == code, kw
    for kw, code in [(dict(n_seq=-1), ARG), (dict(rows=-1), ARG), (dict(max_new=-1), ARG), (dict(max_pages=-1), ARG),
                     (dict(q_start=None), ARG), (dict(kv_len=None), ARG), (dict(slot=None), ARG),
                     (dict(page_table=None), ARG), (dict(q_start=0x7002), ALIGN), (dict(n_seq=1 << 25), SHAPE),
                     (dict(rows=1 << 31), SHAPE), (dict(max_pages=1 << 25), SHAPE),
                     (dict(n_seq=1 << 24, rows=1 << 30, max_new=1 << 20), SHAPE if call is not _read else 0)]:
        if kw.get("n_seq") == 1 << 24 and call is _read:
            continue
        assert call(L, b=_batch(**kw)) == code, kw
    assert call(L, b=_batch(n_seq=0, q_start=None, kv_len=None, slot=None, page_table=None)) == 0   # nothing to do
    assert call(L, c=_cache(pages=0, k_codes=None, v_codes=None, k_scales=None, v_scales=None), b=_batch(n_seq=0)) == 0


def test_arrays(L):
    assert _append(L, K=None) == ARG and _append(L, V=None) == ARG
    assert _append(L, Q=None) == ARG                              # heads without queries
    assert _append(L, Qo=None) == ARG
    assert _append(L, hq=3) == SHAPE and _append(L, hq=-1) == ARG
    assert _append(L, K=0x9008) == ALIGN and _append(L, ldK=248) == ALIGN and _append(L, ldV=260) == ALIGN
    assert _append(L, ldQ=504) == ALIGN and _append(L, ldO=504) == ALIGN
    assert _append(L, rope=0xb004) == ALIGN and _append(L, rope=None) == ARG and _append(L, n=-1) == ARG
    assert _append(L, b=_batch(max_new=0)) == 0
    assert _read(L, count=-1) == ARG and _read(L, count=(1 << 29) + 1) == SHAPE
    assert _read(L, K=None) == ARG and _read(L, V=0xa004) == ALIGN and _read(L, first=0x8002) == ALIGN
    assert _read(L, count=0) == 0
    assert _attend(L, Q=None) == ARG and _attend(L, Y=None) == ARG
    assert _attend(L, hq=3) == SHAPE and _attend(L, hq=0) == ARG
    assert _attend(L, ldQ=504) == ALIGN and _attend(L, Y=0x9004) == ALIGN
    assert _attend(L, scale=float("nan")) == ARG and _attend(L, scale=-1.0) == ARG and _attend(L, scale=float("inf")) == ARG
    assert _attend(L, ws=None) == ARG and _attend(L, ws=0xa008) == ALIGN and _attend(L, n=65535) == ARG
    need = L.glowq_kv_attention_workspace_bytes(_cache(), _batch(), 4)
    assert need >= 65536 and _attend(L, n=need - 1) == ARG
    assert L.glowq_kv_attention_workspace_bytes(_cache(), _batch(), 3) == 0
    assert L.glowq_kv_attention_workspace_bytes(_cache(head_dim=80), _batch(), 4) == 0
    assert _attend(L, b=_batch(max_new=0)) == 0


def test_status_has_a_text(L):
    assert b"range" in L.glowq_status_string(8)


def test_binding_refuses():
    import torch
    with pytest.raises(ValueError, match="CUDA"):
        glowq.KVCache(torch.zeros(1, 1, 1, 64, 64, dtype=torch.int8), None, None, None, None, None)
    with pytest.raises(ValueError, match="head_dim"):
        glowq.KVCache.alloc(1, 1, 1, 96, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        i = lambda *s: torch.zeros(*s, dtype=torch.int32)
        glowq.KVBatch(i(3), i(2), i(2, 4), i(2), 2, 1)


@pytest.mark.parametrize("off", [4, 8, 12])
def test_rotation_table_is_read_16_bytes_at_a_time(L, off):
    """A view of a larger table may begin at any float: only 16-byte boundaries are taken."""
    assert _append(L, rope=0xb000 + off) == ALIGN


def test_a_step_without_rows_needs_no_arrays(L):
    for b in (_batch(rows=0), _batch(max_new=0), _batch(n_seq=0)):
        assert _append(L, b=b, Q=None, K=None, V=None, Qo=None, ldQ=512) == 0
        assert _attend(L, b=b, Q=None, Y=None) == 0
    assert _append(L, b=_batch(rows=0), Q=None, hq=3) == SHAPE
