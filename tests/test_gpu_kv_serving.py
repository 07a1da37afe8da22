"""The 8-bit product, cache and attention as a server uses them: scratch that
holds anything, captured steps whose lengths grow, shared prefixes, mixed and
wide batches, large pools."""
import numpy as np
import pytest

from rank_error_correction_b200 import build, glowq

import plain8
import test_gpu_w8a8 as w8
from test_gpu_kv import PAGE, Server, cuda
from test_gpu_kv_extremes import kernel_of

pytestmark = pytest.mark.gpu
HEAD = 65536


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    glowq.lib()
    yield
    assert glowq.device_status() == 0


@pytest.fixture
def filled():
    """New memory holds NaN (floating point) or the largest integer."""
    import torch
    torch.use_deterministic_algorithms(True, warn_only=True)
    yield
    torch.use_deterministic_algorithms(False)


KERNELS = [("pages", 4, 2, 128, [300, 70], [1, 3]), ("pages", 2, 1, 64, [9000], [4]), ("tiles", 4, 2, 64, [100, 0], [150, 90]),
           ("shares", 4, 2, 128, [4000], [200])]


@pytest.mark.parametrize("T", [1, 13, 40, 333, 2000])
def test_product_scratch_may_hold_anything(T, filled):
    """Only its head is cleared, and no other byte of it matters."""
    import torch
    d, outs, r = 2048, [512, 304], 64
    mods, B, X = w8.make(T, d, outs, r, seed=T)
    dm = w8.dev_mods(mods)
    ws = glowq.w8a8_workspace(T, d, r, outs)
    assert int(ws[:HEAD].max()) == 0 and int(ws[HEAD:].min()) == 255
    Ys, R = glowq.group_forward_w8a8(dm, cuda(B), cuda(X))
    w8.check(Ys, R, *plain8.w8a8(X, mods, B))
    Y = glowq.solo_forward_w8a8(dm[1], cuda(B), cuda(X))
    w8.check([Y], None, plain8.w8a8(X, mods[1:], B)[0], (None, None))


@pytest.mark.parametrize("kernel,Hq,Hkv,D,cached,new", KERNELS)
def test_attention_scratch_may_hold_anything(kernel, Hq, Hkv, D, cached, new, filled):
    sv = Server(len(new), Hq, Hkv, D, (max(cached) + max(new)) // PAGE + 2, seed=D)
    sv.step(cached)
    b, Q, qr = sv.step(new)
    assert kernel_of(sv.cache, b, Hq) == kernel
    sv.ws = glowq.kv_attention_workspace(sv.cache, b, Hq)
    assert int(sv.ws[:HEAD].max()) == 0 and (kernel == "tiles" or int(sv.ws[HEAD:].min()) == 255)
    got = sv.check_attention(b, Q, qr, new)[:, :-8]
    assert np.array_equal(glowq.kv_attention(sv.cache, b, Q).cpu().numpy(), got)
