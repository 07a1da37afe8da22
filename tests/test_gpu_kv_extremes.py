"""Attention over the 8-bit cache where single precision is at its ends, on both
kernels: which of them a call runs is read off the workspace that it asks for."""
import numpy as np
import pytest

from rank_error_correction_b200 import build, glowq

import plain8
from test_gpu_kv import PAGE, Server, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    glowq.lib()
    yield
    assert glowq.device_status() == 0


def kernel_of(cache, batch, Hq):
    """'pages' (few rows), 'tiles' or 'shares' (matrix tiles, whole or with a unit's tokens in shares), by the scratch
    behind the workspace's head: [block][2][8 or 16 rows][D + 4] floats, none, or [..][head][share][D + 2][256 rows]."""
    D = cache.head_dim
    n = glowq.kv_attention_workspace(cache, batch, Hq).numel() - 65536
    if n == 0:
        return "tiles"
    few, many = n % (2 * 8 * (D + 4) * 4) == 0, n % (cache.kv_heads * (D + 2) * 256 * 4) == 0
    assert few != many, n
    return "pages" if few else "shares"


def one_page_softmax(q, k, v, start, scale):
    """Rows whose weight is all in one page or the tail, with scores apart from the others' by far more than fp32's
    steps: (Y, bound, which rows).  There equal scores have equal weights and all others none, whatever the scores' size."""
    n, Hq, D = q.shape
    L, G = len(k), Hq // k.shape[1]
    Y, bound, ok = np.zeros((n, Hq, D)), np.ones((n, Hq, D)), np.zeros((n, Hq), bool)
    u16, u32 = 2.0 ** -11, 2.0 ** -23
    for i in range(n):
        m = min(L, start + i + 1)
        for h in range(Hq):
            s = k[:m, h // G] @ q[i, h].astype(np.float64) * scale
            top = s == s.max()
            # fp32 sums of D products and what is applied to them: off by no more than (D + 10) steps of the largest score
            gap = 100.0 + 2 * (D + 10) * u32 * np.abs(s).max()
            if np.any(~top & (s > s.max() - gap)) or len(set(np.nonzero(top)[0] // PAGE)) > 1:
                continue
            ok[i, h] = True
            Y[i, h] = v[:m, h // G][top].mean(0)
            # equal weights, each rounded to fp16 at most once and summed unrounded; sums in fp32; the output's rounding
            b = (u16 + (top.sum() + 8) * u32) * np.abs(v[:m, h // G][top]).mean(0)
            bound[i, h] = b + u16 * (np.abs(Y[i, h]) + b) + 2.0 ** -25
    return Y, bound, ok


@pytest.mark.parametrize("size,scale", [(300.0, None), (1000.0, None), (4000.0, 1.0), (20000.0, None),
                                        (30000.0, 1.0), (60000.0, 1e6)])
@pytest.mark.parametrize("kernel,Hq,Hkv,D,cached,new", [
    ("pages", 4, 2, 128, [1000, 130], [1, 3]), ("pages", 2, 2, 64, [640, 63], [1, 1]), ("pages", 2, 1, 128, [9000], [6]),
    ("pages", 16, 1, 64, [0, 300], [1, 1]), ("tiles", 4, 2, 128, [100, 0], [300, 70]), ("tiles", 4, 2, 64, [300, 64], [128, 200]),
    ("shares", 4, 2, 64, [4000], [200]),
])
def test_scores_of_any_size(kernel, Hq, Hkv, D, cached, new, size, scale):
    """Queries and keys along one direction, so that scores are as large as fp16 allows (past 2^36, past the steps at
    which single precision still counts ones), and the softmax is a choice."""
    sv = Server(len(new), Hq, Hkv, D, (max(cached) + max(new)) // PAGE + 2, seed=D + len(new))

    def data(counts):
        q, k, v = sv.draw(counts)
        T = sum(counts)
        k = np.broadcast_to(sv.g.uniform(0.2, 1.0, (T, Hkv, 1)) * size, k.shape).astype(np.float16)
        q = np.broadcast_to(sv.g.choice([-1.0, 1.0], (T, Hq, 1)) * sv.g.uniform(0.5, 1.0, (T, Hq, 1)) * size, q.shape)
        return q.astype(np.float16), k, v

    if any(cached):
        sv.step(cached, rope=False, data=data(cached))
    b, Q, qr = sv.step(new, rope=False, data=data(new))
    assert kernel_of(sv.cache, b, Hq) == kernel
    got = glowq.kv_attention(sv.cache, b, Q, scale=scale, workspace=sv.ws).cpu().numpy().reshape(-1, Hq, D)
    at, rows, worst = 0, 0, 0.0
    for s, n in zip(sv.seq, new):
        y, bound, ok = one_page_softmax(qr[at:at + n], *s.held(), len(s.k) - n, D ** -0.5 if scale is None else scale)
        worst = max(worst, plain8.within(got[at:at + n][ok], y[ok], bound[ok]))
        rows += ok.sum()
        at += n
    assert worst <= 1.0, worst
    assert rows >= sum(new) * Hq // 2, rows


@pytest.mark.parametrize("kernel,Hq,Hkv,D,cached,new", [
    ("pages", 4, 2, 128, 300, 3), ("tiles", 4, 2, 128, 100, 150), ("tiles", 2, 1, 64, 0, 200), ("shares", 4, 2, 64, 4000, 200),
])
def test_a_row_does_not_depend_on_the_scores_beside_it(kernel, Hq, Hkv, D, cached, new):
    """Every third query's scores pass 2^24 (and so does what a warp does with them): the others keep their bits."""
    sv = Server(1, Hq, Hkv, D, (cached + new) // PAGE + 2, seed=3)
    if cached:
        sv.step([cached])
    b, Q, _ = sv.step([new])
    assert kernel_of(sv.cache, b, Hq) == kernel
    want = glowq.kv_attention(sv.cache, b, Q, scale=500.0, workspace=sv.ws)
    Q2 = Q.clone()
    Q2[::3] *= 6000.0
    assert bool(Q2.isfinite().all())
    got = glowq.kv_attention(sv.cache, b, Q2, scale=500.0, workspace=sv.ws)
    rest = np.arange(new) % 3 != 0
    assert bool(got.isfinite().all())
    assert np.array_equal(got.cpu().numpy()[rest], want.cpu().numpy()[rest])


INFINITE = [
    ("pages", 4, 2, 64, 0, 1, 0), ("pages", 4, 2, 128, 5, 1, 0), ("pages", 2, 1, 128, 63, 1, 0), ("pages", 2, 2, 64, 100, 3, 1),
    ("pages", 2, 1, 64, 6000, 2, 0), ("tiles", 4, 2, 128, 0, 150, 0), ("tiles", 4, 2, 64, 0, 150, 127),
    ("tiles", 2, 1, 128, 100, 150, 149), ("shares", 4, 2, 64, 4000, 200, 7),
]


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("what,kernel,Hq,Hkv,D,cached,new,row", [("query", *c) for c in INFINITE] +
                         [("keys", *c) for c in INFINITE if c[4] + c[5] < PAGE])   # (a page's scale makes NaN of them)
def test_a_row_whose_scores_are_all_minus_infinity(what, kernel, Hq, Hkv, D, cached, new, row, sign):
    """An infinite query where every key has the other sign, or keys of a tail: there is no softmax, and the row is NaN, not
    the zero of a row that sees nothing; no other row changes."""
    out = []
    for value in (None, -sign * np.inf):
        sv = Server(1, Hq, Hkv, D, (cached + new) // PAGE + 2, seed=D + cached)
        (q0, k0, v0), (q1, k1, v1) = sv.draw([cached]), sv.draw([new])
        for k in (k0, k1):
            k[:, 0, 7] = sign * (0.5 + np.abs(k[:, 0, 7]))           # kv head 0: one sign in dimension 7
        q1[:, 0, 7] = sign * (0.5 + np.abs(q1[:, 0, 7]))
        if value is not None:
            if what == "query":
                q1[row, 0, 7] = value
            else:
                k0[:, 0, 7] = k1[:, 0, 7] = value
        if cached:
            sv.step([cached], rope=False, data=(q0, k0, v0))
        b, Q, _ = sv.step([new], rope=False, data=(q1, k1, v1))
        assert kernel_of(sv.cache, b, Hq) == kernel
        out.append(glowq.kv_attention(sv.cache, b, Q, workspace=sv.ws).cpu().numpy().reshape(new, Hq, D))
        assert int(sv.ws[:65536].max()) == 0
    clean, got = out
    hit = np.zeros((new, Hq), bool)
    hit[row, 0] = True
    if what == "keys":
        hit[:, 0] = True
        clean, got = clean[:, Hq // Hkv:], got[:, Hq // Hkv:]        # (the group's other queries have either sign)
        assert np.isnan(out[1][hit]).all()
        assert np.array_equal(got, clean)
        return
    assert np.isnan(got[hit]).all()
    assert np.isfinite(got[~hit]).all() and np.array_equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("code", [121, 100, 60, 0, -5, -20])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_a_tail_have_22_bits(D, code):
    """Two tokens of nearly equal weight and opposite values beside a heavier one, all in a decoding sequence's tail: what is
    left shows the weights themselves.  Sums of D equal fp16 numbers are exact, so the scores are."""
    sv = Server(1, 2, 2, D, 2, seed=5)
    k = np.full((40, 2, D), -1.0, np.float16)
    v = np.zeros((40, 2, D), np.float16)
    k[3] = 1.0
    k[10] = k[20] = np.float16(code / 127)
    k[20, :, 5] = np.float16((code - 1) / 127)
    v[10], v[20] = 1.0, -1.0
    q = np.ones((40, 2, D), np.float16)
    sv.step([39], rope=False, data=(q[:39], k[:39], v[:39]))
    b, Q, qr = sv.step([1], rope=False, data=(q[39:], k[39:], v[39:]))
    assert kernel_of(sv.cache, b, 2) == "pages"
    got = glowq.kv_attention(sv.cache, b, Q, workspace=sv.ws).cpu().numpy().reshape(2, D).astype(np.float64)
    kk, vv = sv.seq[0].held()
    s = kk[:, 0] @ np.ones(D) * D ** -0.5
    p = np.exp(s - s.max())
    y = p @ vv[:, 0, 0] / p.sum()
    # the exponent in log2 units: four roundings of the score, the values' power of two added (2^15 at most), the distance
    # to the largest; 2^x itself 2^-22; a weight 2^-23 of itself and 2^-32 of the largest; then the output's rounding
    u24 = 2.0 ** -24
    x = np.abs(s) * np.log2(np.e)
    rel = np.log(2) * u24 * (6 * (x + x.max()) + 15 + 24) + 2.0 ** -22 + 2.0 ** -23
    b1 = (p[[10, 20]] @ rel[[10, 20]] + 2 * 2.0 ** -32) / p.sum() + 80 * 2 * u24 * abs(y)
    assert abs(y) < 0.01 and np.abs(got - y).max() <= b1 + 2.0 ** -11 * (abs(y) + b1) + 2.0 ** -25


def fixed_point(q, k, v, start, scale):
    """What the weights' fixed point adds to plain8.attention's bound where a sequence has few new tokens: of a complete page
    each weight is off by 2^-23 of the largest of its row and page."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.zeros((n, Hq, D))
    full = len(k) // PAGE * PAGE                                     # (what is behind is in the tail)
    for i in range(n):
        m = min(len(k), start + i + 1)
        for h in range(Hq):
            if m <= 0:
                continue
            s = k[:m, h // G] @ q[i, h].astype(np.float64) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            for p in range(0, min(m, full), PAGE):
                out[i, h] += 2.0 ** -23 * w[p:p + PAGE].max() * np.abs(v[p:min(p + PAGE, m), h // G]).sum(0)
    return out


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("Hq,Hkv,D,cached,new,scale,spread", [
    (3, 3, 128, [100], [63], None, 30.0), (24, 3, 128, [28, 46, 61], [2, 1, 3], 0.5, 1.0), (28, 4, 64, [65, 100], [3, 2], None, 30.0),
    (2, 1, 64, [6], [61], 0.5, 1.0), (4, 2, 64, [900, 700], [1, 3], 2.0, 5.0),
])
def test_one_token_far_ahead_of_the_others(Hq, Hkv, D, cached, new, scale, spread, seed):
    """Rows whose largest weight is 10^5 and more times the next, with values that are zero there: what is left is the small
    weights' share."""
    sv = Server(len(new), Hq, Hkv, D, 17, seed=seed, spread=spread)
    if any(cached):
        sv.step(cached)
    b, Q, qr = sv.step(new)
    assert kernel_of(sv.cache, b, Hq) == "pages"
    got = glowq.kv_attention(sv.cache, b, Q, scale=scale, workspace=sv.ws).cpu().numpy().reshape(-1, Hq, D)
    scale, at = D ** -0.5 if scale is None else scale, 0
    for s, n in zip(sv.seq, new):
        k, v = s.held()
        y, bound = plain8.attention(qr[at:at + n], k, v, len(k) - n, scale)
        bound = bound + fixed_point(qr[at:at + n], k, v, len(k) - n, scale)
        assert plain8.within(got[at:at + n], y, bound) <= 1.0
        at += n
