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


@pytest.mark.parametrize("T", [1, 16, 40, 333, 1500])
def test_product_stays_inside_its_scratch(T):
    """A workspace of exactly the bytes asked for, with a guard behind it."""
    import torch
    d, outs, r = 1152, [400, 256], 40
    mods, B, X = w8.make(T, d, outs, r, seed=T)
    n = glowq.w8a8_workspace_bytes(T, d, r, outs)
    buf = torch.full((n + 65536,), 201, dtype=torch.uint8, device="cuda")
    buf[:HEAD] = 0
    Ys, R = glowq.group_forward_w8a8(w8.dev_mods(mods), cuda(B), cuda(X), workspace=buf[:n])
    w8.check(Ys, R, *plain8.w8a8(X, mods, B))
    assert bool((buf[n:] == 201).all()) and int(buf[:HEAD].max()) == 0


@pytest.mark.parametrize("kernel,Hq,Hkv,D,cached,new", KERNELS)
def test_attention_stays_inside_its_scratch(kernel, Hq, Hkv, D, cached, new):
    import torch
    sv = Server(len(new), Hq, Hkv, D, (max(cached) + max(new)) // PAGE + 2, seed=D)
    sv.step(cached)
    b, Q, qr = sv.step(new)
    n = glowq.kv_attention_workspace(sv.cache, b, Hq).numel()
    buf = torch.full((n + 65536,), 201, dtype=torch.uint8, device="cuda")
    buf[:HEAD] = 0
    sv.ws = buf[:n]
    sv.check_attention(b, Q, qr, new)
    assert bool((buf[n:] == 201).all())


# ------------------------------------------------- special values, few rows ----

def without(q, k, v, start, scale, pos):
    """plain8.attention as if position pos (before every row) were not there."""
    return plain8.attention(q, np.delete(k, pos, 0), np.delete(v, pos, 0), start - 1, scale)


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("where", ["k page", "v page", "k tail", "v tail", "q"])
@pytest.mark.parametrize("Hq,D,cached,new", [(4, 128, [150, 100], [1, 2]), (2, 64, [9000, 200], [1, 3]), (6, 64, [9000, 0], [4, 1])])
def test_values_that_are_not_finite_in_decode(Hq, D, cached, new, where, value):
    """NaN for the rows that see them (a tail's key whose score is -infinity: no weight), in units that one block takes and
    in units cut into parts; every other row and head as without them."""
    at = {"k page": 70, "v page": 70, "k tail": cached[0] - 3, "v tail": cached[0] - 3}.get(where)
    out = []
    for hit in (False, True):
        sv = Server(2, Hq, 2, D, max(cached) // PAGE + 2, seed=D)
        old, step = sv.draw(cached), sv.draw(new)
        if hit and where == "q":
            step[0][0, Hq // 2, 7] = value
        elif hit:
            old[1 if where[0] == "k" else 2][at, 1, 7] = value       # kv head 1
        sv.step(cached, rope=False, data=old)
        b, Q, qr = sv.step(new, rope=False, data=step)
        assert kernel_of(sv.cache, b, Hq) == "pages"
        out.append(glowq.kv_attention(sv.cache, b, Q, workspace=sv.ws).cpu().numpy().reshape(-1, Hq, D))
        assert int(sv.ws[:HEAD].max()) == 0
    clean, got = out
    rows = np.zeros(got.shape[:2], bool)
    if where == "q":
        rows[0, Hq // 2] = True
    else:
        rows[:new[0], Hq // 2:] = True
    assert np.array_equal(got[~rows], clean[~rows]) and np.isfinite(got[~rows]).all()
    if where == "k tail" and np.isinf(value):
        lost = rows[:new[0]] & (qr[:new[0], :, 7] * value < 0)       # a score of -infinity
        k, v = sv.seq[0].held()
        y, bound = without(qr[:new[0]], np.where(np.isfinite(k), k, 0), v, len(k) - new[0], D ** -0.5, at)
        assert plain8.within(got[:new[0]][lost], y[lost], bound[lost]) <= 1.0
        rows[:new[0]] &= ~lost
    assert np.isnan(got[rows]).all()


@pytest.mark.parametrize("size", [1e-4, 6e-8, 30000.0])
def test_small_and_large_values_in_decode(size):
    sv = Server(2, 4, 2, 64, 40, seed=1)
    for new in ([2000, 100], [1, 2]):
        q, k, v = sv.draw(new)
        v = (v.astype(np.float32) * np.float32(size)).clip(-60000, 60000).astype(np.float16)
        b, Q, qr = sv.step(new, data=(q, k, v))
    assert kernel_of(sv.cache, b, 4) == "pages"
    sv.check_held(b)
    sv.check_attention(b, Q, qr, new)


def test_zero_pages_and_rows_that_see_nothing_in_decode():
    sv = Server(2, 4, 2, 128, 5, seed=2)
    q, k, v = sv.draw([250, 70])
    k[:64] = 0
    v[64:128] = 0
    v[250:] = 0
    sv.step([250, 70], data=(q, k, v), rope=False)
    b, Q, qr = sv.step([3, 2], rope=False)
    assert kernel_of(sv.cache, b, 4) == "pages"
    sv.check_attention(b, Q, qr, [3, 2])
    for lens in ([1, 0], [66, 1], [64, 2]):
        b = sv.batch([3, 2], lens=lens)
        before = [(s.k, s.v) for s in sv.seq]
        for s, n in zip(sv.seq, lens):           # what a cache of this length holds: pages, and the tail's slots
            t = n // PAGE * PAGE
            tail = (len(s.k) - 1) // PAGE * PAGE
            s.k, s.v = (np.concatenate([x[:t], x[tail:tail + n - t]]) for x in (s.k, s.v))
        got = sv.check_attention(b, Q, qr, [3, 2], lens=lens)
        for i, n in ((0, 3 - lens[0]), (3, 2 - lens[1])):
            assert n <= 0 or (got[i:i + n, :-8] == 0).all()
        for s, (k, v) in zip(sv.seq, before):
            s.k, s.v = k, v


@pytest.mark.parametrize("code", [121, 100, 60, 0, -5, -20])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_pages_have_24_bits(D, code):
    """Two tokens of nearly equal weight and opposite values in a page whose largest weight is another's: what is left shows
    the weights themselves.  The scores' integer sums are exact, and so are the queries in fixed point here."""
    sv = Server(1, 2, 2, D, 3, seed=5)
    k = np.full((65, 2, D), -1.0, np.float16)
    v = np.zeros((65, 2, D), np.float16)
    k[3] = 1.0                                               # the page's scale is 1/127, codes -127 .. 127
    k[10] = k[20] = np.float16(code / 127)
    k[20, :, 5] = np.float16((code - 1) / 127)
    v[10], v[20] = 1.0, -1.0
    q = np.ones((65, 2, D), np.float16)
    sv.step([64], rope=False, data=(q[:64], k[:64], v[:64]))
    b, Q, qr = sv.step([1], rope=False, data=(q[64:], k[64:], v[64:]))
    assert kernel_of(sv.cache, b, 2) == "pages"
    got = glowq.kv_attention(sv.cache, b, Q, workspace=sv.ws).cpu().numpy().reshape(2, D).astype(np.float64)
    kk, vv = sv.seq[0].held()
    s = kk[:, 0] @ np.ones(D) * D ** -0.5
    p = np.exp(s - s.max())
    y = p @ vv[:, 0, 0] / p.sum()
    # the exponent in log2 units: five roundings of the score, the value scale's logarithm added (log2 127 < 7), the
    # distance to the largest; 2^x itself 2^-22; a weight 2^-24 of the page's largest; then the output's rounding
    u24 = 2.0 ** -24
    x = np.abs(s) * np.log2(np.e)
    rel = np.log(2) * u24 * (8 * (x + x.max()) + 7 + 24) + 2.0 ** -22
    b1 = (p[[10, 20]] @ rel[[10, 20]] + 2 * u24) / p.sum() + 80 * 2 * u24 * abs(y)
    assert abs(y) < 0.01 and np.abs(got - y).max() <= b1 + 2.0 ** -11 * (abs(y) + b1) + 2.0 ** -25


# ------------------------------------------------------------- as it is used ----

@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (8, 1, 64)])
def test_a_captured_step_whose_lengths_grow(Hq, Hkv, D):
    """One graph of append and attention, replayed for every token: lengths on the device, past page borders."""
    import torch
    sv = Server(3, Hq, Hkv, D, 40, seed=D)
    sv.step([60, 2000, 1])
    qkv = [torch.zeros((3, h * D), dtype=torch.float16, device="cuda") for h in (Hq, Hkv, Hkv)]
    kv_len = cuda(np.array([60, 2000, 1], np.int32))
    b = glowq.KVBatch(cuda(np.arange(4, dtype=np.int32)), kv_len, cuda(sv.pages), cuda(sv.slot), 3, 1)
    rot = torch.empty_like(qkv[0])
    append = glowq.KVAppendPlan(sv.cache, b, qkv[1], qkv[2], Q=qkv[0], Q_out=rot, rope=sv.rope_dev)
    attend = glowq.KVAttentionPlan(sv.cache, b, rot)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv_len.add_(1)
        append()
        attend()
    for i in range(140):
        q, k, v = sv.draw([1, 1, 1])
        for t, x in zip(qkv, (q, k, v)):
            t.copy_(cuda(x.reshape(3, -1)))
        qr = np.empty_like(q)
        for j, s in enumerate(sv.seq):
            cs = sv.rope[len(s.k):len(s.k) + 1]
            s.append(plain8.rotate(k[j:j + 1], cs), v[j:j + 1])
            qr[j:j + 1] = plain8.rotate(q[j:j + 1], cs)
        g.replay()
        if i % 9 == 0 or any(len(s.k) % PAGE in (0, 1) for s in sv.seq):
            got = attend.outputs.cpu().numpy().reshape(3, Hq, D)
            for j, s in enumerate(sv.seq):
                y, bound = plain8.attention(qr[j:j + 1], *s.held(), len(s.k) - 1, D ** -0.5)
                assert plain8.within(got[j:j + 1], y, bound) <= 1.0, (i, j)
    sv.check_held(b)


def test_sequences_that_share_a_prefix():
    """Complete pages of one sequence in the tables of others, which go on from there."""
    sv = Server(3, 4, 2, 64, 5, seed=4)
    sv.step([128, 0, 0])
    sv.pages[1, :2], sv.pages[2, :1] = sv.pages[0, :2], sv.pages[0, :1]
    for i, n in ((1, 128), (2, 64)):
        sv.seq[i].k, sv.seq[i].v = sv.seq[0].k[:n], sv.seq[0].v[:n]
    for new in ([1, 3, 70], [60, 62, 1], [1, 1, 1]):
        b, Q, qr = sv.step(new)
        sv.check_held(b)
        sv.check_attention(b, Q, qr, new)


@pytest.mark.parametrize("kernels,Hq,Hkv,D,cols,cached,new", [
    (("tiles", "shares"), 8, 2, 64, 24, [1200, 3, 64, 700, 90, 1, 500, 127], [1, 1, 1, 1, 1, 300, 1, 1]),
    (("tiles", "shares"), 8, 2, 128, 600, [900, 30], [1, 200]), (("pages",), 4, 2, 64, 600, [700, 5, 64], [1, 1, 1]),
    (("tiles", "shares"), 2, 1, 64, 2048, [0], [500]),
])
def test_mixed_steps_and_wide_tables(kernels, Hq, Hkv, D, cols, cached, new):
    """Decoding sequences beside a prompt's chunk, and tables far wider than the lengths."""
    sv = Server(len(new), Hq, Hkv, D, cols, seed=cols)
    if any(cached):
        sv.step(cached)
    b, Q, qr = sv.step(new)
    assert kernel_of(sv.cache, b, Hq) in kernels
    sv.ws = glowq.kv_attention_workspace(sv.cache, b, Hq)
    first = sv.check_attention(b, Q, qr, new)
    assert np.array_equal(first, sv.check_attention(b, Q, qr, new))


@pytest.mark.parametrize("Hq,Hkv,D,cached,new", [
    (64, 1, 128, [700, 64], [1, 1]), (128, 1, 64, [100], [1]), (96, 1, 128, [300], [2]), (40, 8, 64, [65, 0], [1, 30]), (65, 1, 64, [10], [70])])
def test_many_query_heads_of_one_kv_head(Hq, Hkv, D, cached, new):
    sv = Server(len(new), Hq, Hkv, D, (max(cached) + max(new)) // PAGE + 1, seed=Hq)
    sv.step(cached)
    b, Q, qr = sv.step(new)
    sv.check_attention(b, Q, qr, new)


def test_more_blocks_of_rows_than_are_sorted():
    """Hundreds of prompts of some rows each: more (row tile, sequence) pairs than the many-row kernel sorts."""
    g = np.random.default_rng(6)
    n = 270
    sv = Server(n, 4, 1, 64, 4, seed=6)
    sv.step([int(x) for x in g.integers(0, 90, n)])
    new = [int(x) for x in g.choice([0, 1, 20, 33, 70], n)]
    b, Q, qr = sv.step(new)
    assert kernel_of(sv.cache, b, 4) in ("tiles", "shares")
    sv.ws = glowq.kv_attention_workspace(sv.cache, b, 4)
    sv.check_attention(b, Q, qr, new)


def test_pools_of_more_than_32_bits():
    """Pages and tails whose offsets pass 2^31 elements, and 2^32 bytes."""
    import torch
    pages, slots = 36000, 36000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    sv = Server(3, 8, 8, 128, 9, seed=7)
    sv.cache = glowq.KVCache.alloc(pages, slots, 8, 128)
    sv.pages = pages - 1 - sv.g.permutation(27).reshape(3, 9).astype(np.int32)
    sv.slot = np.array([slots - 1, 0, slots - 20], np.int32)
    for new in ([300, 64, 130], [1, 1, 1], [60, 200, 2]):
        b, Q, qr = sv.step(new)
        sv.check_held(b)
        sv.check_attention(b, Q, qr, new)


@pytest.mark.parametrize("T", [1, 12, 40, 200])
def test_weights_of_more_than_32_bits(T):
    """Codes whose offsets pass 2^31: the last rows against the plain product, the zero rows between exactly zero."""
    import torch
    O, d = 264192, 8192
    mods, B, X = w8.make(T, d, [64, 64], 8, seed=T)
    codes = torch.zeros((O, d), dtype=torch.int8, device="cuda")
    scales = torch.ones(O, device="cuda")
    for at, (q, s, _) in ((0, mods[0]), (O - 64, mods[1])):
        codes[at:at + 64] = cuda(q)
        scales[at:at + 64] = cuda(s)
    Ys, _ = glowq.group_forward_w8a8([glowq.Int8Module(codes, scales)], None, cuda(X))
    refs, _ = plain8.w8a8(X, [(q, s, None) for q, s, _ in mods], None)
    w8.check([Ys[0][:, :64], Ys[0][:, O - 64:]], None, refs, (None, None))
    assert float(Ys[0][:, 64:O - 64].abs().max()) == 0.0


@pytest.mark.parametrize("Ts", [(1, 1), (1, 300), (40, 40), (300, 1500), (16, 17)])
def test_products_on_two_streams(Ts):
    """Two plans at once, each with its own scratch: the bits of one after the other."""
    import torch
    plans, want = [], []
    for i, T in enumerate(Ts):
        mods, B, X = w8.make(T, 2048, [1024, 512], 64, seed=i)
        plans.append(glowq.Int8ForwardPlan(w8.dev_mods(mods), cuda(B), cuda(X)))
        plans[-1]()
        w8.check(plans[-1].outputs, plans[-1].R, *plain8.w8a8(X, mods, B))
        want.append([y.clone() for y in plans[-1].outputs])
    streams = [torch.cuda.Stream() for _ in Ts]
    for _ in range(30):
        for p in plans:
            for y in p.outputs:
                y.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            for p, s in zip(plans, streams):
                p(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(y, x) for p, w in zip(plans, want) for y, x in zip(p.outputs, w))


def test_empty_batches():
    import torch
    cache = glowq.KVCache.alloc(2, 1, 2, 64)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    f16 = lambda *s: torch.empty(*s, dtype=torch.float16, device="cuda")
    for b in (glowq.KVBatch(i32(0), i32(), i32().reshape(0, 1), i32(), 0, 0), glowq.KVBatch(i32(0, 0), i32(0), i32(0).reshape(1, 1), i32(0), 0, 1),
              glowq.KVBatch(i32(0, 0), i32(0), i32(0).reshape(1, 1), i32(0), 4, 2)):
        Q = glowq.kv_append(cache, b, f16(b.rows, 128), f16(b.rows, 128), Q=f16(b.rows, 256))
        assert glowq.kv_attention(cache, b, Q).shape == (b.rows, 256)
        assert all(float(x.abs().sum()) == 0 for x in glowq.kv_read(cache, b, 3))
    mods, B, X = w8.make(0, 256, [32, 16], 8, seed=0)
    Ys, R = glowq.group_forward_w8a8(w8.dev_mods(mods), cuda(B), cuda(X))
    assert [tuple(y.shape) for y in (*Ys, R)] == [(0, 32), (0, 16), (0, 8)]
    assert glowq.solo_forward_w8a8(w8.dev_mods(mods)[0], cuda(B), cuda(X)).shape == (0, 32)


@pytest.mark.parametrize("T", [9, 16])
def test_more_tiles_than_the_scratch_counts(T):
    """Few tokens, whose activations need k in shares, and more tiles than the head has tickets for: left to the tensor-core
    product."""
    import torch
    O, d = 140032, 16384
    mods, B, X = w8.make(T, d, [48, 64], 0, seed=T)
    codes = torch.zeros((O, d), dtype=torch.int8, device="cuda")
    scales = torch.ones(O, device="cuda")
    for at, (q, s, _) in ((0, mods[0]), (O - 64, mods[1])):
        codes[at:at + len(q)] = cuda(q)
        scales[at:at + len(q)] = cuda(s)
    Y = glowq.solo_forward_w8a8(glowq.Int8Module(codes, scales), None, cuda(X))
    w8.check([Y[:, :48], Y[:, O - 64:]], None, plain8.w8a8(X, mods, None)[0], (None, None))
    assert float(Y[:, 48:O - 64].abs().max()) == 0.0


def test_a_mixed_step_as_two_calls():
    """Decoding sequences and a prompt's chunk of one step, attended to by a call each over parts of the step's arrays: each
    by its own kernel, rows outside a call's sequences untouched."""
    import torch
    sv = Server(4, 8, 2, 128, 16, seed=9)
    sv.step([700, 64, 5, 300])
    new = [1, 1, 1, 400]
    b, Q, qr = sv.step(new)
    q_start, kv_len, table, slot = b._keep
    few = glowq.KVBatch(q_start[:4], kv_len[:3], table[:3], slot[:3], 3, 1)
    many = glowq.KVBatch(q_start[3:], kv_len[3:], table[3:], slot[3:], 403, 400)
    assert kernel_of(sv.cache, few, 8) == "pages" and kernel_of(sv.cache, many, 8) in ("tiles", "shares")
    Y = torch.full((403, 8 * 128), 3.0, dtype=torch.float16, device="cuda")
    glowq.kv_attention(sv.cache, many, Q, Y=Y)
    assert bool((Y[:3] == 3).all())
    chunk = Y[3:].clone()
    glowq.kv_attention(sv.cache, few, Q, Y=Y)
    assert torch.equal(Y[3:], chunk)
    got, at = Y.cpu().numpy().reshape(403, 8, 128), 0
    for s, n in zip(sv.seq, new):
        y, bound = plain8.attention(qr[at:at + n], *s.held(), len(s.k) - n, 128 ** -0.5)
        assert plain8.within(got[at:at + n], y, bound) <= 1.0
        at += n


def test_tokens_taken_back():
    """Lengths that go back inside the incomplete page, as after rejected draft tokens, and go on with other tokens."""
    sv = Server(2, 4, 2, 64, 4, seed=10)
    sv.step([100, 130])
    for draft, kept, new in (([4, 4], [101, 128], [2, 1]), ([9, 3], [105, 129], [60, 3])):
        sv.step(draft)
        for s, n in zip(sv.seq, kept):
            s.k, s.v = s.k[:n], s.v[:n]
        b, Q, qr = sv.step(new)
        sv.check_held(b)
        sv.check_attention(b, Q, qr, new)
