"""The paged 8-bit key/value cache: what append stores, bit by bit against the
definition, and attention over it element by element against the plain 64-bit
form; batches of uneven sequences, cut into steps in different ways."""
import numpy as np
import pytest

from rank_error_correction_b200 import build, glowq

import plain8

pytestmark = pytest.mark.gpu
PAGE, INDEX = 64, 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    glowq.lib()
    yield
    assert glowq.device_status() == 0


def cuda(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Server:
    """Sequences in a cache whose unused memory holds NaN and odd codes, and beside it their plain form."""

    def __init__(self, n, Hq, Hkv, D, cols, seed, theta=10000.0, spread=1.0):
        import torch
        self.n, self.Hq, self.Hkv, self.D, self.cols = n, Hq, Hkv, D, cols
        self.g = np.random.default_rng(seed)
        self.cache = glowq.KVCache.alloc(n * cols + 3, n + 2, Hkv, D)
        self.cache.k_codes.fill_(91)
        self.cache.v_codes.fill_(-77)
        for t in (self.cache.k_scales, self.cache.v_scales, self.cache.k_tail, self.cache.v_tail):
            t.fill_(float("nan"))
        self.pages = self.g.permutation(n * cols + 3)[: n * cols].reshape(n, cols).astype(np.int32)
        self.slot = self.g.permutation(n + 2)[:n].astype(np.int32)
        self.seq = [plain8.Sequence(Hkv, D) for _ in range(n)]
        self.rope = plain8.rope_table(cols * PAGE, D, theta)
        self.rope_dev = cuda(self.rope)
        self.spread = spread
        self.ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")

    def batch(self, new, pad=0, lens=None, pages=None, slot=None, max_new=None):
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        lens = [len(s.k) for s in self.seq] if lens is None else lens
        return glowq.KVBatch(cuda(starts), cuda(np.asarray(lens, np.int32)), cuda(self.pages if pages is None else pages),
                             cuda(self.slot if slot is None else slot), int(starts[-1]) + pad,
                             max(new, default=0) if max_new is None else max_new)

    def draw(self, new):
        T = sum(new)
        amp = self.spread ** self.g.uniform(-1, 1, (T, 1, 1))       # tokens of very different size
        k = (self.g.standard_normal((T, self.Hkv, self.D)) * amp).astype(np.float16)
        v = (self.g.standard_normal((T, self.Hkv, self.D)) * amp[::-1]).astype(np.float16)
        q = (self.g.standard_normal((T, self.Hq, self.D)) * 2).astype(np.float16)
        return q, k, v

    def step(self, new, pad=0, rope=True, data=None):
        """One append; returns (batch, rotated queries on the device, rotated queries)."""
        import torch
        q, k, v = self.draw(new) if data is None else data
        T = sum(new)
        width = (self.Hq + 2 * self.Hkv) * self.D
        buf = torch.full((T + pad, width + 16), float("nan"), dtype=torch.float16, device="cuda")
        buf[:T, :width] = cuda(np.concatenate([x.reshape(T, -1) for x in (q, k, v)], 1))
        Q, K, V = (buf[:, a:b] for a, b in ((0, self.Hq * self.D), (self.Hq * self.D, (self.Hq + self.Hkv) * self.D),
                                            ((self.Hq + self.Hkv) * self.D, width)))
        at, pos = 0, []
        for s, n in zip(self.seq, new):
            pos.append(np.arange(len(s.k), len(s.k) + n))
        pos = np.concatenate(pos) if pos else np.zeros(0, int)
        kr, qr = (plain8.rotate(k, self.rope[pos]), plain8.rotate(q, self.rope[pos])) if rope else (k, q)
        for s, n in zip(self.seq, new):
            s.append(kr[at:at + n], v[at:at + n])
            at += n
        b = self.batch(new, pad)
        out = torch.full((T + pad, self.Hq * self.D), 5.0, dtype=torch.float16, device="cuda")
        got = glowq.kv_append(self.cache, b, K, V, Q=Q, Q_out=out, rope=self.rope_dev if rope else None)
        assert got.data_ptr() == out.data_ptr()
        assert np.array_equal(out[:T].cpu().numpy().reshape(q.shape), qr, equal_nan=True)
        assert bool((out[T:] == 5).all())
        return b, out, qr

    def check_held(self, b):
        """Everything that the cache holds, by position."""
        most = max(len(s.k) for s in self.seq) + 5
        K, V = (t.cpu().numpy().reshape(self.n, most, self.Hkv, self.D) for t in glowq.kv_read(self.cache, b, most))
        first = np.array([max(0, len(s.k) - 70) for s in self.seq], np.int32)
        K2, V2 = (t.cpu().numpy().reshape(self.n, 80, self.Hkv, self.D)
                  for t in glowq.kv_read(self.cache, b, 80, first=cuda(first)))
        with np.errstate(over="ignore", invalid="ignore"):
            for i, s in enumerate(self.seq):
                for got, part, want in zip((K, V), (K2, V2), s.held()):
                    # the product code x scale is rounded to fp32 and then to fp16
                    w = np.zeros((most + 80, self.Hkv, self.D), np.float16)
                    w[:len(want)] = want.astype(np.float32).astype(np.float16)
                    assert np.array_equal(got[i], w[:most], equal_nan=True)
                    assert np.array_equal(part[i], w[first[i]:first[i] + 80], equal_nan=True)

    def check_attention(self, b, Q, qr, new, scale=None, lens=None):
        import torch
        rows = Q.shape[0]
        Y = torch.full((rows, self.Hq * self.D + 8), 3.0, dtype=torch.float16, device="cuda")
        glowq.kv_attention(self.cache, b, Q, scale=scale, Y=Y[:, :-8], workspace=self.ws)
        got = Y.cpu().numpy()
        scale = self.D ** -0.5 if scale is None else scale
        T = sum(new)
        assert (got[T:] == 3).all() and (got[:, -8:] == 3).all()
        at, worst = 0, 0.0
        for i, (s, n) in enumerate(zip(self.seq, new)):
            L = len(s.k) if lens is None else lens[i]
            k, v = s.held()
            y, bound = plain8.attention(qr[at:at + n], k[:L], v[:L], L - n, scale)
            worst = max(worst, plain8.within(got[at:at + n, :-8].reshape(n, self.Hq, self.D), y, bound))
            at += n
        assert worst <= 1.0, worst
        assert int(self.ws[:65536].max()) == 0
        return got[:T]


HEADS = [(4, 4, 128), (8, 2, 128), (8, 1, 64), (6, 2, 64), (3, 1, 128), (32, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_steps_of_uneven_sequences(Hq, Hkv, D):
    """Prompts, then single tokens across page borders, then a few tokens at once; sequences of no new tokens, a
    padded batch; after every step the cache bit by bit and the attention over it."""
    sv = Server(5, Hq, Hkv, D, 5, seed=Hq + D)
    for new, pad in [([1, 63, 64, 65, 0], 0), ([1, 1, 1, 1, 1], 3), ([0, 1, 0, 62, 127], 1), ([1, 1, 0, 1, 1], 0),
                     ([5, 3, 2, 4, 1], 7), ([130, 2, 64, 1, 0], 0)]:
        b, Q, qr = sv.step(new, pad)
        sv.check_held(b)
        sv.check_attention(b, Q, qr, new)


@pytest.mark.parametrize("cuts", [[200], [64, 64, 72], [1] * 200, [37, 100, 63], [63, 2, 63, 2, 70]])
def test_the_cut_into_steps_does_not_matter(cuts):
    """The same tokens in other steps: the same codes, scales and tails, bit by bit."""
    import torch
    whole, parts = Server(1, 2, 2, 128, 4, seed=3), Server(1, 2, 2, 128, 4, seed=3)
    q, k, v = whole.draw([200])
    b1, _, _ = whole.step([200], data=(q, k, v))
    at = 0
    for n in cuts:
        b2, _, _ = parts.step([n], data=(q[at:at + n], k[at:at + n], v[at:at + n]))
        at += n
    parts.check_held(b2)
    for x, y in ((whole.cache.k_codes, parts.cache.k_codes), (whole.cache.v_codes, parts.cache.v_codes),
                 (whole.cache.k_scales, parts.cache.k_scales), (whole.cache.v_scales, parts.cache.v_scales)):
        ids = torch.from_numpy(whole.pages[0, :3].astype(np.int64)).cuda()
        assert bool((x[ids] == y[ids]).all())


@pytest.mark.parametrize("Hq,Hkv,D,cached,new", [
    (4, 4, 128, [1500, 0, 700], [1, 1, 1]), (8, 2, 128, [2000, 1], [1, 1]), (8, 8, 64, [3000], [1]),
    (4, 2, 128, [300], [200]), (2, 2, 64, [0, 513], [300, 90]), (8, 1, 128, [100, 64, 0], [33, 64, 129]),
    (16, 1, 128, [1000], [1]), (5, 1, 64, [127, 128], [3, 3]),
])
def test_longer_caches(Hq, Hkv, D, cached, new):
    sv = Server(len(new), Hq, Hkv, D, (max(cached) + max(new)) // PAGE + 2, seed=sum(cached) + D)
    if any(cached):
        sv.step(cached)
    b, Q, qr = sv.step(new)
    sv.check_held(b)
    first = sv.check_attention(b, Q, qr, new)
    assert np.array_equal(first, sv.check_attention(b, Q, qr, new))          # the same bits again


@pytest.mark.parametrize("Hq,Hkv,D,cached,new", [
    (8, 1, 128, [1500], [16]), (8, 1, 64, [2000, 0, 900], [9, 30, 70]), (4, 2, 128, [4000, 3000], [33, 1]),
])
def test_many_rows_over_long_tables(Hq, Hkv, D, cached, new):
    """Enough rows for matrix tiles, but too few blocks of them: pages are shared instead."""
    test_longer_caches(Hq, Hkv, D, cached, new)


@pytest.mark.parametrize("Hq,Hkv,D,cached,new", [
    (8, 2, 128, [5000, 10, 2600], [70, 129, 1]), (2, 2, 64, [0], [1500]), (4, 1, 128, [9000], [65]), (8, 1, 64, [3000, 2999], [100, 100]),
])
def test_matrix_tiles_in_shares(Hq, Hkv, D, cached, new):
    """Few blocks of many rows: their tokens in shares, some of which the first rows do not see."""
    test_longer_caches(Hq, Hkv, D, cached, new)


def test_hundreds_of_uneven_sequences():
    """More sequences than a block has threads, many of a page or less, some without new tokens."""
    g = np.random.default_rng(11)
    n = 300
    sv = Server(n, 6, 2, 64, 6, seed=11)
    sv.step([int(x) for x in g.choice([0, 1, 40, 63, 64, 65, 128, 200, 320], n)])
    for new in ([1] * n, [int(x) for x in g.integers(0, 3, n)], [int(i == 299) for i in range(n)]):
        b, Q, qr = sv.step(new)
        first = sv.check_attention(b, Q, qr, new)
        assert np.array_equal(first, sv.check_attention(b, Q, qr, new))


def test_one_sequence_in_the_most_parts():
    sv = Server(1, 2, 1, 64, 1880, seed=12)
    sv.step([120000])
    b, Q, qr = sv.step([1])
    sv.check_attention(b, Q, qr, [1])
    b, Q, qr = sv.step([6])
    sv.check_attention(b, Q, qr, [6])


@pytest.mark.parametrize("Hq,Hkv,D,cached,new", [
    (4, 2, 64, [300], [700]), (4, 2, 128, [300], [700]), (8, 2, 64, [900, 30, 500], [1, 1, 1]),
    (8, 2, 128, [900, 30, 500], [1, 1, 1]), (8, 2, 64, [2000, 10], [70, 129]),
])
def test_the_same_bits_every_time(Hq, Hkv, D, cached, new):
    """Many calls, alone and two at once on two streams, each with its own workspace: no result depends on time."""
    import torch
    sv = Server(len(new), Hq, Hkv, D, (max(cached) + max(new)) // PAGE + 2, seed=D)
    sv.step(cached)
    b, Q, qr = sv.step(new)
    want = torch.from_numpy(sv.check_attention(b, Q, qr, new)[:, :-8].copy()).cuda()
    plans = [glowq.KVAttentionPlan(sv.cache, b, Q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(100):
        for p, s in zip(plans, streams):
            p.outputs.record_stream(s)
            p(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(p.outputs, want) for p in plans)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [64.0, 2000.0])
def test_scales_far_apart(D, spread):
    """Tokens, and so pages and tails, whose sizes differ by orders of magnitude; scores with hard maxima."""
    sv = Server(3, 4, 2, D, 6, seed=D, spread=spread)
    sv.step([200, 64, 301])
    b, Q, qr = sv.step([1, 3, 20])
    sv.check_held(b)
    sv.check_attention(b, Q, qr, [1, 3, 20])
    sv.check_attention(b, Q, qr, [1, 3, 20], scale=2.0)
    sv.check_attention(b, Q, qr, [1, 3, 20], scale=0.0)


@pytest.mark.parametrize("size", [1e-4, 6e-8, 30000.0])
def test_small_and_large_values(size):
    sv = Server(2, 2, 2, 64, 4, seed=1)
    q, k, v = sv.draw([150, 100])
    v = (v.astype(np.float32) * np.float32(size)).clip(-60000, 60000).astype(np.float16)
    b, Q, qr = sv.step([150, 100], data=(q, k, v))
    sv.check_held(b)
    sv.check_attention(b, Q, qr, [150, 100])


def test_zero_pages_and_no_rotation():
    sv = Server(2, 2, 2, 128, 4, seed=2)
    q, k, v = sv.draw([130, 64])
    k[:64] = 0
    v[64:128] = 0
    v[130:] = 0
    b, Q, qr = sv.step([130, 64], data=(q, k, v), rope=False)
    sv.check_held(b)
    sv.check_attention(b, Q, qr, [130, 64])


@pytest.mark.parametrize("where", ["k page", "v page", "k tail", "v tail", "q"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_values_that_are_not_finite(where, value):
    """NaN for the rows that see them, every other row as without them."""
    sv = Server(2, 2, 2, 128, 4, seed=4)
    q, k, v = sv.draw([150, 100])
    row = {"k page": 70, "v page": 70, "k tail": 140, "v tail": 140, "q": 145}[where]
    {"k": k, "v": v, "q": q}[where[0]][row, 1, 7] = value
    b, Q, qr = sv.step([150, 100], data=(q, k, v), rope=False)
    sv.check_held(b)
    Y = glowq.kv_attention(sv.cache, b, Q, workspace=sv.ws).cpu().numpy().reshape(250, 2, 128)
    hit = np.zeros((250, 2), bool)
    if where == "q":
        hit[145, 1] = True
    else:
        hit[(64 if "page" in where else 140):150, 1] = True      # a page's scale is shared by its tokens
    # a row of the hit head may be as it was where an infinite score of -inf gives its key no weight
    clean = ~hit
    assert np.isfinite(Y[clean]).all()
    if not (where == "k tail" and np.isinf(value)):
        assert np.isnan(Y[hit]).all()
    sv2 = Server(2, 2, 2, 128, 4, seed=4)
    q2, k2, v2 = sv2.draw([150, 100])
    b2, Q2, _ = sv2.step([150, 100], data=(q2, k2, v2), rope=False)
    Y2 = glowq.kv_attention(sv2.cache, b2, Q2, workspace=sv2.ws).cpu().numpy().reshape(250, 2, 128)
    assert np.array_equal(Y[clean], Y2[clean])


def test_rows_that_see_nothing_are_zero():
    """A cache shorter than the step's new tokens: the first rows are before position 0."""
    sv = Server(2, 4, 2, 64, 4, seed=5)
    sv.step([70, 30])
    new = [90, 40]
    q = (sv.g.standard_normal((130, 4, 64))).astype(np.float16)
    b = sv.batch(new, lens=[70, 0])
    got = sv.check_attention(b, cuda(q.reshape(130, -1)), q, new, lens=[70, 0])
    assert (got[:20, :-8] == 0).all() and (got[90:, :-8] == 0).all()


def test_data_out_of_range():
    """Bad pages, slots, lengths and rows: reported, nothing outside written, the other sequences as they should be."""
    import torch
    sv = Server(3, 2, 2, 64, 4, seed=6)
    sv.step([130, 100, 60])
    new = [1, 1, 1]
    b, Q, qr = sv.step(new)
    good = sv.check_attention(b, Q, qr, new)
    for field, value in [("pages", 10 ** 6), ("pages", -1), ("slot", 99), ("slot", -3), ("lens", 10 ** 6), ("lens", -5)]:
        pages, slot, lens = sv.pages.copy(), sv.slot.copy(), [len(s.k) for s in sv.seq]
        if field == "pages":
            pages[0, 1] = value
        elif field == "slot":
            slot[0] = value
        else:
            lens[0] = value
        bad = sv.batch(new, pages=pages, slot=slot, lens=lens)
        Y = glowq.kv_attention(sv.cache, bad, Q, workspace=sv.ws)
        assert glowq.device_status() == INDEX and glowq.device_status() == 0
        assert np.array_equal(Y.cpu().numpy()[1:], good[1:, :-8])
        assert field == "lens" or field == "pages" or (Y[0] == 0).all()
        K, V = glowq.kv_read(sv.cache, bad, 140)
        assert glowq.device_status() == INDEX
        assert np.array_equal(K[1].cpu().numpy().reshape(140, 2, 64)[:101], sv.seq[1].held()[0].astype(np.float32).astype(np.float16))
        # append: the tokens of sequence 0 complete its page (or not); no write may land outside its own memory
        before = [t.clone() for t in (sv.cache.k_codes, sv.cache.v_codes)]
        kv = torch.zeros((3, 2 * 64), dtype=torch.float16, device="cuda")
        lens2 = [192 if field == "pages" and value else lens[0], 101, 61]
        if field == "pages":
            pages[0, 2] = value
            lens2[0] = 192
        glowq.kv_append(sv.cache, sv.batch(new, pages=pages, slot=slot, lens=lens2), kv, kv, rope=sv.rope_dev)
        assert glowq.device_status() == INDEX
        assert all(bool((x == y).all()) for x, y in zip(before, (sv.cache.k_codes, sv.cache.v_codes)))
        # put back the values that the zero rows overwrote in the other sequences' tails
        for i in (1, 2):
            n = len(sv.seq[i].k)
            sv.cache.k_tail[int(sv.slot[i]), :, (n - 1) % PAGE] = cuda(sv.seq[i].k[n - 1])
            sv.cache.v_tail[int(sv.slot[i]), :, (n - 1) % PAGE] = cuda(sv.seq[i].v[n - 1])
    # more new tokens than max_new, rows outside the batch: the sequence is skipped, its rows stay
    for b2 in (sv.batch([2, 1, 1], max_new=1),
               glowq.KVBatch(cuda(np.array([0, 1, 2, 9], np.int32)), cuda(np.array([131, 101, 61], np.int32)), cuda(sv.pages), cuda(sv.slot), 4, 9),
               glowq.KVBatch(cuda(np.array([-1, 1, 2, 3], np.int32)), cuda(np.array([131, 101, 61], np.int32)), cuda(sv.pages), cuda(sv.slot), 4, 9)):
        Y = torch.full((4, 2 * 64), 3.0, dtype=torch.float16, device="cuda")
        glowq.kv_attention(sv.cache, b2, torch.zeros_like(Y), Y=Y, workspace=torch.zeros(1 << 22, dtype=torch.uint8, device="cuda"))
        assert glowq.device_status() == INDEX
        assert int((Y == 3).all(1).sum()) >= 1
    # a position that the rotation's table does not have
    kv = torch.zeros((3, 2 * 64), dtype=torch.float16, device="cuda")
    before = sv.cache.k_tail.clone()
    glowq.kv_append(sv.cache, b, kv, kv, rope=sv.rope_dev[:61].contiguous())
    assert glowq.device_status() == INDEX
    for i in (0, 1):
        assert torch.equal(before[int(sv.slot[i])].nan_to_num(7), sv.cache.k_tail[int(sv.slot[i])].nan_to_num(7))


def test_in_place_rotation_streams_and_graphs():
    import torch
    sv = Server(2, 4, 2, 128, 4, seed=7)
    sv.step([100, 20])
    q, k, v = sv.draw([1, 1])
    for s, i in zip(sv.seq, range(2)):
        pos = len(s.k)
        s.append(plain8.rotate(k[i:i + 1], sv.rope[pos:pos + 1]), v[i:i + 1])
    qr = np.concatenate([plain8.rotate(q[i:i + 1], sv.rope[len(sv.seq[i].k) - 1:len(sv.seq[i].k)]) for i in range(2)])
    b = sv.batch([1, 1])
    Qin, K, V = (cuda(x.reshape(2, -1)) for x in (q, k, v))
    Q = Qin.clone()
    append = glowq.KVAppendPlan(sv.cache, b, K, V, Q=Q, Q_out=Q, rope=sv.rope_dev)
    attend = glowq.KVAttentionPlan(sv.cache, b, Q, workspace=sv.ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    append(stream=s)
    attend(stream=s)
    s.synchronize()
    assert np.array_equal(Q.cpu().numpy().reshape(qr.shape), qr)
    want = sv.check_attention(b, Q, qr, [1, 1])[:, :-8]
    assert np.array_equal(attend.outputs.cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.copy_(Qin)
        append()
        attend()
    for _ in range(3):
        attend.outputs.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(attend.outputs.cpu().numpy(), want)
    sv.check_held(b)


def test_one_workspace_for_every_call_and_a_graph():
    """8-bit products of all token counts and attention of few and of many rows, whole and in shares, one after another on
    the same workspace, alone and in a graph: the same bits, and its head left zero."""
    import torch
    import test_gpu_w8a8 as w
    sv = Server(2, 8, 2, 64, 40, seed=13)
    sv.step([2000, 10])
    ws, calls = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda"), []
    many, Qm, qm = sv.step([70, 129])
    few, Qf, qf = sv.step([1, 1])
    lens = [[2070, 139], [2071, 140]]
    for b, Q, n in ((many, Qm, 0), (few, Qf, 1)):
        calls.append(glowq.KVAttentionPlan(sv.cache, sv.batch([70, 129] if n == 0 else [1, 1], lens=lens[n]), Q, workspace=ws))
    for T in (1, 40, 300):
        mods, B, X = w.make(T, 512, [512, 128], 64, seed=T)
        calls.append(glowq.Int8ForwardPlan(w.dev_mods(mods), cuda(B), cuda(X), workspace=ws))
    flat = lambda c: torch.cat([y.reshape(-1) for y in (c.outputs if isinstance(c.outputs, (list, tuple)) else [c.outputs])])
    want = []
    for c in calls:
        c()
        want.append(flat(c).clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls + calls[::-1]:
            c()
    for _ in range(3):
        for c in calls:
            for y in c.outputs if isinstance(c.outputs, (list, tuple)) else [c.outputs]:
                y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(flat(c), x) for c, x in zip(calls, want))
    assert int(ws[:65536].max()) == 0


def test_a_layers_attention_half():
    """The Q/K/V group, append, attention and o_proj as one step after another, 8-bit throughout, on the same buffers:
    each stage against its plain form from the stage's own inputs."""
    import torch
    import test_gpu_w8a8 as w
    n, Hq, Hkv, D, d, r = 3, 4, 2, 64, 256, 16
    sv = Server(n, Hq, Hkv, D, 4, seed=8)
    outs = [Hq * D, Hkv * D, Hkv * D]
    mods, B, _ = w.make(1, d, outs, r, seed=8)
    solo, Bo, _ = w.make(1, Hq * D, [d], r, seed=9)
    dm, ds = w.dev_mods(mods), w.dev_mods(solo)
    for new in ([70, 5, 64], [1, 1, 1], [1, 1, 1], [2, 60, 3]):
        T = sum(new)
        X = sv.g.standard_normal((T, d)).astype(np.float16)
        buf = torch.empty((T, sum(outs)), dtype=torch.float16, device="cuda")
        Ys, R = glowq.group_forward_w8a8(dm, cuda(B), cuda(X), Ys=list(buf.split(outs, 1)))
        w.check(Ys, R, *plain8.w8a8(X, mods, B))
        q, k, v = (y.cpu().numpy().reshape(T, -1, D) for y in Ys)
        at = 0
        qr = np.empty_like(q)
        for s, m in zip(sv.seq, new):
            cs = sv.rope[len(s.k):len(s.k) + m]
            s.append(plain8.rotate(k[at:at + m], cs), v[at:at + m])
            qr[at:at + m] = plain8.rotate(q[at:at + m], cs)
            at += m
        b = sv.batch(new)
        glowq.kv_append(sv.cache, b, Ys[1], Ys[2], Q=Ys[0], Q_out=Ys[0], rope=sv.rope_dev)
        sv.check_held(b)
        att = sv.check_attention(b, Ys[0], qr, new)[:, :-8]
        out = glowq.solo_forward_w8a8(ds[0], cuda(Bo), cuda(att))
        w.check([out], None, *plain8.w8a8(att, solo, Bo))


def test_binding_refuses():
    import torch
    cache = glowq.KVCache.alloc(2, 1, 2, 64)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    f16 = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    step = (i32(0, 1), i32(1), i32(0).reshape(1, 1), i32(0))
    b = glowq.KVBatch(*step, 1, 1)
    table = torch.zeros((4, 64), dtype=torch.float32, device="cuda")
    for rope in (table[:0], table[:, :32].contiguous(), table.half()):
        with pytest.raises(ValueError, match="rope"):
            glowq.kv_append(cache, b, f16(1, 128), f16(1, 128), rope=rope)
    with pytest.raises(glowq.GlowQError, match="ALIGN"):
        glowq.kv_append(cache, b, f16(1, 128), f16(1, 128), rope=torch.zeros(2 + 4 * 64, device="cuda")[2:].reshape(4, 64))
    for Q in (f16(128), f16(1, 100), f16(1, 2, 64), table):
        with pytest.raises(ValueError, match="Q"):
            glowq.kv_append(cache, b, f16(1, 128), f16(1, 128), Q=Q)
        with pytest.raises(ValueError, match="Q"):
            glowq.kv_attention(cache, b, Q)
    with pytest.raises(ValueError, match="Q_out"):
        glowq.kv_append(cache, b, f16(1, 128), f16(1, 128), Q_out=f16(1, 128))
    for rows, most in ((-1, 1), (1, -1), (1 << 31, 1), (1, 1 << 32)):
        with pytest.raises(ValueError, match="rows"):
            glowq.KVBatch(*step, rows, most)
    with pytest.raises(ValueError, match="Y"):
        glowq.kv_attention(cache, b, f16(1, 128), Y=f16(1, 64))
    with pytest.raises(ValueError, match="K"):
        glowq.kv_append(cache, b, f16(0, 128), f16(1, 128))
