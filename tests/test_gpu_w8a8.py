"""GPU W8A8 path: 8-bit integer weights (a scale per output channel) and
activations (a scale per token), quantisers bit-exact and the corrected group /
solo forward element by element against the plain 64-bit form."""
import numpy as np
import pytest

from rank_error_correction_b200 import build, glowq, synth

import plain8

pytestmark = pytest.mark.gpu


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
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def make(T, d, outs, r, seed, outlier=1.0):
    g = np.random.default_rng(seed)
    mods = []
    for O in outs:
        q, s = plain8.quantize_rows(g.standard_normal((O, d), dtype=np.float32) * np.float32(0.02))
        mods.append((q, s, (g.standard_normal((O, r)) * 0.005).astype(np.float16) if r else None))
    X = g.standard_normal((T, d)) * np.sqrt(synth.power_law_spectrum(d, synth.ALPHA_MLP))
    X[:, g.choice(d, 3)] *= outlier
    B = (g.standard_normal((r, d)) * 0.01).astype(np.float16) if r else None
    return mods, B, X.astype(np.float16)


def dev_mods(mods):
    return [glowq.Int8Module(cuda(q), cuda(s), cuda(A)) for q, s, A in mods]


def check(Ys, R, refs, Rref):
    for Y, (y, b) in zip(Ys, refs, strict=True):
        assert plain8.within(Y.cpu().numpy(), y, b) <= 1.0
    if Rref[0] is not None and R is not None:
        assert plain8.within(R.cpu().numpy(), *Rref) <= 1.0


@pytest.mark.parametrize("O,d", [(16, 128), (48, 640), (5, 4096), (1, 14336)])
def test_pack_and_dequant(O, d):
    W = synth.weights(O, d, seed=O + d, outlier_cols=2)
    W[0, :4] = [0.0, -0.0, 1e-30, -3.0]
    if O > 4:
        W[1] = 0.0                      # scale 1
        W[2, 7] = np.inf                # scale NaN, codes 0
        W[3, 9] = np.nan
        W[4] *= 1e-36                   # subnormal values
    q_ref, s_ref = plain8.quantize_rows(W)
    q, s = glowq.pack_int8(cuda(W))
    assert np.array_equal(q.cpu().numpy(), q_ref)
    assert np.array_equal(s.cpu().numpy(), s_ref, equal_nan=True)
    got = glowq.dequant_int8(q, s).cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        want = (q_ref.astype(np.float32) * s_ref[:, None]).astype(np.float16)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("T,d", [(1, 128), (7, 640), (3, 14336), (300, 1024), (2, 16384)])
def test_quantize_act(T, d):
    X = synth.activations(T, d, synth.ALPHA_QKV, seed=T)
    X[0, :5] = np.array([0.0, -0.0, 6e-8, -6e-8, 60000.0], dtype=np.float16)
    if T > 2:
        X[1] = 0.0
        X[2, d - 1] = np.inf
    q_ref, s_ref = plain8.quantize_rows(X)
    q, s = glowq.quantize_act_int8(cuda(X))
    assert np.array_equal(q.cpu().numpy(), q_ref)
    assert np.array_equal(s.cpu().numpy(), s_ref, equal_nan=True)


# one to long T, odd T, module widths that end inside a tile, every rank rule, d of one block to many
SHAPES = [
    (1, 128, [16], 0), (1, 256, [16, 48], 8), (2, 384, [64], 24), (5, 4096, [272, 144, 16], 64),
    (8, 1024, [512], 64), (9, 1024, [512, 256], 72), (16, 14336, [96], 64), (17, 640, [256, 48, 144], 32),
    (31, 2176, [272], 128), (33, 5120, [160, 32], 256), (64, 4096, [1024], 64), (64, 13824, [80], 16),
    (65, 256, [304], 64), (100, 4096, [64], 0), (129, 896, [528, 16], 8), (257, 1152, [272, 400], 64),
    (300, 768, [256, 48, 144], 40), (520, 2048, [1040], 256), (1000, 384, [2064], 64),
    # more tiles than CTA pairs: whole tiles, a rest that is split or not, short k, several slabs
    (2000, 256, [2560, 272], 72), (1500, 128, [5120], 8), (2500, 640, [4096], 0), (1030, 1152, [10000], 256),
    (4000, 128, [512, 16, 4112], 200), (300, 256, [18944], 64),
]


@pytest.mark.parametrize("T,d,outs,r", SHAPES)
def test_group_and_solo_match_plain(T, d, outs, r):
    mods, B, X = make(T, d, outs, r, seed=T + d, outlier=20.0)
    dm, Bt, Xt = dev_mods(mods), cuda(B), cuda(X)
    Ys, R = glowq.group_forward_w8a8(dm, Bt, Xt)
    refs, Rref = plain8.w8a8(X, mods, B)
    check(Ys, R, refs, Rref)
    Y = glowq.solo_forward_w8a8(dm[-1], Bt, Xt)
    check([Y], None, refs[-1:], Rref)
    # the same bits again, from the same workspace
    outs2 = [m.out_features for m in dm]
    ws = glowq.w8a8_workspace(T, d, r, outs2)
    for _ in range(2):
        Ys2, R2 = glowq.group_forward_w8a8(dm, Bt, Xt, workspace=ws)
        assert all(bool((a == b).all()) for a, b in zip(Ys, Ys2))
        assert int(ws[:65536].max()) == 0


@pytest.mark.parametrize("T", [1, 12, 40, 200])
def test_disabled_modules_and_views(T):
    """A module without A gets the plain product; outputs are column slices of one buffer, whose other columns and
    rows keep their values."""
    import torch
    d, outs, r = 512, [64, 16, 304], 16
    mods, B, X = make(T, d, outs, r, seed=T)
    mods[1] = (mods[1][0], mods[1][1], None)
    buf = torch.full((T + 3, 64 + 8 + 16 + 304 + 24), 7.0, dtype=torch.float16, device="cuda")
    views, at = [], 8
    for O in outs:
        views.append(buf[:T, at:at + O])
        at += O
    Ys, R = glowq.group_forward_w8a8(dev_mods(mods), cuda(B), cuda(X), Ys=views)
    refs, Rref = plain8.w8a8(X, mods, B)
    check(Ys, R, refs, Rref)
    b = buf.cpu().numpy()
    assert (b[T:] == 7).all() and (b[:, :8] == 7).all() and (b[:, at:] == 7).all()


@pytest.mark.parametrize("T", [3, 70, 300])
def test_non_finite_tokens_and_channels(T):
    d, outs = 256, [32, 272]
    mods, B, X = make(T, d, outs, 0, seed=T)
    X[1, 5] = np.nan
    X[2, 0] = -np.inf
    X[0] = 0
    q, s, A = mods[1]
    s[3] = np.nan
    Ys, _ = glowq.group_forward_w8a8(dev_mods(mods), None, cuda(X))
    check(Ys, None, plain8.w8a8(X, mods, None)[0], (None, None))


@pytest.mark.parametrize("T,d", [(1, 131072), (20, 131072), (150, 131072)])
def test_largest_sums(T, d):
    """Codes of +-127 throughout: sums of 127^2 d, just below 2^31."""
    X = np.ones((T, d), np.float16)
    q = np.full((16, d), 127, np.int8)
    q[1] = -127
    q[2, ::2] = -127
    s = np.full(16, 2.0 ** -14, np.float32)
    Y, _ = glowq.group_forward_w8a8([glowq.Int8Module(cuda(q), cuda(s))], None, cuda(X))
    check(Y, None, plain8.w8a8(X, [(q, s, None)], None)[0], (None, None))


@pytest.mark.parametrize("T", [1, 13, 48, 333])
def test_shared_workspace_across_shapes_streams_and_graphs(T):
    """One workspace for calls of other shapes in between; a captured and replayed call; a call on another stream."""
    import torch
    d, outs, r = 2048, [256, 64], 64
    mods, B, X = make(T, d, outs, r, seed=T)
    dm, Bt, Xt = dev_mods(mods), cuda(B), cuda(X)
    refs, Rref = plain8.w8a8(X, mods, B)
    mods2, B2, X2 = make(30, 640, [48], 8, seed=2)
    refs2, Rref2 = plain8.w8a8(X2, mods2, B2)
    n = max(glowq.w8a8_workspace_bytes(T, d, r, outs), glowq.w8a8_workspace_bytes(30, 640, 8, [48]))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    plan = glowq.Int8ForwardPlan(dm, Bt, Xt, workspace=ws)
    other = glowq.Int8ForwardPlan(dev_mods(mods2), cuda(B2), cuda(X2), workspace=ws)
    for _ in range(3):
        check(plan(), plan.R, refs, Rref)
        check(other(), other.R, refs2, Rref2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for Y in plan.outputs:
        Y.zero_()
    torch.cuda.synchronize()
    plan(stream=s)
    s.synchronize()
    check(plan.outputs, plan.R, refs, Rref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan()
        other()
        plan()
    for _ in range(3):
        for Y in plan.outputs + other.outputs:
            Y.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(plan.outputs, plan.R, refs, Rref)
        check(other.outputs, other.R, refs2, Rref2)
    # inputs that change between replays are read anew
    Xt.copy_(cuda(X[::-1].copy()))
    g.replay()
    torch.cuda.synchronize()
    check(plan.outputs, plan.R, *plain8.w8a8(X[::-1].copy(), mods, B))


@pytest.mark.parametrize("T", [1, 5, 16, 40])
@pytest.mark.parametrize("r", [0, 64])
def test_weights_written_by_the_call_before(T, r):
    """A module whose codes and scales the token quantiser, or the weight quantiser, writes on the same stream directly
    ahead of the forward call, which may fetch nothing of them early."""
    import torch
    O, d = 4096, 2048
    g = np.random.default_rng(T)
    L, stream = glowq.lib(), torch.cuda.current_stream()
    Ws = [cuda((g.standard_normal((O, d)) * 0.02).astype(np.float16)) for _ in range(2)]
    _, B, X = make(T, d, [16], r, seed=T)
    A = cuda((g.standard_normal((O, r)) * 0.005).astype(np.float16)) if r else None
    mod = glowq.Int8Module(torch.zeros((O, d), dtype=torch.int8, device="cuda"), torch.zeros(O, device="cuda"), A)
    plan = glowq.Int8ForwardPlan([mod], cuda(B), cuda(X))

    def write(W, packs):
        if packs:
            rc = L.glowq_pack_int8(W.data_ptr(), O, d, mod.codes.data_ptr(), mod.scales.data_ptr(), stream.cuda_stream)
        else:
            rc = L.glowq_quantize_act_int8(W.data_ptr(), O, d, mod.codes.data_ptr(), mod.scales.data_ptr(), stream.cuda_stream)
        assert rc == 0

    want, full = [], [W.float() for W in Ws]
    for W in Ws:
        write(W, False)
        torch.cuda.synchronize()
        plan()
        q, s = plain8.quantize_rows(W.cpu().numpy())
        check(plan.outputs, plan.R, *plain8.w8a8(X, [(q, s, None if A is None else A.cpu().numpy())], B))
        want.append(plan.outputs[0].clone())
    assert not torch.equal(*want)
    for packs in (False, True):
        for i in range(20):
            torch.cuda._sleep(200000)            # all of what follows is enqueued before it begins
            write((full if packs else Ws)[i % 2], packs)
            plan()
            torch.cuda.synchronize()
            assert torch.equal(plan.outputs[0], want[i % 2])


def test_a_plan_holds_the_tensors_whose_addresses_it_has():
    """Fields of modules and caches that are set anew afterwards free nothing that a plan still uses."""
    import gc
    import weakref
    import torch
    mods, B, X = make(2, 256, [32, 16], 8, seed=1)
    dm = dev_mods(mods)
    plan = glowq.Int8ForwardPlan(dm, cuda(B), cuda(X))
    held = [weakref.ref(t) for m in dm for t in (m.codes, m.scales, m.A)] + [weakref.ref(t) for t in plan.outputs]
    for m in dm:
        m.codes = m.scales = m.A = None
    plan.outputs = None
    cache = glowq.KVCache.alloc(2, 1, 1, 64)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    batch = glowq.KVBatch(i32(0, 1), i32(1), i32(0).reshape(1, 1), i32(0), 1, 1)
    plans = [glowq.KVAttentionPlan(cache, batch, torch.zeros((1, 64), dtype=torch.float16, device="cuda")),
             glowq.KVReadPlan(cache, batch, 1)]
    held += [weakref.ref(getattr(cache, f)) for f in ("k_codes", "v_codes", "k_scales", "v_scales", "k_tail", "v_tail")]
    held += [weakref.ref(t) for t in (plans[0].outputs, *plans[1].outputs)]
    cache.k_codes = cache.v_codes = cache.k_scales = cache.v_scales = cache.k_tail = cache.v_tail = None
    for p in plans:
        p.outputs = None
    gc.collect()
    assert all(r() is not None for r in held)
