"""Cases of the 8-bit serving operators and their plain forms.

Three operators that follow one another in a decoder layer's attention half:

  w8a8    the corrected linear with 8-bit integer weights (a scale per output
          channel) and 8-bit integer activations (a scale per token)
  append  rotation of Q and K by position, and keys and values appended to a
          paged cache: complete pages of 64 tokens in 8-bit integers with one
          scale per page and head, the incomplete last page in fp16
  attend  causal attention of the step's queries over that cache

`run` computes them in elementary torch operations in 32 bits (own = False),
or calls the library (own = True).
"""
import math
import random

import torch

own = False

PAGE = 64
MAX_POS_TABLE = 1 << 15


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # decode of one token through the Q/K/V group of LLaMA-2-7B: weight streaming, latency counts
        dict(name="w8a8_7b_qkv_t1", op="w8a8", d=4096, outs="4096,4096,4096", r=64, T=1),
        # decode batch through the gate/up group of LLaMA-2-13B
        dict(name="w8a8_13b_gateup_t32", op="w8a8", d=5120, outs="13824,13824", r=64, T=32),
        # a short ragged prompt through down_proj of LLaMA-3.1-8B (solo: its own factors)
        dict(name="w8a8_8b_down_t333", op="w8a8", d=14336, outs="4096", r=64, T=333),
        # prefill through the gate/up group of LLaMA-2-7B
        dict(name="w8a8_7b_gateup_t2048", op="w8a8", d=4096, outs="11008,11008", r=64, T=2048),
        # one decode step of 64 sequences, LLaMA-3.1-8B heads: one token each, which completes a page for two of them
        dict(name="append_8b_decode_n64", op="append", Hq=32, Hkv=8, D=128, n=64, cached_lo=0, cached_hi=4000,
             new_lo=1, new_hi=1, lens=6),
        # new prompts of uneven lengths, LLaMA-2-13B heads
        dict(name="append_13b_prompts_n6", op="append", Hq=40, Hkv=40, D=128, n=6, cached_lo=0, cached_hi=0,
             new_lo=1, new_hi=700, lens=2),
        # one long prompt chunk behind cached pages, LLaMA-2-7B heads
        dict(name="append_7b_chunk_4096", op="append", Hq=32, Hkv=32, D=128, n=1, cached_lo=1024, cached_hi=1024,
             new_lo=4096, new_hi=4096, lens=3),
        # one sequence decoding, LLaMA-2-7B heads, a short cache: the smallest call
        dict(name="attend_7b_decode_n1", op="attend", Hq=32, Hkv=32, D=128, n=1, cached_lo=499, cached_hi=499,
             new_lo=1, new_hi=1, lens=4),
        # a decode batch of uneven lengths, LLaMA-3.1-8B heads
        dict(name="attend_8b_decode_n64", op="attend", Hq=32, Hkv=8, D=128, n=64, cached_lo=1, cached_hi=4096,
             new_lo=1, new_hi=1, lens=5),
        # a long context decoding, LLaMA-3.1-8B heads: few rows, a long axis
        dict(name="attend_8b_decode_long", op="attend", Hq=32, Hkv=8, D=128, n=2, cached_lo=100001,
             cached_hi=131071, new_lo=1, new_hi=1, lens=6),
        # prefill of one prompt, LLaMA-2-7B heads
        dict(name="attend_7b_prefill_4096", op="attend", Hq=32, Hkv=32, D=128, n=1, cached_lo=0, cached_hi=0,
             new_lo=4096, new_hi=4096, lens=7),
        # chunks of uneven lengths behind uneven caches, LLaMA-3.1-8B heads
        dict(name="attend_8b_chunks_n4", op="attend", Hq=32, Hkv=8, D=128, n=4, cached_lo=0, cached_hi=6000,
             new_lo=100, new_hi=1000, lens=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w8a8", "append", "attend", "attend"])
    if op == "w8a8":
        while True:
            d = 128 * _log_int(rng, 2, 112)
            outs = [16 * _log_int(rng, 4, 896) for _ in range(rng.choice([1, 2, 3]))]
            T = _log_int(rng, 1, 4096)
            if T * sum(outs) * d <= 2048 * 22016 * 4096:
                break
        return dict(op=op, d=d, outs=",".join(map(str, outs)), r=rng.choice([0, 8, 32, 64, 64, 128]), T=T)
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16, 32])
    Hq = Hkv * rng.choice([g for g in (1, 2, 4, 8) if Hkv * g <= 64])
    seed = rng.randrange(1 << 30)
    if op == "append":
        n = _log_int(rng, 1, 64)
        if rng.random() < 0.4:          # decode
            return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, n=n, cached_lo=0, cached_hi=4000, new_lo=1, new_hi=1, lens=seed)
        hi = max(1, min(4096, 4096 * 32 // (n * Hq)))
        return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, n=n, cached_lo=0, cached_hi=4000, new_lo=1,
                    new_hi=_log_int(rng, 1, hi), lens=seed)
    if rng.random() < 0.6:              # decode, some of it with a few tokens of each sequence at once
        n = _log_int(rng, 1, 64)
        most = max(64, min(131072, 2 * 131072 * 8 // (n * Hkv)))
        hi = _log_int(rng, 1, most)
        return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, n=n, cached_lo=rng.randrange(0, hi + 1), cached_hi=hi, new_lo=1,
                    new_hi=rng.choice([1, 1, 1, 4]), lens=seed)
    n = rng.choice([1, 1, 2, 3, 4])
    new = _log_int(rng, 16, 2048 // n)
    cached = rng.choice([0, _log_int(rng, 1, 2048)])
    Hkv = min(Hkv, 32)
    Hq = min(Hq, 32)
    return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, n=n, cached_lo=0, cached_hi=cached, new_lo=max(1, new // 4),
                new_hi=new, lens=seed)


def _lens(case):
    """(cached, new) tokens of each sequence."""
    rng = random.Random(case["lens"])
    got = []
    for _ in range(case["n"]):
        cached, new = rng.randint(case["cached_lo"], case["cached_hi"]), rng.randint(case["new_lo"], case["new_hi"])
        if case["op"] == "append" and case["new_hi"] > 1:
            cached -= cached % PAGE     # a scheduler cuts prompts into whole pages
        got.append((cached, new))
    return got


# ----------------------------------------------------------------- inputs ----

def _quantize_rows(W):
    amax = W.abs().amax(dim=1)
    s = torch.where(amax > 0, amax / 127.0, torch.ones_like(amax))
    return torch.clamp(torch.round(W / s[:, None]), -127, 127).to(torch.int8), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "w8a8":
        d, T, r = case["d"], case["T"], case["r"]
        outs = [int(o) for o in case["outs"].split(",")]
        mods = []
        for O in outs:
            codes, scales = _quantize_rows(randn(O, d) * 0.02)
            mods.append((codes, scales, (randn(O, r) * 0.005).half() if r else None))
        # activations with the power-law spectrum of a layer's input, in a random order of channels
        lam = torch.arange(1, d + 1, device=dev, dtype=torch.float32) ** -0.77
        lam = (lam * (d / lam.sum()))[torch.randperm(d, generator=g, device=dev)]
        X = (randn(T, d) * lam.sqrt()).half()
        B = (randn(r, d) * 0.01).half() if r else None
        return dict(op="w8a8", mods=mods, B=B, X=X)

    n, Hq, Hkv, D = case["n"], case["Hq"], case["Hkv"], case["D"]
    lens = _lens(case)
    new = [q for _, q in lens]
    kv_len = [c + q for c, q in lens]
    n_pages = [-(-k // PAGE) for k in kv_len]
    cols = max(n_pages)
    order = torch.randperm(sum(n_pages), generator=g, device=dev).to(torch.int32)
    table = torch.zeros(n, cols, dtype=torch.int32, device=dev)
    at = 0
    for b, p in enumerate(n_pages):
        table[b, :p] = order[at:at + p]
        at += p
    starts = [0]
    for q in new:
        starts.append(starts[-1] + q)
    T = starts[-1]
    i32 = dict(dtype=torch.int32, device=dev)
    st = dict(op=case["op"], n=n, Hq=Hq, Hkv=Hkv, D=D, T=T, max_new=max(new), max_len=max(kv_len),
              q_start=torch.tensor(starts, **i32), kv_len=torch.tensor(kv_len, **i32), table=table,
              slot=torch.randperm(n, generator=g, device=dev).to(torch.int32),
              row_seq=torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(new, device=dev)),
              scale=1.0 / math.sqrt(D))
    st["row_at"] = torch.arange(T, device=dev) - st["q_start"][st["row_seq"]]
    # keys have a few strong channels, as a layer's keys do
    strong = torch.ones(Hkv, D, device=dev)
    strong[:, torch.randperm(D, generator=g, device=dev)[:3]] = 6.0
    P = sum(n_pages)
    k_codes = torch.empty(P, Hkv, D // 64, PAGE, 64, dtype=torch.int8, device=dev)
    v_codes = torch.empty(P, Hkv, D, PAGE, dtype=torch.int8, device=dev)
    k_scales = torch.empty(P, Hkv, device=dev)
    v_scales = torch.empty(P, Hkv, device=dev)
    if case["op"] == "attend" or case["cached_hi"] > 0:
        for a in range(0, P, 1024):
            b = min(P, a + 1024)
            for codes, scales, strength in ((k_codes, k_scales, strong), (v_codes, v_scales, None)):
                x = randn(b - a, Hkv, PAGE, D)
                if strength is not None:
                    x = x * strength[:, None]
                c, s = _quantize_rows(x.half().float().reshape((b - a) * Hkv, PAGE * D))
                c = c.view(b - a, Hkv, PAGE, D)
                codes[a:b] = (c.view(b - a, Hkv, PAGE, D // 64, 64).transpose(2, 3) if strength is not None
                              else c.transpose(2, 3))
                scales[a:b] = s.view(b - a, Hkv)
    st.update(k_codes=k_codes, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales,
              k_tail=(randn(n, Hkv, PAGE, D) * strong[:, None]).half(), v_tail=randn(n, Hkv, PAGE, D).half())
    if case["op"] == "attend":
        st["Q"] = randn(T, Hq * D).half()
        return st
    # the step's queries, keys and values as a Q/K/V group leaves them: column slices of one buffer
    qkv = torch.cat([randn(T, Hq * D), (randn(T, Hkv, D) * strong).reshape(T, Hkv * D), randn(T, Hkv * D)], 1).half()
    st["Q"], st["K"], st["V"] = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    # cosines and sines by position, theta 500000
    inv = 500000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
    ang = torch.arange(MAX_POS_TABLE, dtype=torch.float64, device=dev)[:, None] * inv
    st["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    # what is read back: the pages that the step touched, from the first one's start
    start = st["kv_len"] - (st["q_start"][1:] - st["q_start"][:-1])
    st["first"] = (start // PAGE * PAGE).to(torch.int32)
    st["count"] = max(-(-k // PAGE) * PAGE - (k - q) // PAGE * PAGE for k, q in zip(kv_len, new))
    return st


# ------------------------------------------------------------ plain forms ----

def _w8a8(st, f=torch.float32):
    X = st["X"].float()
    codes, s_t = _quantize_rows(X)
    codes = codes.to(f)
    R = X.to(f) @ st["B"].to(f).T if st["B"] is not None else None
    Ys = []
    for q, s, A in st["mods"]:
        y = (codes @ q.to(f).T) * s_t[:, None].to(f) * s.to(f)
        Ys.append(y + R @ A.to(f).T if A is not None else y)
    return Ys, R


def _rotated(x, cos, sin):
    a, b = x[..., : x.shape[-1] // 2], x[..., x.shape[-1] // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _stored_pages(st):
    """The cache's complete pages of every sequence by position: n x (pages 64) x Hkv x D, in 32 bits."""
    t = st["table"].long()
    n, cols, Hkv, D = st["n"], t.shape[1], st["Hkv"], st["D"]
    k = st["k_codes"][t].float() * st["k_scales"][t][..., None, None, None]
    v = st["v_codes"][t].float() * st["v_scales"][t][..., None, None]
    k = k.permute(0, 1, 4, 2, 3, 5).reshape(n, cols * PAGE, Hkv, D)
    return k, v.permute(0, 1, 4, 2, 3).reshape(n, cols * PAGE, Hkv, D)


def _append(st, f=torch.float32):
    n, Hq, Hkv, D, T, count = st["n"], st["Hq"], st["Hkv"], st["D"], st["T"], st["count"]
    kv_len, q0 = st["kv_len"].long(), st["q_start"].long()
    start = kv_len - (q0[1:] - q0[:-1])
    at = start[st["row_seq"]] + st["row_at"]
    cos, sin = st["rope"][at].to(f)[:, None].chunk(2, -1)
    Q = _rotated(st["Q"].to(f).reshape(T, Hq, D), cos, sin)
    K = _rotated(st["K"].to(f).reshape(T, Hkv, D), cos, sin).half()
    V = st["V"].reshape(T, Hkv, D)
    # positions first .. first + count of each sequence: from the tail before `start`, from the new rows behind it
    pos = st["first"].long()[:, None] + torch.arange(count, device=kv_len.device)
    row = (q0[:-1, None] + pos - start[:, None]).clamp(0, T - 1)
    is_new, inside = pos >= start[:, None], pos < kv_len[:, None]
    complete = (pos // PAGE + 1) * PAGE <= kv_len[:, None]
    out = []
    for fresh, tail in ((K, st["k_tail"]), (V, st["v_tail"])):
        old = tail[st["slot"].long()].transpose(1, 2)[torch.arange(n, device=pos.device)[:, None], pos % PAGE]
        x = torch.where(is_new[..., None, None], fresh[row], old).float()
        x = torch.where(inside[..., None, None], x, torch.zeros_like(x))
        p = x.view(n, count // PAGE, PAGE, Hkv, D)
        s = p.abs().amax(dim=(2, 4), keepdim=True).clamp(min=2.0 ** -24) / 127.0
        held = (torch.clamp(torch.round(p / s), -127, 127) * s).view(n, count, Hkv, D)
        out.append(torch.where(complete[..., None, None], held, x).reshape(n, count, Hkv * D))
    return Q.reshape(T, Hq * D), out[0], out[1]


def _attend(st, f=torch.float32):
    n, Hq, Hkv, D, T, most = st["n"], st["Hq"], st["Hkv"], st["D"], st["T"], st["max_new"]
    kv_len, q0 = st["kv_len"].long(), st["q_start"].long()
    new = q0[1:] - q0[:-1]
    k, v = _stored_pages(st)
    L = k.shape[1]
    pos = torch.arange(L, device=k.device)
    # the incomplete last page comes from the tail
    in_tail = (pos[None] >= (kv_len // PAGE * PAGE)[:, None])[..., None, None]
    slot = st["slot"].long()
    k = torch.where(in_tail, st["k_tail"][slot].transpose(1, 2).repeat(1, L // PAGE, 1, 1).float(), k).to(f)
    v = torch.where(in_tail, st["v_tail"][slot].transpose(1, 2).repeat(1, L // PAGE, 1, 1).float(), v).to(f)
    inside = (pos[None] < kv_len[:, None])[..., None, None]
    v = torch.where(inside, v, torch.zeros_like(v))
    i = torch.arange(most, device=k.device)
    rows = (q0[:-1, None] + i).clamp(max=T - 1)
    Q = st["Q"].to(f)[rows].view(n, most, Hkv, Hq // Hkv, D)
    s = torch.einsum("nqhgd,nlhd->nhgql", Q, k) * st["scale"]
    sees = pos[None, None] <= (kv_len - new)[:, None, None] + i[None, :, None]      # n x most x L
    s.masked_fill_(~(sees & inside[:, None, :, 0, 0])[:, None, None], float("-inf"))
    p = torch.exp_(s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("nhgql,nlhd->nhgqd", p, v) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(n, most, Hq * D)[st["row_seq"], st["row_at"]]


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "w8a8":
        Ys, R = _w8a8(st)
        return [y.half() for y in Ys], None if R is None else R.half()
    if st["op"] == "append":
        return [x.half() for x in _append(st)]
    return _attend(st).half()


# -------------------------------------------------------- the library's calls ----

def _run_own(st):
    from rank_error_correction_b200 import glowq
    if "plan" not in st:                # the program's own buffers and arguments, made once
        if st["op"] == "w8a8":
            mods = [glowq.Int8Module(q, s, A) for q, s, A in st["mods"]]
            st["plan"] = glowq.Int8ForwardPlan(mods, st["B"], st["X"])
        else:
            cache = glowq.KVCache(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"], st["k_tail"],
                                  st["v_tail"])
            batch = glowq.KVBatch(st["q_start"], st["kv_len"], st["table"], st["slot"], st["T"], st["max_new"])
            if st["op"] == "append":
                st["plan"] = glowq.KVAppendPlan(cache, batch, st["K"], st["V"], Q=st["Q"], rope=st["rope"])
                st["read"] = glowq.KVReadPlan(cache, batch, st["count"], first=st["first"])
            else:
                st["plan"] = glowq.KVAttentionPlan(cache, batch, st["Q"], scale=st["scale"])
    if st["op"] == "w8a8":
        Ys = st["plan"]()
        return Ys, st["plan"].R
    if st["op"] == "append":
        Q = st["plan"]()
        K, V = st["read"]()
        return [Q, K, V]
    return st["plan"]()


# ------------------------------------------------------------ in 64 bits ----

def exact(case, seed):
    st = prepare(case, seed)
    f = torch.float64
    if case["op"] == "w8a8":
        X = st["X"].float()
        amax = X.abs().max(dim=1).values
        s_t = torch.where(amax == 0, torch.ones_like(amax), amax / 127)     # the scales and codes are defined in 32 bits
        c = (X / s_t[:, None]).round().clamp(-127, 127).to(f)
        R = None if st["B"] is None else torch.matmul(X.to(f), st["B"].to(f).t())
        Ys = []
        for q, s, A in st["mods"]:
            y = torch.outer(s_t.to(f), s.to(f)) * torch.matmul(c, q.to(f).t())
            Ys.append(y if A is None else y + torch.matmul(R, A.to(f).t()))
        return Ys, R
    n, Hq, Hkv, D = case["n"], case["Hq"], case["Hkv"], case["D"]
    lens = _lens(case)
    G = Hq // Hkv
    q0 = [0]
    for _, q in lens:
        q0.append(q0[-1] + q)
    slots, table = st["slot"].tolist(), st["table"].tolist()
    if case["op"] == "append":
        half = D // 2
        Qs = torch.empty(st["T"], Hq * D, dtype=f, device="cuda")
        outs = [torch.zeros(n, st["count"], Hkv, D, dtype=f, device="cuda") for _ in range(2)]
        for b, (cached, new) in enumerate(lens):
            rows = slice(q0[b], q0[b + 1])
            cs = st["rope"][cached:cached + new].to(f)
            z = torch.complex(cs[:, :half], cs[:, half:])[:, None]

            def turn(x, H):
                x = x[rows].to(f).reshape(new, H, D)
                t = torch.complex(x[..., :half], x[..., half:]) * z
                return torch.cat([t.real, t.imag], -1)

            Qs[rows] = turn(st["Q"], Hq).reshape(new, Hq * D)
            first = cached - cached % PAGE
            for out, x, tail in ((outs[0], turn(st["K"], Hkv).half(), st["k_tail"]),
                                 (outs[1], st["V"][rows].reshape(new, Hkv, D), st["v_tail"])):
                x = torch.cat([tail[slots[b], :, :cached - first].transpose(0, 1), x])      # from `first` on
                done = (cached + new) // PAGE * PAGE - first
                out[b, :x.shape[0]] = x.to(f)
                if done > 0:
                    p = x[:done].float().view(-1, PAGE, Hkv, D)
                    s = torch.maximum(p.abs().amax(3).amax(1), torch.full((), 2.0 ** -24, device="cuda")) / 127
                    s = s[:, None, :, None]
                    out[b, :done] = ((p / s).round().clamp(-127, 127).to(f) * s.to(f)).view(done, Hkv, D)
        return [Qs, outs[0].view(n, -1, Hkv * D), outs[1].view(n, -1, Hkv * D)]
    Y = torch.zeros(st["T"], Hq, D, dtype=f, device="cuda")
    for b, (cached, new) in enumerate(lens):
        kv = cached + new
        pages = torch.tensor(table[b][:kv // PAGE], dtype=torch.long, device="cuda")
        rest = kv % PAGE
        for h in range(Hkv):
            K = st["k_codes"][pages, h].to(f).transpose(1, 2).reshape(-1, PAGE, D) * st["k_scales"][pages, h].to(f)[:, None, None]
            V = st["v_codes"][pages, h].to(f).transpose(1, 2) * st["v_scales"][pages, h].to(f)[:, None, None]
            K = torch.cat([K.reshape(-1, D), st["k_tail"][slots[b], h, :rest].to(f)])
            V = torch.cat([V.reshape(-1, D), st["v_tail"][slots[b], h, :rest].to(f)])
            Q = st["Q"][q0[b]:q0[b + 1]].to(f).view(new, Hq, D)[:, h * G:(h + 1) * G]
            s = torch.matmul(Q.transpose(0, 1), K.t()) * st["scale"]
            later = torch.arange(kv, device="cuda")[None] > cached + torch.arange(new, device="cuda")[:, None]
            w = torch.softmax(s.masked_fill(later, -math.inf), -1)
            Y[q0[b]:q0[b + 1], h * G:(h + 1) * G] = torch.matmul(w, V).transpose(0, 1)
    return Y.view(st["T"], Hq * D)


# ------------------------------------------------------------------- work ----

def work(case):
    if case["op"] == "w8a8":
        d, T, r = case["d"], case["T"], case["r"]
        O = sum(int(o) for o in case["outs"].split(","))
        return dict(bytes=O * d + 4 * O + 2 * T * d + 2 * r * d + 2 * O * r + 2 * T * O + 2 * T * r,
                    flops=2 * T * O * d + 2 * T * r * (d + O))
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    lens = _lens(case)
    T = sum(q for _, q in lens)
    if case["op"] == "append":
        stored = read = 0
        for c, q in lens:
            first, kv = c // PAGE * PAGE, c + q
            done = kv // PAGE * PAGE
            if done > first:                            # completed pages in codes, what is behind them in fp16
                stored += (done - first) + 2 * (kv - done)
                read += 2 * (c - first)
            else:
                stored += 2 * q
        held = sum(c % PAGE + q for c, q in lens)
        most = max(-(-(c + q) // PAGE) * PAGE - c // PAGE * PAGE for c, q in lens)
        b = 2 * T * (Hq + 2 * Hkv) * D + 4 * T * D + 2 * T * Hq * D + 2 * Hkv * D * (stored + read)
        b += 2 * 2 * Hkv * D * case["n"] * most         # the values that are read back
        return dict(bytes=b, flops=3 * T * (Hq + Hkv) * D + 4 * held * Hkv * D)
    seen = sum(q * c + q * (q + 1) // 2 for c, q in lens)
    codes = sum((c + q) // PAGE * PAGE + 2 * ((c + q) % PAGE) for c, q in lens)
    return dict(bytes=2 * codes * Hkv * D + 2 * 2 * T * Hq * D, flops=4 * D * Hq * seen)
