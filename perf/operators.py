"""Cases of the packed and paged attention calls, with their plain forms.

Five operators: attention over packed prompts with grouped heads (``fwd_packed``)
and its gradients (``bwd_packed``), the write of new keys and values into a paged
cache (``paged_append``), attention of one new token over that cache
(``paged_decode``), and the eviction of the keys that drew the least attention
(``paged_evict``).  ``run`` computes each in elementary torch operations in 32
bits, or, where ``own`` is true, through the framework's calls; ``exact`` computes
the definitions again in 64 bits, one sequence at a time.

Shapes.  Packed tensors are [tokens, heads, d]; sequence b owns rows
[cu[b], cu[b + 1]).  Cache pools are [pages, kv_heads, page, d]; position p of
sequence b lives in row p % page of page table[b, p // page].
"""
import math
import random

import torch

own = False

F32 = torch.float32
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # a handful of chat turns answered together, one of them a single token: launch-bound
        dict(name="fwd_chat_d64", op="fwd", B=6, lo=1, hi=400, prefix=0, Hq=16, Hkv=4, d=64, causal=True, pick=1),
        # prompts of mixed length, each a chunk behind keys that are already there
        dict(name="fwd_batch_prefix_d128", op="fwd", B=8, lo=200, hi=2048, prefix=500, Hq=32, Hkv=8, d=128,
             causal=True, pick=2),
        # two long documents, of the benchmark's length and heads
        dict(name="fwd_long_d128", op="fwd", B=2, lo=6100, hi=8192, prefix=0, Hq=16, Hkv=4, d=128, causal=True, pick=3),
        # one packed training row of short documents, every head with its own keys (the GPT-2 shape's heads)
        dict(name="bwd_docs_d64", op="bwd", B=8, lo=30, hi=1024, prefix=0, Hq=12, Hkv=12, d=64, causal=True, pick=4),
        # a long-context training step with grouped heads
        dict(name="bwd_long_d128", op="bwd", B=2, lo=6100, hi=8192, prefix=0, Hq=16, Hkv=4, d=128, causal=True, pick=5),
        # the cache write of one decoding step of a full batch
        dict(name="append_step", op="append", B=64, lo=1, hi=1, held=500, Hkv=8, d=128, page=16, e4m3=False, pick=6),
        # prompts written to an 8-bit cache after their forward pass
        dict(name="append_prompts_e4m3", op="append", B=8, lo=300, hi=2000, held=0, Hkv=8, d=128, page=64, e4m3=True,
             pick=7),
        # one user, a short history: the smallest decoding step
        dict(name="decode_one", op="decode", B=1, lo=777, hi=777, Hq=32, Hkv=8, d=128, page=16, e4m3=False,
             weights=False, pick=8),
        # a serving batch of mixed lengths, with the weights that eviction goes by
        dict(name="decode_batch_weights", op="decode", B=32, lo=1, hi=8192, Hq=32, Hkv=8, d=128, page=16, e4m3=False,
             weights=True, pick=9),
        # long contexts (the decode workload's 32K) in an 8-bit cache
        dict(name="decode_long_e4m3", op="decode", B=4, lo=30001, hi=32768, Hq=32, Hkv=8, d=128, page=64, e4m3=True,
             weights=False, pick=10),
        # a small cache cut to a quarter
        dict(name="evict_small_d64", op="evict", B=2, lo=500, hi=1000, budget=250, recent=64, Hkv=4, d=64, page=16,
             e4m3=False, pick=11),
        # a serving batch's caches cut to a quarter
        dict(name="evict_batch", op="evict", B=8, lo=7000, hi=8192, budget=2048, recent=256, Hkv=8, d=128, page=64,
             e4m3=False, pick=12),
    ]


HEADS = [(32, 8), (16, 4), (16, 16), (12, 12), (8, 1), (24, 8), (10, 2), (16, 1), (40, 2), (3, 1)]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.25 / hi))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "append", "decode", "decode", "evict"])
    Hq, Hkv = rng.choice(HEADS)
    c = dict(op=op, Hkv=Hkv, d=rng.choice([64, 128]), pick=rng.randrange(1, 1 << 30))
    if op in ("fwd", "bwd"):
        hi = _log(rng, 64, 6000) if op == "bwd" else _log(rng, 16, 6000)
        B = _log(rng, 1, 24)
        B = max(1, min(B, (2 * 16 * 8192 * 8192) // (Hq * hi * (hi + hi // 2))))
        # (the gradients of a row that sees a key or two are differences of nearly equal numbers)
        c.update(B=B, hi=hi, lo=rng.randint(16 if op == "bwd" else 1, hi), prefix=rng.choice([0, 0, rng.randint(1, max(1, hi // 2))]), Hq=Hq,
                 causal=rng.random() < 0.8)
    elif op == "append":
        one = rng.random() < 0.5
        hi = 1 if one else _log(rng, 2, 2000)
        c.update(B=_log(rng, 1, 128 if one else 8), lo=1 if one else rng.randint(1, hi), hi=hi, held=_log(rng, 1, 600) - 1,
                 page=rng.choice([8, 16, 24, 64, 128]), e4m3=rng.random() < 0.5)
    elif op == "decode":
        hi = _log(rng, 1, 32768)
        B = max(1, min(_log(rng, 1, 64), (32 * 8192 * 8) // (hi * Hkv)))
        c.update(B=B, hi=hi, lo=rng.randint(1, hi), Hq=Hq, page=rng.choice([8, 16, 24, 64, 128]),
                 e4m3=rng.random() < 0.5, weights=rng.random() < 0.5)
    else:
        hi = _log(rng, 16, 16384)
        B = max(1, min(_log(rng, 1, 16), (8 * 8192 * 8) // (hi * Hkv)))
        budget = rng.randint(1, hi)
        c.update(B=B, hi=hi, lo=rng.randint(1, hi), budget=budget, recent=rng.randint(0, budget),
                 page=rng.choice([8, 16, 24, 64, 128]), e4m3=rng.random() < 0.5)
    return c


def lengths(c):
    """The sequences' lengths (and the keys held before each, for a prefix or a cache), from the case alone."""
    r = random.Random(c["pick"])
    n = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    n[0], n[-1] = c["lo"], c["hi"]
    more = c.get("prefix", c.get("held", 0))
    return n, [r.randint(0, more) for _ in n]


# ----------------------------------------------------------------- inputs ---
def _cu(n, dev):
    return torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32, device=dev)


def _table(g, lens, page, first, width, dev):
    """Pages first, first + 1, ... dealt to the sequences in a shuffled order; -1 behind each sequence's last."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need), generator=g, device=dev).to(torch.int32) + first
    t = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = ids[at:at + k]
        at += k
    return t, at


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed * 1000003 + c["pick"] % 99991)
    randn = lambda *s: torch.randn(s, generator=g, device=dev, dtype=F32).to(torch.bfloat16)
    op, Hkv, d = c["op"], c["Hkv"], c["d"]
    n, held = lengths(c)
    st = dict(case=c, scale=float(torch.tensor(d ** -0.5, dtype=F32)))
    if op in ("fwd", "bwd"):
        nk = [a + b for a, b in zip(n, held)]
        st.update(Q=randn(sum(n), c["Hq"], d), K=randn(sum(nk), Hkv, d), V=randn(sum(nk), Hkv, d), cu_q=_cu(n, dev),
                  cu_k=_cu(nk, dev), Lq=max(n), Lk=max(nk))
        if op == "bwd":
            st["dO"] = randn(*st["Q"].shape)
            st["O"], st["LSE"] = plain_fwd(st)
        st["ws"] = {}
        return st
    page, e4m3 = c["page"], c["e4m3"]
    total = [a + b for a, b in zip(n, held)]
    W = -(-max(total) // page)
    table, pages = _table(g, total, page, 0, W, dev)
    spare = 0
    if op == "evict":
        Wo = -(-c["budget"] // page)
        st["table_out"], spare = _table(g, [c["budget"]] * c["B"], page, pages, Wo, dev)
    pool = lambda: randn(pages + spare, Hkv, page, d)
    K, V = pool(), pool()
    if e4m3:  # codes of values whose largest is near the type's, as a calibrated cache holds them
        st["ks"] = torch.rand(Hkv, generator=g, device=dev) * 0.01 + 0.01
        st["vs"] = torch.rand(Hkv, generator=g, device=dev) * 0.01 + 0.01
        enc = lambda x, s: (x.float() / s[:, None, None]).clamp(-448, 448).to(E4M3)
        K, V = enc(K, st["ks"]), enc(V, st["vs"])
    else:
        st["ks"] = st["vs"] = None
    st.update(kc=K, vc=V, table=table, lens=torch.tensor(total, dtype=torch.int32, device=dev), L=W * page)
    if op == "append":
        st.update(K=randn(sum(n), Hkv, d), V=randn(sum(n), Hkv, d), cu=_cu(n, dev),
                  lens=torch.tensor(held, dtype=torch.int32, device=dev))
    elif op == "decode":
        st["Q"] = randn(c["B"], c["Hq"], d)
        st["w"] = torch.zeros(c["B"], Hkv, st["L"], device=dev) if c["weights"] else None
        st["ws"] = {}
    else:
        # what decoding leaves behind: a few keys hold most of the weight, many recent ones next to none
        w = torch.randn(c["B"], Hkv, st["L"], generator=g, device=dev).mul(2).exp()
        st["w"] = torch.where(torch.rand(w.shape, generator=g, device=dev) < 0.05, 0.0, w)
        st["w_out"] = torch.zeros(c["B"], Hkv, c["budget"] + 64, device=dev)
        st["ws"] = {}
    return st


# ------------------------------------------------------------- plain forms ---
def _pad(x, cu, L):
    """[tokens, H, d] -> fp32 [B, H, L, d], and which of the L rows of each sequence exist."""
    at = torch.arange(L, device=x.device)
    ok = at < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + at).clamp(max=x.shape[0] - 1).long()
    return x[rows].float().masked_fill(~ok[:, :, None, None], 0.0).transpose(1, 2), ok


def _place(cu, T):
    """Sequence and position of each packed row."""
    t = torch.arange(T, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b]


def _scores(st):
    c = st["case"]
    q, okq = _pad(st["Q"], st["cu_q"], st["Lq"])
    k, okk = _pad(st["K"], st["cu_k"], st["Lk"])
    v, _ = _pad(st["V"], st["cu_k"], st["Lk"])
    B, Hkv, Lk, d = k.shape
    G = c["Hq"] // Hkv
    s = (q.reshape(B, Hkv, G * st["Lq"], d) @ k.transpose(2, 3)).mul_(st["scale"]).view(B, Hkv, G, st["Lq"], Lk)
    see = okk[:, None, :] & okq[:, :, None]
    if c["causal"]:
        off = (st["cu_k"][1:] - st["cu_k"][:-1]) - (st["cu_q"][1:] - st["cu_q"][:-1])
        i, j = torch.arange(st["Lq"], device=s.device), torch.arange(Lk, device=s.device)
        see = see & (j <= i[:, None] + off[:, None, None])
    return q, k, v, s, see[:, None, None]


def plain_fwd(st):
    q, k, v, s, see = _scores(st)
    B, Hkv, G, Lq, Lk = s.shape
    s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * Lq, Lk) @ v).view(B, Hkv, G, Lq, -1) / l.masked_fill(l == 0, 1.0)
    lse = (m + l.log()).view(B, Hkv * G, Lq)
    b, i = _place(st["cu_q"], st["Q"].shape[0])
    return o.view(B, Hkv * G, Lq, -1)[b, :, i].to(torch.bfloat16), lse[b, :, i].t().contiguous()


def plain_bwd(st):
    q, k, v, s, see = _scores(st)
    B, Hkv, G, Lq, Lk = s.shape
    o, _ = _pad(st["O"], st["cu_q"], Lq)
    do, _ = _pad(st["dO"], st["cu_q"], Lq)
    lse, _ = _pad(st["LSE"].t()[:, :, None], st["cu_q"], Lq)
    rows = lambda x: x.reshape(B, Hkv, G * Lq, -1)
    p = rows(s.sub_(lse.masked_fill(lse == -math.inf, 0.0).view(B, Hkv, G, Lq, 1)).exp_().masked_fill_(~see, 0.0))
    dv = p.transpose(2, 3) @ rows(do)
    ds = (rows(do) @ v.transpose(2, 3)).sub_(rows((do * o).sum(-1, keepdim=True))).mul_(p).mul_(st["scale"])
    dk = ds.transpose(2, 3) @ rows(q)
    dq = (ds @ k).view(B, Hkv * G, Lq, -1)
    b, i = _place(st["cu_q"], st["Q"].shape[0])
    bk, j = _place(st["cu_k"], st["K"].shape[0])
    return dq[b, :, i].to(torch.bfloat16), dk[bk, :, j].to(torch.bfloat16), dv[bk, :, j].to(torch.bfloat16)


def _values(st):
    """The pools as the values they stand for."""
    if st["ks"] is None:
        return st["kc"], st["vc"]
    return st["kc"].float() * st["ks"][:, None, None], st["vc"].float() * st["vs"][:, None, None]


def _raw(x):
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def plain_append(st):
    b, i = _place(st["cu"], st["K"].shape[0])
    pos = st["lens"][b] + i
    page = st["case"]["page"]
    where = st["table"][b, (pos // page).long()].long(), pos.long() % page

    def put(pool, x, s):
        if s is not None:
            x = (x.float() / s[:, None]).clamp(-448, 448).to(E4M3)
        _raw(pool)[where[0], :, where[1]] = _raw(x)

    put(st["kc"], st["K"], st["ks"])
    put(st["vc"], st["V"], st["vs"])
    return _values(st)


def _read(pool, table, s):
    """The rows of each sequence's pages, in order: fp32 [B, Hkv, pages x page, d]."""
    x = _raw(pool)[table.clamp(min=0).long()].transpose(1, 2)
    x = (x.view(E4M3) if s is not None else x).float()
    B, Hkv, W, page, d = x.shape
    x = x.reshape(B, Hkv, W * page, d)
    return x if s is None else x * s[:, None, None]


def plain_decode(st):
    c = st["case"]
    k, v = _read(st["kc"], st["table"], st["ks"]), _read(st["vc"], st["table"], st["vs"])
    B, Hkv, L, d = k.shape
    ok = (torch.arange(L, device=k.device) < st["lens"][:, None])[:, None, None]
    q = st["Q"].float().view(B, Hkv, c["Hq"] // Hkv, d)
    s = (q @ k.transpose(2, 3)).mul_(st["scale"]).masked_fill_(~ok, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v.masked_fill(~ok.view(B, 1, L, 1), 0.0)) / l
    out = [o.view(B, c["Hq"], d).to(torch.bfloat16), (m + l.log()).view(B, c["Hq"])]
    if c["weights"]:
        torch.where(ok[:, :, 0], (p / l).sum(2), st["w"], out=st["w"])
        out.append(st["w"])
    return out


def plain_evict(st):
    c = st["case"]
    n, recent, keep, page = st["lens"], c["recent"], c["budget"], c["page"]
    B, Hkv, L = st["w"].shape
    at = torch.arange(L, device=n.device)
    old = at < (n - recent)[:, None]
    late = (at < n[:, None]) & ~old
    w = st["w"].masked_fill(~old[:, None], -math.inf)
    order = w.sort(dim=-1, descending=True, stable=True)[1]  # equal weights: the lowest position first
    rank = torch.empty_like(order).scatter_(-1, order, at.expand(B, Hkv, L))
    stay = ((rank < keep - recent) & old[:, None]) | late[:, None]
    kept = (~stay).to(torch.uint8).sort(dim=-1, stable=True)[1][..., :keep]  # in their order
    if L < keep:
        kept = torch.nn.functional.pad(kept, (0, keep - L))
    left = n.clamp(max=keep)
    row = torch.arange(keep, device=n.device)
    live = (row < left[:, None])[:, None].expand(B, Hkv, keep)
    b, h = torch.arange(B, device=n.device)[:, None, None], torch.arange(Hkv, device=n.device)[:, None]
    src = st["table"][b, kept // page].clamp(min=0).long()
    dst = st["table_out"][:, None, row // page].long().expand(B, Hkv, keep)

    def move(pool):
        x = _raw(pool)
        x[dst, h, row % page] = torch.where(live[..., None], x[src, h, kept % page], x[dst, h, row % page])

    move(st["kc"])
    move(st["vc"])
    st["w_out"].zero_()
    st["w_out"][..., :keep] = st["w"].gather(-1, kept).masked_fill(~live, 0.0)
    return [kept.masked_fill(~live, -1).to(torch.int32), left.to(torch.int32), st["w_out"], *_values(st)]


PLAIN = dict(fwd=plain_fwd, bwd=plain_bwd, append=plain_append, decode=plain_decode, evict=plain_evict)


# -------------------------------------------------------------- own calls ---
def _ws(st, size, *sizes):
    """The workspace that a program keeps next to its buffers."""
    if "t" not in st["ws"]:
        st["ws"]["t"] = torch.empty(max(1, size(*sizes)), dtype=torch.uint8, device="cuda")
    return st["ws"]["t"]


def own_fwd(st, fa):
    c = st["case"]
    ws = _ws(st, fa.fwd_packed_workspace_size, c["B"], st["Q"].shape[0], c["Hq"], c["Hkv"], c["d"])
    return fa.fwd_packed(st["Q"], st["K"], st["V"], st["cu_q"], st["cu_k"], mask="causal" if c["causal"] else "none",
                         scale=st["scale"], workspace=ws)


def own_bwd(st, fa):
    c = st["case"]
    ws = _ws(st, fa.bwd_packed_workspace_size, c["B"], st["Q"].shape[0], st["K"].shape[0], c["Hq"], c["Hkv"], c["d"])
    return fa.bwd_packed(st["Q"], st["K"], st["V"], st["O"], st["dO"], st["LSE"], st["cu_q"], st["cu_k"],
                         mask="causal" if c["causal"] else "none", scale=st["scale"], workspace=ws)


def own_append(st, fa):
    fa.paged_append(st["K"], st["V"], st["cu"], st["lens"], st["kc"], st["vc"], st["table"], k_scale=st["ks"],
                    v_scale=st["vs"])
    return _values(st)


def own_decode(st, fa):
    c = st["case"]
    ws = _ws(st, fa.paged_decode_workspace_size, c["B"], c["Hq"], c["Hkv"], c["d"], st["L"], c["weights"])
    o, lse = fa.paged_decode(st["Q"], st["kc"], st["vc"], st["table"], st["lens"], scale=st["scale"], k_scale=st["ks"],
                             v_scale=st["vs"], weights=st["w"], workspace=ws)
    return [o, lse] + ([st["w"]] if c["weights"] else [])


def own_evict(st, fa):
    c = st["case"]
    kept, left = fa.paged_evict(st["w"], st["kc"], st["vc"], st["table"], st["lens"], st["table_out"], c["budget"],
                                c["recent"], st["w_out"])
    return [kept, left, st["w_out"], *_values(st)]


OWN = dict(fwd=own_fwd, bwd=own_bwd, append=own_append, decode=own_decode, evict=own_evict)


def run(state):
    if own:
        import exact_io_aware_65_b200 as fa

        return OWN[state["case"]["op"]](state, fa)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ---
def work(case):
    c = case
    n, held = lengths(c)
    T, d, Hkv = sum(n), c["d"], c["Hkv"]
    if c["op"] in ("fwd", "bwd"):
        nk = [a + b for a, b in zip(n, held)]
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(n, nk)) if c["causal"] else sum(a * b for a, b in zip(n, nk))
        q, k, lse = T * c["Hq"] * d * 2, sum(nk) * Hkv * d * 2, T * c["Hq"] * 4
        if c["op"] == "fwd":
            return dict(bytes=2 * q + 2 * k + lse, flops=4 * d * pairs * c["Hq"])
        return dict(bytes=4 * q + 4 * k + lse, flops=10 * d * pairs * c["Hq"])
    size = 1 if c["e4m3"] else 2
    row = Hkv * d
    if c["op"] == "append":
        pool = sum(-(-(a + b) // c["page"]) * c["page"] for a, b in zip(n, held)) * row
        values = 2 * pool * (1 + 4) if c["e4m3"] else 0  # the 8-bit pools are returned as values
        return dict(bytes=2 * T * row * (2 + size) + values, flops=2 * T * row)
    if c["op"] == "decode":
        b = 2 * T * row * size + c["B"] * c["Hq"] * (4 * d + 4) + (T * Hkv * 4 if c["weights"] else 0)
        return dict(bytes=b, flops=4 * T * c["Hq"] * d)
    left = sum(min(a, c["budget"]) for a in n)
    pages = sum(-(-a // c["page"]) for a in n) + c["B"] * -(-c["budget"] // c["page"])
    values = 2 * pages * c["page"] * row * (1 + 4) if c["e4m3"] else 0
    return dict(bytes=4 * left * row * size + T * Hkv * 4 + c["B"] * Hkv * (8 * c["budget"] + 256) + values, flops=T * Hkv)


# ------------------------------------------------------- definitions, 64 bits ---
def _e4m3_nearest(x):
    """The value of the 8-bit type (4 exponent bits, 3 of fraction) next to each x, ties to even."""
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _heads(st, b):
    q0, q1, k0, k1 = (int(st[n][b + e]) for n in ("cu_q", "cu_k") for e in (0, 1))
    return q0, q1, k0, k1


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    D = torch.float64
    Hkv, d = c["Hkv"], c["d"]
    if c["op"] in ("fwd", "bwd"):
        G = c["Hq"] // Hkv
        outs = dict(O=torch.zeros(st["Q"].shape, dtype=D, device="cuda"),
                    LSE=torch.zeros(c["Hq"], st["Q"].shape[0], dtype=D, device="cuda"))
        grads = [torch.zeros(st[n].shape, dtype=D, device="cuda") for n in "QKV"]
        for b in range(c["B"]):
            q0, q1, k0, k1 = _heads(st, b)
            hide = torch.zeros(q1 - q0, k1 - k0, dtype=torch.bool, device="cuda")
            if c["causal"]:
                hide = torch.ones_like(hide).triu((k1 - k0) - (q1 - q0) + 1)
            for h in range(c["Hq"]):
                q, k, v = st["Q"][q0:q1, h].to(D), st["K"][k0:k1, h // G].to(D), st["V"][k0:k1, h // G].to(D)
                logits = torch.einsum("id,jd->ij", q, k) * st["scale"]
                logits[hide] = -math.inf
                lse = torch.logsumexp(logits, 1)
                p = torch.exp(logits - lse[:, None])
                o = torch.einsum("ij,jd->id", p, v)
                outs["O"][q0:q1, h], outs["LSE"][h, q0:q1] = o, lse
                if c["op"] == "bwd":
                    do = st["dO"][q0:q1, h].to(D)
                    dp = torch.einsum("id,jd->ij", do, v)
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) * st["scale"]
                    grads[0][q0:q1, h] = torch.einsum("ij,jd->id", ds, k)
                    grads[1][k0:k1, h // G] += torch.einsum("ij,id->jd", ds, q)
                    grads[2][k0:k1, h // G] += torch.einsum("ij,id->jd", p, do)
        return tuple(grads) if c["op"] == "bwd" else (outs["O"], outs["LSE"])
    page, table = c["page"], st["table"].tolist()
    n, held = lengths(c)
    if c["op"] == "append":
        outs = [x.to(D) * (1 if s is None else s.to(D)[:, None, None])
                for x, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"]))]
        at = 0
        for b in range(c["B"]):
            for i in range(n[b]):
                p = held[b] + i
                for o, x, s in zip(outs, (st["K"], st["V"]), (st["ks"], st["vs"])):
                    x = x[at].to(D)
                    if s is not None:
                        x = _e4m3_nearest(x / s.to(D)[:, None]) * s.to(D)[:, None]
                    o[table[b][p // page], :, p % page] = x
                at += 1
        return outs
    if c["op"] == "decode":
        G = c["Hq"] // Hkv
        O, LSE = torch.zeros(c["B"], c["Hq"], d, dtype=D, device="cuda"), torch.zeros(c["B"], c["Hq"], dtype=D, device="cuda")
        W = torch.zeros(c["B"], Hkv, st["L"], dtype=D, device="cuda")
        for b in range(c["B"]):
            rows = []
            for pool, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
                x = torch.cat([pool[t] for t in table[b][:-(-n[b] // page)]], dim=1)[:, :n[b]].to(D)
                rows.append(x if s is None else x * s.to(D)[:, None, None])
            for h in range(c["Hq"]):
                logits = (rows[0][h // G] @ st["Q"][b, h].to(D)) * st["scale"]
                LSE[b, h] = torch.logsumexp(logits, 0)
                p = torch.exp(logits - LSE[b, h])
                O[b, h] = p @ rows[1][h // G]
                W[b, h // G, :n[b]] += p
        return [O, LSE] + ([W] if c["weights"] else [])
    return None  # eviction only selects and moves
