"""What the attention layers' operators are measured on: the per-head norm with the position
rotation, the append to a paged cache, and the attention over that cache.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` makes one pass
through the operator, either in elementary torch operations in fp32 (``own = False``) or through
the library's entry points (``own = True``), and ``exact`` gives the same outputs in 64 bits.

    rope_fwd     norm of every head of q and k, and the rotation by position
    rope_train   the same with its backward: outputs and every gradient
    append       new tokens' q normed and rotated, k normed and rotated into the pages, v copied there
    attn         attention of the new tokens of N sequences over their pages
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}
EPS = 1e-6

# 12 requests of a packed prefill batch, 8192 tokens together
_PACKED = "2500,1536,1024,900,700,512,413,300,150,90,40,27"


def _rope(name, op, B, T, Hq, Hk, d, rot, dtype="bf16", interleaved=False, norm=True, start=0, base=10000.0, amp=1.0,
          token_major=True):
    c = {"op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot, "dtype": dtype, "interleaved": interleaved,
         "norm": norm, "start": start, "base": base, "amp": amp, "token_major": token_major}
    return dict(c, name=name) if name else c


def _append(name, new, past, Hq, Hk, dk, dv, rot, page, dtype="bf16", interleaved=False, norm=True, base=10000.0, amp=1.0):
    c = {"op": "append", "new": new, "past": past, "Hq": Hq, "Hk": Hk, "dk": dk, "dv": dv, "rot": rot, "page": page,
         "dtype": dtype, "interleaved": interleaved, "norm": norm, "base": base, "amp": amp}
    return dict(c, name=name) if name else c


def _attn(name, new, past, Hq, Hk, dk, dv, page, window=0, lse=False):
    c = {"op": "attn", "new": new, "past": past, "Hq": Hq, "Hk": Hk, "dk": dk, "dv": dv, "page": page, "window": window,
         "lse": lse}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one stream of a chat server: one token at a far position
        _rope("rope_fwd_1x40x128", "rope_fwd", 1, 1, 32, 8, 128, 128, start=1000003),
        # an 8K prompt of a model with half-rotated, interleaved heads and a context scaled past its training
        _rope("rope_fwd_8192x40x128", "rope_fwd", 1, 8192, 32, 8, 128, 64, interleaved=True, base=500000.0, amp=1.2079),
        # a training step of the norm and the rotation on 8K tokens
        _rope("rope_train_8192x40x128", "rope_train", 1, 8192, 32, 8, 128, 128),
        # a small fp32 model: ragged length, heads off the vector width, head-major rows
        _rope("rope_train_fp32_2x777x6x90", "rope_train", 2, 777, 5, 1, 90, 42, dtype="fp32", token_major=False),
        # a decode batch of 256 sequences, one new token each
        _append("append_256x1", "256x1", "256~1..255", 32, 8, 128, 128, 128, 64),
        # a prefill batch of mixed requests, resumed from cached prefixes that end inside pages
        _append("append_packed_8192", _PACKED, "12~0..1000", 32, 8, 128, 128, 64, 16, interleaved=True),
        # one stream: one token over 8K cached ones
        _attn("attn_decode_1x8192", "1x1", "8191", 32, 8, 128, 128, 64),
        # a decode batch of 256 sequences of very different lengths
        _attn("attn_decode_256x16384", "256x1", "256~1..16383", 32, 8, 128, 128, 64),
        # four drafted tokens of each of 32 sequences checked at once, heads of 64, a window, small pages
        _attn("attn_verify_32x4", "32x4", "32~100..4000", 32, 4, 64, 64, 16, window=1024, lse=True),
        # an 8K prompt with nothing cached
        _attn("attn_prefill_8192", "8192", "0", 32, 8, 128, 128, 64),
        # mixed requests in one packed batch, resumed from cached prefixes
        _attn("attn_packed_8192", _PACKED, "12~0..4000", 32, 8, 128, 128, 64, lse=True),
        # the next 4K tokens of a 64K document
        _attn("attn_chunk_4096_of_65536", "4096", "61440", 32, 8, 128, 128, 512),
    ]


def _lens(text):
    """"3,0,5": these; "4x7": four of 7; "4~1..9": four spread between 1 and 9."""
    if "~" in text:
        n, r = text.split("~")
        lo, hi = map(int, r.split(".."))
        return [lo + int((hi - lo + 1) * ((s * 0.6180339887498949 + 0.37) % 1.0)) for s in range(int(n))]
    if "x" in text:
        n, v = text.split("x")
        return [int(v)] * int(n)
    return [int(v) for v in text.split(",")]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_train", "rope_train", "append", "append", "attn", "attn", "attn", "attn"])
    interleaved, norm = rng.random() < 0.5, rng.random() < 0.8
    base, amp = rng.choice([(10000.0, 1.0), (500000.0, 1.0), (10000.0, 1.1386)])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op.startswith("rope"):
        d = rng.choice([64, 128, 128, 16 * _logint(rng, 1, 16), 2 * _logint(rng, 1, 128)])
        rot = rng.choice([d, d, 2 * rng.randint(0, d // 2), 16 * (d // 32)])
        Hk = _logint(rng, 1, 16)
        most = 8192 * 40 * 128 // (2 if dtype == "fp32" else 1)
        T = _logint(rng, 1, max(1, min(32768, most // ((G + 1) * Hk * d))))
        B = max(1, min(_logint(rng, 1, 8), most // ((G + 1) * Hk * d * T)))
        return _rope(None, op, B, T, G * Hk, Hk, d, rot, dtype=dtype, interleaved=interleaved, norm=norm,
                     start=rng.choice([0, 0, _logint(rng, 1, 1000000)]), base=base, amp=amp, token_major=rng.random() < 0.5)
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (128, 64), (64, 128)])
    page = rng.choice([16, 32, 64, 64, 128, 512])
    Hk = _logint(rng, 1, 16)
    Hq = G * Hk
    if op == "append":
        N = _logint(rng, 1, 256)
        most = max(N, 8192 * 48 * 128 // ((Hq + 2 * Hk) * 128) // (2 if dtype == "fp32" else 1))
        T = max(N, _logint(rng, 1, most))
        new, past = _cuts(rng, T, N), [rng.randint(0, 255) for _ in range(N)]
        return _append(None, ",".join(map(str, new)), ",".join(map(str, past)), Hq, Hk, dk, dv,
                       rng.choice([dk, dk // 2, 0]), page, dtype=dtype, interleaved=interleaved, norm=norm, base=base, amp=amp)
    kind = rng.choice(["decode", "decode", "few", "prefill", "packed"])
    window = rng.choice([0, 0, 0, _logint(rng, 1, 4096)])
    N = {"decode": _logint(rng, 1, 256), "few": _logint(rng, 1, 64), "prefill": _logint(rng, 1, 4),
         "packed": _logint(rng, 2, 32)}[kind]
    if kind == "decode":
        new = [1] * N
    elif kind == "few":
        new = [rng.randint(2, 8)] * N
    elif kind == "prefill":
        new = [_logint(rng, 16, 8192 // N)] * N
    else:
        new = _cuts(rng, _logint(rng, N, 8192), N)
    keys = 8192 * 256 * 8 // (N * Hk) * 64 // max(dk, dv)                     # a sequence's share of the cache
    top = max(1, min(65536 if max(new) == 1 or N == 1 else 16384, keys))
    past = [_logint(rng, 1, top) - 1 for _ in range(N)]
    pairs = 4096 * 32 * 63488                                                 # those of the longest listed case
    while Hq * sum(n * (p + n) for n, p in zip(new, past)) > pairs:
        new = [max(1, n // 2) for n in new]
    return _attn(None, ",".join(map(str, new)), ",".join(map(str, past)), Hq, Hk, dk, dv, page, window=window,
                 lse=rng.random() < 0.3)


def _cuts(rng, T, N):
    """T tokens over N sequences, ragged; some may be empty."""
    cuts = sorted(rng.randint(0, T) for _ in range(N - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


# ---- inputs -----------------------------------------------------------------------------------

def _inv_freq(rot, base, dev):
    """Frequencies of the rotated pairs in fp32, as a model's buffer holds them."""
    if rot == 0:
        return None
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)
    c, st = case, {"case": case}
    Hq, Hk = c["Hq"], c["Hk"]
    if c["op"].startswith("rope"):
        dt, B, T, d = _DT[c["dtype"]], c["B"], c["T"], c["d"]
        if c["token_major"]:     # q and k are slices of one projection's output
            qkv = randn(B, T, Hq + 2 * Hk, d).to(dt)
            st["q"], st["k"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
        else:
            st["q"], st["k"] = randn(B, Hq, T, d).to(dt), randn(B, Hk, T, d).to(dt)
        st["wq"] = 1.0 + 0.1 * randn(d) if c["norm"] else None
        st["wk"] = 1.0 + 0.1 * randn(d) if c["norm"] else None
        st["inv_freq"] = _inv_freq(c["rot"], c["base"], dev)
        st["pos"] = (c["start"] + torch.arange(T, dtype=torch.int32, device=dev)).repeat(B, 1)
        if c["op"] == "rope_train":
            if c["token_major"]:
                st["dq"], st["dk"] = randn(B, T, Hq, d).to(dt).transpose(1, 2), randn(B, T, Hk, d).to(dt).transpose(1, 2)
            else:
                st["dq"], st["dk"] = randn(B, Hq, T, d).to(dt), randn(B, Hk, T, d).to(dt)
        return st
    new, past = _lens(c["new"]), _lens(c["past"])
    N, T, page, dk, dv = len(new), sum(new), c["page"], c["dk"], c["dv"]
    kv = [n + p for n, p in zip(new, past)]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(N, max(need), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    st.update(new=new, kv=kv, table=table, kv_lens=torch.tensor(kv, dtype=torch.int32, device=dev))
    st["same"] = len(set(new)) == 1                  # sequences of one length: [N,H,n,d], else packed [H,T,d]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu_host"] = cu
    st["cu"] = None if st["same"] else torch.tensor(cu, dtype=torch.int32, device=dev)
    st["k_cache"] = torch.empty(pages, Hk, page, dk, dtype=torch.bfloat16, device=dev)
    st["v_cache"] = torch.empty(pages, Hk, page, dv, dtype=torch.bfloat16, device=dev)
    for t in (st["k_cache"], st["v_cache"]):
        t.normal_(generator=g)
    heads = (lambda t: t.unflatten(0, (N, new[0])).transpose(1, 2)) if st["same"] else (lambda t: t.transpose(0, 1))
    if c["op"] == "append":
        dt = _DT[c["dtype"]]
        row = randn(T, Hq * dk + Hk * (dk + dv)).to(dt)          # q, k and v of a token side by side
        q, k, v = row.split([Hq * dk, Hk * dk, Hk * dv], 1)
        st["q"], st["k"], st["v"] = (heads(t.unflatten(1, (h, -1))) for t, h in ((q, Hq), (k, Hk), (v, Hk)))
        st["wq"] = 1.0 + 0.1 * randn(dk) if c["norm"] else None
        st["wk"] = 1.0 + 0.1 * randn(dk) if c["norm"] else None
        st["inv_freq"] = _inv_freq(c["rot"], c["base"], dev)
        return st
    st["q"] = heads((2.0 * randn(T, Hq, dk)).to(torch.bfloat16))  # scores of deviation 2
    return st


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"rope_fwd": _plain_rope, "rope_train": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](state)


def _own(op, s):
    import gated_delta_rule_78_amd as kda
    c = s["case"]
    if op == "attn":
        r = kda.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], cu_seqlens=s["cu"],
                           window=c["window"], return_lse=c["lse"])
        return {"o": r[0], "lse": r[1]} if c["lse"] else {"o": r}
    kw = dict(interleaved=c["interleaved"], rope_scale=c["amp"], q_weight=s["wq"], k_weight=s["wk"], norm=c["norm"], eps=EPS)
    if op == "append":
        q = kda.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["inv_freq"],
                          cu_seqlens=s["cu"], **kw)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    q, k = kda.head_rope_fwd(s["q"], s["k"], s["inv_freq"], s["pos"], **kw)
    out = {"q": q, "k": k}
    if op == "rope_train":
        out.update(zip(("dq", "dk", "dwq", "dwk"),
                       kda.head_rope_bwd(s["q"], s["k"], s["inv_freq"], s["dq"], s["dk"], s["pos"], **kw)))
    return {n: t for n, t in out.items() if t is not None}


# ---- the plain forms: fp32, elementary operations ---------------------------------------------

def _pairs(x, rot, interleaved):
    """The rotated channels of x as their pairs' two members."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _turn(x, cos, sin, rot, interleaved):
    """x with its first rot channels turned: (a, b) -> (a cos - b sin, b cos + a sin)."""
    if rot == 0:
        return x
    a, b = _pairs(x, rot, interleaved)
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _angles(pos, inv_freq, amp):
    """cos and sin of position times frequency, from a 64-bit product: far positions lose the angle in fp32."""
    if inv_freq is None:
        return None, None
    th = pos.double()[..., None] * inv_freq.double()
    return (th.cos() * amp).float(), (th.sin() * amp).float()


def _norm_turn(x, w, c, cos, sin):
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _turn(x, cos, sin, c["rot"], c["interleaved"])


def _plain_rope(s):
    c = s["case"]
    dt = s["q"].dtype
    cos, sin = _angles(s["pos"][:, None], s["inv_freq"], c["amp"])
    out = {n: _norm_turn(s[n], s[w], c, cos, sin).to(dt) for n, w in (("q", "wq"), ("k", "wk"))}
    if c["op"] == "rope_fwd":
        return out
    for n, w in (("q", "wq"), ("k", "wk")):
        dy = _turn(s["d" + n].float(), cos, -sin if sin is not None else None, c["rot"], c["interleaved"])
        if c["norm"]:
            x = s[n].float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            xh = x * r
            out["dw" + n] = (dy * xh).sum((0, 1, 2))
            t = dy * s[w]
            dy = r * (t - xh * (t * xh).mean(-1, keepdim=True))
        out["d" + n] = dy.to(dt)
    return out


def _rows(s, t):
    """Heads' rows in packed order, [T, H, d]."""
    return t.transpose(1, 2).flatten(0, 1) if s["same"] else t.transpose(0, 1)


def _unrows(s, t):
    return t.unflatten(0, (len(s["new"]), s["new"][0])).transpose(1, 2) if s["same"] else t.transpose(0, 1)


def _plain_append(s):
    c = s["case"]
    N, T, page = len(s["new"]), sum(s["new"]), c["page"]
    dev = s["q"].device
    if s["cu"] is None:
        seq = torch.arange(N, device=dev).repeat_interleave(s["new"][0])
        first = torch.arange(N, device=dev) * s["new"][0]
        n = s["new"][0]
    else:
        seq = torch.searchsorted(s["cu"][1:].contiguous(), torch.arange(T, dtype=torch.int32, device=dev), right=True)
        first = s["cu"][:-1].long()
        n = (s["cu"][1:] - s["cu"][:-1]).long()[seq]
    pos = s["kv_lens"].long()[seq] - n + torch.arange(T, device=dev) - first[seq]
    where = s["table"].long()[seq, pos // page], pos % page
    cos, sin = _angles(pos[:, None], s["inv_freq"], c["amp"])
    q = _norm_turn(_rows(s, s["q"]), s["wq"], c, cos, sin).to(torch.bfloat16)
    s["k_cache"][where[0], :, where[1]] = _norm_turn(_rows(s, s["k"]), s["wk"], c, cos, sin).to(torch.bfloat16)
    s["v_cache"][where[0], :, where[1]] = _rows(s, s["v"]).to(torch.bfloat16)
    return {"q": _unrows(s, q), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    """Sequence by sequence over its gathered keys, blocks of queries against all keys."""
    c = s["case"]
    Hq, Hk, dk, dv, page = c["Hq"], c["Hk"], c["dk"], c["dv"], c["page"]
    G, T = Hq // Hk, sum(s["new"])
    dev = s["q"].device
    q = _rows(s, s["q"]).float() * (1.0 / math.sqrt(dk))
    o = torch.empty(T, Hq, dv, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(T, Hq, device=dev)
    for i, n in enumerate(s["new"]):
        if n == 0:
            continue
        kv, t0 = s["kv"][i], s["cu_host"][i]
        own_pages = s["table"][i, :-(-kv // page)].long()
        K = s["k_cache"][own_pages].transpose(0, 1).reshape(Hk, -1, dk)[:, :kv].float()
        V = s["v_cache"][own_pages].transpose(0, 1).reshape(Hk, -1, dv)[:, :kv].float()
        step = max(1, (1 << 29) // (Hq * kv))
        key = torch.arange(kv, device=dev)
        for a in range(0, n, step):
            b = min(n, a + step)
            pos = torch.arange(kv - n + a, kv - n + b, device=dev)[:, None]
            hidden = key > pos
            if c["window"]:
                hidden |= key <= pos - c["window"]
            qb = q[t0 + a:t0 + b].unflatten(1, (Hk, G)).transpose(0, 1).reshape(Hk, (b - a) * G, dk)
            x = torch.matmul(qb, K.transpose(1, 2)).view(Hk, b - a, G, kv)
            x.masked_fill_(hidden[None, :, None], float("-inf"))
            m = x.amax(-1, keepdim=True)
            x.sub_(m).exp_()
            l = x.sum(-1, keepdim=True)
            r = torch.matmul(x.view(Hk, -1, kv), V).view(Hk, b - a, G, dv) / l
            o[t0 + a:t0 + b] = r.transpose(0, 1).reshape(b - a, Hq, dv)
            lse[t0 + a:t0 + b] = (m + l.log()).squeeze(-1).transpose(0, 1).reshape(b - a, Hq)
    out = {"o": _unrows(s, o)}
    if c["lse"]:
        out["lse"] = _unrows(s, lse)
    return out


# ---- the definitions in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rope"):
        return _exact_rope(s)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)


def _exact_rows(x, w, c, rot, d, pos, inv_freq):
    """x[..., d] normed by its definition and multiplied, pair by pair, as complex numbers."""
    if c["norm"]:
        x = w * x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
    if not rot:
        return x
    th = pos.double().unsqueeze(-1) * inv_freq.double()
    e = torch.polar(torch.full_like(th, c["amp"]), th)
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
    z = torch.complex(x[..., ia], x[..., ib]) * e
    out = torch.empty_like(x)
    out[..., ia], out[..., ib], out[..., rot:] = z.real, z.imag, x[..., rot:]
    return out


def _exact_rope(s):
    """The formula through 64-bit automatic differentiation."""
    c = s["case"]
    leaf = {n: s[n].double().requires_grad_() for n in ("q", "k", "wq", "wk") if s[n] is not None}
    out = {}
    for n in ("q", "k"):
        out[n] = _exact_rows(leaf[n], leaf.get("w" + n), c, c["rot"], c["d"], s["pos"][:, None], s["inv_freq"])
    if c["op"] == "rope_train":
        loss = (out["q"] * s["dq"].double()).sum() + (out["k"] * s["dk"].double()).sum()
        for n, gr in zip(leaf, torch.autograd.grad(loss, list(leaf.values()))):
            out["d" + n] = gr
    return {n: t.detach() for n, t in out.items()}


def _exact_append(s):
    c = s["case"]
    q, k, v = (_rows(s, s[n]).double() for n in ("q", "k", "v"))
    wq, wk = (w.double() if w is not None else None for w in (s["wq"], s["wk"]))
    K, V, qo = s["k_cache"].double(), s["v_cache"].double(), torch.empty_like(q)
    table = s["table"].tolist()
    for i, n in enumerate(s["new"]):
        t0, p0 = s["cu_host"][i], s["kv"][i] - n
        if n == 0:
            continue
        pos = torch.arange(p0, p0 + n, device=q.device)[:, None]
        qo[t0:t0 + n] = _exact_rows(q[t0:t0 + n], wq, c, c["rot"], c["dk"], pos, s["inv_freq"])
        kr = _exact_rows(k[t0:t0 + n], wk, c, c["rot"], c["dk"], pos, s["inv_freq"])
        at = p0
        while at < p0 + n:                           # the part of the run inside one page
            end = min(p0 + n, (at // c["page"] + 1) * c["page"])
            pg, r = table[i][at // c["page"]], at % c["page"]
            K[pg, :, r:r + end - at] = kr[at - p0:end - p0].transpose(0, 1)
            V[pg, :, r:r + end - at] = v[t0 + at - p0:t0 + end - p0].transpose(0, 1)
            at = end
    return {"q": _unrows(s, qo), "k_cache": K, "v_cache": V}


def _exact_attn(s):
    """One key head at a time over each sequence: weights exp(x) by their definition, shifted by the row's largest."""
    c = s["case"]
    G, dk, dv, page = c["Hq"] // c["Hk"], c["dk"], c["dv"], c["page"]
    q = _rows(s, s["q"])
    o = torch.zeros(q.shape[0], c["Hq"], dv, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[0], c["Hq"], dtype=torch.float64, device=q.device)
    if sum(n * k for n, k in zip(s["new"], s["kv"])) * c["Hq"] * (dk + dv) > 1 << 43:
        return None                                  # over some 20 seconds
    for i, n in enumerate(s["new"]):
        kv, t0 = s["kv"][i], s["cu_host"][i]
        pg = s["table"][i, :-(-kv // page)].long()
        for h in range(c["Hk"] if n else 0):
            K = s["k_cache"][pg, h].reshape(-1, dk)[:kv].double()
            V = s["v_cache"][pg, h].reshape(-1, dv)[:kv].double()
            step = max(1, (1 << 27) // (G * kv))
            for a in range(0, n, step):
                b = min(n, a + step)
                j = torch.arange(kv, device=q.device)
                p = torch.arange(a, b, device=q.device)[:, None] + kv - n
                seen = (j <= p) & ((j > p - c["window"]) if c["window"] else torch.ones_like(j, dtype=torch.bool))
                x = q[t0 + a:t0 + b, h * G:(h + 1) * G].double() @ K.t() / dk ** 0.5
                x = torch.where(seen[:, None], x, torch.full_like(x, float("-inf")))
                lse_b = torch.logsumexp(x, -1)
                o[t0 + a:t0 + b, h * G:(h + 1) * G] = torch.exp(x - lse_b.unsqueeze(-1)) @ V
                lse[t0 + a:t0 + b, h * G:(h + 1) * G] = lse_b
    out = {"o": _unrows(s, o)}
    if c["lse"]:
        out["lse"] = _unrows(s, lse)
    return out


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    c = case
    if c["op"].startswith("rope"):
        n = c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["d"]
        e = _BYTES[c["dtype"]]
        small = c["B"] * c["T"] * 4 + 2 * c["rot"] + (8 * c["d"] if c["norm"] else 0)
        per = 5 * c["norm"] + 3 * c["rot"] / c["d"]
        if c["op"] == "rope_fwd":
            return {"bytes": 2 * n * e + small, "flops": n * per}
        # the outputs' gradients in, the inputs' out
        return {"bytes": 4 * n * e + small + (8 * c["d"] if c["norm"] else 0), "flops": n * (3 * per + 4 * c["norm"])}
    new, past = _lens(c["new"]), _lens(c["past"])
    T, N, Hq, Hk, dk, dv = sum(new), len(new), c["Hq"], c["Hk"], c["dk"], c["dv"]
    if c["op"] == "append":
        n = T * (Hq * dk + Hk * (dk + dv))
        return {"bytes": n * (_BYTES[c["dtype"]] + 2) + 12 * N,
                "flops": T * (Hq + Hk) * dk * (5 * c["norm"] + 3 * c["rot"] / dk)}
    w = c["window"]
    pairs = keys = tables = 0
    for n, p in zip(new, past):
        if n:
            if not w:
                pairs += n * p + n * (n + 1) // 2
            else:
                full = max(0, min(n, n + p - w))                              # queries whose window is whole
                a, b = p + 1, p + n - full                                    # the others see 1 .. their position
                pairs += full * w + (max(0, b - a + 1) * (a + b)) // 2
            keys += min(p + n, n + w - 1) if w else p + n
            tables += -(-(p + n) // c["page"])
    return {"bytes": T * Hq * (2 * (dk + dv) + 4 * c["lse"]) + keys * Hk * 2 * (dk + dv) + 4 * tables + 12 * N,
            "flops": pairs * Hq * 2 * (dk + dv)}
