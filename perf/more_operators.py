"""Measured cases of the attention blocks that stand between recurrent ones: norm and position rotation of every query and key
head (prompts, training, and tokens written into a paged cache), causal attention over prompts and packed documents with
grouped heads, forward and backward, and a single token's attention over the cache. Each case has a plain form (elementary
torch operations in 32 bits), the framework's own call, and the definition in 64 bits."""
import math
import random

import torch

own = False

EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # queries and keys of an 8192-token prompt, four query heads to a key head
        {"name": "rope prompt", "op": "rope", "batch": 1, "tokens": 8192, "docs": 0, "heads": 16, "kv_heads": 4, "dim": 128, "rotary": 128,
         "interleaved": False, "theta": 1e6, "train": False},
        # a training step at the 2 x 4096 training shape, half of each head rotated, both directions
        {"name": "rope train", "op": "rope", "batch": 2, "tokens": 4096, "docs": 0, "heads": 16, "kv_heads": 16, "dim": 128, "rotary": 64,
         "interleaved": False, "theta": 1e4, "train": True},
        # four sequences' next tokens, far into their texts, written into a paged cache: latency counts
        {"name": "store token", "op": "store", "batch": 4, "tokens": 1, "docs": 0, "heads": 16, "kv_heads": 4, "dim": 128, "rotary": 128,
         "interleaved": False, "theta": 1e6, "page": 64, "longest": 8192},
        # packed prompts enter the cache, lengths as they come
        {"name": "store prompts", "op": "store", "batch": 1, "tokens": 4093, "docs": 7, "heads": 16, "kv_heads": 4, "dim": 128, "rotary": 128,
         "interleaved": False, "theta": 1e6, "page": 64, "longest": 0},
        # one short prompt: latency counts
        {"name": "attention short", "op": "attention", "batch": 1, "tokens": 77, "docs": 0, "heads": 16, "kv_heads": 4, "dim": 128, "causal": True, "train": False},
        # one long prompt
        {"name": "attention prompt", "op": "attention", "batch": 1, "tokens": 8192, "docs": 0, "heads": 16, "kv_heads": 4, "dim": 128, "causal": True, "train": False},
        # sequences of an odd length that see themselves whole, small heads
        {"name": "attention both ways", "op": "attention", "batch": 8, "tokens": 1001, "docs": 0, "heads": 16, "kv_heads": 8, "dim": 64, "causal": False, "train": False},
        # a training step over 12 documents packed in one row
        {"name": "attention documents", "op": "attention", "batch": 1, "tokens": 16384, "docs": 12, "heads": 16, "kv_heads": 4, "dim": 128, "causal": True, "train": True},
        # a training step at the 2 x 4096 training shape, both directions
        {"name": "attention train", "op": "attention", "batch": 2, "tokens": 4096, "docs": 0, "heads": 16, "kv_heads": 16, "dim": 128, "causal": True, "train": True},
        # the next token of one sequence of 32768
        {"name": "step one", "op": "step", "batch": 1, "heads": 16, "kv_heads": 4, "dim": 128, "page": 64, "longest": 32768},
        # the next tokens of a serving batch, lengths as they come, some rows only padding
        {"name": "step many", "op": "step", "batch": 120, "heads": 16, "kv_heads": 4, "dim": 128, "page": 64, "longest": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "store", "attention", "attention", "attention", "step", "step"])
    kv = rng.choice([1, 2, 4, 4, 8, 16])
    heads = kv * rng.choice([g for g in (1, 2, 4, 7, 8) if kv * g <= 32])
    dim = rng.choice([64, 128, 128])
    rope = {"rotary": rng.choice([dim, dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.3, "theta": rng.choice([1e4, 5e5, 1e6])}
    if op == "step":
        longest = _log(rng, 1, 32768)
        most = max(1, 2000000 // (longest * kv))
        return {"op": op, "batch": min(_log(rng, 1, 160), most), "heads": heads, "kv_heads": kv, "dim": dim, "page": rng.choice([16, 64, 64, 100, 256]), "longest": longest}
    docs = rng.choice([0, 0, 1, 3, 9])
    batch = 1 if docs else rng.choice([1, 2, 3])
    if op == "rope":
        most = min(8192, 134217728 // (heads * dim * 8)) // batch
        return {"op": op, "batch": batch, "tokens": max(docs, _log(rng, 1, most)), "docs": docs, "heads": heads, "kv_heads": kv, "dim": dim, **rope, "train": rng.random() < 0.5}
    if op == "store":
        single = rng.random() < 0.5
        batch, docs = (_log(rng, 1, 160), 0) if single else (batch, docs)
        tokens = 1 if single else max(docs, _log(rng, 2, min(8192, 4194304 // (heads * dim)) // batch))
        return {"op": op, "batch": batch, "tokens": tokens, "docs": docs, "heads": heads, "kv_heads": kv, "dim": dim, **rope,
                "page": rng.choice([16, 64, 64, 100, 256]), "longest": _log(rng, 1, min(32768, 262144 // batch)) if single else 0}
    train = rng.random() < 0.5
    most = min(8192, math.isqrt((268435456 if train else 536870912) // heads // batch))
    return {"op": op, "batch": batch, "tokens": max(docs, _log(rng, 1, most)), "docs": docs, "heads": heads, "kv_heads": kv, "dim": dim,
            "causal": rng.random() < 0.8, "train": train}


# ------------------------------------------------------------------------------------------- inputs

def _offsets(case):
    """Offsets of the sequences in the rows (batch rows one after the other)."""
    B, T, docs = case["batch"], case["tokens"], case["docs"]
    if not docs:
        return [b * T for b in range(B + 1)]
    cuts = random.Random(T * 131 + docs).sample(range(1, T), docs - 1) if docs > 1 else []
    return [0, *sorted(cuts), T]


def _lengths(case):
    """Tokens of every sequence, new ones among them: ragged up to the longest; in a batch of over eight, every eighth row is padding."""
    if case["op"] == "store" and not case["longest"]:
        starts = _offsets(case)
        return [b - a for a, b in zip(starts, starts[1:])]
    rng, B = random.Random(case["batch"] * 7 + case["longest"]), case["batch"]
    return [0 if B > 8 and b % 8 == 7 else case["longest"] if b == 0 else rng.randint((case["longest"] + 3) // 4, case["longest"]) for b in range(B)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)

    def rn(*shape, std=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    op, H, Hk, D = case["op"], case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case}
    if op in ("rope", "store"):
        lead = (case["batch"],) if op == "store" and case["tokens"] == 1 and not case["docs"] else (case["batch"], case["tokens"])
        mixed = rn(*lead, (H + 2 * Hk) * D)     # one projection's output, of which q, k and v are views
        q, k, v = mixed.split([H * D, Hk * D, Hk * D], -1)
        s.update(q=q.unflatten(-1, (H, D)), k=k.unflatten(-1, (Hk, D)), v=v.unflatten(-1, (Hk, D)), q_weight=1 + rn(D, std=0.1, dtype=F32), k_weight=1 + rn(D, std=0.1, dtype=F32))
        s["inv_freq"] = (1 / case["theta"] ** (torch.arange(0, case["rotary"], 2, dtype=F64) / case["rotary"])).to(F32).cuda()
        s["starts"] = _offsets(case)
        s["cu_seqlens"] = s["starts"] if case["docs"] else None
        if case.get("train"):
            s.update(dq=rn(*lead, H, D), dk=rn(*lead, Hk, D))
    elif op == "attention":
        B, T = case["batch"], case["tokens"]
        s.update(q=rn(B, T, H, D), k=rn(B, T, Hk, D), v=rn(B, T, Hk, D))     # as normalised: unit variance, logits of unit variance
        s["starts"] = _offsets(case)
        s["cu_seqlens"] = s["starts"] if case["docs"] else None
        if case["train"]:
            s["do"] = rn(B, T, H, D)
    else:
        s["q"] = rn(case["batch"], H, D)
    if op in ("store", "step"):
        page, lengths = case["page"], _lengths(case)
        need = [(n + page - 1) // page for n in lengths]
        pages = sum(need) + 8
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at: at + n]
            at += n
        s.update(page_table=table, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"), host_lengths=lengths,
                 k_cache=rn(pages, page, Hk, D), v_cache=rn(pages, page, Hk, D))
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _own_rope(s):
    import chunked_gated_delta_05_gb300 as lib
    kw = dict(cu_seqlens=s["cu_seqlens"], eps=EPS, interleaved=s["case"]["interleaved"])
    q, k = lib.qk_norm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"], **kw)
    if not s["case"]["train"]:
        return {"q": q, "k": k}
    dq, dk, dqw, dkw = lib.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"], **kw)
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _own_store(s):
    import chunked_gated_delta_05_gb300 as lib
    q, k = lib.qk_norm_rope_store(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["inv_freq"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"],
                                  cu_seqlens=s["cu_seqlens"], eps=EPS, interleaved=s["case"]["interleaved"])
    return {"q": q, "k": k, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import chunked_gated_delta_05_gb300 as lib
    kw = dict(causal=s["case"]["causal"], cu_seqlens=s["cu_seqlens"])
    o, lse = lib.attention_fwd(s["q"], s["k"], s["v"], **kw)
    if not s["case"]["train"]:
        return {"o": o, "lse": lse}
    dq, dk, dv = lib.attention_bwd(s["do"], s["q"], s["k"], s["v"], o, lse, **kw)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _own_step(s):
    import chunked_gated_delta_05_gb300 as lib
    return lib.attention_step(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"])


_OWN = {"rope": _own_rope, "store": _own_store, "attention": _own_attention, "step": _own_step}


# ------------------------------------------------------------------------------------------- the plain forms

def _positions(s):
    """Every row's position in its sequence, on the device."""
    if "lengths" in s:
        first = [n - (b - a) for n, a, b in zip(s["host_lengths"], s["starts"], s["starts"][1:])]
    else:
        first = [0] * (len(s["starts"]) - 1)
    return torch.cat([torch.arange(f, f + b - a, device="cuda") for f, a, b in zip(first, s["starts"], s["starts"][1:])])


def _cos_sin(s):
    angle = _positions(s).double()[:, None] * s["inv_freq"].double()      # in 64 bits: far positions turn many times
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _rotate(x, cos, sin, interleaved, back=False):
    """The first channels of x [R,H,D] in pairs turned by the angles; the rest stay."""
    n = cos.shape[-1]
    if back:
        sin = -sin
    a, b = (x[..., : 2 * n: 2], x[..., 1: 2 * n: 2]) if interleaved else (x[..., :n], x[..., n: 2 * n])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _normed(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _flat(t):
    return t.reshape(-1, *t.shape[-2:]).float()


def _plain_rope(s):
    inter = s["case"]["interleaved"]
    cos, sin = _cos_sin(s)
    out = {}
    for n in ("q", "k"):
        out[n] = _rotate(_normed(_flat(s[n])) * s[n + "_weight"], cos, sin, inter).to(BF16).view(s[n].shape)
    if not s["case"]["train"]:
        return out
    for n in ("q", "k"):
        x, w = _flat(s[n]), s[n + "_weight"]
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        d = _rotate(_flat(s["d" + n]), cos, sin, inter, back=True)
        xh, dx = x * rstd, d * w
        out["d" + n] = (rstd * (dx - xh * (dx * xh).mean(-1, keepdim=True))).to(BF16).view(s[n].shape)
        out[f"d{n}_weight"] = (d * xh).sum((0, 1))
    return out


def _cache_rows(s):
    """Rows of the batch that are stored, and their rows in the cache."""
    page, starts = s["case"]["page"], s["starts"]
    rows, at = [], []
    for n, length in enumerate(s["host_lengths"]):
        if length > 0:
            a, b = starts[n], starts[n + 1]
            pos = torch.arange(length - (b - a), length, device="cuda")
            rows.append(torch.arange(a, b, device="cuda"))
            at.append(s["page_table"][n].long()[pos // page] * page + pos % page)
    return torch.cat(rows), torch.cat(at)


def _plain_store(s):
    cos, sin = _cos_sin(s)
    rows, at = _cache_rows(s)
    out = {}
    for n in ("q", "k"):
        y = torch.zeros_like(_flat(s[n]))
        y[rows] = _rotate(_normed(_flat(s[n])[rows]) * s[n + "_weight"], cos[rows], sin[rows], s["case"]["interleaved"])
        out[n] = y.to(BF16).view(s[n].shape)
    Hk, D = s["case"]["kv_heads"], s["case"]["dim"]
    s["k_cache"].view(-1, Hk, D)[at] = out["k"].view(-1, Hk, D)[rows]
    s["v_cache"].view(-1, Hk, D)[at] = s["v"].reshape(-1, Hk, D)[rows]
    return {**out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    """Softmax of the scaled products, one sequence and key head at a time, its query heads together."""
    c = s["case"]
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    G, scale = H // Hk, c["dim"] ** -0.5
    q, k, v = (_flat(s[n]) for n in ("q", "k", "v"))
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    if c["train"]:
        do = _flat(s["do"])
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for a, b in zip(s["starts"], s["starts"][1:]):
        late = torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1) if c["causal"] else None
        for h in range(Hk):
            heads = slice(h * G, (h + 1) * G)
            K, V = k[a:b, h], v[a:b, h]
            Q = q[a:b, heads].transpose(0, 1)
            S = Q @ K.t() * scale
            if late is not None:
                S = S.masked_fill(late, -math.inf)
            top = S.amax(-1, keepdim=True)
            P = torch.exp(S - top)
            total = P.sum(-1, keepdim=True)
            P = P / total
            o[a:b, heads] = (P @ V).transpose(0, 1)
            lse[a:b, heads] = (top + torch.log(total))[..., 0].t()
            if c["train"]:
                dO = do[a:b, heads].transpose(0, 1)
                dP = dO @ V.t()
                dS = P * (dP - (P * dP).sum(-1, keepdim=True)) * scale
                dv[a:b, h] = (P.transpose(1, 2) @ dO).sum(0)
                dk[a:b, h] = (dS.transpose(1, 2) @ Q).sum(0)
                dq[a:b, heads] = (dS @ K).transpose(0, 1)
    out = {"o": o.to(BF16).view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}
    if c["train"]:
        out.update(dq=dq.to(BF16).view(s["q"].shape), dk=dk.to(BF16).view(s["k"].shape), dv=dv.to(BF16).view(s["v"].shape))
    return out


def _plain_step(s):
    c = s["case"]
    Hk, D, page = c["kv_heads"], c["dim"], c["page"]
    o = torch.zeros_like(s["q"])
    for b, n in enumerate(s["host_lengths"]):
        if n == 0:
            continue
        pages = s["page_table"][b, : (n + page - 1) // page].long()
        K, V = (s[name][pages].view(-1, Hk, D)[:n].transpose(0, 1).float() for name in ("k_cache", "v_cache"))
        S = s["q"][b].float().view(Hk, -1, D) @ K.transpose(1, 2) * D ** -0.5
        P = torch.exp(S - S.amax(-1, keepdim=True))
        o[b] = (P @ V / P.sum(-1, keepdim=True)).view(-1, D).to(BF16)
    return o


_PLAIN = {"rope": _plain_rope, "store": _plain_store, "attention": _plain_attention, "step": _plain_step}


# ------------------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, H, Hk, D = case["op"], case["heads"], case["kv_heads"], case["dim"]
    if op == "step":
        seen = sum(_lengths(case))
        live = sum(n > 0 for n in _lengths(case))
        return {"bytes": seen * Hk * D * 4 + (live + case["batch"]) * H * D * 2 + 4 * (case["batch"] + -(-seen // case["page"])), "flops": seen * H * D * 4}
    R, el = case["batch"] * case["tokens"], H + Hk
    if op == "rope":
        out = {"bytes": R * el * D * 4 + 8 * D + 2 * case["rotary"], "flops": R * el * D * 8}
        if case["train"]:
            out["bytes"] += R * el * D * 6 + 16 * D + 2 * case["rotary"]
            out["flops"] += R * el * D * 16
        return out
    if op == "store":
        starts = _offsets(case)
        live = sum(b - a for n, a, b in zip(_lengths(case), starts, starts[1:]) if n > 0)
        return {"bytes": live * (H + 2 * Hk) * D * 2 + R * el * D * 2 + live * 2 * Hk * D * 2 + 8 * D + 2 * case["rotary"], "flops": live * el * D * 8}
    starts = _offsets(case)
    lens = [b - a for a, b in zip(starts, starts[1:])]
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens) * H
    out = {"bytes": R * (2 * H + 2 * Hk) * D * 2 + R * H * 4, "flops": pairs * D * 4}
    if case["train"]:     # q, k, v, o, do and the row sums in, three gradients out
        out["bytes"] += R * (4 * H + 4 * Hk) * D * 2 + R * H * 4
        out["flops"] += pairs * D * 10
    return out


# ------------------------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _turns(case, s):
    """Complex numbers e^(i angle) of every row."""
    pos = []
    for i, (a, b) in enumerate(zip(s["starts"], s["starts"][1:])):
        last = s["host_lengths"][i] if "host_lengths" in s else b - a
        pos += range(last - (b - a), last)
    angle = torch.tensor(pos, dtype=F64, device="cuda").unsqueeze(1) * s["inv_freq"].to(F64)
    return torch.polar(torch.ones_like(angle), angle).unsqueeze(1)


def _exact_turned(case, x, w, turn):
    y = x * w / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS)
    r = case["rotary"]
    first = torch.arange(0, r, 2, device="cuda") if case["interleaved"] else torch.arange(r // 2, device="cuda")
    second = first + 1 if case["interleaved"] else first + r // 2
    pair = torch.complex(y[..., first], y[..., second]) * turn
    return y.index_copy(-1, first, pair.real).index_copy(-1, second, pair.imag)


def _exact_rope(case, s):
    turn, out = _turns(case, s), {}
    for n in ("q", "k"):
        x = s[n].reshape(-1, *s[n].shape[-2:]).to(F64).requires_grad_(case["train"])
        w = s[n + "_weight"].to(F64).requires_grad_(case["train"])
        y = _exact_turned(case, x, w, turn)
        out[n] = y.detach().view(s[n].shape)
        if case["train"]:
            dx, dw = torch.autograd.grad((y * s["d" + n].reshape(y.shape).to(F64)).sum(), [x, w])
            out["d" + n], out[f"d{n}_weight"] = dx.view(s[n].shape), dw
    return {k: out[k] for k in ("q", "k", "dq", "dk", "dq_weight", "dk_weight") if k in out}


def _exact_store(case, s):
    turn, out = _turns(case, s), {}
    for n in ("q", "k"):
        out[n] = _exact_turned(case, s[n].reshape(-1, *s[n].shape[-2:]).to(F64), s[n + "_weight"].to(F64), turn)
    caches = {"k_cache": s["k_cache"].to(F64), "v_cache": s["v_cache"].to(F64)}
    v, table = s["v"].reshape(-1, *s["v"].shape[-2:]).to(F64), s["page_table"].tolist()
    for i, length in enumerate(s["host_lengths"]):
        a, b = s["starts"][i], s["starts"][i + 1]
        if length == 0:
            out["q"][a:b] = 0
            out["k"][a:b] = 0
            continue
        at = a
        while at < b:     # page by page
            pos = length - (b - at)
            page, inside = table[i][pos // case["page"]], pos % case["page"]
            n = min(case["page"] - inside, b - at)
            caches["k_cache"][page, inside: inside + n] = out["k"][at: at + n]
            caches["v_cache"][page, inside: inside + n] = v[at: at + n]
            at += n
    return {"q": out["q"].view(s["q"].shape), "k": out["k"].view(s["k"].shape), **caches}


def _exact_attention(case, s):
    H, D, G = case["heads"], case["dim"], case["heads"] // case["kv_heads"]
    names = ("q", "k", "v", "do") if case["train"] else ("q", "k", "v")
    x = {n: s[n].reshape(-1, *s[n].shape[-2:]).to(F64) for n in names}
    o, lse = torch.zeros_like(x["q"]), torch.zeros(x["q"].shape[:2], dtype=F64, device="cuda")
    grads = {n: torch.zeros_like(x[n]) for n in ("q", "k", "v")}
    for a, b in zip(s["starts"], s["starts"][1:]):
        for h in range(H):
            K, V = x["k"][a:b, h // G], x["v"][a:b, h // G]
            for i in range(a, b, 2048):     # queries in pieces, with the keys they see
                j = min(b, i + 2048)
                n = j - a if case["causal"] else b - a
                logits = torch.mm(x["q"][i:j, h], K[:n].t()).div_(math.sqrt(D))
                if case["causal"]:
                    logits[:, i - a:].masked_fill_(torch.ones(j - i, j - i, dtype=torch.bool, device="cuda").triu(1), -math.inf)
                L = torch.logsumexp(logits, 1)
                P = logits.sub_(L[:, None]).exp_()
                o[i:j, h], lse[i:j, h] = P @ V[:n], L
                if case["train"]:
                    dO = x["do"][i:j, h]
                    grads["v"][a: a + n, h // G] += P.t() @ dO
                    dS = P * (dO @ V[:n].t() - (dO * o[i:j, h]).sum(1, keepdim=True)) / math.sqrt(D)
                    grads["q"][i:j, h] = dS @ K[:n]
                    grads["k"][a: a + n, h // G] += dS.t() @ x["q"][i:j, h]
    out = {"o": o.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}
    if case["train"]:
        out.update({"d" + n: grads[n].view(s[n].shape) for n in ("q", "k", "v")})
    return out


def _exact_step(case, s):
    D, G = case["dim"], case["heads"] // case["kv_heads"]
    o, q, table = torch.zeros(s["q"].shape, dtype=F64, device="cuda"), s["q"].to(F64), s["page_table"].tolist()
    for b, n in enumerate(s["host_lengths"]):
        if n:
            used = table[b][: -(-n // case["page"])]
            K, V = (torch.cat([s[name][p] for p in used])[:n].to(F64) for name in ("k_cache", "v_cache"))
            for h in range(case["heads"]):
                P = torch.softmax(K[:, h // G] @ q[b, h] / math.sqrt(D), 0)
                o[b, h] = P @ V[:, h // G]
    return o


_EXACT = {"rope": _exact_rope, "store": _exact_store, "attention": _exact_attention, "step": _exact_step}
