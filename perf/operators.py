"""Measured cases of the operators around the gated delta rule: the selective state space scan (prompts,
training, single tokens), the single-token forms of the short convolution and of the delta rule, and the
norms before and after a block. Each case has a plain form (elementary torch operations in 32 bits), the
framework's own call, and the definition in 64 bits."""
import math
import random

import torch

own = False

EPS = 1e-6          # norms
L2_EPS = 1e-6       # q/k normalisation of the delta rule
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # four sequences' next tokens enter a block: the residual sum and the norm, where latency counts
        {"name": "add_norm token", "op": "add_norm", "rows": 4, "width": 2048, "residual": "f32", "train": False},
        # a training step's 8192 tokens enter a block of the 2 x 4096 training shape's width, both directions
        {"name": "add_norm train", "op": "add_norm", "rows": 8192, "width": 2048, "residual": "f32", "train": True},
        # the gated norm of every head after the recurrence, an 8192-token prompt with 16 heads
        {"name": "gated_norm prompt", "op": "gated_norm", "rows": 131072, "width": 128, "activation": "silu", "train": False},
        # the same in training, 8192 tokens with 32 heads and a sigmoid gate, both directions
        {"name": "gated_norm train", "op": "gated_norm", "rows": 262144, "width": 128, "activation": "sigmoid", "train": True},
        # one sequence's next token through the short convolution of mixed q/k/v channels
        {"name": "conv_step one", "op": "conv_step", "batch": 1, "slots": 1, "channels": 6144, "taps": 4, "dilation": 1,
         "bias": True, "indexed": False},
        # a full serving batch, its states spread over a pool of slots, some rows only padding
        {"name": "conv_step many", "op": "conv_step", "batch": 250, "slots": 320, "channels": 6144, "taps": 4, "dilation": 1,
         "bias": False, "indexed": True},
        # one sequence's next token through the delta rule, 16 heads
        {"name": "gdn_step one", "op": "delta_step", "batch": 1, "slots": 1, "heads": 16, "qk_heads": 16, "gate": "scalar", "indexed": False},
        # a serving batch with grouped query and key heads and pooled states
        {"name": "gdn_step many", "op": "delta_step", "batch": 120, "slots": 160, "heads": 16, "qk_heads": 4, "gate": "scalar", "indexed": True},
        # a serving batch of the per-channel gate, 32 heads, the gate activated in the kernel
        {"name": "kda_step many", "op": "delta_step", "batch": 48, "slots": 48, "heads": 32, "qk_heads": 32, "gate": "logits", "indexed": False},
        # one long prompt through a selective scan block, its last state kept for decoding
        {"name": "scan prompt", "op": "scan", "batch": 1, "tokens": 8192, "docs": 0, "channels": 4096, "states": 16, "groups": 1,
         "z": True, "skip": True, "softplus": True, "h0": False, "train": False},
        # a training step over documents packed in one row, lengths as they come
        {"name": "scan train", "op": "scan", "batch": 1, "tokens": 4093, "docs": 7, "channels": 2048, "states": 16, "groups": 1,
         "z": True, "skip": True, "softplus": True, "h0": False, "train": True},
        # the next token of a serving batch through the scan block
        {"name": "scan_step many", "op": "scan_step", "batch": 120, "slots": 160, "channels": 4096, "states": 16, "groups": 1, "indexed": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add_norm", "gated_norm", "conv_step", "delta_step", "scan", "scan", "scan_step"])
    if op == "add_norm":
        width = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024)])
        return {"op": op, "rows": min(_log(rng, 1, 16384), 16777216 // width), "width": width,
                "residual": rng.choice(["f32", "bf16", "none"]), "train": rng.random() < 0.5}
    if op == "gated_norm":
        width = rng.choice([128, 128, _log(rng, 16, 4096)])
        return {"op": op, "rows": min(_log(rng, 1, 262144), 33500000 // width), "width": width,
                "activation": rng.choice(["silu", "sigmoid"]), "train": rng.random() < 0.5}
    if op == "conv_step":
        batch = _log(rng, 1, 250)
        return {"op": op, "batch": batch, "slots": batch + rng.randrange(64), "channels": 8 * _log(rng, 8, 768), "taps": rng.choice([2, 3, 4, 4]),
                "dilation": rng.choice([1, 1, 2]), "bias": rng.random() < 0.5, "indexed": rng.random() < 0.7}
    if op == "delta_step":
        heads = rng.choice([1, 2, 4, 6, 8, 12, 16, 32])
        batch = min(_log(rng, 1, 120), 1920 // heads)
        return {"op": op, "batch": batch, "slots": batch + rng.randrange(16), "heads": heads, "qk_heads": heads // rng.choice([1, 1, 2 if heads % 2 == 0 else 1]),
                "gate": rng.choice(["scalar", "channel", "logits"]), "indexed": rng.random() < 0.7}
    if op == "scan_step":
        groups = rng.choice([1, 1, 2, 4])
        batch = _log(rng, 1, 120)
        return {"op": op, "batch": batch, "slots": batch + rng.randrange(40), "channels": groups * _log(rng, 16, 4096 // groups),
                "states": rng.choice([4, 8, 13, 16, 16]), "groups": groups, "indexed": rng.random() < 0.7}
    train = rng.random() < 0.5
    groups = rng.choice([1, 1, 2, 4])
    channels = groups * _log(rng, 16, (2048 if train else 4096) // groups)
    docs = rng.choice([0, 0, 1, 3, 9])
    batch = 1 if docs else rng.choice([1, 2, 3])
    most = min(16384 if not train else 8192, (8388608 if train else 33554432) // channels) // batch
    return {"op": op, "batch": batch, "tokens": max(docs, _log(rng, 1, most)), "docs": docs, "channels": channels, "states": rng.choice([4, 8, 13, 16, 16]),
            "groups": groups, "z": rng.random() < 0.7, "skip": rng.random() < 0.7, "softplus": rng.random() < 0.8, "h0": rng.random() < 0.5, "train": train}


# ------------------------------------------------------------------------------------------- inputs

def _offsets(case):
    """Document offsets of the rows (batch rows one after the other): a dense batch's are its sequences."""
    B, T, docs = case["batch"], case["tokens"], case["docs"]
    if not docs:
        return [b * T for b in range(B + 1)]
    cuts = random.Random(T * 131 + docs).sample(range(1, T), docs - 1) if docs > 1 else []
    return [0, *sorted(cuts), T]


def _indices(case, g):
    """Each row's slot in the pool, none twice; in a batch of over eight, every eighth row is padding."""
    idx = torch.randperm(case["slots"], generator=g, device="cuda")[: case["batch"]].to(torch.int32)
    if case["batch"] > 8:
        idx[7::8] = -1
    return idx


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)

    def rn(*shape, std=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def ru(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": case}
    op = case["op"]
    if op == "add_norm":
        R, W = case["rows"], case["width"]
        kind = {"f32": F32, "bf16": BF16, "none": None}[case["residual"]]
        s.update(x=rn(R, W), weight=1 + rn(W, std=0.1, dtype=F32), scale=1.0 if kind is None else 0.7)
        s["residual"] = None if kind is None else rn(R, W, std=2.0, dtype=kind)
        if case["train"]:
            s.update(dy=rn(R, W), dstream=rn(R, W, dtype=BF16 if kind is None else kind))
    elif op == "gated_norm":
        R, W = case["rows"], case["width"]
        s.update(x=rn(R, W, std=0.5), gate=rn(R, W), weight=1 + rn(W, std=0.1, dtype=F32))
        if case["train"]:
            s["dy"] = rn(R, W)
    elif op == "conv_step":
        B, C, W = case["batch"], case["channels"], case["taps"]
        s.update(x=rn(B, C), weight=rn(C, W, std=0.25, dtype=F32), bias=rn(C, std=0.01, dtype=F32) if case["bias"] else None,
                 state=rn(case["slots"], (W - 1) * case["dilation"], C))
    elif op == "delta_step":
        B, H, Hk = case["batch"], case["heads"], case["qk_heads"]
        mixed = rn(B, (2 * Hk + H) * 128)     # the short convolution's output: q, k and v are views of it
        s.update(q=mixed[:, : Hk * 128].view(B, Hk, 128), k=mixed[:, Hk * 128: 2 * Hk * 128].view(B, Hk, 128),
                 v=mixed[:, 2 * Hk * 128:].view(B, H, 128), state=rn(case["slots"], H, 128, 128, std=0.1, dtype=F32))
        if case["gate"] == "scalar":
            s.update(g=-torch.log1p(torch.exp(rn(B, H, dtype=F32))), beta=torch.sigmoid(rn(B, H, dtype=F32)).to(BF16))
        else:
            s["beta"] = rn(B, H)
            if case["gate"] == "channel":
                s["g"] = -torch.log1p(torch.exp(rn(B, H, 128, dtype=F32)))
            else:
                s.update(g=rn(B, H, 128, dtype=F32), A_log=torch.log(1 + 3 * ru(H)), dt_bias=rn(H, 128, std=0.5, dtype=F32), lower_bound=-5.0)
    else:
        D, N, G = case["channels"], case["states"], case["groups"]
        B, T = case["batch"], case.get("tokens")
        lead = (B, T) if op == "scan" else (B,)
        dt = torch.exp(ru(D) * math.log(100.0) + math.log(1e-3))     # step sizes from 0.001 to 0.1, as such layers start
        s.update(A=-(1 + torch.arange(N, device="cuda", dtype=F32)) * torch.exp(0.2 * rn(D, N, dtype=F32)))
        BC = rn(*lead, 2 * G * N + 8)     # a projection's output, of which B and C are views
        s.update(u=rn(*lead, D), B=BC[..., 8: 8 + G * N].view(*lead, G, N), C=BC[..., 8 + G * N:].view(*lead, G, N))
        if case.get("softplus", True):
            s.update(delta=rn(*lead, D, std=0.5), delta_bias=dt + torch.log(-torch.expm1(-dt)))
        else:
            s.update(delta=(dt * torch.exp(0.5 * rn(*lead, D, dtype=F32))).to(BF16), delta_bias=None)
        s["D"] = 1 + rn(D, std=0.1, dtype=F32) if case.get("skip", True) else None
        s["z"] = rn(*lead, 2 * D)[..., D:] if case.get("z", True) else None     # half of the block's input projection
        if op == "scan":
            s["starts"] = _offsets(case)
            s["cu_seqlens"] = s["starts"] if case["docs"] else None
            docs = len(s["starts"]) - 1
            s["h0"] = rn(docs, D, N, dtype=F32) if case["h0"] else None
            if case["train"]:
                s.update(dy=rn(B, T, D), dfinal=rn(docs, D, N, dtype=F32) if case["h0"] else None)
        else:
            s["state"] = rn(case["slots"], D, N, dtype=F32)
    if "slots" in case:
        s["index"] = _indices(case, g) if case["indexed"] else None
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _own_add_norm(s):
    import chunked_gated_delta_05_gb300 as lib
    y, stream = lib.add_rms_norm_fwd(s["x"], s["residual"], s["weight"], eps=EPS, residual_scale=s["scale"])
    if not s["case"]["train"]:
        return {"y": y, "stream": stream}
    dx, dres, dw = lib.add_rms_norm_bwd(s["dy"], s["dstream"], stream, s["weight"], eps=EPS, residual_scale=s["scale"],
                                        has_residual=s["residual"] is not None)
    return {"y": y, "stream": stream, "dx": dx, "dresidual": dres, "dweight": dw}


def _own_gated_norm(s):
    import chunked_gated_delta_05_gb300 as lib
    act = s["case"]["activation"]
    y = lib.gated_rms_norm_fwd(s["x"], s["gate"], s["weight"], eps=EPS, activation=act)
    if not s["case"]["train"]:
        return y
    dx, dgate, dw = lib.gated_rms_norm_bwd(s["x"], s["gate"], s["weight"], s["dy"], eps=EPS, activation=act)
    return {"y": y, "dx": dx, "dgate": dgate, "dweight": dw}


def _own_conv_step(s):
    import chunked_gated_delta_05_gb300 as lib
    y = lib.causal_conv1d_step(s["state"], s["x"], s["weight"], s["bias"], dilation=s["case"]["dilation"], state_indices=s["index"])
    return {"y": y, "state": s["state"]}


def _own_delta_step(s):
    import chunked_gated_delta_05_gb300 as lib
    if s["case"]["gate"] == "scalar":
        o = lib.gdn_step(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], state_indices=s["index"])
    else:
        o = lib.kda_step(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], state_indices=s["index"], A_log=s.get("A_log"),
                         dt_bias=s.get("dt_bias"), lower_bound=s.get("lower_bound"))
    return {"o": o, "state": s["state"]}


def _own_scan(s):
    import chunked_gated_delta_05_gb300 as lib
    c = s["case"]
    kw = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], delta_softplus=c["softplus"], initial_state=s["h0"], cu_seqlens=s["cu_seqlens"])
    if not c["train"]:
        y, final = lib.selective_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], output_final_state=True, **kw)
        return {"y": y, "final": final}
    y, final, saved = lib.selective_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], output_final_state=True, save=True, **kw)
    grads = lib.selective_scan_bwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dy"], dfinal=s["dfinal"], saved=saved, **kw)
    return {"y": y, "final": final, **dict(zip(_SCAN_GRADS, grads))}


def _own_scan_step(s):
    import chunked_gated_delta_05_gb300 as lib
    y = lib.selective_scan_step(s["state"], s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"],
                                delta_softplus=True, state_indices=s["index"])
    return {"y": y, "state": s["state"]}


_SCAN_GRADS = ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dh0")
_OWN = {"add_norm": _own_add_norm, "gated_norm": _own_gated_norm, "conv_step": _own_conv_step, "delta_step": _own_delta_step,
        "scan": _own_scan, "scan_step": _own_scan_step}


# ------------------------------------------------------------------------------------------- the plain forms

def _plain_add_norm(s):
    """stream = residual + scale x, rounded to the residual's type; y = stream / rms(stream) * weight."""
    kind = BF16 if s["residual"] is None else s["residual"].dtype
    stream = s["x"] if s["residual"] is None else (s["residual"].float() + s["scale"] * s["x"].float()).to(kind)
    h, w = stream.float(), s["weight"]
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = (h * rstd * w).to(BF16)
    if not s["case"]["train"]:
        return {"y": y, "stream": stream}
    dy = s["dy"].float()
    xhat, dxhat = h * rstd, dy * w
    dh = s["dstream"].float() + rstd * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True))
    return {"y": y, "stream": stream, "dx": (s["scale"] * dh).to(BF16), "dresidual": None if s["residual"] is None else dh.to(kind),
            "dweight": (dy * xhat).sum(0)}


def _plain_gated_norm(s):
    """y = x / rms(x) * weight * act(gate)."""
    x, gate, w = s["x"].float(), s["gate"].float(), s["weight"]
    sig = 1 / (1 + torch.exp(-gate))
    silu = s["case"]["activation"] == "silu"
    act = gate * sig if silu else sig
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * rstd
    y = (xhat * w * act).to(BF16)
    if not s["case"]["train"]:
        return y
    dy = s["dy"].float()
    dact = sig * (1 + gate * (1 - sig)) if silu else sig * (1 - sig)
    dn = dy * act
    dxhat = dn * w
    dx = rstd * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(BF16), "dgate": (dy * xhat * w * dact).to(BF16), "dweight": (dn * xhat).sum(0)}


def _rows(s):
    """The live rows of a pooled batch and their slots."""
    B = s["case"]["batch"]
    if s["index"] is None:
        every = torch.arange(B, device="cuda")
        return every, every
    live = torch.nonzero(s["index"] >= 0).flatten()
    return live, s["index"][live].long()


def _plain_conv_step(s):
    rows, slots = _rows(s)
    d, taps = s["case"]["dilation"], s["case"]["taps"]
    x = s["x"][rows]
    seen = torch.cat([s["state"][slots], x[:, None]], 1)       # the last (taps-1) dilation inputs and this one
    z = (seen[:, ::d].float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        z = z + s["bias"]
    y = torch.zeros_like(s["x"])
    y[rows] = (z / (1 + torch.exp(-z))).to(BF16)
    s["state"][slots] = seen[:, 1:]
    return {"y": y, "state": s["state"]}


def _plain_delta_step(s):
    c = s["case"]
    rows, slots = _rows(s)
    share = c["heads"] // c["qk_heads"]
    q, k = (t[rows].float().repeat_interleave(share, 1) for t in (s["q"], s["k"]))
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + L2_EPS)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + L2_EPS)
    g, beta = s["g"][rows], s["beta"][rows].float()
    if c["gate"] != "scalar":
        beta = 1 / (1 + torch.exp(-beta))
    if c["gate"] == "logits":
        g = s["lower_bound"] / (1 + torch.exp(-torch.exp(s["A_log"])[:, None] * (g + s["dt_bias"])))
    decay = torch.exp(g)[..., None, None] if c["gate"] == "scalar" else torch.exp(g)[..., None]
    S = s["state"][slots] * decay
    delta = beta[..., None] * (s["v"][rows].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * delta[..., None, :]
    o = torch.zeros(c["batch"], c["heads"], 128, dtype=BF16, device="cuda")
    o[rows] = ((S * q[..., None]).sum(-2) / math.sqrt(128.0)).to(BF16)
    s["state"][slots] = S
    return {"o": o, "state": s["state"]}


def _step_sizes(s, delta):
    x = delta.float() if s["delta_bias"] is None else delta.float() + s["delta_bias"]
    if not s["case"].get("softplus", True):
        return x, torch.ones_like(x)
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs())), 1 / (1 + torch.exp(-x))


def _running(a, b):
    """In place in b: h_t = a_t h_{t-1} + b_t along the first dimension, by doubling; a is used up."""
    n = 1
    while n < b.shape[0]:
        b[n:] += a[n:] * b[:-n]
        a[n:] = a[n:] * a[:-n]
        n *= 2
    return b


def _spread(t, D):
    """[R, G, N] to [R, D, N]: every channel of a group reads the group's vector."""
    R, G, N = t.shape
    return t.float()[:, :, None].expand(R, G, D // G, N).reshape(R, D, N)


def _plain_scan(s):
    c = s["case"]
    R, D, N, G = c["batch"] * c["tokens"], c["channels"], c["states"], c["groups"]
    flat = lambda t: t.reshape(R, *t.shape[2:])
    first, last = torch.tensor(s["starts"][:-1], device="cuda"), torch.tensor(s["starts"][1:], device="cuda") - 1
    u, A = flat(s["u"]).float(), s["A"]
    dt, slope = _step_sizes(s, flat(s["delta"]))
    Bs, Cs = _spread(flat(s["B"]), D), _spread(flat(s["C"]), D)
    decay = torch.exp(dt[..., None] * A)
    h = (dt * u)[..., None] * Bs
    if s["h0"] is not None:
        h[first] += decay[first] * s["h0"]
    a = decay.clone()
    a[first] = 0                                    # nothing flows from one document to the next
    h = _running(a, h)
    del a
    y0 = (h * Cs).sum(-1)
    if s["D"] is not None:
        y0 = y0 + s["D"] * u
    y = y0
    if s["z"] is not None:
        z = flat(s["z"]).float()
        sig = 1 / (1 + torch.exp(-z))
        y = y0 * z * sig
    out = {"y": y.to(BF16).view(s["u"].shape), "final": h[last]}
    if not c["train"]:
        return out
    dy = flat(s["dy"]).float()
    dy0 = dy if s["z"] is None else dy * z * sig
    dh = dy0[..., None] * Cs
    if s["dfinal"] is not None:
        dh[last] += s["dfinal"]
    a = torch.cat([decay[1:], torch.zeros_like(decay[:1])])     # dh_t = C_t dy_t + decay_{t+1} dh_{t+1}
    a[last] = 0
    dh = _running(a.flip(0), dh.flip(0)).flip(0)
    del a
    grouped = lambda t: t.view(R, G, D // G, N).sum(2).to(BF16).view(s["B"].shape)
    dC, dB = grouped(h * dy0[..., None]), grouped(dh * (dt * u)[..., None])
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = 0 if s["h0"] is None else s["h0"]
    fell = dh * decay * before                      # d exp(dt A) dt A / d (dt A)
    dhB = (dh * Bs).sum(-1)
    ddt = u * dhB + (fell * A).sum(-1)
    ddelta = ddt * slope
    du = dt * dhB if s["D"] is None else dt * dhB + s["D"] * dy0
    out.update(du=du.to(BF16).view(s["u"].shape), ddelta=ddelta.to(BF16).view(s["u"].shape), dA=(fell * dt[..., None]).sum(0), dB=dB, dC=dC,
               dD=None if s["D"] is None else (dy0 * u).sum(0),
               dz=None if s["z"] is None else (dy * y0 * sig * (1 + z * (1 - sig))).to(BF16).view(s["u"].shape),
               ddelta_bias=None if s["delta_bias"] is None else ddelta.sum(0), dh0=None if s["h0"] is None else (decay * dh)[first])
    return out


def _plain_scan_step(s):
    D = s["case"]["channels"]
    rows, slots = _rows(s)
    u = s["u"][rows].float()
    dt, _ = _step_sizes(s, s["delta"][rows])
    h = torch.exp(dt[..., None] * s["A"]) * s["state"][slots] + (dt * u)[..., None] * _spread(s["B"][rows], D)
    z = s["z"][rows].float()
    y = torch.zeros_like(s["u"])
    y[rows] = (((h * _spread(s["C"][rows], D)).sum(-1) + s["D"] * u) * z / (1 + torch.exp(-z))).to(BF16)
    s["state"][slots] = h
    return {"y": y, "state": s["state"]}


_PLAIN = {"add_norm": _plain_add_norm, "gated_norm": _plain_gated_norm, "conv_step": _plain_conv_step, "delta_step": _plain_delta_step,
          "scan": _plain_scan, "scan_step": _plain_scan_step}


# ------------------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "add_norm":
        e, R, W = {"f32": 4, "bf16": 2, "none": 0}[case["residual"]], case["rows"], case["width"]
        el = R * W
        out = {"bytes": el * (2 + 2 + 2 * e) + 4 * W, "flops": 6 * el}
        if case["train"]:     # dy, the stream's gradient; dx and, where there is a residual, its gradient; the stream is read again
            out["bytes"] += el * (2 + 2 * (e or 2) + 2 + e) + 8 * W
            out["flops"] += 14 * el
        return out
    if op == "gated_norm":
        el, W = case["rows"] * case["width"], case["width"]
        out = {"bytes": el * 6 + 4 * W, "flops": 10 * el}
        if case["train"]:
            out["bytes"] += el * 10 + 8 * W
            out["flops"] += 24 * el
        return out
    live = case["batch"] - (case["batch"] // 8 if case.get("indexed") and case["batch"] > 8 else 0)
    if op == "conv_step":
        C, HW = case["channels"], (case["taps"] - 1) * case["dilation"]
        return {"bytes": live * C * (2 * HW * 2 + 2) + case["batch"] * C * 2 + C * case["taps"] * 4 + C * 4 * case["bias"], "flops": live * C * (2 * case["taps"] + 5)}
    if op == "delta_step":
        H, Hk = case["heads"], case["qk_heads"]
        per = 2 * 128 * 128 * 4 * H + 2 * Hk * 256 + H * 256 + 2 * H + 4 * H * (1 if case["gate"] == "scalar" else 128)
        return {"bytes": live * per + case["batch"] * H * 256, "flops": live * H * 128 * 128 * 7}
    D, N, G = case["channels"], case["states"], case["groups"]
    if op == "scan_step":
        return {"bytes": live * (2 * D * N * 4 + 3 * 2 * D + 4 * G * N) + case["batch"] * D * 2 + D * N * 4 + 8 * D, "flops": live * D * (7 * N + 20)}
    R, docs = case["batch"] * case["tokens"], case["docs"] or case["batch"]
    z = 1 if case["z"] else 0
    par = D * N * 4 + 4 * D * (case["skip"] + case["softplus"])
    out = {"bytes": R * D * 2 * (3 + z) + R * 4 * G * N + par + docs * D * N * 4 * (1 + case["h0"]), "flops": R * D * (7 * N + 20)}
    if case["train"]:     # u, delta, z, dy in and their gradients out, B and C and their gradients, parameters and theirs, states and theirs
        out["bytes"] += R * D * 2 * (3 + z + 2 + z) + R * 8 * G * N + 2 * par + docs * D * N * 4 * 3 * case["h0"]
        out["flops"] += R * D * (18 * N + 40)
    return out


# ------------------------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, {k: v.to(F64) if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}, s)


def _exact_add_norm(case, s, raw):
    x, w = s["x"].requires_grad_(case["train"]), s["weight"].clone().requires_grad_(case["train"])
    res = s["residual"]
    if res is None:
        stream = x
    else:
        res.requires_grad_(case["train"])
        exact_sum = res + s["scale"] * x
        stream = exact_sum + (exact_sum.detach().to(raw["residual"].dtype).to(F64) - exact_sum.detach())   # what is kept of it
    y = stream * w / torch.sqrt(stream.pow(2).sum(-1, keepdim=True) / case["width"] + EPS)
    out = {"y": y.detach(), "stream": None if res is None else exact_sum.detach()}
    if not case["train"]:
        return out
    wrt = [x, w] if res is None else [x, w, res]
    grads = torch.autograd.grad((y * s["dy"]).sum() + (stream * s["dstream"]).sum(), wrt)
    return {**out, "dx": grads[0], "dresidual": None if res is None else grads[2], "dweight": grads[1]}


def _exact_gated_norm(case, s, raw):
    x, gate, w = (s[k].requires_grad_(case["train"]) for k in ("x", "gate", "weight"))
    y = x * w / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["width"] + EPS) * torch.sigmoid(gate)
    if case["activation"] == "silu":
        y = y * gate
    if not case["train"]:
        return y
    dx, dgate, dw = torch.autograd.grad((y * s["dy"]).sum(), [x, gate, w])
    return {"y": y.detach(), "dx": dx, "dgate": dgate, "dweight": dw}


def _live(case, s):
    idx = range(case["batch"]) if s["index"] is None else s["index"].tolist()
    return [(b, i) for b, i in enumerate(idx) if i >= 0]


def _exact_conv_step(case, s, raw):
    y, state = torch.zeros_like(s["x"]), s["state"].clone()
    d, W = case["dilation"], case["taps"]
    for b, slot in _live(case, s):
        past = s["state"][slot]
        acc = s["x"][b] * s["weight"][:, W - 1]
        for i in range(W - 1):
            acc = acc + past[i * d] * s["weight"][:, i]
        if s["bias"] is not None:
            acc = acc + s["bias"]
        y[b] = acc * torch.sigmoid(acc)
        if past.shape[0]:
            state[slot, :-1] = past[1:]
            state[slot, -1] = s["x"][b]
    return {"y": y, "state": state}


def _exact_delta_step(case, s, raw):
    H, share = case["heads"], case["heads"] // case["qk_heads"]
    o, state = torch.zeros(case["batch"], H, 128, dtype=F64, device="cuda"), s["state"].clone()
    head = torch.arange(H, device="cuda") // share
    for b, slot in _live(case, s):
        q, k, g, beta = s["q"][b][head], s["k"][b][head], s["g"][b], s["beta"][b]
        q, k = (t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) + L2_EPS) for t in (q, k))
        if case["gate"] == "logits":
            g = s["lower_bound"] * torch.sigmoid(torch.exp(s["A_log"])[:, None] * (g + s["dt_bias"]))
        if case["gate"] != "scalar":
            beta = torch.sigmoid(beta)
        S = state[slot] * torch.exp(g.view(H, -1, 1))
        miss = s["v"][b] - torch.einsum("hkv,hk->hv", S, k)
        S = S + torch.einsum("hk,hv->hkv", k, beta[:, None] * miss)
        o[b] = torch.einsum("hkv,hk->hv", S, q) * 128 ** -0.5
        state[slot] = S
    return {"o": o, "state": state}


def _dt64(s, case, delta):
    x = delta if s["delta_bias"] is None else delta + s["delta_bias"]
    return torch.logaddexp(x, torch.zeros_like(x)) if case.get("softplus", True) else x


def _exact_scan(case, s, raw):
    R, D, G = case["batch"] * case["tokens"], case["channels"], case["groups"]
    if case["train"] and R * D * case["states"] > 150_000_000:
        return None
    names = [k for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0") if s[k] is not None]
    if case["train"]:
        for k in names:
            s[k] = s[k].detach().clone().requires_grad_(True)
    u, delta, Bm, Cm = (s[k].reshape(R, *s[k].shape[2:]) for k in ("u", "delta", "B", "C"))
    group = torch.arange(D, device="cuda") // (D // G)
    dt = _dt64(s, case, delta)
    ys, finals = [], []
    for i, (a, b) in enumerate(zip(s["starts"][:-1], s["starts"][1:])):
        h = torch.zeros_like(s["A"]) if s["h0"] is None else s["h0"][i]
        for t in range(a, b):
            h = torch.exp(dt[t, :, None] * s["A"]) * h + (dt[t] * u[t])[:, None] * Bm[t][group]
            ys.append(torch.einsum("dn,dn->d", h, Cm[t][group]))
        finals.append(h)
    y, final = torch.stack(ys), torch.stack(finals)
    if s["D"] is not None:
        y = y + s["D"] * u
    if s["z"] is not None:
        z = s["z"].reshape(R, D)
        y = y * z * torch.sigmoid(z)
    out = {"y": y.detach().view(raw["u"].shape), "final": final.detach()}
    if not case["train"]:
        return out
    loss = (y * s["dy"].reshape(R, D)).sum()
    if s["dfinal"] is not None:
        loss = loss + (final * s["dfinal"]).sum()
    grads = dict(zip(names, torch.autograd.grad(loss, [s[k] for k in names])))
    return {**out, **{"d" + k: grads.get(k) for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0")}}


def _exact_scan_step(case, s, raw):
    group = torch.arange(case["channels"], device="cuda") // (case["channels"] // case["groups"])
    y, state = torch.zeros_like(s["u"]), s["state"].clone()
    for b, slot in _live(case, s):
        dt = _dt64(s, case, s["delta"][b])
        h = torch.exp(dt[:, None] * s["A"]) * state[slot] + (dt * s["u"][b])[:, None] * s["B"][b][group]
        y[b] = (torch.einsum("dn,dn->d", h, s["C"][b][group]) + s["D"] * s["u"][b]) * s["z"][b] * torch.sigmoid(s["z"][b])
        state[slot] = h
    return {"y": y, "state": state}


_EXACT = {"add_norm": _exact_add_norm, "gated_norm": _exact_gated_norm, "conv_step": _exact_conv_step, "delta_step": _exact_delta_step,
          "scan": _exact_scan, "scan_step": _exact_scan_step}
