"""The operators of a hybrid recurrent stack, in their plain form and as the framework's calls.

Three operators sit next to the delta-rule recurrence in such a stack: attention with a sliding
window and a few first tokens that stay visible (sinks), the short causal convolution in front of
a recurrent layer, and the selective state space scan.  Each has a prompt form, a training form
(forward and backward) and a form for single tokens that updates a state of constant size.

A case names its path in ``op``:

attn_prompt   T queries at positions start .. start+T-1 over start+T keys
attn_train    forward and backward over a whole sequence
attn_step     one token per sequence over a ring cache of sinks + window slots
conv_prompt, conv_train, conv_step
scan_prompt, scan_train, scan_step
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a short first message of one conversation: one small launch, latency is all
        _attn("attn_prompt", "attn_prompt_first", B=1, T=96, H=8, Hk=2, d=64, window=1024, sinks=4),
        # a batch of prompts of different lengths, as a server packs them
        _attn("attn_prompt", "attn_prompt_batch", B=2, T=4096, H=16, Hk=4, d=128, window=1024,
              sinks=4, ragged=True),
        # one long document
        _attn("attn_prompt", "attn_prompt_long", B=1, T=16384, H=16, Hk=4, d=128, window=2048,
              sinks=4),
        # the next piece of a prompt over the keys so far, odd sizes, full precision
        _attn("attn_prompt", "attn_chunk_fp32", B=2, T=333, H=6, Hk=3, d=64, window=257, sinks=3,
              start=1000, dtype="fp32"),
        # a training step of an attention layer
        _attn("attn_train", "attn_train", B=2, T=4096, H=16, Hk=4, d=128, window=512, sinks=4),
        # a serving step of a large batch, whose sequences have different lengths
        _attn("attn_step", "attn_step_batch", B=256, T=1, H=16, Hk=4, d=128, window=1024, sinks=4,
              ragged=True),
        # one conversation with a long window: few rows, a long axis
        _attn("attn_step", "attn_step_one", B=1, T=1, H=16, Hk=4, d=128, window=32768, sinks=4),
        # a training step of the convolution in front of a recurrent layer
        _ssm("conv_train", "conv_train", B=8, T=2048, D=2048, K=4),
        # a serving step of it
        _ssm("conv_step", "conv_step", B=256, T=1, D=4096, K=4),
        # one long prompt through a scan layer: few rows, a long axis
        _ssm("scan_prompt", "scan_prompt", B=1, T=8192, D=2048, N=16, K=4),
        # a training step of a scan layer
        _ssm("scan_train", "scan_train", B=4, T=2048, D=2048, N=16, K=4),
        # a serving step of it
        _ssm("scan_step", "scan_step", B=256, T=1, D=4096, N=16, K=4),
    ]


def _attn(op, name=None, *, B, T, H, Hk, d, window, sinks, start=0, ragged=False, dtype="bf16"):
    case = dict(op=op, B=B, T=T, H=H, Hk=Hk, d=d, window=window, sinks=sinks, start=start,
                ragged=ragged, dtype=dtype)
    return case if name is None else dict(case, name=name)


def _ssm(op, name=None, *, B, T, D, K, N=16, G=1, gated=True, ragged=False, dtype="bf16"):
    case = dict(op=op, B=B, T=T, D=D, K=K, N=N, G=G, gated=gated, ragged=ragged, dtype=dtype)
    return case if name is None else dict(case, name=name)


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_prompt", "attn_prompt", "attn_train", "attn_train", "attn_step",
                     "conv_prompt", "conv_train", "conv_step", "scan_prompt", "scan_train",
                     "scan_step"])
    dtype, train = rng.choice(["bf16", "bf16", "bf16", "fp32"]), op == "attn_train"
    like = "conv_train" if op == "conv_prompt" else op
    most = max(_cost(c) for c in listed() if c["op"] == like)
    while True:
        if op.startswith("attn"):
            Hk = rng.choice([1, 2, 3, 4, 8])
            case = _attn(op, B=_log_int(rng, 1, 256) if op == "attn_step" else rng.randint(1, 5),
                         T=1 if op == "attn_step" else _log_int(rng, 32 if train else 1, 16384),
                         H=Hk * rng.choice([1, 2, 4, 5, 8]), Hk=Hk, d=rng.choice([64, 128, 128]),
                         window=_log_int(rng, 16 if train else 1,
                                         32768 if op == "attn_step" else 8192),
                         sinks=rng.choice([0, 1, 4, 4, 16, 100]),
                         start=rng.choice([0, 0, _log_int(rng, 1, 4000)]) if op == "attn_prompt" else 0,
                         ragged=rng.random() < 0.5, dtype=dtype)
        else:
            G = rng.choice([1, 1, 2])
            case = _ssm(op, B=_log_int(rng, 1, 512) if op.endswith("step") else rng.randint(1, 8),
                        T=1 if op.endswith("step") else _log_int(rng, 1, 8192),
                        D=G * rng.choice([_log_int(rng, 16, 4096), 8 * _log_int(rng, 2, 512)]),
                        K=rng.choice([2, 3, 4, 4]), N=rng.choice([8, 16, 16, 32]), G=G,
                        gated=rng.random() < 0.7, ragged=rng.random() < 0.3, dtype=dtype)
        if _cost(case) <= most and _footprint(case) <= 1 << 32:
            return case


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 50 * (8 if case["dtype"] == "fp32" else 1)


def _footprint(case):
    """Values of the largest array that the plain form holds."""
    c = case
    if c["op"].startswith("attn"):
        if c["op"] == "attn_step":
            return c["B"] * c["H"] * (c["window"] + c["sinks"]) * c["d"]
        return c["B"] * c["H"] * c["T"] * (c["start"] + c["T"]) * (4 if c["op"] == "attn_train" else 1)
    return c["B"] * c["T"] * c["D"] * (c["N"] if c["op"].startswith("scan") else 1) * 4


def _pairs(c):
    """(query, key) pairs that are visible in full-length sequences, per head."""
    def upto(p):                       # keys that position p sees
        return min(p + 1, c["window"]) + max(0, min(c["sinks"], p + 1 - c["window"]))
    first, last = c["start"], c["start"] + c["T"]
    knee = c["window"] + c["sinks"]    # from here on the count is constant
    total = sum(map(upto, range(first, min(last, max(first, knee)))))
    return total + max(0, last - max(first, knee)) * upto(knee)


def work(case):
    c, e = case, 4 if case["dtype"] == "fp32" else 2
    if c["op"] in ("attn_prompt", "attn_train"):
        rows, keys = c["B"] * c["T"] * c["H"] * c["d"], c["B"] * (c["start"] + c["T"]) * c["Hk"] * c["d"]
        pairs = c["B"] * c["H"] * _pairs(c)
        if c["op"] == "attn_prompt":   # q, k, v in; out and lse out
            return {"bytes": e * (2 * rows + 2 * keys) + 4 * c["B"] * c["T"] * c["H"],
                    "flops": 4 * c["d"] * pairs}
        return {"bytes": e * (4 * rows + 4 * keys) + 4 * c["B"] * c["T"] * c["H"],
                "flops": 14 * c["d"] * pairs}
    if c["op"] == "attn_step":         # the visible slots of both caches, the new token's rows
        slots = c["window"] + c["sinks"]
        slots = slots / 2 if c["ragged"] else slots
        return {"bytes": e * (2 * c["B"] * c["Hk"] * c["d"] * (slots + 2) + 2 * c["B"] * c["H"] * c["d"]),
                "flops": 4 * c["B"] * c["H"] * slots * c["d"]}
    n = c["B"] * c["T"] * c["D"]
    if c["op"] == "conv_step":         # x, state in; y, state out; weights
        return {"bytes": e * n * (2 + 2 * (c["K"] - 1)) + 4 * c["D"] * (c["K"] + 1),
                "flops": 2 * c["K"] * n}
    if c["op"].startswith("conv"):
        train = c["op"] == "conv_train"
        return {"bytes": e * n * (4 if train else 2) + 4 * c["D"] * (c["K"] + 1) * (2 if train else 1),
                "flops": (6 if train else 2) * c["K"] * n}
    N, groups = c["N"], 2 * c["B"] * c["T"] * c["G"] * c["N"]
    act = 3 + c["gated"]               # x, dt, y and z
    state = 4 * c["B"] * c["D"] * N
    weights = 4 * c["D"] * (N + 2)
    if c["op"] == "scan_step":
        return {"bytes": e * (n * act + groups) + 2 * state + weights, "flops": 7 * n * N}
    if c["op"] == "scan_prompt":
        return {"bytes": e * (n * act + groups) + state + weights, "flops": 7 * n * N}
    return {"bytes": e * (n * (act + act) + 2 * groups) + 2 * weights, "flops": 24 * n * N}


# ----------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DTYPES[c["dtype"]]

    def rand(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def lengths(n, lo, hi):
        return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)

    s = {"case": c}
    if c["op"].startswith("attn"):
        B, T, H, Hk, d = c["B"], c["T"], c["H"], c["Hk"], c["d"]
        # queries lean towards one direction per kv head and the first tokens' keys lie along it,
        # as the keys of sink tokens do
        u = torch.nn.functional.normalize(torch.randn(Hk, d, generator=g, device="cuda"), dim=-1)
        lean = u.repeat_interleave(H // Hk, 0) * (0.15 * math.sqrt(d))
        if c["op"] == "attn_step":
            C = c["sinks"] + c["window"]
            s["q"] = (rand(B, H, d, dtype=torch.float32) + lean).to(dt)
            s["k"], s["v"] = rand(B, Hk, d), rand(B, Hk, d)
            s["k_cache"], s["v_cache"] = rand(B, Hk, C, d), rand(B, Hk, C, d)
            if c["sinks"]:
                s["k_cache"][:, :, :c["sinks"]] += (2 * u[:, None]).to(dt)
            # ragged: from sequences that have just begun to ones that have filled the ring,
            # and free places of the batch (-1)
            s["pos"] = (lengths(B, -1, c["window"] + c["sinks"] - 1) if c["ragged"]
                        else lengths(B, C, 3 * C))
            return s
        S = c["start"] + T
        # slices of one projection's output, as a layer has them
        qkv = rand(B, S, (H + 2 * Hk), d)
        qkv[:, :, :H] += lean.to(dt)
        if c["sinks"]:
            qkv[:, :c["sinks"], H:H + Hk] += (2 * u).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, c["start"]:, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:]
        s["lens"] = lengths(B, (S + 1) // 2, S) if c["ragged"] else None
        if c["op"] == "attn_train":
            s["d_out"] = rand(B, T, H, d)
        return s
    B, T, D, K = c["B"], c["T"], c["D"], c["K"]
    s["lens"] = lengths(B, (T + 1) // 2, T) if c["ragged"] and T > 1 else None
    if c["op"].startswith("conv"):
        s["x"] = rand(B, T, D)
        s["weight"] = rand(D, K, dtype=torch.float32, scale=1 / math.sqrt(K))
        s["bias"] = rand(D, dtype=torch.float32, scale=0.2)
        s["state"] = rand(B, K - 1, D)
        if c["op"] == "conv_train":
            s["d_y"] = rand(B, T, D)
        if c["op"] == "conv_step":
            s["x"] = s["x"][:, 0]
        return s
    N, G = c["N"], c["G"]
    s["x"] = torch.nn.functional.silu(rand(B, T, D, dtype=torch.float32)).to(dt)
    s["dt"] = rand(B, T, D, scale=0.5)
    s["z"] = rand(B, T, D) if c["gated"] else None
    s["B"], s["C"] = rand(B, T, G, N), rand(B, T, G, N)
    # decay rates 1 .. N and time steps 0.001 .. 0.1, as such layers begin with
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(rand(D, N, dtype=torch.float32, scale=0.1))
    step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = rand(D, dtype=torch.float32, scale=0.2) + 1
    s["state"] = rand(B, D, N, dtype=torch.float32, scale=0.3)
    if c["op"] == "scan_train":
        s["d_y"], s["state"] = rand(B, T, D), None
    if c["op"] == "scan_step":
        for k in ("x", "dt", "z", "B", "C"):
            s[k] = None if s[k] is None else s[k][:, 0]
    return s


# ------------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from recurrent_associative_memory_gb300 import attention, ssm
    c, op = s["case"], s["case"]["op"]
    if op == "attn_prompt":
        out, _ = attention.window_attn_fwd(s["q"], s["k"], s["v"], c["window"], c["sinks"],
                                           q_start=c["start"], lens=s["lens"])
        return {"out": out}
    if op == "attn_train":
        out, lse = attention.window_attn_fwd(s["q"], s["k"], s["v"], c["window"], c["sinks"],
                                             lens=s["lens"], want_lse=True)
        g = attention.window_attn_bwd(s["q"], s["k"], s["v"], out, lse, s["d_out"], c["window"],
                                      c["sinks"], lens=s["lens"])
        return {"out": out, "lse": lse, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    if op == "attn_step":
        out = attention.window_attn_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                         s["pos"], c["window"], c["sinks"])
        return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "conv_prompt":
        y, state = ssm.short_conv_fwd(s["x"], s["weight"], s["bias"], init_state=s["state"],
                                      lens=s["lens"])
        return {"y": y, "state": state}
    if op == "conv_train":
        y, _ = ssm.short_conv_fwd(s["x"], s["weight"], s["bias"], lens=s["lens"], want_final=False)
        g = ssm.short_conv_bwd(s["x"], s["weight"], s["bias"], s["d_y"], lens=s["lens"])
        return {"y": y, "dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"]}
    if op == "conv_step":
        y, state = ssm.short_conv_step(s["x"], s["weight"], s["bias"], s["state"],
                                       state_out=torch.empty_like(s["state"]))
        return {"y": y, "state": state}
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "scan_prompt":
        y, state = ssm.selective_scan_fwd(*args, **kw, init_state=s["state"], lens=s["lens"])
        return {"y": y, "state": state}
    if op == "scan_train":
        y, _ = ssm.selective_scan_fwd(*args, **kw, lens=s["lens"], want_final=False)
        g = ssm.selective_scan_bwd(*args, s["d_y"], **kw, lens=s["lens"])
        return {"y": y, **{k: g[k] for k in ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "ddt_bias")
                           if k in g}}
    y, state = ssm.selective_scan_step(*args, s["state"], **kw, state_out=torch.empty_like(s["state"]))
    return {"y": y, "state": state}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "attn_step":
        return _plain_attn_step(s)
    if op.startswith("attn"):
        return _plain_attn(s)
    if op == "conv_step":
        return _plain_conv_step(s)
    if op.startswith("conv"):
        return _plain_conv(s)
    if op == "scan_step":
        return _plain_scan_step(s)
    return _plain_scan(s)


# ------------------------------------------------------------------------------ plain forms

def _plain_attn(s):
    c = s["case"]
    B, T, H, Hk, d = c["B"], c["T"], c["H"], c["Hk"], c["d"]
    S, r, scale, dt = c["start"] + T, H // Hk, 1 / math.sqrt(d), s["q"].dtype
    q = s["q"].float().permute(0, 2, 1, 3).reshape(B, Hk, r, T, d)
    k = s["k"].float().permute(0, 2, 1, 3)[:, :, None]
    v = s["v"].float().permute(0, 2, 1, 3)[:, :, None]
    p = c["start"] + torch.arange(T, device="cuda")[:, None]
    j = torch.arange(S, device="cuda")[None]
    seen = (j <= p) & ((p - j < c["window"]) | (j < c["sinks"]))
    if s["lens"] is not None:
        seen = seen & (j < s["lens"][:, None, None])
        seen = seen[:, None, None]
    w = (q * scale) @ k.transpose(-1, -2)
    w.masked_fill_(~seen, -math.inf)
    m = w.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    w.sub_(m).exp_()
    l = w.sum(-1, keepdim=True)
    some = l > 0
    out = torch.where(some, (w @ v) / torch.where(some, l, torch.ones_like(l)), torch.zeros_like(q))
    lay = lambda t, h: t.reshape(B, h, -1, d).permute(0, 2, 1, 3).contiguous()  # noqa: E731
    if c["op"] == "attn_prompt":
        return {"out": lay(out, H).to(dt)}
    lse = (m + torch.log(l)).reshape(B, H, T)
    w.div_(torch.where(some, l, torch.ones_like(l)))
    do = s["d_out"].float().permute(0, 2, 1, 3).reshape(B, Hk, r, T, d)
    dv = (w.transpose(-1, -2) @ do).sum(2)
    ds = do @ v.transpose(-1, -2)
    ds.sub_((do * out).sum(-1, keepdim=True)).mul_(w)
    dq = ds @ k * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2) * scale
    return {"out": lay(out, H).to(dt), "lse": lse, "dq": lay(dq, H).to(dt), "dk": lay(dk, Hk).to(dt),
            "dv": lay(dv, Hk).to(dt)}


def _plain_attn_step(s):
    c = s["case"]
    B, H, Hk, d, W, n = c["B"], c["H"], c["Hk"], c["d"], c["window"], c["sinks"]
    p = s["pos"].long()
    slot = torch.where(p < n, p, n + (p - n) % W)
    rows = torch.arange(B, device="cuda")
    live, at = (p >= 0)[:, None, None], slot.clamp(min=0)
    s["k_cache"][rows, :, at] = torch.where(live, s["k"], s["k_cache"][rows, :, at])
    s["v_cache"][rows, :, at] = torch.where(live, s["v"], s["v_cache"][rows, :, at])
    e = torch.arange(n + W, device="cuda")[None]
    held = torch.where(e < n, e, p[:, None] - (p[:, None] - e) % W)   # the position in each slot
    seen = (held <= p[:, None]) & ((e < n) | (held >= n))
    q = s["q"].float().reshape(B, Hk, H // Hk, d) / math.sqrt(d)
    w = q @ s["k_cache"].float().transpose(-1, -2)
    w = w.masked_fill(~seen[:, None, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = w.sum(-1, keepdim=True)
    out = (w @ s["v_cache"].float()) / torch.where(l > 0, l, torch.ones_like(l))
    return {"out": out.reshape(B, H, d).to(s["q"].dtype), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _plain_conv(s):
    c, x, w = s["case"], s["x"].float(), s["weight"]
    B, T, D, K = c["B"], c["T"], c["D"], c["K"]
    train = c["op"] == "conv_train"
    past = torch.zeros(B, K - 1, D, device="cuda") if train else s["state"].float()
    ext = torch.cat([past, x], 1)
    pre = s["bias"] + sum(ext[:, j:j + T] * w[:, j] for j in range(K))
    sig = torch.sigmoid(pre)
    y = pre * sig
    lens = s["lens"]
    if lens is None:
        end = ext[:, T:]
    else:
        real = (torch.arange(T, device="cuda")[None] < lens[:, None])[..., None]
        y = torch.where(real, y, torch.zeros_like(y))
        at = lens.long()[:, None] + torch.arange(K - 1, device="cuda")
        end = torch.gather(ext, 1, at[..., None].expand(-1, -1, D))
    dt = s["x"].dtype
    if not train:
        return {"y": y.to(dt), "state": end.to(dt)}
    dpre = s["d_y"].float() * sig * (1 + pre * (1 - sig))
    if lens is not None:
        dpre = torch.where(real, dpre, torch.zeros_like(dpre))
    later = torch.cat([dpre, torch.zeros(B, K - 1, D, device="cuda")], 1)
    dx = sum(later[:, K - 1 - j:K - 1 - j + T] * w[:, j] for j in range(K))
    dw = torch.stack([(ext[:, j:j + T] * dpre).sum((0, 1)) for j in range(K)], 1)
    return {"y": y.to(dt), "dx": dx.to(dt), "dweight": dw, "dbias": dpre.sum((0, 1))}


def _plain_conv_step(s):
    ext = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = s["bias"] + (ext.float() * s["weight"].t()).sum(1)
    return {"y": (pre * torch.sigmoid(pre)).to(s["x"].dtype), "state": ext[:, 1:].contiguous()}


def _doubling_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from zero, by doubling the span."""
    span, T = 1, a.shape[1]
    while span < T:
        b = torch.cat([b[:, :span], b[:, span:] + a[:, span:] * b[:, :-span]], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return b


def _plain_scan(s):
    c, dt_ = s["case"], s["x"].dtype
    B, T, D, N, G = c["B"], c["T"], c["D"], c["N"], c["G"]
    x, A = s["x"].float(), s["A"]
    raw = s["dt"].float() + s["dt_bias"]
    dt = torch.nn.functional.softplus(raw)
    if s["lens"] is not None:
        real = (torch.arange(T, device="cuda")[None] < s["lens"][:, None])[..., None]
        dt = torch.where(real, dt, torch.zeros_like(dt))
    Bt = s["B"].float().repeat_interleave(D // G, 2)
    Ct = s["C"].float().repeat_interleave(D // G, 2)
    a = torch.exp(dt[..., None] * A)
    b = (dt * x)[..., None] * Bt
    if s["state"] is not None:
        b[:, 0] += a[:, 0] * s["state"]
    h = _doubling_scan(a, b)
    y = (h * Ct).sum(-1) + s["D"] * x
    gate = 1.0
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        gate = z * sig
    out = y * gate
    if s["lens"] is not None:
        out = torch.where(real, out, torch.zeros_like(out))
    if c["op"] == "scan_prompt":
        return {"y": out.to(dt_), "state": h[:, -1].contiguous()}
    do = s["d_y"].float()
    if s["lens"] is not None:
        do = torch.where(real, do, torch.zeros_like(do))
    r = {"y": out.to(dt_)}
    if s["z"] is not None:
        r["dz"] = (do * y * sig * (1 + z * (1 - sig))).to(dt_)
    dy = do * gate
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _doubling_scan(after.flip(1), (dy[..., None] * Ct).flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    e = g * a * before
    gB = (g * Bt).sum(-1)
    ddt = (e * A).sum(-1) + gB * x
    ddt = ddt * torch.sigmoid(raw)
    if s["lens"] is not None:
        ddt = torch.where(real, ddt, torch.zeros_like(ddt))
    per_group = lambda t: t.reshape(B, T, G, D // G, N).sum(3).to(dt_)  # noqa: E731
    return r | {"dx": (gB * dt + s["D"] * dy).to(dt_), "ddt": ddt.to(dt_),
                "dA": (e * dt[..., None]).sum((0, 1)),
                "dB": per_group(g * (dt * x)[..., None]), "dC": per_group(h * dy[..., None]),
                "dD": (dy * x).sum((0, 1)), "ddt_bias": ddt.sum((0, 1))}


def _plain_scan_step(s):
    D, G = s["case"]["D"], s["case"]["G"]
    x, dt = s["x"].float(), torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
    Bt = s["B"].float().repeat_interleave(D // G, 1)
    Ct = s["C"].float().repeat_interleave(D // G, 1)
    h = torch.exp(dt[..., None] * s["A"]) * s["state"] + (dt * x)[..., None] * Bt
    y = (h * Ct).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": y.to(s["x"].dtype), "state": h}


# --------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn_step":
        return _exact_attn_step(s)
    if op.startswith("attn"):
        return _exact_attn(s)
    if op.startswith("conv"):
        return _exact_conv(s)
    return _exact_scan(s)


def _exact_attn(s):
    """Block of queries by block of queries, over the keys that the block can see."""
    c = s["case"]
    B, T, H, Hk, d, W, n = c["B"], c["T"], c["H"], c["Hk"], c["d"], c["window"], c["sinks"]
    start, S, r = c["start"], c["start"] + T, H // Hk
    train = c["op"] == "attn_train"
    out = torch.zeros(B, T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(out)
    dk = torch.zeros(B, S, Hk, d, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    step = 512
    for b in range(B):
        n_keys = S if s["lens"] is None else int(s["lens"][b])
        for h in range(H):
            kh, vh = s["k"][b, :, h // r].double(), s["v"][b, :, h // r].double()
            for i in range(0, T, step):
                pos = start + torch.arange(i, min(T, i + step), device="cuda")
                lo, hi = max(0, int(pos[0]) - W + 1), min(n_keys, int(pos[-1]) + 1)
                lo = min(lo, max(hi, 0))
                first = torch.arange(0, min(n, lo, n_keys), device="cuda")
                at = torch.cat([first, torch.arange(lo, max(lo, hi), device="cuda")])
                if not len(at):
                    continue
                ok = (at <= pos[:, None]) & ((pos[:, None] - at < W) | (at < n))
                any_ = ok.any(1)
                qb = s["q"][b, i:i + step, h].double()
                logits = (qb @ kh[at].t() / math.sqrt(d)).masked_fill(~ok, -math.inf)
                total = torch.logsumexp(logits, 1)
                pr = torch.exp(logits - torch.where(any_, total, 0.0)[:, None])
                ob = pr @ vh[at]
                out[b, i:i + step, h], lse[b, h, i:i + step] = ob, total
                if train:
                    gb = s["d_out"][b, i:i + step, h].double()
                    dlog = pr * (gb @ vh[at].t() - (gb * ob).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[b, i:i + step, h] = dlog @ kh[at]
                    dk[b, :, h // r].index_add_(0, at, dlog.t() @ qb)
                    dv[b, :, h // r].index_add_(0, at, pr.t() @ gb)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else {"out": out}


def _exact_attn_step(s):
    """Sequence by sequence, over the visible positions in their order."""
    c = s["case"]
    H, Hk, W, n = c["H"], c["Hk"], c["window"], c["sinks"]
    out = torch.zeros(c["B"], H, c["d"], dtype=torch.float64, device="cuda")
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    for b, p in enumerate(s["pos"].tolist()):
        if p < 0:
            continue
        here = p if p < n else n + (p - n) % W
        kc[b, :, here], vc[b, :, here] = s["k"][b], s["v"][b]
        at = torch.cat([torch.arange(0, min(n, p + 1)), torch.arange(max(min(n, p + 1), p - W + 1), p + 1)])
        at = torch.where(at < n, at, n + (at - n) % W).cuda()
        kb, vb = kc[b][:, at].double(), vc[b][:, at].double()
        pr = torch.softmax(s["q"][b].double().reshape(Hk, H // Hk, -1) @ kb.transpose(1, 2)
                           / math.sqrt(c["d"]), -1)
        out[b] = (pr @ vb).reshape(H, -1)
    return {"out": out, "k_cache": kc, "v_cache": vc}


def _exact_conv(s):
    """Through the library's convolution and automatic differentiation, in 64 bits."""
    c = s["case"]
    B, D, K = c["B"], c["D"], c["K"]
    x = s["x"].double().reshape(B, -1, D).requires_grad_()
    w, bias = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    past = torch.zeros_like(s["state"]) if c["op"] == "conv_train" else s["state"]
    ext = torch.cat([past.double(), x], 1)
    y = torch.nn.functional.silu(torch.nn.functional.conv1d(ext.transpose(1, 2), w[:, None], bias,
                                                            groups=D).transpose(1, 2))
    lens = [x.shape[1]] * B if s["lens"] is None else s["lens"].tolist()
    keep = torch.tensor(lens, device="cuda")[:, None] > torch.arange(x.shape[1], device="cuda")
    y = y * keep[..., None]
    if c["op"] == "conv_train":
        dx, dw, db = torch.autograd.grad(y, (x, w, bias), s["d_y"].double())
        return {"y": y.detach(), "dx": dx, "dweight": dw, "dbias": db}
    end = torch.stack([ext[b, n:n + K - 1] for b, n in enumerate(lens)]).detach()
    y = y.detach()
    return {"y": y[:, 0] if c["op"] == "conv_step" else y, "state": end}


def _exact_scan(s):
    """Token by token, and back again."""
    c = s["case"]
    B, T, D, N, G = c["B"], c["T"], c["D"], c["N"], c["G"]
    train = c["op"] == "scan_train"
    if train and T * B * D * N > 1 << 30:
        return None
    full = lambda t, *sh: t.double().reshape(B, T, *sh)  # noqa: E731
    x, A = full(s["x"], D), s["A"].double()
    raw = full(s["dt"], D) + s["dt_bias"].double()
    dt = torch.where(raw > 40, raw, torch.log1p(torch.exp(raw.clamp(max=40))))
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"]
    keep = (torch.arange(T, device="cuda") < lens[:, None])[..., None].double()
    dt = dt * keep
    of = torch.arange(D, device="cuda") // (D // G)
    Bm, Cm = full(s["B"], G, N), full(s["C"], G, N)
    h = torch.zeros(B, D, N, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    y, past = torch.zeros_like(x), []
    for t in range(T):
        if train:
            past.append(h)
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * Bm[:, t][:, of]
        y[:, t] = torch.einsum("bdn,bdn->bd", h, Cm[:, t][:, of]) + s["D"].double() * x[:, t]
    z = None if s["z"] is None else full(s["z"], D)
    gate = torch.ones_like(x) if z is None else z / (1 + torch.exp(-z))
    out = y * gate * keep
    if not train:
        return {"y": out[:, 0] if c["op"] == "scan_step" else out, "state": h}
    do = full(s["d_y"], D) * keep
    dy = do * gate
    r = {"y": out}
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        r["dz"] = do * y * (sg + z * sg * (1 - sg))
    dx, ddt = s["D"].double() * dy, torch.zeros_like(x)
    dA = torch.zeros_like(A)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    g = torch.zeros_like(h)
    for t in reversed(range(T)):
        a, b = torch.exp(dt[:, t, :, None] * A), Bm[:, t][:, of]
        now = a * past[t] + (dt[:, t] * x[:, t])[..., None] * b
        dC[:, t] = (now * dy[:, t, :, None]).reshape(B, G, -1, N).sum(2)
        g = g + dy[:, t, :, None] * Cm[:, t][:, of]
        dB[:, t] = (g * (dt[:, t] * x[:, t])[..., None]).reshape(B, G, -1, N).sum(2)
        gb = (g * b).sum(-1)
        dx[:, t] += gb * dt[:, t]
        g = g * a
        ddt[:, t] = (g * past[t] * A).sum(-1) + gb * x[:, t]
        dA += (g * past[t] * dt[:, t, :, None]).sum(0)
    ddt = ddt * keep / (1 + torch.exp(-raw))
    return r | {"dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": (dy * x).sum((0, 1)),
                "ddt_bias": ddt.sum((0, 1))}
