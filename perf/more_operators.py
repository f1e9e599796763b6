"""What stands between the mixers of a hybrid stack, in its plain form and as the framework's calls.

Two operators make a block of a mixer: the matrix product with its bias, activation and residual
(projections into and out of a mixer, the two layers of a channel mixer), and the norms before
and after the mixer, fused with the gate and the scale of what it adds to the residual stream.

    y = act(x W + bias) + residual

    h' = h + scale * f(gate) * n(branch; post_weight)
    y  = n(h'; pre_weight)            n(x; w) = w * x / sqrt(mean(x^2) + eps)

A case names its path in ``op``:

linear         the product, for prompts and for single tokens
linear_train   with its gradients
norm           the norms around a block, for prompts and for single tokens
norm_train     with their gradients
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the projection out of a mixer for one conversation's next token: latency is all
        _linear("linear", "linear_token", M=1, K=2048, N=2048, residual=True),
        # the wide layer of a channel mixer in a serving step: every weight is read once
        _linear("linear", "linear_step", M=64, K=4096, N=16384, act="silu", bias=True),
        # the projection out of a mixer over a batch of prompts
        _linear("linear", "linear_prompt", M=8192, K=4096, N=4096, residual=True),
        # a ragged batch and sizes that no tile divides, the weight stored the other way round
        _linear("linear", "linear_odd", M=1003, K=1511, N=2051, act="gelu_tanh", bias=True,
                residual=True, transposed=True),
        # full precision, a short prompt
        _linear("linear", "linear_fp32", M=300, K=2048, N=2048, bias=True, dtype="fp32"),
        # a training step of the wide layer of a channel mixer
        _linear("linear_train", "linear_train", M=8192, K=2048, N=8192, act="silu", bias=True),
        # a smaller one in full precision
        _linear("linear_train", "linear_train_fp32", M=2048, K=1024, N=4096, act="gelu_tanh",
                bias=True, dtype="fp32"),
        # between two blocks for one conversation's next token
        _norm("norm", "norm_token", M=1, D=2048, gate="none"),
        # between two blocks in a serving step
        _norm("norm", "norm_step", M=256, D=4096, gate="silu", post=True, scale=True),
        # between two blocks over a batch of prompts
        _norm("norm", "norm_prompt", M=16384, D=4096, gate="sigmoid", post=True, scale=True),
        # a training step
        _norm("norm_train", "norm_train", M=8192, D=4096, gate="silu", post=True, scale=True),
        # a training step of odd sizes, the residual stream in full precision
        _norm("norm_train", "norm_train_odd", M=2731, D=1111, gate="sigmoid", post=True,
              scale=True, stream="fp32"),
    ]


def _linear(op, name=None, *, M, K, N, act="none", bias=False, residual=False, transposed=False,
            dtype="bf16"):
    case = dict(op=op, M=M, K=K, N=N, act=act, bias=bias, residual=residual,
                transposed=transposed, dtype=dtype)
    return case if name is None else dict(case, name=name)


def _norm(op, name=None, *, M, D, gate="none", post=False, scale=False, dtype="bf16",
          stream=None):
    """``stream``: the type of the residual stream.  ``gate``: the gate's function, or "none"
    for a block without a gate."""
    case = dict(op=op, M=M, D=D, gate=gate, post=post, scale=scale, dtype=dtype,
                stream=stream or dtype)
    return case if name is None else dict(case, name=name)


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_train", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    most = max(_cost(c) for c in listed() if c["op"] == op)

    def size(lo, hi):                  # half of them as models have them
        n = _log_int(rng, lo, hi)
        return n if rng.random() < 0.5 else max(64, n // 64 * 64)

    while True:
        if op.startswith("linear"):
            case = _linear(op, M=_log_int(rng, 1, 16384), K=size(16, 8192), N=size(16, 16384),
                           act=rng.choice(["none", "silu", "gelu_tanh"]), bias=rng.random() < 0.5,
                           residual=rng.random() < 0.4, transposed=rng.random() < 0.3, dtype=dtype)
        else:
            case = _norm(op, M=_log_int(rng, 1, 32768), D=size(32, 8192),
                         gate=rng.choice(["none", "sigmoid", "silu"]), post=rng.random() < 0.6,
                         scale=rng.random() < 0.6, dtype=dtype,
                         stream=rng.choice([dtype, "fp32"]))
        if _cost(case) <= most:
            return case


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 50 * (8 if case["dtype"] == "fp32" else 1)


def work(case):
    c, e = case, 4 if case["dtype"] == "fp32" else 2
    if c["op"].startswith("linear"):
        M, K, N = c["M"], c["K"], c["N"]
        io = M * K + K * N + M * N * (1 + c["residual"]) + N * c["bias"]
        if c["op"] == "linear":
            return {"bytes": e * io, "flops": 2 * M * K * N}
        # d_y in; dx, dweight and dbias out
        return {"bytes": e * (io + M * N + M * K + K * N + N * c["bias"]), "flops": 6 * M * K * N}
    n, w = c["M"] * c["D"], 4 * c["D"] * (1 + c["post"] + c["scale"])
    gated, es = c["gate"] != "none", 4 if c["stream"] == "fp32" else 2
    if c["op"] == "norm":              # h, branch and gate in; h and y out
        return {"bytes": n * (2 * es + e * (2 + gated)) + w, "flops": 10 * n}
    # and the gradients of h' and y in; of h, branch and gate out
    return {"bytes": n * (2 * es + e * (2 + gated) + 2 * es + e * (2 + gated)) + 2 * w,
            "flops": 40 * n}


# ----------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    dt = DTYPES[c["dtype"]]

    def rand(*shape, dtype=dt, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)

    s = {"case": c}
    if c["op"].startswith("linear"):
        M, K, N = c["M"], c["K"], c["N"]
        s["x"] = rand(M, K)
        s["weight"] = (rand(N, K, scale=K ** -0.5).t() if c["transposed"]
                       else rand(K, N, scale=K ** -0.5))
        s["bias"] = rand(N, scale=0.3) if c["bias"] else None
        s["residual"] = rand(M, N) if c["residual"] else None
        if c["op"] == "linear_train":
            s["d_y"] = rand(M, N)
        return s
    M, D, st = c["M"], c["D"], DTYPES[c["stream"]]
    # the stream has grown over the blocks before; a few of its channels are far larger
    size = torch.where(torch.rand(D, generator=g, device="cuda") < 0.01, 12.0, 1.5)
    s["h"] = (rand(M, D, dtype=torch.float32) * size).to(st)
    s["branch"] = rand(M, D, scale=0.7)
    s["gate"] = rand(M, D) if c["gate"] != "none" else None
    s["scale"] = rand(D, dtype=torch.float32, scale=0.1) + 0.5 if c["scale"] else None
    s["post_weight"] = rand(D, dtype=torch.float32, scale=0.1) + 1 if c["post"] else None
    s["pre_weight"] = rand(D, dtype=torch.float32, scale=0.1) + 1
    if c["op"] == "norm_train":
        s["d_h"], s["d_y"] = rand(M, D, dtype=st), rand(M, D)
    return s


# ------------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from recurrent_associative_memory_gb300 import block
    c, op = s["case"], s["case"]["op"]
    if op == "linear":
        y, _ = block.linear_fwd(s["x"], s["weight"], s["bias"], act=c["act"],
                                residual=s["residual"])
        return {"y": y}
    if op == "linear_train":
        y, slope = block.linear_fwd(s["x"], s["weight"], s["bias"], act=c["act"],
                                    residual=s["residual"], want_slope=True)
        g = block.linear_bwd(s["x"], s["weight"], s["d_y"], slope=slope, want_dbias=c["bias"])
        return {"y": y, **{k: g[k] for k in ("dx", "dweight", "dbias") if k in g}}
    kw = dict(gate=s["gate"], gate_act=c["gate"], scale=s["scale"], post_norm=c["post"],
              post_weight=s["post_weight"], pre_weight=s["pre_weight"], eps=EPS)
    y, h = block.block_norm_fwd(s["h"], s["branch"], **kw)
    if op == "norm":
        return {"y": y, "h": h}
    g = block.block_norm_bwd(s["h"], s["branch"], d_h=s["d_h"], d_y=s["d_y"], **kw)
    return {"y": y, "h": h, **{k: g[k] for k in _NORM_GRADS if k in g}}


_NORM_GRADS = ("dh", "dbranch", "dgate", "dscale", "dpost_weight", "dpre_weight")


def _run_plain(s):
    return _plain_linear(s) if s["case"]["op"].startswith("linear") else _plain_norm(s)


# ------------------------------------------------------------------------------ plain forms

def _plain_linear(s):
    act, dt = s["case"]["act"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    pre = x @ w
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    if act == "silu":
        sig = torch.sigmoid(pre)
        y = pre * sig
    elif act == "gelu_tanh":
        tanh = torch.tanh(pre * (_GELU + _GELU * 0.044715 * pre * pre))
        y = 0.5 * pre * (1 + tanh)
    else:
        y = pre
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if s["case"]["op"] == "linear":
        return {"y": y.to(dt)}
    d = s["d_y"].float()
    if act == "silu":
        d = d * sig * (1 + pre * (1 - sig))
    elif act == "gelu_tanh":
        inner = _GELU + 3 * _GELU * 0.044715 * pre * pre
        d = d * (0.5 * (1 + tanh) + 0.5 * pre * (1 - tanh * tanh) * inner)
    r = {"y": y.to(dt), "dx": (d @ w.t()).to(dt), "dweight": (x.t() @ d).to(dt)}
    if s["bias"] is not None:
        r["dbias"] = d.sum(0).to(dt)
    return r


_GELU = math.sqrt(2 / math.pi)


def _plain_norm(s):
    c, dt, st = s["case"], s["branch"].dtype, s["h"].dtype
    h, u = s["h"].float(), s["branch"].float()
    if c["post"]:
        rstd_u = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
        hat = u * rstd_u
        u = hat * s["post_weight"]
    a = torch.ones((), device="cuda")
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = torch.sigmoid(z)
        a = z * sig if c["gate"] == "silu" else sig
    scale = a if s["scale"] is None else s["scale"] * a
    h = h + scale * u
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    normed = h * rstd
    r = {"y": (normed * s["pre_weight"]).to(dt), "h": h.to(st)}
    if c["op"] == "norm":
        return r
    dy = s["d_y"].float()
    t = dy * s["pre_weight"]
    dh = s["d_h"].float() + rstd * (t - normed * (t * normed).mean(-1, keepdim=True))
    r["dh"] = dh.to(st)
    du = dh * scale
    if c["post"]:
        t = du * s["post_weight"]
        r["dbranch"] = (rstd_u * (t - hat * (t * hat).mean(-1, keepdim=True))).to(dt)
    else:
        r["dbranch"] = du.to(dt)
    if s["gate"] is not None:
        slope = sig * (1 + z * (1 - sig)) if c["gate"] == "silu" else sig * (1 - sig)
        dgate = dh * u * slope
        r["dgate"] = (dgate if s["scale"] is None else dgate * s["scale"]).to(dt)
    if s["scale"] is not None:
        r["dscale"] = (dh * a * u).sum(0)
    if c["post"]:
        r["dpost_weight"] = (du * hat).sum(0)
    r["dpre_weight"] = (dy * normed).sum(0)
    return r


# --------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(s) if case["op"].startswith("linear") else _exact_norm(s)


def _leaf(t):
    return None if t is None else t.detach().double().requires_grad_()


def _exact_linear(s):
    """Through automatic differentiation, in 64 bits."""
    c = s["case"]
    train = c["op"] == "linear_train"
    x, w, bias = _leaf(s["x"]), _leaf(s["weight"]), _leaf(s["bias"])
    with torch.set_grad_enabled(train):
        y = torch.einsum("mk,kn->mn", x, w)
        if bias is not None:
            y = y + bias
        if c["act"] == "silu":
            y = y / (1 + torch.exp(-y))
        elif c["act"] == "gelu_tanh":
            y = torch.nn.functional.gelu(y, approximate="tanh")
        if s["residual"] is not None:
            y = y + s["residual"].double()
    if not train:
        return {"y": y}
    wanted = {"dx": x, "dweight": w} | ({} if bias is None else {"dbias": bias})
    grads = torch.autograd.grad(y, list(wanted.values()), s["d_y"].double())
    return {"y": y.detach(), **dict(zip(wanted, grads))}


def _exact_norm(s):
    """Through automatic differentiation, in 64 bits, blocks of rows by blocks of rows."""
    c = s["case"]
    train = c["op"] == "norm_train"
    vec = {k: _leaf(s[k]) for k in ("scale", "post_weight", "pre_weight") if s[k] is not None}
    names = ["h", "branch"] + (["gate"] if s["gate"] is not None else [])
    parts, sums = [], {k: torch.zeros_like(v) for k, v in vec.items()}

    def n(x, w):
        return x * w * (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) ** -0.5

    for i in range(0, c["M"], 4096):
        rows = {k: _leaf(s[k][i:i + 4096]) for k in names}
        with torch.set_grad_enabled(train):
            add = rows["branch"]
            if c["post"]:
                add = n(add, vec["post_weight"])
            if "gate" in rows:
                f = 1 / (1 + torch.exp(-rows["gate"]))
                add = add * (f * rows["gate"] if c["gate"] == "silu" else f)
            if "scale" in vec:
                add = add * vec["scale"]
            h = rows["h"] + add
            y = n(h, vec["pre_weight"])
        part = {"y": y.detach(), "h": h.detach()}
        if train:
            leaves = rows | vec
            got = dict(zip(leaves, torch.autograd.grad(
                (h, y), list(leaves.values()),
                (s["d_h"][i:i + 4096].double(), s["d_y"][i:i + 4096].double()))))
            part |= {"d" + k: got[k] for k in names}
            for k in vec:
                sums[k] += got[k]
        parts.append(part)
    r = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return {**r, **{"d" + k: v.detach() for k, v in sums.items()}} if train else r
