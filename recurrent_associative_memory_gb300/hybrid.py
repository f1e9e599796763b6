"""A small hybrid stack: a delta-rule layer, a selective scan layer and a window-attention
layer, as a model would run them together, for prompts and for single tokens.

Each layer is ``h + mixer(norm(h))``.  Between two mixers one call adds what the first has given
to the residual stream and takes the norm for the second (``block.block_norm_fwd``), and every
projection is ``block.linear_fwd``:

* ``DeltaLayer``   projections to q, k, v -> short convolutions -> the Kaczmarz linear
  attention recurrence (``dr_chunk_fwd`` / ``dr_decode_step``)
* ``ScanLayer``    projection -> short convolution -> time step, B and C projections ->
  selective scan with its gate
* ``WindowLayer``  projections to q, k, v -> attention with a sliding window and sinks
* ``ChannelLayer`` (with ``channels``) a wide layer with bias and activation and one back; its
  block norms what it gives and adds it with a gate and a scale

``prefill`` runs a batch of prompts of different lengths and returns the logits and the
state; ``step`` takes one token per sequence.  Every layer's serving state has a constant
size: the recurrences' matrices, the convolutions' last inputs, the window's ring of keys
and values.  Weights are random; the projections are plain matrix products.

Run as a program it decodes a few tokens and checks them against the prompt form:
``python -m recurrent_associative_memory_gb300.hybrid``.
"""

from __future__ import annotations

import torch

from . import attention, block, dr, runner, ssm

__all__ = ["HybridStack"]

HEAD = 128   # head size of the delta-rule layer (chunked tensor-core path)


EPS = torch.finfo(torch.float32).eps


def _project(x, weight, **kw):
    return block.linear_fwd(x, weight, **kw)[0]


def _norm(x):
    return torch.nn.functional.rms_norm(x.float(), x.shape[-1:])


def _join(h, o=None, *, gate=None, gate_act="none", scale=None, post_norm=False, post_weight=None):
    """The end of a block that gave o (None: the first one begins) and the start of the next: (the
    norm of h', h').  Rows wider than the norms' kernels take go through plain operations."""
    if h.shape[-1] <= block.MAX_CHANNELS:
        return block.block_norm_fwd(h, o, gate=gate, gate_act=gate_act, scale=scale, post_norm=post_norm,
                                    post_weight=post_weight, eps=EPS)
    if o is not None:
        u = _norm(o) * post_weight if post_norm else o.float()
        if gate is not None:
            u = u * (torch.sigmoid(gate.float()) if gate_act == "sigmoid" else gate.float())
        h = (h.float() + (u if scale is None else u * scale)).to(h.dtype)
    return _norm(h).to(h.dtype), h


class _Layer:
    end = {}     # how its block adds what it gives to the stream, besides the layer's gate

    def __init__(self, gen, dim, device):
        self.gen, self.dim, self.device = gen, dim, device

    def matrix(self, n_in, n_out):
        w = torch.randn(n_in, n_out, generator=self.gen) * n_in ** -0.5
        return w.to(self.device, torch.bfloat16)

    def gate(self, x):
        """A gate on what the layer gives, from the layer's input."""
        return None

    def vector(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.gen) * scale).to(self.device)


class DeltaLayer(_Layer):
    """Short convolutions on q, k and v, then the Kaczmarz recurrence with a decay per head."""

    def __init__(self, gen, dim, device, K=4):
        super().__init__(gen, dim, device)
        self.H = dim // HEAD
        self.qkv, self.out = self.matrix(dim, 3 * dim), self.matrix(dim, dim)
        self.gates = self.matrix(dim, 2 * self.H)
        self.conv_w = self.vector(3 * dim, K, scale=K ** -0.5)

    def inputs(self, x, mixed):
        """The recurrence's inputs from the layer's input and the convolved projections."""
        q, k, v = (t.reshape(*t.shape[:-1], self.H, HEAD).contiguous()
                   for t in mixed.chunk(3, -1))
        g = _project(x, self.gates).float()
        return dict(q=q, k=k, v=v, variant="kla", chunk=64, q_l2norm=True, eps=1e-6,
                    eta=torch.sigmoid(g[..., :self.H]).contiguous(),
                    log_alpha=-torch.nn.functional.softplus(g[..., self.H:] + 2.0).contiguous())

    def prefill(self, x, lens):
        mixed, conv = ssm.short_conv_fwd(_project(x, self.qkv), self.conv_w, lens=lens)
        inp = self.inputs(x, mixed)
        # tokens past a sequence's end neither write to the memory nor let it decay
        past = torch.arange(x.shape[1], device=x.device)[None] >= lens[:, None]
        inp["eta"].masked_fill_(past[..., None], 0.0)
        inp["log_alpha"].masked_fill_(past[..., None], 0.0)
        o, memory, _ = runner.chunk_fwd(inp)
        return _project(o.flatten(2), self.out), (conv, memory)

    def step(self, x, state, pos):
        conv, memory = state
        mixed, _ = ssm.short_conv_step(_project(x, self.qkv), self.conv_w, None, conv)
        return _project(runner.decode_step(self.inputs(x, mixed), memory).flatten(1), self.out)


class ScanLayer(_Layer):
    """A short convolution, then the selective scan with N states per channel and a gate."""

    def __init__(self, gen, dim, device, K=4, N=16):
        super().__init__(gen, dim, device)
        self.N = N
        self.xz, self.out = self.matrix(dim, 2 * dim), self.matrix(dim, dim)
        self.select = self.matrix(dim, dim + 2 * N)   # time step, B, C
        self.conv_w = self.vector(dim, K, scale=K ** -0.5)
        self.A = -torch.arange(1, N + 1, device=device).float().repeat(dim, 1)
        self.D = torch.ones(dim, device=device)
        self.dt_bias = self.vector(dim, scale=0.5) - 3.0

    def scan_inputs(self, mixed, z):
        s = _project(mixed, self.select)
        bc = s[..., self.dim:].unflatten(-1, (2, 1, self.N))
        return dict(x=mixed, dt=s[..., :self.dim], A=self.A, B=bc[..., 0, :, :], C=bc[..., 1, :, :],
                    D=self.D, z=z, dt_bias=self.dt_bias)

    def prefill(self, x, lens):
        xz = _project(x, self.xz)
        mixed, conv = ssm.short_conv_fwd(xz[..., :self.dim], self.conv_w, lens=lens)
        y, states = ssm.selective_scan_fwd(**self.scan_inputs(mixed, xz[..., self.dim:]), lens=lens)
        return _project(y, self.out), (conv, states)

    def step(self, x, state, pos):
        conv, states = state
        xz = _project(x, self.xz)
        mixed, _ = ssm.short_conv_step(xz[:, :self.dim], self.conv_w, None, conv)
        y, _ = ssm.selective_scan_step(**self.scan_inputs(mixed, xz[:, self.dim:]), state=states)
        return _project(y, self.out)


class WindowLayer(_Layer):
    """Attention with a sliding window and sinks, grouped heads of 64 channels."""

    def __init__(self, gen, dim, device, window=96, n_sink=4, groups=4):
        super().__init__(gen, dim, device)
        self.H, self.Hkv = dim // 64, dim // 64 // groups
        self.window, self.n_sink = window, n_sink
        self.qkv, self.out = self.matrix(dim, (self.H + 2 * self.Hkv) * 64), self.matrix(dim, dim)

    def heads(self, x):
        qkv = _project(x, self.qkv).unflatten(-1, (-1, 64))
        return qkv.split((self.H, self.Hkv, self.Hkv), -2)

    def prefill(self, x, lens):
        q, k, v = self.heads(x)
        o, _ = attention.window_attn_fwd(q, k, v, self.window, self.n_sink, lens=lens)
        cache = attention.window_cache(x.shape[0], self.Hkv, 64, self.window, self.n_sink,
                                       x.dtype, x.device)
        attention.window_cache_fill(k, v, *cache, self.window, self.n_sink, lens=lens)
        return _project(o.flatten(2), self.out), cache

    def step(self, x, state, pos):
        q, k, v = (t.contiguous() for t in self.heads(x))
        o = attention.window_attn_step(q, k, v, *state, pos, self.window, self.n_sink)
        return _project(o.flatten(1), self.out)


class ChannelLayer(_Layer):
    """A wide layer and one back; its block takes the norm of what they give, gated and scaled."""

    def __init__(self, gen, dim, device, channels):
        super().__init__(gen, dim, device)
        self.up, self.down = self.matrix(dim, channels * dim), self.matrix(channels * dim, dim)
        self.up_bias, self.gates = self.vector(channels * dim, scale=0.3).bfloat16(), self.matrix(dim, dim)
        self.end = dict(post_norm=True, post_weight=self.vector(dim, scale=0.1) + 1,
                        scale=self.vector(dim, scale=0.1) + 0.5, gate_act="sigmoid")

    def gate(self, x):
        return _project(x, self.gates)

    def prefill(self, x, lens):
        return self.step(x, None, None), None

    def step(self, x, state, pos):
        return _project(_project(x, self.up, bias=self.up_bias, act="silu"), self.down)


class HybridStack:
    """Delta-rule, scan and window layers in turn over a small vocabulary; with ``channels`` a
    channel layer of that many times the width after each of them."""

    def __init__(self, dim=512, vocab=256, repeats=1, window=96, n_sink=4, seed=0, device="cuda",
                 channels=0):
        gen = torch.Generator().manual_seed(seed)
        base = _Layer(gen, dim, device)
        self.embed, self.unembed = base.vector(vocab, dim).bfloat16(), base.matrix(dim, vocab)
        self.layers = []
        for _ in range(repeats):
            for mixer in (DeltaLayer(gen, dim, device), ScanLayer(gen, dim, device),
                          WindowLayer(gen, dim, device, window, n_sink)):
                self.layers += [mixer] + ([ChannelLayer(gen, dim, device, channels)] if channels else [])

    def prefill(self, tokens, lens):
        """tokens [B,T], lens int32 [B]: (logits [B,T,vocab], state) after each sequence's
        lens[b] tokens.  Logits past a sequence's end mean nothing."""
        h, states = self.embed[tokens], []
        x, _ = _join(h)
        for layer in self.layers:
            o, state = layer.prefill(x, lens)
            x, h = _join(h, o, gate=layer.gate(x), **layer.end)
            states.append(state)
        return _project(x, self.unembed), (states, lens.clone())

    def step(self, tokens, state):
        """One token [B] per sequence: logits [B,vocab]; the state goes on in place."""
        states, pos = state
        h = self.embed[tokens]
        x, _ = _join(h)
        for layer, s in zip(self.layers, states):
            o = layer.step(x, s, pos)
            x, h = _join(h, o, gate=layer.gate(x), **layer.end)
        pos += 1
        return _project(x, self.unembed)


def main(B=3, T=150, more=20, **kw):
    model = HybridStack(**kw)
    gen = torch.Generator().manual_seed(1)
    tokens = torch.randint(0, 256, (B, T + more), generator=gen).cuda()
    lens = torch.tensor([T, T - 37, 5][:B], dtype=torch.int32, device="cuda")
    full = lens + more
    want, _ = model.prefill(tokens, full)
    _, state = model.prefill(tokens[:, :T], lens)
    worst = 0.0
    for i in range(more):
        at = (lens + i).long()
        rows = torch.arange(B, device="cuda")
        got = model.step(tokens[rows, at], state)
        ref = want[rows, at].float()
        worst = max(worst, float((got.float() - ref).norm() / ref.norm()))
    dr.check(dr.dr_get_device_status(), "hybrid")
    print(f"{more} decoded tokens against the prompt form: relative error {worst:.1e}")
    return worst


if __name__ == "__main__":
    main()
