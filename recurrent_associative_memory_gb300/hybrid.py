"""A small hybrid stack: a delta-rule layer, a selective scan layer and a window-attention
layer, as a model would run them together, for prompts and for single tokens.

Each layer is ``h + mixer(norm(h))``:

* ``DeltaLayer``   projections to q, k, v -> short convolutions -> the Kaczmarz linear
  attention recurrence (``dr_chunk_fwd`` / ``dr_decode_step``)
* ``ScanLayer``    projection -> short convolution -> time step, B and C projections ->
  selective scan with its gate
* ``WindowLayer``  projections to q, k, v -> attention with a sliding window and sinks

``prefill`` runs a batch of prompts of different lengths and returns the logits and the
state; ``step`` takes one token per sequence.  Every layer's serving state has a constant
size: the recurrences' matrices, the convolutions' last inputs, the window's ring of keys
and values.  Weights are random; the projections are plain matrix products.

Run as a program it decodes a few tokens and checks them against the prompt form:
``python -m recurrent_associative_memory_gb300.hybrid``.
"""

from __future__ import annotations

import torch

from . import attention, dr, runner, ssm

__all__ = ["HybridStack"]

HEAD = 128   # head size of the delta-rule layer (chunked tensor-core path)


def _norm(h):
    return torch.nn.functional.rms_norm(h.float(), h.shape[-1:]).to(h.dtype)


class _Layer:
    def __init__(self, gen, dim, device):
        self.gen, self.dim, self.device = gen, dim, device

    def matrix(self, n_in, n_out):
        w = torch.randn(n_in, n_out, generator=self.gen) * n_in ** -0.5
        return w.to(self.device, torch.bfloat16)

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
        g = (x @ self.gates).float()
        return dict(q=q, k=k, v=v, variant="kla", chunk=64, q_l2norm=True, eps=1e-6,
                    eta=torch.sigmoid(g[..., :self.H]).contiguous(),
                    log_alpha=-torch.nn.functional.softplus(g[..., self.H:] + 2.0).contiguous())

    def prefill(self, x, lens):
        mixed, conv = ssm.short_conv_fwd(x @ self.qkv, self.conv_w, lens=lens)
        inp = self.inputs(x, mixed)
        # tokens past a sequence's end neither write to the memory nor let it decay
        past = torch.arange(x.shape[1], device=x.device)[None] >= lens[:, None]
        inp["eta"].masked_fill_(past[..., None], 0.0)
        inp["log_alpha"].masked_fill_(past[..., None], 0.0)
        o, memory, _ = runner.chunk_fwd(inp)
        return o.flatten(2) @ self.out, (conv, memory)

    def step(self, x, state, pos):
        conv, memory = state
        mixed, _ = ssm.short_conv_step(x @ self.qkv, self.conv_w, None, conv)
        return runner.decode_step(self.inputs(x, mixed), memory).flatten(1) @ self.out


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
        s = mixed @ self.select
        bc = s[..., self.dim:].unflatten(-1, (2, 1, self.N))
        return dict(x=mixed, dt=s[..., :self.dim], A=self.A, B=bc[..., 0, :, :], C=bc[..., 1, :, :],
                    D=self.D, z=z, dt_bias=self.dt_bias)

    def prefill(self, x, lens):
        xz = x @ self.xz
        mixed, conv = ssm.short_conv_fwd(xz[..., :self.dim], self.conv_w, lens=lens)
        y, states = ssm.selective_scan_fwd(**self.scan_inputs(mixed, xz[..., self.dim:]), lens=lens)
        return y @ self.out, (conv, states)

    def step(self, x, state, pos):
        conv, states = state
        xz = x @ self.xz
        mixed, _ = ssm.short_conv_step(xz[:, :self.dim], self.conv_w, None, conv)
        y, _ = ssm.selective_scan_step(**self.scan_inputs(mixed, xz[:, self.dim:]), state=states)
        return y @ self.out


class WindowLayer(_Layer):
    """Attention with a sliding window and sinks, grouped heads of 64 channels."""

    def __init__(self, gen, dim, device, window=96, n_sink=4, groups=4):
        super().__init__(gen, dim, device)
        self.H, self.Hkv = dim // 64, dim // 64 // groups
        self.window, self.n_sink = window, n_sink
        self.qkv, self.out = self.matrix(dim, (self.H + 2 * self.Hkv) * 64), self.matrix(dim, dim)

    def heads(self, x):
        qkv = (x @ self.qkv).unflatten(-1, (-1, 64))
        return qkv.split((self.H, self.Hkv, self.Hkv), -2)

    def prefill(self, x, lens):
        q, k, v = self.heads(x)
        o, _ = attention.window_attn_fwd(q, k, v, self.window, self.n_sink, lens=lens)
        cache = attention.window_cache(x.shape[0], self.Hkv, 64, self.window, self.n_sink,
                                       x.dtype, x.device)
        attention.window_cache_fill(k, v, *cache, self.window, self.n_sink, lens=lens)
        return o.flatten(2) @ self.out, cache

    def step(self, x, state, pos):
        q, k, v = (t.contiguous() for t in self.heads(x))
        o = attention.window_attn_step(q, k, v, *state, pos, self.window, self.n_sink)
        return o.flatten(1) @ self.out


class HybridStack:
    """Delta-rule, scan and window layers in turn over a small vocabulary."""

    def __init__(self, dim=512, vocab=256, repeats=1, window=96, n_sink=4, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        base = _Layer(gen, dim, device)
        self.embed, self.unembed = base.vector(vocab, dim).bfloat16(), base.matrix(dim, vocab)
        self.layers = []
        for _ in range(repeats):
            self.layers += [DeltaLayer(gen, dim, device), ScanLayer(gen, dim, device),
                            WindowLayer(gen, dim, device, window, n_sink)]

    def prefill(self, tokens, lens):
        """tokens [B,T], lens int32 [B]: (logits [B,T,vocab], state) after each sequence's
        lens[b] tokens.  Logits past a sequence's end mean nothing."""
        h, states = self.embed[tokens], []
        for layer in self.layers:
            o, state = layer.prefill(_norm(h), lens)
            h = h + o
            states.append(state)
        return _norm(h) @ self.unembed, (states, lens.clone())

    def step(self, tokens, state):
        """One token [B] per sequence: logits [B,vocab]; the state goes on in place."""
        states, pos = state
        h = self.embed[tokens]
        for layer, s in zip(self.layers, states):
            h = h + layer.step(_norm(h), s, pos)
        pos += 1
        return _norm(h) @ self.unembed


def main(B=3, T=150, more=20):
    model = HybridStack()
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
