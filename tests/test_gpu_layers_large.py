"""Tensors of more than 2^31 values: the last sequence of a large batch gives, bit for bit,
what it gives alone (each sequence's arithmetic does not depend on the batch)."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def noise(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=BF)


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def test_attention_step_over_a_large_cache():
    """The caches' last rows lie past 2^31 values; a batch this large is never cut along the
    slots, so the sequence alone runs without a workspace."""
    from recurrent_associative_memory_gb300 import attention
    B, Hk, H, d, window = 72, 8, 16, 128, 32768
    kc, vc = noise(B, Hk, window + 4, d, seed=1), noise(B, Hk, window + 4, d, seed=2)
    q, k, v = noise(B, H, d, seed=3), noise(B, Hk, d, seed=4), noise(B, Hk, d, seed=5)
    pos = torch.full((B,), 100000, dtype=torch.int32, device="cuda")
    k1, v1 = kc[-1:].clone(), vc[-1:].clone()
    out = attention.window_attn_step(q, k, v, kc, vc, pos, window, 4, workspace=None)
    one = attention.window_attn_step(q[-1:], k[-1:], v[-1:], k1, v1, pos[-1:], window, 4, workspace=None)
    assert torch.equal(out[-1:], one) and torch.equal(kc[-1:], k1) and torch.equal(vc[-1:], v1)


def test_attention_of_a_large_batch():
    from recurrent_associative_memory_gb300 import attention
    B, T, H, Hk, d = 9, 65536, 30, 6, 128
    q, k, v = noise(B, T, H, d, seed=1), noise(B, T, Hk, d, seed=2), noise(B, T, Hk, d, seed=3)
    do = noise(B, T, H, d, seed=4)
    assert q.numel() > 2 ** 31
    out, lse = attention.window_attn_fwd(q, k, v, 64, 4, want_lse=True)
    g = attention.window_attn_bwd(q, k, v, out, lse, do, 64, 4)
    one, l1 = attention.window_attn_fwd(q[-1:], k[-1:], v[-1:], 64, 4, want_lse=True)
    g1 = attention.window_attn_bwd(q[-1:], k[-1:], v[-1:], one, l1, do[-1:], 64, 4)
    assert torch.equal(out[-1:], one) and torch.equal(lse[-1:], l1)
    assert all(torch.equal(g[n][-1:], g1[n]) for n in g)


def test_conv_and_scan_of_a_large_batch():
    from recurrent_associative_memory_gb300 import ssm
    B, T, D, N = 17, 65536, 2048, 8
    x, dt = noise(B, T, D, seed=1), noise(B, T, D, seed=2)
    assert x.numel() > 2 ** 31
    w = noise(D, 4, seed=3).float()
    y, end = ssm.short_conv_fwd(x, w)
    y1, end1 = ssm.short_conv_fwd(x[-1:], w)
    assert torch.equal(y[-1:], y1) and torch.equal(end[-1:], end1)
    g = ssm.short_conv_bwd(x, w, None, dt)
    assert torch.equal(g["dx"][-1:], ssm.short_conv_bwd(x[-1:], w, None, dt[-1:])["dx"])
    del g, y
    A, bc = -torch.arange(1, N + 1, device="cuda").float().repeat(D, 1), noise(B, T, 2, 1, N, seed=4)
    kw = dict(A=A, dt_bias=torch.full((D,), -3.0, device="cuda"))
    y, h = ssm.selective_scan_fwd(x, dt, B=bc[:, :, 0], C=bc[:, :, 1], workspace=None, **kw)
    y1, h1 = ssm.selective_scan_fwd(x[-1:], dt[-1:], B=bc[-1:, :, 0], C=bc[-1:, :, 1], workspace=None, **kw)
    assert torch.equal(y[-1:], y1) and torch.equal(h[-1:], h1)
    g = ssm.selective_scan_bwd(x, dt, B=bc[:, :, 0], C=bc[:, :, 1], d_y=dt, **kw)
    g1 = ssm.selective_scan_bwd(x[-1:], dt[-1:], B=bc[-1:, :, 0], C=bc[-1:, :, 1], d_y=dt[-1:], **kw)
    assert all(torch.equal(g[n][-1:], g1[n]) for n in ("dx", "ddt", "dB", "dC"))
