"""The hybrid stack: decoding token by token continues what the prompt form computes.

Both forms round every layer's output to bf16 (unit 2^-8), at different sums; with three
layers and the unembedding the relative error stays well below 3 (3 + 1) 2^-8 = 4.7e-2,
a misplaced position, slot or state is of order 1."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_decoding_continues_the_prompt():
    from recurrent_associative_memory_gb300 import hybrid
    assert hybrid.main() < 4.7e-2


def test_a_prompt_is_not_changed_by_its_neighbours():
    """Each sequence of a ragged batch gives what it gives alone."""
    from recurrent_associative_memory_gb300.hybrid import HybridStack
    model = HybridStack(window=40)
    tokens = torch.randint(0, 256, (3, 130), generator=torch.Generator().manual_seed(2)).cuda()
    lens = torch.tensor([130, 64, 1], dtype=torch.int32, device="cuda")
    both, _ = model.prefill(tokens, lens)
    for b, n in enumerate(lens.tolist()):
        alone, _ = model.prefill(tokens[b:b + 1, :n].contiguous(), lens[b:b + 1])
        ref = both[b, :n].float()
        assert float((alone[0].float() - ref).norm() / ref.norm()) < 4.7e-2


def test_decoding_continues_the_prompt_with_channel_layers():
    """Six layers and the unembedding: 3 (6 + 1) 2^-8 = 8.2e-2."""
    from recurrent_associative_memory_gb300 import hybrid
    assert hybrid.main(channels=3) < 8.2e-2
