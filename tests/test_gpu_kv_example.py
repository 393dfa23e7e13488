"""The draft head and the 4-bit KV cache in one loop (examples/speculative_decoding.py): with drafts the target says what it says without."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    from speculative_decoding_serial_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("speculative_decoding", os.path.join(ROOT, "examples", "speculative_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# Logits are sums of 256 products of size 1/16 to 1 and an attention whose outputs carry bf16's 2^-8; 0.05 is several times what the two
# ways of computing it (one query token, and gamma + 1 of them) can differ by.
GAP = 0.05


@pytest.mark.parametrize("gamma,sequences", [(4, 1), (7, 3), (16, 4)])
def test_what_is_said_with_drafts_is_the_targets_own_choice(example, gamma, sequences):
    """Every token said, against the target alone, one token at a time over the same text: none is better by more than GAP."""
    import torch
    target = example.Target()
    prompt = torch.arange(0, 3000, 37, dtype=torch.int32, device="cuda")
    tokens = 40
    said, steps = example.generate(target, prompt, sequences, tokens, gamma)
    _, plain_steps = example.generate(target, prompt, sequences, tokens, 0)
    assert steps < plain_steps == tokens - 1
    text = torch.tensor(said, dtype=torch.int32, device="cuda")
    cache, first = example.start(target, prompt, sequences, prompt.numel() + tokens)
    assert torch.equal(first, text[:, 0])
    for i in range(tokens - 1):
        logits = target.forward(cache, text[:, i:i + 1].contiguous())[:, 0]
        short = logits.max(-1).values - logits.gather(1, text[:, i + 1:i + 2].long())[:, 0]
        assert short.max().item() <= GAP, (i, short.tolist())
    assert cache.status() == 0
