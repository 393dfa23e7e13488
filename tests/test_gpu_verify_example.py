"""Drafting, attention, verification, compaction and scoring together, as examples/speculative_decoding.py uses them: sampled, and over streams
with a window and first tokens that stay visible."""
import importlib.util
import os

import numpy as np
import pytest

import verify_reference as R

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


@pytest.mark.parametrize("temperature", [0.0, 0.8])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_steps_keep_their_books(example, temperature, window, sinks):
    """Several steps: what verify says of the step's own logits is the model's, the cache holds the last token and the drafts that stay, and
    log probabilities are those of the logits."""
    import torch
    from speculative_decoding_serial_gb300 import verify, whead
    n, gamma, seed = 3, 5, 77
    target = example.Target(vocab=1024, window=window, sinks=sinks)
    prompt = torch.arange(0, 900, 13, dtype=torch.int32, device="cuda")
    cache, last = example.start(target, prompt, n, prompt.numel() + 100)
    head = whead.Head(target.out, target.embed, max_B=n, max_gamma=gamma, flags=whead.FLAG_LOGITS_F32)
    accepted = 0
    for step in range(4):
        begin = cache.lens.clone()
        base = torch.zeros((n, gamma, 1024), device="cuda")
        drawn = torch.empty_like(base)
        drafts = head.walk_ex(base, target.embed[last.long()].float(), T=temperature, seed=seed, t0=step * (gamma + 1), out_logits=drawn)
        said, count, logits = example.draft_step(target, cache, head, last, gamma, temperature, seed, step * (gamma + 1))
        for i in range(n):
            want, c, margin = R.verify(logits[i].double().cpu().numpy(), drafts[i].cpu().numpy(), drawn[i].double().cpu().numpy() if temperature else None,
                                       temperature, temperature, seed, step * (gamma + 1), i, gamma)
            assert margin < 2.0 ** -20 or (said[i].tolist() == want.tolist() and int(count[i]) == c)
            accepted += int(count[i]) - 1
            lse, _, lp, best = R.logprobs(logits[i, 0].double().cpu().numpy(), 1.0, 3)
            r = verify.logprobs(logits[i:i + 1], said[i:i + 1], top=3)
            # sums of 1024 exponentials of fp32 logits: well inside 2^-16 of the log probability's size
            assert abs(r.logprob[0, 0].item() - lp[int(said[i, 0])]) <= 2.0 ** -16 * max(1.0, abs(lp[int(said[i, 0])]))
            np.testing.assert_array_equal(r.top_tokens[0, 0].cpu().numpy(), best)
            assert torch.isneginf(r.logprob[0, int(count[i]):]).all()  # -1 is no token
        assert torch.equal(cache.lens, begin + count)
        last = said.gather(1, count.long()[:, None] - 1)[:, 0].contiguous()
    assert accepted > 0 and cache.status() == 0 and head.status() == 0
    head.close()


# as in test_gpu_kv_example.py: several times what the two ways of computing a logit can differ by
GAP = 0.05


def test_a_stream_with_drafts_says_what_the_target_chooses(example):
    """Greedy, a window and first tokens: every token said against the target alone, one token at a time: none is better by more than GAP."""
    import torch
    target = example.Target(window=48, sinks=4)
    prompt = torch.arange(0, 3000, 37, dtype=torch.int32, device="cuda")
    tokens = 40
    said, steps = example.generate(target, prompt, 3, tokens, 7)
    assert steps < tokens - 1
    text = torch.tensor(said, dtype=torch.int32, device="cuda")
    cache, first = example.start(target, prompt, 3, prompt.numel() + tokens)
    assert torch.equal(first, text[:, 0])
    for i in range(tokens - 1):
        logits = target.forward(cache, text[:, i:i + 1].contiguous())[:, 0]
        short = logits.max(-1).values - logits.gather(1, text[:, i + 1:i + 2].long())[:, 0]
        assert short.max().item() <= GAP, (i, short.tolist())
    assert cache.status() == 0


def test_sampled_generation_runs_with_and_without_drafts(example):
    import torch
    target = example.Target()
    prompt = torch.arange(0, 3000, 37, dtype=torch.int32, device="cuda")
    for gamma in (0, 4):
        scores = []
        said, steps = example.generate(target, prompt, 2, 12, gamma, 0.7, 5, scores)
        assert [len(s) for s in said] == [12, 12] and all(0 <= x < 4096 for s in said for x in s)
        assert len(scores) == steps and all(torch.isfinite(s).all() and (s <= 0).all() for s in scores)
        again, _ = example.generate(target, prompt, 2, 12, gamma, 0.7, 5)
        assert again == said
