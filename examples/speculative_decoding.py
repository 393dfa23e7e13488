"""Speculative decoding with the serial draft head and the 4-bit KV cache, on a small target model with random weights.

One step: the head drafts gamma tokens; the last token and the drafts go through the target together, their keys and values into the
cache (append), their queries over everything that is cached (attend); the drafts that the target would have chosen too stay,
the others leave the cache again (compact). A prompt is cached once and its pages are shared by all sequences (fork).

    python examples/speculative_decoding.py [--gamma 16] [--sequences 4] [--tokens 64]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Target:
    """One attention layer over embeddings: logits = (x + attention(x)) . output embeddings. The head's W and E are its embeddings,
    so that a draft is what the target would say without its attention."""

    def __init__(self, vocab=4096, heads=8, kv_heads=2, dim=64, width=256, weight=0.5, seed=0, device="cuda"):
        import torch
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape, s=1.0: torch.randn(shape, generator=g, device=device) * s  # noqa: E731
        self.heads, self.kv_heads, self.dim, self.width, self.weight = heads, kv_heads, dim, width, weight
        self.embed = normal(vocab, width).bfloat16()
        self.out = normal(vocab, width, s=width ** -0.5).bfloat16()
        self.wq = normal(width, heads * dim, s=width ** -0.5)
        self.wk = normal(width, kv_heads * dim, s=width ** -0.5)
        self.wv = normal(width, kv_heads * dim, s=width ** -0.5)
        self.wo = normal(heads * dim, width, s=(heads * dim) ** -0.5)

    def forward(self, cache, tokens, slots=None):
        """Logits (n, t, vocab) after each of tokens (n, t), which go to the ends of the slots."""
        n, t = tokens.shape
        x = self.embed[tokens.long()].float().view(n * t, self.width)
        q = (x @ self.wq).bfloat16().view(n * t, self.heads, self.dim)
        k = (x @ self.wk).bfloat16().view(n * t, self.kv_heads, self.dim)
        v = (x @ self.wv).bfloat16().view(n * t, self.kv_heads, self.dim)
        cache.append(k, v, slots=slots)
        o, _ = cache.attend(q, slots=slots)
        x = x + self.weight * (o.float().view(n * t, -1) @ self.wo)
        return (x @ self.out.float().T).view(n, t, -1)


def start(target, prompt, sequences, room, page_size=16):
    """A cache with the prompt in every slot (its full pages held once), and the first token after it for each."""
    import torch
    from speculative_decoding_serial_gb300 import kv
    pages = -(-room // page_size)
    cache = kv.KvCache(sequences * pages + 1, page_size, target.kv_heads, target.dim, sequences, pages)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    last = target.forward(cache, prompt.view(1, -1), slots=one)[:, -1].argmax(-1).to(torch.int32)
    cache.fork(torch.zeros(sequences, dtype=torch.int32, device="cuda"))
    # sequences go on from different tokens, or they would all say the same
    others = torch.arange(1, sequences, dtype=torch.int32, device="cuda") * 131 % target.embed.shape[0]
    return cache, torch.cat([last, others])


def plain_step(target, cache, last):
    """One token for each sequence, (n,)."""
    import torch
    return target.forward(cache, last[:, None])[:, 0].argmax(-1).to(torch.int32)


def draft_step(target, cache, head, last, gamma):
    """One speculative step: (tokens (n, gamma + 1), how many of them are the target's (n,))."""
    import torch
    n, vocab = last.shape[0], target.embed.shape[0]
    begin = cache.lens.clone()
    base = torch.zeros((n, gamma, vocab), device="cuda")
    drafts = head.walk(base, target.embed[last.long()].float())
    chosen = target.forward(cache, torch.cat([last[:, None], drafts], 1)).argmax(-1).to(torch.int32)
    good = (drafts == chosen[:, :gamma]).int().cumprod(1).sum(1).to(torch.int32)
    keep = torch.arange(gamma + 1, dtype=torch.int32, device="cuda").repeat(n, 1)
    cache.compact(begin, keep, good + 1)  # the last token and the drafts that were right
    return chosen, good + 1


def generate(target, prompt, sequences, tokens, gamma):
    """`tokens` greedy tokens for each sequence, with drafts (gamma > 0) or without: (lists of tokens, number of steps)."""
    from speculative_decoding_serial_gb300 import whead
    # room for a sequence whose drafts are always right while another's never are
    cache, last = start(target, prompt, sequences, prompt.numel() + (tokens + 1) * (gamma + 1))
    said, steps = [[x] for x in last.tolist()], 0
    head = whead.Head(target.out, target.embed, max_B=sequences, max_gamma=gamma) if gamma else None
    while min(map(len, said)) < tokens:
        if gamma:
            chosen, count = draft_step(target, cache, head, last, gamma)
            last = chosen.gather(1, count.long()[:, None] - 1)[:, 0].contiguous()
            for s, row, c in zip(said, chosen.tolist(), count.tolist()):
                s += row[:c]
        else:
            last = plain_step(target, cache, last)
            for s, x in zip(said, last.tolist()):
                s.append(x)
        steps += 1
    cache.status(check=True)
    if head:
        if head.status():
            raise RuntimeError("the draft head reported an error")
        head.close()
    return [s[:tokens] for s in said], steps


def main():
    import torch
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--gamma", type=int, default=16)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    target = Target()
    prompt = torch.arange(0, 4000, 41, dtype=torch.int32, device="cuda")
    plain, plain_steps = generate(target, prompt, a.sequences, a.tokens, 0)
    said, steps = generate(target, prompt, a.sequences, a.tokens, a.gamma)
    same = sum(x == y for p, s in zip(plain, said) for x, y in zip(p, s))
    print(f"{a.sequences} sequences of {a.tokens} tokens: {plain_steps} steps without drafts, {steps} with {a.gamma} drafts a step; "
          f"{same} of {a.sequences * a.tokens} tokens the same")


if __name__ == "__main__":
    main()
