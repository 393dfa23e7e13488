"""Forms of the verification's kernels and corners of its values that tests/test_gpu_verify.py does not come to; its bounds and helpers.

Which form a call takes follows from its rows and bytes (divide() in csrc/verify_common.cuh, launch() in csrc/verify_drafts.cu); the sizes here are for
152 SMs.
"""
import math

import numpy as np
import pytest

import verify_reference as R
from test_gpu_verify import KINDS, NEAR, U, V, case, check_logprobs, check_verify, torch  # noqa: F401  (fixtures, too)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab", [(1, 151936), (3, 32003), (150, 5003)])
def test_draws_do_not_depend_on_which_warp_comes_first(torch, V, n, vocab):  # noqa: F811
    """What a warp has found bounds what the others look at, whenever they read it: 100 calls say the same."""
    x, y, tokens = case(torch, n, 2, vocab, torch.bfloat16, torch.float32)
    want = V.verify(x, tokens, y, temperature=1.0, seed=13)
    for _ in range(100):
        got = V.verify(x, tokens, y, temperature=1.0, seed=13)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def check_rows(r, x, tokens, top, temperature, rows):
    """Some rows of a call's results against the model, within test_gpu_verify's bounds."""
    for i in rows:
        z = x[i].double().cpu().numpy()
        lse, entropy, lp, best = R.logprobs(z, temperature, top)
        p = np.exp(lp)
        mean = (p[p > 0] * np.abs((z - z.max())[p > 0])).sum() / temperature / math.log(2)
        S = 6 * 2.0 ** -22 + U * (x.shape[1] / 512 + 20) + 3 * U * math.log(2) * mean
        assert abs(r.lse[i].item() - lse) <= S + 4 * U * abs(lse), i
        assert abs(r.entropy[i].item() - entropy) <= S * (2 + mean) + 16 * U, i
        want = lp[int(tokens[i])]
        assert abs(r.logprob[i].item() - want) <= S + 4 * U * abs(want), i
        if top:
            np.testing.assert_array_equal(r.top_tokens[i].cpu().numpy(), best)
            assert (np.abs(r.top_logprobs[i].cpu().numpy() - lp[best]) <= S + 4 * U * np.abs(lp[best])).all(), i


# ---------------------------------------------------------------------------------------------------- references near 2^23

def steps_around(torch, shape, temperature, sign, low, high, seed):  # noqa: F811
    """f32 logits a few of fp32's steps around sign 2^23 T / log2(e), where a reference's k = x log2(e) / T passes 2^23 (a step is 0.69 of k's units)."""
    g = np.random.RandomState(seed)
    at = np.float32(2.0 ** 23 * temperature / R.LOG2E)
    bits = np.asarray(at.view(np.int32) + sign * g.randint(low, high + 1, shape), np.int32)
    return torch.from_numpy(np.array(np.float32(sign) * bits.view(np.float32))).cuda()


@pytest.mark.parametrize("temperature", [1e-6, 1.0])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("rows,vocab", [(3, 40), (3, 4001), (2, 30011), (600, 4001)])
def test_logprobs_where_references_pass_the_border(torch, V, temperature, sign, rows, vocab):  # noqa: F811
    """Threads and CTAs with references on both sides of 2^23 in one row: k is rounded on one side, to steps of a half, and not formed on the other."""
    x = steps_around(torch, (rows, vocab), temperature, sign, -9, 0, rows + vocab)
    x[0, vocab // 2] = steps_around(torch, (), temperature, sign, 2, 2, 0)   # one on the other side, or none
    if rows > 1:
        x[1, ::97] = steps_around(torch, (), temperature, sign, 1, 1, 0)
    tokens = (torch.arange(rows, device="cuda") * 37 % vocab).to(torch.int32)
    r = V.logprobs(x, tokens, top=3, temperature=temperature)
    check_logprobs(torch, V, x[:3].contiguous(), tokens[:3].contiguous(), 3, temperature)
    if rows > 3:
        check_rows(r, x, tokens, 3, temperature, [0, 1, 2, rows - 1])


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,vocab", [(200, 64), (40, 3001), (500, 700)])
def test_verify_where_references_pass_the_border(torch, V, sign, n, vocab):  # noqa: F811
    x = steps_around(torch, (n, 3, vocab), 1e-6, sign, -9, 0, vocab)
    x[:, :, 5::60] = steps_around(torch, (n, 3, len(range(5, vocab, 60))), 1e-6, sign, -1, 2, vocab + 1)
    y = steps_around(torch, (n, 2, vocab), 1e-6, sign, -5, 1, vocab + 2)
    tokens = y.argmax(-1).to(torch.int32)
    check_verify(torch, V, x, tokens, y, 1e-6, seed=31)


# ---------------------------------------------------------------------------------------------------- drawing from small differences

def test_draws_where_the_drafts_are_near_the_target(torch, V):  # noqa: F811
    """2,000,000 entries draw from max(p - q, 0) where that is p / 129: p and q, off by some 2^-20 in fp32, leave it off by 10^-4, in opposite directions
    for the tokens of this row. The sums are of one exponential of 0 and of some 2^-18, so that their rounding, below 2^-20, counts for all
    tokens alike (p / (p - q) differs by 2^-19 from token to token): keys that differ by more than 2^-24 are to be told apart."""
    n, seed = 2000000, 99
    g = np.random.RandomState(1263)
    x = np.concatenate([[0], -12.5 - g.rand(7) / 32]).astype(np.float32)
    y = (x - np.float32(2.0 ** -7)).astype(np.float32)
    y[0] = 0
    p, q = R.distribution(x, 1.0), R.distribution(y, 1.0)
    u = R.uniform(np.stack([np.stack(R.philox(seed, k, 0, np.arange(n), 1), 1) for k in range(2)], 1).reshape(n, 8))
    key = np.maximum(p - q, 0) / -np.log(u)
    want, ordered = key.argmax(1), np.sort(key, 1)
    sure = ordered[:, -1] - ordered[:, -2] > 2.0 ** -24 * ordered[:, -1]
    target, draft = (torch.from_numpy(z).cuda().expand(n, k, 8) for z, k in ((x, 2), (y, 1)))
    said, count = V.verify(target, torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), draft, temperature=1.0, seed=seed)
    assert (count == 1).all()
    got = said[:, 0].cpu().numpy()
    assert sure.mean() > 0.99999 and int((got != want)[sure].sum()) == 0


# ---------------------------------------------------------------------------------------------------- forms of the kernels

@pytest.mark.parametrize("kind,rows,vocab", [
    ("bfloat16", 64, 248064), ("float16", 100, 151936), ("float32", 100, 70001),   # 8 CTAs a row, streamed
    ("bfloat16", 150, 151936), ("float32", 200, 40003),                            # 4
    ("float16", 300, 100003), ("bfloat16", 450, 40001), ("float32", 310, 20001),   # 2
    ("bfloat16", 1000, 40000), ("float32", 470, 40000)])                           # 1
@pytest.mark.parametrize("top", [0, 5, 20])
def test_logprobs_of_many_rows(torch, V, kind, rows, vocab, top):  # noqa: F811
    """Rows streamed by clusters of every size, against the model itself; equal and sorted rows among them, which go the exact way."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn((rows, vocab), generator=g, device="cuda") * 3).to(getattr(torch, kind))
    x[1] = 1.5
    x[2] = x[2].sort()[0]
    x[3, 100:] = torch.finfo(x.dtype).min
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tokens[3] = 50
    r = V.logprobs(x, tokens, top=top, temperature=0.9)
    check_rows(r, x, tokens, top, 0.9, [0, 1, 2, 3, rows // 2, rows - 1])


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float32"])
def test_logprobs_of_rows_with_more_groups_than_a_cta_keeps(torch, V, kind):  # noqa: F811
    """500 times one row of 2^24 - 1 logits, a CTA each: it keeps the largest values of runs of 16 groups (f32) or 8. A few tokens stand out; then all are
    equal; then they are in order, with many equal ones."""
    dtype, vocab, rows, top = getattr(torch, kind), 2 ** 24 - 1, 500, 32
    g = torch.Generator(device="cuda").manual_seed(8)
    few = torch.full((vocab,), -4.0, device="cuda")
    at = torch.randperm(vocab, generator=g, device="cuda")[:60]
    at[:6] = torch.tensor([0, 1, vocab - 1, vocab - 2, vocab // 2, vocab // 2 + 1], device="cuda")
    few[at] = torch.randint(0, 9, (60,), generator=g, device="cuda").float()
    order = torch.arange(vocab, device="cuda") // 8192 / 64.0
    for x in (few, torch.full_like(few, 0.25), order, order.flip(0)):
        x = x.to(dtype)
        best, high = [], x.unique(sorted=True).flip(0)
        for value in high:  # equal ones: the lower tokens first
            best += (x == value).nonzero()[:top, 0].tolist()
            if len(best) >= top:
                break
        best = best[:top]
        r = V.logprobs(x.expand(rows, -1), top=top)
        z = x.double()
        lse = torch.logsumexp(z, 0).item()
        S = 6 * 2.0 ** -22 + U * (vocab / 512 + 20) + 3 * U * (torch.softmax(z, 0) * (z.max() - z)).sum().item()
        for i in (0, 1, rows - 1):
            assert r.top_tokens[i].tolist() == best
            assert abs(r.lse[i].item() - lse) <= S + 4 * U * abs(lse)
            want = z[best].cpu().numpy() - lse
            assert (np.abs(r.top_logprobs[i].cpu().numpy() - want) <= S + 4 * U * np.abs(want)).all()
        assert torch.equal(r.top_tokens, r.top_tokens[:1].expand(rows, -1))


@pytest.mark.parametrize("n,gamma,vocab,kind", [(500, 4, 5003, "bf16"), (470, 8, 2000, "f32"), (30, 5, 151936, "bf16"), (60, 16, 151936, "f16"), (120, 3, 70001, "f32")])
def test_rows_behind_a_refused_draft_left_out(torch, V, n, gamma, vocab, kind):  # noqa: F811
    """Greedy, and sampled drafts without logits: so many entries that what is decided in time is left out, by rows of one part and of several; ragged."""
    x, _, tokens = case(torch, n, gamma, vocab, getattr(torch, KINDS[kind]), None)
    best = x[:, :gamma].float().argmax(-1).to(torch.int32)
    g = torch.Generator(device="cuda").manual_seed(n)
    some = torch.where(torch.rand((n, gamma), generator=g, device="cuda") < 0.7, best, tokens)
    drafted = torch.randint(0, gamma + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    few = list(range(0, n, -(-n // 12))) + [n - 1]
    host = {i: x[i].double().cpu().numpy() for i in few}
    for temperature in (0.0, 0.8):
        for have in (None, drafted):
            a, b = (V.verify(x, some, temperature=temperature, seed=6, step=1, drafted=have) for _ in range(2))
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            for i in few:
                want, c, margin = R.verify(host[i], some[i].cpu().numpy(), None, temperature, temperature, 6, 1, i, gamma if have is None else int(have[i]))
                assert margin < NEAR or (a[0][i].tolist() == want.tolist() and int(a[1][i]) == c), (i, a[0][i].tolist(), want.tolist())
            if have is None and temperature == 0:
                assert 1 < a[1].float().mean().item() < gamma + 1
    # greedy, every entry: against torch
    said, count = V.verify(x, some, drafted=drafted)
    full = x.float()
    token = torch.stack([(full[:, t] == full[:, t].amax(-1, keepdim=True)).int().argmax(-1) for t in range(gamma + 1)], 1).to(torch.int32)
    stay = ((token[:, :gamma] == some) & (torch.arange(gamma, device="cuda") < drafted[:, None])).int().cumprod(1).sum(1)
    at = torch.arange(gamma + 1, device="cuda")[None]
    assert torch.equal(count.long(), stay + 1)
    assert torch.equal(said, torch.where(at <= stay[:, None], token, torch.full_like(token, -1)))


# ---------------------------------------------------------------------------------------------------- gradients that go forward

def test_forward_mode_tangents_are_refused(torch, V):  # noqa: F811
    from torch.autograd import forward_ad
    x, y, tokens = case(torch, 2, 3, 100, torch.float32, torch.float32)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for call in (lambda: V.logprobs(dual), lambda: V.verify(dual, tokens, y, temperature=1.0),
                     lambda: V.verify(x, tokens, forward_ad.make_dual(y, torch.ones_like(y)), temperature=1.0)):
            with pytest.raises(ValueError, match="gradients"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="gradients"):  # which keeps no tangent back
                call()
        V.logprobs(x)
        V.logprobs(forward_ad.unpack_dual(dual).primal)
    V.logprobs(x)
