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
