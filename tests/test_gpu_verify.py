"""Log probabilities and the verification of drafts on the GPU, against a model in 64 bits (tests/verify_reference.py).

Bounds. With u = 2^-24 (half a step of fp32, relative) and d = (x - m) log2(e) / T: a thread's d is off by 3 u |d| (difference, factor,
product), each 2^d by 2^-22 more (the exponential), and a sum by u for each addition on its way: at most V / 256 / 2 in a thread
(fewer where a row has several CTAs), and 20 joins, of which 5 multiply by another exponential. So a sum of exponentials is off by
    S = 6 * 2^-22 + u (V / 512 + 20) + 3 u ln 2 E|d|    relative, E|d| = sum p |d|;
log p by S + 4 u |log p|, lse by S + 4 u |lse|, and the entropy by S (2 + E|d|) + 16 u (a's reference is up to 8 units off, twice).
"""
import math

import numpy as np
import pytest

import verify_reference as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32 = lambda x: np.float64(x).astype(np.float32)  # noqa: E731
# the settled border: decisions whose sides differ by less than what their numbers are off by may go either way
NEAR = 2.0 ** -20


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    from speculative_decoding_serial_gb300 import build
    build.build()
    return torch


@pytest.fixture(scope="module")
def V(torch):
    from speculative_decoding_serial_gb300 import verify
    return verify


def check_logprobs(torch, V, x, tokens, top, temperature=1.0):
    """One call against the model, every row; x (rows, V) on the GPU."""
    r = V.logprobs(x, tokens, top=top, temperature=temperature)
    torch.cuda.synchronize()
    got = [y.cpu().numpy() if y is not None else None for y in r]
    flat, rows = x.double().cpu().numpy(), x.shape[0]
    for i in range(rows):
        lse, entropy, lp, best = R.logprobs(flat[i], temperature, top)
        if np.isnan(lse):
            assert all(np.isnan(got[k][i]).all() for k in (0, 1, 2, 4) if got[k] is not None)
            assert got[3] is None or (got[3][i] == -1).all()
            continue
        p = np.exp(lp)
        mean = (p[p > 0] * np.abs((flat[i] - flat[i].max())[p > 0])).sum() / temperature / math.log(2) if np.isfinite(lse) else 0.0
        S = 6 * 2.0 ** -22 + U * (x.shape[1] / 512 + 20) + 3 * U * math.log(2) * mean
        # what lies past fp32's range rounds to an infinity there: -3.39e38 - 3.39e38 = -6.78e38 < -3.403e38 does
        close = lambda a, b, tol: a == b or a == F32(b) or abs(a - b) <= tol  # noqa: E731
        assert close(got[2][i], lse, S + 4 * U * abs(lse)), (i, got[2][i], lse)
        assert close(got[1][i], entropy, S * (2 + mean) + 16 * U), (i, got[1][i], entropy)
        if tokens is not None:
            t = int(tokens[i])
            want = lp[t] if 0 <= t < x.shape[1] else -np.inf
            assert close(got[0][i], want, S + 4 * U * abs(want)), (i, got[0][i], want)
        if top:
            np.testing.assert_array_equal(got[3][i], best)
            for k in range(top):
                want = lp[best[k]] if best[k] >= 0 else -np.inf
                assert close(got[4][i][k], want, S + 4 * U * abs(want)), (i, k, got[4][i][k], want)
    return r


def logits(torch, rows, vocab, dtype, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * vocab + rows)
    x = torch.randn((rows, vocab), generator=g, device="cuda") * spread
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return x.to(dtype), tokens


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 127, 255, 256, 257, 1000, 2049, 4099, 32003])
def test_logprobs_sizes(torch, V, kind, vocab):
    for rows, top, temperature in ((1, 5, 1.0), (3, 32, 0.7), (2, 0, 2.5), (5, 1, 0.1)):
        x, tokens = logits(torch, rows, vocab, getattr(torch, kind))
        check_logprobs(torch, V, x, tokens, top, temperature)


@pytest.mark.parametrize("kind,rows", [("bfloat16", 1), ("float32", 17), ("float16", 40), ("bfloat16", 130), ("float32", 470), ("bfloat16", 1000)])
def test_logprobs_rows_by_clusters_of_every_size(torch, V, kind, rows):
    """1000 rows have a CTA each, fewer have more, up to 16."""
    vocab = 151936 if rows < 50 else 40000
    x, tokens = logits(torch, rows, vocab, getattr(torch, kind))
    if rows > 50:  # the model takes its time: 12 rows of them
        r = V.logprobs(x, tokens, top=20)
        some = list(range(0, rows, rows // 12))
        one = check_logprobs(torch, V, x[some].contiguous(), tokens[some].contiguous(), 20)
        for a, b in zip(r, one):
            if a.dtype == torch.int32:
                assert torch.equal(a[some], b)
            else:  # both within the bound of the same value
                assert (a[some] - b).abs().max().item() <= 2 * (6 * 2.0 ** -22 + U * (vocab / 512 + 20) + 40 * U) + 80 * U
    else:
        check_logprobs(torch, V, x, tokens, 20)


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float32"])
def test_logprobs_of_strange_rows(torch, V, kind):
    dtype = getattr(torch, kind)
    vocab, inf = 5003, math.inf
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    g = torch.Generator(device="cuda").manual_seed(5)
    base = torch.randn(vocab, generator=g, device="cuda").to(dtype)
    rows = []

    def row(change):
        x = base.clone()
        change(x)
        rows.append(x)
    row(lambda x: x.fill_(-inf))
    row(lambda x: x.fill_(low))                                    # nothing left, by the type's lowest value: all alike
    row(lambda x: x.fill_(high))
    row(lambda x: (x.fill_(-inf), x[4999:5000].fill_(2)))          # one token that can be
    row(lambda x: x[1000:].fill_(-inf))
    row(lambda x: x[:4000].fill_(low))
    row(lambda x: (x.fill_(low), x[17:18].fill_(high)))
    row(lambda x: (x.fill_(-inf), x[3:4].fill_(low)))
    row(lambda x: x[100:101].fill_(math.nan))
    row(lambda x: x[5002:].fill_(inf))
    row(lambda x: (x[7:8].fill_(inf), x[9:10].fill_(math.nan)))
    row(lambda x: x.fill_(math.nan))
    row(lambda x: x.fill_(1.5))                                    # all equal: the first tokens
    row(lambda x: (x.fill_(0.0), x[::2].neg_()))                   # -0 and 0 are equal
    row(lambda x: x.copy_(torch.sort(x)[0]))
    row(lambda x: x.copy_(torch.sort(x, descending=True)[0]))
    row(lambda x: x.copy_((torch.arange(vocab, device="cuda") // 40).to(dtype)))
    row(lambda x: x.mul_(1000))
    row(lambda x: x.mul_(2.0 ** -20))
    row(lambda x: x[:8].fill_(60000.0))
    row(lambda x: (x.fill_(-5), x[2500:].fill_(5)))
    x = torch.stack(rows)
    n = len(rows)
    tokens = torch.tensor([(0, 4999, 17, 3, -1, vocab, 2 ** 31 - 1, -2 ** 31)[i % 8] for i in range(n)], dtype=torch.int32, device="cuda")
    for top in (32, 1):
        for temperature in (1.0, 0.3):
            check_logprobs(torch, V, x, tokens, top, temperature)
    # a given token at the type's lowest value, which a mask by it leaves a finite log probability
    check_logprobs(torch, V, x, torch.full_like(tokens, 11), 0)
    # as rows of few CTAs each: many of them
    many = x.repeat(60, 1)
    a, b = V.logprobs(x, tokens, top=32), V.logprobs(many, tokens.repeat(60), top=32)
    assert torch.equal(a.top_tokens.repeat(60, 1), b.top_tokens)
    for i in range(0, 60 * n, 19 * n):
        check_logprobs(torch, V, many[i:i + n], tokens, 32)


@pytest.mark.parametrize("temperature", [1e-30, 1e-3, 1e30])
def test_logprobs_at_the_ends_of_temperature(torch, V, temperature):
    x, tokens = logits(torch, 4, 3001, torch.float32)
    if temperature < 1e-20:  # all on the largest, whose log probability is 0, or shared by equal ones
        x[1, 77] = x[1, 88] = x[1].max() + 1
        r = V.logprobs(x, x.argmax(1).to(torch.int32), top=2, temperature=temperature)
        np.testing.assert_allclose(r.logprob.cpu().numpy(), [0, -math.log(2), 0, 0], atol=1e-6)
        assert r.top_tokens[1].tolist() == [77, 88] and r.entropy.cpu().tolist()[0] == 0.0
    else:
        check_logprobs(torch, V, x, tokens, 5, temperature)


def test_logprobs_of_strided_rows(torch, V):
    """Rows that start anywhere, that are far apart, that are one row, that run backwards through a batch; three dimensions."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for dtype in (torch.bfloat16, torch.float32):
        big = torch.randn((4, 7, 1003), generator=g, device="cuda").to(dtype)
        for view in (big[:, :, 1:], big[:, ::2, 5:900], big.transpose(0, 1)[:, :, 3:], big[1:2].expand(6, -1, -1), big[:, :1], big[:, :, 10:11]):
            tokens = torch.randint(0, view.shape[2], view.shape[:2], generator=g, device="cuda", dtype=torch.int32)
            got, want = V.logprobs(view, tokens, top=3), check_logprobs(torch, V, view.reshape(-1, view.shape[2]).contiguous(), tokens.reshape(-1), 3)
            assert got.entropy.shape == view.shape[:2] and got.top_tokens.shape == (*view.shape[:2], 3)
            assert torch.equal(got.top_tokens.reshape(-1, 3), want.top_tokens)
            for a, b in zip(got, want):
                assert torch.allclose(a.reshape(b.shape), b, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("kind,rows,vocab", [("float32", 1, 2 ** 24 - 1), ("bfloat16", 460, 1100003)])
def test_logprobs_of_very_long_rows(torch, V, kind, rows, vocab):
    """More groups of vectors than a CTA keeps: it keeps the largest of several."""
    dtype = getattr(torch, kind)
    x = torch.full((rows, vocab), -4.0, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    at = torch.randperm(vocab, generator=g, device="cuda")[:40]
    at[:6] = torch.tensor([0, 1, vocab - 1, vocab - 2, vocab // 2, vocab // 2 + 1], device="cuda")
    values = torch.randint(0, 12, (40,), generator=g, device="cuda").to(dtype)   # with equal ones
    x[-1, at] = values
    x[0, at] = values
    r = V.logprobs(x, top=32)
    order = sorted(range(40), key=lambda k: (-float(values[k]), int(at[k])))[:32]
    for i in (0, rows - 1):
        assert r.top_tokens[i].tolist() == [int(at[k]) for k in order]
        z = x[i].double()
        lse = torch.logsumexp(z, 0).item()
        assert abs(r.lse[i].item() - lse) <= 6 * 2.0 ** -22 + U * (vocab / 512 + 20) + 60 * U
        assert torch.equal(r.top_logprobs[i].argsort(descending=True, stable=True), torch.arange(32, device="cuda"))
    assert r.logprob is None


def test_logprobs_twice_on_another_stream_and_replayed(torch, V):
    x, tokens = logits(torch, 33, 20011, torch.bfloat16)
    want = V.logprobs(x, tokens, top=7)
    again = V.logprobs(x, tokens, top=7)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        third = V.logprobs(x, tokens, top=7)
    torch.cuda.current_stream().wait_stream(other)
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fourth = V.logprobs(held, tokens, top=7)
    held.copy_(x.flip(0))
    graph.replay()
    flipped = V.logprobs(held, tokens, top=7)
    for a, b, c, d, e in zip(want, again, third, fourth, flipped):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(d, e)


def test_logprobs_refusals(torch, V):
    x, tokens = logits(torch, 4, 100, torch.float32)
    from speculative_decoding_serial_gb300 import whead as wh
    for bad in (dict(tokens=tokens.long()), dict(tokens=tokens[:3]), dict(tokens=tokens.cpu()), dict(top=33), dict(top=-1)):
        with pytest.raises(ValueError):
            V.logprobs(x, **bad)
    for bad in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(wh.WheadError):
            V.logprobs(x, temperature=bad)
    y = x.clone().requires_grad_()
    with pytest.raises(ValueError):
        V.logprobs(y)
    with torch.no_grad():
        V.logprobs(y)
    with pytest.raises(ValueError):
        V.logprobs(x.t())
    assert V.logprobs(x[:0], tokens[:0], top=3).top_tokens.shape == (0, 3)


# ---------------------------------------------------------------------------------------------------- verify

def case(torch, n, gamma, vocab, target_dtype, draft_dtype, seed=0, spread=0.6):
    """Target's logits, drafts' logits near them, and drafts drawn from those."""
    g = torch.Generator(device="cuda").manual_seed(seed + 100 * n + gamma + vocab)
    x = torch.randn((n, gamma + 1, vocab), generator=g, device="cuda") * 2.5
    x.scatter_add_(2, torch.randint(0, vocab, (n, gamma + 1, 4), generator=g, device="cuda"), torch.rand((n, gamma + 1, 4), generator=g, device="cuda") * 8)
    y = x[:, :gamma] + torch.randn((n, gamma, vocab), generator=g, device="cuda") * spread
    noise = -torch.log(-torch.log(torch.rand(y.shape, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))
    tokens = (y + noise).argmax(-1).to(torch.int32) if gamma else torch.empty((n, 0), dtype=torch.int32, device="cuda")
    return x.to(target_dtype), (y.to(draft_dtype) if draft_dtype else None), tokens


def check_verify(torch, V, target, tokens, draft, temperature, draft_temperature=None, seed=0, step=0, drafted=None):
    said, count = V.verify(target, tokens, draft, temperature=temperature, draft_temperature=draft_temperature, seed=seed, step=step, drafted=drafted)
    torch.cuda.synchronize()
    n, rows, _ = target.shape
    p, q = target.double().cpu().numpy(), draft.double().cpu().numpy() if draft is not None else None
    x, h = tokens.cpu().numpy(), drafted.cpu().numpy() if drafted is not None else np.full(n, rows - 1)
    near = 0
    for i in range(n):
        want, c, margin = R.verify(p[i], x[i], q[i] if q is not None else None, temperature, draft_temperature or temperature, seed & (2 ** 64 - 1), step, i, int(h[i]))
        same = said[i].tolist() == want.tolist() and int(count[i]) == c
        near += margin < NEAR
        assert same or margin < NEAR, (i, said[i].tolist(), want.tolist(), margin)
    assert near <= 1 + n // 50
    return said, count


KINDS = {"bf16": "bfloat16", "f16": "float16", "f32": "float32", "": None}


@pytest.mark.parametrize("n,gamma,vocab", [(1, 0, 1), (1, 1, 1), (2, 1, 2), (3, 2, 5), (1, 16, 4099), (5, 7, 1000), (9, 3, 257), (2, 40, 131), (1, 255, 63), (3, 5, 32003), (40, 4, 2048)])
@pytest.mark.parametrize("target,draft", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16"), ("bf16", "")])
def test_verify_sizes_and_types(torch, V, n, gamma, vocab, target, draft):
    x, y, tokens = case(torch, n, gamma, vocab, getattr(torch, KINDS[target]), getattr(torch, KINDS[draft]) if draft else None)
    check_verify(torch, V, x, tokens, y, 1.0, seed=-5, step=3)
    check_verify(torch, V, x, tokens, y, 0.6, draft_temperature=0.8, seed=2 ** 63 + 11, step=2 ** 32 - 300)
    check_verify(torch, V, x, tokens, y, 0.0)


@pytest.mark.parametrize("n", [1, 12, 200])
def test_verify_large_vocabulary(torch, V, n):
    x, y, tokens = case(torch, min(n, 12), 3, 151936, torch.bfloat16, torch.float32)
    if n > 12:
        x, y, tokens = x[:1].expand(n, -1, -1), y[:1].expand(n, -1, -1), tokens[:1].expand(n, -1).contiguous()
        said, count = V.verify(x, tokens, y, temperature=1.0, seed=5)
        for i in range(0, n, 40):
            want, c, margin = R.verify(x[0].double().cpu().numpy(), tokens[0].cpu().numpy(), y[0].double().cpu().numpy(), 1.0, 1.0, 5, 0, i, 3)
            assert margin < NEAR or (said[i].tolist() == want.tolist() and int(count[i]) == c)
        return
    check_verify(torch, V, x, tokens, y, 1.0, seed=17, step=4)
    check_verify(torch, V, x, tokens, None, 0.9, seed=17)


@pytest.mark.parametrize("target,draft", [("bf16", "f32"), ("f16", ""), ("f32", "f32")])
def test_verify_many_entries_some_refused_early(torch, V, target, draft):
    """So many that places behind a refused draft are left out; ragged; entries looked at here and there, and twice the same."""
    n, gamma, vocab = 300, 6, 20011
    x, y, tokens = case(torch, n, gamma, vocab, getattr(torch, KINDS[target]), getattr(torch, KINDS[draft]) if draft else None, spread=0.4)
    best = x[:, :gamma].float().argmax(-1).to(torch.int32)
    g = torch.Generator(device="cuda").manual_seed(12)
    drafted = torch.randint(0, gamma + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    for temperature, said_tokens in ((0.0, torch.where(torch.rand((n, gamma), generator=g, device="cuda") < 0.8, best, tokens)), (1.0, tokens)):
        for have in (None, drafted):
            a, b = (V.verify(x, said_tokens, y, temperature=temperature, seed=6, step=1, drafted=have) for _ in range(2))
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            for i in range(0, n, 23):
                h = gamma if have is None else int(have[i])
                want, c, margin = R.verify(x[i].double().cpu().numpy(), said_tokens[i].cpu().numpy(), y[i].double().cpu().numpy() if draft else None,
                                           temperature, temperature, 6, 1, i, h)
                assert margin < NEAR or (a[0][i].tolist() == want.tolist() and int(a[1][i]) == c), (i, a[0][i].tolist(), want.tolist())
            assert 1 < a[1].float().mean().item() < gamma


@pytest.mark.parametrize("n,vocab", [(1, 7), (3, 5003), (2, 151936), (400, 900)])
def test_verify_where_nothing_is_left_of_the_difference(torch, V, n, vocab):
    """Drafts that are no tokens, of the target's own distribution: the token after is drawn from that."""
    x, _, tokens = case(torch, n, 2, vocab, torch.float32, torch.float32)
    tokens = torch.full_like(tokens, -1)
    check_verify(torch, V, x, tokens, x[:, :2], 1.0, seed=21)


def test_verify_ragged(torch, V):
    x, y, tokens = case(torch, 12, 6, 3001, torch.bfloat16, torch.bfloat16, spread=0.1)
    drafted = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 100, -1, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    for temperature in (0.0, 1.0):
        said, count = check_verify(torch, V, x, tokens, y, temperature, seed=3, drafted=drafted)
        assert int(count[0]) == int(count[9]) == int(count[10]) == 1
    # what lies past an entry's drafts is not looked at
    x2, y2, t2 = x.clone(), y.clone(), tokens.clone()
    for i, h in enumerate(drafted.clamp(0, 6).tolist()):
        x2[i, h + 1:] = math.nan
        y2[i, h:] = math.nan
        t2[i, h:] = -7
    for temperature in (0.0, 1.0):
        a, b = (V.verify(*z, temperature=temperature, seed=3, drafted=drafted) for z in ((x, tokens, y), (x2, t2, y2)))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_verify_strange_rows_and_tokens(torch, V, temperature):
    inf = math.inf
    for dtype in (torch.bfloat16, torch.float32):
        x, y, tokens = case(torch, 14, 4, 777, dtype, dtype, spread=0.05)
        low = torch.finfo(dtype).min
        best = x.float().argmax(-1).to(torch.int32)
        if temperature == 0:
            tokens = best[:, :4].contiguous()
        x[0, 1, 5] = math.nan
        x[1, 0, 700] = inf
        x[2, 2] = -inf
        x[3, 1] = low                                   # all alike
        x[4, 2, :700] = -inf
        x[5, 0] = -inf
        x[5, 0, 776] = low                              # the last token is all there is
        tokens[6, 1] = -1
        tokens[7, 1] = 777
        tokens[8, 0] = 2 ** 31 - 1
        if temperature:
            y[9, 1, 3] = math.nan
            y[10, 0] = -inf
            y[11, 2, 0] = inf
            y[12, 0] = -inf
            y[12, 0, tokens[12, 0]] = 0                 # the draft had no choice
            x[12, 0, tokens[12, 0]] = -inf              # and the target would never say it
            x[13], y[13] = x[13, :1], x[13, :1]         # the same distribution: all stay
        check_verify(torch, V, x, tokens, y, temperature, seed=8)
        check_verify(torch, V, x, tokens, None, temperature, seed=8)
        if temperature:
            assert int(V.verify(x, tokens, y, temperature=1.0, seed=8)[1][13]) == 5


def test_verify_greedy_takes_the_lowest_of_equal_tokens(torch, V):
    x = torch.zeros((3, 3, 9001), dtype=torch.float16, device="cuda")
    x[:, :, 8000] = x[:, :, 17] = x[:, :, 400] = 3
    x[1, :, ::2] = -0.0
    x[2] = 0
    x[2, :, 1::2] = -0.0
    tokens = torch.tensor([[17, 17], [17, 400], [0, 0]], dtype=torch.int32, device="cuda")
    said, count = V.verify(x, tokens)
    assert said.tolist() == [[17, 17, 17], [17, 17, -1], [0, 0, 0]] and count.tolist() == [3, 2, 3]


def test_verify_strides(torch, V):
    g = torch.Generator(device="cuda").manual_seed(9)
    big = torch.randn((6, 5, 1501), generator=g, device="cuda")
    near = big + torch.randn(big.shape, generator=g, device="cuda") * 0.3
    for off in (0, 1, 2, 3):
        x, y = big.bfloat16()[::2, :, off:1400], near[1::2, 1:, off:1400]
        tokens = y.argmax(-1).to(torch.int32)
        check_verify(torch, V, x, tokens, y, 1.0, seed=off)
        check_verify(torch, V, big[:, :, off:1001].transpose(0, 1)[:, :3], tokens[:1, :2].repeat(5, 1).clamp(max=900), None, 0.5, seed=off)


def test_tokens_said_are_distributed_as_the_target_says(torch, V):
    """20,000 entries of the same five-token distributions: shares of each position's token within 5 deviations of the target's."""
    n = 20000
    p = torch.tensor([[0.4, 0.3, 0.2, 0.05, 0.05], [0.1, 0.1, 0.1, 0.3, 0.4], [0.2, 0.2, 0.2, 0.2, 0.2]], device="cuda")
    q = torch.tensor([[0.1, 0.2, 0.3, 0.2, 0.2], [0.3, 0.3, 0.2, 0.1, 0.1]], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    tokens = torch.stack([torch.multinomial(r, n, True, generator=g) for r in q], 1).to(torch.int32)
    x, y = p.log()[None].expand(n, -1, -1), q.log()[None].expand(n, -1, -1)
    said, count = V.verify(x, tokens, y, temperature=1.0, seed=1234)
    for t in range(3):
        here = said[count > t, t]
        m = here.numel()
        share = torch.bincount(here.long(), minlength=5).float() / m
        assert (share - p[t]).abs().max().item() <= 5 * math.sqrt(0.25 / m), (t, share.tolist())
    stay = torch.minimum(p[0], q[0]).sum().item()
    assert abs((count > 1).float().mean().item() - stay) <= 5 * math.sqrt(0.25 / n)


def test_verify_of_logits_far_from_zero(torch, V):
    """4,000,000 entries of four tokens whose logits lie around 1,000: a reference rounded to fp32 is off by up to 6e-5 there (in log2 units), which the
    sums must not take over into p and q. Decisions nearer than 2^-19 may go either way: p and q are off by some 2^-21 each (the sum's
    exponentials 2^-22, its additions, the factor log2(e) rounded times differences below 16)."""
    n, temperature = 4000000, 1.0
    g = torch.Generator(device="cuda").manual_seed(4)
    at = torch.rand((n, 1, 1), generator=g, device="cuda") * 400 + 800
    x = at + torch.randn((n, 2, 4), generator=g, device="cuda") * 2
    y = at + 50 + torch.randn((n, 1, 4), generator=g, device="cuda") * 2
    tokens = torch.randint(0, 4, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    said, count = V.verify(x, tokens, y, temperature=temperature, seed=99)
    i = tokens.long()
    p, q = (torch.softmax(z[:, 0].double() / temperature, -1).gather(1, i)[:, 0].cpu().numpy() for z in (x, y))
    u = R.uniform(R.philox(99, 0, 0, np.arange(n), 2)[0])
    stays, sure = u * q < p, np.abs(u * q - p) > 2.0 ** -19 * p
    got = (count > 1).cpu().numpy()
    assert (got == stays)[sure].all(), int((got != stays)[sure].sum())
    assert sure.mean() > 0.9999 and torch.equal(said[:, 0][count > 1], tokens[:, 0][count > 1])


def test_seeds_and_steps_of_any_integer_type(torch, V):
    x, y, tokens = case(torch, 2, 3, 100, torch.float32, torch.float32)
    want = V.verify(x, tokens, y, temperature=1.0, seed=2 ** 63 + 5, step=7)
    got = V.verify(x, tokens, y, temperature=1.0, seed=np.uint64(2 ** 63 + 5), step=np.int64(7))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    a, b = V.verify(x, tokens, y, temperature=1.0, seed=-1), V.verify(x, tokens, y, temperature=1.0, seed=2 ** 64 - 1)
    assert torch.equal(a[0], b[0])


def test_first_calls_of_a_process_inside_a_capture(torch):
    """Nothing of a call needs to have run before it is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
from speculative_decoding_serial_gb300 import verify as V
x = torch.randn((3, 5, 4001), device="cuda").bfloat16()
y, t = x[:, :4].float(), x[:, :4].argmax(-1).to(torch.int32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = V.logprobs(x, top=5)
    b = V.verify(x, t, y, temperature=1.0, seed=3)
    c = V.verify(x, t)
g.replay()
torch.cuda.synchronize()
for got, want in ((a, V.logprobs(x, top=5)), (b, V.verify(x, t, y, temperature=1.0, seed=3)), (c, V.verify(x, t))):
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, want))
print("same")
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "same" in run.stdout, run.stderr


def test_verify_twice_on_another_stream_and_replayed(torch, V):
    x, y, tokens = case(torch, 7, 5, 9001, torch.bfloat16, torch.bfloat16)
    want, again = (V.verify(x, tokens, y, temperature=1.0, seed=1) for _ in range(2))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        third = V.verify(x, tokens, y, temperature=1.0, seed=1)
    torch.cuda.current_stream().wait_stream(other)
    held = x.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for k, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            outs.append(V.verify(held, tokens, y, temperature=1.0 if k else 0.0, seed=1))
    held.copy_(x.flip(0))
    for graph in graphs:
        graph.replay()
    for graph in graphs:
        graph.replay()
    for k, out in enumerate(outs):
        for a, b in zip(out, V.verify(held, tokens, y, temperature=1.0 if k else 0.0, seed=1)):
            assert torch.equal(a, b)
    for a, b, c in zip(want, again, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_verify_refusals(torch, V):
    from speculative_decoding_serial_gb300 import whead as wh
    x, y, tokens = case(torch, 2, 3, 100, torch.float32, torch.float32)
    for bad in ((x, tokens[:, :2], y), (x, tokens.long(), y), (x, tokens, y[:, :2]), (x, tokens, y[..., :50]), (x[0], tokens, y), (x, tokens.cpu(), y),
                (x, tokens, y.cpu()), (x.transpose(1, 2), tokens, y), (x[:, :0], tokens, None)):
        with pytest.raises(ValueError):
            V.verify(*bad)
    with pytest.raises(TypeError):
        V.verify(x, tokens, y.double())
    for bad in (dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=1.0, draft_temperature=0.0), dict(temperature=1e-40)):
        with pytest.raises(wh.WheadError):
            V.verify(x, tokens, y, **bad)
    for bad in (dict(step=-1), dict(step=2 ** 32), dict(drafted=tokens[:, 0].long()), dict(drafted=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            V.verify(x, tokens, y, **bad)
    with pytest.raises(ValueError):
        V.verify(x.clone().requires_grad_(), tokens, y)
    said, count = V.verify(x[:0], tokens[:0], y[:0], temperature=1.0)
    assert said.shape == (0, 4) and count.shape == (0,)
