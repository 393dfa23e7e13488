"""Attention over the 4-bit cache with a window and first tokens that stay visible, against the model in 64 bits (tests/kv_reference.py, whose
visible() gets the first tokens here). The bounds are those of tests/test_gpu_kv.py."""
import math

import numpy as np
import pytest

import kv_reference as R
from test_gpu_kv import held, make, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    from speculative_decoding_serial_gb300 import build
    build.build()
    return torch


@pytest.fixture(scope="module")
def kv(torch):
    from speculative_decoding_serial_gb300 import kv
    return kv


def fill(torch, kv, lens, h, d, page, seed=0):
    """A cache with sequences of these lengths, and what it holds of them."""
    c = make(kv, torch, len(lens), max(lens) + 1, h, d, page, seed=seed)
    total = sum(lens)
    k, v = randn(torch, (total, h, d), torch.bfloat16, seed + 5), randn(torch, (total, h, d), torch.bfloat16, seed + 6)
    ip = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    c.append(k, v, ip)
    assert c.status() == 0
    hk, hv = held(torch, k, c.k_scale).astype(np.float64), held(torch, v, c.v_scale).astype(np.float64)
    return c, [(hk[a:b], hv[a:b]) for a, b in zip(ip[:-1].tolist(), ip[1:].tolist())]


def see(length, tokens, t, window, sinks, bits):
    x = R.visible(length, tokens, t, True, window, bits)
    if window and sinks:
        x |= R.visible(length, tokens, t, True, 0, bits) & (np.arange(length) < sinks)
    return x


def check(torch, c, kvs, q, counts, out, lse, window, sinks, tree=None, rows=None):
    """Every row, or those of `rows`, of every entry."""
    heads, d = q.shape[1:]
    group, u = heads // c.kv_heads, 2.0 ** (-8 if q.dtype == torch.bfloat16 else -11)
    qf, o, l = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    at = 0
    for (k, v), t in zip(kvs, counts):
        for tok in range(t) if rows is None else [x for x in rows if x < t]:
            bits = None if tree is None else [int(x) & (2 ** 64 - 1) for x in np.atleast_1d(tree[at + tok])]
            x = see(len(k), t, tok, window, sinks, bits)
            n = int(x.sum())
            for a in range(heads):
                want, log, spread, mass = R.attend(qf[at + tok, a], k[:, a // group], v[:, a // group], d ** -0.5, x)
                if n == 0:
                    assert not o[at + tok, a].any() and l[at + tok, a] == -np.inf
                    continue
                e = (d + 8) * 2.0 ** -23 * spread
                bound = u * np.abs(want) + (4 * e + 2.0 ** -11 + 2.0 ** -20 + (n + 256) * 2.0 ** -25) * mass + 2.0 ** -24 * np.abs(v[x, a // group]).max()
                assert (np.abs(o[at + tok, a] - want) <= bound).all(), (at, tok, a)
                assert abs(l[at + tok, a] - log) <= 2 * e + 2.0 ** -20 + (n + 256) * 2.0 ** -25 + 2.0 ** -22 * abs(log), (at, tok, a)
        at += t


# lengths, query tokens, query heads a KV head, KV heads, channels, page, window, first tokens, type
CASES = [
    ([700, 33, 1, 64], 1, 4, 2, 128, 64, 100, 4, "bfloat16"),     # a gap; shorter than the window; a single token
    ([700, 300], 1, 1, 2, 64, 16, 7, 1, "float16"),
    ([2000], 1, 4, 2, 128, 16, 64, 130, "bfloat16"),              # more first tokens than window
    ([500, 501, 502, 503, 504, 505], 2, 2, 1, 64, 32, 33, 17, "float16"),
    ([900], 3, 4, 1, 256, 128, 50, 5, "bfloat16"),
    ([900, 260], 9, 4, 1, 256, 16, 1, 33, "bfloat16"),            # a window of the token itself
    ([1500, 200, 66], 17, 4, 2, 128, 64, 128, 4, "bfloat16"),     # many rows, one tile
    ([1300], 33, 4, 1, 64, 16, 40, 129, "float16"),               # first tokens that end in their second block
    ([1400, 777], 70, 4, 1, 128, 64, 200, 64, "bfloat16"),        # two tiles
    ([3000], 1, 8, 1, 128, 64, 250, 260, "bfloat16"),
    ([400], 1, 4, 1, 128, 64, 300, 99, "bfloat16"),               # the window begins in the unit after the first tokens'
    ([400], 1, 4, 1, 128, 64, 300, 100, "bfloat16"),              # where they end
    ([400], 40, 4, 1, 128, 64, 300, 2 ** 31 - 1, "bfloat16"),     # all of them
    ([400], 1, 4, 1, 128, 64, 2 ** 31 - 1, 5, "bfloat16"),
    ([400, 90], 2, 4, 1, 128, 64, 0, 5, "bfloat16"),              # no window: they change nothing
    ([5000, 4000, 3001], 1, 4, 8, 64, 32, 400, 4, "bfloat16"),    # more CTAs than items
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend_with_first_tokens(torch, kv, case):
    lens, t, group, h, d, page, window, sinks, dtype = CASES[case]
    c, kvs = fill(torch, kv, lens, h, d, page, seed=case)
    q = randn(torch, (len(lens) * t, h * group, d), getattr(torch, dtype), 100 + case)
    counts = [t] * len(lens)
    out, lse = c.attend(q, window=window, sinks=sinks)
    assert c.status() == 0
    check(torch, c, kvs, q, counts, out, lse, window, sinks, rows=None if t < 20 else sorted({0, 1, t // 2, t - 1}))
    if not window:
        a, b = c.attend(q)
        assert torch.equal(a, out) and torch.equal(b, lse)


@pytest.mark.parametrize("window,sinks", [(1, 1), (15, 16), (16, 15), (100, 31), (31, 100), (128, 128), (256, 1), (3, 255), (250, 257)])
@pytest.mark.parametrize("t,d", [(1, 128), (2, 64), (5, 256), (12, 128), (40, 64), (40, 128)])
def test_attend_where_window_and_first_tokens_end(torch, kv, window, sinks, t, d):
    """Windows and first tokens that end in, at and around the units of keys, the last ones and the first ones of a slot."""
    lens = [max(t, x) for x in (sinks + window, sinks + window + 1, sinks + window + 130, 3 * sinks + 2 * window + 300, sinks, window)]
    c, kvs = fill(torch, kv, lens, 1, d, 16, seed=window + sinks)
    q = randn(torch, (len(lens) * t, 4, d), torch.bfloat16, t)
    out, lse = c.attend(q, window=window, sinks=sinks)
    assert c.status() == 0
    check(torch, c, kvs, q, [t] * len(lens), out, lse, window, sinks, rows=sorted({0, t // 2, t - 1}))


@pytest.mark.parametrize("d,group", [(128, 4), (64, 2), (256, 1)])
def test_attend_ragged_trees_with_first_tokens(torch, kv, d, group):
    """Trees of drafts, ragged, on slots so short that the first tokens are drafts themselves, and on long ones."""
    counts, lens = [9, 0, 33, 5, 64], [700, 50, 40, 5, 64 + 900]
    c, kvs = fill(torch, kv, lens, 2, d, 16)
    total = sum(counts)
    g = np.random.RandomState(d)
    tree = np.zeros(total, np.uint64)
    at = 0
    for t in counts:
        for u in range(t):
            tree[at + u] = (np.uint64(1) << np.uint64(u)) | (tree[at + g.randint(u)] if u and g.rand() < 0.9 else np.uint64(0))
        at += t
    tree[3] = 0  # sees none of the drafts, not even itself
    q = randn(torch, (total, 2 * group, d), torch.bfloat16, 7)
    ip = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    bits = torch.from_numpy(tree.view(np.int64)).cuda()
    for window, sinks in ((20, 3), (64, 20), (3, 40)):
        out, lse = c.attend(q, ip, window=window, sinks=sinks, tree=bits)
        assert c.status() == 0
        check(torch, c, kvs, q, counts, out, lse, window, sinks, tree.view(np.int64), rows=[0, 3, 4, 20, 63])


@pytest.mark.parametrize("t,d,n", [(1, 64, 700), (9, 64, 700), (17, 64, 900), (1, 256, 700)])
def test_attend_many_entries_with_first_tokens(torch, kv, t, d, n):
    """So many entries that their division is planned ahead; a few looked at."""
    g = np.random.RandomState(n + t)
    lens = g.randint(t, 300, n).tolist()
    c, kvs = fill(torch, kv, lens, 1, d, 16, seed=3)
    q = randn(torch, (n * t, 4, d), torch.bfloat16, 4)
    out, lse = c.attend(q, window=37, sinks=20)
    assert c.status() == 0
    for i in list(range(0, n, 97)) + [n - 1]:
        check(torch, c, [kvs[i]], q[i * t:(i + 1) * t], [t], out[i * t:(i + 1) * t], lse[i * t:(i + 1) * t], 37, 20, rows=[0, t - 1])


def test_first_tokens_in_shared_pages_and_other_slots(torch, kv):
    """A prompt's pages shared by forks, entries in another order, strides, and what lies past a slot's end."""
    h, d, t = 2, 128, 3
    c = make(kv, torch, 4, 600, h, d, 64)
    k, v = randn(torch, (400, h, d), torch.bfloat16, 1), randn(torch, (400, h, d), torch.bfloat16, 2)
    c.append(k, v, torch.tensor([0, 400], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    c.fork(torch.zeros(4, dtype=torch.int32, device="cuda"))
    more = [randn(torch, (4 * t, h, d), torch.bfloat16, 3 + i) for i in range(2)]
    c.append(*more)
    hk, hv = (held(torch, torch.cat([a, b]), s).astype(np.float64) for a, b, s in ((k, more[0], c.k_scale), (v, more[1], c.v_scale)))
    kvs = [(np.concatenate([hk[:400], hk[400 + t * i:400 + t * i + t]]), np.concatenate([hv[:400], hv[400 + t * i:400 + t * i + t]])) for i in range(4)]
    wide = randn(torch, (4 * t, 2, 8, d), torch.bfloat16, 9)
    q = wide[:, 1]
    order = [2, 0, 3]
    slots = torch.tensor(order, dtype=torch.int32, device="cuda")
    out, lse = c.attend(q[:3 * t], slots=slots, window=60, sinks=6)
    assert c.status() == 0
    check(torch, c, [kvs[i] for i in order], q[:3 * t], [t] * 3, out, lse, 60, 6)


def test_first_tokens_replayed_and_refused(torch, kv):
    c, kvs = fill(torch, kv, [900, 300], 2, 128, 64)
    q = randn(torch, (2, 8, 128), torch.bfloat16, 1)
    graph = torch.cuda.CUDAGraph()
    c.attend(q, window=50, sinks=4)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = c.attend(q, window=50, sinks=4)
    for _ in range(2):
        graph.replay()
    assert c.status() == 0
    check(torch, c, kvs, q, [1, 1], out, lse, 50, 4)
    from speculative_decoding_serial_gb300 import whead as wh
    with pytest.raises(wh.WheadError):
        c.attend(q, window=50, sinks=-1)
    for sinks in (2 ** 31, -2 ** 31 - 1, 2 ** 40):
        with pytest.raises(ValueError):
            c.attend(q, window=50, sinks=sinks)
    assert c.status() == 0
