"""The 4-bit paged KV cache on the GPU against a plain model in 64 bits (tests/kv_reference.py).

Bounds. Quantization and bookkeeping are exact: codes, scales, tables, references and lengths have to be equal. For the
attention, u = 2^-8 (bf16, 8 significant bits) or 2^-11 (f16, 11) is a rounding's largest relative error, S the largest
sum |q||k| scale over a row's keys, A = sum p |v| / l, n the row's keys, d the head's channels:
  a score's products are exact and their fp32 sum and factors are off by at most (d + 8) 2^-23 S =: e;
  p is then off by a relative e^2e - 1, its exponential by 2^-21, its rounding to f16 by 2^-11 (largest, not half: the
  pieces of a sum whose reference was raised lie lower), and the fp32 sums by (n / 4 + 64) 2^-24;
  so |out - o| <= u |o| + (4 e + 2^-11 + 2^-20 + (n + 256) 2^-25) A + 2^-24 max|v|, and
  |lse - exact| <= 2 e + 2^-20 + (n + 256) 2^-25 + 2^-22 |exact|.
"""
import math

import numpy as np
import pytest

import kv_reference as R

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


def scales(torch, h, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(h, generator=g) * 0.02 + 0.004).cuda()


def make(kv, torch, n, room, h, d, page, spare=3, seed=0):
    """A cache whose pool is full of bytes that no kernel may let through: NaN scales, largest codes."""
    max_pages = max(1, -(-room // page))
    num = n * max_pages + spare
    pool = torch.full((num, h, page // 16, 18 * d), 0xFF, dtype=torch.uint8, device="cuda")
    return kv.KvCache(num, page, h, d, n, max_pages, k_scale=scales(torch, h, seed), v_scale=scales(torch, h, seed + 1), pool=pool)


def held(torch, x, g):
    """What the cache holds of x [tokens, heads, d], f32."""
    x, g = x.float().cpu().numpy(), g.cpu().numpy()
    return np.stack([R.dequantize(*R.quantize(x[:, i], g[i]), g[i]) for i in range(x.shape[1])], 1)


def randn(torch, shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# ------------------------------------------------------------------------------------------------ append and read

@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
def test_what_is_read_is_what_was_quantized(torch, kv, dtype, d, page):
    """Several appends of odd counts, so that groups and pages are filled in parts; every held value exactly."""
    dtype, h, counts = getattr(torch, dtype), 3, [[1, 0, 17, 5], [16, 1, 30, 0], [2, 129, 1, 64], [1, 1, 1, 1]]
    c = make(kv, torch, 4, 256, h, d, page)
    want = [[] for _ in range(4)]
    for step, n in enumerate(counts):
        k, v = (randn(torch, (sum(n), h, d), dtype, 10 * step + i) * (1 + 5 * i) for i in range(2))
        ip = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        c.append(k, v, ip)
        hk, hv = held(torch, k, c.k_scale), held(torch, v, c.v_scale)
        for i in range(4):
            want[i].append((hk[ip[i]:ip[i + 1]], hv[ip[i]:ip[i + 1]]))
    assert c.status() == 0
    start = torch.tensor([0, 3, 16, 40], dtype=torch.int32, device="cuda")
    k, v = (x.cpu().numpy() for x in c.read(start, 150, dtype=torch.float32))
    for i in range(4):
        for got, w in ((k, np.concatenate([a for a, _ in want[i]])), (v, np.concatenate([b for _, b in want[i]]))):
            w = w[int(start[i]):][:150]
            np.testing.assert_array_equal(got[i, :len(w)], w)
            assert not got[i, len(w):].any()
    assert c.lens.tolist() == [sum(x) for x in zip(*counts)]


def test_bytes_lie_where_the_header_says(torch, kv):
    h, d = 2, 64
    c = make(kv, torch, 1, 32, h, d, 32)
    k, v = randn(torch, (32, h, d), torch.float32, 1), randn(torch, (32, h, d), torch.float32, 2)
    c.append(k, v)
    assert c.status() == 0
    pool = c.pool[int(c.tables[0, 0])].cpu().numpy()
    for head in range(h):
        for part in range(2):
            kc, ks, vc, vs = R.unpack(pool[head, part], d)
            for code, scale, x, g in ((kc, ks, k, c.k_scale), (vc, vs, v, c.v_scale)):
                wc, ws = R.quantize(x[part * 16:part * 16 + 16, head].cpu().numpy(), float(g[head]))
                np.testing.assert_array_equal(scale, ws)
                np.testing.assert_array_equal(R.E2M1[code], R.E2M1[wc])


def test_values_outside_the_ordinary(torch, kv):
    """Zeros, signed zeros, ties of the codes, blocks below and above the scales' range, infinities, NaN."""
    d = 64
    c = make(kv, torch, 1, 16, 1, d, 16)
    c.k_scale.fill_(0.25)
    c.v_scale.fill_(0.25)
    x = torch.zeros(8, 1, d)
    x[1, 0] = torch.linspace(-6, 6, d) * 0.25
    x[2, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6]) * 0.25  # ties
    x[3] = 1e-30
    x[4] = 1e30
    x[5, 0, ::7] = float("nan")
    x[5, 0, 1] = 2.0
    x[6, 0, 3] = float("inf")
    x[6, 0, 20] = -float("inf")
    x[7, 0] = -0.0
    x = x.cuda()
    c.append(x, x)
    got = c.read(torch.zeros(1, dtype=torch.int32, device="cuda"), 8, dtype=torch.float32)
    assert c.status() == 0
    for y in got:
        assert torch.isfinite(y).all()
        np.testing.assert_array_equal(y[0].cpu().numpy(), held(torch, x, c.k_scale))


def test_strided_and_unaligned_inputs(torch, kv):
    h, d, n = 3, 128, 21
    c = make(kv, torch, 2, 64, h, d, 16)
    big = randn(torch, (n, 2, h, d), torch.bfloat16, 3)           # k and v interleaved, as one projection leaves them
    odd = randn(torch, (h * n * d + 1,), torch.float16, 4)[1:]    # heads outermost, an odd address
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    c.append(big[:, 0], big[:, 1], slots=one)
    t = odd.view(h, n, d).transpose(0, 1)
    c.append(t, t, slots=one - 1)
    assert c.status() == 0
    k, v = c.read(torch.zeros(2, dtype=torch.int32, device="cuda"), n, dtype=torch.float32)
    np.testing.assert_array_equal(k[1].cpu().numpy(), held(torch, big[:, 0], c.k_scale))
    np.testing.assert_array_equal(v[1].cpu().numpy(), held(torch, big[:, 1], c.v_scale))
    np.testing.assert_array_equal(k[0].cpu().numpy(), held(torch, t, c.k_scale))
    np.testing.assert_array_equal(v[0].cpu().numpy(), held(torch, t, c.v_scale))


# ------------------------------------------------------------------------------------------------ attend

def fill(torch, c, lens, seed):
    n, h, d = len(lens), c.kv_heads, c.head_dim
    k, v = randn(torch, (sum(lens), h, d), torch.bfloat16, seed), randn(torch, (sum(lens), h, d), torch.bfloat16, seed + 1)
    ip = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    if sum(lens):
        c.append(k, v, ip, slots=torch.arange(n, dtype=torch.int32, device="cuda"))
    hk, hv = held(torch, k, c.k_scale).astype(np.float64), held(torch, v, c.v_scale).astype(np.float64)
    return [(hk[ip[i]:ip[i + 1]], hv[ip[i]:ip[i + 1]]) for i in range(n)]


def check(torch, c, kvs, q, out, lse, counts, slots=None, causal=True, window=0, tree=None, scale=None, rows=None):
    """Every row (or the given query tokens of each entry) against 64 bits, under the bounds above."""
    d = c.head_dim
    heads = q.shape[1]
    group = heads // c.kv_heads
    scale = d ** -0.5 if scale is None else scale
    u = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    qq, oo, ll = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    at = 0
    for i, n in enumerate(counts):
        k, v = kvs[slots[i] if slots is not None else i]
        for t in range(n):
            if rows is not None and t not in rows:
                continue
            bits = None if tree is None else tree[at + t].cpu().numpy().view(np.uint64).reshape(-1)
            see = R.visible(len(k), n, t, causal, window, bits)
            for a in range(heads):
                o, l, big, spread = R.attend(qq[at + t, a], k[:, a // group], v[:, a // group], scale, see)
                where = f"entry {i} token {t} head {a}"
                if not see.any():
                    assert not oo[at + t, a].any() and ll[at + t, a] == -np.inf, where
                    continue
                e, m = (d + 8) * 2.0 ** -23 * big, int(see.sum())
                tol = u * np.abs(o) + (4 * e + 2.0 ** -11 + 2.0 ** -20 + (m + 256) * 2.0 ** -25) * spread + 2.0 ** -24 * np.abs(v).max()
                bad = np.abs(oo[at + t, a] - o) - tol
                assert bad.max() <= 0, f"{where}: out off by {np.abs(oo[at + t, a] - o)[bad.argmax()]:.3g}, allowed {tol[bad.argmax()]:.3g}"
                off, may = abs(ll[at + t, a] - l), 2 * e + 2.0 ** -20 + (m + 256) * 2.0 ** -25 + 2.0 ** -22 * abs(l)
                assert off <= may, f"{where}: lse off by {off:.3g}, allowed {may:.3g}"
        at += n


CASES = [
    # lens, query tokens of each, kv heads, group, d, page, dtype, options
    ([1], 1, 1, 1, 64, 16, "bfloat16", {}),
    ([0, 1, 15, 16, 17], 1, 2, 4, 128, 16, "bfloat16", {}),                    # an empty slot, and lengths about a group's
    ([63, 64, 65, 129, 1000], 1, 1, 8, 128, 64, "float16", {}),
    ([5, 300], 3, 2, 1, 256, 128, "bfloat16", {}),
    ([200, 31, 2], 2, 2, 7, 64, 32, "float16", {}),                           # 14 rows
    ([400, 77], 8, 1, 4, 128, 16, "bfloat16", {}),                            # 32 rows
    ([3, 0, 50], 5, 2, 3, 128, 64, "bfloat16", {}),                           # fewer keys than query tokens: rows that see nothing
    ([70, 129, 33], 17, 2, 4, 128, 64, "bfloat16", {}),                       # 68 rows
    ([260, 17], 17, 1, 8, 128, 16, "float16", {}),                            # 136 rows: past one tile of 128
    ([140, 9], 40, 2, 5, 64, 32, "bfloat16", {}),                             # 200 rows
    ([300], 130, 1, 2, 256, 64, "bfloat16", {}),
    ([500, 20], 1, 2, 4, 128, 32, "bfloat16", {"window": 1}),
    ([500, 100], 9, 1, 4, 128, 64, "bfloat16", {"window": 70}),
    ([700, 3], 33, 1, 4, 64, 16, "float16", {"window": 130}),
    ([90, 257], 12, 2, 2, 128, 32, "bfloat16", {"causal": False}),
    ([300, 0], 48, 1, 4, 128, 64, "float16", {"causal": False}),
    ([100, 40], 7, 1, 4, 128, 16, "bfloat16", {"tree": "drafts"}),
    ([170, 64], 64, 1, 3, 128, 64, "bfloat16", {"tree": "drafts"}),
    ([150, 80], 70, 2, 2, 64, 32, "float16", {"tree": "drafts"}),             # two words a mask
    ([8, 8], 8, 1, 4, 128, 16, "bfloat16", {"tree": "empty"}),                # masks without a bit and nothing before them
    ([64, 64], 40, 1, 4, 64, 64, "float16", {"tree": "empty"}),
    ([90], 6, 1, 4, 128, 64, "float16", {"scale": -0.3}),
    ([90], 40, 1, 4, 128, 64, "float16", {"scale": 0.0}),
    ([3000, 1, 2500], 1, 4, 4, 128, 128, "bfloat16", {}),                      # items cut over many CTAs
    ([2100, 900], 20, 2, 4, 128, 64, "bfloat16", {}),
    ([2000], 6, 2, 4, 256, 32, "float16", {}),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend(torch, kv, case):
    lens, t, h, group, d, page, dtype, more = CASES[case]
    n, dtype = len(lens), getattr(torch, dtype)
    c = make(kv, torch, n, max(lens), h, d, page, seed=case)
    kvs = fill(torch, c, lens, 100 + case)
    q = randn(torch, (n * t, h * group, d), dtype, 200 + case) * 1.5
    more = dict(more)
    kind = more.pop("tree", None)
    if kind:
        words = -(-t // 64)
        b = np.zeros((n * t, words), np.uint64)
        if kind == "drafts":
            g = np.random.RandomState(case)
            for i in range(n):
                for u in range(t):
                    if u and g.rand() < 0.9:
                        b[i * t + u] = b[i * t + g.randint(u)]
                    if g.rand() < 0.95:
                        b[i * t + u, u // 64] |= np.uint64(1) << np.uint64(u % 64)
        more["tree"] = torch.from_numpy(b.view(np.int64)).cuda()
    before = c.state.clone()
    out, lse = c.attend(q, **more)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, [t] * n, **more)
    assert torch.equal(before, c.state)
    again = c.attend(q, **more)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse.view(torch.int32), again[1].view(torch.int32))


@pytest.mark.parametrize("d,group,counts", [(128, 4, [1, 0, 9, 2]), (128, 4, [40, 0, 3, 70]), (64, 2, [5, 100, 0, 33]), (256, 1, [2, 40, 0, 9])])
def test_attend_ragged_queries_any_slots_and_strides(torch, kv, d, group, counts):
    """Entries with different numbers of query tokens, in slots out of order; q with heads outermost, at an odd address."""
    lens, h = [300, 7, 110, 0, 201, 64], 2
    c = make(kv, torch, 6, 320, h, d, 32, seed=d)
    kvs = fill(torch, c, lens, 7)
    slots = [4, 0, 5, 2]
    total, heads = sum(counts), h * group
    q = randn(torch, (heads * total * d + 1,), torch.float16, 8)[1:].view(heads, total, d).transpose(0, 1)
    ip = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    out, lse = c.attend(q, ip, sl, max_q=max(counts))
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, counts, slots=slots)


@pytest.mark.parametrize("t", [3, 40])
def test_attend_longest_window(torch, kv, t):
    """A window as long as an int holds limits nothing, also where an entry has more query tokens than keys."""
    lens, h, d = [2, 0, 100], 2, 64
    c = make(kv, torch, 3, 128, h, d, 16)
    kvs = fill(torch, c, lens, 11)
    q = randn(torch, (3 * t, h * 2, d), torch.bfloat16, 12)
    out, lse = c.attend(q, window=2 ** 31 - 1)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, [t] * 3)
    for bad in (2 ** 31, 2 ** 32 + 5, -1):
        with pytest.raises((ValueError, RuntimeError)):
            c.attend(q, window=bad)


def test_attend_many_entries(torch, kv):
    """More (entry, row tile) pairs than a CTA scans for itself, for both ways of dividing the rows."""
    n, h, d = 600, 1, 64
    lens = [int(x) for x in np.random.RandomState(0).randint(0, 90, n)]
    c = make(kv, torch, n, 96, h, d, 16)
    kvs = fill(torch, c, lens, 1)
    for t, group in ((1, 2), (25, 3)):
        q = randn(torch, (n * t, h * group, d), torch.bfloat16, 2)
        out, lse = c.attend(q)
        assert c.status() == 0
        check(torch, c, kvs, q, out, lse, [t] * n, rows=(0, t - 1))


@pytest.mark.parametrize("t", [1, 40])
def test_attend_rows_do_not_touch_one_another(torch, kv, t):
    """A NaN or an infinity in one query row changes that row alone; very large and very small rows keep their accuracy."""
    h, d, group = 1, 128, 4
    c = make(kv, torch, 1, 200, h, d, 16)
    kvs = fill(torch, c, [200], 3)
    q = randn(torch, (t, group, d), torch.bfloat16, 4)
    clean, clean_lse = c.attend(q)
    q2 = q.clone()
    q2[0, 1, 5] = float("nan")
    q2[0, 2, 6] = float("inf")
    out, lse = c.attend(q2)
    keep = torch.ones(t, group, dtype=torch.bool, device="cuda")
    keep[0, 1] = keep[0, 2] = False
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    for factor in (2.0 ** -60, 2.0 ** 60):
        big = q * factor
        out, lse = c.attend(big, scale=d ** -0.5 / factor)
        check(torch, c, kvs, big, out, lse, [t], scale=d ** -0.5 / factor)
    assert c.status() == 0


@pytest.mark.parametrize("t", [1, 40])
def test_attend_growing_scores(torch, kv, t):
    """Keys in order of their score, so that the running maximum is raised again and again, by little and by much."""
    h, d, L = 1, 128, 700
    c = make(kv, torch, 2, L, h, d, 64)
    base = randn(torch, (1, 1, d), torch.float32, 5)
    for s, top in enumerate((4.0, 40.0)):
        k = (base * torch.linspace(0.01, top, L).cuda()[:, None, None]).to(torch.bfloat16)
        c.append(k, randn(torch, (L, h, d), torch.bfloat16, 6 + s), slots=torch.tensor([s], dtype=torch.int32, device="cuda"))
    assert c.status() == 0
    kk, vv = c.read(torch.zeros(2, dtype=torch.int32, device="cuda"), L, dtype=torch.float32)
    kvs = [(kk[i].double().cpu().numpy(), vv[i].double().cpu().numpy()) for i in range(2)]
    q = base.expand(2 * t, 2, d).to(torch.float16).contiguous()
    out, lse = c.attend(q)
    check(torch, c, kvs, q, out, lse, [t, t])


def test_attend_past_32_bit_offsets(torch, kv):
    """Pages whose bytes lie past 4 GB in the pool."""
    h, d, page = 8, 128, 128
    each = kv.page_bytes(page, h, d)
    num = (1 << 32) // each + 40
    c = kv.KvCache(num, page, h, d, 2, 16, k_scale=scales(torch, h), v_scale=scales(torch, h, 1))
    c.refs[:num - 24] = 1
    kvs = fill(torch, c, [1500, 700], 1)
    assert int(c.tables[:, 0].min()) >= num - 24 and c.status() == 0
    for t in (1, 30):
        q = randn(torch, (2 * t, 2 * h, d), torch.bfloat16, 2)
        out, lse = c.attend(q)
        check(torch, c, kvs, q, out, lse, [t, t], rows=(0, t - 1))
    k, _ = c.read(torch.zeros(2, dtype=torch.int32, device="cuda"), 1500, dtype=torch.float32)
    np.testing.assert_array_equal(k[0].cpu().numpy(), kvs[0][0].astype(np.float32))
    parents = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    c.fork(parents)
    k2, _ = c.read(torch.zeros(2, dtype=torch.int32, device="cuda"), 1500, dtype=torch.float32)
    assert torch.equal(k2[0], k2[1]) and torch.equal(k2[0], k[0]) and c.status() == 0


# ------------------------------------------------------------------------------------------------ pages

def same(c, model, what):
    np.testing.assert_array_equal(c.state.cpu().numpy(), model.state(), err_msg=what)


@pytest.mark.parametrize("page,d,seed", [(16, 64, 0), (32, 128, 1), (64, 64, 2), (128, 256, 3), (16, 128, 4)])
def test_pages_against_the_model(torch, kv, page, d, seed):
    """A hundred random steps of all calls; tables, references and lengths after each, every held token at the end of each tenth."""
    g = np.random.RandomState(seed)
    n, h, max_pages, num = 6, 2, 400 // page + 2, 5 * (400 // page) + 6
    pool = torch.full((num, h, page // 16, 18 * d), 0xFF, dtype=torch.uint8, device="cuda")
    c = kv.KvCache(num, page, h, d, n, max_pages, k_scale=scales(torch, h, seed), v_scale=scales(torch, h, seed + 1), pool=pool)
    model = R.Model(num, page, n, max_pages)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    refused = 0
    for step in range(100):
        op = g.choice(["append", "append", "compact", "compact", "fork", "cut", "free"])
        slots = [int(x) for x in g.permutation(n)[:g.randint(1, n + 1)]]
        ok = True
        if op == "append":
            counts = [int(g.choice([0, 1, 5, 17, 60, 130])) for _ in slots]
            k, v = (randn(torch, (sum(counts), h, d), torch.bfloat16, 1000 * seed + 2 * step + i) for i in range(2))
            hk, hv = held(torch, k, c.k_scale), held(torch, v, c.v_scale)
            at = np.concatenate([[0], np.cumsum(counts)])
            ok = model.append([[(hk[x], hv[x]) for x in range(at[i], at[i + 1])] for i in range(len(slots))], slots)
            if sum(counts):
                c.append(k, v, i32(at), i32(slots))
        elif op in ("compact", "cut"):
            start = [int(max(0, model.lens[s] - g.randint(0, 80))) for s in slots]
            if op == "cut":
                keep = [[] for _ in slots]
                c.compact(i32(start), slots=i32(slots))
            else:
                keep = []
                for s, a in zip(slots, start):
                    block = model.lens[s] - a
                    chosen = np.sort(g.permutation(block)[:g.randint(0, block + 1)]) if g.rand() < 0.6 else np.arange(g.randint(0, block + 1))
                    keep.append([int(x) for x in chosen])
                table = np.full((len(slots), 80), -5)
                for i, x in enumerate(keep):
                    table[i, :len(x)] = x
                c.compact(i32(start), i32(table), i32([len(x) for x in keep]), i32(slots))
            ok = model.compact(slots, start, keep)
        elif op == "fork":
            parents = [int(x) if g.rand() < 0.5 else i for i, x in enumerate(g.randint(-1, n, n))]
            ok = model.fork(parents)
            c.fork(i32(parents))
        else:
            ok = model.compact(slots, [0] * len(slots), [[]] * len(slots))
            c.free(i32(slots))
        status = c.status()
        assert status == (0 if ok else -7), (step, op, status)
        refused += not ok
        same(c, model, f"step {step}: {op}")
        if step % 10 == 9:
            most = max(max(model.lens), 1)
            k, v = (x.cpu().numpy() for x in c.read(i32([0] * n), most, dtype=torch.float32))
            for s in range(n):
                for p, (wk, wv) in enumerate(model.tokens(s)):
                    np.testing.assert_array_equal(k[s, p], wk)
                    np.testing.assert_array_equal(v[s, p], wv)
    assert refused < 60


def test_a_forked_sequence_is_attended_like_its_parent(torch, kv):
    h, d = 2, 128
    c = make(kv, torch, 3, 400, h, d, 64)
    fill(torch, c, [300, 20, 0], 5)
    c.fork(torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda"))
    assert c.lens.tolist() == [300, 300, 20] and c.status() == 0
    q = randn(torch, (1, 8, d), torch.bfloat16, 6)
    out, lse = c.attend(q.expand(3, 8, d).contiguous())
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1]) and not torch.equal(out[0], out[2])


# ------------------------------------------------------------------------------------------------ refusals, streams, graphs

def test_refused_on_the_device_and_nothing_changed(torch, kv):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    h, d = 1, 64
    c = kv.KvCache(5, 16, h, d, 3, 4)
    k = randn(torch, (64, h, d), torch.bfloat16, 1)
    c.append(k[:48], k[:48], i32([0, 30, 48]), i32([0, 1]))  # 2 + 2 of 5 pages
    assert c.status() == 0
    before, pool = c.state.clone(), c.pool.clone()
    bad = [
        (-7, lambda: c.append(k[:40], k[:40], i32([0, 8, 40]), i32([0, 2]))),     # one page is free, three are wanted
        (-7, lambda: c.append(k[:35], k[:35], slots=i32([0]))),                   # five pages in a row of four
        (-1, lambda: c.append(k[:4], k[:4], slots=i32([3]))),                     # no such slot
        (-1, lambda: c.append(k[:4], k[:4], slots=i32([-1]))),
        (-1, lambda: c.append(k[:4], k[:4], i32([0, 5]), i32([0]))),              # offsets past the rows
        (-1, lambda: c.append(k[:4], k[:4], i32([3, 1, 4]), i32([0, 1]))),
        (-1, lambda: c.compact(i32([31]), slots=i32([0]))),                       # past the length
        (-1, lambda: c.compact(i32([-1]), slots=i32([0]))),
        (-1, lambda: c.compact(i32([0]), slots=i32([7]))),
        (-1, lambda: c.compact(i32([10]), i32([[3, 3]]), i32([2]), i32([0]))),    # not ascending
        (-1, lambda: c.compact(i32([10]), i32([[3, 20]]), i32([2]), i32([0]))),   # past the length
        (-1, lambda: c.compact(i32([10]), i32([[-1, 2]]), i32([2]), i32([0]))),
        (-1, lambda: c.compact(i32([10]), i32([[0, 1]]), i32([3]), i32([0]))),    # more than the row has
        (-1, lambda: c.fork(i32([0, 1, 3]))),
        (-1, lambda: c.fork(i32([0, 1, -2]))),
        (-7, lambda: c.fork(i32([0, 0, 0]))),                                     # two copies, one page
    ]
    for code, call in bad:
        call()
        assert c.status() == code and c.status() == 0
        assert torch.equal(c.state, before) and torch.equal(c.pool, pool)
    # a slot that is none reads and attends as an empty one
    out, lse = c.attend(k[:1].expand(1, 1, d).contiguous(), slots=i32([5]))
    assert c.status() == -1 and not out.any() and lse.item() == -math.inf
    a, b = c.read(i32([0]), 4, i32([-3]))
    assert c.status() == -1 and not a.any() and not b.any()
    with pytest.raises(Exception, match="invalid argument"):
        c.fork(i32([9, 9, 9]))
        c.status(check=True)


def test_refused_on_the_host(torch, kv):
    from speculative_decoding_serial_gb300.whead import WheadError
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = kv.KvCache(5, 16, 2, 64, 3, 4)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: c.append(x, x[:3]), lambda: c.append(x, x.half()), lambda: c.append(x.cpu(), x.cpu()),
                 lambda: c.append(x.transpose(1, 2), x.transpose(1, 2)), lambda: c.append(x, x, slots=i32([0]).long()),
                 lambda: c.append(x[:, :, ::2], x[:, :, ::2]), lambda: c.attend(x[:, :, :32]), lambda: c.attend(x.float()),
                 lambda: c.attend(x, tree=torch.zeros(3, dtype=torch.int64, device="cuda")), lambda: c.read(i32([0]), 4),
                 lambda: c.compact(i32([0, 0, 0]), i32([[0]] * 3)), lambda: c.fork(i32([0])),
                 lambda: c.attend(x, out=x[:2], slots=i32([0])), lambda: c.append(x.double(), x.double(), slots=i32([0]))):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: c.attend(torch.zeros(3, 3, 64, dtype=torch.bfloat16, device="cuda")),           # 3 heads on 2
                 lambda: c.attend(x, slots=i32([0, 1, 2])), lambda: c.append(x, x),                     # 4 tokens on 3 slots
                 lambda: c.attend(x, slots=i32([0]), window=4, causal=False), lambda: c.attend(x, slots=i32([0]), window=-1),
                 lambda: c.attend(x, slots=i32([0]), scale=float("nan")), lambda: c.attend(x, slots=i32([0]), max_q=2)):
        with pytest.raises(WheadError):
            call()
    for args in ((5, 24, 2, 64, 3, 4), (5, 16, 2, 96, 3, 4), (0, 16, 2, 64, 3, 4), (5, 16, 2, 64, 5000, 4)):
        with pytest.raises((WheadError, ValueError)):
            kv.KvCache(*args)
    assert c.status() == 0


def test_nothing_to_do(torch, kv):
    c = kv.KvCache(5, 16, 2, 64, 3, 4)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    c.append(x, x, slots=none)
    c.append(x, x)
    c.append(x, x, torch.zeros(4, dtype=torch.int32, device="cuda"))
    out, lse = c.attend(x)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    c.read(none, 4, none)
    c.read(torch.zeros(3, dtype=torch.int32, device="cuda"), 0)
    c.compact(none, slots=none)
    c.fork(torch.arange(3, dtype=torch.int32, device="cuda"))
    assert c.status() == 0 and not c.lens.any()


def test_other_streams_and_graphs(torch, kv):
    """One verification step on a side stream, then captured once and replayed: the same state and outputs."""
    h, d, t = 2, 128, 5
    c = make(kv, torch, 2, 200, h, d, 16)
    fill(torch, c, [100, 37], 9)
    kept = c.state.clone()
    k, v = randn(torch, (2 * t, h, d), torch.bfloat16, 1), randn(torch, (2 * t, h, d), torch.bfloat16, 2)
    q = randn(torch, (2 * t, 4 * h, d), torch.bfloat16, 3)
    start = c.lens.clone()
    keep = torch.tensor([[0, 2, 4], [1, 3, 0]], dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2 * t, 4 * h, device="cuda")

    def step():
        c.state.copy_(kept)
        c.append(k, v)
        c.attend(q, out=out, lse=lse)
        c.compact(start, keep, count)

    step()
    assert c.status() == 0
    want = out.clone(), lse.clone(), c.state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        step()
        side.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(c.state, want[2])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for _ in range(3):
            out.zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(c.state, want[2])
        assert c.status() == 0


@pytest.mark.parametrize("t,group,option", [(2, 4, "causal"), (2, 4, "window"), (2, 4, "tree"), (40, 4, "causal"), (40, 2, "window"), (40, 4, "tree")])
def test_a_token_of_nothing_but_nan(torch, kv, t, group, option):
    """A token, and a block of 16 channels, that hold no number at all are held as zeros: where they are seen, and where a mask hides them."""
    h, d, lens = 2, 128, [90, 61]
    c = make(kv, torch, 2, 96, h, d, 32)
    k, v = randn(torch, (sum(lens), h, d), torch.bfloat16, 31), randn(torch, (sum(lens), h, d), torch.bfloat16, 32)
    for x in (k, v):
        x[[0, 50, 88, 89, 95, 150]] = float("nan")
        x[70, :, 16:32] = float("nan")
    ip = torch.tensor([0, 90, 151], dtype=torch.int32, device="cuda")
    c.append(k, v, ip)
    got = c.read(torch.zeros(2, dtype=torch.int32, device="cuda"), 90, dtype=torch.float32)
    hk, hv = held(torch, k, c.k_scale), held(torch, v, c.v_scale)
    for y, w in zip(got, (hk, hv)):
        np.testing.assert_array_equal(y[0].cpu().numpy(), w[:90])
        np.testing.assert_array_equal(y[1, :61].cpu().numpy(), w[90:])
    kvs = [(hk[a:b].astype(np.float64), hv[a:b].astype(np.float64)) for a, b in ((0, 90), (90, 151))]
    more = {"window": {"window": 3}, "causal": {}}.get(option)
    if more is None:
        bits = torch.ones(2 * t, dtype=torch.int64, device="cuda") << torch.arange(t, device="cuda").repeat(2)
        more = {"tree": torch.where(torch.arange(2 * t, device="cuda") % t == t - 1, 1, bits)}  # the last sees the first, the others themselves
    q = randn(torch, (2 * t, h * group, d), torch.bfloat16, 33)
    out, lse = c.attend(q, **more)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, [t, t], **more)


@pytest.mark.parametrize("d,group,most,count", [(128, 4, 17, 32), (128, 4, 3, 4), (64, 2, 70, 100), (64, 1, 3, 8), (256, 1, 5, 8), (128, 4, 17, 200), (64, 4, 2, 40)])
def test_attend_more_tokens_than_max_q(torch, kv, d, group, most, count):
    """Reported, whether the row tile has room for them or not; that entry's rows are left alone and the others' are right."""
    h, lens = 2, [3000, 2900, 64]
    c = make(kv, torch, 3, 3000, h, d, 64, seed=d)
    kvs = fill(torch, c, lens, 41)
    counts = [most, count, 1]
    ip = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    q = randn(torch, (sum(counts), h * group, d), torch.bfloat16, 42)
    out, lse = torch.full_like(q, 7.0), torch.full((sum(counts), h * group), 9.0, device="cuda")
    c.attend(q, ip, max_q=most, out=out, lse=lse)
    assert c.status() == -1
    assert (out[most:most + count] == 7.0).all() and (lse[most:most + count] == 9.0).all()
    keep = torch.ones(sum(counts), dtype=torch.bool, device="cuda")
    keep[most:most + count] = False
    check(torch, c, [kvs[0], kvs[2]], q[keep], out[keep], lse[keep], [most, 1])
    c.attend(q, ip, max_q=max(counts), out=out, lse=lse)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, counts, rows=(0, 1, count - 1))


@pytest.mark.parametrize("t", [1, 40])
@pytest.mark.parametrize("power", [124, 104, -104, -122, -130])
def test_attend_query_rows_over_the_types_range(torch, kv, t, power):
    """Rows of bf16 up to its largest values and down among those below its normal ones, with the scale the other way."""
    h, d, group = 1, 128, 4
    c = make(kv, torch, 1, 200, h, d, 16)
    kvs = fill(torch, c, [200], 3)
    q = randn(torch, (t, group, d), torch.float32, 4).mul(2.0 ** (power / 2)).mul(2.0 ** (power / 2)).bfloat16()
    assert torch.isfinite(q).all() and q.any()
    scale = d ** -0.5 * 2.0 ** -max(power, -126)
    out, lse = c.attend(q, scale=scale)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, [t], scale=scale)


@pytest.mark.parametrize("factor", [-2.0 ** 110, -2.0 ** 33, 2.0 ** 33, 2.0 ** 110])
@pytest.mark.parametrize("d,group,t", [(128, 4, 1), (64, 4, 2), (128, 4, 5), (64, 2, 40), (128, 2, 130), (256, 1, 3)])
def test_attend_equal_scores_of_any_size(torch, kv, d, group, t, factor):
    """Keys that are all alike, with scores from 1e9 to 1e33 of either sign: every one counts the same, in one CTA or in many."""
    h, L = 2, 2500
    c = make(kv, torch, 2, L, h, d, 64)
    base = randn(torch, (1, h, d), torch.bfloat16, 51)
    v = randn(torch, (L + 20, h, d), torch.bfloat16, 52)
    c.append(base.expand(L + 20, h, d), v, torch.tensor([0, L, L + 20], dtype=torch.int32, device="cuda"))
    k = held(torch, base, c.k_scale).astype(np.float64)[0]
    vv = held(torch, v, c.v_scale).astype(np.float64)
    q = (base.float() * factor).bfloat16()[:, :, None].expand(2 * t, h, group, d).reshape(2 * t, h * group, d).contiguous()
    out, lse = c.attend(q)
    assert c.status() == 0
    o, l, qq = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for i, (lo, n) in enumerate(((0, L), (L, 20))):
        for row in range(t):
            see = max(n - t + row + 1, 0)
            for a in range(h * group):
                x, at = vv[lo:lo + see, a // group], (i * t + row, a)
                if not see:
                    assert not o[at].any() and l[at] == -np.inf
                    continue
                # p is the same for all: what is left of the bounds above is the rounding of the sums and of the output
                tol = 2.0 ** -8 * np.abs(x.mean(0)) + (see + 256) * 2.0 ** -25 * np.abs(x).mean(0) + 2.0 ** -24 * np.abs(x).max()
                assert (np.abs(o[at] - x.mean(0)) <= tol).all(), at
                want = k[a // group] @ qq[at] * d ** -0.5 + np.log(see)
                assert abs(want) > 1e9 and abs(l[at] - want) <= (d + 8) * 2.0 ** -23 * abs(want), at


@pytest.mark.parametrize("t", [1, 3, 40, 130])
@pytest.mark.parametrize("factor", [2.0 ** 28, 2.0 ** 100])
def test_attend_large_scores_that_grow(torch, kv, t, factor):
    """Runs of like keys whose scores, far past the 24 bits of an fp32 number, grow from run to run: the latest run alone counts."""
    h, d, group, L, run = 8, 128, 2, 6000, 500
    c = make(kv, torch, 2, L, h, d, 64)
    base = randn(torch, (1, h, d), torch.float32, 53)
    k = (base * 0.2 * 1.25 ** torch.arange(L // run).cuda().repeat_interleave(run)[:, None, None]).bfloat16()
    v = randn(torch, (L, h, d), torch.bfloat16, 54)
    for slot in range(2):
        c.append(k, v, slots=torch.tensor([slot], dtype=torch.int32, device="cuda"))
    kk, vv = (held(torch, x, g).astype(np.float64) for x, g in ((k[::run], c.k_scale), (v, c.v_scale)))
    q = (base * factor).bfloat16().repeat_interleave(group, 1).expand(2 * t, h * group, d).contiguous()
    scores = np.einsum("rhd,hd->rh", kk, q[0, ::group].double().cpu().numpy())
    assert (scores[0] > 1e8).all() and (scores[1:] > 1.1 * scores[:-1]).all()
    out, lse = c.attend(q)
    assert c.status() == 0
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in range(2):
        for row in sorted({0, t // 2, t - 1}):
            see = L - t + row + 1
            first = (see - 1) // run * run
            for a in range(h * group):
                x, at = vv[first:see, a // group], (i * t + row, a)
                tol = 2.0 ** -8 * np.abs(x.mean(0)) + (see + 256) * 2.0 ** -25 * np.abs(x).mean(0) + 2.0 ** -24 * np.abs(x).max()
                assert (np.abs(o[at] - x.mean(0)) <= tol).all(), at
                want = scores[first // run, a // group] * d ** -0.5
                assert abs(l[at] - want) <= (d + 8) * 2.0 ** -23 * want, at


def test_sizes_that_do_not_fit_are_refused(torch, kv):
    """Windows and most tokens of an entry that wrap to a right number in 32 bits."""
    c = make(kv, torch, 2, 64, 1, 64, 16)
    fill(torch, c, [20, 30], 61)
    q = randn(torch, (2, 1, 64), torch.bfloat16, 62)
    for bad in (-2 ** 32, -2 ** 32 + 5, -2 ** 31, 2 ** 32, 2 ** 32 + 5, -1):
        with pytest.raises((ValueError, RuntimeError)):
            c.attend(q, window=bad)
        with pytest.raises((ValueError, RuntimeError)):
            c.attend(q, max_q=bad)
    assert c.status() == 0


def test_gradients_are_refused(torch, kv):
    c = make(kv, torch, 1, 64, 2, 64, 16)
    x = randn(torch, (4, 2, 64), torch.bfloat16, 63)
    y = x.clone().requires_grad_()
    for call in (lambda: c.append(y, x), lambda: c.append(x, y), lambda: c.attend(y)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert c.lens.item() == 0
    with torch.no_grad():
        c.append(y, y)
        out, _ = c.attend(y)
    assert c.lens.item() == 4 and not out.requires_grad and c.status() == 0


@pytest.mark.parametrize("page", [-1, 5, 2 ** 31 - 1])
def test_a_table_that_names_no_page_is_not_written_through(torch, kv, page):
    """A caller's table whose entry is no page: append and compact report it and write nowhere."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = kv.KvCache(5, 16, 2, 64, 2, 2)
    x = randn(torch, (40, 2, 64), torch.bfloat16, 64)
    c.append(x[:30], x[:30], i32([0, 10, 30]))
    assert c.status() == 0
    c.tables[1, 1] = page
    pool = c.pool.clone()
    c.compact(i32([17]), i32([[1, 2]]), i32([2]), i32([1]))
    assert c.status() == -6 and torch.equal(c.pool, pool)
    c.append(x[:1], x[:1], slots=i32([1]))
    assert c.status() == -6 and torch.equal(c.pool, pool)


def test_compact_that_keeps_no_column(torch, kv):
    """keep without a column keeps nothing, as keep with columns and counts of zero does."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = kv.KvCache(8, 16, 1, 64, 2, 4)
    x = randn(torch, (60, 1, 64), torch.bfloat16, 65)
    c.append(x, x)
    c.compact(i32([17, 3]), torch.empty(2, 0, dtype=torch.int32, device="cuda"), i32([0, 0]))
    assert c.status() == 0 and c.lens.tolist() == [17, 3] and int((c.refs > 0).sum()) == 3
    c.compact(i32([17, 3]), torch.empty(2, 0, dtype=torch.int32, device="cuda"), i32([0, 1]))  # a count past the row
    assert c.status() == -1 and c.lens.tolist() == [17, 3]


@pytest.mark.parametrize("lens,t,d,page,dtype,more", [
    ([6000, 2987], 300, 128, 64, "bfloat16", {}),                     # two tiles, some 20 blocks a CTA
    ([5003, 4000], 261, 64, 16, "float16", {"window": 1500}),
    ([4000, 4999], 200, 128, 128, "float16", {"causal": False}),
    ([9000, 3000, 6001], 17, 128, 64, "bfloat16", {}),                # one tile, some 6
    ([9000, 3000, 6001], 20, 64, 32, "float16", {"causal": False}),
])
def test_attend_many_blocks_a_cta(torch, kv, lens, t, d, page, dtype, more):
    """CTAs that go through many blocks of keys and several items: every buffer and barrier comes round again."""
    h, group, n = 8, 4, len(lens)
    c = make(kv, torch, n, max(lens), h, d, page, seed=t)
    kvs = fill(torch, c, lens, 71)
    q = randn(torch, (n * t, h * group, d), getattr(torch, dtype), 72) * 1.5
    out, lse = c.attend(q, **more)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, [t] * n, rows=(0, 1, t // 2, t - 1), **more)
    again = c.attend(q, **more)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse.view(torch.int32), again[1].view(torch.int32))


@pytest.mark.parametrize("t", [40, 130])
def test_attend_growing_scores_over_many_blocks(torch, kv, t):
    """Scores that grow from block to block within a CTA, for one tile and two: outputs in tensor memory come down again and again."""
    h, d, L = 8, 128, 6000
    c = make(kv, torch, 2, L, h, d, 64)
    base = randn(torch, (1, h, d), torch.float32, 5)
    for s, top in enumerate((4.0, 40.0)):
        k = (base * torch.linspace(0.01, top, L).cuda()[:, None, None]).to(torch.bfloat16)
        c.append(k, randn(torch, (L, h, d), torch.bfloat16, 6 + s), slots=torch.tensor([s], dtype=torch.int32, device="cuda"))
    assert c.status() == 0
    kk, vv = c.read(torch.zeros(2, dtype=torch.int32, device="cuda"), L, dtype=torch.float32)
    kvs = [(kk[i].double().cpu().numpy(), vv[i].double().cpu().numpy()) for i in range(2)]
    q = base.repeat_interleave(2, 1).expand(2 * t, 2 * h, d).to(torch.float16).contiguous()
    out, lse = c.attend(q)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, [t, t], rows=(0, t // 2, t - 1))


@pytest.mark.parametrize("d,group", [(64, 4), (256, 1)])
def test_attend_ragged_trees(torch, kv, d, group):
    """Masks of one word for entries whose tokens together are more than 64, without max_q: the words say how many tokens an entry may have."""
    h, lens, counts = 2, [300, 45, 120], [33, 20, 40]
    c = make(kv, torch, 3, 320, h, d, 32, seed=d)
    kvs = fill(torch, c, lens, 81)
    b, g = [], np.random.RandomState(82)
    for n in counts:
        own = []
        for u in range(n):
            own.append((own[g.randint(u)] if u else 0) | 1 << u)
        b += own
    tree = torch.tensor(np.array(b, np.uint64).view(np.int64), device="cuda")
    ip = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    q = randn(torch, (sum(counts), h * group, d), torch.bfloat16, 83)
    out, lse = c.attend(q, ip, tree=tree)
    assert c.status() == 0
    check(torch, c, kvs, q, out, lse, counts, tree=tree)
    c.attend(q, torch.tensor([0, 5, 6, 93], dtype=torch.int32, device="cuda"), tree=tree)  # 87 tokens
    assert c.status() == -1
