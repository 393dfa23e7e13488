"""The 4-bit paged KV cache's operators as they are measured: cases, inputs, a plain form of each and its value in 64 bits.

The cache holds keys and values as e2m1 codes with an e4m3 scale for each 16 channels of a token and an f32 scale for each
KV head. A page holds `page` tokens of every KV head; inside it, 16 tokens of one head are a group of 18 * dim bytes:
the keys' codes (8 * dim bytes), the keys' scales (dim), the values' codes (8 * dim), the values' scales (dim), each in the
order in which the lanes of a warp take them (include/whead_kv.h says which byte is whose; `unpack` below is that text).
"""
import math

import numpy as np
import torch

own = False

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # e2m1 magnitudes by their three bits; bit 3 is the sign
CUTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)       # halfway points; a tie goes to the even code
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------------- the cases

def listed():
    at = dict(op="attend", causal=True, window=0, tree=False)
    return [
        # a single user's next token after a short prompt: latency alone
        dict(at, name="attend: 1 x 1 on 513", n=1, new=1, shortest=513, longest=513, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # an ordinary decoding batch of ragged lengths
        dict(at, name="attend: 16 x 1 on 300-8200", n=16, new=1, shortest=300, longest=8200, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # long contexts: the cache is far larger than L2
        dict(at, name="attend: 32 x 1 on 2000-32768", n=32, new=1, shortest=2000, longest=32768, heads=32, kv_heads=8, dim=128, page=128, dtype="bf16"),
        # verification of 16 drafted tokens for eight sequences (gamma = 16: 17 query tokens each)
        dict(at, name="attend: 8 x 17 on 900-6100", n=8, new=17, shortest=900, longest=6100, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # verification of a tree of drafts: masks among the new tokens, 7 query heads a KV head, small pages, f16
        dict(at, name="attend: 4 x 33 tree on 777-3001", n=4, new=33, shortest=777, longest=3001, heads=14, kv_heads=2, dim=64, page=16, dtype="f16", tree=True),
        # a chunk of a prompt on what is already cached
        dict(at, name="attend: 2 x 2048 on 4100-6200", n=2, new=2048, shortest=4100, longest=6200, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # one more token for each of a batch's sequences
        dict(op="append", name="append: 16 x 1", n=16, shortest=1, longest=1, past=2000, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # ragged prompts
        dict(op="append", name="append: 6 x 400-8000", n=6, shortest=400, longest=8000, past=0, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # the end of a verification step: drafts in, what was accepted stays (a chain of 17, and a tree's path of up to 33)
        dict(op="compact", name="compact: 8 x 17 chain", n=8, new=17, tree=False, past=2000, kv_heads=8, dim=128, page=64, dtype="bf16"),
        dict(op="compact", name="compact: 64 x 33 tree", n=64, new=33, tree=True, past=3000, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # candidates of a beam replace one another: every fourth is dropped, others take over a better one's sequence
        dict(op="fork", name="fork: 8 on 2000", n=8, past=2000, kv_heads=8, dim=128, page=64, dtype="bf16"),
        dict(op="fork", name="fork: 128 on 12000", n=128, past=12000, kv_heads=4, dim=128, page=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(v):
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "compact", "fork"])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kv_heads=kv_heads, dim=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "f16"]))
    if op == "attend":
        c["heads"] = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
        c["n"] = _log(rng, 1, 48)
        c["new"] = _log(rng, 1, 1500)
        c["longest"] = _log(rng, max(c["new"], 16), 40000)
        # no more pairs than a quarter of the listed prompt chunk's, no more cache than the listed long contexts', and no more scores in
        # the plain form than it holds at once there
        while c["n"] > 1 and (c["n"] * c["heads"] * c["new"] * c["longest"] * c["dim"] > 2e10 or c["n"] * kv_heads * c["longest"] * c["dim"] > 4e8):
            c["n"] = max(1, c["n"] // 2)
        while c["new"] > 1 and c["n"] * c["heads"] * c["new"] * c["longest"] * c["dim"] > 4e10:
            c["new"] = max(1, c["new"] // 2)
        c["longest"] = _size(c["longest"])
        c["shortest"] = max(c["new"], _log(rng, 1, c["longest"]))
        c["tree"] = c["new"] <= 64 and rng.random() < 0.3
        c["causal"] = c["tree"] or rng.random() < 0.8
        c["window"] = _log(rng, 16, 4000) if c["causal"] and not c["tree"] and rng.random() < 0.25 else 0
    elif op == "append":
        c["n"] = _log(rng, 1, 64)
        c["longest"] = _size(min(_log(rng, 1, 8000), max(1, 20000 // c["n"])))
        c["shortest"] = _log(rng, 1, c["longest"])
        c["past"] = rng.choice([0, _size(_log(rng, 1, 4000))])
    elif op == "compact":
        c["n"] = _log(rng, 1, 64)
        c["new"] = _log(rng, 2, 64)
        c["tree"] = rng.random() < 0.5
        c["past"] = _size(_log(rng, 1, 4000))
    else:
        c["n"] = _log(rng, 2, 128)
        c["past"] = _size(_log(rng, 1, 12000))
    return c


def _lengths(case):
    """What the case's host knows: lengths before the call, and tokens that come new, for each sequence (from the case alone)."""
    g = np.random.RandomState(sum(v * (i + 3) for i, (k, v) in enumerate(sorted(case.items())) if isinstance(v, int)) % 2**31)
    n = case["n"]
    if case["op"] == "attend":
        a = g.randint(case["shortest"], case["longest"] + 1, n)
        a[0] = case["longest"]
        return a, np.full(n, case["new"])
    past = g.randint(case["past"] // 2, case["past"] + 1, n) if case["past"] else np.zeros(n, np.int64)
    if case["op"] == "append":
        new = g.randint(case["shortest"], case["longest"] + 1, n)
        new[0] = case["longest"]
        return past, new
    return past, np.full(n, case.get("new", 0))


def _pairs(case):
    """Visible (query token, key) pairs of an attend case; a tree's drafts count as a chain."""
    length, new = _lengths(case)
    total = 0
    for a, t in zip(length.tolist(), new.tolist()):
        if not case["causal"]:
            total += a * t
            continue
        end = np.arange(a - t + 1, a + 1)
        total += int(np.minimum(end, case["window"]).sum() if case["window"] else end.sum())
    return total


def work(case):
    past, new = _lengths(case)
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    token = h * d * 9 // 8                      # bytes of a cached token's keys and values
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "attend":
        w, t = case["window"], int(new[0])
        seen = int(np.minimum(past, w + t - 1).sum() if w else past.sum())
        q = case["n"] * t * case["heads"] * d
        return {"bytes": seen * token + 2 * q * e + case["n"] * t * case["heads"] * 4 + 4 * seen // p, "flops": 4 * d * case["heads"] * _pairs(case)}
    if case["op"] == "append":                  # the tokens in, their codes out and in again, their values out
        total = int(new.sum())
        return {"bytes": total * (2 * 2 * h * d * e + 2 * token), "flops": total * 4 * h * d}
    if case["op"] == "compact":                 # drafts in, codes out, kept ones moved, kept ones' values out
        total = int(new.sum())
        return {"bytes": total * (2 * h * d * e + 3 * token + 2 * h * d * e), "flops": total * 4 * h * d}
    rows = -(-past // p)
    return {"bytes": int(rows.sum()) * 8 + case["n"] // 2 * 2 * p * token + case["n"] * p * (token + 2 * h * d * e), "flops": case["n"] * p * 2 * h * d}


# --------------------------------------------------------------------------------------------------- inputs

def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _fill(pool, pages, k_scale, v_scale, g):
    """Fills the given pages with quantised normal keys (some channels larger than others, as they are after a rotary
    embedding) and values, a few hundred MB at a time."""
    heads, groups, bytes_ = pool.shape[1:]
    d = bytes_ // 18
    wide = 1.0 + 3.0 * (torch.rand((heads, 1, d), generator=g, device="cuda") > 0.95).float()
    step = max(1, (1 << 27) // (heads * groups * 16 * d))
    for at in range(0, len(pages), step):
        part = pages[at:at + step]
        shape = (len(part), heads, groups * 16, d)
        k = quantise(_normal(shape, g) * wide, k_scale[:, None])
        v = quantise(_normal(shape, g), v_scale[:, None])
        pool[part] = pack(*k, *v)


def prepare(case, seed):
    """The cache with the sequences it already holds (their pages spread over the pool in no order), and the call's inputs."""
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    n, h, d, p = case["n"], case["kv_heads"], case["dim"], case["page"]
    past, new = _lengths(case)
    op = case["op"]
    room = past if op == "attend" else past + new
    max_pages = int(-(-int(room.max()) // p)) + 1
    used = -(-past // p)
    first = np.concatenate([[0], np.cumsum(used)])
    extra = 0 if op == "attend" else int((-(-room // p) - used).sum()) + n
    num_pages = int(first[-1]) + extra + 7
    pages = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    state = torch.empty(n + num_pages + n * max_pages, dtype=torch.int32, device="cuda")
    lens, refs, tables = state[:n], state[n:n + num_pages], state[n + num_pages:].view(n, max_pages)
    lens.copy_(torch.from_numpy(past.astype(np.int32)))
    col = torch.arange(max_pages, device="cuda")[None, :]
    start, count = (torch.from_numpy(x.astype(np.int64)).cuda()[:, None] for x in (first[:-1], used))
    tables.copy_(torch.where(col < count, pages[(start + col).clamp(max=num_pages - 1)], -1))
    refs.zero_()
    refs[pages[:int(first[-1])].long()] = 1
    k_scale = torch.rand(h, generator=g, device="cuda") * 0.01 + 0.005
    v_scale = torch.rand(h, generator=g, device="cuda") * 0.01 + 0.005
    pool = torch.zeros((num_pages, h, p // 16, 18 * d), dtype=torch.uint8, device="cuda")
    held = pages[:int(first[-1])].long()
    if op == "attend" or op == "fork":
        _fill(pool, held, k_scale, v_scale, g)
    else:  # what lies before the block is not read: one group's worth of bytes in every page will do
        pool.copy_(torch.randint(0, 120, pool.shape[-1:], generator=g, device="cuda", dtype=torch.uint8))
    s = dict(case, pool=pool, state=state, start=state.clone(), k_scale=k_scale, v_scale=v_scale, num_pages=num_pages, max_pages=max_pages,
             most=int(room.max()), slots=torch.arange(n, dtype=torch.int32, device="cuda"))
    dtype = DTYPES[case["dtype"]]
    if op == "attend":
        t = case["new"]
        s["q"] = _normal((n * t, case["heads"], d), g, dtype)
        if case["tree"]:  # token u hangs on an earlier token of the block; bit v of its mask: v is u or above it
            up = (torch.rand((n, t), generator=g, device="cuda") * torch.arange(t, device="cuda")).long().cpu().numpy()
            bits = np.zeros((n, t), np.uint64)
            for u in range(t):
                bits[:, u] = np.uint64(1) << np.uint64(u)
                if u:
                    bits[:, u] |= bits[np.arange(n), up[:, u]]
            s["bits"] = torch.from_numpy(bits.view(np.int64)).cuda().reshape(n * t)
    elif op in ("append", "compact"):
        total = int(new.sum())
        s["k"], s["v"] = _normal((total, h, d), g, dtype), _normal((total, h, d), g, dtype)
        s["indptr"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        s["from"] = torch.from_numpy(past.astype(np.int32)).cuda()
        s["reads"] = int(new.max())
        if op == "compact":
            t = case["new"]
            if case["tree"]:  # a path of random depth through the block's tokens
                on = torch.rand((n, t), generator=g, device="cuda") < torch.rand((n, 1), generator=g, device="cuda")
                count = on.sum(1)
                keep = torch.sort(torch.where(on, torch.arange(t, device="cuda")[None], t), dim=1)[0]
                s["keep"] = torch.where(keep < t, keep, 0).to(torch.int32)
            else:
                count = (torch.rand(n, generator=g, device="cuda") * (t + 1)).long()
                s["keep"] = torch.arange(t, device="cuda", dtype=torch.int32)[None].repeat(n, 1)
            s["count"] = count.to(torch.int32)
    else:
        parent = torch.arange(n, device="cuda")
        other = (torch.rand(n, generator=g, device="cuda") * n).long()
        s["parents"] = torch.where(torch.arange(n, device="cuda") % 4 == 3, -1, torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, other, parent)).to(torch.int32)
        s["reads"] = p
    if own:
        from speculative_decoding_serial_gb300 import kv
        s["cache"] = kv.KvCache(num_pages, p, h, d, n, max_pages, k_scale=k_scale, v_scale=v_scale, pool=pool, state=state)
    return s


# --------------------------------------------------------------------------------------------------- the plain form

def quantise(x, g):
    """(codes, scale bytes) of x [..., dim] in groups of 16 channels; g: the heads' scales, of a shape that x[..., 0] takes."""
    x = x.float()
    b = x.reshape(*x.shape[:-1], -1, 16)
    g = g[..., None].float()
    s = ((b.abs().amax(-1)) / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = b * (1.0 / (s.float() * g))[..., None]
    y = torch.where(torch.isnan(y), 0.0, y)
    m = y.abs()
    code = torch.zeros(m.shape, dtype=torch.uint8, device=x.device)
    for i, cut in enumerate(CUTS):
        code += (m >= cut if i % 2 else m > cut).to(torch.uint8)
    code += (y < 0).to(torch.uint8) * 8
    return code.reshape(x.shape), s.view(torch.uint8)


def values(code, scale, g):
    """The f32 values that codes [..., dim] and scale bytes [..., dim / 16] stand for."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=code.device)
    y = table[code.int()].reshape(*scale.shape, 16) * (scale.view(torch.float8_e4m3fn).float() * g[..., None])[..., None]
    return y.reshape(code.shape)


def pack(kc, ks, vc, vs):
    """Codes [..., tokens, dim] and scale bytes [..., tokens, dim / 16] as groups [..., tokens / 16, 18 * dim]."""
    lead, (t, d) = kc.shape[:-2], kc.shape[-2:]
    r, c4, m = t // 16, d // 64, len(lead)
    lay = lambda x, shape, order: x.reshape(*lead, r, *shape).permute(*range(m + 1), *(m + 1 + i for i in order))  # noqa: E731
    a = lay(kc, (2, 8, c4, 4, 4, 2, 2), (2, 1, 4, 3, 5, 0, 6))          # hi g | c b t u2 un -> c g t b u2 hi un
    b = lay(ks, (2, 8, d // 16), (1, 2, 0))                             # hi g b -> g b hi
    c = lay(vc, (2, 4, 2, c4, 4, 8, 2), (3, 5, 1, 4, 0, 6, 2))          # hi t un | c b g e -> c g t b hi e un
    e = lay(vs, (2, 4, 2, d // 16), (1, 3, 0, 2))                       # hi t un | b -> t b hi un
    two = lambda x: x[..., 0] + x[..., 1] * 16  # noqa: E731
    return torch.cat([x.reshape(*lead, r, -1) for x in (two(a), b, two(c), e)], -1)


def unpack(x):
    """The inverse of pack."""
    d = x.shape[-1] // 18
    lead, r, c4, m = x.shape[:-2], x.shape[-2], d // 64, x.dim() - 2
    kc, ks, vc, vs = x.split([8 * d, d, 8 * d, d], -1)
    nib = lambda y: torch.stack([y & 15, y >> 4], -1)  # noqa: E731
    lay = lambda y, shape, order, last: y.reshape(*lead, r, *shape).permute(*range(m + 1), *(m + 1 + i for i in order)).reshape(*lead, r * 16, last)  # noqa: E731
    return (lay(nib(kc), (c4, 8, 4, 4, 2, 2, 2), (5, 1, 0, 3, 2, 4, 6), d), lay(ks, (8, d // 16, 2), (2, 0, 1), d // 16),
            lay(nib(vc), (c4, 8, 4, 4, 2, 2, 2), (4, 2, 6, 0, 3, 1, 5), d), lay(vs, (4, d // 16, 2, 2), (2, 0, 3, 1), d // 16))


def _views(s):
    n, num = s["n"], s["num_pages"]
    return s["state"][:n], s["state"][n:n + num], s["state"][n + num:].view(n, s["max_pages"])


def _read(s, start, count):
    """The values of `count` tokens of every sequence from its `start` on, in the case's type; zeros past the length."""
    lens, _, tables = _views(s)
    p = s["page"]
    width = -(-count // p) + 1
    first = start.long() // p
    page = tables.gather(1, (first[:, None] + torch.arange(width, device="cuda")).clamp(max=s["max_pages"] - 1)).long().clamp(min=0)
    kc, ks, vc, vs = unpack(s["pool"][page])                                             # [n, width, heads, page, ..]
    at = (start.long() - first * p)[:, None] + torch.arange(count, device="cuda")        # place among these tokens
    live = (start.long()[:, None] + torch.arange(count, device="cuda")) < lens[:, None]
    rows = torch.arange(s["n"], device="cuda")[:, None]
    out = []
    for code, scale, g in ((kc, ks, s["k_scale"]), (vc, vs, s["v_scale"])):
        y = values(code[rows, at // p, :, at % p], scale[rows, at // p, :, at % p], g)   # [n, count, heads, dim]
        out.append(torch.where(live[..., None, None], y, 0.0).to(DTYPES[s["dtype"]]))
    return out


def _free(refs, ranks):
    """The free pages of the given ranks, lowest first."""
    free = refs == 0
    order = torch.zeros(len(refs) + 1, dtype=torch.int32, device="cuda")
    order[torch.where(free, torch.cumsum(free, 0) - 1, len(refs))] = torch.arange(len(refs), dtype=torch.int32, device="cuda")
    return order[ranks.clamp(0, len(refs))]


def _append(s):
    lens, refs, tables = _views(s)
    n, p, indptr = s["n"], s["page"], s["indptr"].long()
    past = lens.long()
    now = past + indptr[1:] - indptr[:-1]
    col = torch.arange(s["max_pages"], device="cuda")[None]
    want = (col >= (-(-past // p))[:, None]) & (col < (-(-now // p))[:, None])
    rank = (torch.cumsum(want.reshape(-1), 0) - 1).reshape(want.shape)
    page = _free(refs, rank)
    tables.copy_(torch.where(want, page, tables))
    refs[page[want].long()] = 1
    lens.copy_(now)
    total = s["k"].shape[0]
    token = torch.arange(total, device="cuda")
    seq = torch.searchsorted(indptr[1:], token, right=True)
    pos = past[seq] + token - indptr[seq]
    # the pages that the new tokens lie in, each once: taken apart, given the new tokens, put together again
    touched = (col >= (past // p)[:, None]) & (col < (-(-now // p))[:, None]) & (now > past)[:, None]
    place = (torch.cumsum(touched.reshape(-1), 0) - 1).reshape(touched.shape)
    held = tables[touched].long()
    kc, ks, vc, vs = unpack(s["pool"][held])
    a, b = place[seq, pos // p], pos % p
    (kc[a, :, b], ks[a, :, b]), (vc[a, :, b], vs[a, :, b]) = quantise(s["k"], s["k_scale"]), quantise(s["v"], s["v_scale"])
    s["pool"][held] = pack(kc, ks, vc, vs)


def _compact(s):
    lens, refs, tables = _views(s)
    n, p, t = s["n"], s["page"], s["new"]
    start, keep, count = s["from"].long(), s["keep"].long(), s["count"].long()
    i = torch.arange(t, device="cuda")[None]
    live = i < count[:, None]
    stay = ((keep == i) & live).sum(1)                                  # the first kept tokens that are in place already
    before, now = -(-lens.long() // p), -(-(start + count) // p)
    col = torch.arange(s["max_pages"], device="cuda")[None]
    written = (col >= ((start + stay) // p)[:, None]) & (col < now[:, None])
    shared = written & (refs[tables.long().clamp(min=0)] > 1)
    rank = (torch.cumsum(shared.reshape(-1), 0) - 1).reshape(shared.shape)
    page = torch.where(shared, _free(refs, rank), tables)
    page = torch.where(col < now[:, None], page, -1)
    # the block's pages with the kept tokens moved up
    width = -(-t // p) + 1
    first = start // p
    region = (first[:, None] + torch.arange(width, device="cuda"))
    old = tables.gather(1, region.clamp(max=s["max_pages"] - 1)).long().clamp(min=0)
    src = torch.arange(width * p, device="cuda")[None].repeat(n, 1)
    src.scatter_(1, ((start - first * p)[:, None] + i), torch.where(live, (start - first * p)[:, None] + keep, (start - first * p)[:, None] + i))
    rows = torch.arange(n, device="cuda")[:, None]
    moved = [x[rows, src // p, :, src % p].reshape(n, width, p, x.shape[2], -1).transpose(2, 3) for x in unpack(s["pool"][old])]
    write = written.gather(1, region.clamp(max=s["max_pages"] - 1)) & (region < s["max_pages"])
    packed = pack(*moved)
    s["pool"][page.gather(1, region.clamp(max=s["max_pages"] - 1))[write].long()] = packed[write]
    gone = (col < before[:, None]) & ((col >= now[:, None]) | shared)
    refs.index_add_(0, tables[gone].long(), torch.full_like(tables[gone], -1))
    refs[page[shared].long()] = 1
    tables.copy_(page)
    lens.copy_(start + count)


def _fork(s):
    lens, refs, tables = _views(s)
    n, p = s["n"], s["page"]
    parent, me = s["parents"].long(), torch.arange(n, device="cuda")
    takes, leaves = (parent >= 0) & (parent != me), parent != me
    of = parent.clamp(min=0)
    length = torch.where(parent >= 0, lens.long()[of], 0)
    col = torch.arange(s["max_pages"], device="cuda")[None]
    part = takes & (length % p != 0)
    fresh = _free(refs, torch.cumsum(part, 0) - 1)
    last = (length // p)[:, None]
    row = torch.where(part[:, None] & (col == last), fresh[:, None], tables[of])
    row = torch.where(col < (-(-length // p))[:, None], row, -1)
    s["pool"][fresh[part].long()] = s["pool"][tables[of].gather(1, last.clamp(max=s["max_pages"] - 1))[part][:, 0].long()]
    gone = tables[leaves[:, None] & (col < (-(-lens.long() // p))[:, None])].long()
    more = row[takes[:, None] & (col < last)].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    refs.index_add_(0, more, torch.ones_like(more, dtype=torch.int32))
    refs[fresh[part].long()] = 1
    tables.copy_(row)
    lens.copy_(length)


def _attend(s):
    lens, _, tables = _views(s)
    n, t, h, d, p, most = s["n"], s["new"], s["kv_heads"], s["dim"], s["page"], s["most"]
    pages = -(-most // p)
    x = s["pool"][tables[:, :pages].long().clamp(min=0)].transpose(1, 2).reshape(n, h, -1, 18 * d)     # [n, heads, groups, bytes]
    kc, ks, vc, vs = unpack(x)
    del x
    k = values(kc, ks, s["k_scale"][None, :, None])
    del kc, ks
    q = s["q"].float().reshape(n, t, h, -1, d).permute(0, 2, 3, 1, 4).reshape(n, h, -1, d)             # [n, heads, group * t, dim]
    score = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    j = torch.arange(score.shape[-1], device="cuda")[None, None]
    end = lens.long()[:, None, None]
    pos = end - t + torch.arange(t, device="cuda")[None, :, None]
    see = (j < end).expand(n, t, -1)
    if s["causal"]:
        see = see & (j <= pos)
    if s["window"]:
        see = see & (j > pos - s["window"])
    if s["tree"]:
        u = (j - (end - t)).clamp(0, 63)
        see = see & ((j < end - t) | ((s["bits"].reshape(n, t, 1) >> u) & 1).bool())
    score = score.reshape(n, h, -1, t, score.shape[-1])
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    v = values(vc, vs, s["v_scale"][None, :, None])
    o = (score.reshape(n, h, -1, score.shape[-1]) @ v).reshape(n, h, -1, t, d) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(n * t, -1, d).to(s["q"].dtype)
    return o, lse.permute(0, 3, 1, 2).reshape(n * t, -1)


# --------------------------------------------------------------------------------------------------- one pass

def run(s):
    """attend: outputs and log sums. The others set the cache's state back to where the pass begins, work on it, and read back what
    it then holds of the tokens that they wrote."""
    op, cache = s["op"], s.get("cache")
    if op == "attend":
        if own:
            return cache.attend(s["q"], causal=s["causal"], window=s["window"], tree=s.get("bits"))
        return _attend(s)
    s["state"].copy_(s["start"])
    if own:
        if op != "fork":
            cache.append(s["k"], s["v"], s["indptr"])
        if op == "compact":
            cache.compact(s["from"], s["keep"], s["count"])
        if op == "fork":
            cache.fork(s["parents"])
            begin = ((cache.lens - 1).clamp_(min=0) // s["page"]) * s["page"]
        else:
            begin = s["from"]
        held = cache.read(begin, s["reads"], dtype=DTYPES[s["dtype"]])
        return [*held, cache.state]
    if op != "fork":
        _append(s)
    if op == "compact":
        _compact(s)
    if op == "fork":
        _fork(s)
        begin = ((_views(s)[0] - 1).clamp(min=0) // s["page"]) * s["page"]
    else:
        begin = s["from"]
    return [*_read(s, begin, s["reads"]), s["state"]]


# --------------------------------------------------------------------------------------------------- in 64 bits

class _Cache64:
    """The same inputs, taken one sequence at a time and with one byte's place worked out from the format's text."""

    def __init__(self, s):
        self.s, d = s, s["dim"]
        r, c = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
        b, u, hi, g = c // 16, c % 16, r // 8, r % 8
        lane = 4 * g + u // 4
        self.k_byte = (b // 4) * 512 + lane * 16 + (b % 4) * 4 + (u % 4 // 2) * 2 + hi
        self.k_nib = u % 2
        lane = 4 * (u // 2) + (r % 8) // 2
        self.v_byte = 9 * d + (b // 4) * 512 + lane * 16 + (b % 4) * 4 + hi * 2 + u % 2
        self.v_nib = r % 2
        r, b = np.meshgrid(np.arange(16), np.arange(d // 16), indexing="ij")
        self.k_scale = 8 * d + (r % 8) * (d // 8) + b * 2 + r // 8
        self.v_scale = 17 * d + (r % 8 // 2) * (d // 4) + b * 4 + (r // 8) * 2 + r % 2
        e = np.arange(256)
        f = np.where((e >> 3) & 15, (1 + (e & 7) / 8) * 2.0 ** (((e >> 3) & 15) - 7), (e & 7) / 8 * 2.0 ** -6)
        self.e4m3 = torch.from_numpy(f).cuda()
        mag = np.array([0, 1, 2, 3, 4, 6, 8, 12]) / 2
        self.e2m1 = torch.from_numpy(np.concatenate([mag, -mag])).cuda()

    def tokens(self, pages, head):
        """Keys and values, f64 [tokens, dim], of the given pages of one head."""
        x = self.s["pool"][pages, head].reshape(-1, self.s["pool"].shape[-1])
        out = []
        for byte, nib, scale, g in ((self.k_byte, self.k_nib, self.k_scale, self.s["k_scale"]), (self.v_byte, self.v_nib, self.v_scale, self.s["v_scale"])):
            y = x[:, torch.from_numpy(byte).cuda()]
            y = self.e2m1[torch.where(torch.from_numpy(nib).cuda() == 1, y >> 4, y & 15).int()]
            f = self.e4m3[x[:, torch.from_numpy(scale).cuda()].int()] * g[head].double()
            out.append((y * f.repeat_interleave(16, -1)).reshape(-1, self.s["dim"]))
        return out


def _round64(x, g):
    """x [..., dim] as the nearest values that the cache can hold: the block's scale rounded to e4m3 and each value to e2m1, in 64 bits."""
    b = x.double().reshape(*x.shape[:-1], -1, 16)
    g = g.double()[..., None]
    r = (b.abs().amax(-1) / (6 * g)).clamp(max=448.0)
    e = torch.floor(torch.log2(r.clamp(min=2.0 ** -6)))
    s = torch.round(r / 2 ** (e - 3)) * 2 ** (e - 3) * g
    y = (b / s[..., None]).nan_to_num(0.0)
    m = y.abs().clamp(max=6.0)
    q = torch.where(m < 2, torch.round(m * 2) / 2, torch.where(m < 4, torch.round(m), torch.round(m / 2) * 2))
    return (torch.sign(y) * q * s[..., None]).reshape(x.shape)


def _exact_attend(case, s):
    past, _ = _lengths(case)
    n, t, h, d, p = case["n"], case["new"], case["kv_heads"], case["dim"], case["page"]
    if _pairs(case) * case["heads"] * d * 4 > 3e12:
        return None
    held, tables = _Cache64(s), _views(s)[2]
    group = case["heads"] // h
    o = torch.zeros((n, t, case["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((n, t, case["heads"]), dtype=torch.float64, device="cuda")
    for i, length in enumerate(past.tolist()):
        j = torch.arange(length, device="cuda")[None]
        pos = length - t + torch.arange(t, device="cuda")[:, None]
        see = torch.ones((t, length), dtype=torch.bool, device="cuda")
        if case["causal"]:
            see &= j <= pos
        if case["window"]:
            see &= pos - j < case["window"]
        if case["tree"]:
            bits = s["bits"].reshape(n, t)[i].cpu().numpy().view(np.uint64)
            draft = torch.tensor([[bool((int(w) >> u) & 1) for u in range(t)] for w in bits], device="cuda")
            see[:, length - t:] &= draft
        for head in range(h):
            k, v = held.tokens(tables[i, :-(-length // p)].long(), head)
            for q_head in range(head * group, (head + 1) * group):
                q = s["q"].reshape(n, t, case["heads"], d)[i, :, q_head].double()
                z = torch.where(see, q @ k[:length].T / math.sqrt(d), -math.inf)
                lse[i, :, q_head] = torch.logsumexp(z, -1)
                o[i, :, q_head] = torch.softmax(z, -1).nan_to_num(0.0) @ v[:length]
    return o.reshape(n * t, -1, d), lse.reshape(n * t, -1)


def exact(case, seed):
    """attend: from the definition. append and compact: the values by rounding the inputs; fork: by reading the parents' pages. The state (whole
    numbers) has no value in 64 bits."""
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "attend":
        return _exact_attend(case, s)
    past, new = _lengths(case)
    n, h, d, p = case["n"], case["kv_heads"], case["dim"], case["page"]
    k = torch.zeros((n, s["reads"], h, d), dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    if case["op"] == "fork":
        held, tables, parents = _Cache64(s), _views(s)[2], s["parents"].tolist()
        for i, j in enumerate(parents):
            if j >= 0 and past[j]:
                last = (int(past[j]) - 1) // p
                live = int(past[j]) - last * p
                for head in range(h):
                    a, b = held.tokens(tables[j, last:last + 1].long(), head)
                    k[i, :live, head], v[i, :live, head] = a[:live], b[:live]
        return [k, v, None]
    at = np.concatenate([[0], np.cumsum(new)])
    a, b = _round64(s["k"], s["k_scale"]), _round64(s["v"], s["v_scale"])
    for i in range(n):
        pick = torch.arange(at[i], at[i + 1], device="cuda")
        if case["op"] == "compact":
            pick = at[i] + s["keep"][i, :int(s["count"][i])].long()
        k[i, :len(pick)], v[i, :len(pick)] = a[pick], b[pick]
    return [k, v, None]
