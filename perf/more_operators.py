"""The operators of a verification step as they are measured: cases, inputs, a plain form of each and its value in 64 bits.

    logprobs   log probabilities of given tokens under rows of logits, with the rows' entropy, log sum of exponentials and top alternatives
    verify     which drafted tokens stay under the target's logits, and the token after them
    attend     attention over the 4-bit paged cache with a sliding window and a few first tokens that stay visible

Random numbers come from Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", SC'11) with the call's seed as key,
so that they are inputs: both forms draw the same.
"""
import math
from statistics import NormalDist

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------------------------------------- the cases

def listed():
    lp = dict(op="logprobs", masked=0.0, temperature=1.0)
    ver = dict(op="verify", ragged=False)
    att = dict(op="attend", heads=32, kv_heads=8, dim=128, page=64, dtype="bf16")
    return [
        # a single user's next token, with the five alternatives that a client asks for: latency alone
        dict(lp, name="logprobs: 1 x 151936 top 5", rows=1, vocab=151936, dtype="bf16", top=5),
        # what the target gave a walk of 16 drafts: 17 rows, f32, no alternatives
        dict(lp, name="logprobs: 17 x 151936", rows=17, vocab=151936, dtype="f32", top=0),
        # a decoding batch with a full list of alternatives
        dict(lp, name="logprobs: 64 x 248064 top 20", rows=64, vocab=248064, dtype="bf16", top=20),
        # half the vocabulary ruled out by a grammar, an odd vocabulary (rows start anywhere), a temperature
        dict(lp, name="logprobs: 97 x 32003 masked", rows=97, vocab=32003, dtype="f16", top=8, masked=0.5, temperature=0.7),
        # a prompt scored: every token's log probability and the best alternative
        dict(lp, name="logprobs: 4096 x 151936 top 1", rows=4096, vocab=151936, dtype="bf16", top=1),
        # one sequence's 16 drafts, sampled
        dict(ver, name="verify: 1 x 16 sampled", n=1, gamma=16, vocab=151936, dtype="bf16", draft="bf16", temperature=1.0, accept=0.8),
        # greedy verification of a batch
        dict(ver, name="verify: 8 x 16 greedy", n=8, gamma=16, vocab=151936, dtype="f32", draft="", temperature=0.0, accept=0.8),
        # drafts without logits (found in the text, say), as many as each sequence has
        dict(ver, name="verify: 16 x 5 ragged", n=16, gamma=5, vocab=32003, dtype="f16", draft="", temperature=0.8, accept=0.6, ragged=True),
        # a large batch, drafts' logits in the f32 that the walk samples from
        dict(ver, name="verify: 64 x 16 sampled", n=64, gamma=16, vocab=151936, dtype="bf16", draft="f32", temperature=1.0, accept=0.8),
        # a stream's next token
        dict(att, name="attend: 1 x 1, 1024 + 4 of 20001", n=1, new=1, shortest=20001, longest=20001, window=1024, sinks=4),
        # a batch of streams
        dict(att, name="attend: 32 x 1, 4096 + 4 of 2000-32768", n=32, new=1, shortest=2000, longest=32768, window=4096, sinks=4),
        # chunks of two prompts, a system prompt's tokens staying visible
        dict(att, name="attend: 2 x 2048, 1024 + 100 of 4100-6200", n=2, new=2048, shortest=4100, longest=6200, window=1024, sinks=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "verify", "attend"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "logprobs":
        c = dict(op=op, vocab=_log(rng, 1000, 262144), dtype=kind, top=rng.choice([0, 1, 5, 20, 32]), masked=rng.choice([0.0, 0.0, 0.5, 0.9]),
                 temperature=rng.choice([1.0, 1.0, 0.6, 1.7]))
        # no more than the listed prompt's logits, and no more rounds of a search for the largest over them
        c["rows"] = _log(rng, 1, max(1, min(4096, 4096 * 151936 // (c["vocab"] * max(4, c["top"])))))
        return c
    if op == "verify":
        c = dict(op=op, vocab=_log(rng, 500, 262144), dtype=kind, temperature=rng.choice([0.0, 1.0, 0.7]), accept=rng.choice([0.4, 0.7, 0.9]),
                 ragged=rng.random() < 0.3, draft=rng.choice(["", kind, "f32"]), gamma=rng.choice([0, 1, 3, 5, 7, 8, 15, 16, 24]))
        c["n"] = _log(rng, 1, max(1, min(96, 64 * 33 * 151936 // (c["vocab"] * (2 * c["gamma"] + 1)))))
        return c
    kv_heads = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 4, 7, 8]), dim=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]),
             dtype=rng.choice(["bf16", "bf16", "f16"]), window=_log(rng, 8, 5000), sinks=rng.choice([1, 4, 4, 16, 33, 100, 200]), n=_log(rng, 1, 48), new=_log(rng, 1, 1200))
    c["longest"] = _log(rng, max(c["new"], 16), 40000)
    # no more pairs than in the listed chunks of prompts, no more cache than in the listed batch of streams
    while c["n"] > 1 and (c["n"] * c["heads"] * c["new"] * (c["window"] + c["new"]) * c["dim"] > 2e10 or c["n"] * kv_heads * c["longest"] * c["dim"] > 4e8):
        c["n"] = max(1, c["n"] // 2)
    while c["new"] > 1 and c["heads"] * c["new"] * (c["window"] + c["new"]) * c["dim"] > 2e10:
        c["new"] = max(1, c["new"] // 2)
    c["shortest"] = max(c["new"], _log(rng, 1, c["longest"]))
    return c


def _lengths(case):
    """The slots' lengths (from the case alone)."""
    g = np.random.RandomState(sum(v * (i + 3) for i, (k, v) in enumerate(sorted(case.items())) if isinstance(v, int)) % 2**31)
    a = g.randint(case["shortest"], case["longest"] + 1, case["n"])
    a[0] = case["longest"]
    return a


def work(case):
    if case["op"] == "logprobs":
        x = case["rows"] * case["vocab"]
        return {"bytes": x * SIZE[case["dtype"]] + case["rows"] * (4 + 12 + 8 * case["top"]), "flops": 8 * x}
    if case["op"] == "verify":
        # the rows up to the first draft that does not stay, as many as are to be expected; each draft stays with probability `accept`
        n, g, v, a = case["n"], case["gamma"] / (2 if case["ragged"] else 1), case["vocab"], case["accept"]
        tried = sum(a ** t for t in range(int(round(g))))   # drafts looked at
        rows = tried + a ** g                               # and the row after the last, where all stay
        size = rows * SIZE[case["dtype"]] + (tried * SIZE[case["draft"]] if case["draft"] and case["temperature"] else 0)
        return {"bytes": int(n * v * size) + n * (8 * case["gamma"] + 8), "flops": int(n * v * rows * 4)}
    past, t, w, s, d = _lengths(case), case["new"], case["window"], case["sinks"], case["dim"]
    seen = pairs = 0
    for a in past.tolist():
        end = np.arange(a - t + 1, a + 1)
        pairs += int((np.minimum(end, w) + np.minimum(np.maximum(end - w, 0), s)).sum())
        late = min(a, w + t - 1)
        seen += late + min(s, a - late)
    q = case["n"] * t * case["heads"]
    return {"bytes": seen * case["kv_heads"] * d * 9 // 8 + 2 * q * d * 2 + q * 4, "flops": 4 * d * case["heads"] * pairs}


# --------------------------------------------------------------------------------------------------- inputs

def _logits(rows, vocab, g):
    """Rows of f32 logits as language models give them: a broad bell, and a few tokens that stand out of it."""
    x = torch.randn((rows, vocab), generator=g, device="cuda") * 2.5
    at = torch.randint(0, vocab, (rows, 8), generator=g, device="cuda")
    return x.scatter_add_(1, at, torch.rand((rows, 8), generator=g, device="cuda") * 10 + 2)


def _sample(x, g):
    """A token of each row of f32 logits."""
    return (x - torch.log(-torch.log(torch.rand(x.shape, generator=g, device="cuda").clamp(1e-20, 1 - 1e-7)))).argmax(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    if case["op"] == "logprobs":
        rows, vocab, dtype = case["rows"], case["vocab"], DTYPES[case["dtype"]]
        x = torch.empty((rows, vocab), dtype=dtype, device="cuda")
        tokens = torch.empty(rows, dtype=torch.int32, device="cuda")
        for i in range(0, rows, 512):
            y = _logits(min(512, rows - i), vocab, g)
            if case["masked"]:
                y.masked_fill_(torch.rand(y.shape, generator=g, device="cuda") < case["masked"], -math.inf)
            tokens[i:i + 512] = _sample(y, g)
            x[i:i + 512] = y
        return dict(case, logits=x, tokens=tokens)
    if case["op"] == "verify":
        n, t, vocab, a = case["n"], case["gamma"], case["vocab"], case["accept"]
        target = torch.empty((n, t + 1, vocab), dtype=DTYPES[case["dtype"]], device="cuda")
        draft = torch.empty((n, t, vocab), dtype=DTYPES[case["draft"]], device="cuda") if case["draft"] else None
        tokens = torch.empty((n, t), dtype=torch.int32, device="cuda")
        # two softmaxes whose logits differ by normal noise of deviation s share 2 Phi(-s / 2) of their mass, which is how often a draft stays
        spread = -2 * NormalDist().inv_cdf(a / 2)
        for i in range(n):
            x = _logits(t + 1, vocab, g)
            if draft is not None:
                y = x[:t] + torch.randn((t, vocab), generator=g, device="cuda") * spread
                draft[i] = y
                say = _sample(y / (case["temperature"] or 1.0), g) if t else None
            else:
                # one token that the target likes as much as drafts are to stay, and the drafts are that token
                like = torch.randint(0, vocab, (t + 1, 1), generator=g, device="cuda")
                if case["temperature"]:
                    z = x / case["temperature"]
                    z.scatter_(1, like, -math.inf)
                    x.scatter_(1, like, ((torch.logsumexp(z, 1, keepdim=True) + math.log(a / (1 - a))) * case["temperature"]))
                    say = like[:t, 0]
                else:
                    x.scatter_(1, like, x.amax(1, keepdim=True) + 1)
                    say = torch.where(torch.rand(t, generator=g, device="cuda") < a, like[:t, 0], (like[:t, 0] + 1) % vocab)
            target[i] = x
            if t:
                tokens[i] = say
        drafted = (torch.rand(n, generator=g, device="cuda") * (t + 1)).to(torch.int32) if case["ragged"] else None
        return dict(case, target=target, draft=draft if case["temperature"] else None, tokens=tokens, drafted=drafted, seed=seed * 1000003 + 29, step=seed % 97)
    n, h, d, p, t = case["n"], case["kv_heads"], case["dim"], case["page"], case["new"]
    past = _lengths(case)
    used = -(-past // p)
    first = np.concatenate([[0], np.cumsum(used)])
    num, most = int(first[-1]) + 7, int(used.max())
    pages = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    state = torch.zeros(n + num + n * most, dtype=torch.int32, device="cuda")
    state[:n] = torch.from_numpy(past.astype(np.int32))
    col = torch.arange(most, device="cuda")[None]
    start, count = (torch.from_numpy(x.astype(np.int64)).cuda()[:, None] for x in (first[:-1], used))
    state[n + num:].view(n, most).copy_(torch.where(col < count, pages[(start + col).clamp(max=num - 1)], -1))
    state[n:n + num][pages[:int(first[-1])].long()] = 1
    # codes of normal values in the units of their block's scale, and scales that make them some 0.5 to 2: every place of a page is alike
    cut = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    pool = torch.empty((num, h, p // 16, 18 * d), dtype=torch.uint8, device="cuda")
    for part in pool.split(max(1, (1 << 26) // pool[0].numel())):
        x = torch.randn((*part.shape, 2), generator=g, device="cuda") * 2.6
        code = torch.bucketize(x.abs(), cut) + 8 * (x < 0)
        part.copy_((code[..., 0] + 16 * code[..., 1]).to(torch.uint8))
        for at in (8 * d, 17 * d):
            part[..., at:at + d] = torch.randint(0x58, 0x66, (*part.shape[:-1], d), generator=g, device="cuda", dtype=torch.uint8)
    scales = [torch.rand(h, generator=g, device="cuda") * 0.01 + 0.005 for _ in range(2)]
    q = torch.randn((n * t, case["heads"], d), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    s = dict(case, pool=pool, state=state, num=num, most=most, k_scale=scales[0], v_scale=scales[1], q=q)
    if own:
        from speculative_decoding_serial_gb300 import kv
        s["cache"] = kv.KvCache(num, p, h, d, n, most, k_scale=scales[0], v_scale=scales[1], pool=pool, state=state)
    return s


# --------------------------------------------------------------------------------------------------- the plain forms

def _logprobs(s):
    out = []
    for x, token in zip(s["logits"].split(256), s["tokens"].split(256)):
        x = x.float()
        z = x / s["temperature"]
        m = z.amax(-1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(-1, keepdim=True)
        lse = m + torch.log(total)
        entropy = torch.log(total) - torch.where(e > 0, e * (z - m), 0.0).sum(-1, keepdim=True) / total
        part = [z.gather(1, token.long()[:, None])[:, 0] - lse[:, 0], entropy[:, 0], lse[:, 0]]
        if s["top"]:  # the largest, the lowest index of those; then without it
            left, index, best = x.clone(), torch.arange(x.shape[1], device=x.device)[None], []
            for _ in range(s["top"]):
                best.append(torch.where(left == left.amax(-1, keepdim=True), index, x.shape[1]).amin(-1, keepdim=True))
                left.scatter_(1, best[-1], -math.inf)
            best = torch.cat(best, 1)
            part += [best.to(torch.int32), z.gather(1, best) - lse]
        out.append(part)
    return [torch.cat(x) for x in zip(*out)]


def _philox(seed, c0, c1, c2, c3):
    """The four words of Philox4x32-10 for counters of int64 tensors that broadcast, as int64."""
    mask = 0xFFFFFFFF
    k0, k1 = seed & mask, (seed >> 32) & mask
    c = [torch.as_tensor(x, device="cuda", dtype=torch.int64) for x in (c0, c1, c2, c3)]
    for r in range(10):
        if r:
            k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & mask) ^ c[1] ^ k0, b & mask, ((a >> 32) & mask) ^ c[3] ^ k1, a & mask]
    return torch.broadcast_tensors(*c)


def _uniform(w):
    return ((w >> 9).double() + 0.5) * 2.0 ** -23


def _stats(x, temperature):
    """Largest value and sum of exponentials (its additions in 64 bits) of every row of x (.., vocab)."""
    m, total = [], []
    for part in x.reshape(-1, x.shape[-1]).split(256):
        z = part.float()
        top = z.amax(-1, keepdim=True)
        m.append(top[:, 0])
        total.append(torch.exp((z - top) / temperature).sum(-1, dtype=torch.float64))
    return torch.cat(m).reshape(x.shape[:-1]).double(), torch.cat(total).reshape(x.shape[:-1])


def _verify(s):
    target, tokens, n, t, vocab, temperature = s["target"], s["tokens"].long(), s["n"], s["gamma"], s["vocab"], s["temperature"]
    column, entry = torch.arange(t, device="cuda")[None], torch.arange(n, device="cuda")
    have = s["drafted"].long() if s["ragged"] else torch.full((n,), t, device="cuda")
    index = torch.arange(vocab, device="cuda")
    if not temperature:
        z = target.float()
        choice = torch.where(z == z.amax(-1, keepdim=True), index, vocab).amin(-1)
        stay = ((tokens == choice[:, :t]) & (column < have[:, None])).long().cumprod(1).sum(1)
        following = choice[entry, stay]
    else:
        m, total = _stats(target, temperature)
        p = torch.exp((target[:, :t].gather(2, tokens[..., None])[..., 0].double() - m[:, :t]) / temperature) / total[:, :t]
        if s["draft"] is not None:
            md, td = _stats(s["draft"], temperature) if t else (m[:, :0], m[:, :0])
            q = torch.exp((s["draft"].gather(2, tokens[..., None])[..., 0].double() - md) / temperature) / td
        else:
            q = torch.ones_like(p)
        u = _uniform(_philox(s["seed"], 0, s["step"] + column, entry[:, None], 2)[0])
        stay = ((u * q < p) & (column < have[:, None])).long().cumprod(1).sum(1)
        # the row after them: what the target has more of than the draft, or all of it where no draft is left
        left = torch.exp((target[entry, stay].double() - m[entry, stay, None]) / temperature) / total[entry, stay, None]
        some = stay < have
        if t:
            at = stay.clamp(max=t - 1)
            if s["draft"] is not None:
                had = torch.exp((s["draft"][entry, at].double() - md[entry, at, None]) / temperature) / td[entry, at, None]
            else:
                had = (index == tokens[entry, at][:, None]).double()
            rest = (left - had).clamp(min=0)
            left = torch.where((some & (rest.amax(-1) > 0))[:, None], rest, left)
        words = _philox(s["seed"], torch.arange((vocab + 3) // 4, device="cuda")[None], s["step"] + stay[:, None], entry[:, None], 1)
        wait = -torch.log(_uniform(torch.stack(words, -1).reshape(n, -1)[:, :vocab]))
        key = left / wait
        following = torch.where(key == key.amax(-1, keepdim=True), index, vocab).amin(-1)
    wide = torch.arange(t + 1, device="cuda")[None]
    said = torch.where(wide < stay[:, None], torch.cat([tokens, tokens.new_zeros(n, 1)], 1), torch.where(wide == stay[:, None], following[:, None], -1))
    return [said.to(torch.int32), (stay + 1).to(torch.int32)]


def _held(x, d):
    """Groups [.., 18 d] of 16 tokens as (keys' codes, keys' scales, values' codes, values' scales) [.., 16, channels or blocks]: their bytes
    in the order of tokens and channels."""
    lead, m = x.shape[:-1], x.dim() - 1
    kc, ks, vc, vs = x.split([8 * d, d, 8 * d, d], -1)
    nib = lambda y: torch.stack([y & 15, y >> 4], -1)  # noqa: E731
    lay = lambda y, shape, order: y.reshape(*lead, *shape).permute(*range(m), *(m + i for i in order)).reshape(*lead, 16, -1)  # noqa: E731
    return (lay(nib(kc), (d // 64, 8, 4, 4, 2, 2, 2), (5, 1, 0, 3, 2, 4, 6)), lay(ks, (8, d // 16, 2), (2, 0, 1)),
            lay(nib(vc), (d // 64, 8, 4, 4, 2, 2, 2), (4, 2, 6, 0, 3, 1, 5)), lay(vs, (4, d // 16, 2, 2), (2, 0, 3, 1)))


def _attend(s):
    n, t, h, d, p, w, first = s["n"], s["new"], s["kv_heads"], s["dim"], s["page"], s["window"], s["sinks"]
    lens, tables = s["state"][:n].long(), s["state"][n + s["num"]:].view(n, s["most"])
    # the groups of 16 tokens that anything is seen of: the first ones, and those from the first query token's window on
    early, late = -(-first // 16), (w + t - 1) // 16 + 2
    group = torch.cat([torch.arange(early, device="cuda")[None].expand(n, -1),
                       (lens - t - w + 1).clamp(min=0)[:, None] // 16 + torch.arange(late, device="cuda")], 1)
    page = tables.gather(1, (group * 16 // p).clamp(max=s["most"] - 1)).long().clamp(min=0)
    x = s["pool"][page, :, group % (p // 16)].transpose(1, 2)                                          # [n, heads, groups, bytes]
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    table = torch.cat([mag, -mag])
    kc, ks, vc, vs = _held(x, d)
    value = lambda c, e, g: (table[c.int()].unflatten(-1, (-1, 16)) * (e.view(torch.float8_e4m3fn).float() * g[:, None, None, None])[..., None]).reshape(n, h, -1, d)  # noqa: E731
    k = value(kc, ks, s["k_scale"])
    q = s["q"].float().reshape(n, t, h, -1, d).permute(0, 2, 3, 1, 4).reshape(n, h, -1, d)             # [n, heads, group * t, dim]
    score = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    j = (group[:, :, None] * 16 + torch.arange(16, device="cuda")).reshape(n, 1, -1)
    head = torch.arange(j.shape[-1], device="cuda") < early * 16
    pos = lens[:, None, None] - t + torch.arange(t, device="cuda")[None, :, None]
    see = (j <= pos) & torch.where(head, j < first, (j >= first) & (j > pos - w))
    # a first token inside the window is seen once, in its place among the first ones
    score = score.reshape(n, h, -1, t, score.shape[-1])
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    o = (score.reshape(n, h, -1, score.shape[-1]) @ value(vc, vs, s["v_scale"])).reshape(n, h, -1, t, d) / total
    return [o.permute(0, 3, 1, 2, 4).reshape(n * t, -1, d).to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(n * t, -1)]


# --------------------------------------------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "attend":
        return list(s["cache"].attend(s["q"], window=s["window"], sinks=s["sinks"])) if own else _attend(s)
    if not own:
        return _logprobs(s) if s["op"] == "logprobs" else _verify(s)
    from speculative_decoding_serial_gb300 import verify
    if s["op"] == "logprobs":
        r = verify.logprobs(s["logits"], s["tokens"], top=s["top"], temperature=s["temperature"])
        return [r.logprob, r.entropy, r.lse] + ([r.top_tokens, r.top_logprobs] if s["top"] else [])
    return list(verify.verify(s["target"], s["tokens"], s["draft"], temperature=s["temperature"], seed=s["seed"], step=s["step"], drafted=s["drafted"]))


# --------------------------------------------------------------------------------------------------- in 64 bits

def _exact_logprobs(s):
    x, k = s["logits"], s["top"]
    out = [torch.empty(s["rows"], dtype=torch.float64, device="cuda") for _ in range(3)]
    out += [torch.empty((s["rows"], k), dtype=torch.int32, device="cuda"), torch.empty((s["rows"], k), dtype=torch.float64, device="cuda")] if k else []
    for i in range(s["rows"]):
        z = x[i].double() / s["temperature"]
        lse = torch.logsumexp(z, 0)
        log_p = z - lse
        out[0][i], out[2][i] = log_p[int(s["tokens"][i])], lse
        out[1][i] = -(log_p.exp() * log_p.clamp(min=-1e4)).sum()
        if k:
            order = torch.sort(x[i].double(), descending=True, stable=True)[1][:k]
            out[3][i], out[4][i] = order, log_p[order]
    return out


def _words64(seed, c0, c1, c2, c3):
    """Philox4x32-10 in numpy, for an array of first words."""
    m32, c = np.uint64(0xFFFFFFFF), np.zeros((4, len(c0)), np.uint64)
    c[0], c[1], c[2], c[3] = c0, c1, c2, c3
    key = [np.uint64(seed & 0xFFFFFFFF), np.uint64((seed >> 32) & 0xFFFFFFFF)]
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = np.stack([(p1 >> np.uint64(32)) ^ c[1] ^ key[0], p1 & m32, (p0 >> np.uint64(32)) ^ c[3] ^ key[1], p0 & m32])
        key = [(key[0] + np.uint64(0x9E3779B9)) & m32, (key[1] + np.uint64(0xBB67AE85)) & m32]
    return ((c >> np.uint64(9)).astype(np.float64) + 0.5) / 2 ** 23


def _exact_verify(s):
    n, t, vocab, temperature, seed = s["n"], s["gamma"], s["vocab"], s["temperature"], s["seed"]
    said = np.full((n, t + 1), -1, np.int32)
    count = np.zeros(n, np.int32)
    tokens = s["tokens"].cpu().numpy()
    have = s["drafted"].cpu().numpy() if s["ragged"] else np.full(n, t)
    first = lambda x: int((x == x.max()).nonzero()[0, 0])  # noqa: E731
    for i in range(n):
        for a in range(t + 1):
            z = s["target"][i, a].double()
            if not temperature:
                choice = first(z)
                if a < have[i] and choice == tokens[i, a]:
                    said[i, a] = choice
                    continue
                break
            p = torch.softmax(z / temperature, 0)
            q = None
            if a < have[i]:
                x = int(tokens[i, a])
                if s["draft"] is None:
                    q = torch.zeros_like(p)
                    q[x] = 1.0
                else:
                    q = torch.softmax(s["draft"][i, a].double() / temperature, 0)
                u = _words64(seed, np.zeros(1), s["step"] + a, i, 2)[0, 0]
                if u * float(q[x]) < float(p[x]):
                    said[i, a] = x
                    continue
                rest = (p - q).clamp(min=0)
                p = rest if float(rest.max()) > 0 else p
            u = _words64(seed, np.arange((vocab + 3) // 4), s["step"] + a, i, 1).T.reshape(-1)[:vocab]
            choice = first(p / torch.from_numpy(-np.log(u)).cuda())
            break
        said[i, a] = choice
        count[i] = a + 1
    return [torch.from_numpy(said).cuda(), torch.from_numpy(count).cuda()]


def _exact_attend(case, s):
    n, t, h, d, p, heads = case["n"], case["new"], case["kv_heads"], case["dim"], case["page"], case["heads"]
    past, tables = _lengths(case), s["state"][n + s["num"]:].view(n, s["most"])
    if work(case)["flops"] > 2e12:
        return None
    # one byte's place worked out from the format's text: r the token in the group, c the channel, b = c / 16, u = c % 16
    r, c = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    b, u, hi, g = c // 16, c % 16, r // 8, r % 8
    place = [(b // 4) * 512 + (4 * g + u // 4) * 16 + (b % 4) * 4 + (u % 4 // 2) * 2 + hi, u % 2, 8 * d + g * (d // 8) + b * 2 + hi,
             9 * d + (b // 4) * 512 + (4 * (u // 2) + g // 2) * 16 + (b % 4) * 4 + hi * 2 + u % 2, r % 2, 17 * d + (g // 2) * (d // 4) + b * 4 + hi * 2 + r % 2]
    place = [torch.from_numpy(x).cuda() for x in place]
    e = np.arange(256)
    e4m3 = torch.from_numpy(np.where((e >> 3) & 15, (1 + (e & 7) / 8) * 2.0 ** (((e >> 3) & 15) - 7), (e & 7) / 512)).cuda()
    e2m1 = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], device="cuda").double() / 2
    o = torch.zeros((n, t, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((n, t, heads), dtype=torch.float64, device="cuda")
    for i, length in enumerate(past.tolist()):
        pos = torch.arange(length - t, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None]
        j = j[:, (j[0] < case["sinks"]) | (j[0] > length - t - case["window"])]
        see = (j <= pos) & ((j < case["sinks"]) | (pos - j < case["window"]))
        for head in range(h):
            x = s["pool"][tables[i, j[0] // p].long(), head, j[0] % p // 16].long()                    # [keys, bytes]
            at = j[0] % 16
            kv = []
            for code, nib, scale, f in ((*place[:3], s["k_scale"]), (*place[3:], s["v_scale"])):
                y = x.gather(1, code[at])
                kv.append(e2m1[torch.where(nib[at] == 1, y >> 4, y & 15)] * e4m3[x.gather(1, scale[at])] * f[head].double())
            for a in range(head * (heads // h), (head + 1) * (heads // h)):
                q = s["q"].reshape(n, t, heads, d)[i, :, a].double()
                z = torch.where(see, q @ kv[0].T / math.sqrt(d), -math.inf)
                lse[i, :, a] = torch.logsumexp(z, -1)
                o[i, :, a] = torch.softmax(z, -1) @ kv[1]
    return [o.reshape(n * t, -1, d), lse.reshape(n * t, -1)]


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_logprobs(s) if case["op"] == "logprobs" else _exact_verify(s)
