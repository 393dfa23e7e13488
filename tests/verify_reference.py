"""A plain model of the verification of drafts in numpy, in 64 bits, written from include/whead_verify.h."""
import numpy as np

LOG2E = 1.4426950408889634


def philox(seed, c0, c1, c2, c3):
    """Philox4x32-10's four words for counters that broadcast."""
    c0, c1, c2, c3 = np.broadcast_arrays(*(np.asarray(x, np.uint64) for x in (c0, c1, c2, c3)))
    m = np.uint64(0xFFFFFFFF)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        a, b = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        c0, c1, c2, c3 = (b >> np.uint64(32)) ^ c1 ^ np.uint64(k0), b & m, (a >> np.uint64(32)) ^ c3 ^ np.uint64(k1), a & m
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c0, c1, c2, c3


def uniform(w):
    return ((w >> np.uint64(9)).astype(np.float64) + 0.5) * 2.0 ** -23


def distribution(x, temperature):
    """Probabilities of a row, or None where it has none."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
        return None
    z = (x - x.max()) / temperature
    e = np.exp(z)
    return e / e.sum()


def logprobs(x, temperature, top):
    """A row's lse, entropy, log probabilities, and the alternatives' tokens (-1 past the last)."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (x == np.inf).any():
        return np.nan, np.nan, np.full(x.shape, np.nan), np.full(top, -1)
    if (x == -np.inf).all():
        return -np.inf, 0.0, np.full(x.shape, -np.inf), np.full(top, -1)
    d = (x - x.max()) / temperature
    e = np.exp(d)
    log_s = np.log(e.sum())
    p = e / e.sum()
    entropy = log_s - (p[e > 0] * d[e > 0]).sum()
    order = np.argsort(-x, kind="stable")[:top]
    order = order[x[order] > -np.inf]
    return x.max() / temperature + log_s, entropy, d - log_s, np.concatenate([order, np.full(top - len(order), -1)]).astype(np.int64)


def verify(target, tokens, draft, temperature, draft_temperature, seed, step, i, have):
    """One entry, target (gamma + 1, V), draft (gamma, V) or None: (said, count, margin). margin: how near the nearest of its decisions
    was, relative to the larger side."""
    gamma, V = target.shape[0] - 1, target.shape[1]
    said, margin = np.full(gamma + 1, -1, np.int64), np.inf
    have = min(max(have, 0), gamma)
    for a in range(gamma + 1):
        p = distribution(target[a], temperature or 1.0)
        following = -1
        if p is not None:
            if temperature == 0:
                following = int(np.argmax(np.asarray(target[a], np.float64)))
                if a < have and following == tokens[a]:
                    said[a] = following
                    continue
            else:
                w = p
                if a < have:
                    x, q = int(tokens[a]), None
                    if draft is not None:
                        q = distribution(draft[a], draft_temperature)
                    else:
                        q = np.zeros(V)
                        if 0 <= x < V:
                            q[x] = 1.0
                    if q is not None and 0 <= x < V:
                        u = float(uniform(philox(seed, 0, step + a, i, 2)[0]))
                        big = max(u * q[x], p[x])
                        margin = min(margin, abs(u * q[x] - p[x]) / big if big > 0 else np.inf)
                        if u * q[x] < p[x]:
                            said[a] = x
                            continue
                    if q is not None and (p > q).any():
                        w = np.maximum(p - q, 0)
                u = uniform(np.stack(philox(seed, np.arange((V + 3) // 4), step + a, i, 1), 1).reshape(-1)[:V])
                key = w / -np.log(u)
                following = int(np.argmax(key))
                rest = np.delete(key, following)
                if len(rest):
                    # p - q is off by what p and q are off by
                    second = int(np.argmax(rest)) if rest.max() > 0 else 0
                    second += second >= following
                    loss = max(p[j] / w[j] if w[j] > 0 else 1.0 for j in (following, second))
                    margin = min(margin, (key[following] - rest.max()) / key[following] / loss)
        said[a] = following
        return said, a + 1, margin
