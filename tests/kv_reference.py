"""A plain model of the 4-bit paged KV cache in numpy: the format's bytes, the quantization, the bookkeeping of pages, and
attention in 64 bits. Written from include/whead_kv.h, one token and one byte at a time."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)
    v = np.where(b & 127 == 127, np.nan, v)
    return np.where(b & 128, -v, v)


E4M3 = e4m3_values()
_POS = E4M3[:127]  # ascending, 0 .. 448


def nearest(v, table, even):
    """Index of the table's value nearest to v >= 0 (ascending table); a tie goes to the even index; past the end: the last."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = v - table[lo], table[hi] - v
    return np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(lo % 2 == 0, lo, hi))) if even else np.where(dh < dl, hi, lo)


def quantize(x, g):
    """(codes, scale bytes) of x [..., dim] (any float type, exact in fp32) with the head's scale g (fp32 scalar)."""
    x = np.asarray(x, np.float32)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        amax = np.nanmax(np.where(np.isnan(b), 0, np.abs(b)), -1).astype(np.float32)
        r = (amax / (np.float32(6) * g)).astype(np.float32)
        s = nearest(np.minimum(r.astype(np.float64), 1e30), _POS, True)
        inv = (np.float32(1) / (E4M3[s].astype(np.float32) * g)).astype(np.float32)
        y = (b * inv[..., None]).astype(np.float32)
    y = np.where(np.isnan(y), np.float32(0), y)
    code = nearest(np.minimum(np.abs(y.astype(np.float64)), 1e30), E2M1[:8], True)
    code = code + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def dequantize(code, scale, g):
    s = E4M3[scale].astype(np.float32) * np.float32(g)
    return (E2M1[code].astype(np.float32).reshape(*scale.shape, 16) * s[..., None]).reshape(code.shape)


def byte_maps(d):
    """Places in a group of 16 tokens: keys' code bytes and nibbles [16, d], values' likewise, scales' bytes [16, d / 16]."""
    kb, kn, vb, vn = (np.zeros((16, d), np.int64) for _ in range(4))
    ks, vs = (np.zeros((16, d // 16), np.int64) for _ in range(2))
    for r in range(16):
        g, hi = r % 8, r // 8
        for c in range(d):
            b, u = c // 16, c % 16
            kb[r, c] = (b // 4) * 512 + (4 * g + u // 4) * 16 + (b % 4) * 4 + (u % 4 // 2) * 2 + hi
            kn[r, c] = u % 2
            vb[r, c] = 9 * d + (b // 4) * 512 + (4 * (u // 2) + (r % 8) // 2) * 16 + (b % 4) * 4 + hi * 2 + u % 2
            vn[r, c] = r % 2
        for b in range(d // 16):
            ks[r, b] = 8 * d + g * (d // 8) + b * 2 + hi
            vs[r, b] = 17 * d + ((r % 8) // 2) * (d // 4) + b * 4 + hi * 2 + r % 2
    return kb, kn, vb, vn, ks, vs


def unpack(group, d):
    """One group's bytes [18 d] as (key codes [16, d], key scales [16, d / 16], value codes, value scales)."""
    kb, kn, vb, vn, ks, vs = byte_maps(d)
    nib = lambda b, n: (group[b] >> (4 * n)) & 15  # noqa: E731
    return nib(kb, kn), group[ks], nib(vb, vn), group[vs]


class Model:
    """The cache's bookkeeping, with each held token's (k, v) values as python objects."""

    def __init__(self, num_pages, page, max_seqs, max_pages):
        self.page, self.max_pages = page, max_pages
        self.refs = [0] * num_pages
        self.rows = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.held = {}  # (page, place) -> token

    def _take(self, need):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        return free[:need] if len(free) >= need else None

    def _pages(self, n):
        return -(-n // self.page)

    def tokens(self, s):
        return [self.held[self.rows[s][p // self.page], p % self.page] for p in range(self.lens[s])]

    def append(self, tokens, slots):
        need = sum(self._pages(self.lens[s] + len(t)) - len(self.rows[s]) for s, t in zip(slots, tokens))
        if any(self._pages(self.lens[s] + len(t)) > self.max_pages for s, t in zip(slots, tokens)):
            return False
        fresh = self._take(need)
        if fresh is None:
            return False
        for s, t in zip(slots, tokens):
            while len(self.rows[s]) < self._pages(self.lens[s] + len(t)):
                p = fresh.pop(0)
                self.refs[p] = 1
                self.rows[s].append(p)
            for x in t:
                self.held[self.rows[s][self.lens[s] // self.page], self.lens[s] % self.page] = x
                self.lens[s] += 1
        return True

    def compact(self, slots, start, keep):
        plans = []
        for s, a, k in zip(slots, start, keep):
            stay = sum(1 for j, x in enumerate(k) if j == x)
            written = range((a + stay) // self.page, self._pages(a + len(k)))
            plans.append([p for p in written if self.refs[self.rows[s][p]] > 1])
        fresh = self._take(sum(map(len, plans)))
        if fresh is None:
            return False
        old = [self.tokens(s) for s in slots]
        for s, a, k, shared, was in zip(slots, start, keep, plans, old):
            for p in shared:
                new = fresh.pop(0)
                self.refs[self.rows[s][p]] -= 1
                self.refs[new] = 1
                for place in range(self.page):
                    if (self.rows[s][p], place) in self.held:
                        self.held[new, place] = self.held[self.rows[s][p], place]
                self.rows[s][p] = new
            for p in self.rows[s][self._pages(a + len(k)):]:
                self.refs[p] -= 1
            self.rows[s] = self.rows[s][:self._pages(a + len(k))]
            self.lens[s] = a + len(k)
            for j, x in enumerate(k):
                if j != x:
                    self.held[self.rows[s][(a + j) // self.page], (a + j) % self.page] = was[a + x]
        return True

    def fork(self, parents):
        take = [i for i, p in enumerate(parents) if p >= 0 and p != i]
        need = [i for i in take if self.lens[parents[i]] % self.page]
        fresh = self._take(len(need))
        if fresh is None:
            return False
        rows, lens = [list(r) for r in self.rows], list(self.lens)
        for i, p in enumerate(parents):
            if p == i:
                continue
            for q in self.rows[i]:
                self.refs[q] -= 1
            rows[i], lens[i] = ([], 0) if p < 0 else (list(self.rows[p]), self.lens[p])
            if i in need:
                new = fresh.pop(0)
                for place in range(self.page):
                    if (rows[i][-1], place) in self.held:
                        self.held[new, place] = self.held[rows[i][-1], place]
                rows[i][-1] = new
            for q in rows[i]:
                self.refs[q] += 1
        self.rows, self.lens = rows, lens
        return True

    def state(self):
        table = [r + [-1] * (self.max_pages - len(r)) for r in self.rows]
        return np.array(self.lens + self.refs + [x for r in table for x in r], np.int32)


def visible(length, tokens, t, causal, window, bits):
    """Which of a slot's keys query token t of `tokens` sees."""
    j = np.arange(length)
    pos = length - tokens + t
    see = np.ones(length, bool)
    if causal:
        see &= j <= pos
    if window:
        see &= j > pos - window
    if bits is not None:
        for u in range(tokens):
            if 0 <= length - tokens + u < length and not (int(bits[u // 64]) >> (u % 64)) & 1:
                see[length - tokens + u] = False
    return see


def attend(q, k, v, scale, see):
    """Outputs, log sums and the bound's parts for one query row: q [d], k and v [L, d], see [L]."""
    if not see.any():
        return np.zeros(k.shape[1]), -np.inf, 0.0, np.zeros(k.shape[1])
    s = k[see] @ q * scale
    m = s.max()
    p = np.exp(s - m)
    total = p.sum()
    spread = np.abs(k[see]) @ np.abs(q) * abs(scale)
    return p @ v[see] / total, m + np.log(total), spread.max(), p @ np.abs(v[see]) / total
