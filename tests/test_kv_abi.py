"""What the 4-bit KV cache's C ABI promises and refuses without a GPU, and the plain model's own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

import kv_reference as R
from speculative_decoding_serial_gb300 import build, kv
from speculative_decoding_serial_gb300 import whead as wh

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned, never read


@pytest.fixture(scope="module")
def L():
    build.build()
    return kv.load()


def declared():
    text = open(os.path.join(ROOT, "include", "whead_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(whead_kv_\w+)\s*\(", text, flags=re.M)))


def test_header_binding_and_library_agree(L):
    assert declared() == sorted(kv.EXPORTS)
    for name in declared():
        assert hasattr(L, name)
    assert wh.strerror(-7).startswith("a KV cache's page pool")


@pytest.mark.parametrize("args,want", [((64, 8, 128), 8 * 4 * 18 * 128), ((16, 1, 64), 18 * 64), ((128, 2, 256), 2 * 8 * 18 * 256),
                                       ((24, 8, 128), wh.ERR_UNSUPPORTED), ((64, 8, 80), wh.ERR_UNSUPPORTED), ((64, 0, 128), wh.ERR_INVALID_ARG)])
def test_page_bytes(L, args, want):
    assert L.whead_kv_page_bytes(*args) == want


def params(**kw):
    p = kv.KvParams(page_size=64, kv_heads=8, head_dim=128, max_seqs=4, max_pages=16, num_pages=64, pool=FAKE, lens=FAKE, refs=FAKE,
                    tables=FAKE, k_scale=FAKE, v_scale=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD = [(dict(page_size=48), wh.ERR_UNSUPPORTED), (dict(head_dim=96), wh.ERR_UNSUPPORTED), (dict(kv_heads=2000), wh.ERR_UNSUPPORTED),
       (dict(max_seqs=5000), wh.ERR_UNSUPPORTED), (dict(max_seqs=0), wh.ERR_INVALID_ARG), (dict(num_pages=0), wh.ERR_INVALID_ARG),
       (dict(max_pages=1 << 26), wh.ERR_UNSUPPORTED), (dict(pool=None), wh.ERR_INVALID_ARG), (dict(pool=FAKE + 8), wh.ERR_INVALID_ARG),
       (dict(workspace=None), wh.ERR_INVALID_ARG), (dict(workspace=FAKE + 16), wh.ERR_INVALID_ARG), (dict(k_scale=None), wh.ERR_INVALID_ARG),
       (dict(lens=FAKE + 2), wh.ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,code", BAD)
def test_a_bad_cache_is_refused_by_every_call(L, kw, code):
    if "max_seqs" in kw and kw["max_seqs"] == 0:
        kw = dict(kw)
    p = ctypes.addressof(keep := params(**kw))
    x = ctypes.c_void_p(FAKE)
    assert L.whead_kv_status(p) == code
    assert L.whead_kv_fork(p, x) == code
    if keep.max_seqs >= 1:
        assert L.whead_kv_append(p, x, x, 0, 1024, 128, 1024, 128, None, None, 1, 4) == code
        assert L.whead_kv_read(p, x, None, 1, 4, 0, x, x) == code
        assert L.whead_kv_compact(p, x, x, x, None, 1, 4) == code
        if keep.kv_heads in (1, 2, 4, 8):
            a = attend_args()
            assert L.whead_kv_attend(p, ctypes.addressof(a)) == code


@pytest.mark.parametrize("page", [16, 64, 128])
def test_longest_slot(L, page):
    """Positions are ints: the keys of a block that begins before a slot's end, and of the two after it, have to stay below 2^31."""
    most = (2 ** 31 - 1024) // page
    for extra, refused in ((0, False), (1, True), (1024 // page - 1, True)):
        p = params(page_size=page, max_seqs=1, max_pages=most + extra)
        assert (L.whead_kv_workspace_bytes(ctypes.addressof(p)) == wh.ERR_UNSUPPORTED) == refused


def attend_args(**kw):
    a = kv.KvAttendArgs(q=FAKE, out=FAKE, lse=FAKE, total=8, q_token_stride=4096, q_head_stride=128, n=2, heads=32, max_q=4, dtype=0,
                        causal=1, scale=0.1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), wh.ERR_INVALID_ARG), (dict(out=FAKE + 8), wh.ERR_INVALID_ARG), (dict(heads=31), wh.ERR_INVALID_ARG),
    (dict(heads=0), wh.ERR_INVALID_ARG), (dict(n=5), wh.ERR_INVALID_ARG), (dict(n=-1), wh.ERR_INVALID_ARG), (dict(total=9), wh.ERR_INVALID_ARG),
    (dict(max_q=3), wh.ERR_INVALID_ARG), (dict(dtype=2), wh.ERR_UNSUPPORTED), (dict(dtype=7), wh.ERR_UNSUPPORTED),
    (dict(window=-1), wh.ERR_INVALID_ARG), (dict(window=3, causal=0), wh.ERR_INVALID_ARG), (dict(scale=float("inf")), wh.ERR_INVALID_ARG),
    (dict(tree=FAKE), wh.ERR_INVALID_ARG), (dict(tree=FAKE, tree_words=1, causal=0), wh.ERR_INVALID_ARG),
    (dict(tree=FAKE + 4, tree_words=1), wh.ERR_INVALID_ARG)])
def test_attend_refuses(L, kw, code):
    p, a = params(), attend_args(**kw)
    assert L.whead_kv_attend(ctypes.addressof(p), ctypes.addressof(a)) == code


def test_attend_refuses_more_items_than_its_scans_hold(L):
    """512 x 4,194,303 row tiles end 513 below 2^31: a scan of 1,024 items a step would step past it. What total rules out is no item."""
    p = params(max_seqs=4096)
    call = lambda **kw: L.whead_kv_attend(ctypes.addressof(p), ctypes.addressof(keep := attend_args(**dict(dict(n=512, heads=8, indptr=FAKE), **kw))))  # noqa: E731
    assert call(total=4194303 * 256, max_q=4194303 * 256) == wh.ERR_UNSUPPORTED
    assert call(total=2 ** 31 - 2, max_q=2 ** 30 - 1) == wh.ERR_UNSUPPORTED


def test_other_calls_refuse(L):
    p, x = params(), ctypes.c_void_p(FAKE)
    q = ctypes.addressof(p)
    assert L.whead_kv_append(q, x, x, 3, 1, 1, 1, 1, None, None, 1, 4) == wh.ERR_INVALID_ARG
    assert L.whead_kv_append(q, None, x, 0, 1, 1, 1, 1, None, None, 1, 4) == wh.ERR_INVALID_ARG
    assert L.whead_kv_append(q, x, x, 0, 1, 1, 1, 1, None, None, 3, 4) == wh.ERR_INVALID_ARG   # 4 tokens on 3 entries
    assert L.whead_kv_append(q, x, x, 0, 1, 1, 1, 1, None, None, 0, 4) == wh.ERR_INVALID_ARG
    assert L.whead_kv_append(q, ctypes.c_void_p(FAKE + 1), x, 0, 1, 1, 1, 1, None, None, 1, 4) == wh.ERR_INVALID_ARG
    assert L.whead_kv_read(q, x, None, 1, 4, 0, ctypes.c_void_p(FAKE + 4), x) == wh.ERR_INVALID_ARG
    assert L.whead_kv_read(q, x, None, 1, -1, 0, x, x) == wh.ERR_INVALID_ARG
    assert L.whead_kv_compact(q, x, x, None, None, 1, 4) == wh.ERR_INVALID_ARG
    assert L.whead_kv_compact(q, x, None, None, None, 1, 4) == wh.ERR_INVALID_ARG
    assert L.whead_kv_compact(q, x, x, x, None, 1, kv.MAX_BLOCK + 1) == wh.ERR_INVALID_ARG
    assert L.whead_kv_fork(q, None) == wh.ERR_INVALID_ARG
    for name in kv.EXPORTS[2:]:
        args = {"whead_kv_append": (x, x, 0, 1, 1, 1, 1, None, None, 1, 4), "whead_kv_read": (x, None, 1, 4, 0, x, x),
                "whead_kv_attend": (x,), "whead_kv_compact": (x, x, x, None, 1, 4), "whead_kv_fork": (x,), "whead_kv_status": ()}[name]
        assert getattr(L, name)(None, *args) == wh.ERR_INVALID_ARG


def test_model_layout_is_a_bijection():
    for d in (64, 128, 256):
        kb, kn, vb, vn, ks, vs = R.byte_maps(d)
        nibbles = np.concatenate([(kb * 2 + kn).ravel(), (vb * 2 + vn).ravel()])
        scales = np.concatenate([ks.ravel(), vs.ravel()])
        every = np.concatenate([nibbles // 2, scales])
        assert len(set(nibbles.tolist())) == nibbles.size and len(set(scales.tolist())) == scales.size
        assert set(every.tolist()) == set(range(18 * d))


def test_model_rounding_pins():
    """e4m3 and e2m1 to nearest even against torch's conversion and the halfway points by hand."""
    torch = pytest.importorskip("torch")
    x = np.concatenate([np.linspace(0, 460, 20001), 2.0 ** np.linspace(-12, 9, 5000)]).astype(np.float32)
    want = torch.from_numpy(np.minimum(x, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(R.nearest(x.astype(np.float64), R._POS, True), want)
    half = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    np.testing.assert_array_equal(R.nearest(half, R.E2M1[:8], True), [0, 2, 2, 4, 4, 6, 6, 7])


@pytest.mark.parametrize("seed", range(4))
def test_model_keeps_its_books(seed):
    """Every page is referenced as often as rows name it; a partial last page has one holder; forks equal their parents."""
    g = np.random.RandomState(seed)
    m = R.Model(40, 16, 5, 12)
    serial = 0
    for _ in range(200):
        op = g.randint(3)
        if op == 0:
            slots = [int(x) for x in g.permutation(5)[:2]]
            tokens = [[(serial := serial + 1) for _ in range(g.randint(0, 40))] for _ in slots]
            want = [m.tokens(s) + t for s, t in zip(slots, tokens)]
            if m.append(tokens, slots):
                assert [m.tokens(s) for s in slots] == want
        elif op == 1:
            s = int(g.randint(5))
            start = int(max(0, m.lens[s] - g.randint(0, 30)))
            was = m.tokens(s)
            keep = [int(x) for x in np.sort(g.permutation(m.lens[s] - start)[:g.randint(0, m.lens[s] - start + 1)])]
            others = [m.tokens(x) for x in range(5) if x != s]
            if m.compact([s], [start], [keep]):
                assert m.tokens(s) == was[:start] + [was[start + x] for x in keep]
            assert others == [m.tokens(x) for x in range(5) if x != s]
        else:
            parents = [int(x) for x in g.randint(-1, 5, 5)]
            was = [m.tokens(s) for s in range(5)]
            if m.fork(parents):
                assert [m.tokens(s) for s in range(5)] == [was[p] if p >= 0 else [] for p in parents]
        count = np.bincount([p for r in m.rows for p in r], minlength=40)
        assert count.tolist() == m.refs
        assert all(m.refs[r[-1]] == 1 for r, n in zip(m.rows, m.lens) if n % 16)
