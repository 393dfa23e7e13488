"""What the verification's C ABI promises and refuses without a GPU, what its binding refuses, and the plain model's own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

import verify_reference as R
from oracle import oracle as O
from speculative_decoding_serial_gb300 import build, verify
from speculative_decoding_serial_gb300 import whead as wh

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned, never read


@pytest.fixture(scope="module")
def L():
    build.build()
    return verify.load()


def test_header_binding_and_library_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "whead_verify.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(whead_\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(verify.EXPORTS)
    for name in declared:
        assert hasattr(L, name)
    assert f"WHEAD_MAX_TOP {verify.MAX_TOP}\n" in text and f"WHEAD_MAX_DRAFTS {verify.MAX_DRAFTS}\n" in text


def logprobs_args(**kw):
    a = verify.LogprobsArgs(logits=FAKE, tokens=FAKE, logprob=FAKE, entropy=FAKE, lse=FAKE, top_tokens=FAKE, top_logprobs=FAKE, stride_n=100, stride_t=0,
                            n=2, t=1, V=100, temperature=1.0, dtype=0, top=5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), wh.ERR_INVALID_ARG), (dict(logits=FAKE + 1), wh.ERR_INVALID_ARG), (dict(logits=FAKE + 2, dtype=2), wh.ERR_INVALID_ARG),
    (dict(n=-1), wh.ERR_INVALID_ARG), (dict(t=-1), wh.ERR_INVALID_ARG), (dict(V=0), wh.ERR_INVALID_ARG), (dict(dtype=3), wh.ERR_INVALID_ARG),
    (dict(dtype=-1), wh.ERR_INVALID_ARG), (dict(top=-1), wh.ERR_INVALID_ARG), (dict(top=33), wh.ERR_UNSUPPORTED), (dict(V=1 << 24), wh.ERR_UNSUPPORTED),
    (dict(n=1 << 27), wh.ERR_UNSUPPORTED), (dict(n=1 << 14, t=1 << 13), wh.ERR_UNSUPPORTED), (dict(n=1 << 62, t=1 << 62), wh.ERR_UNSUPPORTED),
    (dict(temperature=0.0), wh.ERR_INVALID_ARG), (dict(temperature=-1.0), wh.ERR_INVALID_ARG), (dict(temperature=float("nan")), wh.ERR_INVALID_ARG),
    (dict(temperature=float("inf")), wh.ERR_INVALID_ARG), (dict(temperature=1e-39), wh.ERR_INVALID_ARG), (dict(temperature=1e39), wh.ERR_INVALID_ARG),
    (dict(tokens=None), wh.ERR_INVALID_ARG), (dict(logprob=None), wh.ERR_INVALID_ARG), (dict(tokens=FAKE + 2), wh.ERR_INVALID_ARG),
    (dict(entropy=FAKE + 2), wh.ERR_INVALID_ARG), (dict(lse=FAKE + 1), wh.ERR_INVALID_ARG), (dict(top_tokens=None), wh.ERR_INVALID_ARG),
    (dict(top_logprobs=None), wh.ERR_INVALID_ARG), (dict(top_logprobs=FAKE + 2), wh.ERR_INVALID_ARG)])
def test_logprobs_refuses(L, kw, code):
    assert L.whead_logprobs(ctypes.addressof(keep := logprobs_args(**kw))) == code
    assert keep is not None


def test_first_tokens_below_zero_are_refused(L):
    """sinks of the cache's attention (whead_kv.h)."""
    from speculative_decoding_serial_gb300 import kv
    K = kv.load()
    p = kv.KvParams(page_size=64, kv_heads=8, head_dim=128, max_seqs=4, max_pages=16, num_pages=64, pool=FAKE, lens=FAKE, refs=FAKE, tables=FAKE,
                    k_scale=FAKE, v_scale=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    a = kv.KvAttendArgs(q=FAKE, out=FAKE, lse=FAKE, total=8, q_token_stride=4096, q_head_stride=128, n=2, heads=32, max_q=4, causal=1, window=9, scale=0.1,
                        sinks=-1)
    assert K.whead_kv_attend(ctypes.addressof(p), ctypes.addressof(a)) == wh.ERR_INVALID_ARG


def test_no_rows_are_no_work(L):
    assert L.whead_logprobs(None) == wh.ERR_INVALID_ARG
    assert L.whead_verify(None) == wh.ERR_INVALID_ARG
    for kw in (dict(n=0), dict(t=0)):
        assert L.whead_logprobs(ctypes.addressof(keep := logprobs_args(logits=None, **kw))) == wh.OK
    assert L.whead_verify(ctypes.addressof(keep := verify_args(n=0, target=None))) == wh.OK
    assert keep is not None


def verify_args(**kw):
    a = verify.VerifyArgs(target=FAKE, draft=FAKE, tokens=FAKE, said=FAKE, count=FAKE, target_stride_n=500, target_stride_t=100, draft_stride_n=400,
                          draft_stride_t=100, n=2, V=100, gamma=4, temperature=1.0, draft_temperature=1.0, workspace=FAKE, workspace_bytes=1 << 20)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(target=None), wh.ERR_INVALID_ARG), (dict(target=FAKE + 1), wh.ERR_INVALID_ARG), (dict(target=FAKE + 2, target_dtype=2), wh.ERR_INVALID_ARG),
    (dict(draft=FAKE + 1), wh.ERR_INVALID_ARG), (dict(draft_dtype=5), wh.ERR_INVALID_ARG), (dict(target_dtype=3), wh.ERR_INVALID_ARG),
    (dict(tokens=None), wh.ERR_INVALID_ARG), (dict(tokens=FAKE + 1), wh.ERR_INVALID_ARG), (dict(drafted=FAKE + 2), wh.ERR_INVALID_ARG),
    (dict(said=None), wh.ERR_INVALID_ARG), (dict(count=None), wh.ERR_INVALID_ARG), (dict(n=-1), wh.ERR_INVALID_ARG), (dict(gamma=-1), wh.ERR_INVALID_ARG),
    (dict(gamma=256), wh.ERR_UNSUPPORTED), (dict(n=1 << 27), wh.ERR_UNSUPPORTED), (dict(V=0), wh.ERR_INVALID_ARG), (dict(V=1 << 24), wh.ERR_UNSUPPORTED),
    (dict(temperature=-0.5), wh.ERR_INVALID_ARG), (dict(temperature=float("nan")), wh.ERR_INVALID_ARG), (dict(temperature=float("inf")), wh.ERR_INVALID_ARG),
    (dict(draft_temperature=0.0), wh.ERR_INVALID_ARG), (dict(draft_temperature=float("nan")), wh.ERR_INVALID_ARG), (dict(workspace=None), wh.ERR_INVALID_ARG),
    (dict(workspace=FAKE + 8), wh.ERR_INVALID_ARG), (dict(workspace_bytes=100), wh.ERR_INVALID_ARG)])
def test_verify_refuses(L, kw, code):
    assert L.whead_verify(ctypes.addressof(keep := verify_args(**kw))) == code
    assert keep is not None


def test_workspace(L):
    assert L.whead_verify_workspace_bytes(-1, 4) == wh.ERR_INVALID_ARG
    assert L.whead_verify_workspace_bytes(1, -1) == wh.ERR_INVALID_ARG
    assert L.whead_verify_workspace_bytes(1, 256) == wh.ERR_UNSUPPORTED
    assert L.whead_verify_workspace_bytes(1 << 40, 0) == wh.ERR_UNSUPPORTED
    assert L.whead_verify_workspace_bytes(0, 0) >= 0
    assert L.whead_verify_workspace_bytes(3, 16) >= 3 * 33 * 8


def test_binding_refuses_without_a_gpu(L):
    """CPU tensors, wrong types, shapes and strides are refused before anything is called."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 5, 100)
    i = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        verify.logprobs(x)
    with pytest.raises(ValueError):
        verify.logprobs(x.transpose(1, 2))
    with pytest.raises(ValueError):
        verify.logprobs(x[0, 0])
    with pytest.raises(TypeError):
        verify.logprobs(x.double())
    with pytest.raises(ValueError):
        verify.verify(x, i)
    with pytest.raises(ValueError):
        verify.verify(x[0], i)


def test_model_draws_as_the_oracle_does():
    """The model's Philox and uniforms against the oracle's own."""
    O.build()
    seed = 0x0123456789ABCDEF
    for ctr in ((0, 0, 0, 2), (37983, 15, 3, 1), (0xFFFFFFFF, 0xFFFFFFFF, 0xFFFFFFFF, 1)):
        words = [int(x) for x in R.philox(seed, *ctr)]
        assert words == O.philox4x32_10(ctr, (seed & 0xFFFFFFFF, seed >> 32))
        assert [float(R.uniform(np.uint64(w))) for w in words] == [O.uniform(w) for w in words]


def test_model_logprobs_by_hand():
    lse, entropy, lp, top = R.logprobs([0.0, np.log(3.0), -np.inf, 0.0], 1.0, 5)
    assert np.allclose([lse, entropy], [np.log(5), np.log(5) - 0.6 * np.log(3)])
    assert np.allclose(lp[[0, 1, 3]], np.log([0.2, 0.6, 0.2])) and lp[2] == -np.inf
    assert top.tolist() == [1, 0, 3, -1, -1]


def test_model_says_what_the_target_would():
    """Tokens said by drawing, checking and drawing again are distributed as the target's own (4 tokens, 40,000 entries, one draft)."""
    p, q = np.array([0.5, 0.3, 0.15, 0.05]), np.array([0.1, 0.2, 0.3, 0.4])
    g = np.random.RandomState(0)
    n, seed = 40000, 99
    draft = g.choice(4, n, p=q)
    u = R.uniform(R.philox(seed, 0, 7, np.arange(n), 2)[0])
    stay = u * q[draft] < p[draft]
    words = np.stack(R.philox(seed, 0, 7, np.arange(n), 1), 1)
    drawn = np.argmax(np.maximum(p - q, 0) / -np.log(R.uniform(words)), 1)
    said = np.where(stay, draft, drawn)
    share = np.bincount(said, minlength=4) / n
    assert np.abs(share - p).max() < 5 * np.sqrt(0.25 / n)
    for i in range(50):  # and the model's own function says the same, entry by entry
        s, count, _ = R.verify(np.log(np.stack([p, p])), [draft[i]], np.log(q[None]), 1.0, 1.0, seed, 7, i, 1)
        assert s[0] == said[i] and count == 1 + stay[i]
