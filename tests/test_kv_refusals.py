"""What the cache's C ABI looks at and what not, without a GPU: calls without entries, which launch nothing."""
import ctypes

import pytest

from speculative_decoding_serial_gb300 import build, kv
from speculative_decoding_serial_gb300 import whead as wh

FAKE = 0x10000  # aligned, never read


@pytest.fixture(scope="module")
def attend():
    build.build()
    L = kv.load()

    def call(**kw):
        p = kv.KvParams(page_size=64, kv_heads=8, head_dim=128, max_seqs=4, max_pages=16, num_pages=64, pool=FAKE, lens=FAKE, refs=FAKE, tables=FAKE,
                        k_scale=FAKE, v_scale=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
        a = kv.KvAttendArgs(q=FAKE, out=FAKE, lse=FAKE, total=0, q_token_stride=4096, q_head_stride=128, n=0, heads=32, max_q=0, causal=1, scale=0.1, **kw)
        return L.whead_kv_attend(ctypes.addressof(p), ctypes.addressof(a))
    return call


def test_first_tokens_count_with_a_window_alone(attend):
    """A caller built before the arguments had `sinks` has anything there: without a window it is not looked at."""
    fine = attend(sinks=0)
    assert fine != wh.ERR_INVALID_ARG
    for sinks in (-1, -2 ** 31, 5, 2 ** 31 - 1):
        assert attend(sinks=sinks) == fine
    assert attend(window=9, sinks=-1) == wh.ERR_INVALID_ARG
    assert attend(window=9, sinks=5) == fine
