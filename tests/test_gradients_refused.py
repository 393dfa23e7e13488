"""What the bindings take for a call that is asked for gradients, without a GPU: the refusals come before anything else of a tensor is looked at."""
import pytest

torch = pytest.importorskip("torch")
from torch.autograd import forward_ad  # noqa: E402

from speculative_decoding_serial_gb300 import build, verify  # noqa: E402
from speculative_decoding_serial_gb300 import whead as wh  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


def test_who_asks():
    x, y = torch.zeros(3), torch.zeros(3, requires_grad=True)
    assert not wh.asks_for_gradients(x) and wh.asks_for_gradients(x, y)
    with torch.no_grad():
        assert not wh.asks_for_gradients(x, y)
    with torch.inference_mode():
        assert not wh.asks_for_gradients(x, y)
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x, torch.ones(3))
        assert not wh.asks_for_gradients(x) and wh.asks_for_gradients(d) and wh.asks_for_gradients(x, d) and wh.asks_for_gradients(d[1:])
        with torch.no_grad():
            assert wh.asks_for_gradients(d) and not wh.asks_for_gradients(y)
        assert not wh.asks_for_gradients(forward_ad.unpack_dual(d).primal)
    assert not wh.asks_for_gradients(d)


def test_verification_refuses_them():
    x, tokens = torch.zeros(2, 5, 100), torch.zeros(2, 4, dtype=torch.int32)
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x, torch.ones_like(x))
        for call in (lambda: verify.logprobs(d), lambda: verify.verify(d, tokens)):
            with pytest.raises(ValueError, match="gradients"):
                call()
    with pytest.raises(ValueError, match="gradients"):
        verify.logprobs(x.clone().requires_grad_())
    with pytest.raises(ValueError, match="CUDA"):
        verify.logprobs(x)
