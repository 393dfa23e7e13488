"""What the cache's binding refuses beyond tests/test_gpu_kv.py."""
import pytest

from test_gpu_kv import make, randn
from test_gpu_kv_sinks import kv, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def test_forward_mode_tangents_are_refused(torch, kv):  # noqa: F811
    from torch.autograd import forward_ad
    c = make(kv, torch, 1, 64, 1, 64, 16)
    k, v, q = (randn(torch, (1, 1, 64), torch.bfloat16, i) for i in range(3))
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(k, torch.ones_like(k))
        for call in (lambda: c.append(dual, v), lambda: c.append(k, dual), lambda: c.attend(dual)):
            with pytest.raises(ValueError, match="gradients"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="gradients"):  # which keeps no tangent back
                call()
        assert c.lens.item() == 0
        c.append(k, v)
    c.attend(q)
    assert c.lens.item() == 1 and c.status() == 0


def test_first_tokens_below_zero_are_refused_without_a_window(torch, kv):  # noqa: F811
    """The library looks at them only with a window; the binding always does."""
    c = make(kv, torch, 1, 64, 1, 64, 16)
    k, v, q = (randn(torch, (1, 1, 64), torch.bfloat16, i) for i in range(3))
    c.append(k, v)
    with pytest.raises(ValueError):
        c.attend(q, sinks=-1)
    assert c.status() == 0
