"""Forms of the verification's kernels and corners of its values that tests/test_gpu_verify.py does not come to; its bounds and helpers."""
import pytest

from test_gpu_verify import V, case, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab", [(1, 151936), (3, 32003), (150, 5003)])
def test_draws_do_not_depend_on_which_warp_comes_first(torch, V, n, vocab):  # noqa: F811
    """What a warp has found bounds what the others look at, whenever they read it: 100 calls say the same."""
    x, y, tokens = case(torch, n, 2, vocab, torch.bfloat16, torch.float32)
    want = V.verify(x, tokens, y, temperature=1.0, seed=13)
    for _ in range(100):
        got = V.verify(x, tokens, y, temperature=1.0, seed=13)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
