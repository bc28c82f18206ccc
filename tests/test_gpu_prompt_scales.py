"""Scores at the ends of fp32's range in the prompt attention. Tolerances and cases
are those of the attention's tests."""
import pytest

import gpu_common as gc
from test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


@pytest.mark.parametrize("cache", [None, "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -132, -2.0 ** -132])
def test_large_products_with_a_small_scale(cache, dim, scale):
    """Products of q and k of 2^126 and its negative: 2^-132 of them is a score of
    1 / 64, none of them the mean of v."""
    c = Case([300, 9, 5000], [300, 9, 5000] if cache is None else [3, 9, 1], 4, 2, dim, "bf16", cache, seed=dim)
    c.scale = scale
    k = c.k if cache is None else c.kc
    c.q.zero_()
    c.q[..., 0] = 2.0 ** 63
    k.copy_(k.sign() * 2.0 ** 63)
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_queries_and_a_large_scale_over_keys_of_zero(dim):
    """bf16 queries of 2^120 over an e4m3 cache: their power of two times the scale is
    past fp32's range, the scores are 0."""
    c = Case([300, 9], [3, 9], 4, 2, dim, "bf16", "e4m3", seed=dim)
    c.scale = 2.0 ** 30
    c.q.fill_(2.0 ** 120)
    c.kc.copy_(c.kc.float().zero_())
    out, lse, st = c.call()
    assert st == 0
    c.check(out, lse)
