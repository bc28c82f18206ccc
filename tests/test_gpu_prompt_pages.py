"""The chunk attention over pages of odd sizes with small heads: tokens are copied
one by one. Tolerances and cases are those of the attention's tests."""
import pytest

import gpu_common as gc
from test_gpu_prompt_attention import CHUNKS, TYPES, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("page", [1, 2, 3, 7, 12, 129])
def test_small_and_odd_pages(kind, cache, dim, page):
    run(*CHUNKS, 8, 2, dim, kind, cache, page, bool(page % 2), seed=page + dim)
    run([3000, 6000, 1], [2, 70, 1], 8, 2, dim, kind, cache, page, seed=page)
