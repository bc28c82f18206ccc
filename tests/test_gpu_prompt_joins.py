"""The prompt attention's units that are cut between blocks, beside units of which
nothing is seen. Tolerances and cases are those of the attention's tests."""
import math

import pytest

import gpu_common as gc
from test_gpu_prompt_attention import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length,empty,count", [(16000, 2, 12), (5000, 7, 16)])
def test_padded_rows_behind_long_sequences(kind, cache, dim, length, empty, count):
    """Sequences that decode, each with rows of length 0 behind it (a padded batch):
    blocks join a part of a cut unit when the queries of units without keys have
    only just been asked for. Long ones right and the same bits every time, the others
    0 and -infinity."""
    lens = ([length] + [0] * empty) * count
    c = Case(lens, [1] * len(lens), 64, 8, dim, kind, cache, 64, seed=dim)
    first, first_lse, st = c.call()
    assert st == 0
    c.check(first, first_lse)
    for _ in range(20):
        out, lse, st = c.call()
        assert st == 0 and bool((out == first).all()) and bool((lse == first_lse).all())
    none = [i for i, n in enumerate(lens) if n == 0]
    assert bool((first[none] == 0).all()) and bool((first_lse[none] == -math.inf).all())
