"""The limits of the prompt attention's sizes as its header states them, without a
GPU: a size within them gets as far as the check of the workspace."""
import pytest

from test_decoder_boundary import rope
from test_prompt_boundary import OK, SHAPE, SMALL, chunk, norm, prompt
import test_prompt_boundary as tb


@pytest.fixture(scope="module", autouse=True)
def _built():
    import awq_int4_moe_gb300.build as b
    b.build()


def within(tokens, group, kv_heads, batch, longest):
    """The header's limits."""
    u = group * (longest + tokens + 640) + 512
    return tokens * group <= 2 ** 31 - 256 and u * (longest // 128 + 1) <= 4 * 10 ** 18 and \
        u * (tokens * group / 120 + 1) * kv_heads * batch <= 4 * 10 ** 18


@pytest.mark.parametrize("group", [1, 8, 43, 65, 86, 100, 129, 300])
@pytest.mark.parametrize("dim", [64, 136])
def test_sizes_within_the_limits_are_taken(group, dim):
    """The largest batch that the header allows, with units of as few as 65 rows (65
    heads of one, of more than 128 elements)."""
    tokens = (2 ** 31 - 256) // group
    u = group * (2 * tokens + 640) + 512
    batch = int(4 * 10 ** 18 / (u * (tokens * group / 120 + 1)))
    assert within(tokens, group, 1, batch, tokens)
    over = dict(tokens=tokens, batch=batch, q_heads=group, kv_heads=1, dim=dim, ws_bytes=1000)
    assert prompt(**over) == SMALL
    assert prompt(**{**over, "batch": 8 * batch}) == SHAPE
    assert prompt(**{**over, "tokens": (2 ** 31 - 256) // group + 1}) == SHAPE


def test_sizes_within_the_limits_of_a_cache_are_taken():
    # 8 heads of one, 2^20 new tokens in all, pages of 16
    tokens, group, pages = 1 << 20, 8, 1 << 22
    u = group * (pages * 16 + tokens + 640) + 512
    batch = int(4 * 10 ** 18 / (u * (tokens * group / 120 + 1) * 2))
    assert within(tokens, group, 2, batch, pages * 16)
    over = dict(tokens=tokens, batch=batch, q_heads=16, pages=pages, stride=pages, cache=tb.cache(heads=2), ws_bytes=1000)
    assert chunk(**over) == SMALL
    assert chunk(**{**over, "batch": 8 * batch}) == SHAPE


@pytest.mark.parametrize("append", [norm, rope])
def test_rows_of_a_token_that_32_bits_do_not_count(append):
    most = 2 ** 31 - 2048 - 2 * 2
    assert append(q_heads=most + 1) == SHAPE
    assert append(q_heads=2 ** 31 - 1) == SHAPE
    assert append(q_heads=8, cache=tb.cache(heads=2 ** 30)) == SHAPE
    assert append(q_heads=most, tokens=0) == OK
