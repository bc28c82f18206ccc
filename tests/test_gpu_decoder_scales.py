"""Scores at the ends of fp32's range in the decode attention. Tolerances and cases
are those of the prompt attention's tests, whose weights are rounded to fewer bits."""
import pytest

import gpu_common as gc
from test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


def decode(c):
    import torch
    import awq_int4_moe_gb300 as awq
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    ws, st = torch.zeros(awq.paged_attention_workspace_bytes(c.dim), dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    awq.paged_attention(c.q, c.kc, c.vc, c.table, c.seq, out, ws, st, scale=c.scale, lse=lse, k_scale=c.scales[0], v_scale=c.scales[1])
    torch.cuda.synchronize()
    assert int(st) == 0
    return out, lse


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -132, -2.0 ** -132])
def test_large_products_with_a_small_scale(dim, scale):
    """Products of q and k of 2^126 and its negative: 2^-132 of them is a score of
    1 / 64, none of them the mean of v."""
    c = Case([300, 9, 5000], [1, 1, 1], 4, 2, dim, "bf16", "bf16", seed=dim)
    c.scale = scale
    c.q.zero_()
    c.q[..., 0] = 2.0 ** 63
    c.kc.copy_(c.kc.sign() * 2.0 ** 63)
    c.check(*decode(c))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_queries_and_a_large_scale_over_keys_of_zero(dim):
    """bf16 queries of 2^120 over an e4m3 cache: their power of two times the scale is
    past fp32's range, the scores are 0."""
    c = Case([300, 9], [1, 1], 4, 2, dim, "bf16", "e4m3", seed=dim)
    c.scale = 2.0 ** 30
    c.q.fill_(2.0 ** 120)
    c.kc.copy_(c.kc.float().zero_())
    c.check(*decode(c))
