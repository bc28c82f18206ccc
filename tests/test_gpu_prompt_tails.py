"""What lies behind a sequence's last token in the chunk attention. Cases are those
of the attention's tests."""
import math

import pytest

import gpu_common as gc
from test_gpu_prompt_attention import TYPES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


def shortest(call):
    """The shortest of some calls, in microseconds."""
    import torch
    best = math.inf
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1000)
    return best


@pytest.mark.parametrize("kind,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_what_lies_behind_the_last_token_costs_nothing(kind, cache, dim):
    """Values that no row sees, NaN or not, are not looked for in any row's output: the
    same bits, and no more than twice the time (a look at them takes some thirty
    times as long)."""
    import torch
    import awq_int4_moe_gb300 as awq
    c = Case([5000, 2100, 1533], [1000, 700, 333], 20, 4, dim, kind, cache, 64, seed=dim)
    results, times = [], []
    for bad in (0.0, math.nan):
        for plane in (c.kc, c.vc):
            raw = plane.float()
            for b, n in enumerate(c.lens):
                raw[c.table[b, n // 64].long(), n % 64:] = bad
            plane.copy_(raw.to(plane.dtype))
        results.append(c.call())
        out, st, ws = torch.empty_like(c.q), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(
            awq.prompt_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
        times.append(shortest(lambda: awq.chunk_attention(c.q, c.kc, c.vc, c.table, c.cu_t, c.seq, out, ws, st, scale=c.scale,
                                                          k_scale=c.scales[0], v_scale=c.scales[1])))
    assert results[0][2] == results[1][2] == 0
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert times[1] < 2 * times[0], times
