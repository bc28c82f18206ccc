"""The time limit of the prompt attention's wait for the other blocks' parts."""
import time

import pytest

import gpu_common as gc
from test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    gc.require_gpu()
    gc.build_all()


@pytest.mark.parametrize("dim,cache,lens", [(64, "f16", [20000]), (128, "e4m3", [20000, 9000, 12345]), (256, "f16", [9000, 12345, 7000])])
def test_parts_that_never_come(dim, cache, lens):
    """Counters of parts (the workspace's first words, two for each block) that are
    short of some: the blocks that share a unit give up after a second, the call
    says so, and with the workspace zeroed again the next one is right."""
    import torch
    import awq_int4_moe_gb300 as awq
    c = Case(lens, [1] * len(lens), 4, 2, dim, "f16", cache, 64, seed=dim)
    ws = torch.zeros(awq.prompt_attention_workspace_bytes(dim), dtype=torch.uint8, device="cuda")
    assert c.call(workspace=ws)[2] == 0                                 # (loads the kernel)
    ws.view(torch.int32)[0:320:2] = -1000
    torch.cuda.synchronize()
    t0 = time.monotonic()
    assert c.call(workspace=ws)[2] == awq.ERR_DEVICE_TIMEOUT
    assert 0.9 < time.monotonic() - t0 < 6
    ws.zero_()
    for _ in range(2):
        out, lse, st = c.call(workspace=ws)
        assert st == 0
        c.check(out, lse)
    assert not bool(ws.view(torch.int32)[:320].any())
