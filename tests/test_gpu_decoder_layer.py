"""The decoder layer of examples/decoder_layer.py: the calls together, as a
user's program makes them, against 64-bit results.

Tolerance of the attention half. Its only coarse roundings are the two e4m3
quantisations of activations (a 64-bit form of the same layer with the same
8-bit weights has none): at most 2^-4 relative per element, uniform, so 0.036
in the 2-norm at most each; a product passes the relative 2-norm on, the
softmax averages it and shifts weights by less than as much again. Three such
terms stay below 0.11 of the output's 2-norm. The expert half is compared bit
for bit with the same calls made one by one."""
import importlib.util
import os

import pytest

import gpu_common as gc

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    gc.require_gpu()
    gc.build_all()
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def weight64(q, s):
    n, k = q.shape
    return q.float().double() * s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


class Reference:
    """The attention half in 64 bits, its own keys and values kept."""

    def __init__(self, layer):
        self.l = layer
        self.k, self.v = [], []

    def step(self, x, residual):
        import torch
        l = self.l
        r = x.double() + residual.double()
        h = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * l.norm1.double()
        qkv = (h @ weight64(l.qkv_w, l.qkv_s).t()).view(l.batch, -1, l.dim)
        row = l.cos_sin[len(self.k)].double()
        half = l.dim // 2

        def turn(t):
            a, b = t[..., :half], t[..., half:]
            return torch.cat([a * row[:half] - b * row[half:], b * row[:half] + a * row[half:]], 2)

        qh, kh = l.q_heads, l.kv_heads
        q = turn(qkv[:, :qh])
        self.k.append(turn(qkv[:, qh:qh + kh]))
        self.v.append(qkv[:, qh + kh:])
        k, v = torch.stack(self.k, 1), torch.stack(self.v, 1)
        g = qh // kh
        s = torch.einsum("bhgd,bnhd->bhgn", q.view(l.batch, kh, g, l.dim), k) * l.dim ** -0.5
        o = torch.einsum("bhgn,bnhd->bhgd", s.softmax(3), v).reshape(l.batch, qh * l.dim)
        return r, o @ weight64(l.o_w, l.o_s).t()


@pytest.mark.parametrize("batch", [1, 5])
def test_layer_against_64_bits(example, batch):
    import torch
    import awq_int4_moe_gb300 as awq
    layer = example.DecoderLayer(batch, 64, seed=batch)
    ref = Reference(layer)
    layer.x.normal_()
    for step in range(20):
        x, residual = layer.x.clone(), layer.residual.clone()
        layer.attention_half()
        torch.cuda.synchronize()
        r, o = ref.step(x, residual)
        assert bool(((layer.residual.double() - r).abs() <= r.abs() * 2.0 ** -11 + 2.0 ** -25).all())
        far = float((layer.o.double() - o).norm() / o.norm())
        assert far < 0.11, (step, far)
        mid = layer.residual.clone()
        layer.expert_half()
        # the same calls, one by one
        h, res = torch.empty_like(layer.h), torch.empty_like(layer.h)
        awq.add_rmsnorm(layer.o, layer.norm2, 1e-6, residual=mid, residual_out=res, out=h)
        ids, w = torch.empty_like(layer.ids), torch.empty_like(layer.weights)
        awq.moe_router_topk(h.float() @ layer.router.t(), batch, layer.shape, ids, w)
        torch.cuda.synchronize()
        assert bool((h == layer.h).all()) and bool((res == layer.residual).all()) and bool((ids == layer.ids).all())
        assert bool(layer.x.isfinite().all()) and int(layer.status) == 0
        layer.x.mul_(8.0 / layer.x.float().norm(dim=1, keepdim=True).clamp(min=1e-3)).clamp_(-50, 50)   # random experts: keep the scale
    assert layer.seq_lens.tolist() == [20] * batch


def test_graph_replay_matches_eager_steps(example):
    import torch
    outs = []
    for graphed in (False, True):
        layer = example.DecoderLayer(4, 40, seed=3)
        g = torch.Generator(device="cuda")
        g.manual_seed(9)
        layer.x.normal_(generator=g)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.step()
        torch.cuda.current_stream().wait_stream(side)
        if graphed:
            keep = [t.clone() for t in (layer.x, layer.residual, layer.seq_lens)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                layer.step()
            for t, k in zip((layer.x, layer.residual, layer.seq_lens), keep):
                t.copy_(k)
        for _ in range(10):
            graph.replay() if graphed else layer.step()
        torch.cuda.synchronize()
        assert int(layer.status) == 0
        outs.append((layer.x.clone(), layer.residual.clone(), layer.seq_lens.clone()))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("batch", [1, 5])
def test_expert_half_against_the_calls_one_by_one_and_the_oracle(example, batch, oracle_lib):
    """The routing weights and the stage's output bit for bit, and the output
    within the stage's tolerance of the oracle's."""
    import numpy as np
    import synth
    import torch
    import awq_int4_moe_gb300 as awq
    layer = example.DecoderLayer(batch, 8, seed=20 + batch)
    layer.x.normal_()
    layer.attention_half()
    before, o = layer.residual.clone(), layer.o.clone()
    layer.expert_half()
    h, res = torch.empty_like(layer.h), torch.empty_like(layer.h)
    awq.add_rmsnorm(o, layer.norm2, 1e-6, residual=before, residual_out=res, out=h)
    logits = h.float() @ layer.router.t()
    ids, w = torch.empty_like(layer.ids), torch.empty_like(layer.weights)
    awq.moe_router_topk(logits, batch, layer.shape, ids, w)
    out, status = torch.empty_like(layer.x), torch.zeros_like(layer.status)
    ws = torch.zeros_like(layer.moe_ws)
    awq.moe_layer(h, ids, w, batch, layer.shape, layer.experts, out, ws, layer.moe_ws_bytes, status)
    torch.cuda.synchronize()
    assert int(status) == 0 and int(layer.status) == 0
    assert torch.equal(h, layer.h) and torch.equal(res, layer.residual)
    assert torch.equal(ids, layer.ids) and torch.equal(w, layer.weights)
    assert torch.equal(out, layer.x)
    expert = synth.ExpertShape(num_experts=512, top_k=10, hidden=2560, inter=160, meta_bytes=4)
    ref, _ = oracle_lib.layer_from_synth(expert, 20 + batch, 0, h.cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy())
    err = np.abs(layer.x.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= gc.ATOL + gc.RTOL * np.abs(ref)), float(err.max())
