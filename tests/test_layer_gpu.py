"""block_norm, lora_linear and moe_route as a program runs them, with the linears,
the cache and the experts: one decoder layer of a step of several requests, each
with its adapter, and its mixture of experts.  Every stage is checked against its
64-bit form on the very inputs it had, eagerly and as one graph replayed on other
inputs."""
import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
import oracle
from tests import layer_util as lu
from tests.gpu_util import host_codes, host_values, need_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
H, HQ, HKV, D, P = 256, 4, 2, 64, 16
ROWS, SEQS, E, TOPK, INTER, ADAPTERS, RANK = 9, 4, 8, 2, 128, 3, 16
QKV = (HQ + 2 * HKV) * D


class Layer:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g = g
        rnd = lambda *s, k=1.0: (k * torch.randn(*s, generator=g, device="cuda")).to(BF)
        self.rnd = rnd
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.h, self.residual = rnd(ROWS, H), torch.zeros(ROWS, H, device="cuda")
        self.norms = [1 + rnd(H, k=0.1) for _ in range(4)]
        self.w_qkv, self.w_o = rnd(QKV, H, k=0.06), rnd(H, HQ * D, k=0.06)
        self.w_router = rnd(E, H, k=0.1)
        self.bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        self.lora_qkv = sg.make_lora(
            [rnd(ADAPTERS, RANK, H, k=0.06), None, rnd(ADAPTERS, RANK, H, k=0.06)],
            [rnd(ADAPTERS, HQ * D, RANK, k=0.2), HKV * D, rnd(ADAPTERS, HKV * D, RANK, k=0.2)])
        self.ranks, self.scale = i32(RANK, 5, 8), torch.rand(ADAPTERS, generator=g, device="cuda")
        self.lora_o = sg.make_lora(rnd(ADAPTERS, RANK, HQ * D, k=0.06), rnd(ADAPTERS, H, RANK, k=0.2),
                                   scale=self.scale, ranks=self.ranks)
        self.ids = i32(0, 0, 2, 2, 2, -1, 1, 1, 1)
        self.q_start, self.kv_len = i32(0, 2, 5, 6, 9), i32(20, 3, 17, 40)
        self.table = torch.randperm(12, generator=g, device="cuda").to(torch.int32).view(SEQS, 3)
        self.cache = sg.make_kv_cache(rnd(12, HKV, P, D), rnd(12, HKV, P, D))
        self.batch = sg.make_batch(self.q_start, self.kv_len, self.table, ROWS)
        self.freq = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
        self.w_experts = rnd(E, 2 * INTER, H, k=0.06), rnd(E, H, INTER, k=0.09)
        self.gate_up, self.down = (sg.make_experts(w) for w in self.w_experts)
        nan = lambda *s, t=BF: torch.full(s, float("nan"), dtype=t, device="cuda")
        self.x, self.qkv, self.q, self.att, self.o = nan(ROWS, H), nan(ROWS, QKV), \
            nan(ROWS, HQ * D), nan(ROWS, HQ * D), nan(ROWS, H)
        self.res1, self.x2, self.logits = nan(ROWS, H, t=torch.float32), nan(ROWS, H), nan(ROWS, E)
        self.route_ids = torch.full((ROWS, TOPK), -1, dtype=torch.int32, device="cuda")
        self.route_w = nan(ROWS, TOPK, t=torch.float32)
        self.y, self.res2, self.out = nan(ROWS * TOPK, H), nan(ROWS, H, t=torch.float32), nan(ROWS, H)
        self.base_qkv, self.base_o = nan(ROWS, QKV), nan(ROWS, H)
        n = max(sg.workspace_bytes(sg.BF16, ROWS, QKV, H), sg.workspace_bytes(sg.BF16, ROWS, H, HQ * D),
                sg.workspace_bytes(sg.BF16, ROWS, E, H), sg.lora_workspace_bytes(self.lora_qkv, ROWS),
                sg.lora_workspace_bytes(self.lora_o, ROWS),
                sg.kv_attention_workspace_bytes(self.cache, self.batch, HQ))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.ws_moe = torch.zeros(sg.moe_mlp_workspace_bytes(self.gate_up, self.down, ROWS, TOPK),
                                  dtype=torch.uint8, device="cuda")

    def run(self):
        """One workspace serves every stage but the experts', in stream order."""
        n1, n2, n3, n4 = self.norms
        sg.block_norm(self.x, n1, block=self.h, residual_out=self.residual)
        sg.skinny_gemm_bf16(self.x, self.w_qkv, self.qkv, self.ws)
        self.base_qkv.copy_(self.qkv)
        sg.lora_linear(self.lora_qkv, self.x, self.ids, self.qkv, self.ws)
        sg.kv_append(self.cache, self.batch, self.qkv, self.freq, self.q)
        sg.kv_attention(self.cache, self.batch, self.q, self.att, self.ws)
        sg.skinny_gemm_bf16(self.att, self.w_o, self.base_o, self.ws)
        sg.lora_linear(self.lora_o, self.att, self.ids, self.o, self.ws, base=self.base_o)
        sg.block_norm(self.x2, n3, residual=self.residual, block=self.o, residual_out=self.res1,
                      post_weight=n2)
        sg.skinny_gemm_bf16(self.x2, self.w_router, self.logits, self.ws)
        sg.moe_route(self.logits, self.route_ids, self.route_w, scoring=sg.ROUTE_SIGMOID,
                     bias=self.bias, groups=4, top_groups=2, scale=1.5)
        sg.moe_mlp_swiglu(self.gate_up, self.down, self.x2, self.route_ids, self.y, self.ws_moe)
        sg.block_norm(self.out, n4, residual=self.res1, block=self.y, residual_out=self.res2,
                      route_weights=self.route_w)

    def check(self):
        torch.cuda.synchronize()
        n1, n2, n3, n4 = (lu.host(n) for n in self.norms)
        host = lu.host
        _, _, want, bound = lu.block_norm(host(self.h), None, n1)
        lu.near(lu.values(self.x), want, bound)
        assert torch.equal(self.residual, self.h.float())
        for x, w, y in ((self.x, self.w_qkv, self.base_qkv), (self.att, self.w_o, self.base_o),
                        (self.x2, self.w_router, self.logits)):
            y_ref, a, _ = oracle.linear_bf16(host_codes(x), host_codes(w))
            ok, worst, _ = oracle.check(host_values(y), y_ref, a)
            assert ok, worst
        ids = self.ids.tolist()
        for lora, x, base, y in ((self.lora_qkv, self.x, self.base_qkv, self.qkv),
                                 (self.lora_o, self.att, self.base_o, self.o)):
            tensors = list(lora.tensors)
            if lora is self.lora_qkv:
                a0, a2, b0, b2 = tensors
                want, bound = lu.lora(host(x), ids, host(base), [host(a0), None, host(a2)],
                                      [host(b0), HKV * D, host(b2)], None, None)
            else:
                want, bound = lu.lora(host(x), ids, host(base), [host(tensors[0])], [host(tensors[1])],
                                      self.ranks.tolist(), host(self.scale))
            lu.near(lu.values(y), want, bound)
        h, eh, want, bound = lu.block_norm(host(self.o), host(self.residual), n3, post_weight=n2)
        lu.near(lu.values(self.res1), h, eh, lu.U32, 2.0 ** -148)
        lu.near(lu.values(self.x2), want, bound)
        rid, rw = lu.route(host(self.logits), TOPK, True, bias=host(self.bias), groups=4, top_groups=2,
                           scale=1.5)
        np.testing.assert_array_equal(self.route_ids.cpu().numpy(), rid)
        lu.near(host(self.route_w), rw, 2.0 ** -40 * rw, lu.U32, 2.0 ** -149)
        h, eh, want, bound = lu.block_norm(host(self.y), host(self.res1), n4, routes=TOPK,
                                           route_weights=host(self.route_w))
        lu.near(lu.values(self.res2), h, eh, lu.U32, 2.0 ** -148)
        lu.near(lu.values(self.out), want, bound)
        assert not self.y.isnan().any()


def test_layer_runs_together():
    need_gpu()
    layer = Layer()
    layer.run()
    layer.check()


def test_layer_as_a_graph():
    """Captured once, replayed with other inputs, adapters and lengths in the same
    buffers, with eager work between the replays."""
    need_gpu()
    layer = Layer(seed=1)
    layer.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    for step in range(3):
        layer.h.copy_(layer.rnd(ROWS, H))
        layer.ids.copy_(torch.randint(-1, ADAPTERS, (ROWS,), generator=layer.g, device="cuda"))
        layer.kv_len += 3
        graph.replay()
        layer.check()
        kept = [t.clone() for t in (layer.out, layer.res2, layer.qkv)]
        layer.run()
        torch.cuda.synchronize()
        for a, b in zip(kept, (layer.out, layer.res2, layer.qkv)):
            assert torch.equal(a, b)


def test_two_streams_with_their_own_workspaces():
    """Adapters of a long call and of a short one at once give what each gives alone."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    lora = sg.make_lora(rnd(5, 32, 512), rnd(5, 700, 32))
    calls = []
    for rows in (3, 40, 300, 2000):
        ids = torch.randint(-1, 5, (rows,), generator=g, device="cuda").to(torch.int32)
        ws = torch.empty(sg.lora_workspace_bytes(lora, rows), dtype=torch.uint8, device="cuda")
        calls.append((rnd(rows, 512), ids, rnd(rows, 700), ws))
    alone = []
    for x, ids, base, ws in calls:
        y = torch.empty_like(base)
        sg.lora_linear(lora, x, ids, y, ws, base=base)
        torch.cuda.synchronize()
        alone.append(y)
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        together = [torch.empty_like(base) for _, _, base, _ in calls]
        torch.cuda.synchronize()
        for s, y, (x, ids, base, ws) in zip(streams, together, calls):
            sg.lora_linear(lora, x, ids, y, ws, base=base, stream=s)
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert torch.equal(a, b)
