"""block_norm, lora_linear and moe_route, and their binding, refuse bad arguments
on the host, before anything is enqueued (no GPU; the addresses are never touched)."""
import pytest
import torch

import gemv_skinny_gemm_amd as sg

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = [0x10000000 * (i + 1) for i in range(12)]
NAN, INF = float("nan"), float("inf")


def norm(**kw):
    a = dict(kind=sg.NORM_RMS, rows=4, width=100, routes=2, residual_dtype=sg.VALUES_F32,
             weight_dtype=sg.VALUES_BF16, gate_rows=0, reserved=0, eps=1e-6, residual_scale=1.0,
             block_scale=1.0, weight_offset=0.0, block=P[0], route_weights=P[1], post_weight=P[2],
             post_bias=P[3], gate=P[4], residual=P[5], residual_out=P[6], weight=P[7], bias=P[8],
             out=P[9])
    a.update(kw)
    return sg.lib().skinny_block_norm(sg.Norm(*a.values()), None)


NO_BLOCK = dict(block=None, route_weights=None, post_weight=None, post_bias=None, gate=None, routes=1)


@pytest.mark.parametrize("kw,status", [
    (dict(kind=2), INVALID), (dict(rows=0), INVALID), (dict(width=0), INVALID),
    (dict(routes=0), INVALID), (dict(residual_dtype=2), INVALID), (dict(weight_dtype=-1), INVALID),
    (dict(gate_rows=2), INVALID), (dict(gate_rows=1, gate=None), INVALID), (dict(reserved=1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(residual_scale=INF), INVALID), (dict(block_scale=NAN), INVALID),
    (dict(weight_offset=INF), INVALID), (dict(block=None), INVALID),
    (dict(NO_BLOCK, residual=None), INVALID), (dict(NO_BLOCK, routes=2), INVALID),
    (dict(NO_BLOCK, gate=P[4]), INVALID), (dict(NO_BLOCK, post_weight=P[4]), INVALID),
    (dict(NO_BLOCK, route_weights=P[4]), INVALID), (dict(post_weight=None), INVALID),
    (dict(out=None, residual_out=None, weight=None, bias=None), INVALID), (dict(out=None), INVALID),
    (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(width=32769), UNSUPPORTED),
    (dict(routes=17), UNSUPPORTED), (dict(block=P[0] + 1), UNSUPPORTED),
    (dict(residual=P[5] + 2), UNSUPPORTED), (dict(residual_out=P[6] + 2), UNSUPPORTED),
    (dict(route_weights=P[1] + 2), UNSUPPORTED), (dict(out=P[9] + 1), UNSUPPORTED),
    (dict(weight_dtype=sg.VALUES_F32, bias=P[8] + 2), UNSUPPORTED),
    (dict(out=P[0]), INVALID), (dict(out=P[5] + 64), INVALID), (dict(out=P[6]), INVALID),
    (dict(residual_out=P[0] + 1596), INVALID), (dict(residual_out=P[5] + 4), INVALID),
    (dict(residual_out=P[7]), INVALID), (dict(residual=P[0], residual_out=P[0]), INVALID),
])
def test_norm_refuses(kw, status):
    assert norm(**kw) == status


def lora(call=None, rows=5, ws=P[11], n=None, x=P[8], ids=P[9], base=P[7], y=P[10], **kw):
    l = sg.Lora(3, 16, 64, 2)
    for i in range(2):
        l.n[i], l.a[i], l.b[i] = 40 + i, P[i], P[2 + i]
    l.ranks, l.scale = P[4], P[5]
    for k, v in kw.items():
        if k[0] in "nab" and k[1:].isdigit():
            getattr(l, k[0])[int(k[1:])] = v
        else:
            setattr(l, k, v)
    return sg.lib().skinny_lora_linear(l, x, ids, rows, base, y, ws, 1 << 27 if n is None else n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), INVALID), (dict(adapters=0), INVALID), (dict(rank=0), INVALID), (dict(K=0), INVALID),
    (dict(slices=0), INVALID), (dict(n0=0), INVALID), (dict(a0=None), INVALID), (dict(b1=None), INVALID),
    (dict(a0=None, b0=None, a1=None, b1=None), INVALID), (dict(x=None), INVALID),
    (dict(ids=None), INVALID), (dict(y=None), INVALID), (dict(slices=5), UNSUPPORTED),
    (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(adapters=8193), UNSUPPORTED),
    (dict(rank=12), UNSUPPORTED), (dict(rank=256, K=1 << 23), UNSUPPORTED), (dict(rank=264), UNSUPPORTED), (dict(K=60), UNSUPPORTED),
    (dict(a1=P[1] + 8), UNSUPPORTED), (dict(b0=P[2] + 2), UNSUPPORTED), (dict(x=P[8] + 8), UNSUPPORTED),
    (dict(ids=P[9] + 2), UNSUPPORTED), (dict(ranks=P[4] + 1), UNSUPPORTED),
    (dict(scale=P[5] + 2), UNSUPPORTED), (dict(y=P[10] + 1), UNSUPPORTED),
    (dict(base=P[7] + 1), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(n=200), WORKSPACE),
    (dict(ws=P[11] + 8), UNSUPPORTED), (dict(y=P[8]), INVALID), (dict(y=P[9]), INVALID),
    (dict(y=P[7] + 2), INVALID), (dict(y=P[1] + 16), INVALID), (dict(ws=P[3]), INVALID),
    (dict(ws=P[10]), INVALID), (dict(ws=P[7]), INVALID), (dict(ws=P[4]), INVALID),
    (dict(y=P[5]), INVALID), (dict(ids=P[11] + 64), INVALID),
])
def test_lora_refuses(kw, status):
    assert lora(**kw) == status


def test_lora_workspace():
    l = sg.Lora(3, 16, 64, 1)
    l.n[0], l.a[0], l.b[0] = 40, P[0], P[1]
    need = sg.lora_workspace_bytes(l, 5)
    assert need >= 256 and sg.lora_workspace_bytes(l, 0) == 0
    assert sg.lora_workspace_bytes(l, 1 << 20) >= (1 << 20) * 16 * 4
    assert lora(n=need - 1 if need > 256 else 255) == WORKSPACE
    l.rank = 20
    assert sg.lora_workspace_bytes(l, 5) == 0
    assert sg.lib().skinny_lora_linear(None, P[0], P[1], 1, None, P[2], P[3], 1 << 20, None) == INVALID


def route(**kw):
    a = dict(dtype=sg.VALUES_BF16, scoring=sg.ROUTE_SOFTMAX, rows=5, experts=32, topk=4, groups=4,
             top_groups=2, renormalize=1, scale=1.0, reserved=0, logits=P[0], bias=P[1], ids=P[2],
             weights=P[3])
    a.update(kw)
    return sg.lib().skinny_moe_route(sg.Route(*a.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), INVALID), (dict(scoring=2), INVALID), (dict(rows=0), INVALID),
    (dict(experts=0), INVALID), (dict(topk=0), INVALID), (dict(groups=0), INVALID),
    (dict(top_groups=0), INVALID), (dict(top_groups=5), INVALID), (dict(groups=5), INVALID),
    (dict(topk=16, top_groups=1), INVALID), (dict(renormalize=2), INVALID), (dict(scale=INF), INVALID),
    (dict(reserved=1), INVALID), (dict(logits=None), INVALID), (dict(ids=None), INVALID),
    (dict(weights=None), INVALID), (dict(rows=(1 << 20) + 1), UNSUPPORTED),
    (dict(experts=1028), UNSUPPORTED), (dict(topk=17, top_groups=4), UNSUPPORTED),
    (dict(experts=130, groups=65, top_groups=65), UNSUPPORTED), (dict(logits=P[0] + 1), UNSUPPORTED),
    (dict(dtype=sg.VALUES_F32, logits=P[0] + 2), UNSUPPORTED), (dict(bias=P[1] + 2), UNSUPPORTED),
    (dict(ids=P[2] + 2), UNSUPPORTED), (dict(weights=P[3] + 1), UNSUPPORTED),
    (dict(ids=P[3]), INVALID), (dict(ids=P[0] + 4), INVALID), (dict(weights=P[1]), INVALID),
    (dict(weights=P[0]), INVALID), (dict(ids=P[1] + 64), INVALID),
])
def test_route_refuses(kw, status):
    assert route(**kw) == status


def test_null():
    assert sg.lib().skinny_block_norm(None, None) == INVALID
    assert sg.lib().skinny_moe_route(None, None) == INVALID


BF = torch.bfloat16


def refuses(fn, match, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_norm_binding():
    z = lambda *s, t=BF: torch.zeros(s, dtype=t)
    out, w, x, r = z(4, 32), z(32), z(4, 32), z(4, 32, t=torch.float32)
    refuses(sg.block_norm, "one of out and residual_out", None, w, block=x)
    refuses(sg.block_norm, "weight: shape", out, z(31), block=x)
    refuses(sg.block_norm, "bias: dtype", out, w, block=x, bias=z(32, t=torch.float32))
    refuses(sg.block_norm, "dtype float16", out, z(32, t=torch.float16), block=x)
    refuses(sg.block_norm, "block: shape", out, w, block=z(6, 32))
    refuses(sg.block_norm, "block: dtype", out, w, block=r)
    refuses(sg.block_norm, "block: shape", out, w, block=x, route_weights=z(4, 2, t=torch.float32))
    refuses(sg.block_norm, "route_weights: shape", out, w, block=x, route_weights=z(3, 1))
    refuses(sg.block_norm, "residual: shape", out, w, residual=z(4, 33))
    refuses(sg.block_norm, "residual: dtype", out, w, residual=z(4, 32, t=torch.float16))
    refuses(sg.block_norm, "residual_out: dtype", out, w, residual=x, residual_out=r)
    refuses(sg.block_norm, "gate: shape", out, w, block=x, gate=z(3, 32))
    refuses(sg.block_norm, "need a block", out, w, residual=x, gate=w)
    refuses(sg.block_norm, "contiguous", out, w, block=z(32, 4).t())
    refuses(sg.block_norm, "must be on the GPU", out, w, block=x)


def test_lora_binding():
    z = lambda *s, t=BF: torch.zeros(s, dtype=t)
    a, b = z(3, 16, 64), z(3, 40, 16)
    refuses(sg.make_lora, "same number", [a], [b, b])
    refuses(sg.make_lora, "same number", [a] * 5, [b] * 5)
    refuses(sg.make_lora, "3-D", [None], [40])
    refuses(sg.make_lora, r"a\[1\]: shape", [a, z(3, 8, 64)], [b, b])
    refuses(sg.make_lora, r"a\[0\]: dtype", a.float(), b)
    for bad, what in ((z(3, 40, 8), r"b\[0\]: shape"), (40, "3-D tensor"), (b.float(), r"b\[0\]: dtype")):
        with pytest.raises(ValueError, match=what):
            sg.make_lora(a, bad)
    refuses(sg.make_lora, "must be on the GPU", a, b)


def test_route_binding():
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t)
    ids, w, l = z(4, 2, t=torch.int32), z(4, 2), z(4, 8)
    refuses(sg.moe_route, "logits: dtype", l.double(), ids, w)
    refuses(sg.moe_route, "ids: shape", l, z(3, 2, t=torch.int32), w)
    refuses(sg.moe_route, "ids: dtype", l, z(4, 2, t=torch.int64), w)
    refuses(sg.moe_route, "weights: shape", l, ids, z(4, 3))
    refuses(sg.moe_route, "bias: shape", l, ids, w, bias=z(9))
    refuses(sg.moe_route, "must be on the GPU", l, ids, w)


def test_lora_filled_by_hand():
    """A Lora without make_lora: y's width is the sum of its slices'."""
    z = lambda *s, t=BF: torch.zeros(s, dtype=t)
    lora = sg.Lora(3, 16, 64, 2)
    for i in range(2):
        lora.n[i], lora.a[i], lora.b[i] = 40 + i, P[i], P[2 + i]
    x, ids, ws = z(5, 64), z(5, t=torch.int32), z(4096, t=torch.uint8)
    refuses(sg.lora_linear, "y: shape", lora, x, ids, z(5, 80), ws)
    refuses(sg.lora_linear, "base: shape", lora, x, ids, z(5, 81), ws, base=z(5, 40))
    refuses(sg.lora_linear, "must be on the GPU", lora, x, ids, z(5, 81), ws)
