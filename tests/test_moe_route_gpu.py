"""moe_route against its 64-bit form: ids equal, weights rounded once."""
import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
from tests import layer_util as lu
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def run_and_check(logits, topk, bias=None, **kw):
    rows = logits.shape[0]
    ids = torch.full((rows + 2, topk), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((rows + 2, topk), NAN, device="cuda")
    sg.moe_route(logits, ids[1:-1], weights[1:-1], bias=bias, **kw)
    torch.cuda.synchronize()
    assert (ids[0] == -7).all() and (ids[-1] == -7).all()
    assert weights[0].isnan().all() and weights[-1].isnan().all()
    sigmoid = kw.pop("scoring", sg.ROUTE_SOFTMAX) == sg.ROUTE_SIGMOID
    want, w = lu.route(lu.host(logits), topk, sigmoid, bias=lu.host(bias), **kw)
    np.testing.assert_array_equal(ids[1:-1].cpu().numpy(), want)
    # One rounding; the 64-bit sums and exponentials leave less than 2^-40.
    lu.near(weights[1:-1].double().cpu().numpy(), w, 2.0 ** -40 * np.abs(w), lu.U32, 2.0 ** -149)


def rand(rows, experts, dtype, seed, k=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (k * torch.randn(rows, experts, generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("experts", [1, 2, 8, 63, 64, 65, 128, 161, 256, 257, 512, 1000, 1024])
@pytest.mark.parametrize("scoring", [sg.ROUTE_SOFTMAX, sg.ROUTE_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_experts(experts, scoring, dtype):
    need_gpu()
    for topk in sorted({1, min(6, experts), min(16, experts)}):
        run_and_check(rand(7, experts, dtype, experts), topk, scoring=scoring,
                      renormalize=topk > 1, scale=1.0 if topk > 1 else 2.5)


@pytest.mark.parametrize("experts,groups,top", [(8, 2, 1), (256, 8, 4), (60, 5, 2), (64, 64, 16),
                                                (1024, 32, 3), (21, 3, 3), (1000, 4, 1)])
@pytest.mark.parametrize("scoring", [sg.ROUTE_SOFTMAX, sg.ROUTE_SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(experts, groups, top, scoring, biased):
    need_gpu()
    bias = rand(1, experts, torch.float32, 5, 0.2)[0] if biased else None
    topk = min(8, experts // groups * top)
    run_and_check(rand(13, experts, torch.float32, groups), topk, bias=bias, scoring=scoring,
                  groups=groups, top_groups=top)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 1027])
def test_rows(rows):
    need_gpu()
    run_and_check(rand(rows, 96, torch.bfloat16, rows), 4)


def test_equal_logits_go_by_index():
    need_gpu()
    l = torch.zeros(3, 200, device="cuda")
    l[1, 150:] = 1.0
    l[2, ::7] = -0.0
    for dtype in (torch.float32, torch.bfloat16):
        run_and_check(l.to(dtype), 5)
        run_and_check(l.to(dtype), 5, groups=10, top_groups=3)
        run_and_check(l.to(dtype), 5, bias=torch.zeros(200, device="cuda"), groups=10, top_groups=3,
                      scoring=sg.ROUTE_SIGMOID)


def test_values_that_are_no_numbers():
    need_gpu()
    l = rand(9, 70, torch.float32, 3)
    l[0, :] = -INF
    l[1, :] = NAN
    l[2, 3:] = -INF                    # fewer experts than choices
    l[3, 10] = INF
    l[4, 10] = l[4, 60] = INF
    l[5, ::2] = NAN
    l[6, 20] = torch.finfo(torch.float32).max
    l[7, 20] = torch.finfo(torch.float32).min
    l[8] *= 300.0                      # sigmoids that are 1 in 64 bits keep the logits' order
    bias = torch.zeros(70, device="cuda")
    bias[5], bias[6], bias[7] = -INF, NAN, INF
    for scoring in (sg.ROUTE_SOFTMAX, sg.ROUTE_SIGMOID):
        for renormalize in (True, False):
            for kw in (dict(), dict(groups=7, top_groups=2), dict(groups=35, top_groups=3)):
                run_and_check(l, 6, scoring=scoring, renormalize=renormalize, **kw)
                run_and_check(l, 6, bias=bias, scoring=scoring, renormalize=renormalize, **kw)


@pytest.mark.parametrize("biased", [False, True])
def test_long_offsets(biased):
    """The most rows and experts, logits of 2^32 bytes: a row gives what it gives alone."""
    need_gpu()
    rows, experts, topk = 1 << 20, 1024, 16
    logits = rand(rows, experts, torch.float32, 8)
    bias = rand(1, experts, torch.float32, 5, 0.2)[0] if biased else None
    ids = torch.full((rows, topk), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((rows, topk), NAN, device="cuda")
    sg.moe_route(logits, ids, weights, bias=bias, groups=64, top_groups=8)
    one, one_w = torch.empty_like(ids[:1]), torch.empty_like(weights[:1])
    for t in (0, 1, rows // 2 - 1, rows // 2, rows - 1):
        sg.moe_route(logits[t:t + 1], one, one_w, bias=bias, groups=64, top_groups=8)
        assert torch.equal(ids[t:t + 1], one) and torch.equal(weights[t:t + 1], one_w)


@pytest.mark.parametrize("experts,groups,top", [(64, 1, 1), (161, 1, 1), (256, 8, 4), (1000, 4, 1),
                                                (1024, 64, 16)])
def test_bf16_values_that_are_no_numbers(experts, groups, top):
    """And bf16 neighbours: equal ones by index, its largest behind infinity, its smallest."""
    need_gpu()
    l = rand(12, experts, torch.bfloat16, experts)
    l[0, :] = -INF
    l[1, :] = NAN
    l[2, 3:] = -INF                    # fewer experts than choices
    l[3, 40] = INF
    l[3, 2] = l[3, 50] = torch.finfo(torch.bfloat16).max
    l[4, 10] = l[4, 60] = INF
    l[5, ::2] = NAN
    l[6, :] = torch.finfo(torch.bfloat16).min
    l[6, 7] = -INF
    l[7, :] = -1.0                     # equal but for the sign of zeros and the smallest numbers
    l[7, 30:] = -0.0
    l[7, 45:] = 0.0
    l[7, 62] = 2.0 ** -133
    l[7, 63] = -2.0 ** -133
    l[8] *= 100.0
    l[9] = l[9].round()                # many equal ones
    l[10, :] = 0.5
    for scoring in (sg.ROUTE_SOFTMAX, sg.ROUTE_SIGMOID):
        for renormalize in (True, False):
            run_and_check(l, 8, scoring=scoring, renormalize=renormalize, groups=groups,
                          top_groups=top)
