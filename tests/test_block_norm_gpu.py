"""block_norm against its 64-bit form: every operand there and not there, both
kinds, both types, widths from one value to the largest, odd ones among them, and
rows with values at the ends of the types."""
import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
from tests import layer_util as lu
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(rows, width, routes=1, residual=BF, weight=BF, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, k=1.0, m=0.0: m + k * torch.randn(*s, generator=g, device="cuda")
    return dict(residual=rnd(rows, width, k=3 * spread).to(residual),
                block=rnd(rows * routes, width, k=spread).to(BF),
                weight=rnd(width, k=0.2, m=1.0).to(weight), bias=rnd(width, k=0.1).to(weight),
                post_weight=rnd(width, k=0.2, m=0.5).to(weight),
                post_bias=rnd(width, k=0.1).to(weight), gate=rnd(width, k=0.5).to(weight),
                gate_rows=rnd(rows, width, k=0.5).to(weight),
                route_weights=torch.softmax(rnd(rows, routes), dim=1))


def run_and_check(rows, width, t, routes=1, res_type=BF, in_place=False, want_out=True,
                  want_res=True, **kw):
    """t: the operands by block_norm's names."""
    scalars = {k: kw[k] for k in ("eps", "residual_scale", "block_scale", "weight_offset") if k in kw}
    host = {k: lu.host(v) for k, v in t.items() if k != "weight"}
    block, residual = host.pop("block", None), host.pop("residual", None)
    h, eh, want, bound = lu.block_norm(block, residual, lu.host(t.get("weight")), routes=routes,
                                       layer=kw.get("kind") == sg.NORM_LAYER, **host, **scalars)
    guard = 64                        # values on both sides that must stay as they were
    out = torch.full((rows * width + 2 * guard,), 7.0, dtype=BF, device="cuda")
    inner = out[guard:guard + rows * width].view(rows, width)
    res = None
    if want_res:
        res = t["residual"] if in_place else torch.full((rows, width), float("nan"),
                                                        dtype=res_type, device="cuda")
    args = {k: v for k, v in t.items() if k != "weight"}
    sg.block_norm(inner if want_out else None, t.get("weight") if want_out else None,
                  residual_out=res, **args, **kw)
    torch.cuda.synchronize()
    if want_out:
        lu.near(lu.values(inner), want, bound)
    assert (out[:guard] == 7).all() and (out[guard + rows * width:] == 7).all()
    if want_res:
        half, tiny = (lu.U16, lu.TINY16) if res_type is BF else (lu.U32, 2.0 ** -148)
        lu.near(lu.values(res), h + np.zeros((rows, width)), eh, half, tiny)


@pytest.mark.parametrize("width", [1, 7, 8, 63, 64, 100, 512, 513, 520, 1001, 2048, 2049, 4096, 5001,
                                   8191, 8192, 8193, 16384, 16391, 32768])
@pytest.mark.parametrize("kind", [sg.NORM_RMS, sg.NORM_LAYER])
def test_widths(width, kind):
    need_gpu()
    rows = 5
    t = make(rows, width, seed=width)
    del t["gate_rows"], t["route_weights"]
    run_and_check(rows, width, t, kind=kind)


@pytest.mark.parametrize("rows,width", [(1, 8192), (3, 264), (130, 72), (1030, 504), (2050, 1544),
                                        (515, 8192), (300, 5001)])
@pytest.mark.parametrize("res_type,w_type", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_rows_and_types(rows, width, res_type, w_type):
    need_gpu()
    t = make(rows, width, residual=res_type, weight=w_type, seed=rows)
    run_and_check(rows, width, {k: t[k] for k in ("residual", "block", "weight")}, res_type=res_type)


@pytest.mark.parametrize("routes", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("weighted", [False, True])
def test_routes(routes, weighted):
    need_gpu()
    t = make(9, 1016, routes, residual=F32, seed=routes)
    names = ["residual", "block", "weight"] + (["route_weights"] if weighted else [])
    run_and_check(9, 1016, {k: t[k] for k in names}, routes=routes, res_type=F32)


FORMS = [
    ("residual", "weight"), ("block", "weight"), ("residual",), ("block",),
    ("residual", "block", "weight", "gate"), ("residual", "block", "weight", "gate_rows"),
    ("residual", "block", "post_weight", "weight"),
    ("residual", "block", "post_weight", "post_bias", "gate", "weight", "bias"),
    ("block", "post_weight", "gate_rows"),
]


@pytest.mark.parametrize("form", FORMS, ids="+".join)
@pytest.mark.parametrize("kind", [sg.NORM_RMS, sg.NORM_LAYER])
@pytest.mark.parametrize("width", [72, 6001])
def test_forms(form, kind, width):
    need_gpu()
    t = make(6, width, seed=len(form))
    t = {("gate" if k == "gate_rows" else k): t[k] for k in form}
    run_and_check(6, width, t, kind=kind, residual_scale=0.75, block_scale=-1.25, weight_offset=1.0,
                  eps=1e-5)


def test_in_place_and_one_output():
    need_gpu()
    names = ("residual", "block", "weight")
    for res_type in (BF, F32):
        t = make(7, 3000, residual=res_type)
        run_and_check(7, 3000, {k: t[k] for k in names}, res_type=res_type, in_place=True)
        t = make(7, 3000, residual=res_type)
        run_and_check(7, 3000, {k: t[k] for k in names}, res_type=res_type, want_res=False)
        t = make(7, 3000, residual=res_type)
        run_and_check(7, 3000, {k: t[k] for k in ("residual", "block")}, res_type=res_type,
                      want_out=False)


@pytest.mark.parametrize("spread", [1e-30, 1e-18, 1e18, 1e36])
@pytest.mark.parametrize("kind", [sg.NORM_RMS, sg.NORM_LAYER])
def test_ends_of_the_types(spread, kind):
    """Squares pass fp32's range on both sides; sums are held in 64 bits."""
    need_gpu()
    t = make(3, 777, residual=F32, spread=spread)
    for names in (("residual", "block", "weight"), ("residual", "block", "post_weight", "weight")):
        run_and_check(3, 777, {k: t[k] for k in names}, res_type=F32, kind=kind, eps=0.0)


def test_not_finite_rows_stay_alone():
    need_gpu()
    for width in (200, 2000, 8192):
        t = make(6, width)
        t["residual"][1, 3] = float("nan")
        t["block"][2, width - 1] = float("inf")
        t["residual"][4, 0] = -float("inf")
        run_and_check(6, width, {k: t[k] for k in ("residual", "block", "weight")})


def test_zero_and_constant_rows():
    need_gpu()
    z = torch.zeros(4, 300, dtype=BF, device="cuda")
    w = torch.ones(300, dtype=BF, device="cuda")
    out = torch.empty_like(z)
    sg.block_norm(out, w, residual=z)
    assert (out == 0).all()
    sg.block_norm(out, w, residual=z, eps=0.0)              # 0 / 0
    assert out.isnan().all()
    for eps in (1e-6, 1e-12):                               # a constant row has no deviation
        sg.block_norm(out, w, residual=z + 1000.0, kind=sg.NORM_LAYER, eps=eps)
        assert (out == 0).all()


def test_reproducible_on_another_stream():
    need_gpu()
    t = make(33, 4104)
    outs = []
    side = torch.cuda.Stream()
    for stream in (None, side, side):
        out = torch.empty(33, 4104, dtype=BF, device="cuda")
        torch.cuda.synchronize()
        sg.block_norm(out, t["weight"], residual=t["residual"], block=t["block"], stream=stream)
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[1], outs[2])


def test_long_offsets():
    """The most rows, and more than 2^31 values: a row gives what it gives alone."""
    need_gpu()
    rows, width = 1 << 20, 2056
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)
    residual, block, gate, weight = rnd(rows, width), rnd(rows, width), rnd(rows, width), rnd(width)
    out, kept = torch.empty_like(residual), torch.empty_like(residual)
    sg.block_norm(out, weight, residual=residual, block=block, gate=gate, residual_out=kept)
    one, one_kept = torch.empty_like(out[:1]), torch.empty_like(kept[:1])
    for t in (0, 1, (1 << 31) // width, (1 << 31) // width + 1, rows - 1):
        sg.block_norm(one, weight, residual=residual[t:t + 1], block=block[t:t + 1],
                      gate=gate[t:t + 1], residual_out=one_kept)
        assert torch.equal(out[t:t + 1], one) and torch.equal(kept[t:t + 1], one_kept)


WIDE = [("residual", "block", "weight"),
        ("residual", "block", "post_weight", "post_bias", "gate", "weight", "bias"),
        ("block", "post_weight", "gate_rows")]


@pytest.mark.parametrize("width", [8200, 12001, 16385, 20000, 32767])
@pytest.mark.parametrize("res_type,w_type", [(F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("form", WIDE, ids="+".join)
def test_wide_rows_of_32_bits(width, res_type, w_type, form):
    """Several units per thread with fp32 operands."""
    need_gpu()
    for kind in (sg.NORM_RMS, sg.NORM_LAYER):
        t = make(4, width, residual=res_type, weight=w_type, seed=width)
        run_and_check(4, width, {("gate" if k == "gate_rows" else k): t[k] for k in form}, kind=kind,
                      res_type=res_type if "residual" in form else BF, residual_scale=0.75,
                      block_scale=-1.25, weight_offset=1.0)


@pytest.mark.parametrize("width", [8191, 8192, 9000, 16384, 16391, 32768])
@pytest.mark.parametrize("res_type", [BF, F32])
def test_routes_of_wide_rows(width, res_type):
    need_gpu()
    for routes, weighted in ((2, True), (3, False), (8, True)):
        t = make(5, width, routes, residual=res_type, seed=width)
        names = ["residual", "block", "weight"] + (["route_weights"] if weighted else [])
        run_and_check(5, width, {k: t[k] for k in names}, routes=routes, res_type=res_type)


@pytest.mark.parametrize("width", [5, 64, 777, 8200, 16400])
@pytest.mark.parametrize("res_type,w_type", [(BF, BF), (F32, F32)])
def test_addresses_of_a_value(width, res_type, w_type):
    """Every operand at a multiple of its type's bytes; values beside them do not count or change."""
    need_gpu()
    rows = 3
    t = make(rows, width, residual=res_type, weight=w_type, seed=width)
    del t["gate_rows"], t["route_weights"]
    aligned, apart, guards = [torch.empty(rows, width, dtype=BF, device="cuda"),
                              torch.empty(rows, width, dtype=res_type, device="cuda")], {}, []

    def placed(v, offset, fill):
        buf = torch.full((v.numel() + 64,), fill, dtype=v.dtype, device="cuda")
        guards.append((buf, 16 + offset, 16 + offset + v.numel()))
        inner = buf[16 + offset:16 + offset + v.numel()].view(v.shape)
        return inner.copy_(v)

    for i, (k, v) in enumerate(sorted(t.items())):
        apart[k] = placed(v, 1 + i % 3 * 2, float("nan"))
    guards.clear()
    out, res = placed(aligned[0], 1, 7.0), placed(aligned[1], 3, 7.0)
    for kind in (sg.NORM_RMS, sg.NORM_LAYER):
        for operands, o, r in ((t, *aligned), (apart, out, res)):
            kw = {k: v for k, v in operands.items() if k != "weight"}
            sg.block_norm(o, operands["weight"], residual_out=r, kind=kind, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, aligned[0]) and torch.equal(res, aligned[1])
        for buf, lo, hi in guards:
            assert (buf[:lo] == 7).all() and (buf[hi:] == 7).all()
    apart["residual"].copy_(t["residual"])
    kw = {k: v for k, v in apart.items() if k != "weight"}
    sg.block_norm(out, apart["weight"], residual_out=apart["residual"], kind=sg.NORM_LAYER, **kw)
    torch.cuda.synchronize()           # in place, as the last pass of the loop
    assert torch.equal(out, aligned[0]) and torch.equal(apart["residual"], aligned[1])
