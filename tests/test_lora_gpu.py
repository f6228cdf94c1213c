"""lora_linear against its 64-bit form: whole numbers, whose sums hold no
rounding, bitwise; other values within what fp32 sums leave."""
import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
from tests import layer_util as lu
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF, NAN, INF = torch.bfloat16, float("nan"), float("inf")


class Call:
    def __init__(self, rows, K, n, adapters, rank, ids=None, ranks=None, scaled=True, whole=False,
                 bare=(), seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s, most=2, k=1.0):
            if whole:
                return torch.randint(-most, most + 1, s, generator=g, device="cuda").to(BF)
            return (k * torch.randn(*s, generator=g, device="cuda")).to(BF)

        self.rows, self.N = rows, sum(n)
        self.x, self.base = rnd(rows, K), rnd(rows, sum(n), most=100)
        self.a = [None if i in bare else rnd(adapters, rank, K, k=K ** -0.5) for i in range(len(n))]
        self.b = [w if i in bare else rnd(adapters, w, rank) for i, w in enumerate(n)]
        if ids is None:
            ids = torch.randint(-1, adapters, (rows,), generator=g, device="cuda")
        self.ids = torch.as_tensor(ids, device="cuda").to(torch.int32)
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
        self.scale = None
        if scaled:
            self.scale = torch.randint(-2, 3, (adapters,), generator=g, device="cuda").float() if whole \
                else torch.randn(adapters, generator=g, device="cuda")
        self.lora = sg.make_lora(self.a, self.b, scale=self.scale, ranks=self.ranks)
        self.ws = torch.full((sg.lora_workspace_bytes(self.lora, rows),), 0xFF, dtype=torch.uint8,
                             device="cuda")

    def want(self):
        part = lambda v: v if v is None or isinstance(v, int) else lu.host(v)
        return lu.lora(lu.host(self.x), self.ids.tolist(), lu.host(self.base),
                       [part(v) for v in self.a], [part(v) for v in self.b],
                       None if self.ranks is None else self.ranks.tolist(), lu.host(self.scale))

    def run(self, in_place=False):
        guard = 40
        y = torch.full((self.rows * self.N + 2 * guard,), 7.0, dtype=BF, device="cuda")
        inner = y[guard:guard + self.rows * self.N].view(self.rows, self.N)
        if in_place:
            inner.copy_(self.base)
        else:
            inner.fill_(NAN)
        sg.lora_linear(self.lora, self.x, self.ids, inner, self.ws,
                       base=None if in_place else self.base)
        torch.cuda.synchronize()
        assert (y[:guard] == 7).all() and (y[guard + self.rows * self.N:] == 7).all()
        return inner

    def check(self, whole=False):
        want, bound = self.want()
        for in_place in (False, True):
            got = self.run(in_place)
            if whole:                  # every sum is a whole number below 2^24
                rounded = torch.from_numpy(want).to(torch.float32).to(BF)
                assert np.abs(want).max() < 2 ** 24
                assert torch.equal(got.cpu(), rounded)
            else:
                lu.near(lu.values(got), want, bound)
        return got


SIZES = [
    (1, 8, [1], 1, 8), (1, 8192, [1024], 3, 16), (2, 64, [64], 2, 8), (3, 72, [65], 2, 24),
    (16, 1000, [256, 100, 31], 5, 32), (17, 520, [257], 1, 64), (33, 128, [300], 40, 40),
    (64, 256, [70], 64, 16), (65, 256, [70, 3], 3, 72), (200, 328, [513], 9, 128),
    (300, 64, [40], 2, 256), (1000, 136, [96, 17], 70, 8), (2500, 72, [130], 4, 48),
    (600, 200, [64, 33], 3, 256), (9000, 24, [19], 200, 8), (9001, 16, [8], 3, 16),
]


@pytest.mark.parametrize("rows,K,n,adapters,rank", SIZES)
def test_whole_numbers(rows, K, n, adapters, rank):
    need_gpu()
    Call(rows, K, n, adapters, rank, whole=True, seed=rows).check(whole=True)


@pytest.mark.parametrize("rows,K,n,adapters,rank", SIZES)
def test_values(rows, K, n, adapters, rank):
    need_gpu()
    ranks = [(7 * e + 3) % (rank + 1) for e in range(adapters)]
    Call(rows, K, n, adapters, rank, seed=rows).check()
    Call(rows, K, n, adapters, rank, ranks=ranks, scaled=False, seed=rows + 1).check()


def test_ranks_hide_what_is_behind_them():
    need_gpu()
    ranks = [0, 1, 15, 16, 17, 40, 99, -3]
    c = Call(50, 136, [90, 33], 8, 40, ranks=ranks, whole=True)
    for e, r in enumerate(ranks):
        r = min(max(r, 0), 40)
        for a, b in zip(c.a, c.b):
            a[e, r:] = NAN
            b[e, :, r:] = float("inf")
    c.check(whole=True)


def test_slices_without_adapters():
    need_gpu()
    for bare in ((0,), (1,), (2,), (0, 2), (1, 2)):
        for rows in (3, 90):
            Call(rows, 64, [33, 300, 8], 4, 16, whole=True, bare=bare).check(whole=True)


@pytest.mark.parametrize("ids", [[-1] * 70, [9, -5, 1 << 30, -(1 << 31)] * 20, [0] * 130,
                                 list(range(3)) * 22, [2] * 15 + [-1] * 34 + [1] * 81])
def test_ids(ids):
    need_gpu()
    Call(len(ids), 128, [100], 3, 16, ids=ids, whole=True).check(whole=True)


def test_values_that_are_no_numbers_stay_in_their_row():
    need_gpu()
    c = Call(40, 128, [70], 3, 16, whole=True)
    c.ids.copy_(torch.arange(40) % 4 - 1)
    c.x[5, 3], c.x[6, 127], c.base[9, 0] = NAN, float("inf"), NAN
    c.scale.fill_(1.0)
    c.a[0][:, :, 127] = 1.0
    c.b[0][c.b[0] == 0] = 1.0
    c.b[0][:, :35].abs_()
    rows = [t for t in range(40) if t not in (5, 6)]
    want = torch.from_numpy(c.want()[0]).to(torch.float32).to(BF)
    got = c.run().cpu()
    same = (got[rows] == want[rows]) | (got[rows].isnan() & want[rows].isnan())
    assert same.all() and got[5].isnan().all()
    # An infinite A x gives infinities where B has one sign, NaN where both meet.
    infinite = want[6].isinf()
    assert infinite[:35].all()
    assert torch.equal(got[6][infinite], want[6][infinite])


def test_largest_numbers():
    """A x beyond bf16's largest number and within fp32's keeps its value."""
    need_gpu()
    c = Call(4, 64, [16], 1, 8, ids=[0] * 4, scaled=False, whole=True)
    top = float(torch.finfo(torch.float32).max)
    c.x.zero_()
    c.a[0].zero_()
    c.x[:, 0], c.x[:, 1] = 2.0 ** 64, 2.0 ** 64
    c.a[0][0, :, 0], c.a[0][0, :, 1] = 2.0 ** 63, 2.0 ** 62 * 1.9921875     # sum below 2^128
    c.b[0].zero_()
    c.b[0][0, :, 0] = 2.0 ** -100
    v = 2.0 ** 127 + 2.0 ** 126 * 1.9921875
    assert float(torch.finfo(BF).max) < v < top
    c.base.zero_()
    got = c.run()
    want = torch.full_like(c.base, v * 2.0 ** -100)
    assert torch.equal(got, want)


def test_many_adapters():
    need_gpu()
    ids = torch.arange(700) * 37 % 8192
    Call(700, 64, [33], 8192, 8, ids=ids, whole=True).check(whole=True)


@pytest.mark.parametrize("rows,rank", [(5, 256), (70, 16), (600, 256)])
def test_as_a_graph(rows, rank):
    """Replays take the ids and values that are in the buffers then."""
    need_gpu()
    c = Call(rows, 136, [65, 40], 6, rank, whole=True)
    y = torch.empty_like(c.base)
    go = lambda: sg.lora_linear(c.lora, c.x, c.ids, y, c.ws, base=c.base)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for step in range(3):
        c.ids.copy_(torch.randint(-1, 6, (rows,), device="cuda"))
        c.x.copy_(torch.randint(-2, 3, c.x.shape, device="cuda"))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), torch.from_numpy(c.want()[0]).to(torch.float32).to(BF))


def test_long_offsets():
    """More than 2^31 values of y."""
    need_gpu()
    rows, N = 110000, 20001
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(BF)
    x, a, b = ints(rows, 8), ints(2, 8, 8), ints(2, N, 8)
    ids = torch.randint(-1, 2, (rows,), generator=g, device="cuda").to(torch.int32)
    y = torch.ones(rows, N, dtype=BF, device="cuda")
    lora = sg.make_lora(a, b)
    ws = torch.empty(sg.lora_workspace_bytes(lora, rows), dtype=torch.uint8, device="cuda")
    sg.lora_linear(lora, x, ids, y, ws)
    for t in (0, 1, 53687, 107368, 107369, rows - 2, rows - 1):
        e = int(ids[t])
        want = torch.ones(N, device="cuda")
        if e >= 0:
            want = want + b[e].float() @ (a[e].float() @ x[t].float())
        assert torch.equal(y[t], want.to(BF))


def test_long_x():
    """The most rows, and more than 2^31 values of x."""
    need_gpu()
    rows, K, N = 1 << 20, 2056, 17
    g = torch.Generator(device="cuda").manual_seed(2)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda", dtype=torch.int8).to(BF)
    x, a, b = ints(rows, K), ints(3, 8, K), ints(3, N, 8)
    ids = torch.randint(-1, 3, (rows,), generator=g, device="cuda").to(torch.int32)
    y = torch.ones(rows, N, dtype=BF, device="cuda")
    lora = sg.make_lora(a, b)
    ws = torch.empty(sg.lora_workspace_bytes(lora, rows), dtype=torch.uint8, device="cuda")
    sg.lora_linear(lora, x, ids, y, ws)
    for t in (0, 1, (1 << 31) // K, (1 << 31) // K + 1, rows - 2, rows - 1):
        e = int(ids[t])
        want = torch.ones(N, device="cuda")
        if e >= 0:                     # whole numbers below 2^24, exact in fp32
            want = want + b[e].float() @ (a[e].float() @ x[t].float())
        assert torch.equal(y[t], want.to(BF))


@pytest.mark.parametrize("rows,rank", [(1, 8), (5, 40), (30, 128), (64, 256), (70, 16), (200, 64),
                                       (300, 256), (600, 8), (700, 72), (1100, 200)])
def test_sums_of_24_bits_stay_whole(rows, rank):
    """A x of up to 23 bits, whose differences y shows: pairs of A's rows differ where x counts
    once only.  Every partial sum is a whole number below 2^24, exact in fp32 in any order."""
    need_gpu()
    adapters, K, N = 3, 24, 70
    c = Call(rows, K, [N], adapters, rank, ids=[t % 4 for t in range(rows)], whole=True, scaled=False)
    g = torch.Generator(device="cuda").manual_seed(rank)
    ints = lambda most, *s: torch.randint(-most, most + 1, s, generator=g, device="cuda")
    step = 2 ** (torch.arange(K, device="cuda") % 12)
    a = ints(255, adapters, rank // 2, 1, K) * step
    a = a.repeat(1, 1, 2, 1)
    a[..., ::12] = ints(255, adapters, rank // 2, 2, K // 12)
    c.a[0].copy_(a.reshape(adapters, rank, K))
    pair = torch.randint(0, rank // 2, (adapters, N, 1), generator=g, device="cuda")
    b = torch.zeros(adapters, N, rank, device="cuda")
    b.scatter_(2, 2 * pair, 1.0).scatter_(2, 2 * pair + 1, -1.0)
    c.b[0].copy_(b)
    c.check(whole=True)
    x, A = lu.host(c.x), lu.host(c.a[0])
    size = max(float((np.abs(A[i]) @ np.abs(x[t])).max()) for t, i in enumerate(c.ids.tolist()) if i < adapters)
    assert 2 * size + 100 < 2 ** 24


@pytest.mark.parametrize("rows,rank", [(1, 8), (20, 64), (40, 128), (64, 256), (90, 16), (200, 40),
                                       (600, 64), (700, 200)])
@pytest.mark.parametrize("most", [2, 255])
def test_infinities_in_b(rows, rank, most):
    """B's infinities and NaN within the rank: y is infinite where A x is not 0 there, whether
    A x is a bf16 number (most 2) or needs more bits, and other columns and rows are whole."""
    need_gpu()
    adapters, K, N = 3, 64, 150
    c = Call(rows, K, [N], adapters, rank, ids=[t % 4 for t in range(rows)], whole=True, scaled=False)
    g = torch.Generator(device="cuda").manual_seed(rows)
    c.a[0].copy_(torch.randint(-most, most + 1, c.a[0].shape, generator=g, device="cuda"))
    b = c.b[0]
    b[:, 3, rank - 1], b[0, 70, 0], b[1, 71, 1], b[2, 72, 2] = INF, -INF, NAN, INF
    b[0, 149, 5], b[0, 149, 6] = INF, -INF
    want = torch.from_numpy(c.want()[0]).to(torch.float32).to(BF)
    assert want[:, 3].isinf().any() and torch.isfinite(want[:, 4:70]).all()
    for in_place in (False, True):
        got = c.run(in_place).cpu()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(nan=0.5, posinf=INF, neginf=-INF),
                           want.nan_to_num(nan=0.5, posinf=INF, neginf=-INF))


def test_smallest_numbers():
    """A x of 2^-115 + 2^-132 and 2^-115: parts below bf16's normal numbers count, too."""
    need_gpu()
    for rows in (2, 70, 600):
        c = Call(rows, 64, [16], 1, 8, ids=[0] * rows, scaled=False, whole=True)
        for t in (c.x, c.a[0], c.b[0], c.base):
            t.zero_()
        c.x[:, 0], c.x[:, 1] = 2.0 ** -60, 2.0 ** -66
        c.a[0][0, :2, 0], c.a[0][0, 0, 1] = 2.0 ** -55, 2.0 ** -66
        c.b[0][0, :, 0], c.b[0][0, :, 1] = 2.0 ** 120, -2.0 ** 120
        assert (c.run() == 2.0 ** -12).all()


def test_filled_by_hand():
    """A descriptor that a program fills itself is make_lora's."""
    need_gpu()
    c = Call(20, 64, [33, 40], 3, 16, whole=True, scaled=False)
    made, c.lora = c.lora, sg.Lora(3, 16, 64, 2)
    for i in range(2):
        c.lora.n[i], c.lora.a[i], c.lora.b[i] = made.n[i], made.a[i], made.b[i]
    assert sg.lora_workspace_bytes(c.lora, 20) == sg.lora_workspace_bytes(made, 20)
    c.check(whole=True)


@pytest.mark.parametrize("rows", [2, 17, 63, 64])
@pytest.mark.parametrize("step", [1, 7, 13])
def test_rows_of_an_adapter_anywhere(rows, step):
    """The rows of an adapter, spread over the call, as the first launch lists them for the second."""
    need_gpu()
    Call(rows, 72, [100], 4, 24, ids=[t * step % 5 for t in range(rows)], whole=True).check(whole=True)


def placed(values, offset, fill):
    """A copy of a 2-D tensor, `offset` values behind an aligned address, and the whole buffer."""
    n = values.numel()
    buf = torch.full((n + 48,), fill, dtype=values.dtype, device="cuda")
    inner = buf[16 + offset:16 + offset + n].view(values.shape)
    inner.copy_(values)
    return inner, buf


@pytest.mark.parametrize("rows,n,rank", [(1, [8], 8), (5, [64], 40), (5, [65], 16), (40, [7, 70], 136),
                                         (70, [64], 16), (300, [129], 72), (600, [130], 16),
                                         (600, [3, 129], 136)])
def test_addresses_of_a_value(rows, n, rank):
    """base and y at any multiple of 2 bytes, each at its own; nothing beside them counts or
    changes, nor what lies behind a workspace of just the bytes that it has to have."""
    need_gpu()
    c = Call(rows, 64, n, 3, rank, ids=[t % 4 for t in range(rows)], whole=True)
    want = torch.from_numpy(c.want()[0]).to(torch.float32).to(BF)
    need = sg.lora_workspace_bytes(c.lora, rows)
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    for base_at, y_at in ((0, 1), (1, 0), (1, 1), (3, 2), (2, 3), (7, 5), (None, 1), (None, 3)):
        y, buf = placed(torch.full_like(c.base, NAN) if base_at is not None else c.base, y_at, 7.0)
        base = None if base_at is None else placed(c.base, base_at, NAN)[0]
        sg.lora_linear(c.lora, c.x, c.ids, y, ws[:need], base=base)
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want)
        assert (buf[:16 + y_at] == 7).all() and (buf[16 + y_at + y.numel():] == 7).all()
        assert (ws[need:] == 0xAB).all()
