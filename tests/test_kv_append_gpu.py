"""skinny_kv_append against its 64-bit form: every byte of the pools and scales
(those it must leave alone among them) and the rotated queries, over both cache
types, head layouts, rotations, page sizes, ragged batches and bad batches."""
import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
from tests import kv_util as kv
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def check(c, freq, interleaved=False, what=""):
    c.upload()
    c.append(freq, interleaved)
    torch.cuda.synchronize()
    kv.assert_append(c, freq, interleaved, what)


RAGGED = [(1, 1), (0, 40), (3, 3), (5, 37), (1, 16), (1, 17), (2, 33), (20, 70), (0, 0), (16, 16)]


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 4000)], [(1, 64)], [(6, 66)], [(70, 90)], RAGGED],
                         ids=["first", "far", "page-end", "two-pages", "many", "ragged"])
@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (128, 256)])
def test_shapes(dtype, seqs, P, D):
    c = kv.Case(seqs, P=P, D=D, hq=6, hkv=2, dtype=dtype, seed=P + D, tail=2)
    check(c, kv.frequencies(D))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 48, 64, 128])
def test_rotations(dtype, interleaved, rot):
    c = kv.Case([(3, 50), (2, 2)], D=128, dtype=dtype, seed=rot)
    check(c, kv.frequencies(rot) if rot else None, interleaved)


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("P,D,rot,interleaved", [(64, 128, 128, False), (16, 64, 48, True),
                                                 (128, 256, 256, False), (32, 128, 0, False),
                                                 (128, 128, 16, True)])
def test_many_rows(dtype, P, D, rot, interleaved):
    """The kernel of long steps, ragged, with rows of no sequence, a sequence in
    the middle of a page, one that begins and one without rows."""
    c = kv.Case([(700, 1003), (1, 77), (0, 40), (333, 333), (3, 300), (40, 40 + P)], P=P, D=D,
                hq=5 if D < 256 else 2, hkv=1, dtype=dtype, seed=D + rot, tail=5)
    check(c, kv.frequencies(rot) if rot else None, interleaved)


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_many_rows_bad_batches(dtype):
    """Long steps with lengths below the rows and past the table, pages outside
    the pool and values that are no finite numbers."""
    c = kv.Case([(600, 700), (500, 900), (30, 50)], D=64, hq=3, hkv=3, dtype=dtype, seed=70, tail=3,
                max_pages=50)
    c.kv_len[0] = 580                     # 20 rows at positions below 0
    c.table[1, 28] = -1                   # 900 positions: 100 past the table's 800
    c.table[1, 45] = c.pages
    x = c.qkv.reshape(c.T, -1)
    x[40, 3 * 64 + 5] = kv.BF16_NAN
    x[300, 6 * 64 + 7] = kv.BF16_INF
    check(c, kv.frequencies(64) if dtype == "bf16" else None)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (64, 8), (5, 5), (40, 8), (33, 3)])
def test_heads(hq, hkv):
    check(kv.Case([(2, 30), (1, 5)], hq=hq, hkv=hkv, D=64, seed=hq), kv.frequencies(64))


def test_far_positions():
    """Positions near 2^20 and 2^24: angles whose fp32 products are off by whole
    turns; the page table is short, so q alone is written there."""
    for far in (1 << 20, (1 << 24) - 3):
        c = kv.Case([(4, 4)], D=128, seed=9)
        c.kv_len[:] = far
        check(c, kv.frequencies(128, 1e4), what=str(far))


def test_scale_growth_and_rounding():
    """A page filled row by row with growing values: the scale grows, older codes
    are rounded again, and smaller rows later keep it; subnormal codes, zeros,
    ties and the border of 448 among the values."""
    edge = np.array([0.0, 448.0, 449.0, 447.9, 1.75, 1.7578125, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10,
                     1.0625, 1.1875, 3e38, 1e-38, -448.0, -2.0 ** -10, 240.0], np.float64)
    c = kv.Case([(1, 1)], D=64, hq=2, hkv=2, seed=3, max_pages=2)
    c.upload()
    for step, mag in enumerate([2.0 ** -80, 0.0, 1.0, 2.0 ** -12, 37.0, 2.0 ** 40, 2.0 ** 100, 1.0]):
        row = np.tile(edge, c.qkv.shape[1] // 16) * mag
        row = np.clip(row, -3e38, 3e38)
        c.qkv[0] = kv.bf16_round(row)
        c.kv_len[0] = step + 1
        for n in ("k", "v"):
            c.codes[n] = c.dev[n].cpu().numpy()
            c.scales[n] = c.dev[n + "_scale"].cpu().numpy()
        c.dev["qkv"].copy_(torch.from_numpy(c.qkv.view(np.int16)).view(torch.bfloat16))
        c.dev["kv_len"].copy_(torch.from_numpy(c.kv_len))
        c.append(None)
        torch.cuda.synchronize()
        kv.assert_append(c, None, what=f"step {step}")


def test_every_bf16_to_every_code():
    """All finite bf16 numbers of magnitude 2^-30 .. 448 * 2^-10 as one page's
    values: each code is the nearest even one."""
    D, P, hkv = 64, 128, 1
    codes = np.arange(1 << 16, dtype=np.uint16)
    v = np.abs(kv.bf16_values(codes))
    pick = codes[(v <= 448 * 2.0 ** -10) & (v >= 2.0 ** -30)]
    pick = np.resize(pick, P * D * (-(-pick.size // (P * D)))).reshape(-1, P, D)
    for block in pick:
        c = kv.Case([(P, P)], P=P, D=D, hq=1, hkv=hkv, seed=1)
        c.qkv[:, :D] = block
        c.qkv[:, D:2 * D] = block
        c.qkv[:, 2 * D:] = block
        c.qkv[0, D:] = kv.bf16_round(np.full(2 * D, 448 * 2.0 ** -10))
        check(c, None)


def test_nonfinite_values():
    c = kv.Case([(3, 20)], D=64, seed=5)
    x = c.qkv.reshape(3, -1)
    x[0, 8 * 64 + 3] = kv.BF16_NAN
    x[1, 8 * 64 + 70] = kv.BF16_INF
    x[2, 10 * 64 + 9] = kv.BF16_INF | 0x8000
    x[1, 11 * 64:12 * 64] = kv.BF16_NAN          # a head of NaN only
    check(c, None)


def test_unusual_old_scale():
    """A page scaled by the user (not a power of two): kept while large enough."""
    for old in (0.013, 3.7, 1e-30):
        c = kv.Case([(1, 9)], D=64, seed=6)
        for n in ("k", "v"):
            c.scales[n][c.table[0, 0]] = old
            c.codes[n][c.table[0, 0], :, :8] = kv.e4m3_round(
                np.clip(20 * c.rng.normal(size=(2, 8, 64)), -448, 448))
        c.upload()
        c.append(None)
        torch.cuda.synchronize()
        if old == 3.7:
            kv.assert_append(c, None, what=str(old))
        else:                       # older codes: within a step of the fp32 ratio's rounding
            got = c.dev["k_scale"].cpu().numpy()[c.table[0, 0]]
            assert (got >= np.float32(old)).all()


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_bad_batches(dtype):
    """Lengths below the rows or past the table, pages outside the pool, row
    ranges outside the step: only slots that exist are written."""
    c = kv.Case([(4, 20), (5, 30), (3, 40), (2, 18)], dtype=dtype, seed=8, tail=3, max_pages=3)
    c.kv_len[0] = 2                       # two rows at positions below 0
    c.kv_len[1] = 50                      # two rows past the page table (48)
    c.table[2, 2] = c.pages               # the page of sequence 2's rows
    c.table[3, 1] = -1
    check(c, kv.frequencies(64), what="bad lengths and pages")
    c = kv.Case([(4, 20)], dtype=dtype, seed=8)
    c.table[0, 1] = np.iinfo(np.int32).max
    check(c, kv.frequencies(64), what="huge page")
    c = kv.Case([(4, 20), (3, 9)], dtype=dtype, seed=8)
    c.upload()
    before = {n: c.dev[n].clone() for n in ("k", "v")}
    c.dev["q_start"].copy_(torch.tensor([-5, -2, -1], dtype=torch.int32))
    c.append(kv.frequencies(64))
    c.dev["q_start"].copy_(torch.tensor([900, 901, 902], dtype=torch.int32))
    c.append(kv.frequencies(64))
    c.dev["q_start"].copy_(torch.tensor([0, 4, 7], dtype=torch.int32))
    c.dev["kv_len"].copy_(torch.tensor([-3, np.iinfo(np.int32).min], dtype=torch.int32))
    c.append(kv.frequencies(64))
    torch.cuda.synchronize()
    for n in before:
        assert torch.equal(before[n].view(torch.uint8), c.dev[n].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_many_sequences(dtype):
    """More sequences than a wave has lanes, empty ones among them."""
    rng = np.random.default_rng(2)
    seqs = [(int(n), int(n + rng.integers(0, 60))) for n in rng.integers(0, 4, 200)]
    check(kv.Case(seqs, dtype=dtype, hq=2, hkv=1, seed=4, tail=1), kv.frequencies(64))


def test_twice_is_once():
    c = kv.Case(RAGGED, D=64, seed=11)
    f = kv.frequencies(64)
    check(c, f)
    first = {n: c.dev[n].clone() for n in ("k", "v", "k_scale", "v_scale", "out")}
    c.append(f)
    torch.cuda.synchronize()
    for n, t in first.items():
        assert torch.equal(t.view(torch.uint8), c.dev[n].view(torch.uint8)), n


@pytest.mark.parametrize("rows", [63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("dtype,D", [("fp8", 64), ("fp8", 256), ("bf16", 128)])
def test_row_counts_around_the_kernels_border(rows, dtype, D):
    check(kv.Case([(rows - 3, rows + 30), (3, 3)], P=128, D=D, hq=2, hkv=1, dtype=dtype, seed=rows),
          kv.frequencies(D))


def test_few_and_many_rows_agree():
    """The same rows in one long step and in short ones: the same cache and
    queries (bf16, where a row's bytes do not depend on its neighbours)."""
    f = kv.frequencies(128)
    long = kv.Case([(1500, 1600)], P=64, D=128, hq=4, hkv=2, dtype="bf16", seed=71).upload()
    long.append(f)
    torch.cuda.synchronize()
    want = {n: long.dev[n].clone() for n in ("k", "v", "out")}
    short = kv.Case([(1500, 1600)], P=64, D=128, hq=4, hkv=2, dtype="bf16", seed=71).upload()
    freq = torch.from_numpy(f).cuda()
    for at in range(0, 1500, 60):
        q0 = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
        n = torch.tensor([100 + at + 60], dtype=torch.int32, device="cuda")
        batch = sg.make_batch(q0, n, short.dev["table"], 60)
        sg.kv_append(short.cache, batch, short.dev["qkv"][at:at + 60], freq,
                     short.dev["out"][at:at + 60])
    torch.cuda.synchronize()
    for name, t in want.items():
        assert torch.equal(t.view(torch.uint8), short.dev[name].view(torch.uint8)), name


def test_graph_replays_and_streams():
    """Captured once, replayed with other lengths, rows and pages; and run on a
    stream of its own."""
    f = kv.frequencies(64)
    c = kv.Case([(2, 30), (3, 40)], seed=12, max_pages=8, spare=8).upload()
    freq = torch.from_numpy(f).cuda()
    call = lambda stream=None: sg.kv_append(c.cache, c.batch, c.dev["qkv"], freq, c.dev["out"],
                                            stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed, lens in ((13, (31, 41)), (14, (32, 64)), (15, (2, 3))):
        n = kv.Case([(2, lens[0]), (3, lens[1])], seed=seed, max_pages=8,
                    spare=c.pages - sum(-(-x // 16) for x in lens)).upload()
        for name in ("k", "v", "k_scale", "v_scale", "q_start", "kv_len", "table", "qkv"):
            c.dev[name].copy_(n.dev[name])
        c.dev["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        own, c_dev = n.dev, c.dev
        n.dev = {**own, **{k: c_dev[k] for k in ("k", "v", "k_scale", "v_scale", "out")}}
        kv.assert_append(n, f, what=f"replay {seed}")
        n.dev = own
        n.append(f, stream=side)
        torch.cuda.synchronize()
        kv.assert_append(n, f, what=f"stream {seed}")
