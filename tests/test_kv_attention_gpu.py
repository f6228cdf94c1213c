"""skinny_kv_attention against its 64-bit form: both cache types, head sizes and
groups, lengths around every boundary, ragged batches with empty sequences, NaN
and infinities in places that a row does not see, bad batches, and the ways a
program runs it (streams, graphs, threads of work on one workspace)."""
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


def check(c, scale=None, what=""):
    got = c.upload().attend(scale=scale)
    torch.cuda.synchronize()
    return kv.assert_attention(c, got, scale, what)


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 128])
def test_lengths(dtype, D, P):
    check(kv.Case([(1, n) for n in EDGES], P=P, D=D, dtype=dtype, seed=D, tail=1))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 6, 7, 11, 16])
@pytest.mark.parametrize("hq,hkv,D", [(8, 1, 128), (16, 2, 64), (4, 2, 256)])
def test_rows(dtype, rows, hq, hkv, D):
    """One to sixteen rows per sequence: every count of row tiles and groups."""
    check(kv.Case([(rows, rows), (rows, rows + 1), (rows, 130), (rows, 777)], hq=hq, hkv=hkv, D=D,
                  P=32, dtype=dtype, seed=rows))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 5), (12, 4), (17, 1), (64, 8), (40, 1)])
def test_groups(hq, hkv):
    check(kv.Case([(1, 90), (4, 300)], hq=hq, hkv=hkv, D=64, seed=hq))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_ragged(dtype):
    seqs = [(0, 100), (1, 1), (9, 9), (1, 0), (2, 1500), (0, 0), (5, 77), (1, 2049), (3, 2), (30, 40)]
    check(kv.Case(seqs, hq=8, hkv=2, D=64, dtype=dtype, seed=21, tail=4))


@pytest.mark.parametrize("dtype,D", [("fp8", 128), ("bf16", 128), ("fp8", 64), ("bf16", 256)])
def test_long(dtype, D):
    """Split over many workgroups and joined."""
    check(kv.Case([(1, 20011)], hq=8, hkv=1, D=D, P=64, dtype=dtype, seed=D))
    check(kv.Case([(6, 9000), (2, 123), (1, 4097)], hq=8, hkv=1, D=D, P=16, dtype=dtype, seed=D))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_prompt(dtype):
    """Hundreds of rows, their causal triangle among the keys."""
    check(kv.Case([(200, 200), (90, 400)], hq=4, hkv=2, D=64, dtype=dtype, seed=23))
    check(kv.Case([(70, 100)], hq=8, hkv=1, D=128, dtype=dtype, seed=24))


@pytest.mark.parametrize("seqs", [3, 70])
@pytest.mark.parametrize("wider", [0, 1])
@pytest.mark.parametrize("dtype,D,tiles", [("fp8", 64, 4), ("fp8", 128, 4), ("fp8", 256, 2),
                                           ("bf16", 64, 4), ("bf16", 128, 2), ("bf16", 256, 1)])
def test_whole_items(dtype, D, tiles, wider, seqs):
    """Both sides of the page table's width up to which items stay whole, and
    more items than workgroups."""
    keys = tiles * 32 * (4 if D == 256 else 8)
    lens = [(1, keys), (2, 3), (1, keys - 37)]
    lens += [(int(i % 7 > 0), 1 + 7 * i % keys) for i in range(seqs - 3)]
    check(kv.Case(lens, P=16, hq=8, hkv=4, D=D, dtype=dtype, seed=D + seqs,
                  max_pages=keys // 16 + wider))


def test_many_sequences():
    rng = np.random.default_rng(5)
    seqs = [(int(n), int(n + rng.integers(0, 200))) for n in rng.integers(0, 3, 150)]
    check(kv.Case(seqs, hq=2, hkv=1, seed=25))


def test_peaked_and_flat():
    """Scores far apart (one key takes all) and all equal."""
    c = kv.Case([(2, 700)], D=128, seed=26)
    c.q = kv.bf16_round(30 * kv.bf16_values(c.q))
    check(c, what="peaked")
    c = kv.Case([(2, 700)], D=128, seed=26)
    check(c, scale=0.0, what="flat")
    check(c, scale=-0.3, what="negative scale")


def test_unusual_scales():
    """Page scales that are no powers of two, from 2^-40 to 2^30."""
    c = kv.Case([(3, 300)], D=64, seed=27)
    c.scales["k"] = (c.scales["k"] * c.rng.uniform(0.3, 3.0, c.scales["k"].shape)).astype(np.float32)
    c.scales["v"] = (c.scales["v"] * np.exp2(c.rng.uniform(-32, 38, c.scales["v"].shape))).astype(np.float32)
    check(c)


def put(c, name, s, pos, heads, cols, value):
    """Write a code (bf16 or e4m3) into the cache at a position of a sequence."""
    c.codes[name][c.table[s, pos // c.P], heads, pos % c.P, cols] = value


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("rows", [1, 6, 40])
def test_nonfinite_keys_and_values(dtype, rows):
    """NaN and infinities reach the rows that see them and no other: a later
    row's key or value (behind an earlier row's mask), and a shared one."""
    nan = kv.BF16_NAN if dtype == "bf16" else kv.E4M3_NAN
    for name in ("k", "v"):
        for back in (0, rows // 2, rows + 3, 150):
            c = kv.Case([(rows, 200), (1, 60)], hq=8, hkv=2, D=64, dtype=dtype, seed=28)
            put(c, name, 0, 199 - back, 1, slice(5, 9), nan)
            check(c, what=f"{name} back {back}")
    if dtype == "bf16":
        for back in (0, rows // 2, 150):
            c = kv.Case([(rows, 200)], hq=8, hkv=2, D=64, dtype=dtype, seed=29)
            put(c, "v", 0, 199 - back, 0, slice(0, 3), kv.BF16_INF)
            put(c, "v", 0, 199 - back, 0, slice(9, 12), kv.BF16_INF | 0x8000)
            check(c, what=f"inf back {back}")
    else:
        c = kv.Case([(rows, 200)], P=16, hq=8, hkv=2, D=64, dtype=dtype, seed=29)
        for name in ("k", "v"):            # the scale of the last page, which early rows do not see
            c.scales[name][c.table[0, 199 // 16], 1] = np.nan
        check(c, what="NaN scale")


def test_nan_query():
    c = kv.Case([(3, 100)], hq=8, hkv=2, D=64, seed=30)
    c.q.reshape(3, 8, 64)[1, 5, 7] = kv.BF16_NAN
    check(c)


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_bad_batches(dtype):
    c = kv.Case([(2, 300), (3, 100), (1, 70)], dtype=dtype, P=16, seed=31, max_pages=10)
    c.table[0, 3] = -1
    c.table[0, 7] = c.pages
    c.table[1, :] = np.iinfo(np.int32).max           # no page at all
    c.kv_len[2] = -4
    check(c, what="pages and lengths")               # kv_len 300 > 160: cut to the table
    c = kv.Case([(4, 20), (3, 9)], dtype=dtype, seed=8)
    c.upload()
    c.dev["q_start"].copy_(torch.tensor([900, -5, -1], dtype=torch.int32))
    got = c.attend()
    torch.cuda.synchronize()
    assert torch.isnan(got).all()                    # no rows
    c.dev["q_start"].copy_(torch.tensor([0, 7, 3], dtype=torch.int32))
    c.attend()                                       # descending: sequence 1 has no rows
    torch.cuda.synchronize()


@pytest.mark.parametrize("case", [dict(seqs=[(1, 9001)], hq=8, hkv=1, D=128),
                                  dict(seqs=[(6, 500), (1, 1200)], hq=16, hkv=2, D=64),
                                  dict(seqs=[(3, 700)], hq=8, hkv=2, D=256, dtype="bf16")])
def test_workspace_is_enough_and_results_repeat(case):
    c = kv.Case(**case, seed=32).upload()
    n = sg.kv_attention_workspace_bytes(c.cache, c.batch, c.hq)
    full = torch.full((n + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    first = c.attend(full[:n]).clone()
    torch.cuda.synchronize()
    assert bool((full[n:] == 0xA5).all())
    for fill in (0x00, 0xFF):
        full[:n].fill_(fill)
        assert torch.equal(first.view(torch.int16), c.attend(full[:n]).view(torch.int16))
    with pytest.raises(sg.SkinnyError, match="WORKSPACE"):
        c.attend(full[:n - 1])


def test_graphs_share_a_workspace():
    """Two captured graphs on one workspace, replayed in turn with eager calls
    and new lengths between: every replay equals the eager call."""
    a = kv.Case([(1, 5000)], hq=8, hkv=1, D=128, P=64, seed=33, max_pages=90, spare=20).upload()
    b = kv.Case([(6, 3000), (2, 40)], hq=8, hkv=1, D=128, P=64, seed=34).upload()
    n = max(c.workspace().numel() for c in (a, b))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.attend(ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.attend(ws)
        graphs.append(g)
    for turn in range(4):
        a.kv_len[0] = (5000, 17, 1300, 4999)[turn]
        a.dev["kv_len"].copy_(torch.from_numpy(a.kv_len))
        for c, g in zip((a, b), graphs):
            c.dev["out"].fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            got = c.dev["out"].clone()
            kv.assert_attention(c, got, what=f"turn {turn}")
            c.attend(ws)
            torch.cuda.synchronize()
            assert torch.equal(got.view(torch.int16), c.dev["out"].view(torch.int16))


def test_streams_with_own_workspaces():
    cases = [kv.Case([(1, 3000 + 700 * i)], hq=8, hkv=1, D=128, seed=40 + i).upload() for i in range(3)]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [c.workspace() for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, w in zip(cases, streams, spaces):
            c.attend(w, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        kv.assert_attention(c, c.dev["out"])


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: the sequence's pages lie at its end."""
    P, D, hkv = 64, 128, 8
    pages = (1 << 32) // (P * D * hkv) + 40
    small = kv.Case([(2, 500)], P=P, D=D, hq=16, hkv=hkv, seed=50)
    small.upload()
    k = torch.empty((pages, hkv, P, D), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.full((pages, hkv), float("nan"), device="cuda")
    vs = torch.full_like(ks, float("nan"))
    n = small.pages
    for big, name in ((k, "k"), (v, "v"), (ks, "k_scale"), (vs, "v_scale")):
        big[pages - n:] = small.dev[name]
    small.dev["table"] += pages - n                  # -7 entries stay unused
    small.cache = sg.make_kv_cache(k, v, ks, vs)
    got = small.attend()
    torch.cuda.synchronize()
    kv.assert_attention(small, got)
    f = kv.frequencies(D)
    small.append(f)
    torch.cuda.synchronize()
    for big, name in ((k, "k"), (v, "v"), (ks, "k_scale"), (vs, "v_scale")):
        small.dev[name] = big[pages - n:]
    kv.assert_append(small, f)
