"""skinny_kv_attention's forms that the other tests pass by: four row waves at
head_dim 256, infinities and NaN at every head size, bad row ranges beside good
ones; and pages whose scale the caller chose."""
import numpy as np
import pytest
import torch

from tests import kv_util as kv
from tests.gpu_util import need_gpu
from tests.test_kv_attention_gpu import check, put

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("rows", [4, 5, 6, 8, 9, 16])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 2), (9, 1)])
def test_rows_of_wide_heads(dtype, rows, hq, hkv):
    """32 rows under a KV head are two row waves, 33 to 64 four, more are several
    row groups."""
    check(kv.Case([(rows, rows), (rows, rows + 1), (rows, 130), (rows, 777)], hq=hq, hkv=hkv, D=256,
                  P=32, dtype=dtype, seed=rows))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_prompts_of_wide_heads(dtype):
    check(kv.Case([(70, 70), (90, 400), (1, 30)], hq=4, hkv=1, D=256, dtype=dtype, seed=70, tail=3))
    check(kv.Case([(20, 20)], hq=8, hkv=2, D=256, P=64, dtype=dtype, seed=71))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("length", [6007, 12000])
def test_verify_rows_of_wide_heads_split_and_joined(dtype, length):
    check(kv.Case([(6, length), (7, 900), (5, 33)], hq=8, hkv=1, D=256, P=64, dtype=dtype, seed=72))


@pytest.mark.parametrize("dtype,pages", [("fp8", 2), ("fp8", 3), ("bf16", 2), ("bf16", 3)])
def test_short_verify_rows_of_wide_heads(dtype, pages):
    """Page tables of 32 and 48 positions: items stay whole, or just do not."""
    check(kv.Case([(6, 6), (6, 16 * pages), (5, 19), (7, 32)], hq=8, hkv=1, D=256, P=16, dtype=dtype,
                  seed=73, max_pages=pages))


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("rows", [1, 3, 6, 40])
def test_nonfinite_values_at_every_head_size(dtype, D, rows):
    """NaN and infinities reach the rows that see them and no other, in the last
    tile, behind earlier rows' masks, and in tiles that all rows see."""
    nan = kv.BF16_NAN if dtype == "bf16" else kv.E4M3_NAN
    for name in ("k", "v"):
        for back in (0, rows // 2, rows + 3, 150):
            c = kv.Case([(rows, 200), (1, 60)], hq=8, hkv=2, D=D, dtype=dtype, seed=74)
            put(c, name, 0, 199 - back, 1, slice(D - 9, D - 5), nan)
            check(c, what=f"{name} back {back}")
    if dtype == "bf16":
        for back in (0, rows // 2, 150):
            c = kv.Case([(rows, 200)], hq=8, hkv=2, D=D, dtype=dtype, seed=75)
            put(c, "v", 0, 199 - back, 0, slice(0, 3), kv.BF16_INF)
            put(c, "v", 0, 199 - back, 0, slice(D - 12, D - 9), kv.BF16_INF | 0x8000)
            check(c, what=f"inf back {back}")


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_descending_row_ranges(dtype):
    """q_start 0, 7, 3 in a step of 9 rows: sequence 0 has rows 0 to 6, sequence 1
    none, and rows 7 and 8 are left as they were."""
    c = kv.Case([(7, 20), (2, 9)], hq=4, hkv=2, D=64, dtype=dtype, seed=76)
    c.upload()
    c.dev["q_start"].copy_(torch.tensor([0, 7, 3], dtype=torch.int32))
    got = c.attend()
    torch.cuda.synchronize()
    want, tol, _ = kv.attention_oracle(c)
    got = got.float().cpu().double().numpy()
    assert (np.abs(got - want) <= tol)[:7].all() and np.isnan(got[7:]).all()


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("old", [0.013, 3.7, 1e-30, 2.0 ** -70, 1e30])
def test_pages_of_a_callers_scale(old, rows):
    """kv_append behind codes of any scale: both scales and every code, where the
    scale grows and where it stays."""
    c = kv.Case([(rows, 8 + rows)] * 2, D=64, seed=77)
    for n in ("k", "v"):
        for s in range(2):
            c.scales[n][c.table[s, 0]] = old
            c.codes[n][c.table[s, 0], :, :8] = kv.e4m3_round(
                np.clip(120 * c.rng.normal(size=(2, 8, 64)), -448, 448))
    c.upload()
    c.append(None)
    torch.cuda.synchronize()
    kv.assert_append(c, None, what=str(old))
