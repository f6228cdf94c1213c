"""skinny_kv_attention and skinny_kv_append where fewer bits, or a number that is
no finite one, could show: against the 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import kv_util as kv
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def attend(c):
    got = c.upload().attend()
    torch.cuda.synchronize()
    return got.float().cpu().double().numpy()


def aligned_queries(c, size):
    """Every row's query along the first value of each head, `size` long; keys
    then score by their own first value."""
    q = np.zeros((c.T, c.hq, c.D))
    q[:, :, 0] = size
    c.q = kv.bf16_round(q.reshape(c.T, -1))


def first_key_values(c, s, start, stop, value):
    """Sets value 0 of the keys at positions start .. stop - 1 of a sequence."""
    for pos in range(start, stop):
        c.codes["k"][c.table[s, pos // c.P], :, pos % c.P, 0] = kv.bf16_round([value])[0]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,length", [(1, 200), (6, 300), (40, 200), (2, 9000)])
def test_infinite_values_of_small_probability(D, rows, length):
    """A seen value of +-inf gives that infinity however small its probability:
    here e^-200, which is no fp32 number, in tiles that every row sees and in
    tiles with a mask."""
    for back in (0, rows + 3, length - 10):
        c = kv.Case([(rows, length), (1, 50)], hq=8, hkv=2, D=D, dtype="bf16", seed=60 + D)
        aligned_queries(c, D ** 0.5)
        first_key_values(c, 0, 0, length, 0.0)
        pos = length - 1 - back
        first_key_values(c, 0, pos, pos + 1, -200.0)
        put = c.codes["v"][c.table[0, pos // c.P], :, pos % c.P]
        put[:, 1], put[:, D - 1] = kv.BF16_INF, kv.BF16_INF | 0x8000
        got = attend(c)
        want, tol, _ = kv.attention_oracle(c)
        assert np.isinf(want).any()
        assert np.array_equal(np.isnan(got), np.isnan(want)), f"NaN, {back} back"
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf]), f"infinities, {back} back"
        ok = np.isfinite(want)
        assert (np.abs(got - want)[ok] <= tol[ok]).all(), f"the rest, {back} back"
