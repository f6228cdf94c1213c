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


@pytest.mark.parametrize("rows,length,finite", [(1, 20, []), (1, 300, []), (7, 300, []), (1, 9000, []),
                                                (1, 300, [5]), (1, 300, [299]), (1, 9000, [4500]),
                                                (3, 9000, [8998])])
def test_scores_of_minus_infinity(rows, length, finite):
    """Scores of -inf take no part where a row has a finite one; a row with no
    other scores is 0 / 0 (zeros are for rows that see no position)."""
    c = kv.Case([(rows, length), (2, 33)], hq=4, hkv=2, D=64, dtype="bf16", seed=61)
    aligned_queries(c, 1.0)
    first_key_values(c, 0, 0, length, -np.inf)
    for pos in finite:
        first_key_values(c, 0, pos, pos + 1, 0.5)
    got = attend(c)
    v = c.values("v")
    for r in range(rows):
        end = length - rows + r + 1
        seen = [p for p in finite if p < end]
        for h in range(c.hq):
            row = got[r, h * c.D:(h + 1) * c.D]
            if not seen:
                assert np.isnan(row).all(), f"row {r}"
            else:
                pos = seen[0]
                assert np.array_equal(row, v[c.table[0, pos // c.P], h // 2, pos % c.P]), f"row {r}"
    want, tol, _ = kv.attention_oracle(c)                # the other sequence
    assert (np.abs(got - want) <= tol)[rows:].all()
