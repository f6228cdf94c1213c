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


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("seqs,hq,hkv,D", [([(1, 3), (1, 7), (2, 40)], 8, 2, 64),
                                           ([(6, 9), (6, 500)], 16, 2, 128),
                                           ([(12, 12), (3, 6000)], 8, 1, 256),
                                           ([(1, 20000)], 8, 1, 128)])
def test_probabilities_keep_16_bits(dtype, seqs, hq, hkv, D):
    """The output's own rounding is the only one to 8 bits.  With p held to 2^-16
    of itself (bf16 of p and of the rest), scores as in the oracle's bound, and A
    = sum p |v|: |err| <= 2^-8 |out| + (2^-16 + 4 (D + 4) 2^-24 max|q||k| + 2 (L +
    64) 2^-24) A, and 1e-3 of the rounding for what it does to a rounded error."""
    c = kv.Case(seqs, hq=hq, hkv=hkv, D=D, P=32, dtype=dtype, seed=62)
    # Short keys and queries: what the scores' fp32 sums may lose stays below 2^-14.
    c.q = kv.bf16_round(0.25 * kv.bf16_values(c.q))
    if dtype == "bf16":
        k = kv.bf16_values(c.codes["k"])
        c.codes["k"] = np.where(np.isnan(k), c.codes["k"], kv.bf16_round(0.25 * k)).astype(np.uint16)
    else:
        c.scales["k"] *= np.float32(0.25)
    got = attend(c)
    want, rough, _ = kv.attention_oracle(c)
    vals = {n: c.values(n) for n in ("k", "v")}
    G, worst = hq // hkv, 0.0
    for s in range(len(seqs)):
        n, length = seqs[s]
        ids = c.table[s, :-(-length // c.P)]
        kk, vv = (vals[x][ids].transpose(1, 0, 2, 3).reshape(hkv, -1, D)[:, :length] for x in ("k", "v"))
        q = kv.bf16_values(c.q).reshape(c.T, hq, D)
        for r in range(n):
            end = length - n + r + 1
            for h in range(hq):
                row, k, v = q[c.q_start[s] + r, h], kk[h // G][:end], vv[h // G][:end]
                p = np.exp(D ** -0.5 * (k @ row))
                p /= p.sum()
                big = D ** -0.5 * (np.abs(k) @ np.abs(row)).max()
                rel = 2.0 ** -16 + 4 * (D + 4) * kv.ULP32 * big + 2 * (end + 64) * kv.ULP32
                at = slice(h * D, (h + 1) * D)
                out = want[c.q_start[s] + r, at]
                tol = 1.001 * kv.HALF_BF16 * np.abs(out) + 1.01 * rel * (p @ np.abs(v)) + 1e-30
                worst = max(worst, np.max(np.abs(got[c.q_start[s] + r, at] - out) / tol))
    assert worst <= 1.0, worst


def odd_scale(seqs, count, seed, scale, codes, row):
    """`seqs` sequences of `count` rows each behind 8 older ones in their pages;
    scale(s, h), codes(s, h) and row(s, h) give a page's scale, its older codes
    and its new values (for k and v alike)."""
    c = kv.Case([(count, 8 + count)] * seqs, D=64, hq=2, hkv=2, seed=seed, x_sigma=0.5)
    x = c.qkv.reshape(c.T, 6, 64)
    for s in range(seqs):
        page = c.table[s, 0]
        for h in range(2):
            for n, lo in (("k", 2), ("v", 4)):
                c.scales[n][page, h] = scale(s, h)
                c.codes[n][page, h, :8] = codes(s, h)
                x[s * count:(s + 1) * count, lo + h] = kv.bf16_round(row(s, h))
    return c


MIDDLES = (kv.E4M3[8:126] + kv.E4M3[9:127]) / 2         # half way between two codes


@pytest.mark.parametrize("count", [1, 3])
@pytest.mark.parametrize("seqs", [15, 100])               # the kernels of few and of many rows
def test_older_codes_of_any_scale_are_rounded_once(seqs, count):
    """A page's scale that is no power of two grows: older codes land next to the
    middle between two codes, nearer to it than fp32 can tell."""
    rng = np.random.default_rng(63)
    code = rng.integers(32, 127, (seqs, 2))
    middle = np.empty((seqs, 2))
    for i in np.ndindex(seqs, 2):
        r = MIDDLES / kv.E4M3[code[i]]
        middle[i] = rng.choice(MIDDLES[(r > 0.3) & (r < 0.99)])
    had = (middle / kv.E4M3[code]).astype(np.float32)
    c = odd_scale(seqs, count, 63, lambda s, h: had[s, h],
                  lambda s, h: np.where(rng.random((8, 64)) < 0.7, code[s, h],
                                        rng.integers(0, 127, (8, 64))).astype(np.uint8),
                  lambda s, h: np.full(64, 448.0))        # needs a scale of 1
    c.upload()
    c.append(None)
    torch.cuda.synchronize()
    kv.assert_append(c, None)
    assert (c.dev["k_scale"].cpu().numpy()[c.table[:, 0]] == 1.0).all()


@pytest.mark.parametrize("count", [1, 3])
@pytest.mark.parametrize("seqs", [15, 100])
def test_new_codes_of_any_scale_are_rounded_once(seqs, count):
    """A page's scale that is no power of two stays: values next to the middle
    between two codes after the division, and exactly there."""
    rng = np.random.default_rng(64)
    x = kv.bf16_values(rng.integers(0x3F80, 0x4080, (seqs, 2)).astype(np.uint16))      # 1 .. 4
    middle = rng.choice(MIDDLES[(MIDDLES > 0.02) & (MIDDLES < 200)], (seqs, 2))
    had = (x / middle).astype(np.float32)
    for s in range(0, seqs, 3):                           # exact ties: 3 * middle is a bf16 number
        had[s], x[s] = 3.0, 3 * middle[s]
    c = odd_scale(seqs, count, 64, lambda s, h: had[s, h], lambda s, h: np.full((8, 64), 0x30, np.uint8),
                  lambda s, h: x[s, h] * rng.choice([-1.0, 1.0, 0.5], 64))
    c.upload()
    c.append(None)
    torch.cuda.synchronize()
    kv.assert_append(c, None)
    assert np.array_equal(c.dev["v_scale"].cpu().numpy()[c.table[:, 0]], had)


@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
@pytest.mark.parametrize("seqs", [1, 80])                 # the kernels of few and of many rows
def test_rotations_past_the_largest_number(seqs, dtype):
    """Two values of bf16's largest number turned by 3 pi / 4: one becomes 1.41
    times that, which is an infinity like any other."""
    freq = np.zeros(32, np.float32)
    freq[5] = np.pi / 4
    c = kv.Case([(1, 4)] * seqs, D=64, hq=2, hkv=1, dtype=dtype, seed=65)
    x = c.qkv.reshape(c.T, 4, 64)
    x[:, :3, 5] = x[:, :3, 37] = 0x7F7F
    c.upload()
    q = c.append(freq).float().cpu().double().numpy().reshape(c.T, 2, 64)
    torch.cuda.synchronize()
    assert (q[:, :, 5] == -np.inf).all() and np.isfinite(np.delete(q, 5, axis=2)).all()
    k = kv.bf16_values(x[:, 2])
    top = 0.0
    for r in range(c.T):
        turned = kv.rotate(k[r], 3, freq, False)
        assert turned[5] < -np.finfo(np.float32).max
        top = max(top, np.abs(np.delete(turned, 5)).max())
    got = c.dev["k"].cpu().view(torch.int16 if dtype == "bf16" else torch.uint8).numpy()
    got = got.astype(np.int64)[c.table[:, 0], 0, 3]
    if dtype == "bf16":
        assert (got[:, 5] & 0xFFFF == kv.BF16_INF | 0x8000).all()
        return
    assert (got[:, 5] == 0xFE).all()                      # -448
    scale = c.dev["k_scale"].cpu().numpy()[c.table[:, 0], 0]
    old = c.scales["k"][c.table[:, 0], 0]
    assert np.array_equal(scale, np.maximum(old, np.float32(kv.pow2_scale(top))))
