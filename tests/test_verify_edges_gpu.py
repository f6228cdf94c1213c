"""skinny_verify_draft where its contract ends: rows of the draft that it does not
ask for, drafts of vanishing probability, vocabularies of many trips."""
import ctypes

import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
from tests.gpu_util import need_gpu
from tests.test_verify_gpu import BELOW_ONE, case, check, compare, oracle, run, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,temps,asked", [([3, 2], [0.9, 0.7], 4), ([3, 4], [0.9, 0.0], 2),
                                              ([4], [1.0], 3), ([5, 1, 1], [0.8], 4)])
def test_rows_of_the_draft_that_are_not_asked(dtype, rows, temps, asked):
    """The last row of a sequence, greedy sequences' rows and rows of no sequence
    need no draft logits; here there are none behind the last row that is asked."""
    c = case(rows, 100003, dtype, seed=40, tail=2, temps=temps)
    d = upload(c)
    T, V = c["logits"].shape
    draft = d["draft"][:asked].clone()
    d["draft"] = None
    address = ctypes.c_void_p
    v = sg.Verify(sg.LOGITS_BF16 if dtype == "bf16" else sg.LOGITS_F32, V, T, len(rows),
                  *(address(t.data_ptr()) for t in (d["q_start"], d["logits"], draft, d["tokens"],
                                                    d["temperature"], d["accept_u"], d["sample_u"],
                                                    d["out"], d["accepted"])))
    assert sg.lib().skinny_verify_draft(v, d["ws"].data_ptr(), d["ws"].numel(), None) == 0
    torch.cuda.synchronize()
    compare(c, d)


@pytest.mark.parametrize("p_at,q_at,au,kept", [
    (-900, -901, BELOW_ONE, 1), (-901, -900, 0.499, 1), (-901, -900, 0.501, 0), (-999, -999, 0.999, 1),
    (-1001, -900, 0.0, 0), (-1001, -1002, 0.5, 0), (-999, -1002, BELOW_ONE, 1), (-20, -900, 0.5, 1)])
def test_drafts_far_below_the_largest(p_at, q_at, au, kept):
    """u q(d) < p(d) at a low temperature, by the ratio of two probabilities of
    2^p_at and 2^q_at; what lies below 2^-1000 is no probability, and is not kept."""
    t = np.float32(2e-3)
    c = case([2], 5000, "f32", seed=30, temps=[t])
    c["logits"][0], c["draft"][0] = -3.0, -3.0           # 2^-2164 and less
    c["logits"][0, 7] = c["draft"][0, 9] = 0.0           # p is 1 at 7, q is 1 at 9
    c["tokens"][1], c["accept_u"][0] = 4321, au
    for name, at in (("logits", p_at), ("draft", q_at)):
        c[name][0, 4321] = at * np.log(2.0) * np.float64(t)
    d = upload(c)
    run(d)
    torch.cuda.synchronize()
    assert d["accepted"].tolist() == [kept]
    assert d["out"].tolist()[0] == (4321 if kept else 7)
    # The same draft, given instead of drawn: q is 1, only a random number of 0 keeps it.
    for u in (0.0, 2.0 ** -22):
        d["accept_u"].fill_(u)
        d["draft"] = None
        run(d)
        torch.cuda.synchronize()
        assert d["accepted"].tolist() == [int(p_at > -1000 and u * 2.0 ** 500 < 2.0 ** (p_at + 500))]


def test_a_wait_that_gives_up_says_so():
    """A spin limit < 0, set from the host, makes every sampling sequence give up:
    -1 for its count and in all its places, nothing else, and the next call is
    as ever."""
    c = case([4, 2, 0, 3], 32003, seed=41, temps=[0.9, 0.0, 1.0, 0.7], tail=1)
    d = upload(c)
    sg.verify_set_spin_limit(-1)
    try:
        run(d)
        torch.cuda.synchronize()
    finally:
        sg.verify_set_spin_limit(1 << 16)
    out, accepted = oracle(c)
    out[[0, 1, 2, 3, 6, 7, 8]] = -1
    assert d["out"].tolist() == out.tolist()
    assert d["accepted"].tolist() == [-1, accepted[1], 0, -1]
    for _ in range(3):
        d["out"].fill_(-9)
        run(d)
        torch.cuda.synchronize()
        compare(c, d)


def check_rows(V, seed, **kw):
    c = case([3, 2, 1, 1], V, "f32", seed=seed, temps=[0.9, 0.7, 1.0, 0.0], **kw)
    check(c, what=f"{V}")
    return c


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [262144, 262145, 600001])
def test_vocabularies_of_several_trips(V, draft):
    """From 65 slices of 4096 entries on, a row's sums and a sequence's words take
    more than one trip."""
    c = check_rows(V, 50, draft=draft)
    for su in (0.0, 0.5, BELOW_ONE):
        c["sample_u"][:] = su
        check(c, what=f"{V} {su}")
        c["accept_u"][:] = 0.0 if su == 0.5 else BELOW_ONE
        check(c, what=f"{V} {su}")


@pytest.mark.parametrize("at", [0, 5, 262143, 262144, 400000, 524287, 524288, 600000])
def test_every_trip_gives_its_entry(at):
    """A flat row's entry at `at`; one that alone is above -inf, or infinite, there;
    and an infinity each in two trips."""
    V = 600001
    c = case([1, 1, 1, 1], V, "f32", seed=51, draft=False)
    l = c["logits"]
    l[0] = 1.0
    l[1] = -np.inf
    l[1, at] = -4.0
    l[2, at] = np.inf
    l[3, [7, at]] = np.inf
    c["sample_u"][:] = (at + 0.5) / V, 0.5, 0.5, 0.75
    d = check(c)
    assert d["out"].tolist() == [at, at, at, max(7, at)]


def test_several_trips_without_a_residual():
    """p = q, and a draft where both are 0: rejected, then drawn from p itself."""
    c = case([2, 2, 2], 600001, "f32", seed=52, close=0.0)
    for x in ("logits", "draft"):
        c[x][[0, 2, 4], 17] = -np.inf
    c["tokens"][[1, 3, 5]] = 17
    for su in (0.0, 0.3, 0.999, BELOW_ONE):
        c["sample_u"][:] = su
        d = check(c, what=str(su))
        assert d["accepted"].tolist() == [0, 0, 0]


def test_the_largest_vocabulary():
    c = case([1], 5, "f32", seed=53, draft=False)
    V = 1 << 24
    row = np.full((1, V), -np.inf, np.float32)
    for at in (0, 9000000, V - 1):
        row[:] = -np.inf
        row[0, at] = 1.5
        c["logits"] = row
        d = upload(c)
        run(d)
        torch.cuda.synchronize()
        assert d["out"].tolist() == [at] and d["accepted"].tolist() == [0]
