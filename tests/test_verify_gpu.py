"""skinny_verify_draft against its definition in 64 bits: tokens and counts are
whole numbers and have to be equal.  Vocabularies around the slice size and the
full one, both logit types, aligned and not, ragged and empty sequences, greedy
and sampled, with and without a draft distribution, masks, NaN and infinities."""
import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BELOW_ONE = np.float32(1) - np.float32(2.0 ** -24)


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def softmax(l, t):
    """p of one row; t <= 0 or NaN: one at the lowest largest; NaN as -inf."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    p = np.zeros_like(l)
    top = l.max()
    if top == -np.inf:
        return p
    if not t > 0:
        p[int(np.argmax(l))] = 1.0
        return p
    with np.errstate(invalid="ignore"):
        e = np.where(l == top, 1.0, np.exp((l - top) / np.float64(t)))
    return e / e.sum()


def oracle(c):
    V, out, accepted = c["logits"].shape[1], c["out"].copy(), []
    for s in range(len(c["sample_u"])):
        lo, hi = c["q_start"][s], c["q_start"][s + 1]
        t = 1.0 if c["temperature"] is None else c["temperature"][s]
        kept = 0
        out[lo:hi] = -1
        for r in range(lo, hi):
            p = softmax(c["logits"][r], t)
            w = p
            if r + 1 < hi:
                d = c["tokens"][r + 1]
                q = np.zeros(V)
                if c["draft"] is not None and t > 0:
                    q = softmax(c["draft"][r], t)
                elif 0 <= d < V:
                    q[d] = 1.0
                if 0 <= d < V and np.float64(c["accept_u"][r]) * q[d] < p[d]:
                    out[r] = d
                    kept += 1
                    continue
                w = np.maximum(p - q, 0.0)
                w = w if w.sum() > 0 else p
            sums = np.cumsum(w)
            u = np.float64(c["sample_u"][s])
            if not t > 0 or sums[-1] == 0:
                out[r] = int(np.argmax(w))
            else:
                first = int(np.searchsorted(sums, (u if u > 0 else 0.0) * sums[-1], side="right"))
                out[r] = min(first, int(np.nonzero(w)[0][-1]))
            break
        accepted.append(kept)
    return out, np.array(accepted)


def case(rows, V, dtype="bf16", draft=True, seed=0, tail=0, temps=None, close=0.5):
    rng = np.random.default_rng(seed)
    q_start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    T, S = int(q_start[-1]) + tail, len(rows)
    l = 2.5 * rng.normal(size=(T, V))
    l[np.arange(T), rng.integers(0, V, T)] += 2.5 + np.log(V)
    dl = l + close * rng.normal(size=(T, V))

    def rounded(x):
        x = torch.from_numpy(x)
        return (x.to(torch.bfloat16) if dtype == "bf16" else x).float().numpy()

    l, dl = rounded(l), rounded(dl)
    drawn = np.array([rng.choice(V, p=softmax(x, 0.8)) for x in dl])
    return dict(q_start=q_start, logits=l, draft=dl if draft else None,
                tokens=np.roll(drawn, 1).astype(np.int32), dtype=dtype,
                temperature=None if temps is None else np.resize(temps, S).astype(np.float32),
                accept_u=rng.random(T).astype(np.float32),
                sample_u=rng.random(S).astype(np.float32), out=np.full(T, -9, np.int32))


def upload(c, offset=0):
    T, V = c["logits"].shape

    def dev(x, dt):
        if x is None:
            return None
        flat = torch.zeros(x.size + offset, dtype=dt, device="cuda")
        flat[offset:] = torch.from_numpy(x.reshape(-1).copy()).to(dt).cuda()
        return flat[offset:].view(*x.shape)

    L = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    d = {n: dev(c[n], L) for n in ("logits", "draft")}
    d.update({n: dev(c[n], torch.int32) for n in ("q_start", "tokens", "out")})
    d.update({n: dev(c[n], torch.float32) for n in ("accept_u", "sample_u", "temperature")})
    d["accepted"] = torch.full((len(c["sample_u"]),), -5, dtype=torch.int32, device="cuda")
    d["ws"] = torch.full((sg.verify_workspace_bytes(T, len(c["sample_u"]), V),), 0xFF,
                         dtype=torch.uint8, device="cuda")
    return d


def run(d, ws=None, stream=None):
    sg.verify_draft(d["q_start"], d["logits"], d["tokens"], d["accept_u"], d["sample_u"], d["out"],
                    d["accepted"], d["ws"] if ws is None else ws, draft_logits=d["draft"],
                    temperature=d["temperature"], stream=stream)


def check(c, offset=0, what=""):
    d = upload(c, offset)
    run(d)
    torch.cuda.synchronize()
    compare(c, d, what)
    return d


def compare(c, d, what=""):
    out, accepted = oracle(c)
    assert d["accepted"].tolist() == accepted.tolist(), what
    assert d["out"].tolist() == out.tolist(), what


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 1000, 4095, 4096, 4097, 32003, 152064])
def test_vocabularies(dtype, draft, V):
    for seed in range(3):
        check(case([6, 1, 3], V, dtype, draft, seed=seed, temps=[0.8, 1.0, 0.0]), what=str(seed))


@pytest.mark.parametrize("V,rows", [(2047, 3), (2048, 3), (2049, 3), (131072, 16), (131073, 3),
                                    (131080, 3), (20480, 102), (20480, 103)])
def test_slices(V, rows):
    """Vocabularies around a slice's end, and both sides of each bound of the
    short slices' rule: 64 of a row, 1024 of all rows."""
    check(case([rows - 2, 2], V, seed=V + rows), what=f"{V} {rows}")


@pytest.mark.parametrize("dtype,offset", [("bf16", 1), ("bf16", 4), ("f32", 1)])
def test_unaligned(dtype, offset):
    check(case([4, 2], 5000, dtype, seed=3, temps=[0.7]), offset=offset)


@pytest.mark.parametrize("draft", [True, False])
def test_ragged(draft):
    rows = [1, 0, 16, 17, 2, 0, 40, 5, 1, 33]
    c = case(rows, 700, draft=draft, seed=4, tail=3, temps=[1.0, 0.5, 0.9, 0.8, 0.0], close=0.05)
    check(c)
    c["accept_u"][:] = 0.0                      # everything is kept: the bonus token of long rows
    check(c)


def test_many_sequences():
    rng = np.random.default_rng(6)
    check(case([int(n) for n in rng.integers(0, 4, 150)], 300, seed=6, temps=[0.9, 0.0, 1.3]))


@pytest.mark.parametrize("draft", [True, False])
def test_random_numbers_at_the_ends(draft):
    for au in (0.0, BELOW_ONE):
        for su in (0.0, BELOW_ONE, 0.5):
            c = case([4, 3, 1], 9000, draft=draft, seed=7)
            c["accept_u"][:], c["sample_u"][:] = au, su
            check(c, what=f"{au} {su}")


def test_temperatures():
    """No array, cold, hot, greedy ones (0, negative, NaN)."""
    check(case([3, 3], 5000, seed=8))
    check(case([3] * 6, 5000, seed=9, temps=[0.02, 5.0, 0.0, -1.0, np.nan, 100.0]))


def test_masked_logits():
    """-inf nearly everywhere, a row with nothing, NaN (as -inf), +inf, the
    type's lowest number; drafts outside what is left."""
    for draft in (True, False):
        c = case([4, 4, 4, 4, 4], 10000, "f32", draft, seed=10, temps=[0.9])
        l = c["logits"]
        l[0:4, 100:] = -np.inf
        l[1, :] = -np.inf
        l[1, 4096] = 3.0
        l[4:6] = -np.inf
        l[8:12, ::3] = np.nan
        l[9] = np.nan
        l[12, [5000, 7000]] = np.inf
        l[14, 9999] = np.inf
        l[16:20, 200:] = np.finfo(np.float32).min
        if draft:
            c["draft"][16, :] = -np.inf
            c["draft"][2, 50:] = -np.inf
        for au in (0.0, 0.5, BELOW_ONE):
            c["accept_u"][:] = au
            check(c, what=f"draft {draft} {au}")


def test_drafts_outside_the_vocabulary():
    c = case([4, 4, 4], 3000, seed=11, temps=[0.9, 0.0, 1.0])
    c["tokens"][[1, 6, 10]] = [-1, 3000, np.iinfo(np.int32).max]
    c["accept_u"][:] = 0.0
    check(c)


def test_equal_distributions():
    """p = q: every draft with q(d) > 0 is kept; one drafted where q(d) = 0 is
    not, and the token then comes from p."""
    c = case([5, 5], 6000, seed=12, close=0.0)
    c["accept_u"][:] = BELOW_ONE
    check(c)
    for x in ("logits", "draft"):
        c[x][0, 17] = -np.inf
    c["tokens"][1] = 17
    d = check(c)
    assert d["accepted"].tolist()[0] == 0


def test_greedy_ties_take_the_lowest():
    c = case([2, 2, 1], 9000, seed=13, temps=[0.0])
    c["logits"][:] = 0.0
    c["logits"][0, [4097, 4096, 8999]] = 5.0
    c["logits"][2, [3, 8000]] = 5.0
    c["tokens"][[1, 3]] = [4096, 8000]
    d = check(c)
    assert d["out"].tolist()[2] == 3 and d["accepted"].tolist() == [1, 0, 0]


def test_every_token_in_turn():
    """A flat row: sample_u = (k + 1/2) / V gives token k."""
    V = 9000
    for k in (0, 1, 4095, 4096, 5000, 8191, 8192, 8999):
        c = case([1], V, "f32", seed=14)
        c["logits"][:] = 1.0
        c["sample_u"][:] = (k + 0.5) / V
        d = check(c)
        assert d["out"].tolist() == [k]


def test_bad_row_ranges():
    """Ranges outside the step or descending: nothing outside is touched."""
    c = case([3, 3], 5000, seed=15, tail=2)
    d = upload(c)
    for q in ([-9, -3, -1], [50, 60, 70]):
        d["q_start"].copy_(torch.tensor(q, dtype=torch.int32))
        run(d)
        torch.cuda.synchronize()
        assert d["out"].tolist() == [-9] * 8 and d["accepted"].tolist() == [0, 0]
    d["q_start"].copy_(torch.tensor([2, 8, 4], dtype=torch.int32))
    run(d)
    torch.cuda.synchronize()
    assert d["out"].tolist()[:2] == [-9, -9] and d["accepted"].tolist()[1] == 0


@pytest.mark.parametrize("temps", [[1.0, 1.0, 0.0], [0.0, 1.0, 1.0]])
def test_rows_of_two_sequences_give_tokens_of_the_vocabulary(temps):
    """Rows 2 and 3 belong to a sampling and to a greedy sequence; which of
    them writes last is open, but not what a token can be."""
    c = case([4, 0, 2], 5000, seed=21, temps=temps)
    d = upload(c)
    d["q_start"].copy_(torch.tensor([0, 4, 2, 6], dtype=torch.int32))
    run(d)
    torch.cuda.synchronize()
    assert all(-1 <= t < 5000 for t in d["out"].tolist())
    assert all(0 <= n <= 3 for n in d["accepted"].tolist())


def test_workspace_is_enough_and_results_repeat():
    c = case([6, 4, 1], 32003, seed=16, temps=[0.9])
    d = upload(c)
    n = d["ws"].numel()
    full = torch.full((n + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    for fill in (0x00, 0xFF, 0x7F):
        full[:n].fill_(fill)
        run(d, full[:n])
        torch.cuda.synchronize()
        compare(c, d)
        run(d, full[:n])                        # on what the last call left
        torch.cuda.synchronize()
        compare(c, d)
    assert bool((full[n:] == 0xA5).all())
    with pytest.raises(sg.SkinnyError, match="WORKSPACE"):
        run(d, full[:n - 1])


def test_graphs_share_a_workspace():
    cs = [case([6, 2], 20000, seed=17, temps=[0.8]), case([1, 1, 5], 20000, seed=18, draft=False)]
    ds = [upload(c) for c in cs]
    ws = torch.empty(max(d["ws"].numel() for d in ds), dtype=torch.uint8, device="cuda")
    graphs = []
    for d in ds:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(d, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(d, ws)
        graphs.append(g)
    rng = np.random.default_rng(0)
    for turn in range(5):
        for c, d, g in zip(cs, ds, graphs):
            for n in ("accept_u", "sample_u"):
                c[n][:] = rng.random(c[n].shape)
                d[n].copy_(torch.from_numpy(c[n]))
            d["out"].fill_(-9)
            g.replay()
            torch.cuda.synchronize()
            compare(c, d, f"turn {turn}")
            d["out"].fill_(-9)
            run(d, ws)
            torch.cuda.synchronize()
            compare(c, d, f"eager {turn}")


def test_streams_with_own_workspaces():
    cs = [case([5, 3], 50000, seed=20 + i, temps=[0.9]) for i in range(3)]
    ds = [upload(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s in zip(ds, streams):
            run(d, stream=s)
    torch.cuda.synchronize()
    for c, d in zip(cs, ds):
        compare(c, d)
