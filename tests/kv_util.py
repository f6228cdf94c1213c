"""Plain 64-bit forms of the paged-cache operators, on host arrays, and the
batches their tests run on."""
import numpy as np
import torch

import gemv_skinny_gemm_amd as sg

BF16_NAN, BF16_INF = 0x7FC0, 0x7F80
E4M3_NAN = 0x7F
HALF_BF16 = 2.0 ** -8            # torch.finfo(torch.bfloat16).eps / 2
ULP32 = 2.0 ** -24


def bf16_round(x):
    """float64 -> bf16 codes, to nearest even (through fp32 rounded to odd)."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        f = x.astype(np.float32)
        u = f.view(np.uint32).copy()
        back = f.astype(np.float64)
        move = np.isfinite(f) & (back != x) & ((u & 1) == 0)
        up = (np.abs(back) < np.abs(x))
        u = np.where(move & up, u + 1, np.where(move & ~up, u - 1, u)).astype(np.uint32)
    nan = np.isnan(x)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    r[nan] = BF16_NAN
    return r


def bf16_values(codes):
    return (np.ascontiguousarray(codes, np.uint16).astype(np.uint32) << 16).view(np.float32) \
        .astype(np.float64)


def _e4m3_table():
    c = np.arange(256)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(s == 1, -v, v)


E4M3 = _e4m3_table()
_POSITIVE = E4M3[:127]           # ascending


def e4m3_round(x):
    """float64 -> e4m3 codes: nearest, ties to the even code, beyond 448 the
    largest, NaN to 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == 0.0, 0, code) | (np.signbit(x).astype(np.int64) << 7)
    return np.where(np.isnan(x), E4M3_NAN, code).astype(np.uint8)


class Case:
    """A ragged batch over a pool with data everywhere: random numbers where a
    sequence's tokens are, and NaN in every other slot, scale and page.
    seqs: [(rows of this step, kv_len)]; `tail` rows belong to no sequence."""

    def __init__(self, seqs, P=16, hq=8, hkv=2, D=64, dtype="fp8", seed=0, tail=0, spare=3,
                 max_pages=None, x_sigma=2.0, poison=True):
        rng = np.random.default_rng(seed)
        self.rng, self.seqs, self.P, self.hq, self.hkv, self.D = rng, seqs, P, hq, hkv, D
        self.dtype = dtype
        rows = [n for n, _ in seqs]
        self.q_start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.kv_len = np.array([k for _, k in seqs], np.int32)
        self.T = int(self.q_start[-1]) + tail
        need = [-(-k // P) for _, k in seqs]
        self.max_pages = max(1, max(need)) + 1 if max_pages is None else max_pages
        need = [min(n, self.max_pages) for n in need]
        self.pages = sum(need) + spare
        ids = rng.permutation(self.pages)
        self.table = np.full((len(seqs), self.max_pages), -7, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        shape = (self.pages, hkv, P, D)
        self.codes, self.scales = {}, {}
        for name in ("k", "v"):
            if dtype == "bf16":
                c = bf16_round(rng.normal(size=shape))
                bad = BF16_NAN
            else:
                c = e4m3_round(np.clip(96 * rng.normal(size=shape), -448, 448))
                bad = E4M3_NAN
                self.scales[name] = (2.0 ** rng.integers(-8, -5, shape[:2])).astype(np.float32)
            if poison:
                keep = np.zeros((self.pages, P), bool)
                for s, (_, k) in enumerate(seqs):
                    for j in range(need[s]):
                        keep[self.table[s, j], :max(0, min(P, k - j * P))] = True
                c = np.where(keep[:, None, :, None], c, bad).astype(c.dtype)
                if dtype == "fp8":
                    self.scales[name][~keep.any(axis=1)] = np.nan
            self.codes[name] = c
        self.qkv = bf16_round(x_sigma * rng.normal(size=(self.T, (hq + 2 * hkv) * D)))
        self.q = bf16_round(rng.normal(size=(self.T, hq * D)))

    def position(self, s, i):
        return int(self.kv_len[s]) - int(self.q_start[s + 1] - self.q_start[s]) + i

    def upload(self):
        def bf(c):
            return torch.from_numpy(np.ascontiguousarray(c).view(np.int16)).view(torch.bfloat16).cuda()
        up = bf if self.dtype == "bf16" else (lambda c: torch.from_numpy(c.copy()).cuda())
        self.dev = {n: up(self.codes[n]) for n in ("k", "v")}
        for n in self.scales:
            self.dev[n + "_scale"] = torch.from_numpy(self.scales[n].copy()).cuda()
        for n in ("q_start", "kv_len", "table"):
            self.dev[n] = torch.from_numpy(getattr(self, n).copy()).cuda()
        self.dev["qkv"], self.dev["q"] = bf(self.qkv), bf(self.q)
        self.cache = sg.make_kv_cache(self.dev["k"], self.dev["v"], self.dev.get("k_scale"),
                                      self.dev.get("v_scale"))
        self.batch = sg.make_batch(self.dev["q_start"], self.dev["kv_len"], self.dev["table"], self.T)
        self.dev["out"] = torch.full((self.T, self.hq * self.D), float("nan"),
                                     dtype=torch.bfloat16, device="cuda")
        return self

    def workspace(self):
        return torch.empty(sg.kv_attention_workspace_bytes(self.cache, self.batch, self.hq),
                           dtype=torch.uint8, device="cuda")

    def attend(self, ws=None, scale=None, stream=None):
        sg.kv_attention(self.cache, self.batch, self.dev["q"], self.dev["out"],
                        self.workspace() if ws is None else ws, scale=scale, stream=stream)
        return self.dev["out"]

    def append(self, freq, interleaved=False, stream=None):
        f = None if freq is None else torch.from_numpy(freq).cuda()
        self.keep = f
        sg.kv_append(self.cache, self.batch, self.dev["qkv"], f, self.dev["out"],
                     interleaved=interleaved, stream=stream)
        return self.dev["out"]

    def values(self, name):
        if self.dtype == "bf16":
            return bf16_values(self.codes[name])
        return E4M3[self.codes[name]] * self.scales[name].astype(np.float64)[:, :, None, None]


def rotate(x, pos, freq, interleaved):
    """x [..., D] float64 at one position."""
    y = x.copy()
    n = len(freq)
    t = float(pos) * freq.astype(np.float64)
    c, s = np.cos(t), np.sin(t)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else \
        (slice(0, n), slice(n, 2 * n))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def pow2_scale(top):
    s = 2.0 ** -64
    while top > 448.0 * s:
        s *= 2
    return s


def append_oracle(c: Case, freq, interleaved=False):
    """What kv_append leaves: q rows (float64; None where none is written), and
    per pool the new codes, the scales and the 64-bit numbers that new rows
    were rounded from (NaN elsewhere)."""
    freq = np.zeros(0, np.float32) if freq is None else freq
    x = bf16_values(c.qkv).reshape(c.T, c.hq + 2 * c.hkv, c.D)
    q = np.full((c.T, c.hq, c.D), np.nan)
    wrote_q = np.zeros(c.T, bool)
    codes = {n: c.codes[n].copy() for n in ("k", "v")}
    scales = {n: c.scales[n].copy() for n in c.scales}
    source = {n: np.full(codes[n].shape, np.nan) for n in ("k", "v")}
    fresh = {n: np.zeros(codes[n].shape, bool) for n in ("k", "v")}
    for s in range(len(c.seqs)):
        places = {}
        for r in range(c.q_start[s], c.q_start[s + 1]):
            pos = c.position(s, r - c.q_start[s])
            q[r] = rotate(x[r, :c.hq], pos, freq, interleaved)
            wrote_q[r] = True
            if 0 <= pos < min(int(c.kv_len[s]), c.max_pages * c.P):
                places.setdefault(pos // c.P, []).append((pos % c.P, r, pos))
        for j, rows in places.items():
            page = c.table[s, j]
            if not 0 <= page < c.pages:
                continue
            slots = [a for a, _, _ in rows]
            for name, lo in (("k", c.hq), ("v", c.hq + c.hkv)):
                new = np.stack([x[r, lo:lo + c.hkv] if name == "v" else
                                rotate(x[r, lo:lo + c.hkv], pos, freq, interleaved)
                                for _, r, pos in rows], axis=1)            # [hkv][rows][D]
                source[name][page][:, slots] = new
                fresh[name][page][:, slots] = True
                if c.dtype == "bf16":
                    codes[name][page][:, slots] = bf16_round(new)
                    continue
                older = slots[0]
                for h in range(c.hkv):
                    fin = np.abs(new[h][np.isfinite(new[h])])
                    need = pow2_scale(fin.max() if fin.size else 0.0)
                    had = float(scales[name][page, h])
                    now = max(had, need) if older else need
                    if older and now != had:
                        old = E4M3[codes[name][page, h, :older]]
                        codes[name][page, h, :older] = e4m3_round(old * (had / now))
                    codes[name][page, h, slots] = e4m3_round(new[h] / now)
                    scales[name][page, h] = now
    return q, wrote_q, codes, scales, source, fresh


def attention_oracle(c: Case, scale=None, codes=None):
    """(out, tolerance, rows written) in float64.

    The tolerance: a probability is rounded to bf16 (HALF_BF16 relative) and so
    is the output; a score's products are exact in fp32 and its sum of D terms,
    the scale and the difference to the maximum are off by at most (D + 4) 2^-24
    of sum |q k| (twice: in p and in the normaliser); the exponential and the sums
    over L keys in fp32 by (L + 64) 2^-24.  A = sum p |v| carries all of them."""
    scale = c.D ** -0.5 if scale is None else scale
    q = bf16_values(c.q).reshape(c.T, c.hq, c.D)
    out = np.zeros((c.T, c.hq, c.D))
    tol = np.zeros_like(out)
    wrote = np.zeros(c.T, bool)
    vals = {n: c.values(n) for n in ("k", "v")}
    G = c.hq // c.hkv
    for s in range(len(c.seqs)):
        cap = min(max(int(c.kv_len[s]), 0), c.max_pages * c.P)
        pages = c.table[s, :-(-cap // c.P)] if cap else np.zeros(0, np.int32)
        good = (pages >= 0) & (pages < c.pages)
        ids = np.where(good, pages, 0)
        seen_page = np.repeat(good, c.P)[:cap]
        kv = {n: vals[n][ids].transpose(1, 0, 2, 3).reshape(c.hkv, -1, c.D)[:, :cap]
              for n in ("k", "v")}
        for r in range(c.q_start[s], c.q_start[s + 1]):
            wrote[r] = True
            end = min(max(c.position(s, r - c.q_start[s]) + 1, 0), cap)
            see = np.nonzero(seen_page[:end])[0]
            if not len(see):
                continue
            for h in range(c.hkv):
                k, v = kv["k"][h][see], kv["v"][h][see]
                qq = q[r, h * G:(h + 1) * G]
                with np.errstate(invalid="ignore"):
                    sc = scale * (qq @ k.T)
                    p = np.exp(sc - sc.max(axis=1, keepdims=True))
                    p /= p.sum(axis=1, keepdims=True)
                    out[r, h * G:(h + 1) * G] = p @ v
                    big = abs(scale) * (np.abs(qq) @ np.abs(k).T).max(axis=1, keepdims=True)
                    rel = 2 * HALF_BF16 + 4 * (c.D + 4) * ULP32 * big + 2 * (len(see) + 64) * ULP32
                    tol[r, h * G:(h + 1) * G] = rel * (p @ np.abs(v))
    return out.reshape(c.T, -1), tol.reshape(c.T, -1), wrote


def assert_attention(c: Case, got, scale=None, what=""):
    want, tol, wrote = attention_oracle(c, scale)
    got = got.float().cpu().double().numpy()
    assert np.isnan(got[~wrote]).all(), f"{what}: a row of no sequence was written"
    got, want, tol = got[wrote], want[wrote], tol[wrote]
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities"
    ok = np.isfinite(want)
    err = np.abs(got - want)[ok]
    worst = np.max(err / (tol[ok] + 1e-30)) if err.size else 0.0
    assert worst <= 1.0, f"{what}: worst err / bound {worst:.3g}"
    return worst


def assert_append(c: Case, freq, interleaved=False, what=""):
    """The device's buffers against the oracle: bitwise where the operator only
    moves or rounds its input, and where it rotates first within half a step of
    the 64-bit value (1e-9 of it: sine and cosine in fp64)."""
    q, wrote, codes, scales, source, fresh = append_oracle(c, freq, interleaved)
    got = c.dev["out"].float().cpu().double().numpy().reshape(c.T, c.hq, c.D)
    assert np.isnan(got[~wrote]).all(), f"{what}: q of a row of no sequence was written"
    fin = np.isfinite(q) & wrote[:, None, None]
    err = np.abs(got - q)[fin]
    assert (err <= (HALF_BF16 + 1e-9) * np.abs(q[fin]) + 1e-38).all(), f"{what}: q {err.max()}"
    for name in scales:
        have = c.dev[name + "_scale"].cpu().numpy()
        assert np.array_equal(have.view(np.uint32), scales[name].view(np.uint32)), f"{what}: {name} scale"
    for name in ("k", "v"):
        t = c.dev[name].cpu()
        have = t.view(torch.int16).numpy().view(np.uint16) if c.dtype == "bf16" else \
            t.view(torch.uint8).numpy()
        f = fresh[name]
        assert np.array_equal(have[~f], codes[name][~f]), f"{what}: {name} outside the new rows"
        if name == "v" or freq is None:
            nan = np.isnan(source[name]) & f
            assert np.array_equal(have[f & ~nan], codes[name][f & ~nan]), f"{what}: {name} codes"
        dec, x = (bf16_values(have), source[name]) if c.dtype == "bf16" else \
            (E4M3[have], source[name] / scales[name].astype(np.float64)[:, :, None, None])
        assert np.array_equal(np.isnan(dec[f]), np.isnan(x[f])), f"{what}: {name} NaN"
        ok = f & np.isfinite(x)
        if c.dtype == "bf16":
            half = HALF_BF16 * np.abs(x[ok]) + 1e-38
        else:
            _, e = np.frexp(np.abs(x[ok]))
            half = 2.0 ** (np.maximum(e - 1, -6) - 4.0)
        assert (np.abs(dec[ok] - x[ok]) <= half + 1e-9 * np.abs(x[ok])).all(), f"{what}: {name}"


def frequencies(rot, base=1e6):
    half = rot // 2
    return (base ** (-np.arange(half) / max(1, half))).astype(np.float32)
