"""The operators around the linears of a decode or verify step, as measured work.

Between a layer's QKV and O linears a step appends the new keys and values to a
paged cache (``kv_append``: position rotation of q and k, the cache in bf16 or
in e4m3 with one scale per page and head) and attends over that cache
(``kv_attention``); after the vocabulary projection it verifies the drafted
tokens against the target's probabilities (``verify_draft``).

Sequences share one ragged batch: sequence s owns rows q_start[s] ..
q_start[s + 1] of the T rows, kv_len[s] counts its cache after them, and its
row i stands at position kv_len[s] - n_s + i.

``run`` computes each operator in elementary torch operations where ``own`` is
false, and calls the library's entry points where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

PREFIX_PAGES = 8          # kv_append: full pages that the sequences' prompts share
MIN_SCALE_EXP = -64       # smallest scale of an 8-bit page: 2^-64
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # One new token of one sequence on a TP=8 shard (8 query heads, 1 KV head): latency.
        dict(name="append_tp8_token", op="append", cache="fp8", seqs=1, tokens=1, q_heads=8,
             kv_heads=1, head_dim=128, page=64, context=4000, rot=128, interleaved=False),
        # Two sequences verifying six tokens each, whole model on one GPU, pages of 16.
        dict(name="append_verify", op="append", cache="fp8", seqs=2, tokens=12, q_heads=64,
             kv_heads=8, head_dim=128, page=16, context=30011, rot=128, interleaved=False),
        # Sixteen decoding sequences, bf16 cache, adjacent pairs, part of each head rotated.
        dict(name="append_batch_bf16", op="append", cache="bf16", seqs=16, tokens=16, q_heads=32,
             kv_heads=8, head_dim=64, page=32, context=120001, rot=32, interleaved=True),
        # Prompts of three sequences entering the cache.
        dict(name="append_prompt", op="append", cache="fp8", seqs=3, tokens=4099, q_heads=64,
             kv_heads=8, head_dim=128, page=64, context=9001, rot=128, interleaved=False),
        # One token of one sequence on a TP=8 shard.
        dict(name="attn_tp8_token", op="attention", cache="fp8", seqs=1, tokens=1, q_heads=8,
             kv_heads=1, head_dim=128, page=64, context=4000),
        # Short chats of a small model, ragged.
        dict(name="attn_short_d64", op="attention", cache="fp8", seqs=5, tokens=7, q_heads=32,
             kv_heads=8, head_dim=64, page=16, context=777),
        # Two sequences verifying six tokens each at about 30k tokens of context.
        dict(name="attn_verify", op="attention", cache="fp8", seqs=2, tokens=12, q_heads=64,
             kv_heads=8, head_dim=128, page=16, context=30011),
        # Sixteen decoding sequences of unequal lengths, bf16 cache.
        dict(name="attn_batch_bf16", op="attention", cache="bf16", seqs=16, tokens=16, q_heads=64,
             kv_heads=8, head_dim=128, page=32, context=16001),
        # One sequence at the model's longest context.
        dict(name="attn_long", op="attention", cache="fp8", seqs=1, tokens=1, q_heads=64,
             kv_heads=8, head_dim=128, page=64, context=131072),
        # One sequence, one drafted token, a small vocabulary of odd size, no draft distribution.
        dict(name="verify_small", op="verify", logits="f32", seqs=1, tokens=2, vocab=32003,
             draft=False),
        # The six-token verify step at the full vocabulary, with the draft's distribution.
        dict(name="verify_six", op="verify", logits="bf16", seqs=1, tokens=6, vocab=152064,
             draft=True),
        # Eight sequences, ragged drafts (some with none), full vocabulary.
        dict(name="verify_batch", op="verify", logits="bf16", seqs=8, tokens=37, vocab=152064,
             draft=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "verify"])
    if op == "verify":
        seqs = _spread(rng, 1, 12)
        return dict(op=op, logits=rng.choice(["bf16", "f32"]), seqs=seqs,
                    tokens=seqs + _spread(rng, 1, 40) - 1, vocab=_spread(rng, 2000, 80000),
                    draft=rng.random() < 0.7)
    kv_heads = rng.choice([1, 2, 4, 8])
    case = dict(op=op, cache=rng.choice(["fp8", "fp8", "bf16"]), kv_heads=kv_heads,
                q_heads=kv_heads * rng.choice([1, 2, 4, 5, 8]),
                head_dim=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        seqs = _spread(rng, 1, 24)
        rot = rng.choice([0, case["head_dim"] // 2, case["head_dim"], case["head_dim"]])
        return dict(case, seqs=seqs, tokens=seqs + _spread(rng, 1, 1500) - 1,
                    context=_spread(rng, 2000, 120000), rot=rot,
                    interleaved=rng.random() < 0.4)
    seqs = _spread(rng, 1, 24)
    per_token = 2 * kv_heads * case["head_dim"] * (2 if case["cache"] == "bf16" else 1)
    most = min(60000, int(2.0e8 / per_token / seqs))
    return dict(case, seqs=seqs, tokens=seqs + _spread(rng, 1, 6 * seqs) - 1,
                context=_spread(rng, 24, max(200, most)))


def _lengths(case):
    """Rows and cache length of each sequence, a function of the case alone: one
    sequence of several has the whole context, the others any part of it; of four
    or more, one has no rows in this step and one begins with it."""
    S, T, context = case["seqs"], case["tokens"], case["context"] if "context" in case else 0
    rng = random.Random("%d %d %d" % (S, T, context))
    rows = [1] * S
    if S >= 4 and T > S:
        rows[2] = 0
    spare = T - sum(rows)
    cuts = sorted(rng.randint(0, spare) for _ in range(S - 1))
    for s, (a, b) in enumerate(zip([0] + cuts, cuts + [spare])):
        if rows[s]:
            rows[s] += b - a
    rows[0] += T - sum(rows)
    lens = [max(n, context)] if S == 1 and (n := rows[0]) else []
    for s in range(S if S > 1 else 0):
        length = context if s == 0 else int(context * rng.random() ** 1.5)
        lens.append(max(rows[s], length))
    if S >= 4:
        lens[1] = rows[1]
    return rows, lens


def _esize(case):
    return 2 if case["cache"] == "bf16" else 1


def work(case):
    rows, lens = _lengths(case)
    T, S = case["tokens"], case["seqs"]
    if case["op"] == "verify":
        e = 2 if case["logits"] == "bf16" else 4
        read = T + (sum(n - 1 for n in rows if n) if case["draft"] else 0)
        return {"bytes": read * case["vocab"] * e + 16 * T + 12 * S,
                "flops": 4.0 * read * case["vocab"]}
    hq, hkv, d, e = case["q_heads"], case["kv_heads"], case["head_dim"], _esize(case)
    if case["op"] == "append":
        return {"bytes": 2 * T * (hq + 2 * hkv) * d + 2 * T * hq * d + 2 * T * hkv * d * e,
                "flops": 3.0 * T * (hq + hkv) * case["rot"] + T * 2 * hkv * d}
    seen = sum(n * length - n * (n - 1) // 2 for n, length in zip(rows, lens))
    read = sum(length for n, length in zip(rows, lens) if n)
    return {"bytes": 2 * read * hkv * d * e + 4 * T * hq * d, "flops": 4.0 * seen * hq * d}


# ---------------------------------------------------------------------------
# Inputs


def _normal(gen, shape, sigma, dtype):
    return (sigma * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(gen, case, pages):
    """A pool of pages with data in every slot: bf16, or e4m3 codes with powers
    of two as scales (keys of standard deviation about 1.5)."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    state = {}
    for name in ("k", "v"):
        if case["cache"] == "bf16":
            state[name] = _normal(gen, shape, 1.5, torch.bfloat16)
            state[name + "_scale"] = None
        else:
            codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
            for part in codes.split(max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))):
                part.copy_((96.0 * torch.randn(part.shape, generator=gen, device="cuda"))
                           .clamp_(-E4M3_MAX, E4M3_MAX))
            state[name] = codes
            exps = torch.randint(-7, -4, shape[:2], generator=gen, device="cuda")
            state[name + "_scale"] = torch.exp2(exps.float())
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, lens = _lengths(case)
    S, T = case["seqs"], case["tokens"]
    q_start = np.concatenate([[0], np.cumsum(rows)]).tolist()
    state = {"op": case["op"], "q_start": _ints(q_start), "rows": max(rows)}
    if case["op"] == "verify":
        _prepare_verify(state, case, gen)
    else:
        P, D = case["page"], case["head_dim"]
        width = max(1, -(-max(lens) // P))
        order = random.Random(seed)
        table = []
        if case["op"] == "append":
            # Pages that receive rows are a sequence's own, all others shared prefix pages.
            firsts = [(length - n) // P for n, length in zip(rows, lens)]
            counts = [(length - 1) // P - f + 1 if n else 0
                      for n, length, f in zip(rows, lens, firsts)]
            pages = sum(counts) + PREFIX_PAGES
            ids = order.sample(range(pages), pages)
            for f, c in zip(firsts, counts):
                mine = [ids.pop() for _ in range(c)]
                table.append([order.choice(ids[:PREFIX_PAGES]) for _ in range(f)] + mine
                             + [0] * (width - f - c))
        else:
            counts = [-(-length // P) for length in lens]
            pages = sum(counts)
            ids = order.sample(range(pages), pages)
            for c in counts:
                table.append([ids.pop() for _ in range(c)] + [0] * (width - c))
        state.update(_cache(gen, case, pages), kv_len=_ints(lens), page_table=_ints(table),
                     page=P, head_dim=D, q_heads=case["q_heads"], kv_heads=case["kv_heads"],
                     longest=max(lens))
        width_q = case["q_heads"] * D
        if case["op"] == "append":
            state["qkv"] = _normal(gen, (T, width_q + 2 * case["kv_heads"] * D), 2.0, torch.bfloat16)
            state["interleaved"], state["rot"] = case["interleaved"], case["rot"]
            half = case["rot"] // 2
            # Base 10^6, as a float32 table; no rotation at all for rot = 0.
            state["inv_freq"] = None if not half else (
                1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
            state["q_out"] = torch.empty((T, width_q), dtype=torch.bfloat16, device="cuda")
        else:
            state["q"] = _normal(gen, (T, width_q), 1.0, torch.bfloat16)
            state["out"] = torch.empty((T, width_q), dtype=torch.bfloat16, device="cuda")
    if own:  # what a program keeps beside its buffers: descriptors of them and a workspace
        _handles(state)
    return state


def _prepare_verify(state, case, gen):
    S, T, V = case["seqs"], case["tokens"], case["vocab"]
    dtype = torch.bfloat16 if case["logits"] == "bf16" else torch.float32
    # Logits with one likely token a row; the draft's are the target's, perturbed.
    logits = 2.5 * torch.randn((T, V), generator=gen, device="cuda")
    peak = torch.randint(0, V, (T, 1), generator=gen, device="cuda")
    logits.scatter_add_(1, peak, 13.0 + 3.0 * torch.rand((T, 1), generator=gen, device="cuda"))
    state["logits"] = logits.to(dtype)
    draft = (logits + 0.5 * torch.randn((T, V), generator=gen, device="cuda")).to(dtype)
    # One sequence in eight is greedy, the others sample at unlike temperatures.
    tau = torch.tensor([0.0 if s % 8 == 3 else 0.6 + 0.1 * (s % 7) for s in range(S)])
    state["temperature"] = tau.float().cuda()
    row_tau = torch.full((T,), 0.8, device="cuda")
    noise = -torch.log(-torch.log(torch.rand((T, V), generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)))
    drawn = torch.argmax(draft.float() / row_tau[:, None] + noise, dim=1)
    # Row r's token is drawn from the draft's distribution at row r - 1.
    state["tokens"] = torch.roll(drawn, 1).to(torch.int32)
    state["draft_logits"] = draft if case["draft"] else None
    state["accept_u"] = torch.rand(T, generator=gen, device="cuda")
    state["sample_u"] = torch.rand(S, generator=gen, device="cuda")
    state["out_tokens"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    state["accepted"] = torch.zeros(S, dtype=torch.int32, device="cuda")


def _handles(st):
    import gemv_skinny_gemm_amd as sg

    def workspace(n):
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    if st["op"] == "verify":
        T, V = st["logits"].shape
        st["workspace"] = workspace(sg.verify_workspace_bytes(T, st["sample_u"].numel(), V))
        return
    st["cache"] = sg.make_kv_cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
    rows = (st["qkv"] if st["op"] == "append" else st["q"]).shape[0]
    st["batch"] = sg.make_batch(st["q_start"], st["kv_len"], st["page_table"], rows)
    if st["op"] == "attention":
        st["workspace"] = workspace(
            sg.kv_attention_workspace_bytes(st["cache"], st["batch"], st["q_heads"]))


# ---------------------------------------------------------------------------
# One pass


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "append":
        return _plain_append(st)
    if st["op"] == "attention":
        return _plain_attention(st)
    return _plain_verify(st)


def _run_own(st):
    import gemv_skinny_gemm_amd as sg
    if st["op"] == "append":
        sg.kv_append(st["cache"], st["batch"], st["qkv"], st["inv_freq"], st["q_out"],
                     interleaved=st["interleaved"])
        return _append_outputs(st)
    if st["op"] == "attention":
        sg.kv_attention(st["cache"], st["batch"], st["q"], st["out"], st["workspace"])
        return {"out": st["out"]}
    sg.verify_draft(st["q_start"], st["logits"], st["tokens"], st["accept_u"], st["sample_u"],
                    st["out_tokens"], st["accepted"], st["workspace"],
                    draft_logits=st["draft_logits"], temperature=st["temperature"])
    return {"tokens": st["out_tokens"], "accepted": st["accepted"]}


def _append_outputs(st):
    """q, and the cache's own buffers (its codes as e4m3 numbers, the scales beside them)."""
    got = {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    if st["k_scale"] is not None:
        got.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
    return got


def _row_sequences(st, T):
    """Sequence of each row."""
    return torch.searchsorted(st["q_start"][1:].long(), torch.arange(T, device="cuda"), right=True)


def _rotate(x, angle, interleaved):
    """x [T][H][D] in float64, the first 2 x angle.shape[1] values of a head rotated."""
    half = angle.shape[1]
    cos, sin = angle.cos()[:, None, :], angle.sin()[:, None, :]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _page_scale(amax):
    """The smallest power of two s with amax <= 448 s, 2^-64 at least."""
    m, e = torch.frexp(amax / E4M3_MAX)
    e = torch.where(m > 0.5, e, e - 1)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_SCALE_EXP)).clamp(min=MIN_SCALE_EXP)
    return torch.exp2(e.double())


def _plain_append(st):
    qkv, P, D, hq, hkv = st["qkv"], st["page"], st["head_dim"], st["q_heads"], st["kv_heads"]
    T = qkv.shape[0]
    seq = _row_sequences(st, T)
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    pos = kv_len[seq] - q_start[seq + 1] + torch.arange(T, device="cuda")
    x = qkv.double().view(T, hq + 2 * hkv, D)
    qk, v = x[:, :hq + hkv], x[:, hq + hkv:]
    if st["inv_freq"] is not None:
        qk = _rotate(qk, pos.double()[:, None] * st["inv_freq"].double()[None, :], st["interleaved"])
    st["q_out"].copy_(qk[:, :hq].reshape(T, hq * D))
    page, slot = st["page_table"].long()[seq, pos // P], pos % P
    if st["k_scale"] is None:
        st["k"][page, :, slot] = qk[:, hq:].to(torch.bfloat16)
        st["v"][page, :, slot] = v.to(torch.bfloat16)
        return _append_outputs(st)
    # The page that a sequence's first new row enters may hold older rows.
    has = q_start[1:] > q_start[:-1]
    first = (kv_len - (q_start[1:] - q_start[:-1])).clamp(min=0)
    at = (first // P).clamp(max=st["page_table"].shape[1] - 1)
    begun = st["page_table"].long().gather(1, at[:, None])[:, 0]
    old_rows = torch.where(has, first % P, torch.zeros_like(first))
    keeps = old_rows > 0
    for name, rows in (("k", qk[:, hq:]), ("v", v)):
        codes, scale = st[name], st[name + "_scale"]
        amax = torch.zeros(scale.shape, dtype=torch.float64, device="cuda")
        amax.index_reduce_(0, page, rows.abs().amax(dim=-1), "amax")
        new = scale.double()
        new[page] = _page_scale(amax[page])
        old = scale.double()[begun]
        ratio = old / torch.maximum(old, new[begun])
        stay = torch.arange(P, device="cuda")[None, :] < old_rows[:, None]
        before = codes[begun].double()
        after = (before * ratio[:, :, None, None]).float().to(torch.float8_e4m3fn)
        raised = torch.where(keeps[:, None], torch.maximum(old, new[begun]), new[begun])
        new.index_reduce_(0, begun, torch.where(keeps[:, None], raised, torch.zeros_like(raised)), "amax")
        kept = torch.where(stay[:, None, :, None], after.view(torch.uint8), codes[begun].view(torch.uint8))
        own_page = torch.where(keeps, begun, begun.new_full((), -1))
        every = torch.cat([codes.view(torch.uint8), codes.new_zeros((1, *codes.shape[1:])).view(torch.uint8)])
        every[own_page] = kept
        every[page, :, slot] = (rows / new[page][:, :, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        codes.view(torch.uint8).copy_(every[:-1])
        scale.copy_(new)
    return _append_outputs(st)


def _plain_attention(st):
    q, P, D, hq, hkv = st["q"], st["page"], st["head_dim"], st["q_heads"], st["kv_heads"]
    T, S, n = q.shape[0], st["kv_len"].numel(), st["rows"]
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    pages = st["page_table"].long()[:, :-(-st["longest"] // P)]

    def gathered(codes, scale):
        x = codes[pages].float()                                   # [S][pages][heads][P][D]
        if scale is not None:
            x = x * scale[pages][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(S, hkv, -1, D)

    row = q_start[:-1, None] + torch.arange(n, device="cuda")      # [S][n], clamped into T below
    count = q_start[1:] - q_start[:-1]
    x = q[row.clamp(max=T - 1)].float().view(S, n, hkv, hq // hkv, D)
    x = x.permute(0, 2, 1, 3, 4).reshape(S, hkv, -1, D) / math.sqrt(D)
    score = torch.matmul(x, gathered(st["k"], st["k_scale"]).transpose(2, 3).contiguous())
    score = score.view(S, hkv, n, hq // hkv, -1)
    last = kv_len[:, None] - count[:, None] + torch.arange(n, device="cuda")
    seen = torch.arange(score.shape[-1], device="cuda") <= last[..., None]
    score = score.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    top = score.amax(dim=-1, keepdim=True)
    weight = torch.exp(score - torch.where(top.isfinite(), top, torch.zeros_like(top)))
    total = weight.sum(dim=-1, keepdim=True)
    value = gathered(st["v"], st["v_scale"])
    y = torch.matmul(weight.view(S, hkv, -1, weight.shape[-1]), value).view(S, hkv, n, -1, D)
    y = y / torch.where(total > 0, total, torch.ones_like(total))
    y = y.permute(0, 2, 1, 3, 4).reshape(S, n, hq * D)
    seq = _row_sequences(st, T)
    st["out"].copy_(y[seq, torch.arange(T, device="cuda") - q_start[seq]])
    return {"out": st["out"]}


def _plain_verify(st):
    logits, T = st["logits"], st["logits"].shape[0]
    seq, q_start = _row_sequences(st, T), st["q_start"].long()
    at = torch.arange(T, device="cuda")
    tau = st["temperature"].double()[seq][:, None]

    def probabilities(x):
        x = x.double()
        top, first = x.max(dim=1, keepdim=True)
        first = (x == top).to(torch.uint8).argmax(dim=1, keepdim=True)      # the lowest of equals
        e = torch.exp((x - top) / torch.where(tau > 0, tau, torch.ones_like(tau)))
        one = torch.zeros_like(e).scatter_(1, first, 1.0)
        return torch.where(tau > 0, e / e.sum(dim=1, keepdim=True), one)

    p = probabilities(logits)
    drafted = torch.roll(st["tokens"].long(), -1)[:, None]
    if st["draft_logits"] is not None:
        q = probabilities(st["draft_logits"])
        q = torch.where(tau > 0, q, torch.zeros_like(q).scatter_(1, drafted, 1.0))
    else:
        q = torch.zeros_like(p).scatter_(1, drafted, 1.0)
    final = at + 1 == q_start[seq + 1]
    taken = st["accept_u"].double() * q.gather(1, drafted)[:, 0] < p.gather(1, drafted)[:, 0]
    # The first row of each sequence that stops: a rejection, or its last row.
    stop = torch.full((q_start.numel() - 1,), T, device="cuda").scatter_reduce(
        0, seq, torch.where(taken & ~final, T, at), "amin")
    has = q_start[1:] > q_start[:-1]
    row = stop.clamp(max=T - 1)
    w = torch.where(final[row][:, None], p[row], (p[row] - q[row]).clamp(min=0))
    w = torch.where(w.sum(dim=1, keepdim=True) > 0, w, p[row])
    sums = w.cumsum(dim=1)
    goal = st["sample_u"].double()[:, None] * sums[:, -1:]
    index = torch.arange(w.shape[1], device="cuda")
    largest = torch.where(w > 0, index, index.new_zeros(())).amax(dim=1)
    token = torch.minimum((sums <= goal).sum(dim=1), largest)
    last = stop[seq]
    out = torch.where(at < last, drafted[:, 0], torch.where(at == last, token[seq], -1))
    st["out_tokens"].copy_(out)
    st["accepted"].copy_(torch.where(has, stop - q_start[:-1], 0))
    return {"tokens": st["out_tokens"], "accepted": st["accepted"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence


def exact(case, seed):
    st = prepare(case, seed)
    starts = st["q_start"].tolist()
    if case["op"] == "verify":
        return _exact_verify(st, starts)
    lens, table = st["kv_len"].tolist(), st["page_table"].tolist()
    return (_exact_append if case["op"] == "append" else _exact_attention)(st, starts, lens, table)


def _to_e4m3(x):
    """Nearest e4m3 number, ties to even, of |x| <= 448 (steps of 2^-9 below 2^-6)."""
    _, e = np.frexp(np.abs(x))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.round(x / step) * step


def _exact_append(st, starts, lens, table):
    P, D, hq, hkv = st["page"], st["head_dim"], st["q_heads"], st["kv_heads"]
    x = st["qkv"].double().cpu().numpy()
    x = x.reshape(x.shape[0], -1, D)
    rot = st["rot"]
    out_q = np.zeros((x.shape[0], hq, D))
    pools = {n: st[n].double().cpu().numpy() for n in ("k", "v")}
    scaled = st["k_scale"] is not None
    scales = {n: st[n + "_scale"].double().cpu().numpy() for n in ("k", "v")} if scaled else {}
    freq = st["inv_freq"].double().cpu().numpy() if rot else None
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        if not n:
            continue
        mine = x[starts[s]:starts[s + 1]].copy()
        place = np.arange(length - n, length)
        if rot:
            even = slice(0, rot, 2) if st["interleaved"] else slice(0, rot // 2)
            odd = slice(1, rot, 2) if st["interleaved"] else slice(rot // 2, rot)
            turned = (mine[:, :hq + hkv, even] + 1j * mine[:, :hq + hkv, odd]) \
                * np.exp(1j * place[:, None] * freq[None, :])[:, None, :]
            mine[:, :hq + hkv, even], mine[:, :hq + hkv, odd] = turned.real, turned.imag
        out_q[starts[s]:starts[s + 1]] = mine[:, :hq]
        for page in range((length - n) // P, (length - 1) // P + 1):
            inside = place // P == page
            slots, older = place[inside] % P, max(0, min(P, length - n - page * P))
            for name, lo in (("k", hq), ("v", hq + hkv)):
                rows = mine[inside, lo:lo + hkv].transpose(1, 0, 2)          # [heads][rows][D]
                pool = pools[name][table[s][page]]
                if not scaled:
                    pool[:, slots] = rows
                    continue
                top = np.abs(rows).max(axis=(1, 2))
                need = np.full(hkv, 2.0 ** MIN_SCALE_EXP)
                while (low := top > E4M3_MAX * need).any():
                    need[low] *= 2
                had = scales[name][table[s][page]].copy()
                now = np.maximum(had, need) if older else need
                pool[:, :older] = _to_e4m3(pool[:, :older] * (had / now)[:, None, None])
                pool[:, slots] = _to_e4m3(rows / now[:, None, None])
                scales[name][table[s][page]] = now
    got = {"q": out_q.reshape(x.shape[0], hq * D), **pools}
    if scaled:
        got.update(k_scale=scales["k"], v_scale=scales["v"])
    return got


def _exact_attention(st, starts, lens, table):
    P, D, hq, hkv = st["page"], st["head_dim"], st["q_heads"], st["kv_heads"]
    q = st["q"].double().view(-1, hq, D)
    out = torch.zeros_like(q)
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        if not n:
            continue
        ids = torch.tensor(table[s][:-(-length // P)], device="cuda")
        for h in range(hkv):
            k, v = st["k"][ids, h].double(), st["v"][ids, h].double()
            if st["k_scale"] is not None:
                k = k * st["k_scale"][ids, h].double()[:, None, None]
                v = v * st["v_scale"][ids, h].double()[:, None, None]
            k, v = k.reshape(-1, D)[:length], v.reshape(-1, D)[:length]
            for i in range(n):
                end = length - n + i + 1
                heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
                score = q[starts[s] + i, heads] @ k[:end].T * D ** -0.5
                out[starts[s] + i, heads] = torch.softmax(score, dim=1) @ v[:end]
    return {"out": out.view(-1, hq * D)}


def _exact_verify(st, starts):
    logits = st["logits"].double().cpu().numpy()
    draft = None if st["draft_logits"] is None else st["draft_logits"].double().cpu().numpy()
    tokens, tau = st["tokens"].tolist(), st["temperature"].double().tolist()
    u, su = st["accept_u"].double().tolist(), st["sample_u"].double().tolist()
    out, accepted = [-1] * len(tokens), []

    def soft(x, t):
        e = np.exp((x - x.max()) / t)
        return e / e.sum()

    for s in range(len(su)):
        lo, hi = starts[s], starts[s + 1]
        taken = 0
        for r in range(lo, hi):
            d = tokens[r + 1] if r + 1 < hi else None
            if tau[s] <= 0:
                best = int(np.argmax(logits[r]))
                if d is not None and d == best and u[r] < 1:
                    out[r] = d
                    taken += 1
                    continue
                out[r] = best
                break
            p = soft(logits[r], tau[s])
            q = np.zeros_like(p)
            if d is not None and draft is not None:
                q = soft(draft[r], tau[s])
            elif d is not None:
                q[d] = 1.0
            if d is not None and u[r] * q[d] < p[d]:
                out[r] = d
                taken += 1
                continue
            w = np.maximum(p - q, 0.0)
            w = w if w.sum() > 0 else p
            sums = np.cumsum(w)
            first = int(np.searchsorted(sums, su[s] * sums[-1], side="right"))
            out[r] = min(first, int(np.nonzero(w)[0][-1]))
            break
        accepted.append(taken)
    return {"tokens": np.array(out), "accepted": np.array(accepted)}
