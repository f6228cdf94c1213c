"""What a decoder layer computes between and beside its linears, as measured work.

``block_norm`` updates the residual with a block's output (its norm, gate, scales
and, behind a mixture of experts, the routes' weighted sum) and makes the next
linear's input; ``lora_linear`` adds the low-rank adapters of many requests beside
a shared projection; ``moe_route`` turns a router's logits into the experts' ids
and weights.

``run`` computes each operator in elementary torch operations where ``own`` is
false, and calls the library's entry points where it is true.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# Cases


def listed():
    return [
        # One decoding token: residual update and the next linear's input. Latency.
        dict(name="norm_token", op="norm", kind="rms", rows=1, width=8192, routes=1, post=False,
             gate="none", residual="bf16", weight="bf16", scales=False),
        # Behind the experts of a 16-token step: two routes a token, fp32 residual.
        dict(name="norm_experts", op="norm", kind="rms", rows=16, width=4096, routes=2, post=False,
             gate="none", residual="f32", weight="bf16", scales=False),
        # Norms before and after a block, a gate per value, layer norm, an odd width.
        dict(name="norm_sandwich_odd", op="norm", kind="layer", rows=777, width=5001, routes=1,
             post=True, gate="value", residual="f32", weight="f32", scales=True),
        # A long prompt through a pre- and post-normed block with a gate per channel.
        dict(name="norm_prompt", op="norm", kind="rms", rows=16384, width=8192, routes=1, post=True,
             gate="channel", residual="bf16", weight="bf16", scales=True),
        # One request's adapter beside the QKV projection: latency.
        dict(name="lora_token", op="lora", rows=1, k=8192, n1=8192, n2=1024, n3=1024, adapters=8,
             rank=16, mixed=False),
        # Sixteen requests beside gate and up, adapters of unlike ranks.
        dict(name="lora_batch", op="lora", rows=16, k=8192, n1=29568, n2=29568, n3=0, adapters=32,
             rank=64, mixed=True),
        # A busy server's batch on a TP=8 shard's projection of odd width.
        dict(name="lora_many_odd", op="lora", rows=251, k=1032, n1=2561, n2=0, n3=0, adapters=64,
             rank=32, mixed=True),
        # Prompts of some requests beside QKV.
        dict(name="lora_prompt", op="lora", rows=4099, k=8192, n1=8192, n2=1024, n3=1024,
             adapters=3, rank=64, mixed=False),
        # One token over a few experts: latency.
        dict(name="route_token", op="route", scoring="softmax", logits="bf16", rows=1, experts=8,
             topk=2, groups=1, top_groups=1, bias=False),
        # A 16-token step over many experts, biased choice within the best groups.
        dict(name="route_groups", op="route", scoring="sigmoid", logits="f32", rows=16, experts=256,
             topk=8, groups=8, top_groups=4, bias=True),
        # A prompt over an odd number of experts.
        dict(name="route_prompt", op="route", scoring="softmax", logits="bf16", rows=16384,
             experts=161, topk=6, groups=1, top_groups=1, bias=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "lora", "lora", "lora", "route"])
    if op == "norm":
        width = _spread(rng, 64, 16384)
        if rng.random() < 0.7:
            width = -(-width // 8) * 8
        routes = rng.choice([1, 1, 1, 2, 4, 8])
        rows = _spread(rng, 1, max(1, min(16384, (1 << 26) // (width * (routes + 1)))))
        return dict(op=op, kind=rng.choice(["rms", "rms", "layer"]), rows=rows, width=width,
                    routes=routes, post=rng.random() < 0.4,
                    gate=rng.choice(["none", "none", "channel", "value"]),
                    residual=rng.choice(["bf16", "f32"]), weight=rng.choice(["bf16", "f32"]),
                    scales=rng.random() < 0.4)
    if op == "lora":
        rows = _spread(rng, 1, 3000)
        k = 8 * _spread(rng, 16, 1024)
        rank = rng.choice([8, 16, 16, 32, 64, 128])
        most = max(64, min(30000, (1 << 26) // rows - k))
        n = [_spread(rng, 32, most) for _ in range(rng.choice([1, 1, 2, 3]))]
        while sum(n) > most:
            n = [-(-w // 2) for w in n]
        n += [0] * (3 - len(n))
        adapters = _spread(rng, 1, min(64, max(2, (1 << 27) // (rank * (3 * k + sum(n))))))
        return dict(op=op, rows=rows, k=k, n1=n[0], n2=n[1], n3=n[2], adapters=adapters, rank=rank,
                    mixed=rng.random() < 0.5)
    groups = rng.choice([1, 1, 2, 4, 8])
    each = _spread(rng, 2, 64) if groups > 1 else _spread(rng, 4, 512)
    top_groups = rng.randint(1, groups)
    return dict(op=op, scoring=rng.choice(["softmax", "sigmoid"]), logits=rng.choice(["bf16", "f32"]),
                rows=_spread(rng, 1, 16384), experts=groups * each,
                topk=rng.randint(1, min(16, top_groups * each)), groups=groups,
                top_groups=top_groups, bias=rng.random() < 0.5)


def _slices(case):
    return [case["n%d" % i] for i in (1, 2, 3) if case["n%d" % i]]


def _row_adapters(case):
    """Adapter of each row, a function of the case alone: requests of neighbouring
    rows (one row each in a batch of few), each with an adapter, one in nine
    without (-1), some adapters shared and some without requests."""
    T, E = case["rows"], case["adapters"]
    rng = random.Random("%d %d %d" % (T, E, case["k"]))
    requests = T if T <= 64 else min(T, max(5, T // 40))
    cuts = sorted(rng.sample(range(1, T), requests - 1)) if requests > 1 else []
    ids = []
    for i, (a, b) in enumerate(zip([0] + cuts, cuts + [T])):
        ids += [-1 if i % 9 == 4 else rng.randrange(E)] * (b - a)
    return ids


def _ranks(case):
    rng = random.Random("ranks %d %d" % (case["adapters"], case["rank"]))
    return [case["rank"] if not case["mixed"] else rng.randint(1, case["rank"])
            for _ in range(case["adapters"])]


def work(case):
    if case["op"] == "norm":
        T, H = case["rows"], case["width"]
        res = 2 if case["residual"] == "bf16" else 4
        w = (2 if case["weight"] == "bf16" else 4) * H
        vectors = (2 if case["kind"] == "layer" else 1) * (2 if case["post"] else 1)
        nbytes = T * H * (2 * case["routes"] + 2 * res + 2) + vectors * w
        if case["gate"] == "channel":
            nbytes += w
        elif case["gate"] == "value":
            nbytes += T * w
        if case["routes"] > 1:
            nbytes += 4 * T * case["routes"]
        return {"bytes": nbytes, "flops": T * H * (2.0 * case["routes"] + 8 + (4 if case["post"] else 0))}
    if case["op"] == "lora":
        ids, ranks, n = _row_adapters(case), _ranks(case), _slices(case)
        T, K, N = case["rows"], case["k"], sum(n)
        weights = sum(2 * ranks[a] * (len(n) * K + N) for a in set(ids) if a >= 0)
        flops = sum(2.0 * ranks[a] * (len(n) * K + N) for a in ids if a >= 0)
        read = sum(1 for a in ids if a >= 0)
        return {"bytes": 2 * read * K + 4 * T * N + weights + 4 * T, "flops": flops}
    e = 2 if case["logits"] == "bf16" else 4
    T, E = case["rows"], case["experts"]
    return {"bytes": T * E * e + T * case["topk"] * 8 + (4 * E if case["bias"] else 0),
            "flops": 4.0 * T * E}


# ---------------------------------------------------------------------------
# Inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0, mean=0.0, dtype=torch.bfloat16):
        return (mean + sigma * torch.randn(shape, generator=gen, device="cuda")).to(dtype)

    return {"norm": _prepare_norm, "lora": _prepare_lora, "route": _prepare_route}[case["op"]](
        case, normal, gen)


def _prepare_norm(case, normal, gen):
    T, H = case["rows"], case["width"]
    wt = torch.bfloat16 if case["weight"] == "bf16" else torch.float32
    rt = torch.bfloat16 if case["residual"] == "bf16" else torch.float32
    st = dict(case, residual=normal(T, H, sigma=3.0, dtype=rt),
              block=normal(T * case["routes"], H), pre=normal(H, sigma=0.2, mean=1.0, dtype=wt),
              pre_bias=None, post=None, post_bias=None, gate=None, route_weights=None)
    # A few channels of a residual are far larger than the others.
    st["residual"][:, :: max(1, H // 5)] *= 16.0
    if case["kind"] == "layer":
        st["pre_bias"] = normal(H, sigma=0.1, dtype=wt)
    if case["post"]:
        st["post"] = normal(H, sigma=0.2, mean=0.5, dtype=wt)
        if case["kind"] == "layer":
            st["post_bias"] = normal(H, sigma=0.1, dtype=wt)
    if case["gate"] != "none":
        st["gate"] = normal(*((H,) if case["gate"] == "channel" else (T, H)), sigma=0.5, dtype=wt)
    if case["routes"] > 1:
        st["route_weights"] = torch.softmax(normal(T, case["routes"], dtype=torch.float32), dim=1)
    st["residual_scale"], st["block_scale"] = (0.875, 1.375) if case["scales"] else (1.0, 1.0)
    st["eps"] = 1e-6
    st["residual_out"] = torch.empty_like(st["residual"])
    st["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    return st


def _prepare_lora(case, normal, gen):
    T, K, E, R = case["rows"], case["k"], case["adapters"], case["rank"]
    n = _slices(case)
    st = {"op": "lora", "x": normal(T, K), "base": normal(T, sum(n)), "n": n,
          "ids": torch.tensor(_row_adapters(case), dtype=torch.int32, device="cuda"),
          "a": [normal(E, R, K, sigma=K ** -0.5) for _ in n],
          "b": [normal(E, w, R, sigma=R ** -0.5) for w in n],
          "scale": 0.5 + torch.rand(E, generator=gen, device="cuda"),
          "ranks": torch.tensor(_ranks(case), dtype=torch.int32, device="cuda") if case["mixed"] else None,
          "y": torch.empty((T, sum(n)), dtype=torch.bfloat16, device="cuda")}
    if own:  # what a program keeps beside its buffers: a descriptor of them and a workspace
        import gemv_skinny_gemm_amd as sg
        st["lora"] = sg.make_lora(st["a"], st["b"], scale=st["scale"], ranks=st["ranks"])
        st["workspace"] = torch.empty(sg.lora_workspace_bytes(st["lora"], T), dtype=torch.uint8,
                                      device="cuda")
    return st


def _prepare_route(case, normal, gen):
    T, E, k = case["rows"], case["experts"], case["topk"]
    lt = torch.bfloat16 if case["logits"] == "bf16" else torch.float32
    return dict(case, logits=normal(T, E, sigma=1.5, dtype=lt),
                bias=normal(E, sigma=0.1, dtype=torch.float32) if case["bias"] else None,
                renormalize=case["topk"] > 1, scale=2.5 if case["bias"] else 1.0,
                ids=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                weights=torch.empty((T, k), dtype=torch.float32, device="cuda"))


# ---------------------------------------------------------------------------
# One pass


def run(st):
    if own:
        return _run_own(st)
    return {"norm": _plain_norm, "lora": _plain_lora, "route": _plain_route}[st["op"]](st)


def _run_own(st):
    import gemv_skinny_gemm_amd as sg
    if st["op"] == "norm":
        sg.block_norm(st["out"], st["pre"], residual=st["residual"], block=st["block"],
                      residual_out=st["residual_out"], bias=st["pre_bias"], post_weight=st["post"],
                      post_bias=st["post_bias"], gate=st["gate"], route_weights=st["route_weights"],
                      kind=sg.NORM_LAYER if st["kind"] == "layer" else sg.NORM_RMS, eps=st["eps"],
                      residual_scale=st["residual_scale"], block_scale=st["block_scale"])
        return {"out": st["out"], "residual": st["residual_out"]}
    if st["op"] == "lora":
        sg.lora_linear(st["lora"], st["x"], st["ids"], st["y"], st["workspace"], base=st["base"])
        return {"y": st["y"]}
    sg.moe_route(st["logits"], st["ids"], st["weights"], bias=st["bias"],
                 scoring=sg.ROUTE_SIGMOID if st["scoring"] == "sigmoid" else sg.ROUTE_SOFTMAX,
                 groups=st["groups"], top_groups=st["top_groups"], renormalize=st["renormalize"],
                 scale=st["scale"])
    return {"ids": st["ids"], "weights": st["weights"]}


def _normed(x, st, weight, bias):
    if st["kind"] == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + st["eps"]) * weight.float()
    return y if bias is None else y + bias.float()


def _plain_norm(st):
    T, H = st["out"].shape
    b = st["block"].float()
    if st["route_weights"] is not None:
        b = (b.view(T, -1, H) * st["route_weights"][:, :, None]).sum(dim=1)
    if st["post"] is not None:
        b = _normed(b, st, st["post"], st["post_bias"])
    if st["gate"] is not None:
        b = b * st["gate"].float()
    h = st["residual_scale"] * st["residual"].float() + st["block_scale"] * b
    st["residual_out"].copy_(h)
    st["out"].copy_(_normed(h, st, st["pre"], st["pre_bias"]))
    return {"out": st["out"], "residual": st["residual_out"]}


def _plain_lora(st):
    x, ids, T = st["x"].float(), st["ids"].long(), st["x"].shape[0]
    y, at = st["base"].float(), 0
    for n, a, b in zip(st["n"], st["a"], st["b"]):
        E, R, K = a.shape
        if T * R * (K + n) <= 1 << 27:                 # few rows: each gets a copy of its adapter
            e = ids.clamp(min=0)
            low = torch.matmul(a[e].float(), x[:, :, None])[:, :, 0] * st["scale"][e][:, None]
            live = (ids >= 0)[:, None]
            if st["ranks"] is not None:
                live = live & (torch.arange(R, device="cuda") < st["ranks"][e][:, None])
            low = torch.where(live, low, 0.0)
            y[:, at:at + n] += torch.matmul(b[e].float(), low[:, :, None])[:, :, 0]
        else:                                          # many rows: every adapter in turn, masked
            for e in range(E):
                low = torch.matmul(x, a[e].float().t()) * st["scale"][e]
                if st["ranks"] is not None:
                    low = torch.where(torch.arange(R, device="cuda") < st["ranks"][e], low, 0.0)
                low = torch.where((ids == e)[:, None], low, 0.0)
                y[:, at:at + n] += torch.matmul(low, b[e].float().t())
        at += n
    st["y"].copy_(y)
    return {"y": st["y"]}


def _plain_route(st):
    l = st["logits"].double()
    T, E = l.shape
    if st["scoring"] == "softmax":
        s = torch.exp(l - l.amax(dim=1, keepdim=True))
        s = s / s.sum(dim=1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    # Without a bias the scores order as the logits do, which hold no roundings.
    c = l if st["bias"] is None else s + st["bias"].double()
    low = torch.full((), float("-inf"), dtype=torch.float64, device="cuda")
    place = torch.arange(E, device="cuda")
    if st["groups"] > 1:
        g = c.view(T, st["groups"], -1)
        best = g.amax(dim=2)
        if st["bias"] is not None and g.shape[2] > 1:
            first = (g == best[:, :, None]).to(torch.uint8).argmax(dim=2, keepdim=True)
            best = best + g.scatter(2, first, low.expand(first.shape)).amax(dim=2)
        kept = torch.zeros_like(best, dtype=torch.bool)
        for _ in range(st["top_groups"]):
            at = (best == best.amax(dim=1, keepdim=True)).to(torch.uint8).argmax(dim=1, keepdim=True)
            kept.scatter_(1, at, True)
            best = best.scatter(1, at, low.expand(at.shape))
        c = torch.where(kept[:, :, None], g, low).view(T, E)
    picked = []
    for _ in range(st["topk"]):
        at = torch.where(c == c.amax(dim=1, keepdim=True), place, E).amin(dim=1, keepdim=True)
        picked.append(at)
        c = c.scatter(1, at, low.expand(at.shape))
    ids = torch.cat(picked, dim=1)
    w = s.gather(1, ids)
    if st["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    st["ids"].copy_(ids)
    st["weights"].copy_(w * st["scale"])
    return {"ids": st["ids"], "weights": st["weights"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits


def exact(case, seed):
    return {"norm": _exact_norm, "lora": _exact_lora, "route": _exact_route}[case["op"]](
        prepare(case, seed), case)


def _exact_norm(st, case):
    T, H, r = case["rows"], case["width"], case["routes"]
    out = torch.empty((T, H), dtype=torch.float64, device="cuda")
    new = torch.empty_like(out)

    def stretch(v, weight, bias):
        if case["kind"] == "layer":
            v = v - v.sum(dim=1, keepdim=True) / H
        v = v / torch.sqrt(torch.linalg.vecdot(v, v)[:, None] / H + st["eps"])
        v = v * weight.double()
        return v if bias is None else v + bias.double()

    step = max(1, (1 << 25) // (H * (r + 2)))
    for lo in range(0, T, step):                       # rows of a part, each by itself
        hi = min(T, lo + step)
        v = st["block"][lo * r:hi * r].double()
        if r > 1:
            w = st["route_weights"][lo:hi].double()
            v = sum(w[:, j:j + 1] * v[j::r] for j in range(r))
        if case["post"]:
            v = stretch(v, st["post"], st["post_bias"])
        if case["gate"] != "none":
            v = v * (st["gate"] if case["gate"] == "channel" else st["gate"][lo:hi]).double()
        v = st["block_scale"] * v + st["residual_scale"] * st["residual"][lo:hi].double()
        new[lo:hi] = v
        out[lo:hi] = stretch(v, st["pre"], st["pre_bias"])
    return {"out": out, "residual": new}


def _exact_lora(st, case):
    ids, ranks = _row_adapters(case), _ranks(case)
    y = st["base"].double()
    for e in sorted(set(ids) - {-1}):
        rows = torch.tensor([t for t, i in enumerate(ids) if i == e], device="cuda")
        x, r, at = st["x"][rows].double(), ranks[e], 0
        for n, a, b in zip(st["n"], st["a"], st["b"]):
            part = (x @ a[e, :r].double().T) @ b[e, :, :r].double().T
            y[rows, at:at + n] += float(st["scale"][e].double()) * part
            at += n
    return {"y": y}


def _exact_route(st, case):
    l = st["logits"].double().cpu().numpy()
    T, E = l.shape
    k, groups = case["topk"], case["groups"]
    if case["scoring"] == "softmax":
        s = np.exp(l - l.max(axis=1, keepdims=True))
        s /= s.sum(axis=1, keepdims=True)
    else:
        s = np.where(l > 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    c = l if not case["bias"] else s + st["bias"].double().cpu().numpy()
    c = c.copy()
    if groups > 1:
        parts = np.sort(c.reshape(T, groups, -1), axis=2)
        best = parts[:, :, -2:].sum(axis=2) if case["bias"] and parts.shape[2] > 1 else parts[:, :, -1]
        order = np.argsort(-best, axis=1, kind="stable")
        out = np.ones((T, groups), dtype=bool)
        np.put_along_axis(out, order[:, :case["top_groups"]], False, axis=1)
        c[np.repeat(out, E // groups, axis=1)] = -np.inf
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, axis=1)
    if st["renormalize"]:
        w = w / w.sum(axis=1, keepdims=True)
    return {"ids": ids, "weights": w * st["scale"]}
