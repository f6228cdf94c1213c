"""The operators of a decode or verify step run as a program runs them: QKV
linear, kv_append, kv_attention, O linear, vocabulary projection with its greedy
token, verify_draft, whose result moves the lengths on for the next step.  Every
stage is checked against its 64-bit form on the very inputs it had, over a prompt
step and several verify steps with drafts kept and rejected (rejected rows stay in
the cache behind the length and are written over), eagerly and as one graph."""
import numpy as np
import pytest
import torch

import gemv_skinny_gemm_amd as sg
import oracle
from tests import kv_util as kv
from tests.gpu_util import host_codes, host_values, need_gpu
from tests.test_verify_gpu import oracle as verify_oracle

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, P, V = 512, 8, 2, 64, 16, 3001
ROWS, SEQS, PAGES, WIDTH = 10, 3, 24, 8
FREQ = kv.frequencies(D)


class Step:
    def __init__(self, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, k=1.0: (k * torch.randn(*s, generator=g, device="cuda")).bfloat16()
        self.dtype = dtype
        self.embed = rnd(V, H)
        self.w_qkv, self.w_o, self.w_head = rnd((HQ + 2 * HKV) * D, H, k=0.05), rnd(H, HQ * D, k=0.05), \
            rnd(V, H, k=0.08)
        shape = (PAGES, HKV, P, D)
        if dtype == "fp8":
            self.k = torch.full(shape, kv.E4M3_NAN, dtype=torch.uint8, device="cuda")
            self.ks = torch.full(shape[:2], float("nan"), device="cuda")
        else:
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            self.ks = None
        self.v, self.vs = self.k.clone(), None if self.ks is None else self.ks.clone()
        order = torch.randperm(PAGES, generator=g, device="cuda").to(torch.int32)
        self.table = order.view(SEQS, WIDTH).contiguous()
        self.freq = torch.from_numpy(FREQ).cuda()
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.q_start, self.kv_len = i32(0, 0, 0, 0), i32(0, 0, 0)
        self.tokens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.au, self.su = torch.zeros(ROWS, device="cuda"), torch.zeros(SEQS, device="cuda")
        self.temps = torch.tensor([0.0, 0.8, 1.0], device="cuda")
        bf = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.x, self.qkv, self.q, self.att = bf(ROWS, H), bf(ROWS, (HQ + 2 * HKV) * D), \
            bf(ROWS, HQ * D), bf(ROWS, HQ * D)
        self.o, self.h, self.logits = bf(ROWS, H), bf(ROWS, H), bf(ROWS, V)
        self.greedy, self.out = torch.zeros_like(self.tokens), torch.zeros_like(self.tokens)
        self.accepted = torch.zeros(SEQS, dtype=torch.int32, device="cuda")
        self.cache = sg.make_kv_cache(self.k, self.v, self.ks, self.vs)
        self.batch = sg.make_batch(self.q_start, self.kv_len, self.table, ROWS)
        self.head = sg.make_linear(self.h, self.w_head, self.logits)
        ws = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
        self.ws = ws(max(sg.workspace_bytes(sg.BF16, ROWS, (HQ + 2 * HKV) * D, H),
                         sg.workspace_bytes(sg.BF16, ROWS, H, HQ * D),
                         sg.lm_head_workspace_bytes(self.head, ROWS),
                         sg.kv_attention_workspace_bytes(self.cache, self.batch, HQ),
                         sg.verify_workspace_bytes(ROWS, SEQS, V)))

    def run(self):
        """One workspace serves every stage, in stream order."""
        self.att.zero_()                       # rows of no sequence are left as they were
        self.x.copy_(self.embed[self.tokens.long()])
        sg.skinny_gemm_bf16(self.x, self.w_qkv, self.qkv, self.ws)
        sg.kv_append(self.cache, self.batch, self.qkv, self.freq, self.q)
        sg.kv_attention(self.cache, self.batch, self.q, self.att, self.ws)
        sg.skinny_gemm_bf16(self.att, self.w_o, self.o, self.ws)
        torch.add(self.x, self.o, out=self.h)
        sg.lm_head_argmax(self.head, ROWS, self.greedy, self.ws)
        sg.verify_draft(self.q_start, self.logits, self.tokens, self.au, self.su, self.out,
                        self.accepted, self.ws, temperature=self.temps)

    def case(self):
        """The batch and the cache as the plain forms take them."""
        c = kv.Case.__new__(kv.Case)
        c.seqs, c.P, c.hq, c.hkv, c.D, c.dtype = [None] * SEQS, P, HQ, HKV, D, self.dtype
        c.q_start, c.kv_len = self.q_start.cpu().numpy(), self.kv_len.cpu().numpy()
        c.T, c.max_pages, c.pages, c.table = ROWS, WIDTH, PAGES, self.table.cpu().numpy()
        code = (lambda t: host_codes(t).copy()) if self.dtype == "bf16" else (lambda t: t.cpu().numpy().copy())
        c.codes = {"k": code(self.k), "v": code(self.v)}
        c.scales = {} if self.ks is None else {"k": self.ks.cpu().numpy(), "v": self.vs.cpu().numpy()}
        c.qkv, c.q = host_codes(self.qkv), host_codes(self.q)
        return c

    def set(self, rows, kv_len, rng):
        self.q_start.copy_(torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32))
        self.kv_len.copy_(kv_len)
        self.au.copy_(torch.from_numpy(rng.random(ROWS).astype(np.float32)))
        self.su.copy_(torch.from_numpy(rng.random(SEQS).astype(np.float32)))
        self.q.fill_(float("nan"))
        self.out.fill_(-9)


def check_step(s, before, what):
    after = s.case()
    before.qkv, before.q_start, before.kv_len = after.qkv, after.q_start, after.kv_len
    before.dev = {"k": s.k, "v": s.v, "out": s.q}
    if s.ks is not None:
        before.dev.update(k_scale=s.ks, v_scale=s.vs)
    kv.assert_append(before, FREQ, what=what)
    n = int(after.q_start[-1])
    att = s.att.clone()
    att[n:] = float("nan")                      # zeroed by the program, checked as untouched
    assert not bool(s.att[n:].any())
    kv.assert_attention(after, att, what=what)
    for x, w, y in ((s.x, s.w_qkv, s.qkv), (s.att, s.w_o, s.o), (s.h, s.w_head, s.logits)):
        ref, a, _ = oracle.linear_bf16(host_codes(x), host_codes(w))
        ok, worst, at = oracle.check(host_values(y), ref, a)
        assert ok, (what, worst, at)
    c = dict(q_start=after.q_start, logits=s.logits.float().cpu().numpy(), draft=None,
             tokens=s.tokens.cpu().numpy(), temperature=s.temps.cpu().numpy(),
             accept_u=s.au.cpu().numpy(), sample_u=s.su.cpu().numpy(), out=np.full(ROWS, -9, np.int32))
    out, accepted = verify_oracle(c)
    assert s.out.tolist() == out.tolist() and s.accepted.tolist() == accepted.tolist(), what
    # The greedy sequence's new token is the vocabulary projection's own.
    if after.q_start[1] > after.q_start[0]:
        row = int(after.q_start[0]) + int(accepted[0])
        assert int(out[row]) == int(s.greedy[row]), what
    return out, accepted


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype", ["fp8", "bf16"])
def test_prompt_then_verify_steps(dtype, graph):
    need_gpu()
    s = Step(dtype, 5)
    rng = np.random.default_rng(6)
    call = s.run
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        call = g.replay
    sure = [0, 0, 0]                                  # tokens of each sequence that are sure
    rows = [4, 3, 2]                                  # the prompts
    s.tokens.copy_(torch.from_numpy(rng.integers(0, V, ROWS).astype(np.int32)))
    kept = 0
    for step in range(18):
        lens = torch.tensor([a + n for a, n in zip(sure, rows)], dtype=torch.int32)
        s.set(rows, lens, rng)
        if step % 4 == 2:
            s.au.zero_()                              # sampled sequences keep every likely draft
        before = s.case()
        call()
        torch.cuda.synchronize()
        out, accepted = check_step(s, before, f"step {step}")
        starts = np.concatenate([[0], np.cumsum(rows)])
        tokens = np.zeros(ROWS, np.int32)
        nxt = [4, 0, 5] if step == 3 else [3, 4, 2] if step % 2 else [1, 5, 4]
        at = 0
        for q in range(SEQS):
            if step == 0:                             # a prompt is sure as a whole
                accepted[q] = rows[q] - 1
            if rows[q]:
                sure[q] += int(accepted[q]) + 1
                kept += int(accepted[q]) if step else 0
                last = int(out[starts[q] + (accepted[q] if step else 0)]) % V
            else:
                last = int(rng.integers(0, V))
            if nxt[q]:
                tokens[at] = last
                # Drafts: the target's likely tokens, some of them good.
                top = torch.topk(s.logits[max(0, starts[q + 1] - 1)].float(), 3).indices.tolist()
                for i in range(1, nxt[q]):
                    tokens[at + i] = top[int(rng.integers(0, 3))]
                at += nxt[q]
        rows = nxt
        s.tokens.copy_(torch.from_numpy(tokens))
    assert min(sure) > P and kept > 0                 # pages were crossed, drafts kept


def test_structs_know_their_tensors_and_gpu():
    """A cache or batch holds the tensors that it points to, and a call whose
    tensors lie on another GPU than either is refused."""
    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    cache = sg.make_kv_cache(k, k.clone())
    batch = sg.make_batch(ints(0, 1), ints(1), ints(0)[None], 1)
    assert cache.v == cache.tensors[1].data_ptr()
    assert batch.page_table == batch.tensors[2].data_ptr()
    qkv = torch.zeros((1, 3 * 64), dtype=torch.bfloat16, device="cuda")
    q = qkv[:, :64].clone()
    ws = torch.empty(sg.kv_attention_workspace_bytes(cache, batch, 1), dtype=torch.uint8,
                     device="cuda")
    for struct in (cache, batch):
        struct.gpu += 1
        with pytest.raises(ValueError, match="the call's tensors on GPU 0"):
            sg.kv_append(cache, batch, qkv, None, q)
        with pytest.raises(ValueError, match="the call's tensors on GPU 0"):
            sg.kv_attention(cache, batch, q, q.clone(), ws)
        struct.gpu -= 1
    with pytest.raises(ValueError, match="on the GPU"):
        sg.kv_attention(cache, batch, q, q.clone(), ws.cpu())
    sg.kv_append(cache, batch, qkv, None, q)
    sg.kv_attention(cache, batch, q, q.clone(), ws)
    torch.cuda.synchronize()
