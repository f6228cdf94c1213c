"""skinny_verify_draft and its binding refuse bad arguments on the host (no GPU;
the addresses are never touched)."""
import pytest
import torch

import gemv_skinny_gemm_amd as sg

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
QS, LOG, DR, TOK, TMP, AU, SU, OUT, ACC, WS = (0x10000000 * (i + 1) for i in range(10))


def call(ws=WS, n=1 << 24, **kw):
    a = dict(dtype=sg.LOGITS_BF16, vocab=1000, rows=4, seqs=2, q_start=QS, logits=LOG, draft=DR,
             tokens=TOK, temperature=TMP, accept_u=AU, sample_u=SU, out=OUT, accepted=ACC)
    a.update(kw)
    return sg.lib().skinny_verify_draft(sg.Verify(*a.values()), ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), INVALID), (dict(vocab=0), INVALID), (dict(rows=0), INVALID),
    (dict(seqs=0), INVALID), (dict(q_start=None), INVALID), (dict(logits=None), INVALID),
    (dict(tokens=None), INVALID), (dict(accept_u=None), INVALID), (dict(sample_u=None), INVALID),
    (dict(out=None), INVALID), (dict(accepted=None), INVALID),
    (dict(vocab=(1 << 24) + 1), UNSUPPORTED), (dict(rows=65536), UNSUPPORTED),
    (dict(seqs=65536), UNSUPPORTED), (dict(logits=LOG + 1), UNSUPPORTED),
    (dict(draft=DR + 1), UNSUPPORTED), (dict(dtype=sg.LOGITS_F32, logits=LOG + 2), UNSUPPORTED),
    (dict(tokens=TOK + 2), UNSUPPORTED), (dict(temperature=TMP + 1), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE), (dict(ws=WS + 8), UNSUPPORTED),
    (dict(out=LOG + 16), INVALID), (dict(out=TOK), INVALID), (dict(accepted=OUT), INVALID),
    (dict(accepted=SU), INVALID), (dict(ws=DR), INVALID), (dict(out=WS + 64), INVALID),
    (dict(ws=TMP), INVALID),
])
def test_refuses(kw, status):
    assert call(**kw) == status


def test_null_and_workspace():
    assert sg.lib().skinny_verify_draft(None, WS, 1 << 20, None) == INVALID
    assert sg.verify_workspace_bytes(0, 1, 10) == 0
    assert sg.verify_workspace_bytes(1, 1, (1 << 24) + 1) == 0
    n = sg.verify_workspace_bytes(4, 2, 1000)
    assert 0 < n < sg.verify_workspace_bytes(4, 2, 100000)
    assert call(n=n - 1) == WORKSPACE


def test_binding_checks_tensors():
    i32 = torch.int32
    good = dict(q_start=torch.zeros(3, dtype=i32), logits=torch.zeros((4, 50), dtype=torch.bfloat16),
                tokens=torch.zeros(4, dtype=i32), accept_u=torch.zeros(4), sample_u=torch.zeros(2),
                out_tokens=torch.zeros(4, dtype=i32), accepted=torch.zeros(2, dtype=i32),
                workspace=(WS, 1 << 20), draft_logits=None, temperature=None, stream=0)
    for kw, what in (
            (dict(logits=good["logits"].double()), "logits: dtype"),
            (dict(draft_logits=good["logits"].float()), "draft_logits: dtype"),
            (dict(draft_logits=good["logits"][:3]), "draft_logits: shape"),
            (dict(q_start=torch.zeros(2, dtype=i32)), "q_start: shape"),
            (dict(tokens=torch.zeros(4, dtype=torch.int64)), "tokens: dtype"),
            (dict(accept_u=torch.zeros(3)), "accept_u: shape"),
            (dict(temperature=torch.zeros(4)), "temperature: shape"),
            (dict(out_tokens=torch.zeros(5, dtype=i32)), "out_tokens: shape"),
            (dict(accepted=torch.zeros(2)), "accepted: dtype"), (dict(), "on the GPU")):
        with pytest.raises(ValueError, match=what):
            sg.verify_draft(**{**good, **kw})


def test_workspace_of_a_larger_step_holds_a_smaller_one():
    """Sized once for the most rows, sequences and entries, it does for less."""
    sizes = [1, 2, 3, 16, 51, 52, 102, 103, 170, 171, 512, 1024, 1025, 4000]
    vocabs = [1, 2048, 2049, 4096, 4097, 12288, 12289, 20480, 32003, 131072, 131073, 152064]
    for most in (sizes, vocabs):
        got = [sg.verify_workspace_bytes(*((n, 5, 20480) if most is sizes else (7, 5, n)))
               for n in most]
        assert got == sorted(got) and got[0] > 0
    got = [sg.verify_workspace_bytes(40, n, 32003) for n in sizes]
    assert got == sorted(got)
    # Either length of slices fits: statistics (16 bytes) of each row's slices,
    # the target's and the draft's, and four sums of each sequence's.
    for rows in sizes:
        for vocab in vocabs:
            short = -(-vocab // 2048)
            slices = short if short <= 64 and rows * short <= 1024 else -(-vocab // 4096)
            need = 2 * rows * slices * 16 + 5 * slices * 32 + 8 * rows + 20
            assert sg.verify_workspace_bytes(rows, 5, vocab) >= need
