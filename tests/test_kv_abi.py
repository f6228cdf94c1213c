"""The paged-cache entry points and their binding refuse bad arguments on the
host, before anything is enqueued (no GPU; the addresses are never touched)."""
import ctypes

import pytest
import torch

import gemv_skinny_gemm_amd as sg

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
K, V, KS, VS = 0x10000000, 0x20000000, 0x30000000, 0x31000000
QS, KL, PT = 0x32000000, 0x33000000, 0x34000000
QKV, Q, OUT, FREQ, WS = 0x40000000, 0x50000000, 0x60000000, 0x70000000, 0x80000000


def cache(**kw):
    a = dict(dtype=sg.KV_FP8, pages=40, kv_heads=2, page_tokens=16, head_dim=64, reserved=0, k=K,
             v=V, k_scale=KS, v_scale=VS)
    a.update(kw)
    return sg.KvCache(*a.values())


def batch(**kw):
    a = dict(seqs=3, tokens=5, max_pages=10, reserved=0, q_start=QS, kv_len=KL, page_table=PT)
    a.update(kw)
    return sg.KvBatch(*a.values())


def append(c=None, b=None, qkv=QKV, q_heads=8, freq=FREQ, rot=64, inter=0, out=OUT):
    c = cache() if c is None else c
    b = batch() if b is None else b
    return sg.lib().skinny_kv_append(c, b, qkv, q_heads, freq, rot, inter, out, None)


def attend(c=None, b=None, q=Q, q_heads=8, scale=0.125, out=OUT, ws=WS, n=None):
    c = cache() if c is None else c
    b = batch() if b is None else b
    n = 1 << 30 if n is None else n
    return sg.lib().skinny_kv_attention(c, b, q, q_heads, scale, out, ws, n, None)


BAD_CACHES = [
    (dict(dtype=2), INVALID), (dict(reserved=1), INVALID), (dict(pages=0), INVALID),
    (dict(kv_heads=0), INVALID), (dict(page_tokens=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_scale=None), INVALID),
    (dict(v_scale=None), INVALID), (dict(dtype=sg.KV_BF16), INVALID),   # scales of a bf16 cache
    (dict(page_tokens=8), UNSUPPORTED), (dict(page_tokens=48), UNSUPPORTED),
    (dict(page_tokens=256), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(kv_heads=2048), UNSUPPORTED), (dict(k=K + 8), UNSUPPORTED), (dict(v=V + 4), UNSUPPORTED),
    (dict(k_scale=KS + 2), UNSUPPORTED),
]
BAD_BATCHES = [
    (dict(seqs=0), INVALID), (dict(tokens=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(reserved=3), INVALID), (dict(q_start=None), INVALID), (dict(kv_len=None), INVALID),
    (dict(page_table=None), INVALID), (dict(seqs=65537), UNSUPPORTED),
    (dict(tokens=(1 << 20) + 1), UNSUPPORTED), (dict(max_pages=(1 << 26) + 1), UNSUPPORTED),
    (dict(q_start=QS + 2), UNSUPPORTED), (dict(page_table=PT + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(kw, status):
    assert append(c=cache(**kw)) == status
    assert attend(c=cache(**kw)) == status
    assert sg.kv_attention_workspace_bytes(cache(**kw), batch(), 8) == 0


@pytest.mark.parametrize("kw,status", BAD_BATCHES)
def test_bad_batches(kw, status):
    assert append(b=batch(**kw)) == status
    assert attend(b=batch(**kw)) == status
    assert sg.kv_attention_workspace_bytes(cache(), batch(**kw), 8) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(qkv=None), INVALID), (dict(out=None), INVALID), (dict(q_heads=0), INVALID),
    (dict(q_heads=7), INVALID), (dict(q_heads=2048), UNSUPPORTED), (dict(rot=-4), INVALID),
    (dict(rot=68), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=0), INVALID),
    (dict(freq=None), INVALID), (dict(inter=2), INVALID), (dict(qkv=QKV + 8), UNSUPPORTED),
    (dict(out=OUT + 2), UNSUPPORTED), (dict(freq=FREQ + 1), UNSUPPORTED),
    (dict(out=QKV), INVALID), (dict(out=K + 64), INVALID), (dict(out=KS + 16), INVALID),
    (dict(out=QS), INVALID), (dict(out=FREQ), INVALID), (dict(qkv=V + 32), INVALID),
    (dict(freq=VS), INVALID), (dict(c=cache(v=K + 128)), INVALID),
    (dict(c=cache(k_scale=K)), INVALID), (dict(c=cache(v_scale=KS + 4)), INVALID),
    (dict(b=batch(kv_len=K)), INVALID),
    (dict(b=batch(tokens=1 << 20), q_heads=1024, c=cache(kv_heads=1024), qkv=1 << 44, out=2 << 44),
     UNSUPPORTED),                                # more workgroups than a launch holds
])
def test_append_refuses(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q_heads=3), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=Q + 8), UNSUPPORTED), (dict(out=OUT + 8), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(n=255), WORKSPACE), (dict(ws=WS + 8), UNSUPPORTED), (dict(out=Q), INVALID),
    (dict(out=WS + 64), INVALID), (dict(q=WS + 64), INVALID), (dict(out=V), INVALID),
    (dict(ws=K), INVALID), (dict(ws=PT), INVALID), (dict(out=KL), INVALID),
])
def test_attention_refuses(kw, status):
    assert attend(**kw) == status


def test_null_structs():
    L = sg.lib()
    assert L.skinny_kv_append(None, batch(), QKV, 8, FREQ, 64, 0, OUT, None) == INVALID
    assert L.skinny_kv_append(cache(), None, QKV, 8, FREQ, 64, 0, OUT, None) == INVALID
    assert L.skinny_kv_attention(None, batch(), Q, 8, 0.1, OUT, WS, 1 << 30, None) == INVALID
    assert L.skinny_kv_attention(cache(), None, Q, 8, 0.1, OUT, WS, 1 << 30, None) == INVALID
    assert L.skinny_kv_attention_workspace_bytes(None, None, 8) == 0


def test_workspace_is_host_arithmetic():
    small = sg.kv_attention_workspace_bytes(cache(), batch(seqs=1, tokens=1, max_pages=1), 2)
    assert small >= 256
    long = sg.kv_attention_workspace_bytes(cache(), batch(seqs=1, tokens=1, max_pages=8192), 8)
    assert small < long
    # It does not grow with the batch beyond the grid's own share.
    wide = sg.kv_attention_workspace_bytes(cache(), batch(seqs=16, tokens=16, max_pages=8192), 8)
    assert wide == long
    # The exact size is accepted (host checks pass as far as the device query).
    assert attend(n=sg.kv_attention_workspace_bytes(cache(), batch(), 8) - 1) == WORKSPACE


def test_binding_checks_tensors():
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    k = torch.zeros((4, 2, 16, 64), dtype=u8)
    s = torch.zeros((4, 2))
    with pytest.raises(ValueError, match="4-D"):
        sg.make_kv_cache(k[0], k[0])
    with pytest.raises(ValueError, match="come together"):
        sg.make_kv_cache(k, k, s)
    with pytest.raises(ValueError, match="v: shape"):
        sg.make_kv_cache(k, k[:, :, :, :32], s, s)
    with pytest.raises(ValueError, match="k: dtype"):
        sg.make_kv_cache(k, k)                                   # e4m3 codes without scales
    with pytest.raises(ValueError, match="k: dtype"):
        sg.make_kv_cache(k.to(bf), k.to(bf), s, s)
    with pytest.raises(ValueError, match="v_scale: shape"):
        sg.make_kv_cache(k, k, s, torch.zeros((4, 1)))
    with pytest.raises(ValueError, match="k_scale: dtype"):
        sg.make_kv_cache(k, k, s.double(), s)
    with pytest.raises(ValueError, match="on the GPU"):
        sg.make_kv_cache(k, k, s, s)
    with pytest.raises(ValueError, match="contiguous"):
        sg.make_kv_cache(torch.zeros((4, 16, 2, 64), dtype=u8).transpose(1, 2), k, s, s)
    q0, n, t = torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros((3, 5), dtype=i32)
    with pytest.raises(ValueError, match="q_start: shape"):
        sg.make_batch(n, n, t, 3)
    with pytest.raises(ValueError, match="kv_len: dtype"):
        sg.make_batch(q0, n.long(), t, 3)
    with pytest.raises(ValueError, match="page_table: dtype"):
        sg.make_batch(q0, n, t.long(), 3)
    with pytest.raises(ValueError, match="on the GPU"):
        sg.make_batch(q0, n, t, 3)
    c, b = cache(), batch()                                       # 2 KV heads of 64, 5 rows
    qkv, q = torch.zeros((5, 12 * 64), dtype=bf), torch.zeros((5, 8 * 64), dtype=bf)
    freq = torch.zeros(32)
    for kw, what in ((dict(qkv=qkv[:4]), "qkv: shape"), (dict(qkv=qkv[:, :-2]), "qkv: shape"),
                     (dict(qkv=qkv.float()), "qkv: dtype"), (dict(q_out=q[:, :64]), "q_out: shape"),
                     (dict(inv_freq=freq.double()), "inv_freq: dtype"),
                     (dict(inv_freq=freq.view(2, 16)), "inv_freq: shape"),
                     (dict(), "on the GPU")):
        a = {**dict(qkv=qkv, inv_freq=freq, q_out=q), **kw}
        with pytest.raises(ValueError, match=what):
            sg.kv_append(c, b, a["qkv"], a["inv_freq"], a["q_out"], stream=0)
    for kw, what in ((dict(q=q[:3]), "q: shape"), (dict(out=q[:, :64]), "out: shape"),
                     (dict(out=q.float()), "out: dtype"), (dict(), "on the GPU")):
        a = {**dict(q=q, out=q.clone()), **kw}
        with pytest.raises(ValueError, match=what):
            sg.kv_attention(c, b, a["q"], a["out"], (WS, 1 << 30), stream=0)
