"""The size of a step that skinny_kv_attention takes: its workspace query and its
call agree (no GPU; the addresses are never touched)."""
import pytest

from tests.test_kv_abi import INVALID, UNSUPPORTED, WORKSPACE, attend, batch, cache
import gemv_skinny_gemm_amd as sg

FAR = dict(q=1 << 44, out=2 << 44, ws=3 << 44)


def sizes(seqs, tokens, max_pages, kv_heads, q_heads, **kw):
    c = cache(kv_heads=kv_heads, page_tokens=16, **kw)
    return c, batch(seqs=seqs, tokens=tokens, max_pages=max_pages, page_table=4 << 44), q_heads


@pytest.mark.parametrize("shape", [
    dict(seqs=1, tokens=1 << 20, max_pages=1 << 16, kv_heads=8, q_heads=64),
    dict(seqs=1024, tokens=1024, max_pages=1 << 26, kv_heads=1, q_heads=1),
    dict(seqs=65536, tokens=1 << 20, max_pages=1 << 15, kv_heads=2, q_heads=16),
    dict(seqs=1, tokens=1 << 20, max_pages=1 << 16, kv_heads=8, q_heads=64, head_dim=256),
])
def test_steps_of_too_much_work_have_no_workspace(shape):
    c, b, heads = sizes(**shape)
    assert attend(c=c, b=b, q_heads=heads, n=1 << 40, **FAR) == UNSUPPORTED
    assert sg.kv_attention_workspace_bytes(c, b, heads) == 0


@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("seqs,tokens,kv_heads,q_heads", [(1, 1, 1, 8), (7, 40, 8, 64), (3, 4099, 2, 10),
                                                          (65536, 1 << 20, 1, 1)])
def test_steps_below_the_stated_bound_have_one(seqs, tokens, kv_heads, q_heads, head_dim):
    items = kv_heads * (tokens * (q_heads // kv_heads) / 16 + seqs)
    max_pages = int(min(1 << 26, ((1 << 31) - 2) / items * 32 / 16 - 2))
    while items * (max_pages * 16 / 32 + 1) >= (1 << 31) - 1:
        max_pages -= 1
    c, b, heads = sizes(seqs, tokens, max_pages, kv_heads, q_heads, head_dim=head_dim)
    n = sg.kv_attention_workspace_bytes(c, b, heads)
    assert n > 0
    assert attend(c=c, b=b, q_heads=heads, n=n - 1, **FAR) == WORKSPACE


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_scales_that_log2_e_takes_past_the_largest_number(scale):
    assert attend(scale=scale) == INVALID
    assert attend(scale=2.3e38, n=255) == WORKSPACE         # the next check
