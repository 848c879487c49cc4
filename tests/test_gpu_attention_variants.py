"""Every variant of the attention kernels (attention_cases.py) against its 64-bit form."""
import pytest
import torch

import attention_cases as C
import test_gpu_attention_decode as D
import test_gpu_attention_prefill as P
import test_gpu_rope_cache as R
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import attention
    return attention


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,q_heads,heads,d", C.PREFILL)
def test_prefill(att, lq, lk, q_heads, heads, d, causal):
    say("prefill variant", lq[:4], lk[:4], len(lq), q_heads, heads, d, causal)
    q, k, v, cq, ck = P.inputs(lq, lk, q_heads, heads, d, sum(lk) + d)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = att.attention_prefill(q, k, v, cq, ck, causal=causal, lse=lse)
    P.check(q, k, v, cq, ck, causal, out, lse)
    again = torch.full_like(out, float("nan"))
    att.attention_prefill(q, k, v, cq, ck, causal=causal, out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lq,lk,q_heads,heads,d", C.PREFILL)
def test_behind_the_mask(att, bad, lq, lk, q_heads, heads, d):
    """A key or value of the first sequence that is not finite: the rows that do not see it, other heads and
    other sequences come out as without it."""
    say("prefill variant behind the mask", bad, lq[:4], lk[:4], len(lq), q_heads, heads, d)
    q, k, v, cq, ck = P.inputs(lq, lk, q_heads, heads, d, 11)
    clean = att.attention_prefill(q, k, v, cq, ck)
    n, m = lq[0], lk[0]
    at = m - 1 - n // 3          # a third of the rows sees it
    first, group = at - (m - n), q_heads // heads
    head = heads - 1
    mine = slice(head * group, q_heads)
    for which in (k, v):
        x = which.clone()
        x[at, head, 7] = bad
        out = att.attention_prefill(q, x if which is k else k, x if which is v else v, cq, ck)
        same = out == clean
        assert bool(same[:first].all()) and bool(same[n:].all()) and bool(same[:, : head * group].all()), which is k
        if which is v:
            assert not bool(out[first:n, mine, 7].isfinite().any())
            assert bool(same[..., :7].all()) and bool(same[..., 8:].all())


@pytest.mark.parametrize("lens,new,q_heads,heads,d,page,wide", C.DECODE)
def test_decode(att, lens, new, q_heads, heads, d, page, wide):
    say("decode variant", lens[:4], len(lens), new, q_heads, heads, d, page, wide)
    s = D.setup(att, lens, new, q_heads, heads, d, page, seed=len(lens) + d)
    if wide:
        table = torch.full((len(lens), wide // page), -7, dtype=torch.int32, device="cuda")
        table[:, : s["block_table"].shape[1]] = s["block_table"]
        s["block_table"] = table
    lse = torch.full(s["q"].shape[:3], 7.0, device="cuda")
    ws = torch.full((att.attention_ws_bytes(len(lens), d),), 0xFF, dtype=torch.uint8, device="cuda")
    out = att.nvfp4_attention_decode(**s, lse=lse, workspace=ws)
    D.check(s, out, lse)
    again = torch.full_like(out, float("nan"))
    att.nvfp4_attention_decode(**s, out=again, workspace=ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,heads,d,sections", C.ROPE)
def test_rope(att, t, heads, d, sections, inter):
    R.test_rope(att, t, heads, d, sections, inter)


@pytest.mark.parametrize("t,heads,d,page", C.ROWS)
def test_append_and_read(att, t, heads, d, page):
    R.test_append_and_read(att, t, heads, d, page)
