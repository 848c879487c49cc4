"""Attention of some thousand sequences in a call."""
import pytest
import torch

import test_gpu_attention_decode as D
import test_gpu_attention_prefill as P
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import attention
    return attention


def some(n):
    """The sequences looked at: runs at the beginning, around the middle and at the end, which cross the
    kernels' steps of 64."""
    return [range(0, 30), range(n // 2 - 40, n // 2 + 40), range(n - 70, n)]


@pytest.mark.parametrize("b,q_heads,heads,d,long", [(4100, 2, 1, 64, 900), (5000, 4, 2, 128, 3000), (65536, 1, 1, 16, 40)])
def test_decode(att, b, q_heads, heads, d, long):
    say("decode batch", b, q_heads, heads, d, long)
    page, pages = 16, 700
    s = D.setup(att, [page * pages], 1, q_heads, heads, d, page, seed=b)   # one long sequence, whose pages all share
    g = torch.Generator(device="cuda").manual_seed(b)
    per = -(-long // page)
    lens = torch.randint(0, min(long, 150) + 1, (b,), device="cuda", generator=g, dtype=torch.int32)
    lens[torch.tensor([3, b // 2, b // 2 + 1, b - 64, b - 1], device="cuda")] = long
    lens[b - 2] = 0
    s.update(block_table=s["block_table"][0, :pages][torch.randint(0, pages, (b, per), device="cuda", generator=g)].contiguous(), lengths=lens,
             q=torch.randn(b, 1, q_heads, d, device="cuda", generator=g).bfloat16())
    lse = torch.full(s["q"].shape[:3], 7.0, device="cuda")
    out = att.nvfp4_attention_decode(**s, lse=lse)
    for part in some(b):
        cut = slice(part.start, part.stop)
        D.check({**s, "q": s["q"][cut], "block_table": s["block_table"][cut], "lengths": lens[cut]}, out[cut], lse[cut])
    if long <= 1024:   # sequences that no call splits: the same bits in small batches
        small = torch.cat([att.nvfp4_attention_decode(**{**s, "q": s["q"][i:i + 512], "block_table": s["block_table"][i:i + 512].contiguous(), "lengths": lens[i:i + 512].contiguous()})
                           for i in range(0, b, 512)])
        assert torch.equal(out, small)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("b,most,prefix,q_heads,heads,d", [(4100, 9, 0, 4, 4, 64), (5000, 70, 30, 8, 2, 128), (20000, 2, 1, 1, 1, 256)])
def test_prefill(att, b, most, prefix, q_heads, heads, d, causal):
    say("prefill batch", b, most, prefix, q_heads, heads, d, causal)
    g = torch.Generator().manual_seed(b)
    lq = torch.randint(0, most + 1, (b,), generator=g)
    lk = lq + torch.randint(0, prefix + 1, (b,), generator=g)
    q, k, v, cq, ck = P.inputs(lq.tolist(), lk.tolist(), q_heads, heads, d, b)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = att.attention_prefill(q, k, v, cq, ck, causal=causal, lse=lse)
    for part in some(b):
        a, c = cq[part.start:part.stop + 1], ck[part.start:part.stop + 1]
        P.check(q, k, v, a, c, causal, out, lse)
