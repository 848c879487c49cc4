"""Attention whose scores, probabilities or values lie many binades apart, against its 64-bit form."""
import pytest
import torch

import attention_ref as A
from gpu_util import say
from serving_ref import gamma

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import attention
    return attention


def one_key_takes_all(q, k, v, scale, seen, out, lse):
    """Scores so large that fp32 holds them to whole units or worse.  Where the largest (or several equal
    ones) lead by more than their error, the others' weights are zero and what comes out is the leaders'
    mean, its probabilities and itself rounded to bf16 at worst (2^-8 each, and 2^-20 of sums); anywhere else it lies among
    the values.  Returns the number of rows with such a lead."""
    x = (q @ k.t() * scale).masked_fill(~seen, -float("inf"))
    dx = (gamma(q.shape[1]) * (q.abs() @ k.abs().t()) * scale + 2.0 ** -21 * x.abs()).masked_fill(~seen, 0).amax(-1)
    top = x.amax(-1, keepdim=True)
    first = x >= top * (1 - 2.0 ** -40 * top.sign())   # (equal but for the 64-bit sums' own rounding)
    lead = top[:, 0] - x.masked_fill(first, -float("inf")).amax(-1) > 2 * dx + 100
    ref = first.double() @ v / first.sum(-1, keepdim=True)
    size = first.double() @ v.abs() / first.sum(-1, keepdim=True)
    assert bool(((out.double() - ref).abs() <= size * (2.0 ** -7 + 2.0 ** -15))[lead].all())
    assert bool((out.double().abs() <= v.abs().amax(0) * (1 + 2.0 ** -6)).all())
    assert bool(((lse.double() - (top[:, 0] + first.sum(-1).log())).abs() <= dx + 2.0 ** -21 * top[:, 0].abs() + 1)[lead].all())
    return int(lead.sum())


@pytest.mark.parametrize("power", [20, 27, 31, 60])
@pytest.mark.parametrize("n,new,q_heads,heads,d", [(900, 1, 8, 2, 128), (3000, 3, 16, 2, 64), (500, 1, 4, 2, 256), (65, 1, 3, 3, 80)])
def test_decode_with_scores_past_the_units_of_fp32(att, n, new, q_heads, heads, d, power):
    say("decode large scores", n, new, q_heads, heads, d, power)
    g = torch.Generator(device="cuda").manual_seed(n)
    page, b = 16, 2
    pages = -(-n // page)
    kv = torch.full((pages, 2, heads, page, d // 2), 0xFF, dtype=torch.uint8, device="cuda")
    sf = torch.full((pages, 2, heads, d // 16, page), 0xFF, dtype=torch.uint8, device="cuda")
    gs = torch.tensor([2688 / 6.0, 2688 / 5.0], device="cuda")
    k, v = (torch.randn(n, heads, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    k[n // 2] = k[n // 3]
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    att.nvfp4_kv_append(k, v, slots, gs, kv, sf)
    q = (torch.randn(b, new, q_heads, d, device="cuda", generator=g) * 2.0 ** power).bfloat16()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(b, -1).contiguous()
    lse = torch.empty(b, new, q_heads, device="cuda")
    out = att.nvfp4_attention_decode(q, kv, sf, gs, table, torch.full((b,), n, dtype=torch.int32, device="cuda"), lse=lse)
    assert bool(out.isfinite().all())
    kk, vv = (A.rows(kv, sf, w, slots) / gs[w].double() for w in (0, 1))
    seen = torch.arange(n, device="cuda") < (n - (new - 1 - torch.arange(new, device="cuda")))[:, None]
    led = sum(one_key_takes_all(q[i, :, h].double(), kk[:, h * heads // q_heads], vv[:, h * heads // q_heads], d ** -0.5, seen, out[i, :, h], lse[i, :, h])
              for i in range(b) for h in range(q_heads))
    assert led >= 0.8 * b * new * q_heads


@pytest.mark.parametrize("power", [20, 31, 33, 60])
@pytest.mark.parametrize("lq,lk,q_heads,heads,d", [((150, 40), (150, 90), 4, 2, 128), ((700,), (700,), 2, 2, 64), ((60,), (60,), 2, 1, 256), ((5,), (3000,), 4, 1, 128),
                                                   ((300,) * 9, (300,) * 9, 16, 8, 96)])
def test_prompts_with_scores_past_the_units_of_fp32(att, lq, lk, q_heads, heads, d, power):
    say("prefill large scores", lq, lk, q_heads, heads, d, power)
    g = torch.Generator(device="cuda").manual_seed(sum(lk))
    q = (torch.randn(sum(lq), q_heads, d, device="cuda", generator=g) * 2.0 ** power).bfloat16()
    k, v = (torch.randn(sum(lk), heads, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    k[9] = k[3]
    cq, ck = (torch.tensor((0,) + n, device="cuda").cumsum(0).int() for n in (lq, lk))
    for causal in (True, False):
        lse = torch.empty(q.shape[:2], device="cuda")
        out = att.attention_prefill(q, k, v, cq, ck, causal=causal, lse=lse)
        assert bool(out.isfinite().all())
        led = 0
        for i, (n, m) in enumerate(zip(lq, lk)):
            r, c = slice(int(cq[i]), int(cq[i + 1])), slice(int(ck[i]), int(ck[i + 1]))
            seen = torch.arange(m, device="cuda") <= ((torch.arange(n, device="cuda") + m - n) if causal else torch.full((n,), m, device="cuda"))[:, None]
            led += sum(one_key_takes_all(q[r, h].double(), k[c, h * heads // q_heads].double(), v[c, h * heads // q_heads].double(), d ** -0.5, seen, out[r, h], lse[r, h])
                       for h in range(q_heads))
        assert led >= 0.8 * sum(lq) * q_heads


# Probabilities enter the product as fp16: half a step is 2^-11 of themselves, or, in fp16's
# subnormals, 2^-25, where the largest is at least 2^12.5: 2^-37.5 of the largest.
HALF_STEP, TINY = 2.0 ** -11, 2.0 ** -37


@pytest.mark.parametrize("depth", [9.0, 14.0, 17.5, 18.5])
@pytest.mark.parametrize("b,n,at,new,q_heads,heads,d,page", [
    (64, 32768, range(100, 32768, 4096), 1, 8, 8, 128, 64), (64, 32768, range(0, 32768, 2048), 1, 8, 8, 64, 64), (3, 1000, (0,), 1, 8, 2, 128, 16),
    (3, 1000, (999,), 1, 4, 2, 256, 16), (40, 9000, range(50, 9000, 1000), 1, 6, 6, 80, 32), (2, 70, (1,), 1, 3, 3, 96, 16),
    (32, 16384, range(16000, 0, -1000), 5, 32, 8, 128, 64), (2, 300, (7, 200), 3, 8, 1, 48, 16),
])
def test_few_keys_far_above_the_others(att, depth, b, n, at, new, q_heads, heads, d, page):
    """Keys `at` score `depth` above all others (which score 0) and hold zeros: what comes out is the
    others' alone, e^-depth each.  All sequences read the same pages, as ones with a prefix in common do."""
    say("decode depth", depth, b, n, new, q_heads, heads, d, page)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    pages = -(-n // page)
    kv = torch.full((pages, 2, heads, page, d // 2), 0xFF, dtype=torch.uint8, device="cuda")
    sf = torch.full((pages, 2, heads, d // 16, page), 0xFF, dtype=torch.uint8, device="cuda")
    gs = torch.tensor([2688 / 2.0, 2688 / 4.0], device="cuda")
    k = torch.zeros(n, heads, d, device="cuda")
    v = 1 + torch.rand(n, heads, d, device="cuda", generator=g)
    k[list(at)], v[list(at)] = 1.0, 0.0
    order = torch.randperm(pages, device="cuda", generator=g).int()
    j = torch.arange(n, device="cuda")
    slots = (order[j // page] * page + j % page).int()
    att.nvfp4_kv_append(k.bfloat16(), v.bfloat16(), slots, gs, kv, sf)
    q = torch.ones(b, new, q_heads, d, device="cuda").bfloat16()
    table = order.expand(b, -1).contiguous()
    lengths = torch.full((b,), n, dtype=torch.int32, device="cuda")
    key = A.rows(kv, sf, 0, slots) / gs[0].double()
    val = A.rows(kv, sf, 1, slots) / gs[1].double()
    scale = depth / key[at[0], 0].sum().item()
    lse = torch.empty(b, new, q_heads, device="cuda")
    out = att.nvfp4_attention_decode(q, kv, sf, gs, table, lengths, scale=scale, lse=lse)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    group = q_heads // heads
    seen = j < (n - (new - 1 - torch.arange(new, device="cuda")))[:, None]
    for h in range(q_heads):
        ref, rl, bound, dl = A.attend(q[0, :, h].double(), key[:, h // group], val[:, h // group], scale, seen, HALF_STEP, TINY)
        worst = A.worst(out[0, :, h], ref, bound)
        assert worst <= 1.0, (h, worst, (out[0, :, h].double() / ref).amin().item())
        assert A.same_lse(lse[0, :, h], rl, dl), h


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,q_heads,heads,d", [
    ((200, 70), (200, 70), 4, 2, 128), ((90,), (300,), 2, 2, 64), ((130,), (257,), 2, 1, 256), ((300,) * 9, (300,) * 9, 16, 8, 96), ((3, 20) * 20, (90, 20) * 20, 32, 8, 128),
    ((7, 16), (5000, 3111), 8, 2, 128), ((5,), (2000,), 3, 3, 64), ((2300, 1900), (2300, 1900), 16, 16, 128), ((200, 300), (200, 300), 64, 64, 256),
])
def test_prompts_with_values_near_the_largest(att, lq, lk, q_heads, heads, d, causal):
    """Values of 2^122, and keys whose scores rise by less than makes the maximum move: the result is an
    average, and fp32 holds every sum on the way while no probability is above one (about a hundred keys
    count as much as the largest at most, of random sign).  Bounds as of any prompt: probabilities and
    outputs in bf16."""
    say("prefill large values", lq[:4], lk[:4], q_heads, heads, d, causal)
    g = torch.Generator(device="cuda").manual_seed(sum(lk) + d)
    r = lambda t, h: torch.randn(t, h, d, device="cuda", generator=g)  # noqa: E731
    q, k, v = r(sum(lq), q_heads), r(sum(lk), heads) * 0.25, r(sum(lk), heads)
    cq, ck = (torch.tensor((0,) + n, device="cuda").cumsum(0).int() for n in (lq, lk))
    q[..., 0] = d ** 0.5
    at = torch.cat([torch.arange(n, device="cuda") for n in lk])
    k[..., 0] = (at > 7).float()[:, None]             # past the first keys
    k[..., 0] += 4.2 * (at % 67 == 66).float()[:, None]   # and now and then a score of 5.2: 2^7.5
    q, k, v = q.bfloat16(), k.bfloat16(), (v.clamp(-3, 3) * 2.0 ** 120.5).bfloat16()
    lse = torch.empty(q.shape[:2], device="cuda")
    out = att.attention_prefill(q, k, v, cq, ck, causal=causal, lse=lse)
    for i, (n, m) in enumerate(zip(lq, lk)):
        a, c = slice(int(cq[i]), int(cq[i + 1])), slice(int(ck[i]), int(ck[i + 1]))
        seen = torch.arange(m, device="cuda") <= ((torch.arange(n, device="cuda") + m - n) if causal else torch.full((n,), m, device="cuda"))[:, None]
        for h in range(q_heads):
            ref, rl, bound, dl = A.attend(q[a, h].double(), k[c, h * heads // q_heads].double(), v[c, h * heads // q_heads].double(), d ** -0.5, seen, 2.0 ** -8, 0.0)
            assert bool(out[a, h].isfinite().all()), (i, h)
            assert A.worst(out[a, h], ref, bound) <= 1.0, (i, h)
            assert A.same_lse(lse[a, h], rl, dl), (i, h)


@pytest.mark.parametrize("scales", [(7e-36, 1e-36), (3e38, 1e37), (float("inf"), 2.0 ** 126), (1e-39, 2.0 ** -149), (2.0 ** -112, 2.0 ** 112), (2.0 ** -113, 2.0 ** 113),
                                    (1.1 * 2.0 ** -116, 1.7 * 2.0 ** 120), (2688 / 3.3895e38, 2688 / 1e-38)])
def test_read_with_any_global_scale(att, scales):
    """bf16 of the correctly rounded fp32 quotient, infinite and subnormal ones among them, for every
    code and scale."""
    say("read scales", scales)
    kv, sf = torch.zeros(16, 2, 1, 16, 16, dtype=torch.uint8, device="cuda"), torch.zeros(16, 2, 1, 2, 16, dtype=torch.uint8, device="cuda")
    flat, fsf = kv.view(16, 2, 16, 16), sf.view(16, 2, 2, 16)
    flat[:] = torch.arange(16, dtype=torch.uint8, device="cuda").repeat(16).view(16, 16) * 16 + torch.arange(16, dtype=torch.uint8, device="cuda")
    fsf[:] = torch.arange(512, device="cuda").remainder(127).to(torch.uint8).view(16, 2, 16).unsqueeze(1)
    slots = torch.arange(256, dtype=torch.int32, device="cuda")
    gs = torch.tensor(scales, dtype=torch.float32, device="cuda")
    for which, o in enumerate(att.nvfp4_kv_read(slots, gs, kv, sf)):
        want = (A.rows(kv, sf, which, slots).float().cpu() / gs[which].cpu()).bfloat16()
        assert not bool(want.isnan().any())
        same = o.cpu() == want
        assert bool(same.all()), (which, int((~same).sum()))


@pytest.mark.parametrize("size", [1e-35, 1e-34, 1e-30, 1e33, 3e37])
@pytest.mark.parametrize("lens,q_heads,heads,d", [((900, 40), 8, 2, 128), ((5000,), 4, 4, 64), ((9000, 30), 6, 1, 256)])
def test_decode_with_very_small_and_large_values(att, size, lens, q_heads, heads, d):
    """The global scale of values near either end of bf16's range, whole sequences and parts."""
    say("decode size of values", size, lens, q_heads, heads, d)
    g = torch.Generator(device="cuda").manual_seed(d)
    page, most, b = 16, max(lens), len(lens)
    pages = -(-most // page)
    kv = torch.full((pages, 2, heads, page, d // 2), 0xFF, dtype=torch.uint8, device="cuda")
    sf = torch.full((pages, 2, heads, d // 16, page), 0xFF, dtype=torch.uint8, device="cuda")
    k = torch.randn(most, heads, d, device="cuda", generator=g).bfloat16()
    v = (torch.randn(most, heads, d, device="cuda", generator=g).clamp(-4, 4) * size).bfloat16()
    gs = torch.stack([2688 / k.abs().amax().float(), 2688 / v.abs().amax().float()])
    slots = torch.arange(most, dtype=torch.int32, device="cuda")
    att.nvfp4_kv_append(k, v, slots, gs, kv, sf)
    q = torch.randn(b, 1, q_heads, d, device="cuda", generator=g).bfloat16()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(b, -1).contiguous()
    out = att.nvfp4_attention_decode(q, kv, sf, gs, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    kk, vv = (A.rows(kv, sf, w, slots) / gs[w].double() for w in (0, 1))
    for i, n in enumerate(lens):
        for h in range(q_heads):
            at = h * heads // q_heads
            ref, _, bound, _ = A.attend(q[i, :, h].double(), kk[:n, at], vv[:n, at], d ** -0.5, torch.ones(1, n, dtype=torch.bool, device="cuda"), HALF_STEP, TINY)
            bound = bound - 1e-37 + 1e-41   # (what attend allows around zero is as large as these values)
            assert A.worst(out[i, :, h], ref, bound) <= 1.0, (i, h, A.worst(out[i, :, h], ref, bound))
