"""Attention over the paged 4-bit cache against its 64-bit form."""
import pytest
import torch

import attention_ref as A
from gpu_util import say

pytestmark = pytest.mark.gpu
HALF_STEP, TINY = 2.0 ** -11, 2.0 ** -25   # fp16 probabilities


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import attention
    return attention


def setup(att, lens, new, q_heads, heads, d, page, seed=0, spare=2, kscale=1.0):
    """A cache filled through nvfp4_kv_append, all other bytes 0xFF (NaN scales)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = max(1, max(-(-n // page) for n in lens)) + 1
    need = sum(-(-n // page) for n in lens)
    pages = need + spare
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((len(lens), per), 0x7FFFFFF, dtype=torch.int32, device="cuda")
    kv = torch.full((pages, 2, heads, page, d // 2), 0xFF, dtype=torch.uint8, device="cuda")
    sf = torch.full((pages, 2, heads, d // 16, page), 0xFF, dtype=torch.uint8, device="cuda")
    gs = torch.tensor([2688 / 6.0, 2688 / 5.0], device="cuda")
    at = 0
    for i, n in enumerate(lens):
        m = -(-n // page)
        table[i, :m] = order[at:at + m]
        at += m
        if n:
            j = torch.arange(n, device="cuda")
            slots = table[i, j // page] * page + (j % page).int()
            k = torch.randn(n, heads, d, device="cuda", generator=g) * kscale
            v = torch.randn(n, heads, d, device="cuda", generator=g)
            att.nvfp4_kv_append(k.bfloat16(), v.bfloat16(), slots.int(), gs, kv, sf)
    q = torch.randn(len(lens), new, q_heads, d, device="cuda", generator=g).bfloat16()
    return dict(q=q, kv=kv, kv_sf=sf, kv_gs=gs, block_table=table, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def check(s, out, lse=None, scale=None, gone=()):
    """Every row against the 64-bit form; `gone`: (sequence, page index) pairs that count as not there."""
    b, new, q_heads, d = s["q"].shape
    heads, page = s["kv"].shape[2:4]
    scale = d ** -0.5 if scale is None else scale
    group = q_heads // heads
    for i, n in enumerate(s["lengths"].tolist()):
        j = torch.arange(max(n, 0), device="cuda")
        there = torch.ones(len(j), dtype=torch.bool, device="cuda")
        tab = s["block_table"][i].clone()
        for a, c in gone:
            if a == i:
                there[(j // page) == c] = False
                tab[c] = 0
        slots = tab[j // page].long() * page + j % page
        k = A.rows(s["kv"], s["kv_sf"], 0, slots) / s["kv_gs"][0].double()
        v = A.rows(s["kv"], s["kv_sf"], 1, slots) / s["kv_gs"][1].double()
        k, v = k.masked_fill(~there[:, None, None], 0), v.masked_fill(~there[:, None, None], 0)
        lim = n - (new - 1 - torch.arange(new, device="cuda"))
        seen = ((j < lim[:, None]) & there).repeat_interleave(group, 0)
        for h in range(heads):
            q = s["q"][i, :, h * group:(h + 1) * group].double().reshape(new * group, d)
            ref, rl, bound, dl = A.attend(q, k[:, h], v[:, h], scale, seen, HALF_STEP, TINY)
            got = out[i, :, h * group:(h + 1) * group].reshape(new * group, d)
            assert bool(got.isfinite().all()), (i, h)
            assert A.worst(got, ref, bound) <= 1.0, (i, h, n, A.worst(got, ref, bound))
            if lse is not None:
                assert A.same_lse(lse[i, :, h * group:(h + 1) * group].reshape(-1), rl, dl), (i, h, n)


@pytest.mark.parametrize("lens,new,q_heads,heads,d,page", [
    ((1,), 1, 1, 1, 32, 16), ((1,), 1, 32, 8, 128, 64), ((63, 64, 65), 1, 8, 2, 128, 16), ((0, 5, 0), 1, 4, 4, 64, 32),
    ((15, 16, 17, 255, 256, 257, 300), 1, 6, 3, 128, 16), ((700, 1, 0, 2900), 1, 40, 8, 128, 64), ((2100,), 1, 16, 1, 64, 128),
    ((333, 1024), 1, 21, 3, 96, 32), ((513, 40), 1, 10, 2, 256, 64), ((90, 777), 1, 5, 5, 160, 16), ((4000, 17), 1, 71, 1, 64, 64),
    ((5, 2, 1, 0, 600), 4, 12, 4, 128, 16), ((1000, 3), 7, 48, 2, 64, 32), ((259, 258, 257), 3, 8, 8, 256, 16), ((40,), 64, 2, 1, 128, 64),
    ((9000, 12000, 64), 1, 8, 8, 128, 256), ((20000,), 2, 4, 1, 128, 4096), ((3000,) * 3, 1, 3, 3, 192, 64), ((70,), 1, 7, 7, 224, 16),
    ((1, 300, 0, 77), 1, 8, 2, 80, 16), ((3000, 65), 1, 21, 3, 80, 64), ((500,), 3, 40, 4, 48, 32), ((200, 18), 1, 5, 5, 16, 16), ((31, 1200), 2, 6, 2, 112, 64),
    ((700, 2), 1, 9, 3, 144, 16), ((100, 400), 5, 16, 2, 240, 128), ((257,), 1, 2, 2, 208, 32), ((1100, 7), 1, 64, 4, 32, 16),
])
def test_decode(att, lens, new, q_heads, heads, d, page):
    say("decode", lens, new, q_heads, heads, d, page)
    s = setup(att, lens, new, q_heads, heads, d, page, seed=len(lens) + d)
    lse = torch.full(s["q"].shape[:3], 7.0, device="cuda")
    ws = torch.full((att.attention_ws_bytes(len(lens), d),), 0xFF, dtype=torch.uint8, device="cuda")
    out = att.nvfp4_attention_decode(**s, lse=lse, workspace=ws)
    check(s, out, lse)
    again = torch.full_like(out, float("nan"))
    att.nvfp4_attention_decode(**s, out=again, workspace=ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("lens,new,q_heads,heads,d,page", [((600, 33, 1, 0, 2000), 4, 64, 8, 128, 64), ((70, 1025), 3, 21, 3, 64, 32), ((40, 3), 17, 8, 4, 96, 64),
                                                           ((513,), 5, 40, 8, 256, 64), ((300, 17, 1400), 5, 24, 4, 80, 16), ((90, 700), 2, 40, 4, 48, 32)])
def test_rows_that_share_a_read(att, lens, new, q_heads, heads, d, page):
    """Tables wide enough that several tiles of rows are taken together."""
    say("decode shared", lens, new, q_heads, heads, d, page)
    s = setup(att, lens, new, q_heads, heads, d, page, seed=new)
    wide = torch.full((len(lens), (1 << 20) // page), -7, dtype=torch.int32, device="cuda")
    wide[:, : s["block_table"].shape[1]] = s["block_table"]
    s["block_table"] = wide
    lse = torch.empty(s["q"].shape[:3], device="cuda")
    check(s, att.nvfp4_attention_decode(**s, lse=lse), lse)


def test_many_sequences(att):
    lens = [(i * 37) % 401 for i in range(300)] + [5000, 0, 1]
    say("decode 303 sequences")
    s = setup(att, lens, 1, 4, 2, 64, 16, seed=5)
    check(s, att.nvfp4_attention_decode(**s))


@pytest.mark.parametrize("q_heads,heads,d,new", [(32, 2, 256, 1), (40, 1, 128, 1), (26, 2, 80, 1), (16, 16, 64, 2)])
def test_many_rows_and_parts(att, q_heads, heads, d, new):
    """A thousand rows and more, some of sequences in many parts."""
    lens = [(i * 53) % 700 for i in range(40)] + [9000, 0, 4500]
    say("decode many rows", q_heads, heads, d, new)
    s = setup(att, lens, new, q_heads, heads, d, 32, seed=d)
    lse = torch.empty(s["q"].shape[:3], device="cuda")
    check(s, att.nvfp4_attention_decode(**s, lse=lse), lse)


def test_scale_and_peaks(att):
    """Scores far apart (one key takes all), a scale of its own, queries of very different size."""
    say("decode peaks")
    s = setup(att, (777, 64, 3), 1, 8, 2, 128, 16, seed=3, kscale=1.5)
    s["q"][:, :, 0] *= 2.0 ** 40
    s["q"][:, :, 0] *= 2.0 ** -36
    s["q"][:, :, 1] *= 2.0 ** -60
    s["q"][:, :, 2] = 0
    for scale in (0.3, 2.0, 1e-4):
        lse = torch.empty(s["q"].shape[:3], device="cuda")
        check(s, att.nvfp4_attention_decode(**s, scale=scale, lse=lse), lse, scale=scale)


def test_rows_of_nan_stay_alone(att):
    say("decode nan rows")
    s = setup(att, (300, 100), 1, 8, 2, 128, 16, seed=9)
    clean = att.nvfp4_attention_decode(**s)
    s["q"][0, 0, 3, 17] = float("nan")
    s["q"][1, 0, 6, 0] = float("inf")
    out = att.nvfp4_attention_decode(**s)
    assert bool(out[0, 0, 3].isnan().all()) and not bool(out[1, 0, 6].isfinite().any())
    keep = torch.ones(2, 8, dtype=torch.bool, device="cuda")
    keep[0, 3] = keep[1, 6] = False
    assert torch.equal(out[:, 0][keep], clean[:, 0][keep])


def test_pages_outside_the_cache_are_not_there(att):
    say("decode bad pages")
    s = setup(att, (600, 200, 30), 2, 8, 4, 128, 16, seed=4)
    gone = [(0, 3), (0, 20), (0, 37), (1, 0), (2, 0), (2, 1)]
    for (i, c), bad in zip(gone, (-1, s["kv"].shape[0], 2 ** 31 - 1, -2 ** 31, -1, 1 << 20)):
        s["block_table"][i, c] = bad
    lse = torch.empty(s["q"].shape[:3], device="cuda")
    check(s, att.nvfp4_attention_decode(**s, lse=lse), lse, gone=gone)


def test_lengths_outside_the_table(att):
    say("decode clamped lengths")
    s = setup(att, (100, 50), 1, 4, 2, 64, 16, seed=6)
    s["block_table"] = s["block_table"][:, :4].contiguous()   # 64 positions
    s["lengths"] = torch.tensor([100, -3], dtype=torch.int32, device="cuda")
    out = att.nvfp4_attention_decode(**s)
    s["lengths"] = torch.tensor([64, 0], dtype=torch.int32, device="cuda")
    assert torch.equal(out, att.nvfp4_attention_decode(**s))
    check(s, out)


def test_cache_past_4_gib(att):
    """Pages whose bytes lie past 32-bit offsets: 9.4 GB of codes."""
    say("decode large cache")
    heads, d, page = 8, 128, 64
    pages = 140000
    kv = torch.empty(pages, 2, heads, page, d // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(pages, 2, heads, d // 16, page, dtype=torch.uint8, device="cuda")
    gs = torch.tensor([400.0, 500.0], device="cuda")
    table = torch.tensor([[pages - 1, 3, pages // 2 + 7], [pages - 2, 65537, 131071]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    j = torch.arange(150, device="cuda")
    for i in range(2):
        k = torch.randn(150, heads, d, device="cuda", generator=g).bfloat16()
        att.nvfp4_kv_append(k, k * 2, (table[i, j // page] * page + (j % page).int()).int(), gs, kv, sf)
    s = dict(q=torch.randn(2, 1, 16, d, device="cuda", generator=g).bfloat16(), kv=kv, kv_sf=sf, kv_gs=gs, block_table=table,
             lengths=torch.tensor([150, 149], dtype=torch.int32, device="cuda"))
    check(s, att.nvfp4_attention_decode(**s))
