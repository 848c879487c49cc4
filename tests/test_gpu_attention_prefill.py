"""Attention of packed prompts against its 64-bit form."""
import pytest
import torch

import attention_ref as A
from gpu_util import say

pytestmark = pytest.mark.gpu
HALF_STEP, TINY = 2.0 ** -8, 0.0   # bf16 probabilities


@pytest.fixture(scope="module")
def att():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import attention
    return attention


def starts(lens, first=0):
    return torch.tensor([first] + list(lens), dtype=torch.int32, device="cuda").cumsum(0).int()


def check(q, k, v, cu_q, cu_k, causal, out, lse=None, scale=None):
    d, q_heads, heads = q.shape[2], q.shape[1], k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    a, c = cu_q.tolist(), cu_k.tolist()
    for i in range(len(a) - 1):
        n, m = a[i + 1] - a[i], c[i + 1] - c[i]
        j = torch.arange(m, device="cuda")
        lim = torch.arange(n, device="cuda") + m - n if causal else torch.full((n,), m, device="cuda")
        seen = j <= lim[:, None]
        for h in range(q_heads):
            kk, vv = (x[c[i]:c[i + 1], h // (q_heads // heads)].double() for x in (k, v))
            ref, rl, bound, dl = A.attend(q[a[i]:a[i + 1], h].double(), kk, vv, scale, seen, HALF_STEP, TINY)
            got = out[a[i]:a[i + 1], h]
            assert bool(got.isfinite().all()), (i, h)
            assert A.worst(got, ref, bound) <= 1.0, (i, h, n, m, A.worst(got, ref, bound))
            if lse is not None:
                assert A.same_lse(lse[a[i]:a[i + 1], h], rl, dl), (i, h)


def inputs(lq, lk, q_heads, heads, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    tq, tk = max(1, sum(lq)), max(1, sum(lk))
    r = lambda t, h: torch.randn(t, h, d, device="cuda", generator=g).bfloat16()  # noqa: E731
    return r(tq, q_heads), r(tk, heads), r(tk, heads), starts(lq), starts(lk)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,q_heads,heads,d", [
    ((1,), (1,), 1, 1, 16), ((1,), (1,), 32, 8, 128), ((61,), (61,), 32, 8, 128), ((64,), (64,), 4, 2, 64), ((65, 127, 1, 128), (65, 127, 1, 128), 6, 3, 128),
    ((0, 7, 0, 33), (0, 7, 5, 33), 2, 1, 64), ((5, 9), (0, 9), 2, 2, 128), ((10, 300), (4, 100), 3, 1, 128), ((129, 255, 256, 257), (129, 255, 256, 257), 2, 2, 96),
    ((1, 1, 40), (700, 129, 1100), 8, 2, 128), ((200,), (1500,), 5, 1, 64), ((70, 3), (70, 259), 2, 1, 256), ((90,), (200,), 2, 2, 224), ((33, 200), (33, 200), 7, 7, 80),
    ((1000,), (1000,), 10, 2, 128), ((513, 700), (600, 701), 3, 3, 64), ((2500,), (2500,), 2, 1, 128),
    # many tiles: 256 rows a workgroup (long), 128 (short), heads of 64, 96 and 256
    ((2300, 1900), (2300, 1900), 16, 2, 128), ((1100, 1, 1990), (1190, 1500, 1990), 24, 4, 96), ((300,) * 9, (300,) * 9, 16, 8, 128), ((257, 2, 900), (257, 2, 900), 64, 8, 64),
    ((513, 320), (513, 1320), 40, 8, 128), ((200, 300), (200, 300), 8, 4, 256), ((7, 16), (5000, 3111), 8, 2, 128), ((1,), (4097,), 16, 4, 64),
    ((31, 32, 33, 1), (31, 96, 65, 64), 4, 4, 256), ((700, 129), (1000, 129), 6, 2, 256), ((100,), (3001,), 32, 32, 208), ((1300,), (1300,), 8, 8, 256),
])
def test_prefill(att, lq, lk, q_heads, heads, d, causal):
    say("prefill", lq, lk, q_heads, heads, d, causal)
    q, k, v, cq, ck = inputs(lq, lk, q_heads, heads, d, sum(lk) + d)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = att.attention_prefill(q, k, v, cq, ck, causal=causal, lse=lse)
    check(q, k, v, cq, ck, causal, out, lse)
    again = torch.full_like(out, float("nan"))
    att.attention_prefill(q, k, v, cq, ck, causal=causal, out=again)
    assert torch.equal(out[:sum(lq)], again[:sum(lq)])


def test_many_sequences(att):
    lens = [(i * 29) % 83 for i in range(150)]
    say("prefill 150 sequences")
    q, k, v, cq, ck = inputs(lens, lens, 2, 1, 64, 3)
    check(q, k, v, cq, ck, True, att.attention_prefill(q, k, v, cq))


def test_strides_and_rows_outside(att):
    """q, k, v as parts of one projection's output, sequences that leave rows before and behind."""
    say("prefill strides")
    g = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn(400, 6 + 2 + 2, 128, device="cuda", generator=g).bfloat16()
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    cu = starts((100, 150), first=30)
    wide = torch.full((400, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = att.attention_prefill(q, k, v, cu, out=wide[:, 1:7])
    assert out.data_ptr() == wide[:, 1:7].data_ptr()
    check(q, k, v, cu, cu, True, out)
    assert bool((wide[:30] == 7).all()) and bool((wide[280:] == 7).all()) and bool((wide[:, 0] == 7).all()) and bool((wide[:, 7] == 7).all())


def test_scale_and_peaks(att):
    say("prefill peaks")
    q, k, v, cq, ck = inputs((300,), (300,), 4, 2, 128, 8)
    q[:, 0] *= 30
    q[:, 1] = 0
    k[150] *= 20
    for scale in (0.5, 1e-5):
        lse = torch.empty(q.shape[:2], device="cuda")
        check(q, k, v, cq, ck, True, att.attention_prefill(q, k, v, cq, ck, scale=scale, lse=lse), lse, scale=scale)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,q_heads,heads,d", [((200, 90), 2, 1, 64), ((200, 90), 2, 1, 128), ((200, 90), 2, 1, 256), ((200, 90), 136, 2, 128),
                                                  ((200, 90), 136, 2, 64), ((1100, 1060), 32, 2, 128)])
def test_values_behind_the_mask_do_not_matter(att, bad, lens, q_heads, heads, d):
    """Rows before a key or value that is not finite, and other sequences, come out as without it."""
    say("prefill behind the mask", bad, lens, q_heads, heads, d)
    q, k, v, cq, ck = inputs(lens, lens, q_heads, heads, d, 11)
    clean = att.attention_prefill(q, k, v, cq, ck)
    at, n = lens[0] - 67, lens[0]
    for which in (k, v):
        x = which.clone()
        x[at, 0, 7] = bad
        out = att.attention_prefill(q, x if which is k else k, x if which is v else v, cq, ck)
        assert torch.equal(out[:at], clean[:at]), which is k
        assert torch.equal(out[n:], clean[n:]), which is k
        if which is v:
            mine = slice(0, q_heads // heads)
            assert not bool(out[at:n, mine, 7].isfinite().any())
            keep = torch.ones(d, dtype=torch.bool)
            keep[7] = False
            assert torch.equal(out[at:n][..., keep], clean[at:n][..., keep])
            assert torch.equal(out[:, q_heads // heads:], clean[:, q_heads // heads:])


def test_neighbours_do_not_matter(att):
    """Keys of the next sequence lie right behind and are all NaN."""
    say("prefill neighbours")
    q, k, v, cq, ck = inputs((70, 60), (70, 60), 2, 2, 128, 12)
    for causal in (True, False):
        clean = att.attention_prefill(q, k, v, cq, ck, causal=causal)
        k2, v2 = k.clone(), v.clone()
        k2[70:], v2[70:] = float("nan"), float("nan")
        out = att.attention_prefill(q, k2, v2, cq, ck, causal=causal)
        assert torch.equal(out[:70], clean[:70]) and bool(out[70:].isnan().all())


def test_offsets_outside_the_tensors(att):
    """Starts that leave the tensors are clamped."""
    say("prefill clamped")
    q, k, v, cq, ck = inputs((70, 60), (70, 60), 2, 2, 64, 13)
    want = att.attention_prefill(q, k, v, cq, ck)
    cq[2], ck[2], cq[0] = 1 << 30, 1000, -5
    assert torch.equal(att.attention_prefill(q, k, v, cq, ck), want)


def test_rows_past_4_gib(att):
    """q, k, v and out as parts of rows whose offsets pass 32 bits: 5 GB."""
    say("prefill large strides")
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.empty(40000, 512, 128, dtype=torch.bfloat16, device="cuda")
    lens, first = (130, 1, 200), 40000 - 331
    wide[first:] = torch.randn(331, 512, 128, device="cuda", generator=g).bfloat16()
    q, k, v, out = wide[:, 500:504], wide[:, 7:9], wide[:, 100:102], wide[:, 300:304]
    cu = starts(lens, first=first)
    kept = wide[first:].clone()
    att.attention_prefill(q, k, v, cu, out=out)
    check(q, k, v, cu, cu, True, out)
    kept[:, 300:304] = out[first:]
    assert torch.equal(wide[first:], kept)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,q_heads,heads,d", [
    ((1,), (8191,), 32, 8, 128), ((61,), (4157,), 6, 2, 64), ((129, 0, 7), (5000, 40, 64), 4, 4, 96), ((16, 1, 30), (2016, 3000, 900), 8, 8, 256), ((300,), (1600,), 16, 2, 80),
    ((2000,), (2000,), 3, 1, 128), ((5, 3, 0, 2), (9000, 0, 2, 130), 7, 1, 64), ((130,), (16500,), 2, 1, 224),
])
def test_few_rows_behind_many_keys(att, lq, lk, q_heads, heads, d, causal):
    """Keys that several workgroups share."""
    say("prefill parts", lq, lk, q_heads, heads, d, causal)
    q, k, v, cq, ck = inputs(lq, lk, q_heads, heads, d, sum(lk) + d)
    need = att.attention_prefill_ws_bytes(len(q), len(k), q_heads, heads, len(lq), d)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = att.attention_prefill(q, k, v, cq, ck, causal=causal, lse=lse, workspace=ws)
    check(q, k, v, cq, ck, causal, out, lse)
    wide = torch.full((len(q) + 9, q_heads + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    more = torch.cat([q[:0].new_zeros(5, q_heads, d), q, q[:0].new_zeros(4, q_heads, d)])
    att.attention_prefill(more, k, v, cq + 5, ck, causal=causal, out=wide[:, 1:])
    assert torch.equal(wide[5:len(q) + 5, 1:], out)
    assert bool((wide[:5] == 7).all()) and bool((wide[len(q) + 5:] == 7).all()) and bool((wide[:, 0] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_keys_behind_the_mask(att, bad, d):
    say("prefill parts behind the mask", bad, d)
    q, k, v, cq, ck = inputs((100, 20), (3000, 2500), 4, 2, d, 21)
    assert att.attention_prefill_ws_bytes(len(q), len(k), 4, 2, 2, d) > 0
    clean = att.attention_prefill(q, k, v, cq, ck)
    at = 2940   # rows up to 39 do not see it
    for which in (k, v):
        x = which.clone()
        x[at, 0, 7] = bad
        out = att.attention_prefill(q, x if which is k else k, x if which is v else v, cq, ck)
        assert torch.equal(out[:40], clean[:40]) and torch.equal(out[100:], clean[100:]) and torch.equal(out[:, 2:], clean[:, 2:])
        if which is v:
            assert not bool(out[40:100, :2, 7].isfinite().any())
            keep = torch.arange(d) != 7
            assert torch.equal(out[40:100][..., keep], clean[40:100][..., keep])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,q_heads,heads,d", [
    ((16, 1, 0, 7) * 16, (16, 1, 0, 7) * 16, 32, 8, 128), ((30, 5) * 20, (530, 5) * 20, 21, 3, 64), ((1,) * 64, (1,) * 64, 40, 4, 80), ((33, 20, 61) * 8, (33, 200, 61) * 8, 30, 2, 96),
    ((3,) * 40, (70,) * 40, 14, 1, 256), ((300,) + (0,) * 60, (300,) + (9,) * 60, 35, 7, 128),
])
def test_heads_that_share_a_tile(att, lq, lk, q_heads, heads, d, causal):
    """Many short sequences with grouped heads."""
    say("prefill packed", lq[:4], lk[:4], len(lq), q_heads, heads, d, causal)
    q, k, v, cq, ck = inputs(lq, lk, q_heads, heads, d, sum(lk) + d)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    wide = torch.full((len(q) + 9, q_heads + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    more = torch.zeros(len(q) + 9, q_heads + 3, d, dtype=torch.bfloat16, device="cuda")
    more[5:len(q) + 5, 2:-1] = q
    att.attention_prefill(more[:, 2:-1], k, v, cq + 5, ck, causal=causal, out=wide[:, 1:])
    out = att.attention_prefill(q, k, v, cq, ck, causal=causal, lse=lse)
    check(q, k, v, cq, ck, causal, out, lse)
    assert torch.equal(wide[5:len(q) + 5, 1:], out)
    assert bool((wide[:5] == 7).all()) and bool((wide[len(q) + 5:] == 7).all()) and bool((wide[:, 0] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_shared_tiles_behind_the_mask(att, bad):
    say("prefill packed behind the mask", bad)
    lens = (14,) * 40
    q, k, v, cq, ck = inputs(lens, lens, 32, 8, 128, 22)
    clean = att.attention_prefill(q, k, v, cq, ck)
    at = 14 * 7 + 5
    for which in (k, v):
        x = which.clone()
        x[at, 3, 7] = bad
        out = att.attention_prefill(q, x if which is k else k, x if which is v else v, cq, ck)
        keep = torch.ones(560, 32, 128, dtype=torch.bool)
        keep[at:14 * 8, 12:16, 7 if which is v else slice(None)] = False
        assert torch.equal(out[keep], clean[keep])
        if which is v:
            assert not bool(out[at:14 * 8, 12:16, 7].isfinite().any())
