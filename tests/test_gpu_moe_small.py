"""nvfp4_moe_small against a plain 64-bit form: routing (ids exactly, weights to
fp32 rounding) and the layer's output within the error its arithmetic allows, at
sizes on both sides of every tile, chunk and workgroup boundary, and on routing
inputs that can go wrong."""
import pytest
import torch

import serving_ref as R
from gpu_util import OUT_CANARY, say

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def serving():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import serving as _s
    return _s


def layer(seed, t, h, inter, E, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = dict(w13=R.rand_fp4(g, E, 2 * inter, k=h), w13_sf=R.rand_sf(g, 2 * inter, h, E),
             alpha13=torch.rand(E, device="cuda", generator=g) / (4 * h ** 0.5) + 0.01,
             w2=R.rand_fp4(g, E, h, k=inter), w2_sf=R.rand_sf(g, h, inter, E),
             alpha2=torch.rand(E, device="cuda", generator=g) / inter ** 0.5 + 0.01)
    x = torch.randn(t, h, device="cuda", generator=g).bfloat16()
    logits = (torch.randn(t, E, device="cuda", generator=g) * 2).to(dtype)
    return x, logits, w


def check(serving, x, logits, w, k, score, renorm):
    t, h = x.shape
    inter = w["w2"].shape[2] * 2
    out = torch.full((t, h), OUT_CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    ids = torch.full((t, k), 77, dtype=torch.int32, device="cuda")
    wts = torch.full((t, k), NAN, device="cuda")
    ws = torch.full((serving.moe_small_ws_bytes(t, k, h, inter),), 0xFF, dtype=torch.uint8, device="cuda")
    serving.nvfp4_moe_small(x, logits, *w.values(), k, score=score, renormalize=renorm, out=out, topk_ids=ids,
                            topk_weights=wts, workspace=ws)
    ref, bound, rid, rw = R.moe(x, logits, *w.values(), k, score, renorm)
    assert torch.equal(ids.cpu(), rid), (ids.cpu(), rid)
    # exp of a difference, a sum of at most 256 and a division, in fp32; the
    # argument's own rounding (half an ulp of |l - max|, at most 2^-24 * 128)
    assert torch.allclose(wts.cpu().double(), rw, rtol=2.0 ** -16, atol=2.0 ** -126, equal_nan=True)
    # the weight's error reaches the output in proportion
    bound = bound + ref.abs() * 2.0 ** -16
    assert R.worst(out, ref, bound) <= 1.0
    return out


CASES = [  # t, h, inter, E, k, score, renormalize, logits
    (1, 16, 16, 1, 1, "softmax", True, "f32"),
    (1, 128, 128, 2, 1, "sigmoid", False, "f32"),
    (2, 144, 48, 3, 2, "softmax", False, "bf16"),
    (15, 48, 208, 8, 2, "sigmoid", True, "bf16"),
    (16, 256, 128, 16, 4, "softmax", True, "f32"),
    (17, 1040, 144, 63, 3, "softmax", False, "f32"),
    (33, 272, 272, 65, 16, "softmax", True, "bf16"),
    (64, 512, 256, 32, 4, "softmax", True, "f32"),
    (64, 128, 640, 256, 8, "sigmoid", True, "f32"),
    (5, 2064, 1104, 130, 9, "softmax", True, "f32"),
    (3, 640, 2048, 200, 1, "sigmoid", False, "bf16"),
    (64, 96, 32, 4, 4, "softmax", False, "f32"),
]


@pytest.mark.parametrize("t,h,inter,E,k,score,renorm,dt", CASES)
def test_layer(serving, t, h, inter, E, k, score, renorm, dt):
    say("moe", t, h, inter, E, k, score, renorm, dt)
    x, lg, w = layer(t + h, t, h, inter, E, torch.bfloat16 if dt == "bf16" else torch.float32)
    check(serving, x, lg, w, k, score, renorm)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("t,E,k", [(6, 9, 4), (2, 100, 4)])
def test_routing_edges(serving, t, E, k, score, renorm):
    """Rows with nothing to choose, fewer than top_k, NaN, equal logits, the
    lowest finite value, very negative ones; with few pairs and with many."""
    say("moe routing edges", t, E, k, score, renorm)
    x, lg, w = layer(3, t, 64, 32, E)
    rows = [torch.full((E,), -INF, device="cuda"), lg[0].clone(), torch.full((E,), 0.25, device="cuda"),
            torch.full((E,), torch.finfo(torch.float32).min, device="cuda"), lg[1].clone() * 4 - 100, lg[0].clone()]
    rows[1][:] = -INF
    rows[1][E - 1], rows[1][2], rows[1][0] = 0.5, 0.5, NAN   # two to choose, equal, and a NaN
    rows[5][1::2] = NAN
    for i in range(0, len(rows), t):
        lg = torch.stack([rows[j % len(rows)] for j in range(i, i + t)])
        check(serving, x, lg, w, k, score, renorm)


def test_no_token_chooses(serving):
    say("moe: every row empty")
    x, lg, w = layer(4, 3, 64, 32, 40)
    out = check(serving, x, torch.full_like(lg, -INF), w, 2, "softmax", True)
    assert not out.any()


@pytest.mark.parametrize("E", [4, 200])
def test_every_token_on_one_expert(serving, E):
    """More rows of an expert than a tile holds, beside experts without any."""
    say("moe: 61 tokens on one expert of", E)
    x, lg, w = layer(5, 61, 160, 96, E)
    lg[:, 3] = 50.0
    check(serving, x, lg, w, 1, "softmax", True)
    check(serving, x, lg, w, 3, "sigmoid", False)


def test_positive_infinity_and_non_finite_tokens(serving):
    """+inf is chosen first and its softmax weight is NaN; a token with NaN or
    inf reaches its own output row only."""
    say("moe: non-finite")
    x, lg, w = layer(6, 5, 64, 32, 8)
    lg[1, 5] = INF
    check(serving, x, lg, w, 2, "sigmoid", False)
    out, ids, wts = serving.nvfp4_moe_small(x, lg, *w.values(), 2)
    assert ids[1, 0] == 5 and wts[1].isnan().all() and out[1].isnan().all() and out[[0, 2, 3, 4]].isfinite().all()
    x[2, 7], x[3, 9] = NAN, INF
    lg[1, 5] = 1.0
    good, _, _ = serving.nvfp4_moe_small(torch.where(x.isfinite(), x, torch.zeros_like(x)), lg, *w.values(), 2)
    out, _, _ = serving.nvfp4_moe_small(x, lg, *w.values(), 2)
    assert out[2].isnan().all() and not out[3].isfinite().all()
    assert torch.equal(out[[0, 1, 4]], good[[0, 1, 4]])


def test_offsets_past_32_bits(serving):
    """Expert weights of more than 2^32 bytes: the last experts are the ones used."""
    say("moe: 6.4 GB of expert weights")
    E, h, inter, t = 256, 4096, 4096 + 128, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rp, cp = (2 * inter + 127) // 128 * 128, h // 16
    w = dict(w13=torch.zeros(E, 2 * inter, h // 2, dtype=torch.uint8, device="cuda"),
             w13_sf=torch.zeros(E, rp * cp, dtype=torch.uint8, device="cuda"),
             alpha13=torch.full((E,), 0.01, device="cuda"),
             w2=torch.zeros(E, h, inter // 2, dtype=torch.uint8, device="cuda"),
             w2_sf=torch.zeros(E, h * (inter // 16), dtype=torch.uint8, device="cuda"),
             alpha2=torch.full((E,), 0.02, device="cuda"))
    assert w["w13"].numel() > 2 ** 32
    for e in (E - 1, E - 2):
        w["w13"][e] = R.rand_fp4(g, 2 * inter, k=h)
        w["w13_sf"][e] = R.rand_sf(g, 2 * inter, h)
        w["w2"][e] = R.rand_fp4(g, h, k=inter)
        w["w2_sf"][e] = R.rand_sf(g, h, inter)
    x = torch.randn(t, h, device="cuda", generator=g).bfloat16()
    lg = torch.randn(t, E, device="cuda", generator=g)
    lg[:, -2:] += 20
    check(serving, x, lg, w, 2, "softmax", True)


# The second launch's form of 16 waves: t > 32 and wide enough h (sixteen_waves).
SIXTEEN = [  # t, h, inter, E, k, score, renormalize, logits
    (33, 2064, 144, 5, 2, "softmax", True, "f32"),        # one share; an odd number of 128-column bands
    (64, 4112, 1040, 4, 3, "sigmoid", False, "bf16"),     # three shares, about 48 tokens an expert, I % 128 != 0
    (64, 4096, 2048, 6, 2, "softmax", True, "f32"),       # whole chunks and bands
    (40, 3088, 512, 40, 8, "softmax", False, "f32"),      # many short experts, 13 shares at most
    (49, 3200, 656, 3, 1, "sigmoid", True, "f32"),
]


def sixteen_waves(t, h):
    """Whether the second launch takes workgroups of 16 waves: most shares of the
    K axis times tiles of 256 columns fill the CUs."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return t > 32 and -(-h // 256) * min(1024 // t, 32) >= cus


@pytest.mark.parametrize("t,h,inter,E,k,score,renorm,dt", SIXTEEN)
def test_layer_of_sixteen_waves(serving, t, h, inter, E, k, score, renorm, dt):
    say("moe, 16 waves", t, h, inter, E, k, score, renorm, dt)
    assert sixteen_waves(t, h)
    x, lg, w = layer(t + h, t, h, inter, E, torch.bfloat16 if dt == "bf16" else torch.float32)
    check(serving, x, lg, w, k, score, renorm)


def test_sixteen_waves_edges(serving):
    """Empty rows, every token on one expert, no token on any, a token of NaN."""
    say("moe, 16 waves: edges")
    t, h, inter, E = 50, 3344, 176, 9
    assert sixteen_waves(t, h)
    x, lg, w = layer(11, t, h, inter, E)
    lg[::3] = -INF
    check(serving, x, lg, w, 4, "softmax", True)
    lg[:] = -INF
    lg[:, 7] = 1.0
    good = check(serving, x, lg, w, 2, "softmax", True)
    x[20, 5] = NAN
    out, _, _ = serving.nvfp4_moe_small(x, lg, *w.values(), 2)
    assert out[20].isnan().all() and torch.equal(out[:20], good[:20]) and torch.equal(out[21:], good[21:])
    assert not check(serving, x.nan_to_num(), torch.full_like(lg, -INF), w, 2, "softmax", True).any()


def test_sixteen_waves_repeats_and_graph(serving):
    """The same bits on a second call and on three replays of a captured graph,
    the workspace and the outputs overwritten in between."""
    say("moe, 16 waves: repeats, graph")
    t, h, inter, k = 64, 4112, 1040, 3
    assert sixteen_waves(t, h)
    x, lg, w = layer(12, t, h, inter, 4)
    ws = torch.full((serving.moe_small_ws_bytes(t, k, h, inter),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty(t, h, dtype=torch.bfloat16, device="cuda")
    go = lambda: serving.nvfp4_moe_small(x, lg, *w.values(), k, out=out, workspace=ws)
    go()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    for replay in range(4):
        out.fill_(3)
        ws.fill_(0xFF)
        if replay:
            graph.replay()
        else:
            go()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        if replay == 0:
            with torch.cuda.graph(graph):
                go()


def test_repeats_streams_and_graph(serving):
    """The same bits on a second call, on another stream, and on three replays of
    a captured graph with the workspace and the outputs overwritten in between."""
    say("moe: repeats, stream, graph")
    x, lg, w = layer(8, 33, 272, 144, 20)
    ws = torch.full((serving.moe_small_ws_bytes(33, 3, 272, 144),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty(33, 272, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(33, 3, dtype=torch.int32, device="cuda")
    wts = torch.empty(33, 3, device="cuda")
    go = lambda: serving.nvfp4_moe_small(x, lg, *w.values(), 3, out=out, topk_ids=ids, topk_weights=wts, workspace=ws)
    go()
    want = [v.clone() for v in (out, ids, wts)]

    def scribble():
        for v in (out, ids, wts):
            v.fill_(3)
        ws.fill_(0xFF)

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip((out, ids, wts), want))

    scribble()
    go()
    assert same()
    scribble()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        scribble()
        graph.replay()
        assert same()


def test_refusals(serving):
    x, lg, w = layer(1, 4, 64, 32, 8)
    v = list(w.values())
    f = serving.nvfp4_moe_small
    say("moe: refusals")
    for bad in (lambda: f(x.float(), lg, *v, 2), lambda: f(x, lg.half(), *v, 2), lambda: f(x, lg[:3], *v, 2),
                lambda: f(x, lg, *v, 2, score="tanh"), lambda: f(x.t(), lg, *v, 2),
                lambda: f(x, lg, v[0][:, :32].contiguous(), *v[1:], 2), lambda: f(x, lg, v[0], v[1][:, :-1].contiguous(), *v[2:], 2),
                lambda: f(x, lg, *v[:3], v[3].cpu(), *v[4:], 2),
                lambda: f(x, lg, *v, 2, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda")),
                lambda: f(x, lg, *v, 2, out=torch.empty(4, 63, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(x, lg, *v, 9), lambda: f(x, lg, *v, 0)):
        with pytest.raises(RuntimeError):
            bad()
    x65, lg65, _ = layer(1, 65, 64, 32, 8)
    out = torch.full((65, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        f(x65, lg65, *v, 2, out=out)
    torch.cuda.synchronize()
    assert bool((out == 5).all())
