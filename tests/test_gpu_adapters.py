"""nvfp4_linear_adapters and nvfp4_gemm_adapters against a plain 64-bit form:
every output within the error the arithmetic allows, at sizes on both sides of
every tile, rank and slice boundary, through every tile the prefill GEMM picks,
and over adapter lists in any order."""
import pytest
import torch

import serving_ref as R
from gpu_util import OUT_CANARY, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from nvfp4_block_scaled_04_amd import ops, serving
    return serving, ops


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def pool(g, m, n, k, r, L, ids="mixed"):
    p = dict(lora_a=(torch.randn(L, r, k, device="cuda", generator=g) / k ** 0.5).bfloat16(),
             lora_b=(torch.randn(L, n, r, device="cuda", generator=g)).bfloat16(),
             scaling=torch.rand(L, device="cuda", generator=g) * 2 + 0.25)
    a = torch.randint(-1, L, (m,), device="cuda", generator=g, dtype=torch.int32)
    if ids == "none":
        a[:] = -1
    elif ids == "one":
        a[:] = L - 1
    elif ids == "each":
        a = (torch.arange(m, device="cuda") % L).int()
    elif ids == "runs":
        a = (torch.arange(m, device="cuda") * 7 // m % L).int()
    elif ids == "wild":   # ids no pool holds: as if there were none
        a = torch.tensor([L, -1, 0, -2 ** 31, 2 ** 31 - 1, L - 1], device="cuda", dtype=torch.int32).repeat(m)[:m].contiguous()
    p["adapter"] = a
    return p


def fresh(m, n):
    return torch.full((m, n), OUT_CANARY, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")


DECODE = [  # m, n, k, r, L, ids, scaling, bias
    (1, 16, 16, 8, 1, "one", True, False),
    (1, 40, 128, 16, 3, "one", False, True),
    (2, 1, 48, 8, 2, "each", True, True),
    (15, 33, 144, 24, 5, "mixed", True, False),
    (16, 1000, 1040, 40, 20, "each", True, True),
    (17, 64, 512, 256, 4, "mixed", True, False),
    (23, 130, 2608, 24, 12, "wild", True, True),
    (32, 48, 272, 64, 40, "each", False, False),
    (33, 96, 640, 128, 7, "mixed", True, False),
    (64, 272, 1024, 32, 48, "each", True, False),
    (64, 272, 1024, 136, 2, "none", True, True),
    (65, 80, 256, 16, 9, "mixed", True, True),
    (200, 144, 384, 72, 33, "runs", True, False),
    (48, 1048, 2576, 200, 30, "each", True, True),
    (64, 520, 4096, 64, 64, "each", True, False),
    (31, 256, 128, 8, 3, "wild", False, True),
    (3, 24, 4240, 16, 3, "each", True, False),          # shared tiles: K beyond one step
    (16, 8210, 400, 40, 9, "mixed", True, True),        # and more columns than workgroups
    (31, 300, 4128, 24, 9, "mixed", False, True),
    (24, 4100, 256, 72, 5, "each", True, False),
    (64, 260, 5136, 136, 70, "each", True, True),
    (47, 4104, 640, 16, 4, "wild", True, False),
    (8200, 24, 48, 16, 5, "runs", True, False),         # projections of many rows: 32-row tiles
    (8193, 40, 272, 32, 40, "mixed", True, True),
    (8225, 16, 144, 200, 6, "runs", False, False),
    (300, 40, 336, 56, 9, "each", True, False),         # 16-row tiles of 16 ranks
    (600, 40, 336, 136, 9, "mixed", True, False),       # and of three tiles of ranks
]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("m,n,k,r,L,ids,scaled,biased", DECODE)
def test_decode(mods, m, n, k, r, L, ids, scaled, biased, split):
    serving, _ = mods
    say("linear_adapters", m, n, k, r, L, ids, split)
    g = gen(m + n + k)
    p = pool(g, m, n, k, r, L, ids)
    s = p["scaling"] if scaled else None
    b, sf = R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    alpha = torch.full((1,), 0.02, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    bias = torch.randn(n, device="cuda", generator=g).bfloat16() if biased else None
    out = fresh(m, n)
    serving.nvfp4_linear_adapters(x, b, sf, alpha, p["lora_a"], p["lora_b"], p["adapter"], scaling=s, bias=bias, out=out,
                                  workspace=workspace(serving.adapters_ws_bytes(m, r, split)))
    w = R.dequant(b, sf)
    ref, bound = R.adapters(x.double() @ w.t() * alpha.double(), x.double().abs() @ w.abs().t() * alpha.double(), k, x,
                            p["lora_a"], p["lora_b"], p["adapter"], s, bias)
    assert R.worst(out, ref, bound) <= 1.0


PREFILL = [  # m, n, k, r, L, ids, bias, workspace of the split-tail schedule
    (1, 32, 16, 8, 1, "one", False, False),            # skinny kernel
    (64, 100, 272, 40, 20, "each", True, False),
    (65, 33, 128, 8, 3, "mixed", True, False),          # 128 x 128 tile
    (300, 520, 1040, 24, 40, "each", False, False),
    (1003, 2056, 2000, 40, 9, "runs", True, False),
    (2000, 1928, 256, 16, 5, "wild", True, False),      # 128 x 256, two K groups
    (1928, 4096, 144, 16, 5, "runs", False, False),
    (2048, 4104, 896, 16, 6, "mixed", False, False),    # 128 x 256, odd number of steps
    (4000, 3480, 272, 32, 6, "runs", True, False),      # one round of 256 x 192
    (4096, 8200, 144, 32, 6, "runs", False, False),     # 256 x 256
    (3968, 2560, 1008, 32, 6, "runs", True, True),      # split tail
    (3968, 2560, 1008, 32, 200, "mixed", True, True),
]


@pytest.mark.parametrize("m,n,k,r,L,ids,biased,split", PREFILL)
def test_prefill(mods, m, n, k, r, L, ids, biased, split):
    serving, ops = mods
    say("gemm_adapters", m, n, k, r, L, ids, split)
    g = gen(m + n + k)
    p = pool(g, m, n, k, r, L, ids)
    a, a_sf, b, b_sf = R.rand_fp4(g, m, k=k), R.rand_sf(g, m, k), R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    alpha = torch.full((1,), 3e-4, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    bias = torch.randn(n, device="cuda", generator=g).bfloat16() if biased else None
    out = fresh(m, n)
    serving.nvfp4_gemm_adapters(a, b, a_sf, b_sf, alpha, x, p["lora_a"], p["lora_b"], p["adapter"], scaling=p["scaling"],
                                bias=bias, out=out, workspace=workspace(serving.adapters_ws_bytes(m, r, split)))
    left, w = R.dequant(a, a_sf), R.dequant(b, b_sf)
    ref, bound = R.adapters(left @ w.t() * alpha.double(), left.abs() @ w.abs().t() * alpha.double(), k, x, p["lora_a"],
                            p["lora_b"], p["adapter"], p["scaling"], bias)
    assert R.worst(out, ref, bound) <= 1.0
    if not split:  # rows without an adapter are the plain GEMM's, bit for bit
        plain = ops.nvfp4_gemm(a, b, a_sf, b_sf, alpha, bias=bias)
        rows = (p["adapter"] < 0) | (p["adapter"] >= L)
        assert torch.equal(out[rows], plain[rows])


def test_non_finite_row_stays_in_its_row(mods):
    """A row with NaN or inf, and an adapter with NaN that one row uses, reach
    those rows only."""
    serving, _ = mods
    say("adapters: non-finite rows")
    g = gen(2)
    m, n, k, r, L = 20, 48, 256, 16, 5
    p = pool(g, m, n, k, r, L, "each")
    b, sf = R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    alpha = torch.full((1,), 0.02, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    p["adapter"][p["adapter"] == 4] = 3
    p["adapter"][11] = 4
    run = lambda x: serving.nvfp4_linear_adapters(x, b, sf, alpha, p["lora_a"], p["lora_b"], p["adapter"])
    good = run(x)
    x[3, 5], x[18, 200] = float("nan"), float("inf")
    p["lora_a"][4, 2, 9] = float("nan")
    out = run(x)
    keep = [i for i in range(m) if i not in (3, 11, 18)]
    assert torch.equal(out[keep], good[keep])
    assert out[3].isnan().all() and out[11].isnan().all() and not out[18].isfinite().any()


def test_adapter_pool_past_32_bits(mods):
    """A pool whose last adapter lies beyond 2^32 bytes."""
    serving, _ = mods
    say("adapters: 4.4 GB pools")
    g = gen(4)
    m, n, k, r, L = 18, 4096, 4096, 128, 4200
    la = torch.zeros(L, r, k, dtype=torch.bfloat16, device="cuda")
    lb = torch.zeros(L, n, r, dtype=torch.bfloat16, device="cuda")
    assert la.numel() * 2 > 2 ** 32
    for a in (0, L - 1):
        la[a] = (torch.randn(r, k, device="cuda", generator=g) / 64).bfloat16()
        lb[a] = torch.randn(n, r, device="cuda", generator=g).bfloat16()
    ids = torch.tensor([0, L - 1, -1] * 6, dtype=torch.int32, device="cuda")
    b, sf = R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    alpha = torch.full((1,), 0.02, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    out = serving.nvfp4_linear_adapters(x, b, sf, alpha, la, lb, ids)
    w = R.dequant(b, sf)
    ref, bound = R.adapters(x.double() @ w.t() * alpha.double(), x.double().abs() @ w.abs().t() * alpha.double(), k, x, la,
                            lb, ids, None, None)
    assert R.worst(out, ref, bound) <= 1.0


@pytest.mark.parametrize("m", [16, 300, 3968])
def test_repeats_streams_and_graph(mods, m):
    """The same bits on a second call, on another stream, and on three replays of
    a captured graph with the workspace and the output overwritten in between."""
    serving, _ = mods
    say("adapters: repeats, stream, graph", m)
    g = gen(6)
    n, k, r, L = 2560, 256, 24, 7
    p = pool(g, m, n, k, r, L, "mixed")
    b, b_sf = R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    a, a_sf = R.rand_fp4(g, m, k=k), R.rand_sf(g, m, k)
    alpha = torch.full((1,), 3e-4, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    ws, out = workspace(serving.adapters_ws_bytes(m, r, True)), fresh(m, n)
    lora = (p["lora_a"], p["lora_b"], p["adapter"])
    calls = [lambda: serving.nvfp4_gemm_adapters(a, b, a_sf, b_sf, alpha, x, *lora, scaling=p["scaling"], out=out,
                                                 workspace=ws)]
    if m <= 300:
        calls.append(lambda: serving.nvfp4_linear_adapters(x, b, b_sf, alpha, *lora, scaling=p["scaling"], out=out,
                                                           workspace=ws))
    for go in calls:
        go()
        want = out.clone()

        def same():
            torch.cuda.synchronize()
            return torch.equal(out, want)

        def scribble():
            out.fill_(3)
            ws.fill_(0xFF)

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


def test_refusals(mods):
    serving, _ = mods
    say("adapters: refusals")
    g = gen(7)
    m, n, k, r, L = 8, 32, 64, 16, 3
    p = pool(g, m, n, k, r, L)
    b, sf = R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    alpha = torch.ones(1, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    la, lb, ad = p["lora_a"], p["lora_b"], p["adapter"]
    f = serving.nvfp4_linear_adapters
    for bad in (lambda: f(x.float(), b, sf, alpha, la, lb, ad), lambda: f(x, b, sf, alpha, la.float(), lb, ad),
                lambda: f(x, b, sf, alpha, la, lb[:, :, :8].contiguous(), ad), lambda: f(x, b, sf, alpha, la, lb, ad.long()),
                lambda: f(x, b, sf, alpha, la, lb, ad[:-1]), lambda: f(x, b, sf, alpha, la[:2], lb, ad),
                lambda: f(x, b[:, :16].contiguous(), sf, alpha, la, lb, ad), lambda: f(x, b, sf[:-1], alpha, la, lb, ad),
                lambda: f(x, b, sf, alpha, la, lb, ad, scaling=torch.ones(2, device="cuda")),
                lambda: f(x, b, sf, alpha, la, lb, ad, bias=torch.ones(n, device="cuda")),
                lambda: f(x, b, sf, alpha, la, lb, ad, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: f(x, b, sf, alpha, la, lb, ad.cpu()),
                lambda: serving.nvfp4_gemm_adapters(b[:7], b, sf, sf, alpha, x, la, lb, ad)):
        with pytest.raises(ValueError):
            bad()
    la12, lb12 = la[:, :12].contiguous(), lb[:, :, :12].contiguous()
    out = torch.full((m, n), 5.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError, match="rank"):
        f(x, b, sf, alpha, la12, lb12, ad, out=out)
    torch.cuda.synchronize()
    assert bool((out == 5).all())


@pytest.mark.parametrize("m", [20, 64, 300, 2048])
def test_non_finite_adapter_stays_with_its_rows(mods, m):
    """An adapter whose second matrix holds NaN or inf reaches the rows that use it
    only, though other rows of the same tile are multiplied beside them."""
    serving, _ = mods
    say("adapters: non-finite lora_b", m)
    g = gen(12)
    n, k, r, L = 272, 256, 24, 6
    p = pool(g, m, n, k, r, L, "mixed")
    b, b_sf, a, a_sf = R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k), R.rand_fp4(g, m, k=k), R.rand_sf(g, m, k)
    alpha = torch.full((1,), 3e-4, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    calls = [lambda: serving.nvfp4_gemm_adapters(a, b, a_sf, b_sf, alpha, x, p["lora_a"], p["lora_b"], p["adapter"])]
    if m <= 300:
        calls.append(lambda: serving.nvfp4_linear_adapters(x, b, b_sf, alpha, p["lora_a"], p["lora_b"], p["adapter"]))
    good = [f() for f in calls]
    p["lora_b"][2, 5, 3] = float("nan")
    p["lora_b"][4, :, 20] = float("inf")
    rows = (p["adapter"] != 2) & (p["adapter"] != 4)
    for f, want in zip(calls, good):
        out = f()
        assert torch.equal(out[rows], want[rows])
        assert out[p["adapter"] == 2][:, 5].isnan().all() and not out[p["adapter"] == 4].isfinite().any()


@pytest.mark.parametrize("m,n,k", [(3, 32, 64), (40, 260, 4240), (100, 48, 64)])
def test_projection_past_the_largest_bf16(mods, m, n, k):
    """A row's projection that is finite in fp32 but rounds to an infinity in bf16
    stays finite; one that is infinite stays infinite, with its sign."""
    serving, _ = mods
    say("adapters: projection past the largest bf16", m, n, k)
    g = gen(m)
    b, b_sf = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda"), R.rand_sf(g, n, k)   # the shared product is 0
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1], x[:, 3] = 2.0 ** 128 - 2.0 ** 120, 1.5 * 2.0 ** 119, 1.0    # 2^128 - 2^118 together; and 1
    x[1::3] = -x[1::3]
    la = torch.zeros(1, 8, k, dtype=torch.bfloat16, device="cuda")
    la[0, 2, :2] = 1.0
    la[0, 5, 3] = 3.0
    lb = torch.full((1, n, 8), 0.0, dtype=torch.bfloat16, device="cuda")
    lb[0, :, 2], lb[0, :, 5] = 2.0 ** -100, torch.randn(n, device="cuda", generator=g).bfloat16()
    ids = torch.zeros(m, dtype=torch.int32, device="cuda")
    alpha = torch.ones(1, device="cuda")
    zero = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    calls = [lambda: serving.nvfp4_linear_adapters(x, b, b_sf, alpha, la, lb, ids),
             lambda: serving.nvfp4_gemm_adapters(torch.zeros(m, k // 2, dtype=torch.uint8, device="cuda"), b, R.rand_sf(g, m, k), b_sf,
                                                 alpha, x, la, lb, ids)]
    ref, bound = R.adapters(zero, zero, k, x, la, lb, ids, None, None)
    assert bool(ref.isfinite().all())
    for f in calls:
        assert R.worst(f(), ref, bound) <= 1.0
    la[0, 2, 0] = 4.0   # the sum is past fp32's largest
    lb[0, :, 5] = 0.0
    sign = torch.where(x[:, :1] > 0, 1.0, -1.0).double()
    for f in calls:
        assert torch.equal(f().double(), (sign * float("inf")).expand(m, n))


def near_pairs(g, m, n, k, r, L):
    """Rows and adapters whose projections are integers of 24 bits (times a power of
    two of the row), two and two a small step apart; column c of the output is the
    step of pair c % (r / 2), exact in every order of the sums.  Returns x, lora_a,
    lora_b, adapter and the output, with a shared product of 0."""
    x = torch.zeros(m, k, device="cuda")
    s = 2.0 ** (torch.arange(m, device="cuda") % 5 - 2)
    cols = [0, k // 2, k - 1]
    for c, v in zip(cols, (65536.0, 256.0, 1.0)):
        x[:, c] = s * v
    step = torch.randint(1, 256, (L, r // 2), device="cuda", generator=g)
    low = torch.randint(2 ** 23, 2 ** 24 - 256, (L, r // 2), device="cuda", generator=g)
    d = torch.stack([low, low + step], -1).view(L, r)
    la = torch.zeros(L, r, k, device="cuda")
    for c, shift in zip(cols, (16, 8, 0)):
        la[:, :, c] = (d >> shift & 255).float()
    pair = torch.arange(n, device="cuda") % (r // 2)
    lb = torch.zeros(L, n, r, device="cuda")
    at = torch.arange(n, device="cuda")
    lb[:, at, 2 * pair], lb[:, at, 2 * pair + 1] = -1.0, 1.0
    ids = torch.randint(-1, L, (m,), device="cuda", generator=g, dtype=torch.int32)
    out = torch.where(ids[:, None] >= 0, s[:, None] * step[ids.clamp(min=0).long()][:, pair], torch.zeros(m, n, device="cuda"))
    return x.bfloat16(), la.bfloat16(), lb.bfloat16(), ids, out.bfloat16()


@pytest.mark.parametrize("m,n,k,r", [(1, 32, 64, 8), (17, 100, 272, 16), (50, 48, 640, 40), (16, 8210, 400, 8), (24, 4100, 256, 72),
                                     (40, 260, 4240, 24), (100, 48, 64, 256)])
def test_projection_keeps_its_fp32_bits_decode(mods, m, n, k, r):
    """The projection onto the ranks is a sum, held in fp32."""
    serving, _ = mods
    say("adapters: fp32 projection, decode", m, n, k, r)
    g = gen(m + n)
    x, la, lb, ids, want = near_pairs(g, m, n, k, r, 5)
    b, sf = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda"), R.rand_sf(g, n, k)
    for split in (False, True):
        out = serving.nvfp4_linear_adapters(x, b, sf, torch.ones(1, device="cuda"), la, lb, ids, out=fresh(m, n),
                                            workspace=workspace(serving.adapters_ws_bytes(m, r, split)))
        assert torch.equal(out, want)


@pytest.mark.parametrize("m,n,k,r,split", [(20, 64, 272, 40, False), (300, 520, 128, 24, False), (2000, 1928, 256, 16, False),
                                           (2048, 4104, 896, 40, False), (4000, 3480, 272, 32, False),
                                           (4096, 8200, 144, 40, False), (3968, 2560, 1008, 72, True)])
def test_projection_keeps_its_fp32_bits_prefill(mods, m, n, k, r, split):
    serving, _ = mods
    say("adapters: fp32 projection, prefill", m, n, k, r)
    g = gen(m + n)
    x, la, lb, ids, want = near_pairs(g, m, n, k, r, 3)
    ids[: m // 2] = ids[0]   # fragments that share an adapter, and mixed ones
    want[: m // 2] = want[0] * (2.0 ** (torch.arange(m // 2, device="cuda") % 5))[:, None].bfloat16()
    a, b = (torch.zeros(v, k // 2, dtype=torch.uint8, device="cuda") for v in (m, n))
    out = serving.nvfp4_gemm_adapters(a, b, R.rand_sf(g, m, k), R.rand_sf(g, n, k), torch.ones(1, device="cuda"), x, la, lb, ids,
                                      out=fresh(m, n), workspace=workspace(serving.adapters_ws_bytes(m, r, split)))
    assert torch.equal(out, want)


@pytest.mark.parametrize("m,n,k,r", [(40, 1040, 272, 24), (300, 1040, 272, 24), (2000, 1928, 256, 16), (4000, 3480, 272, 40),
                                     (4096, 8200, 144, 32)])
def test_prefill_row_does_not_depend_on_its_neighbours(mods, m, n, k, r):
    """A row comes out the same bit for bit whichever adapters the rows beside it use."""
    serving, _ = mods
    say("gemm_adapters: neighbours", m, n, k, r)
    g = gen(m + r)
    p = pool(g, m, n, k, r, 5, "one")
    a, a_sf, b, b_sf = R.rand_fp4(g, m, k=k), R.rand_sf(g, m, k), R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    alpha = torch.full((1,), 3e-4, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    go = lambda ids: serving.nvfp4_gemm_adapters(a, b, a_sf, b_sf, alpha, x, p["lora_a"], p["lora_b"], ids, scaling=p["scaling"])
    one = p["adapter"]
    mixed = torch.where(torch.rand(m, device="cuda", generator=g) < 0.5, one, torch.randint_like(one, -1, 4))
    rows = mixed == one
    assert torch.equal(go(one)[rows], go(mixed)[rows])


def test_most_rows(mods):
    """2^20 rows, the most that are taken."""
    serving, _ = mods
    say("adapters: 2^20 rows")
    g = gen(20)
    m, n, k, r, L = 1 << 20, 24, 16, 24, 6
    p = pool(g, m, n, k, r, L, "runs")
    a, a_sf, b, b_sf = R.rand_fp4(g, m, k=k), R.rand_sf(g, m, k), R.rand_fp4(g, n, k=k), R.rand_sf(g, n, k)
    alpha = torch.full((1,), 0.02, device="cuda")
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    lora = (p["lora_a"], p["lora_b"], p["adapter"])
    w = R.dequant(b, b_sf)
    for left, f in ((x.double(), lambda out: serving.nvfp4_linear_adapters(x, b, b_sf, alpha, *lora, out=out)),
                    (R.dequant(a, a_sf), lambda out: serving.nvfp4_gemm_adapters(a, b, a_sf, b_sf, alpha, x, *lora, out=out))):
        ref, bound = R.adapters(left @ w.t() * alpha.double(), left.abs() @ w.abs().t() * alpha.double(), k, x, *lora, None, None)
        assert R.worst(f(fresh(m, n)), ref, bound) <= 1.0
